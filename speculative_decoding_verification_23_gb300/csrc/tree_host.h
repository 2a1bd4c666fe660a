// Host side of the attention operators, shared by their entry points: checks of
// arguments, the choice of kernel, the kernels' parameters.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "spec_tree.h"
#include "spec_internal.h"
#include "tree_internal.h"

namespace sv {
TreePlan plan_tree_warp(int dim, int num_sms);
bool tree_tc_fits(int dim, int page_size);
TreePlan plan_tree_tc(int rows, int num_sms);
}  // namespace sv

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool mult8(int64_t x) { return x >= 0 && x % 8 == 0; }
bool sixteen(int dtype) { return dtype == SPEC_BF16 || dtype == SPEC_F16; }

// SMs that sizes are planned for where there is no device to ask.
constexpr int kPlanSms = 152;

int sm_count(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_DEVICE;
  }
  return SPEC_OK;
}

int check_cache(const spec_cache& c, bool need_v) {
  if (!c.k || (need_v && !c.v)) return SPEC_ERR_NULL;
  if (!sixteen(c.dtype)) return SPEC_ERR_DTYPE;
  if (c.layers < 1 || c.num_pages < 1 || c.page_size < 1 || c.heads < 1) return SPEC_ERR_SHAPE;
  if (c.dim != 64 && c.dim != 96 && c.dim != 128 && c.dim != 192 && c.dim != 256) return SPEC_ERR_SHAPE;
  if ((long long)c.num_pages * c.page_size > INT32_MAX) return SPEC_ERR_SHAPE;
  if (!aligned16(c.k) || (need_v && !aligned16(c.v))) return SPEC_ERR_ALIGN;
  if (!mult8(c.s_layer) || !mult8(c.s_page) || !mult8(c.s_slot) || !mult8(c.s_head)) return SPEC_ERR_ALIGN;
  return SPEC_OK;
}

// Positions of tokens, and the step past the last of them that a loop takes,
// fit 32 bits.
constexpr int kMaxTokens = INT32_MAX - 65535;
bool table_ok(int ld, int page_size) { return ld >= 1 && (long long)ld * page_size <= kMaxTokens; }
bool row_ok(int ld) { return ld >= 1 && ld <= kMaxTokens; }

// a b c <= most, of positive factors whose product may pass 64 bits.
bool fits32(long long a, long long b, long long c, long long most = INT32_MAX) { return a <= most / b && a * b <= most / c; }

int check_tree(const spec_tree_args* a) {
  if (!a) return SPEC_ERR_NULL;
  int rc = check_cache(a->cache, true);
  if (rc) return rc;
  if (a->B < 1 || a->B > 65535 * 16 || a->total_nodes < 0 || a->max_nodes < 0 || a->max_nodes > SPEC_MAX_TREE)
    return SPEC_ERR_SHAPE;
  if ((long long)a->total_nodes > (long long)a->B * a->max_nodes) return SPEC_ERR_SHAPE;
  if (a->heads_q < 1 || a->heads_q % a->cache.heads != 0) return SPEC_ERR_SHAPE;
  if ((long long)SPEC_MAX_TREE * a->heads_q > INT32_MAX) return SPEC_ERR_SHAPE;
  if (a->layer < 0 || a->layer >= a->cache.layers || !std::isfinite(a->scale)) return SPEC_ERR_SHAPE;
  if (!table_ok(a->ld_table, a->cache.page_size)) return SPEC_ERR_SHAPE;
  if (!a->cu_nodes || !a->block_table || !a->ctx_len) return SPEC_ERR_NULL;
  if (a->tree_mask && (long long)a->mask_words * 32 < a->max_nodes) return SPEC_ERR_SHAPE;
  if (a->total_nodes > 0) {
    if (!a->q || !a->k_new || !a->v_new) return SPEC_ERR_NULL;
    if (!aligned16(a->q) || !aligned16(a->k_new) || !aligned16(a->v_new) || !mult8(a->sq_node) || !mult8(a->sq_head) ||
        !mult8(a->sn_node) || !mult8(a->sn_head))
      return SPEC_ERR_ALIGN;
  }
  return SPEC_OK;
}

// A stride that a TMA copy takes along an axis of n elements.
bool tma_stride(int64_t s, int64_t n) { return n == 1 || (s > 0 && s < (1ll << 38)); }

// The tensor-memory kernel takes the calls whose tiles TMA can copy, with a
// positive scale, and more query rows per key head than one warp tile holds.
// Both kernels measured (us, warp tiles against tensor memory; 28 query and 4
// key heads of 128 channels):
//   8 requests of 4000 tokens: 7 rows 25.6 / 31.1, 14 rows 27.3 / 31.5,
//     21 rows 39.3 / 32.0, 35 rows 44.2 / 31.6, 63 rows 52.0 / 32.4;
//   64 requests of 2000 tokens, 7 rows: 58.6 / 63.2;
//   one of 700 tokens, 64 channels: 7 rows 10.3 / 11.5, 21 rows 9.6 / 10.9.
constexpr int kWarpRows = 16;
// Up to here the kernel finds a row's node in fp32.
constexpr int kMaxTcRows = 1 << 20;

sv::TreePlan plan_tree(const spec_tree_args* a, int num_sms) {
  const spec_cache& c = a->cache;
  const int rows = a->max_nodes * (a->heads_q / c.heads);
  const bool fits = rows <= kMaxTcRows && sv::tree_tc_fits(c.dim, c.page_size) && a->scale > 0.f && a->total_nodes > 0 &&
                    tma_stride(c.s_slot, c.page_size) && tma_stride(c.s_head, c.heads) &&
                    tma_stride(c.s_page, c.num_pages) && tma_stride(a->sn_node, a->total_nodes) &&
                    tma_stride(a->sn_head, c.heads);
  return fits && rows > kWarpRows ? sv::plan_tree_tc(rows, num_sms) : sv::plan_tree_warp(c.dim, num_sms);
}

// Memory that a call reads or writes: n elements of 4 bytes, or of `size`.
struct Span {
  uintptr_t at;
  unsigned long long bytes;
  Span(const void* p, long long n, int size = 4)
      : at(reinterpret_cast<uintptr_t>(p)), bytes(p ? (unsigned long long)n * size : 0ull) {}
};

// Whether results overlap anything that a kernel reads: CTAs do not begin
// together, so one could find results of another for arguments.
bool overlap(std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span& o : out)
    for (const Span& i : in)
      if (o.bytes > 0 && i.bytes > 0 && o.at < i.at + i.bytes && i.at < o.at + o.bytes) return true;
  return false;
}

uint16_t* layer_of(void* p, const spec_cache& c, int layer) {
  return static_cast<uint16_t*>(p) + (long long)layer * c.s_layer;
}

// Whether a call's results overlap what its kernels read.
bool tree_overlap(const spec_tree_args* a, const float* out_lse, const int32_t* out_status) {
  return overlap({{out_lse, (long long)a->total_nodes * a->heads_q}, {out_status, a->B}},
                 {{a->cu_nodes, a->B + 1ll}, {a->ctx_len, a->B}, {a->block_table, (long long)a->B * a->ld_table},
                  {a->tree_mask, (long long)a->total_nodes * a->mask_words}});
}

// The kernels' parameters of a checked call.
void fill_tree(sv::TreeParams& P, const spec_tree_args* a, const sv::TreePlan& plan, const sv::TreeWorkspace& W, void* out,
               int64_t so_node, int64_t so_head, float* out_lse, int32_t* out_status, void* workspace) {
  unsigned char* w = static_cast<unsigned char*>(workspace);
  std::memset(&P, 0, sizeof(P));
  P.cu = a->cu_nodes;
  P.ctx = a->ctx_len;
  P.table = a->block_table;
  P.mask = a->tree_mask;
  P.q = a->q;
  P.k_new = a->k_new;
  P.v_new = a->v_new;
  P.k = layer_of(a->cache.k, a->cache, a->layer);
  P.v = layer_of(a->cache.v, a->cache, a->layer);
  P.sq_node = a->sq_node;
  P.sq_head = a->sq_head;
  P.sn_node = a->sn_node;
  P.sn_head = a->sn_head;
  P.so_node = so_node;
  P.so_head = so_head;
  P.s_page = a->cache.s_page;
  P.s_slot = a->cache.s_slot;
  P.s_head = a->cache.s_head;
  P.out = out;
  P.lse = out_lse;
  P.status = out_status;
  P.start = reinterpret_cast<long long*>(w + W.off_start);
  P.failed = plan.kernel == 1 ? reinterpret_cast<int32_t*>(w + W.off_failed) : nullptr;
  P.part_ml = reinterpret_cast<float4*>(w + W.off_ml);
  P.part_o = reinterpret_cast<float*>(w + W.off_o);
  P.scale_log2 = a->scale * 1.4426950408889634f;
  P.B = a->B;
  P.total = a->total_nodes;
  P.max_nodes = a->max_nodes;
  P.mask_words = a->mask_words;
  P.ld_table = a->ld_table;
  P.num_pages = a->cache.num_pages;
  P.page_size = a->cache.page_size;
  P.heads = a->cache.heads;
  P.group = a->heads_q / a->cache.heads;
  P.dim = a->cache.dim;
  P.grid = plan.grid;
  P.rows = plan.rows;
  P.kt = plan.kt;
}

}  // namespace
