// C ABI of the drafted-tree operators: host-side checks, the choice of
// kernel, launches.
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
int launch_tree_warp(const TreeParams& P, bool bf16, cudaStream_t s);
bool tree_tc_fits(int dim, int page_size);
TreePlan plan_tree_tc(int rows, int num_sms);
int launch_tree_tc(const TreeParams& P, bool bf16, cudaStream_t s);
int launch_tree_join(const TreeParams& P, bool bf16, int num_sms, cudaStream_t s);
int weigh_tc_rows();
int launch_weigh_tc(const TreeParams& P, const float* before, const float* lse, float* out, bool bf16, cudaStream_t s);
int launch_weigh(const WeighParams& P, bool bf16, cudaStream_t s);
int launch_evict(const EvictParams& P, cudaStream_t s);
int launch_commit(const CommitParams& P, cudaStream_t s);
void plan_beams(BeamParams& P, bool bf16, int num_sms);
int launch_beam_select(const BeamParams& P, bool bf16, cudaStream_t s);
long long plan_reorder(ReorderParams& P);
int launch_beam_reorder(const ReorderParams& P, long long blocks, cudaStream_t s);
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

}  // namespace

extern "C" {

size_t spec_tree_workspace_bytes(const spec_tree_args* a) {
  if (check_tree(a)) return 0;
  int sms = kPlanSms;
  if (sm_count(&sms)) sms = kPlanSms;
  const sv::TreePlan p = plan_tree(a, sms);
  return sv::make_tree_workspace(a->B, p.grid, p.rows, a->cache.dim).total;
}

int spec_tree_attention(const spec_tree_args* a, void* out, int64_t so_node, int64_t so_head, float* out_lse,
                        int32_t* out_status, void* workspace, size_t ws_bytes, spec_stream_t stream) {
  NvtxRange nvtx("spec_tree_attention");
  int rc = check_tree(a);
  if (rc) return rc;
  if (a->total_nodes > 0) {
    if (!out) return SPEC_ERR_NULL;
    if (!aligned16(out) || !mult8(so_node) || !mult8(so_head)) return SPEC_ERR_ALIGN;
  }
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  rc = sm_count(&sms);
  const sv::TreePlan plan = plan_tree(a, rc ? kPlanSms : sms);
  const sv::TreeWorkspace W = sv::make_tree_workspace(a->B, plan.grid, plan.rows, a->cache.dim);
  if (ws_bytes < W.total) return SPEC_ERR_WORKSPACE;
  if (rc) return rc;
  if (overlap({{out_lse, (long long)a->total_nodes * a->heads_q}, {out_status, a->B}},
              {{a->cu_nodes, a->B + 1ll}, {a->ctx_len, a->B}, {a->block_table, (long long)a->B * a->ld_table},
               {a->tree_mask, (long long)a->total_nodes * a->mask_words}}))
    return SPEC_ERR_SHAPE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  sv::TreeParams P;
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
  const bool bf16 = a->cache.dtype == SPEC_BF16;
  if (plan.kernel == 1 ? sv::launch_tree_tc(P, bf16, s) : sv::launch_tree_warp(P, bf16, s)) return SPEC_ERR_LAUNCH;
  return sv::launch_tree_join(P, bf16, sms, s) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int spec_attention_weights(const spec_weigh_args* a, const float* before, float* out, int32_t* out_status,
                           spec_stream_t stream) {
  NvtxRange nvtx("spec_attention_weights");
  if (!a) return SPEC_ERR_NULL;
  int rc = check_cache(a->cache, false);
  if (rc) return rc;
  if (a->B < 1 || a->total_rows < 0 || a->max_rows < 0 || !row_ok(a->ld)) return SPEC_ERR_SHAPE;
  if ((long long)a->total_rows > (long long)a->B * a->max_rows) return SPEC_ERR_SHAPE;
  if (a->heads_q < 1 || a->heads_q % a->cache.heads != 0) return SPEC_ERR_SHAPE;
  if ((long long)a->max_rows * a->heads_q > INT32_MAX || (long long)a->B * a->cache.heads > INT32_MAX)
    return SPEC_ERR_SHAPE;
  if ((long long)((a->ld + 63) / 64) * a->B * a->cache.heads > INT32_MAX) return SPEC_ERR_SHAPE;
  if (a->layer < 0 || a->layer >= a->cache.layers || !std::isfinite(a->scale)) return SPEC_ERR_SHAPE;
  if (!table_ok(a->ld_table, a->cache.page_size)) return SPEC_ERR_SHAPE;
  if (!a->cu_rows || !a->block_table || !a->kv_len || !out) return SPEC_ERR_NULL;
  if (a->total_rows > 0) {
    if (!a->q || !a->lse) return SPEC_ERR_NULL;
    if (!aligned16(a->q) || !mult8(a->sq_row) || !mult8(a->sq_head)) return SPEC_ERR_ALIGN;
  }
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  const spec_cache& c = a->cache;
  const long long keys = (long long)a->B * c.heads * a->ld, lens = a->B;
  const Span before_at(before == out ? nullptr : before, keys), lse_at(a->lse, (long long)a->total_rows * a->heads_q),
      cu_at(a->cu_rows, lens + 1), len_at(a->kv_len, lens), table_at(a->block_table, lens * a->ld_table);
  if (overlap({{out, keys}, {out_status, lens}}, {before_at, lse_at, cu_at, len_at, table_at})) return SPEC_ERR_SHAPE;
  const bool bf16 = a->cache.dtype == SPEC_BF16;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long rows = (long long)a->max_rows * (a->heads_q / c.heads);
  // Tensor memory where its rows and tiles fit: on 16 requests of up to 16384
  // tokens, 8 key heads of 128 channels, 4 / 36 / 128 rows per key head, 60.8 /
  // 62.1 / 87.4 us against 149 / 186 / 387 on warp tiles; one request of 36
  // rows 6.4 against 10.1.
  if (sv::tree_tc_fits(c.dim, c.page_size) && rows <= sv::weigh_tc_rows() && tma_stride(c.s_slot, c.page_size) &&
      tma_stride(c.s_head, c.heads) && tma_stride(c.s_page, c.num_pages)) {
    sv::TreeParams P;
    std::memset(&P, 0, sizeof(P));
    P.cu = a->cu_rows;
    P.ctx = a->kv_len;
    P.table = a->block_table;
    P.q = a->q;
    P.k = layer_of(c.k, c, a->layer);
    P.sq_node = a->sq_row;
    P.sq_head = a->sq_head;
    P.s_page = c.s_page;
    P.s_slot = c.s_slot;
    P.s_head = c.s_head;
    P.status = out_status;
    P.scale_log2 = a->scale * 1.4426950408889634f;
    P.B = a->B;
    P.total = a->total_rows;
    P.max_nodes = a->max_rows;
    P.ld_table = a->ld_table;
    P.num_pages = c.num_pages;
    P.page_size = c.page_size;
    P.heads = c.heads;
    P.group = a->heads_q / c.heads;
    P.dim = c.dim;
    P.grid = sms;
    P.rows = 1;
    P.kt = 128;
    P.weigh = 1;
    P.ld = a->ld;
    return sv::launch_weigh_tc(P, before, a->lse, out, bf16, s) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
  }
  sv::WeighParams P;
  std::memset(&P, 0, sizeof(P));
  P.cu = a->cu_rows;
  P.len = a->kv_len;
  P.table = a->block_table;
  P.q = a->q;
  P.k = layer_of(a->cache.k, a->cache, a->layer);
  P.lse = a->lse;
  P.before = before;
  P.out = out;
  P.status = out_status;
  P.sq_row = a->sq_row;
  P.sq_head = a->sq_head;
  P.s_page = a->cache.s_page;
  P.s_slot = a->cache.s_slot;
  P.s_head = a->cache.s_head;
  P.scale_log2 = a->scale * 1.4426950408889634f;
  P.B = a->B;
  P.total = a->total_rows;
  P.max_rows = a->max_rows;
  P.ld_table = a->ld_table;
  P.ld = a->ld;
  P.num_pages = a->cache.num_pages;
  P.page_size = a->cache.page_size;
  P.heads = a->cache.heads;
  P.group = a->heads_q / a->cache.heads;
  P.dim = a->cache.dim;
  return sv::launch_weigh(P, bf16, s) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int spec_cache_evict(const spec_evict_args* a, int32_t* out_index, float* out_kept, int32_t* out_len,
                     int32_t* out_status, spec_stream_t stream) {
  NvtxRange nvtx("spec_cache_evict");
  if (!a) return SPEC_ERR_NULL;
  int rc = check_cache(a->cache, true);
  if (rc) return rc;
  if (a->B < 1 || a->keep < 1 || a->sink < 0 || a->recent < 0 || !row_ok(a->ld)) return SPEC_ERR_SHAPE;
  if ((long long)a->sink + a->recent > a->keep) return SPEC_ERR_SHAPE;
  if (a->layer < 0 || a->layer >= a->cache.layers) return SPEC_ERR_SHAPE;
  if (!table_ok(a->ld_table, a->cache.page_size) || !table_ok(a->ld_to, a->cache.page_size)) return SPEC_ERR_SHAPE;
  if ((long long)a->ld_to * a->cache.page_size < a->keep) return SPEC_ERR_SHAPE;
  // CTAs of the move: at least 8 kept tokens each
  if (!fits32(a->B, a->cache.heads, (a->keep + 7) / 8)) return SPEC_ERR_SHAPE;
  if (!a->weights || !a->kv_len || !a->block_table || !a->to_table || !out_index || !out_len) return SPEC_ERR_NULL;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  const long long rows = (long long)a->B * a->cache.heads, kept = rows * a->keep;
  if (overlap({{out_index, kept}, {out_kept, kept}, {out_len, a->B}, {out_status, a->B}},
              {{a->weights, rows * a->ld}, {out_len == a->kv_len ? nullptr : a->kv_len, a->B},
               {a->block_table, (long long)a->B * a->ld_table}, {a->to_table, (long long)a->B * a->ld_to}}) ||
      overlap({{out_index, kept}, {out_kept, kept}, {out_status, a->B}}, {{a->kv_len, a->B}}))
    return SPEC_ERR_SHAPE;
  sv::EvictParams P;
  std::memset(&P, 0, sizeof(P));
  P.weights = a->weights;
  P.len = a->kv_len;
  P.table = a->block_table;
  P.to = a->to_table;
  P.k = layer_of(a->cache.k, a->cache, a->layer);
  P.v = layer_of(a->cache.v, a->cache, a->layer);
  P.s_page = a->cache.s_page;
  P.s_slot = a->cache.s_slot;
  P.s_head = a->cache.s_head;
  P.index = out_index;
  P.kept = out_kept;
  P.new_len = out_len;
  P.status = out_status;
  P.B = a->B;
  P.keep = a->keep;
  P.sink = a->sink;
  P.recent = a->recent;
  P.ld = a->ld;
  P.ld_table = a->ld_table;
  P.ld_to = a->ld_to;
  P.num_pages = a->cache.num_pages;
  P.page_size = a->cache.page_size;
  P.heads = a->cache.heads;
  P.dim = a->cache.dim;
  return sv::launch_evict(P, reinterpret_cast<cudaStream_t>(stream)) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int spec_cache_commit(const spec_commit_args* a, int32_t* out_len, int32_t* out_status, spec_stream_t stream) {
  NvtxRange nvtx("spec_cache_commit");
  if (!a) return SPEC_ERR_NULL;
  int rc = check_cache(a->cache, true);
  if (rc) return rc;
  if (a->B < 1 || a->total_nodes < 0 || a->ld_path < 1 || a->cache.layers > 65535) return SPEC_ERR_SHAPE;
  if (!fits32(a->ld_path, a->cache.heads, a->cache.dim / 8, kMaxTokens)) return SPEC_ERR_SHAPE;
  if (!table_ok(a->ld_table, a->cache.page_size)) return SPEC_ERR_SHAPE;
  if (!a->cu_nodes || !a->path || !a->path_len || !a->block_table || !a->ctx_len || !out_len) return SPEC_ERR_NULL;
  if (a->total_nodes > 0) {
    if (!a->k_new || !a->v_new) return SPEC_ERR_NULL;
    if (!aligned16(a->k_new) || !aligned16(a->v_new) || !mult8(a->sn_layer) || !mult8(a->sn_node) ||
        !mult8(a->sn_head))
      return SPEC_ERR_ALIGN;
  }
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  const long long lens = a->B;
  if (overlap({{out_len, lens}, {out_status, lens}},
              {{a->cu_nodes, lens + 1}, {a->path, lens * a->ld_path}, {a->path_len, lens},
               {a->block_table, lens * a->ld_table}, {out_len == a->ctx_len ? nullptr : a->ctx_len, lens}}) ||
      overlap({{out_status, lens}}, {{a->ctx_len, lens}}))
    return SPEC_ERR_SHAPE;
  sv::CommitParams P;
  std::memset(&P, 0, sizeof(P));
  P.cu = a->cu_nodes;
  P.path = a->path;
  P.path_len = a->path_len;
  P.table = a->block_table;
  P.ctx = a->ctx_len;
  P.k_new = a->k_new;
  P.v_new = a->v_new;
  P.k = a->cache.k;
  P.v = a->cache.v;
  P.sn_layer = a->sn_layer;
  P.sn_node = a->sn_node;
  P.sn_head = a->sn_head;
  P.s_layer = a->cache.s_layer;
  P.s_page = a->cache.s_page;
  P.s_slot = a->cache.s_slot;
  P.s_head = a->cache.s_head;
  P.new_len = out_len;
  P.status = out_status;
  P.B = a->B;
  P.total = a->total_nodes;
  P.layers = a->cache.layers;
  P.ld_path = a->ld_path;
  P.ld_table = a->ld_table;
  P.num_pages = a->cache.num_pages;
  P.page_size = a->cache.page_size;
  P.heads = a->cache.heads;
  P.dim = a->cache.dim;
  return sv::launch_commit(P, reinterpret_cast<cudaStream_t>(stream)) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // extern "C"

namespace {

int check_beams(const spec_beam_args* a) {
  if (!a) return SPEC_ERR_NULL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (a->B < 1 || a->V < 1 || a->W < 1 || a->W > SPEC_MAX_BEAMS || a->keep < 1 || a->keep > SPEC_MAX_BEAMS)
    return SPEC_ERR_SHAPE;
  // places in the split of the logits and of a request's candidates are 32-bit
  if ((long long)a->W * a->V > INT32_MAX / 2 || (long long)a->B * a->W > INT32_MAX / 4096 ||
      (long long)a->B * a->W * ((a->V + 4095ll) / 4096) > INT32_MAX)
    return SPEC_ERR_SHAPE;
  if (!a->logits || !a->scores) return SPEC_ERR_NULL;
  if (a->ld < a->V) return SPEC_ERR_SHAPE;
  if (a->finished && (a->end_token < 0 || a->end_token >= a->V)) return SPEC_ERR_SHAPE;
  if (!aligned16(a->logits) || (a->ld * (a->dtype == SPEC_BF16 ? 2 : 4)) % 16 != 0) return SPEC_ERR_ALIGN;
  return SPEC_OK;
}

void beam_params(sv::BeamParams& P, const spec_beam_args* a, int num_sms) {
  std::memset(&P, 0, sizeof(P));
  P.B = a->B;
  P.W = a->W;
  P.keep = a->keep;
  P.V = a->V;
  P.end_token = a->end_token;
  sv::plan_beams(P, a->dtype == SPEC_BF16, num_sms);
}

}  // namespace

extern "C" {

size_t spec_beam_workspace_bytes(const spec_beam_args* a) {
  if (check_beams(a)) return 0;
  int sms = kPlanSms;
  if (sm_count(&sms)) sms = kPlanSms;
  sv::BeamParams P;
  beam_params(P, a, sms);
  return sv::make_beam_workspace(a->B, a->W, P.grid, P.spans, P.chunks).total;
}

int spec_beam_select(const spec_beam_args* a, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                     int32_t* out_status, void* workspace, size_t ws_bytes, spec_stream_t stream) {
  NvtxRange nvtx("spec_beam_select");
  int rc = check_beams(a);
  if (rc) return rc;
  if (!out_scores || !out_parents || !out_tokens) return SPEC_ERR_NULL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  rc = sm_count(&sms);
  sv::BeamParams P;
  beam_params(P, a, rc ? kPlanSms : sms);
  const sv::BeamWorkspace W = sv::make_beam_workspace(a->B, a->W, P.grid, P.spans, P.chunks);
  if (ws_bytes < W.total) return SPEC_ERR_WORKSPACE;
  if (rc) return rc;
  const long long rows = (long long)a->B * a->W, kept = (long long)a->B * a->keep;
  if (overlap({{out_scores, kept}, {out_parents, kept}, {out_tokens, kept}, {out_status, a->B}},
              {{a->scores, rows}, {a->finished, rows},
               {a->logits, (rows - 1) * a->ld + a->V, a->dtype == SPEC_BF16 ? 2 : 4}}))
    return SPEC_ERR_SHAPE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  P.logits = a->logits;
  P.ld = a->ld;
  P.scores = a->scores;
  P.finished = a->finished;
  P.out_scores = out_scores;
  P.out_parents = out_parents;
  P.out_tokens = out_tokens;
  P.status = out_status;
  P.counters = reinterpret_cast<unsigned long long*>(w + W.off_counters);
  P.stat = reinterpret_cast<float4*>(w + W.off_stat);
  P.maxima = reinterpret_cast<float*>(w + W.off_maxima);
  rc = sv::call_tag(P.counters, a->B, s, &P.tag);
  if (rc) return rc;
  return sv::launch_beam_select(P, a->dtype == SPEC_BF16, s) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int spec_beam_reorder(int32_t B, int32_t W, int32_t keep, const int32_t* parents, const spec_beam_state* states,
                      int32_t num_states, spec_stream_t stream) {
  NvtxRange nvtx("spec_beam_reorder");
  if (!parents || !states) return SPEC_ERR_NULL;
  if (B < 1 || W < 1 || keep < 1 || num_states < 1 || num_states > SPEC_MAX_STATES) return SPEC_ERR_SHAPE;
  sv::ReorderParams P;
  std::memset(&P, 0, sizeof(P));
  P.parents = parents;
  P.B = B;
  P.W = W;
  P.keep = keep;
  P.num = num_states;
  for (int i = 0; i < num_states; ++i) {
    const spec_beam_state& a = states[i];
    if (a.row_bytes < 0 || a.outer < 0 || a.row_bytes > (1ll << 40)) return SPEC_ERR_SHAPE;
    if (a.row_bytes > 0 && a.outer > 0 && (!a.src || !a.dst)) return SPEC_ERR_NULL;
    // a block at least for every row
    if (a.row_bytes > 0 && a.outer > 0 && !fits32(B, keep, a.outer)) return SPEC_ERR_SHAPE;
    sv::BeamState& s = P.s[i];
    s.src = static_cast<const unsigned char*>(a.src);
    s.dst = static_cast<unsigned char*>(a.dst);
    s.row_bytes = a.row_bytes;
    s.src_outer = a.src_outer;
    s.src_batch = a.src_batch;
    s.src_beam = a.src_beam;
    s.dst_outer = a.dst_outer;
    s.dst_batch = a.dst_batch;
    s.dst_beam = a.dst_beam;
    s.outer = a.outer;
    // the widest access that every row's start and size allow
    const unsigned long long all =
        reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) | (unsigned long long)a.row_bytes |
        (unsigned long long)a.src_batch | (unsigned long long)a.src_beam | (unsigned long long)a.dst_batch |
        (unsigned long long)a.dst_beam | (a.outer > 1 ? (unsigned long long)a.src_outer | (unsigned long long)a.dst_outer : 0ull);
    s.unit = 16;
    while (all & (unsigned long long)(s.unit - 1)) s.unit >>= 1;
  }
  const long long blocks = sv::plan_reorder(P);
  if (blocks > INT32_MAX) return SPEC_ERR_SHAPE;
  int sms = 0;
  const int rc = sm_count(&sms);
  if (rc) return rc;
  if (blocks == 0) return SPEC_OK;
  return sv::launch_beam_reorder(P, blocks, reinterpret_cast<cudaStream_t>(stream)) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // extern "C"
