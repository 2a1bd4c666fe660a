// C ABI of the operators beside the drafted tree: host-side checks, the choice
// of kernel, launches.
#include "spec_serve.h"
#include "serve_internal.h"
#include "tree_host.h"

namespace sv {
int launch_norm_rotate(RotateParams& P, bool bf16, int num_sms, cudaStream_t s);
int launch_window_warp(const TreeParams& P, bool bf16, cudaStream_t s);
int launch_window_tc(const TreeParams& P, bool bf16, cudaStream_t s);
int launch_window_join(const TreeParams& P, bool bf16, int num_sms, cudaStream_t s);
TreePlan plan_cache8_warp(int dim, int num_sms);
int launch_cache8_warp(const Cache8Params& C, bool bf16, cudaStream_t s);
bool cache8_tc_fits(int dim, int page_size, int block);
TreePlan plan_cache8_tc(int rows, int num_sms);
int launch_cache8_tc(const Cache8Params& C, bool bf16, cudaStream_t s);
int launch_commit8(Commit8Params& P, bool bf16, int num_sms, cudaStream_t s);
}  // namespace sv

namespace {

bool mult16(int64_t x) { return x >= 0 && x % 16 == 0; }

// ---------------------------------------------------- norms and positions

// Rows of a strided side: n elements a row from its first to its last.
struct Rows {
  uintptr_t at;
  unsigned long long row, bytes, all;  // between rows, of a row, of all rows
  Rows(const void* p, int rows, int heads, int dim, int64_t s_row, int64_t s_head)
      : at(reinterpret_cast<uintptr_t>(p)),
        row(2ull * s_row),
        bytes(rows > 0 && heads > 0 ? 2ull * ((unsigned long long)(heads - 1) * s_head + dim) : 0ull),
        all(bytes ? row * (unsigned long long)(rows - 1) + bytes : 0ull) {}
};

// Whether two sides share memory.  Rows that lie between one another's, as the
// parts of one projection do, are told apart where their strides are the same.
bool rows_overlap(const Rows& a, const Rows& b) {
  if (!a.bytes || !b.bytes || a.at >= b.at + b.all || b.at >= a.at + a.all) return false;
  if (a.row != b.row || a.bytes > a.row || b.bytes > b.row) return true;
  const unsigned long long d = a.at <= b.at ? (b.at - a.at) % a.row : a.row - 1 - (a.at - b.at - 1) % a.row;
  return d < a.bytes || d + b.bytes > a.row;
}

// Whether rows or heads of a result share memory: the one of smaller stride lies
// within the other's.
bool overlaps_itself(int rows, int heads, int dim, int64_t s_row, int64_t s_head) {
  if (heads < 1 || (rows < 2 && heads < 2)) return false;
  if (rows < 2) return s_head < dim;
  if (heads < 2) return s_row < dim;
  const bool heads_inside = s_head <= s_row;
  const unsigned long long inner = heads_inside ? s_head : s_row, outer = heads_inside ? s_row : s_head;
  return inner < (unsigned)dim || outer < inner * ((heads_inside ? heads : rows) - 1ull) + dim;
}

int check_side(const void* p, int heads, int64_t s_row, int64_t s_head) {
  if (heads == 0) return SPEC_OK;
  if (!p) return SPEC_ERR_NULL;
  return aligned16(p) && mult8(s_row) && mult8(s_head) ? SPEC_OK : SPEC_ERR_ALIGN;
}

// -------------------------------------------------------------- 8-bit cache

int check_cache8(const spec_cache8& c) {
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return SPEC_ERR_NULL;
  if (c.layers < 1 || c.num_pages < 1 || c.page_size < 1 || c.heads < 1 || c.block < 1 || c.page_size % c.block != 0)
    return SPEC_ERR_SHAPE;
  if (c.dim != 64 && c.dim != 96 && c.dim != 128 && c.dim != 192 && c.dim != 256) return SPEC_ERR_SHAPE;
  if ((long long)c.num_pages * c.page_size > INT32_MAX) return SPEC_ERR_SHAPE;
  if (c.c_layer < 0 || c.c_page < 0 || c.c_block < 0 || c.c_head < 0) return SPEC_ERR_SHAPE;
  if (!aligned16(c.k) || !aligned16(c.v) || (reinterpret_cast<uintptr_t>(c.k_scale) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(c.v_scale) & 3u) != 0)
    return SPEC_ERR_ALIGN;
  if (!mult16(c.s_layer) || !mult16(c.s_page) || !mult16(c.s_slot) || !mult16(c.s_head)) return SPEC_ERR_ALIGN;
  return SPEC_OK;
}

// Whether results overlap the scales of `layers` layers from `first` on.
bool scale_overlap(const spec_cache8& c, int first, int layers, std::initializer_list<Span> results) {
  const long long n = (layers - 1) * c.c_layer + (c.num_pages - 1) * c.c_page + (c.page_size / c.block - 1) * c.c_block +
                      (c.heads - 1) * c.c_head + 1;
  return overlap(results, {{c.k_scale + first * c.c_layer, n}, {c.v_scale + first * c.c_layer, n}});
}

// The same call over a 16-bit cache, for the checks and parameters that both
// have (offsets into the cache apart).
spec_tree_args as_tree(const spec_cache8_args& a) {
  spec_tree_args t;
  std::memset(&t, 0, sizeof(t));
  t.B = a.B;
  t.total_nodes = a.total_nodes;
  t.max_nodes = a.max_nodes;
  t.heads_q = a.heads_q;
  t.layer = a.layer;
  t.scale = a.scale;
  t.cu_nodes = a.cu_nodes;
  t.q = a.q;
  t.sq_node = a.sq_node;
  t.sq_head = a.sq_head;
  t.k_new = a.k_new;
  t.v_new = a.v_new;
  t.sn_node = a.sn_node;
  t.sn_head = a.sn_head;
  t.tree_mask = a.tree_mask;
  t.mask_words = a.mask_words;
  t.ld_table = a.ld_table;
  t.cache.k = a.cache.k;
  t.cache.v = a.cache.v;
  t.cache.dtype = a.dtype;
  t.cache.layers = a.cache.layers;
  t.cache.num_pages = a.cache.num_pages;
  t.cache.page_size = a.cache.page_size;
  t.cache.heads = a.cache.heads;
  t.cache.dim = a.cache.dim;
  t.cache.s_layer = a.cache.s_layer;
  t.cache.s_page = a.cache.s_page;
  t.cache.s_slot = a.cache.s_slot;
  t.cache.s_head = a.cache.s_head;
  t.block_table = a.block_table;
  t.ctx_len = a.ctx_len;
  return t;
}

int check_window(int window, int sinks) { return window >= 1 && sinks >= 0 ? SPEC_OK : SPEC_ERR_SHAPE; }

int check_cache8_args(const spec_cache8_args* a, spec_tree_args* t) {
  if (!a) return SPEC_ERR_NULL;
  int rc = check_cache8(a->cache);
  if (rc) return rc;
  if (!sixteen(a->dtype)) return SPEC_ERR_DTYPE;
  *t = as_tree(*a);
  rc = check_tree(t);
  if (rc) return rc;
  return a->window == 0 && a->sinks == 0 ? SPEC_OK : check_window(a->window, a->sinks);
}

// The tensor-memory kernel takes the calls whose tiles TMA can copy, with a
// positive scale, down to one token of one request: against warp tiles, 64
// requests of one token over up to 8192, 28 / 4 heads of 128 channels, 125 us and
// 160; one of 2000 tokens, 32 / 8 heads, 23 and 28; one of 1001 tokens, 14 / 2
// heads of 64, 12.3 and 12.0.
sv::TreePlan plan_cache8(const spec_cache8_args* a, int num_sms) {
  const spec_cache8& c = a->cache;
  const int rows = a->max_nodes * (a->heads_q / c.heads);
  const bool fits = rows <= kMaxTcRows && a->scale > 0.f && sv::cache8_tc_fits(c.dim, c.page_size, c.block) && a->total_nodes > 0 &&
                    tma_stride(c.s_slot, c.page_size) && tma_stride(c.s_head, c.heads) && tma_stride(c.s_page, c.num_pages);
  return fits ? sv::plan_cache8_tc(rows, num_sms) : sv::plan_cache8_warp(c.dim, num_sms);
}

// The largest power of two up to 64 that divides the page size: the copies of
// the tensor-memory kernels hold this many tokens, and warp tiles begin
// anywhere.
int window_align(const sv::TreePlan& plan, int page_size) {
  if (plan.kernel == 0) return 1;
  int a = 1;
  while (a < 64 && page_size % (2 * a) == 0) a *= 2;
  return a;
}

int check_results(const spec_tree_args* a, const void* out, int64_t so_node, int64_t so_head, const void* workspace) {
  if (a->total_nodes > 0) {
    if (!out) return SPEC_ERR_NULL;
    if (!aligned16(out) || !mult8(so_node) || !mult8(so_head)) return SPEC_ERR_ALIGN;
  }
  return workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 ? SPEC_OK : SPEC_ERR_WORKSPACE;
}

}  // namespace

extern "C" {

int spec_norm_rotate(const spec_rotate_args* a, void* out_q, int64_t oq_row, int64_t oq_head, void* out_k,
                     int64_t ok_row, int64_t ok_head, spec_stream_t stream) {
  NvtxRange nvtx("spec_norm_rotate");
  if (!a) return SPEC_ERR_NULL;
  if (!sixteen(a->dtype)) return SPEC_ERR_DTYPE;
  if (a->rows < 0 || a->heads_q < 0 || a->heads_k < 0 || a->heads_q > 65535 || a->heads_k > 65535) return SPEC_ERR_SHAPE;
  if (a->dim != 64 && a->dim != 96 && a->dim != 128 && a->dim != 192 && a->dim != 256) return SPEC_ERR_SHAPE;
  if (a->rot < 0 || a->rot > a->dim || a->rot % 8 != 0 || !(a->eps >= 0.f) || !std::isfinite(a->eps)) return SPEC_ERR_SHAPE;
  const bool any = a->rows > 0 && (a->heads_q > 0 || a->heads_k > 0);
  if (any) {
    if (!a->positions || (a->rot > 0 && !a->inv_freq)) return SPEC_ERR_NULL;
    int rc = check_side(a->q, a->heads_q, a->sq_row, a->sq_head);
    if (!rc) rc = check_side(a->k, a->heads_k, a->sk_row, a->sk_head);
    if (!rc) rc = check_side(out_q, a->heads_q, oq_row, oq_head);
    if (!rc) rc = check_side(out_k, a->heads_k, ok_row, ok_head);
    if (rc) return rc;
    if (!aligned16(a->q_weight) || !aligned16(a->k_weight)) return SPEC_ERR_ALIGN;
    const Rows q(a->q, a->rows, a->heads_q, a->dim, a->sq_row, a->sq_head),
        k(a->k, a->rows, a->heads_k, a->dim, a->sk_row, a->sk_head),
        oq(out_q, a->rows, a->heads_q, a->dim, oq_row, oq_head), ok(out_k, a->rows, a->heads_k, a->dim, ok_row, ok_head);
    const bool q_in_place = out_q == a->q && oq_row == a->sq_row && oq_head == a->sq_head;
    const bool k_in_place = out_k == a->k && ok_row == a->sk_row && ok_head == a->sk_head;
    if (overlaps_itself(a->rows, a->heads_q, a->dim, oq_row, oq_head) ||
        overlaps_itself(a->rows, a->heads_k, a->dim, ok_row, ok_head))
      return SPEC_ERR_SHAPE;
    if ((!q_in_place && rows_overlap(oq, q)) || (!k_in_place && rows_overlap(ok, k)) || rows_overlap(oq, k) ||
        rows_overlap(ok, q) || rows_overlap(oq, ok))
      return SPEC_ERR_SHAPE;
    for (const Rows& o : {oq, ok})
      if (overlap({{reinterpret_cast<const void*>(o.at), (long long)o.all, 1}},
                  {{a->positions, a->rows}, {a->inv_freq, a->rot / 2}, {a->q_weight, a->dim, 2}, {a->k_weight, a->dim, 2}}))
        return SPEC_ERR_SHAPE;
  }
  int sms = 0;
  const int rc = sm_count(&sms);
  if (rc) return rc;
  if (!any) return SPEC_OK;
  sv::RotateParams P;
  std::memset(&P, 0, sizeof(P));
  P.side[0] = {a->q, out_q, a->q_weight, a->sq_row, a->sq_head, oq_row, oq_head, a->heads_q};
  P.side[1] = {a->k, out_k, a->k_weight, a->sk_row, a->sk_head, ok_row, ok_head, a->heads_k};
  P.positions = a->positions;
  P.inv_freq = a->inv_freq;
  P.eps = a->eps;
  P.rows = a->rows;
  P.dim = a->dim;
  P.rot = a->rot;
  P.interleaved = a->interleaved != 0;
  return sv::launch_norm_rotate(P, a->dtype == SPEC_BF16, sms, reinterpret_cast<cudaStream_t>(stream)) == 0 ? SPEC_OK
                                                                                                            : SPEC_ERR_LAUNCH;
}

size_t spec_window_workspace_bytes(const spec_window_args* a) {
  if (!a || check_tree(&a->tree) || check_window(a->window, a->sinks)) return 0;
  int sms = kPlanSms;
  if (sm_count(&sms)) sms = kPlanSms;
  const sv::TreePlan p = plan_tree(&a->tree, sms);
  return sv::make_tree_workspace(a->tree.B, p.grid, p.rows, a->tree.cache.dim).total;
}

int spec_window_attention(const spec_window_args* a, void* out, int64_t so_node, int64_t so_head, float* out_lse,
                          int32_t* out_status, void* workspace, size_t ws_bytes, spec_stream_t stream) {
  NvtxRange nvtx("spec_window_attention");
  if (!a) return SPEC_ERR_NULL;
  int rc = check_tree(&a->tree);
  if (!rc) rc = check_window(a->window, a->sinks);
  if (!rc) rc = check_results(&a->tree, out, so_node, so_head, workspace);
  if (rc) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  const sv::TreePlan plan = plan_tree(&a->tree, rc ? kPlanSms : sms);
  const sv::TreeWorkspace W = sv::make_tree_workspace(a->tree.B, plan.grid, plan.rows, a->tree.cache.dim);
  if (ws_bytes < W.total) return SPEC_ERR_WORKSPACE;
  if (rc) return rc;
  if (tree_overlap(&a->tree, out_lse, out_status)) return SPEC_ERR_SHAPE;
  sv::TreeParams P;
  fill_tree(P, &a->tree, plan, W, out, so_node, so_head, out_lse, out_status, workspace);
  P.window = a->window;
  P.sinks = a->sinks;
  P.align = window_align(plan, a->tree.cache.page_size);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = a->tree.cache.dtype == SPEC_BF16;
  if (plan.kernel == 1 ? sv::launch_window_tc(P, bf16, s) : sv::launch_window_warp(P, bf16, s)) return SPEC_ERR_LAUNCH;
  return sv::launch_window_join(P, bf16, sms, s) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

size_t spec_cache8_workspace_bytes(const spec_cache8_args* a) {
  spec_tree_args t;
  if (check_cache8_args(a, &t)) return 0;
  int sms = kPlanSms;
  if (sm_count(&sms)) sms = kPlanSms;
  const sv::TreePlan p = plan_cache8(a, sms);
  return sv::make_tree_workspace(a->B, p.grid, p.rows, a->cache.dim).total;
}

int spec_cache8_attention(const spec_cache8_args* a, void* out, int64_t so_node, int64_t so_head, float* out_lse,
                          int32_t* out_status, void* workspace, size_t ws_bytes, spec_stream_t stream) {
  NvtxRange nvtx("spec_cache8_attention");
  spec_tree_args t;
  int rc = check_cache8_args(a, &t);
  if (!rc) rc = check_results(&t, out, so_node, so_head, workspace);
  if (rc) return rc;
  int sms = 0;
  rc = sm_count(&sms);
  const sv::TreePlan plan = plan_cache8(a, rc ? kPlanSms : sms);
  const sv::TreeWorkspace W = sv::make_tree_workspace(a->B, plan.grid, plan.rows, a->cache.dim);
  if (ws_bytes < W.total) return SPEC_ERR_WORKSPACE;
  if (tree_overlap(&t, out_lse, out_status) ||
      scale_overlap(a->cache, a->layer, 1, {{out_lse, (long long)a->total_nodes * a->heads_q}, {out_status, a->B}}))
    return SPEC_ERR_SHAPE;
  if (rc) return rc;
  sv::Cache8Params C;
  std::memset(&C, 0, sizeof(C));
  fill_tree(C.t, &t, plan, W, out, so_node, so_head, out_lse, out_status, workspace);
  C.t.k = static_cast<const uint8_t*>(a->cache.k) + (long long)a->layer * a->cache.s_layer;
  C.t.v = static_cast<const uint8_t*>(a->cache.v) + (long long)a->layer * a->cache.s_layer;
  C.t.window = a->window ? a->window : INT32_MAX;
  C.t.sinks = a->sinks;
  C.t.align = window_align(plan, a->cache.page_size);
  C.ks = a->cache.k_scale + (long long)a->layer * a->cache.c_layer;
  C.vs = a->cache.v_scale + (long long)a->layer * a->cache.c_layer;
  C.c_page = a->cache.c_page;
  C.c_block = a->cache.c_block;
  C.c_head = a->cache.c_head;
  C.block = a->cache.block;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = a->dtype == SPEC_BF16;
  if (plan.kernel == 1 ? sv::launch_cache8_tc(C, bf16, s) : sv::launch_cache8_warp(C, bf16, s)) return SPEC_ERR_LAUNCH;
  return sv::launch_window_join(C.t, bf16, sms, s) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

int spec_cache8_commit(const spec_cache8_commit_args* a, int32_t* out_len, int32_t* out_status, spec_stream_t stream) {
  NvtxRange nvtx("spec_cache8_commit");
  if (!a) return SPEC_ERR_NULL;
  const spec_cache8& c = a->cache;
  int rc = check_cache8(c);
  if (rc) return rc;
  if (!sixteen(a->dtype)) return SPEC_ERR_DTYPE;
  if (a->B < 1 || a->total_nodes < 0 || a->ld_path < 1 || c.layers > 65535) return SPEC_ERR_SHAPE;
  // units of a block and head, for keys and values
  if (!fits32((a->ld_path + c.block - 2ll) / c.block + 1, c.heads, 2, kMaxTokens)) return SPEC_ERR_SHAPE;
  if (!table_ok(a->ld_table, c.page_size)) return SPEC_ERR_SHAPE;
  if (!a->cu_nodes || !a->path || !a->path_len || !a->block_table || !a->ctx_len || !out_len) return SPEC_ERR_NULL;
  if (a->total_nodes > 0) {
    if (!a->k_new || !a->v_new) return SPEC_ERR_NULL;
    if (!aligned16(a->k_new) || !aligned16(a->v_new) || !mult8(a->sn_layer) || !mult8(a->sn_node) ||
        !mult8(a->sn_head))
      return SPEC_ERR_ALIGN;
  }
  const long long lens = a->B;
  if (overlap({{out_len, lens}, {out_status, lens}},
              {{a->cu_nodes, lens + 1}, {a->path, lens * a->ld_path}, {a->path_len, lens},
               {a->block_table, lens * a->ld_table}, {out_len == a->ctx_len ? nullptr : a->ctx_len, lens}}) ||
      overlap({{out_status, lens}}, {{a->ctx_len, lens}, {out_len, lens}}) ||
      scale_overlap(c, 0, c.layers, {{out_len, lens}, {out_status, lens}}))
    return SPEC_ERR_SHAPE;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  sv::Commit8Params P;
  std::memset(&P, 0, sizeof(P));
  P.cu = a->cu_nodes;
  P.path = a->path;
  P.path_len = a->path_len;
  P.table = a->block_table;
  P.ctx = a->ctx_len;
  P.x[0] = a->k_new;
  P.x[1] = a->v_new;
  P.held[0] = static_cast<uint8_t*>(c.k);
  P.held[1] = static_cast<uint8_t*>(c.v);
  P.scale[0] = c.k_scale;
  P.scale[1] = c.v_scale;
  P.sn_layer = a->sn_layer;
  P.sn_node = a->sn_node;
  P.sn_head = a->sn_head;
  P.s_layer = c.s_layer;
  P.s_page = c.s_page;
  P.s_slot = c.s_slot;
  P.s_head = c.s_head;
  P.c_layer = c.c_layer;
  P.c_page = c.c_page;
  P.c_block = c.c_block;
  P.c_head = c.c_head;
  P.new_len = out_len;
  P.status = out_status;
  P.B = a->B;
  P.total = a->total_nodes;
  P.layers = c.layers;
  P.ld_path = a->ld_path;
  P.ld_table = a->ld_table;
  P.num_pages = c.num_pages;
  P.page_size = c.page_size;
  P.heads = c.heads;
  P.dim = c.dim;
  P.block = c.block;
  return sv::launch_commit8(P, a->dtype == SPEC_BF16, sms, reinterpret_cast<cudaStream_t>(stream)) == 0 ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // extern "C"
