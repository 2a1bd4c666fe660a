// Attention of drafted trees over a paged cache: warp tiles on mma.sync, and
// the kernel that joins items split over several CTAs.
#include "tree_common.cuh"

namespace sv {
namespace {

constexpr int kWtWarps = 4;
constexpr int kWtKeys = 16 * kWtWarps;  // keys per tile: 16 per warp

template <int D>
struct WtShape {
  static constexpr int kPitch = D + 8;  // elements per staged row: ldmatrix rows on distinct banks
  static constexpr int kWarpStage = 2 * 16 * kPitch * 2;
  static constexpr int kStage = kWtWarps * kWarpStage;
  static constexpr int kStages = D <= 64 ? 5 : (D <= 96 ? 4 : (D <= 128 ? 3 : (D <= 192 ? 4 : 3)));
  static constexpr int kSmem = kStage * kStages + 2 * 16 * kWtWarps * 4;
  static constexpr int kCtas = D <= 128 ? 2 : 1;  // per SM
};

// One item's tiles: each warp takes 16 keys of every tile with a running
// maximum m, sum l and output O of its own,
//   m' = max(m, max_j s_j),  O' = O 2^(m-m') + sum_j 2^(s_j-m') v_j,
//   l' = l 2^(m-m') + sum_j 2^(s_j-m'),
// and the warps' results are joined by the same rule at the segment's end.
//
// Few query rows do a few operations per byte of the cache, so the cache's
// bytes bound the kernel: each warp keeps its own ring of 16-byte asynchronous
// copies in flight (up to 128 KB per SM) and never waits for the others inside
// a segment.  64 requests of one token and 28 / 4 heads of 128 channels over
// 2000 cached tokens: 263 MB in 52 us, 5.1 TB/s (75 % of the copy rate); with
// the launch and the joining kernel, 59 us.  One token of one request over 700
// tokens: 9.2 us, all of it latency.
template <typename T, int D>
__global__ void __launch_bounds__(kWtWarps * 32, WtShape<D>::kCtas) tree_warp_kernel(const TreeParams P) {
  using S = WtShape<D>;
  constexpr int CH = D / 8;    // 16-byte pieces per row
  constexpr int NLD = CH / 2;  // pieces per lane for 16 rows
  extern __shared__ __align__(128) unsigned char smem[];
  float* ml = reinterpret_cast<float*>(smem + S::kStage * S::kStages);  // [warp][16] m, then l
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  unsigned char* ring = smem + warp * S::kWarpStage;
  const PageDiv pd(P.page_size);
  const T* kc = static_cast<const T*>(P.k);
  const T* vc = static_cast<const T*>(P.v);
  const T* kn = static_cast<const T*>(P.k_new);
  const T* vn = static_cast<const T*>(P.v_new);
  const T* q = static_cast<const T*>(P.q);

  after_previous();
  const TreeScan scan = tree_scan(P, lane);
  if (blockIdx.x == 0 && warp == 0) tree_store_starts(P, scan, lane);
  TreeWalk walk;
  walk.begin(P, lane, scan, blockIdx.x);
  TreeSeg g;
  while (walk.next(P, g)) {
    const TreeReq& r = walk.r;
    const int row_lo = g.m * 16;
    const int nrows = min(16, r.n * P.group - row_lo);
    // Q fragments, rows r0 and r0 + 8
    uint32_t qf[D / 16][4];
    int node[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rr = r0 + 8 * h;
      const bool in = rr < nrows;
      node[h] = in ? (row_lo + rr) / P.group : 0;
      const T* src = q + (long long)(r.cu + node[h]) * P.sq_node +
                     (long long)(g.kvh * P.group + (in ? (row_lo + rr) % P.group : 0)) * P.sq_head;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[ks][2 * e + h] = in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + e * 8 + c0) : 0u;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int bad = 0;
    __syncthreads();  // the last segment's join is done with the ring

    // Keys of a tile that this warp holds: [lo, lo + 16) of the cached or drafted ones
    auto tile_lo = [&](int t) { return (t < r.ct ? t : t - r.ct) * kWtKeys + warp * 16; };
    auto load = [&](int t) {
      if (t >= g.t1) return;
      const bool cached = t < r.ct;
      const int lo = tile_lo(t), lim = cached ? r.ctx : r.n;
      if (lo >= lim) return;
      const int j = lo + (lane & 15);
      bool real = j < lim;
      long long off = 0;
      if (real) {
        if (cached) {
          int page, slot;
          pd.split(j, page, slot);
          const int id = P.table[(long long)g.b * P.ld_table + page];
          if (id < 0 || id >= P.num_pages) {
            bad = 1;
            real = false;
          } else {
            off = (long long)id * P.s_page + (long long)slot * P.s_slot + (long long)g.kvh * P.s_head;
          }
        } else {
          off = (long long)(r.cu + j) * P.sn_node + (long long)g.kvh * P.sn_head;
        }
      }
      const T* kb = cached ? kc : kn;
      const T* vb = cached ? vc : vn;
      const uint32_t dst = smem_u32(ring + (t % S::kStages) * S::kStage);
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int idx = i * 32 + lane, row = idx / CH, ch = idx % CH;
        const long long ro = __shfl_sync(0xffffffffu, off, row);
        const bool rl = __shfl_sync(0xffffffffu, (int)real, row) != 0;
        const uint32_t at = dst + (row * S::kPitch + ch * 8) * 2;
        cp_async16(at, kb + ro + ch * 8, rl);
        cp_async16(at + 16 * S::kPitch * 2, vb + ro + ch * 8, rl);
      }
    };

#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      load(g.t0 + i);
      cp_async_commit();
    }
    for (int t = g.t0; t < g.t1; ++t) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      load(t + S::kStages - 1);  // into the slot that tile t - 1 left
      cp_async_commit();
      const bool cached = t < r.ct;
      const int lo = tile_lo(t), lim = cached ? r.ctx : r.n;
      if (lo >= lim) continue;  // warp-uniform
      const uint32_t kb = smem_u32(ring + (t % S::kStages) * S::kStage);
      const uint32_t vb = kb + 16 * S::kPitch * 2;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      // matrices: keys 0-7 (channels 0-7, 8-15), keys 8-15 (0-7, 8-15)
      const uint32_t krow = kb + ((lane & 7) + ((lane & 16) >> 1)) * (S::kPitch * 2) + (lane & 8) * 2;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kf[4];
        ldsm4(krow + ks * 32, kf);
        mma16816<T>(s[0], qf[ks], kf[0], kf[1]);
        mma16816<T>(s[1], qf[ks], kf[2], kf[3]);
      }
      uint32_t see[2];
      if (cached) {
        const int left = lim - lo;
        see[0] = see[1] = left >= 16 ? 0xffffu : (1u << left) - 1u;
      } else {
        see[0] = tree_bits16(P, r.cu, r.n, node[0], lo);
        see[1] = tree_bits16(P, r.cu, r.n, node[1], lo);
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1, key = nt * 8 + c0 + (e & 1);
          s[nt][e] = ((see[h] >> key) & 1u) ? s[nt][e] * P.scale_log2 : -INFINITY;
          mx[h] = fmaxf(mx[h], s[nt][e]);
        }
      float sc[2], ref[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        const float mn = fmaxf(m[h], mx[h]);
        ref[h] = mn == -INFINITY ? 0.f : mn;
        sc[h] = ex2(m[h] - ref[h]);
        m[h] = mn;
        l[h] *= sc[h];
      }
      uint32_t pf[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(s[nt][e] - ref[e >> 1]);
          l[e >> 1] += p[e];
        }
        pf[2 * nt] = pack2<T>(p[0], p[1]);
        pf[2 * nt + 1] = pack2<T>(p[2], p[3]);
      }
      if (__any_sync(0xffffffffu, sc[0] != 1.f || sc[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= sc[0];
          o[i][1] *= sc[0];
          o[i][2] *= sc[1];
          o[i][3] *= sc[1];
        }
      }
      if (!cached) {
        // A value that some rows do not see must not reach them, but 0 times
        // an infinity or NaN would: such values are added to the rows that
        // see them here, and are zero for the matrix product.
        uint32_t* vs = reinterpret_cast<uint32_t*>(ring + (t % S::kStages) * S::kStage + 16 * S::kPitch * 2);
        uint32_t odd = 0;
        for (int i = lane; i < 16 * (D / 2); i += 32) {
          const uint32_t w = vs[(i / (D / 2)) * (S::kPitch / 2) + i % (D / 2)];
          const uint32_t em = exp_mask<T>();
          odd |= (uint32_t)((w & em) == em || ((w >> 16) & em) == em);
        }
        if (__any_sync(0xffffffffu, odd != 0u)) {
          const uint32_t em = exp_mask<T>();
          for (int key = 0; key < 16; ++key)
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const uint32_t w = vs[key * (S::kPitch / 2) + i * 4 + (lane & 3)];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t x = e ? w >> 16 : w & 0xffffu;
                if ((x & em) == em) {
                  if ((see[0] >> key) & 1u) o[i][e] += half_to_f32<T>(x);
                  if ((see[1] >> key) & 1u) o[i][2 + e] += half_to_f32<T>(x);
                }
              }
            }
          __syncwarp();
          for (int i = lane; i < 16 * (D / 2); i += 32) {
            uint32_t& w = vs[(i / (D / 2)) * (S::kPitch / 2) + i % (D / 2)];
            uint32_t x = w;
            if ((x & em) == em) x &= 0xffff0000u;
            if (((x >> 16) & em) == em) x &= 0xffffu;
            w = x;
          }
          __syncwarp();
        }
      }
      // matrices (transposed): keys 0-7, 8-15 of channels 0-7, then of 8-15
      const uint32_t vrow = vb + (lane & 15) * (S::kPitch * 2) + (lane & 16);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t vf[4];
        ldsm4t(vrow + i * 32, vf);
        mma16816<T>(o[2 * i], pf, vf[0], vf[1]);
        mma16816<T>(o[2 * i + 1], pf, vf[2], vf[3]);
      }
      __syncwarp();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    const bool poison = __syncthreads_or(bad) != 0;  // and every warp is done with its ring
    float* so = reinterpret_cast<float*>(smem);  // [warp][16][D]
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(so + (warp * 16 + r0 + 8 * h) * D + i * 8 + c0) =
            make_float2(o[i][2 * h], o[i][2 * h + 1]);
    if ((lane & 3) == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ml[warp * 16 + r0 + 8 * h] = m[h];
        ml[16 * kWtWarps + warp * 16 + r0 + 8 * h] = l[h];
      }
    }
    __syncthreads();
    const bool whole = g.t0 == 0 && g.t1 == r.per_item;
    const int slot = 2 * blockIdx.x + tree_slot(g.t0 == 0);
    for (int i = tid; i < nrows * (D / 2); i += kWtWarps * 32) {
      const int row = i / (D / 2), d = (i % (D / 2)) * 2;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWtWarps; ++w) M = fmaxf(M, ml[w * 16 + row]);
      const float R = M == -INFINITY ? 0.f : M;
      float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWtWarps; ++w) {
        const float f = ex2(ml[w * 16 + row] - R);
        L += ml[16 * kWtWarps + w * 16 + row] * f;
        const float2 v = *reinterpret_cast<const float2*>(so + (w * 16 + row) * D + d);
        x += v.x * f;
        y += v.y * f;
      }
      if (poison) L = x = y = NAN;
      const int R2 = row_lo + row;
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int nd = R2 / P.group, head = g.kvh * P.group + R2 % P.group;
        T* dst = static_cast<T*>(P.out) + (long long)(r.cu + nd) * P.so_node + (long long)head * P.so_head;
        *reinterpret_cast<uint32_t*>(dst + d) = pack2<T>(x * inv, y * inv);
        if (P.lse && d == 0)
          P.lse[(long long)(r.cu + nd) * P.heads * P.group + head] = L == 0.f ? -INFINITY : (R + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float2*>(P.part_o + (((long long)slot * (D / 4) + d / 4) * 16 + row) * 4 + d % 4) = make_float2(x, y);
        if (d == 0) P.part_ml[(long long)slot * 16 + row] = make_float4(M, L, L, 0.f);
      }
    }
  }
}

// Joins the pieces of split items, in tile order.  A warp takes 8 rows of one
// item: lane l the row l % 8 and channels 4 (l / 8) .. + 3 of every 16, so
// that pieces are read by 128 bytes and results written by 32.  Also the
// status of every request, and NaN in the rows of one whose lengths are bad.
//
// A few pieces of an item are read by one warp; many (a long context of few
// heads) by all warps of the CTA, a share each, whose sums are added in warp
// order.  The pieces come from L2, so latency bounds it.  Limits of 1 / 6 / any
// number of pieces for one warp (attention and joining, us): trees of 16
// requests 119 / 89 / 89, two contexts of 128 K tokens 157 / 157 / 166, one
// token over 32000 cached ones 17.5 / 17.5 / 39.4.
template <int D>
constexpr int kJoinOf = D <= 128 ? 8 : 4;  // warps: their sums fit 48 KB of shared memory
constexpr int kJoinFew = 6;  // pieces that one warp reads

template <typename T, int D>
__global__ void __launch_bounds__(kJoinOf<D> * 32) tree_join_kernel(const TreeParams P) {
  constexpr int kJoinWarps = kJoinOf<D>;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  after_previous();
  const TreeReq r = tree_request(P, b);
  const int heads_q = P.heads * P.group;
  if (blockIdx.y == 0 && P.status) {
    int bad = 0;
    if (r.ok) {
      const long long pages = ((long long)r.ctx + P.page_size - 1) / P.page_size;
      for (long long p = threadIdx.x; p < pages; p += kJoinWarps * 32) {
        const int id = P.table[(long long)b * P.ld_table + p];
        bad |= id < 0 || id >= P.num_pages;
      }
    }
    bad = __syncthreads_or(bad);
    int late = 0;
    if (P.failed)
      for (int c = threadIdx.x; c < P.grid; c += kJoinWarps * 32) late |= P.failed[c];
    late = __syncthreads_or(late);
    if (threadIdx.x == 0)
      P.status[b] = (r.ok ? (bad ? kStatusBadPage : 0) : kStatusBadLen) | (late ? kStatusTimeout : 0);
  }
  if (r.cu < 0 || r.n < 0 || (long long)r.cu + r.n > P.total) return;
  T* out = static_cast<T*>(P.out);
  const int sub = lane & 7, quad = lane >> 3;
  if (!r.ok) {
    for (long long i = (long long)blockIdx.y * kJoinWarps + warp; i < (long long)r.n * heads_q;
         i += (long long)gridDim.y * kJoinWarps) {
      const int node = (int)(i / heads_q), head = (int)(i - (long long)node * heads_q);
      T* dst = out + (long long)(r.cu + node) * P.so_node + (long long)head * P.so_head;
      for (int d = 2 * lane; d < D; d += 64) *reinterpret_cast<uint32_t*>(dst + d) = pack2<T>(NAN, NAN);
      if (P.lse && lane == 0) P.lse[(long long)(r.cu + node) * heads_q + head] = NAN;
    }
    return;
  }
  const long long T_ = P.start[P.B], s0 = P.start[b];
  const int used = tree_used(P, T_);
  const int rows = r.n * P.group, blocks = (rows + 7) / 8;  // P.rows is a multiple of 8
  if (rows == 0) return;
  // most pieces of an item of this request
  const int most = (int)(((long long)r.per_item * used + T_ - 1) / T_) + 1;
  const bool many = most > kJoinFew;
  const int step = many ? gridDim.y : gridDim.y * kJoinWarps;
  __shared__ float4 part[kJoinWarps][D / 16][32];
  __shared__ float4 part_ml[kJoinWarps][8];
  for (int i = many ? blockIdx.y : blockIdx.y * kJoinWarps + warp; i < blocks * P.heads; i += step) {
    const int kvh = i / blocks, R0 = (i - kvh * blocks) * 8;
    const long long s = s0 + ((long long)kvh * r.mb + R0 / P.rows) * r.per_item;
    const int c0 = tree_owner(s, T_, used), c1 = tree_owner(s + r.per_item - 1, T_, used);
    if (c0 == c1) continue;  // written whole
    const bool in = R0 + sub < rows;
    const int row = R0 % P.rows + (in ? sub : 0);
    // CTA c0 in slot 1, c0 + 1 .. c1 in slot 0; a running reference as in the
    // main kernel, four pieces' loads at once
    float M = -INFINITY, L = 0.f, N = 0.f;  // N: the outputs' divisor
    float4 acc[D / 16];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int by = many ? kJoinWarps : 1;
    constexpr int U = D <= 64 ? 4 : (D <= 128 ? 2 : 1);
    for (int c = c0 + (many ? warp : 0); c <= c1; c += U * by) {
      float4 ml[U];
      float4 v[U][D / 16];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c + u * by;
        const long long at = 2ll * cu + (cu == c0);
        ml[u] = cu <= c1 ? __ldcg(&P.part_ml[at * P.rows + row]) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        const float4* src = reinterpret_cast<const float4*>(P.part_o) + (at * (D / 4) + quad) * P.rows + row;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          v[u][k] = cu <= c1 ? __ldcg(src + (long long)k * 4 * P.rows) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float to = fmaxf(M, ml[u].x), ref = to == -INFINITY ? 0.f : to;
        const float f = ex2(M - ref), h = ex2(ml[u].x - ref);
        L = L * f + ml[u].y * h;
        N = N * f + ml[u].z * h;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          acc[k].x = acc[k].x * f + v[u][k].x * h;
          acc[k].y = acc[k].y * f + v[u][k].y * h;
          acc[k].z = acc[k].z * f + v[u][k].z * h;
          acc[k].w = acc[k].w * f + v[u][k].w * h;
        }
        M = to;
      }
    }
    if (many) {
      __syncthreads();  // the last block's sums have been read
      if (quad == 0) part_ml[warp][sub] = make_float4(M, L, N, 0.f);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) part[warp][k][lane] = acc[k];
      __syncthreads();
      // channels by warp: a warp adds the sums of D / 16 / kJoinWarps vectors (or one, by some)
      M = -INFINITY;
      for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, part_ml[w][sub].x);
      const float ref = M == -INFINITY ? 0.f : M;
      L = N = 0.f;
      for (int w = 0; w < kJoinWarps; ++w) {
        const float h = ex2(part_ml[w][sub].x - ref);
        L += part_ml[w][sub].y * h;
        N += part_ml[w][sub].z * h;
      }
      const float inv = L == 0.f ? 0.f : 1.f / N;
      const int R = R0 + sub, node = in ? R / P.group : 0, head = kvh * P.group + (in ? R - node * P.group : 0);
      T* dst = out + (long long)(r.cu + node) * P.so_node + (long long)head * P.so_head + quad * 4;
      for (int k = warp; k < D / 16; k += kJoinWarps) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < kJoinWarps; ++w) {
          const float h = ex2(part_ml[w][sub].x - ref);
          const float4 v = part[w][k][lane];
          t.x += v.x * h;
          t.y += v.y * h;
          t.z += v.z * h;
          t.w += v.w * h;
        }
        if (in) {
          uint2 o;
          o.x = pack2<T>(t.x * inv, t.y * inv);
          o.y = pack2<T>(t.z * inv, t.w * inv);
          *reinterpret_cast<uint2*>(dst + k * 16) = o;
        }
      }
      if (in && P.lse && warp == 0 && quad == 0)
        P.lse[(long long)(r.cu + node) * heads_q + head] = L == 0.f ? -INFINITY : (ref + log2f(L)) * kLn2;
      continue;
    }
    if (!in) continue;
    const float ref = M == -INFINITY ? 0.f : M;
    const int R = R0 + sub, node = R / P.group, head = kvh * P.group + R - node * P.group;
    const float inv = L == 0.f ? 0.f : 1.f / N;
    T* dst = out + (long long)(r.cu + node) * P.so_node + (long long)head * P.so_head + quad * 4;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint2 v;
      v.x = pack2<T>(acc[k].x * inv, acc[k].y * inv);
      v.y = pack2<T>(acc[k].z * inv, acc[k].w * inv);
      *reinterpret_cast<uint2*>(dst + k * 16) = v;
    }
    if (P.lse && quad == 0)
      P.lse[(long long)(r.cu + node) * heads_q + head] = L == 0.f ? -INFINITY : (ref + log2f(L)) * kLn2;
  }
}

template <typename T, int D>
int launch_warp(const TreeParams& P, cudaStream_t s) {
  using S = WtShape<D>;
  if (cudaFuncSetAttribute(tree_warp_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(tree_warp_kernel<T, D>, dim3(P.grid), kWtWarps * 32, S::kSmem, s, P);
}

template <typename T>
int launch_warp_dim(const TreeParams& P, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch_warp<T, 64>(P, s);
    case 96: return launch_warp<T, 96>(P, s);
    case 128: return launch_warp<T, 128>(P, s);
    case 192: return launch_warp<T, 192>(P, s);
    case 256: return launch_warp<T, 256>(P, s);
    default: return -1;
  }
}

}  // namespace

TreePlan plan_tree_warp(int dim, int num_sms) {
  TreePlan p;
  p.kernel = 0;
  p.rows = 16;
  p.kt = kWtKeys;
  p.grid = num_sms * (dim <= 128 ? 2 : 1);
  return p;
}

int launch_tree_warp(const TreeParams& P, bool bf16, cudaStream_t s) {
  return bf16 ? launch_warp_dim<__nv_bfloat16>(P, s) : launch_warp_dim<__half>(P, s);
}

namespace {
template <typename T, int D>
int launch_join(const TreeParams& P, int num_sms, cudaStream_t s) {
  // A CTA for every 8 rows of the largest request, up to six per SM in all.
  const long long rows = (long long)P.max_nodes * P.group, want = (rows + 7) / 8 * P.heads;
  const long long most = (6ll * num_sms + P.B - 1) / P.B;
  return launch_kernel(tree_join_kernel<T, D>, dim3(P.B, (unsigned)max(1ll, min(want, most))), kJoinOf<D> * 32, 0, s, P);
}

template <typename T>
int launch_join_dim(const TreeParams& P, int num_sms, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch_join<T, 64>(P, num_sms, s);
    case 96: return launch_join<T, 96>(P, num_sms, s);
    case 128: return launch_join<T, 128>(P, num_sms, s);
    case 192: return launch_join<T, 192>(P, num_sms, s);
    case 256: return launch_join<T, 256>(P, num_sms, s);
    default: return -1;
  }
}
}  // namespace

int launch_tree_join(const TreeParams& P, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? launch_join_dim<__nv_bfloat16>(P, num_sms, s) : launch_join_dim<__half>(P, num_sms, s);
}

}  // namespace sv
