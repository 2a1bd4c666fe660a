// Attention of drafted trees over a paged cache: warp tiles on mma.sync, with or
// without a sliding window.
#pragma once

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
template <typename T, int D, bool WIN>
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
  const TreeScan scan = tree_scan<WIN>(P, lane);
  if (blockIdx.x == 0 && warp == 0) tree_store_starts<WIN>(P, scan, lane);
  TreeWalkOf<WIN> walk;
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
    TreeRow win[2];
    if (WIN) {
      win[0] = tree_row(P, r, node[0]);
      win[1] = tree_row(P, r, node[1]);
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int bad = 0;
    __syncthreads();  // the last segment's join is done with the ring

    auto load = [&](int t) {
      if (t >= g.t1) return;
      // keys of the tile that this warp holds: [lo, lo + 16) of the cached or drafted ones
      const TreeKeys tk = tree_keys<WIN>(r, kWtKeys, t);
      const bool cached = tk.cached;
      const int lo = tk.lo + warp * 16, lim = tk.lim;
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
      const TreeKeys tk = tree_keys<WIN>(r, kWtKeys, t);
      const bool cached = tk.cached;
      const int lo = tk.lo + warp * 16, lim = tk.lim;
      if (lo >= lim) continue;  // warp-uniform
      // keys that some rows see and others do not: drafted, or at a window's beginning
      const bool some = !cached || (WIN && t >= r.st && lo < r.part);
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
        if (WIN && some) {
          see[0] &= tree_window32(lo, win[0].lo, P.sinks);
          see[1] &= tree_window32(lo, win[1].lo, P.sinks);
        }
      } else {
        see[0] = tree_bits16(P, r.cu, r.n, node[0], lo);
        see[1] = tree_bits16(P, r.cu, r.n, node[1], lo);
        if (WIN) {
          see[0] = tree_window_drafted(P, r, win[0], node[0], lo, see[0]);
          see[1] = tree_window_drafted(P, r, win[1], node[1], lo, see[1]);
        }
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
      if (some) {
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

template <typename T, int D, bool WIN>
int launch_warp(const TreeParams& P, cudaStream_t s) {
  using S = WtShape<D>;
  if (cudaFuncSetAttribute(tree_warp_kernel<T, D, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(tree_warp_kernel<T, D, WIN>, dim3(P.grid), kWtWarps * 32, S::kSmem, s, P);
}

template <typename T, bool WIN>
int launch_warp_dim(const TreeParams& P, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch_warp<T, 64, WIN>(P, s);
    case 96: return launch_warp<T, 96, WIN>(P, s);
    case 128: return launch_warp<T, 128, WIN>(P, s);
    case 192: return launch_warp<T, 192, WIN>(P, s);
    case 256: return launch_warp<T, 256, WIN>(P, s);
    default: return -1;
  }
}

}  // namespace
}  // namespace sv
