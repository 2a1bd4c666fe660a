// The kernel that joins attention items split over several CTAs and writes every
// request's status, with or without a sliding window.
#pragma once

#include "tree_common.cuh"

namespace sv {
namespace {

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

template <typename T, int D, bool WIN>
__global__ void __launch_bounds__(kJoinOf<D> * 32) tree_join_kernel(const TreeParams P) {
  constexpr int kJoinWarps = kJoinOf<D>;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  after_previous();
  const TreeReq r = tree_request<WIN>(P, b);
  const int heads_q = P.heads * P.group;
  if (blockIdx.y == 0 && P.status) {
    int bad = 0;
    if (r.ok) {
      const long long pages = ((long long)r.ctx + P.page_size - 1) / P.page_size;
      for (long long p = threadIdx.x; p < pages; p += kJoinWarps * 32) {
        // pages between the sinks and the window are not looked at
        if (WIN && p * P.page_size >= r.sk && (p + 1) * P.page_size <= r.b1) continue;
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

template <typename T, int D, bool WIN>
int launch_join(const TreeParams& P, int num_sms, cudaStream_t s) {
  // A CTA for every 8 rows of the largest request, up to six per SM in all.
  const long long rows = (long long)P.max_nodes * P.group, want = (rows + 7) / 8 * P.heads;
  const long long most = (6ll * num_sms + P.B - 1) / P.B;
  return launch_kernel(tree_join_kernel<T, D, WIN>, dim3(P.B, (unsigned)max(1ll, min(want, most))), kJoinOf<D> * 32, 0, s, P);
}

template <typename T, bool WIN>
int launch_join_dim(const TreeParams& P, int num_sms, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch_join<T, 64, WIN>(P, num_sms, s);
    case 96: return launch_join<T, 96, WIN>(P, num_sms, s);
    case 128: return launch_join<T, 128, WIN>(P, num_sms, s);
    case 192: return launch_join<T, 192, WIN>(P, num_sms, s);
    case 256: return launch_join<T, 256, WIN>(P, num_sms, s);
    default: return -1;
  }
}
}  // namespace
}  // namespace sv
