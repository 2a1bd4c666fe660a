// Beam selection over beams and vocabulary, and the beams' states in their
// new order.
#include "stream_common.cuh"
#include "tree_internal.h"

namespace sv {
namespace {

constexpr int kBmThreads = 256;
constexpr int kBmWarps = kBmThreads / 32;
constexpr int kBmUnroll = 4;   // 16-byte loads in flight per lane
constexpr int kBmCap = 512;    // candidates a warp holds at most

// Unsigned order of a float's value (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t float_key(float z) {
  const uint32_t u = __float_as_uint(z == 0.f ? 0.f : z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long double_key(double z) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(z == 0.0 ? 0.0 : z);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_double(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// A warp's candidates: the tokens seen so far that may be among the best K
// of its part, in shared memory.  Every token that beats (tz, tt) — a larger
// logit, or the same one at a lower token — is added; K of those seen beat
// or equal it.
struct WarpCands {
  float* z;
  int* tok;
  int cnt;
  float tz;
  int tt;
};

// Keeps the best K of the warp's candidates (its count is above K) and makes
// the K-th best the new bound.  A bisection over the order keys, by counts of
// the whole warp, finds the K-th logit; a second one over tokens decides
// among its equals.
struct Bound {
  int cnt;
  float tz;
  int tt;
};

__device__ __noinline__ Bound prune_list(float* cz, int* ct, int cnt, int K, int lane) {
  constexpr int PER = kBmCap / 32;
  uint32_t key[PER];
  int tok[PER];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = i * 32 + lane;
    key[i] = at < cnt ? float_key(cz[at]) : 0u;  // 0: below every finite logit
    tok[i] = at < cnt ? ct[at] : 0x7fffffff;
  }
  uint32_t t = 0;  // the largest key with at least K at or above it
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t probe = t | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += key[i] >= probe;
    if (__reduce_add_sync(0xffffffffu, n) >= K) t = probe;
  }
  int above = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) above += key[i] > t;
  const int need = K - __reduce_add_sync(0xffffffffu, above);  // >= 1 of key t
  int last = 0;  // the largest token of them: fewer than `need` are below it
  for (int bit = 30; bit >= 0; --bit) {
    const int probe = last | (1 << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += key[i] == t && tok[i] < probe;
    if (__reduce_add_sync(0xffffffffu, n) < need) last = probe;
  }
  __syncwarp();
  int at = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool keep = key[i] > t || (key[i] == t && tok[i] <= last);
    const unsigned who = __ballot_sync(0xffffffffu, keep);
    if (keep) {
      const int to = at + __popc(who & ((1u << lane) - 1u));
      cz[to] = __uint_as_float((key[i] & 0x80000000u) ? key[i] & 0x7fffffffu : ~key[i]);
      ct[to] = tok[i];
    }
    at += __popc(who);
  }
  __syncwarp();
  return {at, __uint_as_float((t & 0x80000000u) ? t & 0x7fffffffu : ~t), last};
}

__device__ __forceinline__ void prune(WarpCands& c, int K, int lane) {
  const Bound n = prune_list(c.z, c.tok, c.cnt, K, lane);
  c.cnt = n.cnt;
  c.tz = n.tz;
  c.tt = n.tt;
}

// Adds a vector's tokens (base + e for this lane) that beat the bound.
template <int N>
__device__ __forceinline__ void gather(WarpCands& c, const float (&z)[N], int base, int K, int lane) {
  if (c.cnt + 32 * N > kBmCap) prune(c, K, lane);  // cnt > K here: K + 32 N <= kBmCap
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const bool in = z[e] > c.tz || (z[e] == c.tz && base + e < c.tt);
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (in) {
      const int to = c.cnt + __popc(who & ((1u << lane) - 1u));
      c.z[to] = z[e];
      c.tok[to] = base + e;
    }
    c.cnt += __popc(who);
  }
}

// One CTA per (row, span of its vocabulary): one read of the span's logits
// for the row's sum of exponentials and for its best K tokens.  The last CTA
// of a request picks its continuations.
template <typename T>
__global__ void __launch_bounds__(kBmThreads) beam_select_kernel(const BeamParams P) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float w_ref[kBmWarps], w_sum[kBmWarps];
  __shared__ int w_cnt[kBmWarps], w_at[kBmWarps + 1];
  __shared__ int is_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sp = blockIdx.x % P.spans, row = blockIdx.x / P.spans;
  const int b = row / P.W, K = P.keep;
  const float L = 1.4426950408889634f;
  float* cz = reinterpret_cast<float*>(smem);            // [warps][cap]
  int* ct = reinterpret_cast<int*>(cz + kBmWarps * kBmCap);
  const float cum = P.scores[row];
  const bool ended = P.finished && P.finished[row] != 0;
  if (!ended && cum > -INFINITY) {
    const int lo = sp * P.span, hi = min(P.V, lo + P.span);
    const T* z0 = static_cast<const T*>(P.logits) + (long long)row * P.ld;
    WarpCands c;
    c.z = cz + warp * kBmCap;
    c.tok = ct + warp * kBmCap;
    c.cnt = 0;
    c.tz = -INFINITY;
    c.tt = -1;
    // sum + low: the sum with its rounding errors, of 2^((z - ref) log2(e)).
    // The difference comes first: the lowest finite logits, a mask as a rule,
    // leave fp32's range when they are scaled.
    float ref = -INFINITY, sum = 0.f, low = 0.f;
    bool first = true;
    constexpr int STEP = kBmThreads * N * kBmUnroll;
    for (int at = lo; at < hi; at += STEP) {
      uint4 raw[kBmUnroll];
      int base[kBmUnroll];
#pragma unroll
      for (int u = 0; u < kBmUnroll; ++u) {
        base[u] = at + ((u * kBmWarps + warp) * 32 + lane) * N;
        if (base[u] < hi) raw[u] = __ldg(reinterpret_cast<const uint4*>(z0 + base[u]));
      }
      float z[kBmUnroll][N], mx[kBmUnroll];
#pragma unroll
      for (int u = 0; u < kBmUnroll; ++u) {
        if (base[u] < hi) {
          cvt16(raw[u], z[u]);
          if (base[u] + N > hi) {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (base[u] + e >= hi) z[u][e] = -INFINITY;
          }
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) z[u][e] = -INFINITY;
        }
        mx[u] = z[u][0];
#pragma unroll
        for (int e = 1; e < N; ++e) mx[u] = fmaxf(mx[u], z[u][e]);
      }
      float top = mx[0];
#pragma unroll
      for (int u = 1; u < kBmUnroll; ++u) top = fmaxf(top, mx[u]);
      if (first) {
        // The first vectors' 64 maxima of half a lane's tokens: K tokens are
        // at or above the K-th of them.
        float a = mx[0], d = mx[kBmUnroll / 2];
#pragma unroll
        for (int u = 1; u < kBmUnroll / 2; ++u) {
          a = fmaxf(a, mx[u]);
          d = fmaxf(d, mx[kBmUnroll / 2 + u]);
        }
        int ra = 0, rd = 0;
        for (int o = 0; o < 32; ++o) {
          const float x = __shfl_sync(0xffffffffu, a, o), y = __shfl_sync(0xffffffffu, d, o);
          ra += (x > a || (x == a && o < lane)) + (y > a);
          rd += (x >= d) + (y > d || (y == d && o < lane));
        }
        const unsigned wa = __ballot_sync(0xffffffffu, ra == K - 1), wd = __ballot_sync(0xffffffffu, rd == K - 1);
        if (wa)
          c.tz = __shfl_sync(0xffffffffu, a, __ffs(wa) - 1);
        else if (wd)
          c.tz = __shfl_sync(0xffffffffu, d, __ffs(wd) - 1);
        c.tt = c.tz > -INFINITY ? 0x7fffffff : -1;
        first = false;
      }
      // the reference moves at the first finite logit, and then only where
      // terms would come near fp32's range
      if (top > ref + 40.f) {
        const float f = ex2((ref - top) * L);
        sum *= f;
        low *= f;
        ref = top;
      }
      const float base_z = ref > -INFINITY ? ref : 0.f;
      const float2 L2 = make_float2(L, L), nr = make_float2(-base_z, -base_z);
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kBmUnroll; ++u)
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 y = __fmul2_rn(__fadd2_rn(make_float2(z[u][e], z[u][e + 1]), nr), L2);
          acc = __fadd2_rn(acc, make_float2(ex2(y.x), ex2(y.y)));
        }
      {
        const float x = acc.x + acc.y, s = sum + x, bb = s - sum;
        low += (sum - (s - bb)) + (x - bb);
        sum = s;
      }
#pragma unroll
      for (int u = 0; u < kBmUnroll; ++u)
        if (__any_sync(0xffffffffu, mx[u] >= c.tz && mx[u] > -INFINITY)) gather<N>(c, z[u], base[u], K, lane);
    }
    if (c.cnt > K) prune(c, K, lane);
    __syncwarp();
    const float wr = warp_max(ref);
    const float ws = warp_sum(ref > -INFINITY ? (sum + low) * ex2((ref - wr) * L) : sum);
    if (lane == 0) {
      w_ref[warp] = wr;
      w_sum[warp] = ws;
      w_cnt[warp] = c.cnt;
    }
    __syncthreads();
    if (tid == 0) {
      int s = 0;
      float M = w_ref[0], S = 0.f;
      for (int w = 0; w < kBmWarps; ++w) {
        w_at[w] = s;
        s += w_cnt[w];
        M = fmaxf(M, w_ref[w]);
      }
      w_at[kBmWarps] = s;
      for (int w = 0; w < kBmWarps; ++w) S += w_ref[w] > -INFINITY ? w_sum[w] * ex2((w_ref[w] - M) * L) : w_sum[w];
      __stcg(&P.stat[(long long)row * P.spans + sp], make_float4(M, S, S <= 3.4028235e38f ? 0.f : 1.f, 0.f));
    }
    __syncthreads();
    // the warps' candidates by rank
    const int n = w_at[kBmWarps];
    BeamCand* out = P.cand + ((long long)row * P.spans + sp) * K;
    for (int x = tid; x < kBmWarps * K; x += kBmThreads) {
      const int w = x / K, i = x - w * K;
      if (i >= w_cnt[w]) continue;
      const float z = cz[w * kBmCap + i];
      const int tok = ct[w * kBmCap + i];
      int rank = 0;
      for (int w2 = 0; w2 < kBmWarps; ++w2)
        for (int i2 = 0; i2 < w_cnt[w2]; ++i2) {
          const float z2 = cz[w2 * kBmCap + i2];
          rank += z2 > z || (z2 == z && ct[w2 * kBmCap + i2] < tok);
        }
      if (rank < K) __stcg(reinterpret_cast<int2*>(out + rank), make_int2(__float_as_int(z), tok));
    }
    for (int i = n + tid; i < K; i += kBmThreads)
      __stcg(reinterpret_cast<int2*>(out + i), make_int2(__float_as_int(-INFINITY), -1));
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) is_last = tagged_arrive(&P.counters[b], P.tag) == P.W * P.spans - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();

  // ---- the request's continuations, by the last CTA
  const int lists = P.W * P.spans;
  __shared__ double lse[kBeamMax];
  __shared__ int bad, n_got;
  __shared__ unsigned long long t_key;
  __shared__ int t_flat;
  unsigned long long* hk = reinterpret_cast<unsigned long long*>(smem);  // [lists] heads: order key, flat token
  int* hf = reinterpret_cast<int*>(hk + lists);
  unsigned long long* gk = reinterpret_cast<unsigned long long*>(smem + ((size_t)lists * 12 + 15) / 16 * 16);
  int* gf = reinterpret_cast<int*>(gk + K * K);
  if (tid == 0) {
    bad = 0;
    n_got = 0;
    t_key = 0;
    t_flat = 0x7fffffff;
  }
  __syncthreads();
  for (int w = warp; w < P.W; w += kBmWarps) {
    const float s0 = P.scores[b * P.W + w];
    const bool end = P.finished && P.finished[b * P.W + w] != 0;
    if (!(s0 < INFINITY)) bad = 1;
    if (end || !(s0 > -INFINITY)) continue;
    const float4* st = P.stat + (long long)(b * P.W + w) * P.spans;
    float M = -INFINITY;
    int off = 0;
    for (int i = lane; i < P.spans; i += 32) {
      const float4 v = __ldcg(st + i);
      off |= v.z != 0.f;
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
    M = warp_max(M);
    double S = 0.0;
    for (int i = lane; i < P.spans; i += 32) {
      const float4 v = __ldcg(st + i);
      if (v.y > 0.f) S += (double)v.y * exp2(((double)v.x - (double)M) * (double)L);
    }
    S = warp_sum_d(S);
    if (warp_or(off) && lane == 0) bad = 1;
    // an empty row has no reference (and no continuation)
    if (lane == 0) lse[w] = S > 0.0 ? (double)M + log2(S) / (double)L : 0.0;
  }
  __syncthreads();
  if (bad) {
    for (int i = tid; i < K; i += kBmThreads) {
      P.out_scores[b * K + i] = -INFINITY;
      P.out_parents[b * K + i] = -1;
      P.out_tokens[b * K + i] = -1;
    }
    if (tid == 0 && P.status) P.status[b] = kStatusBadLogits;
    return;
  }
  // The score of entry i of a list; key 0: none.  (A score's key is above 0.)
  auto entry = [&](int list, int i, int& flat) -> unsigned long long {
    const int w = list / P.spans;
    const float s0 = P.scores[b * P.W + w];
    flat = 0x7fffffff;
    if (!(s0 > -INFINITY)) return 0ull;
    if (P.finished && P.finished[b * P.W + w] != 0) {
      if (i > 0 || list != w * P.spans) return 0ull;
      flat = w * P.V + P.end_token;
      return double_key((double)s0);
    }
    const int2 v = __ldcg(reinterpret_cast<const int2*>(P.cand + ((long long)b * lists + list) * K + i));
    if (v.y < 0) return 0ull;
    flat = w * P.V + v.y;
    return double_key((double)s0 + ((double)__int_as_float(v.x) - lse[w]));
  };
  for (int i = tid; i < lists; i += kBmThreads) {
    int f;
    hk[i] = entry(i, 0, f);
    hf[i] = f;
  }
  __syncthreads();
  // K lists' heads are at or above the K-th best head, so no entry below it is kept
  for (int i = tid; i < lists; i += kBmThreads) {
    const unsigned long long k = hk[i];
    const int f = hf[i];
    if (k == 0ull) continue;
    int rank = 0;
    for (int x = 0; x < lists; ++x) rank += hk[x] > k || (hk[x] == k && hf[x] < f);
    if (rank == K - 1) {
      t_key = k;
      t_flat = f;
    }
  }
  __syncthreads();
  const unsigned long long tk = t_key;
  const int tf = t_flat;
  for (int x = tid; x < lists * K; x += kBmThreads) {
    const int list = x / K, i = x - list * K;
    const unsigned long long hk0 = hk[list];
    if (hk0 == 0ull || hk0 < tk || (hk0 == tk && hf[list] > tf)) continue;
    int f;
    const unsigned long long k = entry(list, i, f);
    if (k == 0ull || k < tk || (k == tk && f > tf)) continue;
    const int to = atomicAdd(&n_got, 1);  // at most K lists of K entries
    gk[to] = k;
    gf[to] = f;
  }
  __syncthreads();
  const int n = n_got;
  for (int x = tid; x < n; x += kBmThreads) {
    const unsigned long long k = gk[x];
    const int f = gf[x];
    int rank = 0;
    for (int y = 0; y < n; ++y) rank += gk[y] > k || (gk[y] == k && gf[y] < f);
    if (rank < K) {
      P.out_scores[b * K + rank] = (float)key_double(k);
      P.out_parents[b * K + rank] = f / P.V;
      P.out_tokens[b * K + rank] = f % P.V;
    }
  }
  for (int i = n + tid; i < K; i += kBmThreads) {
    P.out_scores[b * K + i] = -INFINITY;
    P.out_parents[b * K + i] = -1;
    P.out_tokens[b * K + i] = -1;
  }
  if (tid == 0 && P.status) P.status[b] = 0;
}

size_t beam_smem(const BeamParams& P) {
  const size_t lists = (size_t)P.W * P.spans;
  const size_t a = (size_t)kBmWarps * kBmCap * 8;
  const size_t m = (lists * 12 + 15) / 16 * 16 + (size_t)P.keep * P.keep * 12;
  return a > m ? a : m;
}

// ---------------------------------------------------------- reordering
constexpr int kRoThreads = 256;
constexpr int kRoPer = 4;  // accesses per thread

template <typename U>
__device__ __forceinline__ void copy_units(unsigned char* dst, const unsigned char* src, long long n, long long at) {
  U v[kRoPer];
#pragma unroll
  for (int i = 0; i < kRoPer; ++i) {
    const long long x = at + (long long)i * kRoThreads;
    if (x < n && src) v[i] = reinterpret_cast<const U*>(src)[x];
    if (!src) v[i] = U{};
  }
#pragma unroll
  for (int i = 0; i < kRoPer; ++i) {
    const long long x = at + (long long)i * kRoThreads;
    if (x < n) reinterpret_cast<U*>(dst)[x] = v[i];
  }
}

__global__ void __launch_bounds__(kRoThreads) beam_reorder_kernel(const ReorderParams P) {
  int k = 0;
  while (k + 1 < P.num && (long long)blockIdx.x >= P.s[k + 1].first) ++k;
  const BeamState& s = P.s[k];
  const long long x = (long long)blockIdx.x - s.first;
  const long long row = x / s.blocks;
  const int part = (int)(x - row * s.blocks);
  const int j = (int)(row % P.keep), b = (int)(row / P.keep % P.B), o = (int)(row / ((long long)P.keep * P.B));
  const int parent = P.parents[b * P.keep + j];
  const unsigned char* src = parent >= 0 && parent < P.W
                                 ? s.src + o * s.src_outer + b * s.src_batch + parent * s.src_beam
                                 : nullptr;
  unsigned char* dst = s.dst + o * s.dst_outer + b * s.dst_batch + j * s.dst_beam;
  const long long n = s.row_bytes / s.unit, at = (long long)part * kRoThreads * kRoPer + threadIdx.x;
  switch (s.unit) {
    case 16: copy_units<uint4>(dst, src, n, at); break;
    case 8: copy_units<uint2>(dst, src, n, at); break;
    case 4: copy_units<uint32_t>(dst, src, n, at); break;
    case 2: copy_units<uint16_t>(dst, src, n, at); break;
    default: copy_units<uint8_t>(dst, src, n, at); break;
  }
}

}  // namespace

// Spans of a row: enough CTAs to fill the device a few times over, each with
// at least one step of every thread.
int beam_spans(int rows, int V, int num_sms) {
  const int step = kBmThreads * 8 * kBmUnroll;
  const int want = (4 * num_sms + rows - 1) / rows, most = (V + step - 1) / step;
  return want < most ? want : most;
}

int beam_smem_bytes(int W, int spans, int keep) {
  BeamParams P{};
  P.W = W;
  P.spans = spans;
  P.keep = keep;
  return (int)beam_smem(P);
}

int launch_beam_select(const BeamParams& P, bool bf16, cudaStream_t s) {
  const int bytes = (int)beam_smem(P);
  const unsigned grid = (unsigned)((long long)P.B * P.W * P.spans);
  const void* f = bf16 ? (const void*)beam_select_kernel<__nv_bfloat16> : (const void*)beam_select_kernel<float>;
  if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (bf16)
    beam_select_kernel<__nv_bfloat16><<<grid, kBmThreads, bytes, s>>>(P);
  else
    beam_select_kernel<float><<<grid, kBmThreads, bytes, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

// Fills the work split of P's states and returns the number of blocks.
long long plan_reorder(ReorderParams& P) {
  long long at = 0;
  for (int k = 0; k < P.num; ++k) {
    BeamState& s = P.s[k];
    const long long n = s.row_bytes / s.unit, per = kRoThreads * kRoPer;
    s.blocks = (int)((n + per - 1) / per);
    s.first = at;
    at += (long long)s.blocks * s.outer * P.B * P.keep;
  }
  return at;
}

int launch_beam_reorder(const ReorderParams& P, long long blocks, cudaStream_t s) {
  beam_reorder_kernel<<<(unsigned)blocks, kRoThreads, 0, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace sv
