// Beam selection over beams and vocabulary, and the beams' states in their
// new order.
#include "stream_common.cuh"
#include "tree_internal.h"
#include "tree_launch.cuh"

namespace sv {
namespace {

constexpr int kBmThreads = 256;
constexpr int kBmWarps = kBmThreads / 32;
// 16-byte loads of a lane in a chunk, and CTAs per SM.  64 x 8 beams over
// 152064 bf16 logits and one request of 4 over 151936, with reordering, us:
//   loads 4: one CTA 63 and 14.3, two 49 and 15.2, three 53 and 15.5, four 56 and 16.4;
//   two CTAs: 2 loads 57 and 15.1, 8 loads 54 and 16.5.
constexpr int kBmUnroll = 4;
constexpr int kBmCtas = 2;
constexpr int kBmCap = 2048;      // candidates of a request in shared memory
constexpr int kBmHot = 1024;      // chunks that may hold candidates
constexpr float kBmBad = 1.f, kBmLowest = 2.f;  // a piece's flags: no number, nothing but masks
constexpr int kBeamRows = 2048;   // rows up to which those that are read are counted

// A chunk is what a warp reads at once (1024 bf16 or 512 fp32 logits); a step
// of a CTA is a chunk for each warp.
template <typename T>
struct BmShape {
  static constexpr int N = Vec<T>::N;
  static constexpr int kChunk = 32 * N * kBmUnroll;
  static constexpr int kStep = kBmWarps * kChunk;
};

// Unsigned order of a float's value (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t float_key(float z) {
  const uint32_t u = __float_as_uint(z == 0.f ? 0.f : z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long double_key(double z) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(z == 0.0 ? 0.0 : z);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_double(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// 2^d for a whole d <= 0 (0 below fp32's normal range).
__device__ __forceinline__ float pow2_int(float d) { return d > -127.f ? __int_as_float(((int)d + 127) << 23) : 0.f; }

// The largest of kBmUnroll vectors' values (NaN passed over).
template <typename T>
__device__ __forceinline__ float max_of(const uint4 (&v)[kBmUnroll]);
template <>
__device__ __forceinline__ float max_of<float>(const uint4 (&v)[kBmUnroll]) {
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < kBmUnroll; ++u) {
    m = fmaxf(fmaxf(m, __uint_as_float(v[u].x)), __uint_as_float(v[u].y));
    m = fmaxf(fmaxf(m, __uint_as_float(v[u].z)), __uint_as_float(v[u].w));
  }
  return m;
}
template <>
__device__ __forceinline__ float max_of<__nv_bfloat16>(const uint4 (&v)[kBmUnroll]) {
  auto pair = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
  __nv_bfloat162 m = __hmax2(pair(v[0].x), pair(v[0].y));
  m = __hmax2(m, __hmax2(pair(v[0].z), pair(v[0].w)));
#pragma unroll
  for (int u = 1; u < kBmUnroll; ++u) {
    m = __hmax2(m, __hmax2(pair(v[u].x), pair(v[u].y)));
    m = __hmax2(m, __hmax2(pair(v[u].z), pair(v[u].w)));
  }
  const float a = __low2float(m), b = __high2float(m);
  return fmaxf(fmaxf(a, b), -INFINITY);  // NaN where all are
}

// A vector at the end of a span: -inf past it.
template <typename T>
__device__ __forceinline__ uint4 load_tail(const T* z, int at, int hi) {
  constexpr int N = Vec<T>::N;
  const T none = neg_inf<T>();
  __align__(16) T x[N];
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = none;
  uint4 v = *reinterpret_cast<const uint4*>(x);
  if (at < hi) {
    v = load16(z + at);
    if (at + N > hi) {
      *reinterpret_cast<uint4*>(x) = v;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (at + e >= hi) x[e] = none;
      v = *reinterpret_cast<const uint4*>(x);
    }
  }
  return v;
}

// A value with at least K of the CTA's 256 values at or above it, and not many
// more than K where that is quickly found; -inf where fewer are finite.  Any
// such value does: a bisection over the 32 below the largest, where scores
// lie as a rule, and over all floats' order where too few do.
__device__ __forceinline__ float kth_bound(const float* vals, int K, int lane) {
  float v[kBmThreads / 32];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBmThreads / 32; ++i) {
    v[i] = vals[i * 32 + lane];
    top = fmaxf(top, v[i]);
  }
  top = key_float(__reduce_max_sync(0xffffffffu, float_key(top)));
  auto count = [&](float x) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kBmThreads / 32; ++i) n += v[i] >= x;
    return __reduce_add_sync(0xffffffffu, n);
  };
  if (!(top > -INFINITY)) return -INFINITY;
  float lo = top - 32.f, hi = top;
  int n = count(lo);
  if (n >= K) {
#pragma unroll 1
    for (int i = 0; i < 12 && n > K + K / 2; ++i) {
      const float mid = 0.5f * (lo + hi);
      const int m = count(mid);
      if (m >= K) {
        lo = mid;
        n = m;
      } else {
        hi = mid;
      }
    }
    return lo;
  }
  uint32_t t = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t probe = t | (1u << bit);
    const float x = key_float(probe);
    if (x > -INFINITY && count(x) >= K) t = probe;
    if (!(x > -INFINITY)) t = probe;  // -inf and below: everything
  }
  return t > 0u ? key_float(t) : -INFINITY;
}

// ---- the split of all rows' logits over the CTAs
// A row that is read (its beam has not ended and is alive) has `steps` steps.
// All steps of all such rows, in order, are cut evenly over the CTAs; a row's
// piece in a CTA has a record of its sum, and each of its chunks its maximum.
// With more than kBeamRows rows, rows that need not be read keep their places
// in the split and are passed over.
struct BeamSplit {
  const int* rows;   // the rows that are read, or null: all
  int n;             // how many
  int steps, used;   // steps per row, CTAs in use
  long long total;
  bool small;        // (total + 1) * (used + 1) fits 32 bits, whose divisions are much faster
  __device__ __forceinline__ int row(int a) const { return rows ? rows[a] : a; }
  __device__ __forceinline__ long long begin(int c) const {
    return small ? (long long)((uint32_t)total * (uint32_t)c / (uint32_t)used) : total * c / used;
  }
  __device__ __forceinline__ int owner(long long x) const {
    return small ? (int)(((uint32_t)(x + 1) * (uint32_t)used + (uint32_t)total - 1u) / (uint32_t)total) - 1
                 : (int)(((x + 1) * used + total - 1) / total - 1);
  }
  __device__ __forceinline__ int first_cta(int a) const { return owner((long long)a * steps); }
  __device__ __forceinline__ int pieces(int a) const { return owner((long long)(a + 1) * steps - 1) - first_cta(a) + 1; }
  // the record of place a's piece in a CTA, `per` of which a CTA has
  __device__ __forceinline__ int record(int cta, int a, int per) const { return cta * per + a - (int)((uint32_t)begin(cta) / (uint32_t)steps); }
};

__device__ __forceinline__ bool beam_read(const BeamParams& P, int row) {
  return P.scores[row] > -INFINITY && !(P.finished && P.finished[row] != 0);
}

struct BeamShared {
  float w_ref[kBmWarps], w_sum[kBmWarps], w_top[kBmWarps];
  int w_cnt[kBmWarps], w_cnt2[2][kBmWarps];
  float t_max[kBmThreads];
  int is_last, bad, n_got, n_hot, over;
  int place[kBeamMax];                       // of each row of the request in the split, -1: not read
  int pieces[kBeamMax];
  double lse[kBeamMax], row_sum[kBeamMax];
  float row_ref[kBeamMax], row_top[kBeamMax], s0[kBeamMax], add[kBeamMax], err[kBeamMax], z_min[kBeamMax];
  int row_low[kBeamMax];
  unsigned long long best_key[kBeamMax];     // the best K, in order
  int best_flat[kBeamMax];
};

// A row's tokens [lo, hi) in a CTA.
struct BeamPiece {
  int a, row, lo, hi;  // place in the split, row
};

// The loads of a warp's chunk at token x (of this lane) of a piece.
template <typename T>
__device__ __forceinline__ void beam_fetch(const BeamParams& P, const BeamPiece& p, int x, uint4 (&v)[kBmUnroll]) {
  constexpr int N = BmShape<T>::N;
  const T* z0 = static_cast<const T*>(P.logits) + (long long)p.row * P.ld;
  if (x + (kBmUnroll - 1) * 32 * N + N <= p.hi) {
#pragma unroll
    for (int u = 0; u < kBmUnroll; ++u) v[u] = load16(z0 + x + u * 32 * N);
  } else {
#pragma unroll 1
    for (int u = 0; u < kBmUnroll; ++u) {
      const uint4 t = load_tail<T>(z0, x + u * 32 * N, p.hi);
#pragma unroll
      for (int i = 0; i < kBmUnroll; ++i)
        if (i == u) v[i] = t;
    }
  }
}

// The sum and the chunks' maxima of a piece, whose first loads are in `next`;
// the first loads of the piece after it are left there.
template <typename T>
__device__ __forceinline__ void beam_piece(const BeamParams& P, BeamShared& sh, const BeamPiece& p,
                                           const BeamPiece& after, uint4 (&next)[kBmUnroll], float4* stat) {
  const int row = p.row, lo = p.lo, hi = p.hi;
  using S = BmShape<T>;
  constexpr int N = S::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float L = 1.4426950408889634f;
  const T* z0 = static_cast<const T*>(P.logits) + (long long)row * P.ld;
  float* maxima = P.maxima + (long long)row * P.chunks;
  // sum + low: the sum with its rounding errors, of 2^(z log2(e) - ref).
  // References are whole numbers, so that sums move to another one exactly.
  float ref = -INFINITY, sum = 0.f, low = 0.f, best = -INFINITY;
  int at = lo + warp * S::kChunk + lane * N;
  for (int first = lo + warp * S::kChunk; first < hi; first += S::kStep, at += S::kStep) {  // warp-uniform
    uint4 raw[kBmUnroll];
#pragma unroll
    for (int u = 0; u < kBmUnroll; ++u) raw[u] = next[u];
    beam_fetch<T>(P, p, at + S::kStep, next);
    const float top = max_of<T>(raw);
    const uint32_t key = __reduce_max_sync(0xffffffffu, float_key(top));
    if (lane == 0) __stcg(maxima + first / S::kChunk, key_float(key));
    best = fmaxf(best, top);
    // The reference moves at the first finite logit, and then where a lane's
    // maximum has passed it by more than 2^4: an exponent of up to 4 is rounded
    // by 2^-23 at most, and the terms that matter by as little.
    if (top * L > ref + 4.f) {
      const float to = ceilf(top * L), f = pow2_int(ref - to);
      sum *= f;
      low *= f;
      ref = to;
    }
    const float back = ref > -INFINITY ? -ref : 0.f;
    const float2 L2 = make_float2(L, L), nr = make_float2(back, back);
    float2 acc = make_float2(0.f, 0.f), acc2 = acc;
#pragma unroll
    for (int u = 0; u < kBmUnroll; ++u) {
      float z[N];
      cvt16(raw[u], z);
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float2 y = __ffma2_rn(make_float2(z[e], z[e + 1]), L2, nr);
        const float2 y2 = __ffma2_rn(make_float2(z[e + 2], z[e + 3]), L2, nr);
        acc = __fadd2_rn(acc, make_float2(ex2(y.x), ex2(y.y)));
        acc2 = __fadd2_rn(acc2, make_float2(ex2(y2.x), ex2(y2.y)));
      }
    }
    const float x = (acc.x + acc.y) + (acc2.x + acc2.y), s = sum + x, bb = s - sum;
    low += (sum - (s - bb)) + (x - bb);
    sum = s;
  }
  beam_fetch<T>(P, after, after.lo + warp * S::kChunk + lane * N, next);
  best = warp_max(best);
  if (lane == 0) sh.w_top[warp] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBmWarps; ++w) best = fmaxf(best, sh.w_top[w]);
  // A piece of nothing but the lowest finite logits (masks): scaled, they
  // leave fp32's range, so they are summed again relative to their maximum.
  const bool lowest = best > -INFINITY && best * L == -INFINITY;
  if (lowest) {
    ref = 0.f;
    sum = low = 0.f;
    for (int v = lo + tid; v < hi; v += kBmThreads) sum += ex2((to_f32<T>(z0[v]) - best) * L);
  }
  const float wr = warp_max(ref);
  const float ws = warp_sum(ref > -INFINITY ? (sum + low) * pow2_int(ref - wr) : sum);
  if (lane == 0) {
    sh.w_ref[warp] = wr;
    sh.w_sum[warp] = ws;
  }
  __syncthreads();
  if (tid == 0) {
    float M = sh.w_ref[0], sum_all = 0.f;
    for (int w = 1; w < kBmWarps; ++w) M = fmaxf(M, sh.w_ref[w]);
    for (int w = 0; w < kBmWarps; ++w)
      sum_all += sh.w_ref[w] > -INFINITY ? sh.w_sum[w] * pow2_int(sh.w_ref[w] - M) : sh.w_sum[w];
    const float flags = (sum_all <= 3.4028235e38f ? 0.f : kBmBad) + (lowest ? kBmLowest : 0.f);
    __stcg(stat, make_float4(lowest ? best : M, sum_all, flags, best));
  }
}

// As tagged_arrive, by `n` at once.
__device__ __forceinline__ int tagged_add(unsigned long long* ctr, unsigned long long tag, int n) {
  const unsigned long long v = *reinterpret_cast<volatile unsigned long long*>(ctr);
  if ((v >> kTagShift) != tag) atomicCAS(ctr, v, tag << kTagShift);
  return (int)(atomicAdd(ctr, (unsigned long long)n) & ((1ull << kTagShift) - 1ull));
}

// The request's candidates in shared memory.
struct BeamPool {
  unsigned long long* key;
  int* flat;
  int* hot;   // chunks
};

// Leaves the best K of the pool's n > K candidates, in any order: bisections
// over the scores' order keys and, among equals of the K-th, over places.
__device__ __noinline__ void beam_cut(BeamShared& sh, BeamPool pool, int n, int K) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int PER = kBmCap / kBmThreads;
  unsigned long long key[PER];
  int flat[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int x = i * kBmThreads + tid;
    key[i] = x < n ? pool.key[x] : 0ull;  // below every score's
    flat[i] = x < n ? pool.flat[x] : 0x7fffffff;
  }
  int buf = 0;
  auto total = [&](int v) {  // over the CTA
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) sh.w_cnt2[buf][warp] = v;
    __syncthreads();
    v = __reduce_add_sync(0xffffffffu, lane < kBmWarps ? sh.w_cnt2[buf][lane] : 0);
    buf ^= 1;
    return v;
  };
  unsigned long long t = 0ull;  // the K-th best key
  int at = n;
#pragma unroll 1
  for (int bit = 63; bit >= 0 && at != K; --bit) {
    const unsigned long long probe = t | (1ull << bit);
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += key[i] >= probe;
    c = total(c);
    if (c >= K) {
      t = probe;
      at = c;
    }
  }
  int last = 0x7fffffff;  // the last place of an equal that stays
  if (at != K) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += key[i] > t;
    const int need = K - total(c);
    last = 0;
#pragma unroll 1
    for (int bit = 30; bit >= 0; --bit) {
      const int probe = last | (1 << bit);
      c = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) c += key[i] == t && flat[i] < probe;
      if (total(c) < need) last = probe;
    }
  }
  if (tid == 0) sh.n_got = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (key[i] > t || (key[i] == t && key[i] != 0ull && flat[i] <= last)) {
      const int to = atomicAdd(&sh.n_got, 1);
      pool.key[to] = key[i];
      pool.flat[to] = flat[i];
    }
  __syncthreads();
}

// The best K of the pool's n candidates, in order, to sh.best.
__device__ __forceinline__ void beam_best(BeamShared& sh, const BeamPool& pool, int n, int K) {
  if (n > kBmThreads) {
    beam_cut(sh, pool, n, K);
    n = K;
  }
  const int x = threadIdx.x;
  if (x < n) {
    const unsigned long long k = pool.key[x];
    const int f = pool.flat[x];
    int rank = 0;
#pragma unroll 4
    for (int y = 0; y < n; ++y) rank += pool.key[y] > k || (pool.key[y] == k && pool.flat[y] < f);
    if (rank < K) {
      sh.best_key[rank] = k;
      sh.best_flat[rank] = f;
    }
  }
  __syncthreads();
}

// A request's continuations; sh.place and sh.pieces are set.
//
// A chunk's maximum gives its best score.  Each thread keeps the best of its
// share of chunks; the K-th best of these 256 bounds the K-th continuation
// from below, so only chunks at or above it (about K) are read once more.
template <typename T>
__device__ __forceinline__ void beam_finish(const BeamParams& P, BeamShared& sh, unsigned char* smem,
                                            const BeamSplit& sp, int b) {
  using S = BmShape<T>;
  constexpr int N = S::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = P.keep;
  const float L = 1.4426950408889634f;
  BeamPool pool;
  pool.key = reinterpret_cast<unsigned long long*>(smem);
  pool.flat = reinterpret_cast<int*>(pool.key + kBmCap);
  pool.hot = pool.flat + kBmCap;
  if (tid == 0) sh.bad = sh.n_got = sh.n_hot = sh.over = 0;
  // Chunks by thread in turn, eight loads at once; the first eight stay.
  const float* maxima = P.maxima + (long long)b * P.W * P.chunks;
  constexpr int HELD = 8;
  const int n_chunk = P.W * P.chunks;
  float held[HELD];
  // a chunk's row: exact, as a request has fewer than 2^22 chunks
  const float inv_chunks = 1.f / (float)P.chunks;
  auto row_of = [&](int id) { return (int)(((float)id + 0.5f) * inv_chunks); };
  auto fetch = [&](int from, float (&m)[HELD]) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int id = from + i * kBmThreads;
      m[i] = id < n_chunk && sh.place[row_of(id)] >= 0 ? __ldcg(maxima + id) : -INFINITY;
    }
  };
  fetch(tid, held);
  __syncthreads();
  // the rows' sums, by 8 lanes each
#pragma unroll 1
  for (int first = 0; first < P.W; first += kBmThreads / 8) {
    const int w = first + tid / 8, sub = tid & 7;
    const bool in = w < P.W;
    const float s0 = in ? P.scores[b * P.W + w] : 0.f;
    const int a = in ? sh.place[w] : -1, n = a >= 0 ? sh.pieces[w] : 0, cta = a >= 0 ? sp.first_cta(a) : 0;
    // sums of whole references, and of masks alone
    float M = -INFINITY, M_low = -INFINITY, top = -INFINITY;
    double sum = 0.0, sum_low = 0.0;
    int off = !(s0 < INFINITY);
#pragma unroll 1
    for (int i = sub; i < n; i += 32) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = i + 8 * j < n ? __ldcg(P.stat + sp.record(cta + i + 8 * j, a, P.spans)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        off |= v[j].z == kBmBad || v[j].z == kBmBad + kBmLowest;
        if (!(v[j].y > 0.f)) continue;
        top = fmaxf(top, v[j].w);
        if (v[j].z < kBmLowest) {
          const float to = fmaxf(M, v[j].x);
          sum = sum * (double)pow2_int(M - to) + (double)(v[j].y * pow2_int(v[j].x - to));
          M = to;
        } else {
          const float to = fmaxf(M_low, v[j].x);
          sum_low = sum_low * (double)ex2((M_low - to) * L) + (double)(v[j].y * ex2((v[j].x - to) * L));
          M_low = to;
        }
      }
    }
    float M_all = M, low_all = M_low;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      M_all = fmaxf(M_all, __shfl_xor_sync(0xffffffffu, M_all, o));
      low_all = fmaxf(low_all, __shfl_xor_sync(0xffffffffu, low_all, o));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const bool low_row = !(M_all > -INFINITY);  // nothing but the lowest logits
    if (low_row)
      sum = M_low > -INFINITY ? sum_low * (double)ex2((M_low - low_all) * L) : 0.0;
    else
      sum = M > -INFINITY ? sum * (double)pow2_int(M - M_all) : 0.0;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (off) sh.bad = 1;
    if (in && sub == 0) {
      sh.s0[w] = s0;
      sh.row_sum[w] = sum;
      sh.row_ref[w] = low_row ? low_all : M_all;
      sh.row_low[w] = low_row;
      sh.row_top[w] = top;
    }
  }
  __syncthreads();
  // log2 of a sum: its exponent, log2f of its fp32 fraction in [1, 2) (off by
  // 2^-24 at most) and the fraction's rounding.  log2(e) is the fp32 constant
  // by which logits were scaled; an empty row has no sum (and no
  // continuation).  In fp32 a score is z + add, off by less than err plus
  // 2^-22 |z|.
  for (int w = tid; w < P.W; w += kBmThreads) {
    double l2 = 0.0;
    if (sh.row_sum[w] > 0.0) {
      const long long bits = __double_as_longlong(sh.row_sum[w]);
      const double m = __longlong_as_double((bits & 0x000fffffffffffffll) | 0x3ff0000000000000ll);
      const float mf = (float)m;
      l2 = (double)((int)(bits >> 52) - 1023) + (double)log2f(mf) + (double)((float)(m - (double)mf) / mf * L);
    }
    constexpr double inv = 1.0 / 1.4426950216293335;  // of that constant
    // It is the largest logit at least, and is that logit where the sum is its
    // term alone, computed as there (its lane's reference moved to it): one
    // allowed token leaves a beam's score as it is.
    const float top = sh.row_top[w];
    double lse = sh.row_low[w] ? (double)sh.row_ref[w] + l2 * inv : ((double)sh.row_ref[w] + l2) * inv;
    const bool alone = !sh.row_low[w] && sh.row_sum[w] == (double)ex2(fmaf(top, L, -sh.row_ref[w]));
    if (alone || lse < (double)top) lse = (double)top;
    const float s0 = sh.s0[w];
    sh.lse[w] = lse;
    sh.add[w] = (float)((double)s0 - lse);
    sh.err[w] = 4.8e-7f * fabsf((float)((double)s0 - lse));
  }
  __syncthreads();
  if (sh.bad) {
    for (int i = tid; i < K; i += kBmThreads) {
      P.out_scores[b * K + i] = -INFINITY;
      P.out_parents[b * K + i] = -1;
      P.out_tokens[b * K + i] = -1;
    }
    if (tid == 0 && P.status) P.status[b] = kStatusBadLogits;
    return;
  }
  float best = -INFINITY;
  auto take = [&](int from, const float (&m)[HELD]) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (m[i] > -INFINITY) {
        const int w = row_of(from + i * kBmThreads);
        best = fmaxf(best, (m[i] + sh.add[w]) - (sh.err[w] + 2.4e-7f * fabsf(m[i])));
      }
  };
  take(tid, held);
  for (int from = tid + HELD * kBmThreads; from < n_chunk; from += HELD * kBmThreads) {
    float m[HELD];
    fetch(from, m);
    take(from, m);
  }
  sh.t_max[tid] = best;
  __syncthreads();
  const float floor = kth_bound(sh.t_max, K, lane);
  // from below, what a logit of each row has to be to score `floor`
  for (int w = tid; w < P.W; w += kBmThreads) {
    const float z = floor - sh.add[w];
    sh.z_min[w] = z - (sh.err[w] + 4.8e-7f * (fabsf(z) + fabsf(floor)));
  }
  __syncthreads();
  for (int w = tid; w < P.W; w += kBmThreads) {  // an ended beam goes on as it is
    if (sh.place[w] < 0 && sh.s0[w] > -INFINITY && P.finished && P.finished[b * P.W + w] != 0) {
      const int to = atomicAdd(&sh.n_got, 1);
      pool.key[to] = double_key((double)sh.s0[w]);
      pool.flat[to] = w * P.V + P.end_token;
    }
  }
  auto mark = [&](int from, const float (&m)[HELD]) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (m[i] > -INFINITY && m[i] >= sh.z_min[row_of(from + i * kBmThreads)]) {
        const int to = atomicAdd(&sh.n_hot, 1);
        if (to < kBmHot) pool.hot[to] = from + i * kBmThreads;
      }
  };
  mark(tid, held);
  for (int from = tid + HELD * kBmThreads; from < n_chunk; from += HELD * kBmThreads) {
    float m[HELD];
    fetch(from, m);
    mark(from, m);
  }
  __syncthreads();
  const int n_hot = sh.n_hot, n_ended = sh.n_got;
  __syncthreads();
  const T* logits = static_cast<const T*>(P.logits) + (long long)b * P.W * P.ld;
  // adds a chunk's u-th vector's tokens at or above their row's z_min and the
  // bound (tk, tf); the code is run once by a CTA, so it is kept short
  unsigned long long tk = 0ull;
  int tf = 0x7fffffff;
  auto add_vector = [&](int w, int tok, const uint4& raw) {
    float z[N];
    cvt16(raw, z);
    unsigned in = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) in |= (z[e] >= sh.z_min[w] && z[e] > -INFINITY ? 1u : 0u) << e;
    while (in) {
      const int t = tok + __ffs(in) - 1;
      in &= in - 1;
      const double zt = (double)to_f32<T>(logits[(long long)w * P.ld + t]);
      const unsigned long long k = double_key((double)sh.s0[w] + (zt - sh.lse[w]));
      const int f = w * P.V + t;
      if (k < tk || (k == tk && f > tf)) continue;
      const int to = atomicAdd(&sh.n_got, 1);
      if (to >= kBmCap) {
        sh.over = 1;
      } else {
        pool.key[to] = k;
        pool.flat[to] = f;
      }
    }
  };
  if (n_hot <= kBmHot && (n_chunk < 8 * K || n_hot > 2 * K + 16)) {
    // Few chunks (a short vocabulary) bound the K-th best loosely or not at
    // all: the same by threads' maxima over the tokens of these chunks.
    best = -INFINITY;
#pragma unroll 1
    for (int i = warp; i < n_hot * kBmUnroll; i += kBmWarps) {
      const int id = pool.hot[i / kBmUnroll], w = row_of(id);
      const int tok = (id - w * P.chunks) * S::kChunk + (i % kBmUnroll * 32 + lane) * N;
      float z[N];
      cvt16(load_tail<T>(logits + (long long)w * P.ld, tok, P.V), z);
      float top = z[0];
#pragma unroll
      for (int e = 1; e < N; ++e) top = fmaxf(top, z[e]);
      if (top > -INFINITY) best = fmaxf(best, (top + sh.add[w]) - (sh.err[w] + 2.4e-7f * fabsf(top)));
    }
    sh.t_max[tid] = best;
    __syncthreads();
    const float floor2 = kth_bound(sh.t_max, K, lane);
    for (int w = tid; w < P.W; w += kBmThreads) {
      const float z = floor2 - sh.add[w];
      sh.z_min[w] = fmaxf(sh.z_min[w], z - (sh.err[w] + 4.8e-7f * (fabsf(z) + fabsf(floor2))));
    }
    __syncthreads();
  }
  if (n_hot <= kBmHot) {
    uint4 ahead[kBmUnroll];
    int w_next = 0, tok_next = 0;
    auto chunk = [&](int i) {  // the loads of the i-th
      if (i >= n_hot) return;
      const int id = pool.hot[i];
      BeamPiece p;
      w_next = row_of(id);
      tok_next = (id - w_next * P.chunks) * S::kChunk + lane * N;
      p.row = b * P.W + w_next;
      p.hi = P.V;
      beam_fetch<T>(P, p, tok_next, ahead);
    };
    chunk(warp);
#pragma unroll 1
    for (int i = warp; i < n_hot; i += kBmWarps) {
      uint4 v[kBmUnroll];
#pragma unroll
      for (int u = 0; u < kBmUnroll; ++u) v[u] = ahead[u];
      const int w = w_next, tok = tok_next;
      chunk(i + kBmWarps);
#pragma unroll 1
      for (int u = 0; u < kBmUnroll; ++u) {
        add_vector(w, tok + u * 32 * N, v[0]);
#pragma unroll
        for (int j = 0; j + 1 < kBmUnroll; ++j) v[j] = v[j + 1];
      }
    }
  } else if (tid == 0) {
    sh.over = 1;
  }
  __syncthreads();
  int n = min(sh.n_got, kBmCap);
  if (sh.over) {
    // Too many at the bound (long runs of equal logits): chunk by chunk in
    // order, with the K-th best so far as the bound, ties by place.
    __syncthreads();
    if (tid == 0) {
      sh.n_got = n_ended;
      sh.over = 0;
    }
    __syncthreads();
    n = n_ended;
    // whether a chunk may hold a token that beats the bound
    auto may = [&](int id, float m) {
      const int w = row_of(id);
      if (!(m > -INFINITY && m >= sh.z_min[w])) return false;
      const unsigned long long k = double_key((double)sh.s0[w] + ((double)m - sh.lse[w]));
      return k > tk || (k == tk && w * P.V + (id - w * P.chunks) * S::kChunk <= tf);
    };
#pragma unroll 1
    for (int base = 0; base < n_chunk; base += kBmThreads) {
      const int mine = base + tid;
      const float m = mine < n_chunk && sh.place[row_of(mine)] >= 0 ? __ldcg(maxima + mine) : -INFINITY;
      const bool go = m > -INFINITY && may(mine, m);
      sh.t_max[tid] = go ? m : -INFINITY;
      if (__syncthreads_count(go) == 0) continue;
#pragma unroll 1
      for (int i = 0; i < kBmThreads; ++i) {
        if (sh.t_max[i] == -INFINITY || !may(base + i, sh.t_max[i])) continue;  // the same for all threads
        const int id = base + i, w = row_of(id);
        if (warp < kBmUnroll) {  // at most kBmCap - kChunk candidates before
          const int tok = (id - w * P.chunks) * S::kChunk + (warp * 32 + lane) * N;
          add_vector(w, tok, load_tail<T>(logits + (long long)w * P.ld, tok, P.V));
        }
        __syncthreads();
        n = sh.n_got;
        __syncthreads();
        if (n > kBmCap - S::kChunk) {
          beam_best(sh, pool, n, K);
          for (int x = tid; x < K; x += kBmThreads) {
            pool.key[x] = sh.best_key[x];
            pool.flat[x] = sh.best_flat[x];
          }
          tk = sh.best_key[K - 1];
          tf = sh.best_flat[K - 1];
          if (tid == 0) sh.n_got = K;
          __syncthreads();
          n = K;
        }
      }
      __syncthreads();
    }
  }
  beam_best(sh, pool, n, K);
  for (int i = tid; i < K; i += kBmThreads) {
    const bool in = i < n;
    P.out_scores[b * K + i] = in ? (float)key_double(sh.best_key[i]) : -INFINITY;
    P.out_parents[b * K + i] = in ? sh.best_flat[i] / P.V : -1;
    P.out_tokens[b * K + i] = in ? sh.best_flat[i] % P.V : -1;
  }
  if (tid == 0 && P.status) P.status[b] = 0;
}

// One wave of CTAs, each with an even share of all logits that are read; the
// last CTA of a request to arrive picks its continuations.
//
// 64 x 8 beams over 152064 bf16 logits, 156 MB: 46 us, and 49 with the beams'
// states.  Without the continuations, dependent trips to L2 by one CTA a
// request, 37; of these without exponentials 36.4, without any sums 35.8, and
// then with twice as many loads in flight 34.2: the stream is bound by its loads
// in flight, its start and its end, not by what it computes.  4 beams of one
// request: 15 us, latency.
template <typename T>
__global__ void __launch_bounds__(kBmThreads, kBmCtas) beam_select_kernel(const BeamParams P) {
  using S = BmShape<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BeamShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = P.B * P.W;
  after_previous();
  BeamSplit sp;
  sp.steps = (P.V + S::kStep - 1) / S::kStep;
  if (R <= kBeamRows) {
    int* rows = reinterpret_cast<int*>(smem + kBmCap * 12 + kBmHot * 4);
    int n = 0;
    for (int base = 0; base < R; base += kBmThreads) {
      const int r = base + tid;
      const bool in = r < R && beam_read(P, r);
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (lane == 0) sh.w_cnt[warp] = __popc(who);
      __syncthreads();
      int at = n;
      for (int w = 0; w < kBmWarps; ++w) {
        if (w < warp) at += sh.w_cnt[w];
        n += sh.w_cnt[w];
      }
      if (in) rows[at + __popc(who & ((1u << lane) - 1u))] = r;
      __syncthreads();
    }
    sp.rows = rows;
    sp.n = n;
  } else {
    sp.rows = nullptr;
    sp.n = R;
  }
  sp.total = (long long)sp.n * sp.steps;
  sp.used = (int)min((long long)gridDim.x, sp.total);
  sp.small = (sp.total + 1) * (sp.used + 1) < (1ll << 32);
  const int cta = blockIdx.x;
  // the places and pieces of request b's rows; `near`: the place of one
  auto request = [&](int b, int near) {
    for (int w = tid; w < P.W; w += kBmThreads) sh.place[w] = -1;
    __syncthreads();
    const int a = near - kBeamMax + tid;
    if (tid < 2 * kBeamMax && a >= 0 && a < sp.n) {
      const int w = sp.row(a) - b * P.W;
      if (w >= 0 && w < P.W) {
        sh.pieces[w] = sp.pieces(a);
        sh.place[w] = sp.rows || beam_read(P, sp.row(a)) ? a : -1;
      }
    }
    __syncthreads();
  };
  if (cta < sp.used) {
    long long x = sp.begin(cta);
    const long long end = sp.begin(cta + 1);
    // the piece at step y (of no tokens past the range)
    auto piece = [&](long long y) {
      BeamPiece p;
      p.a = (int)((uint32_t)y / (uint32_t)sp.steps);
      p.row = y < end ? sp.row(p.a) : 0;
      const int c0 = (int)(y - (long long)p.a * sp.steps), len = (int)min((long long)(sp.steps - c0), end - y);
      p.lo = c0 * S::kStep;
      p.hi = y < end ? (int)min((long long)P.V, (long long)(c0 + len) * S::kStep) : 0;
      return p;
    };
    BeamPiece p = piece(x);
    uint4 next[kBmUnroll];
    beam_fetch<T>(P, p, p.lo + warp * S::kChunk + lane * S::N, next);
    while (x < end) {
      const int b = p.row / P.W, len = (p.hi - p.lo + S::kStep - 1) / S::kStep;
      const BeamPiece after = piece(x + len);
      if (sp.rows || beam_read(P, p.row))
        beam_piece<T>(P, sh, p, after, next, P.stat + sp.record(cta, p.a, P.spans));
      else
        beam_fetch<T>(P, after, after.lo + warp * S::kChunk + lane * S::N, next);
      // A request's arrivals count steps: its rows in the split have so many.
      const int a = p.a - kBeamMax + tid;
      const bool its = tid < 2 * kBeamMax && a >= 0 && a < sp.n && sp.row(a) >= b * P.W && sp.row(a) < (b + 1) * P.W;
      const int rows = __syncthreads_count(its);  // and what the CTA has written is before this
      if (tid == 0) {
        __threadfence();
        sh.is_last = tagged_add(&P.counters[b], P.tag, len) + len == rows * sp.steps;
      }
      __syncthreads();
      if (sh.is_last) {
        __threadfence();
        request(b, p.a);
        beam_finish<T>(P, sh, smem, sp, b);
        __syncthreads();
      }
      x += len;
      p = after;
    }
  }
  // requests without a row in the split
  if (sp.rows) {
    for (int b = cta; b < P.B; b += gridDim.x) {
      bool some = false;
      for (int w = tid; w < P.W; w += kBmThreads) some |= beam_read(P, b * P.W + w);
      if (__syncthreads_or(some)) continue;
      for (int w = tid; w < P.W; w += kBmThreads) sh.place[w] = -1;
      __syncthreads();
      beam_finish<T>(P, sh, smem, sp, b);
      __syncthreads();
    }
  }
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

// Latency bounds it, parents to rows: 64 x 8 beams' 500 tokens and 3584 values,
// 9.4 MB read and written, 5 us.  Its launch overlaps the selection's end (48.4
// us for both, 49.4 in stream order; 4 beams 15.2, 16.5).
__global__ void __launch_bounds__(kRoThreads) beam_reorder_kernel(const ReorderParams P) {
  after_previous();
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

// The launch: as many CTAs as the device holds at once, of at least one step
// each.  P.spans becomes the most pieces of a CTA, P.chunks a row's chunks.
void plan_beams(BeamParams& P, bool bf16, int num_sms) {
  const int chunk = bf16 ? BmShape<__nv_bfloat16>::kChunk : BmShape<float>::kChunk;
  const long long step = (long long)kBmWarps * chunk, steps = (P.V + step - 1) / step, rows = (long long)P.B * P.W;
  long long g = (long long)kBmCtas * num_sms;
  if (g > rows * steps) g = rows * steps;
  P.grid = (int)g;
  P.chunks = (P.V + chunk - 1) / chunk;
  // a CTA's range is at most this many steps, whichever rows are read
  const long long range = (rows * steps + g - 1) / g;
  P.spans = (int)((range + steps - 1) / steps + 1);
}

int launch_beam_select(const BeamParams& P, bool bf16, cudaStream_t s) {
  // the last CTA's candidates and chunks, then the rows that are read
  const long long rows = (long long)P.B * P.W;
  const int bytes = kBmCap * 12 + kBmHot * 4 + (rows <= kBeamRows ? (int)rows * 4 : 0);
  return bf16 ? launch_kernel(beam_select_kernel<__nv_bfloat16>, dim3(P.grid), kBmThreads, bytes, s, P)
              : launch_kernel(beam_select_kernel<float>, dim3(P.grid), kBmThreads, bytes, s, P);
}

// Fills the work split of P's states and returns the number of blocks, or one
// past 32 bits (a state has at most 2^31 rows of 2^30 blocks, so that the sum
// is not taken further).
long long plan_reorder(ReorderParams& P) {
  long long at = 0;
  for (int k = 0; k < P.num; ++k) {
    BeamState& s = P.s[k];
    const long long n = s.row_bytes / s.unit, per = kRoThreads * kRoPer;
    s.blocks = (int)((n + per - 1) / per);
    s.first = at;
    at += (long long)s.blocks * s.outer * P.B * P.keep;
    if (at > INT32_MAX) break;
  }
  return at;
}

int launch_beam_reorder(const ReorderParams& P, long long blocks, cudaStream_t s) {
  return launch_kernel(beam_reorder_kernel, dim3((unsigned)blocks), kRoThreads, 0, s, P);
}

}  // namespace sv
