// Attention weights: for every cached key, the sum over rows of its softmax
// weight.  Keys are the rows of the matrix product, so that a key's sum
// stays inside a quad of lanes and no row needs to be joined.
#include "tree_common.cuh"

namespace sv {
namespace {

constexpr int kWgWarps = 4;
constexpr int kWgKeys = 16 * kWgWarps;  // keys per tile: 16 per warp
constexpr int kWgRows = 32;             // query rows staged at once

// One CTA per (request, key head, tile of keys).  Each warp keeps its 16
// keys' fragments in registers and passes over the rows, kWgRows at a time:
//   w_j += sum_r 2^(scale q_r.k_j log2(e) - lse_r log2(e)).
// For the heads, pages and row counts that the tensor-memory kernel does not
// take.  The keys' bytes bound it with few rows, its latency with one tile per
// CTA: 16 requests of up to 16384 tokens, 8 key heads of 128 channels, 4 rows
// per key head, 149 us, 2.2 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(kWgWarps * 32) weigh_kernel(const WeighParams P, int tiles) {
  constexpr int CH = D / 8, PITCH = D + 8;
  __shared__ __align__(16) T qs[kWgRows * PITCH];
  __shared__ float ls[kWgRows];
  __shared__ int last_seen[kWgRows];  // last key that a row sees
  after_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % P.heads, b = bh / P.heads;
  const int cu = P.cu[b], n = P.cu[b + 1] - cu, len = P.len[b];
  const long long cap = (long long)P.ld_table * P.page_size;
  const bool ok = cu >= 0 && n >= 0 && n <= P.max_rows && (long long)cu + n <= P.total && len >= n && len <= P.ld &&
                  (long long)len <= cap;
  const float* before = P.before ? P.before + ((long long)b * P.heads + h) * P.ld : nullptr;
  float* out = P.out + ((long long)b * P.heads + h) * P.ld;
  if (h == 0 && tile == 0 && P.status) {
    int bad = 0;
    if (ok)
      for (long long p = tid; p < ((long long)len + P.page_size - 1) / P.page_size; p += kWgWarps * 32) {
        const int id = P.table[(long long)b * P.ld_table + p];
        bad |= id < 0 || id >= P.num_pages;
      }
    bad = __syncthreads_or(bad);
    if (tid == 0) P.status[b] = ok ? (bad ? kStatusBadPage : 0) : kStatusBadLen;
  }
  const int lo = tile * kWgKeys + warp * 16;
  const PageDiv pd(P.page_size);
  // key rows r0 and r0 + 8 of the fragments
  uint32_t kf[D / 16][4];
  bool bad[2] = {false, false};  // a page of their own each
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = lo + (lane >> 2) + 8 * e;
    const T* src = nullptr;
    if (ok && j < len) {
      int page, slot;
      pd.split(j, page, slot);
      const int id = P.table[(long long)b * P.ld_table + page];
      if (id < 0 || id >= P.num_pages)
        bad[e] = true;
      else
        src = static_cast<const T*>(P.k) + (long long)id * P.s_page + (long long)slot * P.s_slot + (long long)h * P.s_head;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        kf[ks][2 * c + e] = src ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + c * 8 + (lane & 3) * 2) : 0u;
  }
  float w[2] = {0.f, 0.f};
  const int rows = ok ? n * P.group : 0;
  for (int r0 = 0; r0 < rows; r0 += kWgRows) {
    __syncthreads();
    for (int i = tid; i < kWgRows * CH; i += kWgWarps * 32) {
      const int row = i / CH, ch = i % CH, R = r0 + row;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (R < rows)
        v = *reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + (long long)(cu + R / P.group) * P.sq_row +
                                            (long long)(h * P.group + R % P.group) * P.sq_head + ch * 8);
      *reinterpret_cast<uint4*>(qs + row * PITCH + ch * 8) = v;
    }
    if (tid < kWgRows) {
      const int R = r0 + tid;
      const bool in = R < rows;
      ls[tid] = in ? P.lse[(long long)(cu + R / P.group) * P.heads * P.group + h * P.group + R % P.group] *
                         1.4426950408889634f
                   : INFINITY;
      // padding and rows of infinite lse see nothing
      last_seen[tid] = in && fabsf(ls[tid]) != INFINITY ? len - n + R / P.group : -1;
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < kWgRows / 8; nt += 2) {
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const uint32_t qrow = smem_u32(qs) + (nt * 8 + (lane & 7) + ((lane & 16) >> 1)) * (PITCH * 2) + (lane & 8) * 2;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t qf[4];
        ldsm4(qrow + ks * 32, qf);
        mma16816<T>(s[0], kf[ks], qf[0], qf[1]);
        mma16816<T>(s[1], kf[ks], qf[2], qf[3]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = (nt + x) * 8 + (lane & 3) * 2 + (e & 1), j = lo + (lane >> 2) + 8 * (e >> 1);
          const float p = ex2(fmaf(s[x][e], P.scale_log2, -ls[row]));
          w[e >> 1] += j <= last_seen[row] ? p : 0.f;
        }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    w[e] += __shfl_xor_sync(0xffffffffu, w[e], 1);
    w[e] += __shfl_xor_sync(0xffffffffu, w[e], 2);
  }
  if ((lane & 3) == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = lo + (lane >> 2) + 8 * e;
      if (j < P.ld) out[j] = !ok ? NAN : (j < len ? (bad[e] ? NAN : (before ? before[j] : 0.f) + w[e]) : 0.f);
    }
  }
}

template <typename T>
int launch_dim(const WeighParams& P, cudaStream_t s) {
  const int tiles = (P.ld + kWgKeys - 1) / kWgKeys;
  const dim3 grid((unsigned)((long long)tiles * P.B * P.heads));
  switch (P.dim) {
    case 64: return launch_kernel(weigh_kernel<T, 64>, grid, kWgWarps * 32, 0, s, P, tiles);
    case 96: return launch_kernel(weigh_kernel<T, 96>, grid, kWgWarps * 32, 0, s, P, tiles);
    case 128: return launch_kernel(weigh_kernel<T, 128>, grid, kWgWarps * 32, 0, s, P, tiles);
    case 192: return launch_kernel(weigh_kernel<T, 192>, grid, kWgWarps * 32, 0, s, P, tiles);
    case 256: return launch_kernel(weigh_kernel<T, 256>, grid, kWgWarps * 32, 0, s, P, tiles);
    default: return -1;
  }
}

}  // namespace

int launch_weigh(const WeighParams& P, bool bf16, cudaStream_t s) {
  return bf16 ? launch_dim<__nv_bfloat16>(P, s) : launch_dim<__half>(P, s);
}

}  // namespace sv
