// Commitment of the accepted path to a cache held in 8 bits.
#include "cache8_common.cuh"

namespace sv {
namespace {

constexpr int kC8Threads = 256;
constexpr int kC8Warps = kC8Threads / 32;
constexpr int kC8Rows = 16;  // tokens that a warp holds in registers

// The smallest power of two from 2^-126 on whose 448-fold (0.875 of 2^9) reaches
// the finite top >= 0; 0 for 0.
__device__ __forceinline__ float scale_for(float top) {
  if (top == 0.f) return 0.f;
  const uint32_t b = __float_as_uint(top);
  // top = (1 + m / 2^23) 2^(e - 127), to be at most 1.75 2^8 2^k
  const int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(k, -126) + 127) << 23);
}

// x * inv, infinities as NaN (the conversion would saturate them).
__device__ __forceinline__ float to8_arg(float x, float inv) { return fmaf(x, 0.f, x * inv); }

// The request's tokens and pages, found sound or not: every thread of a CTA
// comes here.
struct Path8 {
  int cu, m, ctx, status;
};
__device__ __forceinline__ Path8 check_path(const Commit8Params& P, int b) {
  Path8 r;
  r.cu = P.cu[b];
  const int n = P.cu[b + 1] - r.cu;
  r.m = P.path_len[b];
  r.ctx = P.ctx[b];
  const bool ok = r.cu >= 0 && n >= 0 && (long long)r.cu + n <= P.total && r.m >= 0 && r.m <= P.ld_path && r.ctx >= 0 &&
                  (long long)r.ctx + r.m <= (long long)P.ld_table * P.page_size;
  const PageDiv pd(P.page_size);
  int bad = 0;
  if (ok) {
    const int32_t* path = P.path + (long long)b * P.ld_path;
    for (int i = threadIdx.x; i < r.m; i += kC8Threads) {
      const int node = path[i];
      bad |= node < 0 || node >= n ? 1 : 0;
    }
    if (r.m > 0) {
      int first, last, slot;
      pd.split(r.ctx, first, slot);
      pd.split(r.ctx + r.m - 1, last, slot);
      for (int p = first + (int)threadIdx.x; p <= last; p += kC8Threads) {
        const int id = P.table[(long long)b * P.ld_table + p];
        bad |= id < 0 || id >= P.num_pages ? 2 : 0;
      }
    }
  }
  r.status = ok ? 0 : kStatusBadLen;
  if (__syncthreads_or(bad)) {
    if (__syncthreads_or(bad & 1)) r.status |= kStatusBadLen;
    if (__syncthreads_or(bad & 2)) r.status |= kStatusBadPage;
  }
  return r;
}

// One CTA per request: its status and new length.
__global__ void __launch_bounds__(kC8Threads) commit8_check_kernel(const Commit8Params P) {
  after_previous();
  const int b = blockIdx.x;
  const Path8 r = check_path(P, b);
  if (threadIdx.x == 0) {
    if (P.status) P.status[b] = r.status;
    P.new_len[b] = r.status ? -1 : r.ctx + r.m;
  }
}

// A unit is one block of tokens of one head, keys or values: `warps` warps take
// its rows, up to 16 a warp and pass (a lane 8 channels of every R-th row), find
// the largest size, agree on the scale, and write the bytes.  A block of at most
// 16 rows a warp is read once, its rows staying in registers.  Bytes bound it: 2
// read and 1 written for every channel.
//
// CHECKED: the check kernel has run, and a new length of -1 says that the
// request is bad.  Otherwise every CTA checks its request.
template <typename T, int D, bool CHECKED>
__global__ void __launch_bounds__(kC8Threads) commit8_kernel(const Commit8Params P) {
  constexpr int LR = D / 8;                     // lanes per row
  constexpr int R = 32 / LR;                    // rows of a warp at once
  constexpr int N = (kC8Rows + R - 1) / R;      // and how often
  __shared__ float tops[2][kC8Warps];
  after_previous();
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Path8 r;
  if (CHECKED) {
    r.cu = P.cu[b];
    r.m = P.path_len[b];
    const int len = P.new_len[b];
    r.status = len < 0;
    r.ctx = len - r.m;
  } else {
    r = check_path(P, b);
    if (layer == 0 && blockIdx.z == 0 && tid == 0) {
      if (P.status) P.status[b] = r.status;
      P.new_len[b] = r.status ? -1 : r.ctx + r.m;
    }
  }
  if (r.status || r.m == 0) return;
  const PageDiv pd(P.page_size);
  const int32_t* path = P.path + (long long)b * P.ld_path;
  const int32_t* table = P.table + (long long)b * P.ld_table;
  const int W = P.warps, group = warp / W, wsub = warp % W, groups = kC8Warps / W;
  const int first_block = r.ctx / P.block, blocks = (r.ctx + r.m - 1) / P.block - first_block + 1;
  const int units = blocks * P.heads * 2;       // the head changes first: neighbours' rows lie side by side
  const int per = (P.block + W - 1) / W;        // rows of a warp
  const int rsub = lane / LR, ch = (lane % LR) * 8;
  int turn = 0;
  // every warp of a CTA takes the same number of turns
  for (int u0 = blockIdx.z * groups; u0 < units; u0 += gridDim.z * groups, turn ^= 1) {
    const int u = u0 + group;
    const bool mine = u < units;
    const int kv = mine ? u % 2 : 0, h = mine ? (u / 2) % P.heads : 0, j = first_block + (mine ? u / 2 / P.heads : 0);
    const int base = j * P.block;               // the block's first token
    const int lo = max(r.ctx, base), hi = mine ? min(r.ctx + r.m, base + P.block) : lo;
    int page, slot;
    pd.split(base, page, slot);
    const int id = table[page];
    uint8_t* held = P.held[kv] + (long long)layer * P.s_layer + (long long)id * P.s_page + (long long)slot * P.s_slot +
                    (long long)h * P.s_head + ch;
    float* at = P.scale[kv] + (long long)layer * P.c_layer + (long long)id * P.c_page +
                (long long)(slot / P.block) * P.c_block + (long long)h * P.c_head;
    const T* x = static_cast<const T*>(P.x[kv]) + (long long)layer * P.sn_layer + (long long)r.cu * P.sn_node +
                 (long long)h * P.sn_head + ch;
    const bool before = mine && base < r.ctx;   // tokens of the block that were there
    const float old = before ? *at : 0.f;
    const int w0 = base + wsub * per, w1 = min(base + P.block, w0 + per);  // this warp's rows
    uint4 v[N];
    auto load = [&](int c) {  // rows c .. c + 15
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = c + i * R + rsub;
        const bool in = rsub < R && p >= lo && p < hi && p < w1 && i * R + rsub < kC8Rows;
        v[i] = in ? load16(x + (long long)path[p - r.ctx] * P.sn_node) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    uint32_t top = 0;  // the largest size's bits, of two 16-bit values at once
    const uint32_t em = exp_mask<T>();
    for (int c = w0; c < w1 && c < hi; c += kC8Rows) {
      load(c);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t* e = reinterpret_cast<const uint32_t*>(&v[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) top = __vmaxu2(top, finite_size2(e[k], em));
      }
    }
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    float big = half_to_f32<T>(top);
    if (W > 1) {
      if (lane == 0) tops[turn][warp] = big;
      __syncthreads();  // also: every warp has read the old scale
      for (int k = 0; k < W; ++k) big = fmaxf(big, tops[turn][group * W + k]);
    } else {
      __syncwarp();
    }
    if (!mine) continue;
    const float need = scale_for(big);
    const bool grown = before && need > old;
    const float s = before && !grown ? old : need, inv = s == 0.f ? 0.f : 1.f / s;
    if (wsub == 0 && lane == 0 && (!before || grown)) *at = s;
    // new tokens
    for (int c = w0; c < w1 && c < hi; c += kC8Rows) {
      if (per > kC8Rows) load(c);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = c + i * R + rsub;
        if (!(rsub < R && p >= lo && p < hi && p < w1 && i * R + rsub < kC8Rows)) continue;
        const uint32_t* e = reinterpret_cast<const uint32_t*>(&v[i]);
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            f[z] = to8_arg(half_to_f32<T>(z & 1 ? e[2 * k + z / 2] >> 16 : e[2 * k + z / 2] & 0xffffu), inv);
          q[k] = to_e4m3x2(f[0], f[1]) | to_e4m3x2(f[2], f[3]) << 16;
        }
        *reinterpret_cast<uint2*>(held + (long long)(p - base) * P.s_slot) = make_uint2(q[0], q[1]);
      }
    }
    // tokens that were there, under the new scale
    if (!grown) continue;
    for (int p = w0 + rsub; p < min(w1, r.ctx); p += R) {
      if (rsub >= R) break;
      uint2* d = reinterpret_cast<uint2*>(held + (long long)(p - base) * P.s_slot);
      const uint2 w = *d;
      uint32_t q[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t y = k ? w.y : w.x;
        const float2 a = from_e4m3x2(y & 0xffffu), c = from_e4m3x2(y >> 16);
        q[k] = to_e4m3x2(a.x * old * inv, a.y * old * inv) | to_e4m3x2(c.x * old * inv, c.y * old * inv) << 16;
      }
      *d = make_uint2(q[0], q[1]);
    }
  }
}

template <typename T, int D>
int launch_commit(const Commit8Params& P, bool checked, dim3 grid, cudaStream_t s) {
  return checked ? launch_kernel(commit8_kernel<T, D, true>, grid, kC8Threads, 0, s, P)
                 : launch_kernel(commit8_kernel<T, D, false>, grid, kC8Threads, 0, s, P);
}

template <typename T>
int launch_commit_dim(const Commit8Params& P, bool checked, dim3 grid, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch_commit<T, 64>(P, checked, grid, s);
    case 96: return launch_commit<T, 96>(P, checked, grid, s);
    case 128: return launch_commit<T, 128>(P, checked, grid, s);
    case 192: return launch_commit<T, 192>(P, checked, grid, s);
    case 256: return launch_commit<T, 256>(P, checked, grid, s);
    default: return -1;
  }
}

constexpr int kC8OwnCheck = 256;  // longest path that every CTA checks by itself

}  // namespace

int launch_commit8(Commit8Params& P, bool bf16, cudaStream_t s) {
  const int need = (P.block + kC8Rows - 1) / kC8Rows;
  P.warps = 1;
  while (P.warps < kC8Warps && P.warps < need) P.warps *= 2;
  const long long blocks = (P.ld_path + P.block - 2ll) / P.block + 1, units = blocks * P.heads * 2;
  const int groups = kC8Warps / P.warps;
  const long long turns = (units + groups - 1) / groups;
  const unsigned z = (unsigned)(turns < 8 ? turns : turns < 64 ? 8 : turns / 8 < 65535 ? turns / 8 : 65535);
  const bool checked = P.new_len == P.ctx || P.ld_path > kC8OwnCheck;
  if (checked && launch_kernel(commit8_check_kernel, dim3(P.B), kC8Threads, 0, s, P)) return -1;
  const dim3 grid((unsigned)P.B, (unsigned)P.layers, z);
  return bf16 ? launch_commit_dim<__nv_bfloat16>(P, checked, grid, s) : launch_commit_dim<__half>(P, checked, grid, s);
}

}  // namespace sv
