// Norms of the heads of queries and keys, and their rotation to positions.
#include "tree_common.cuh"
#include "serve_internal.h"

namespace sv {
namespace {

constexpr int kRotWarps = 8;

// Lanes of a warp that share a head, 8 channels each (some idle where D / 8 is
// no power of two).
template <int D>
constexpr int kRotLanes = D <= 64 ? 8 : (D <= 128 ? 16 : 32);

template <typename T>
__device__ __forceinline__ void unpack4(uint2 v, float (&x)[4]) {
  x[0] = half_to_f32<T>(v.x & 0xffffu);
  x[1] = half_to_f32<T>(v.x >> 16);
  x[2] = half_to_f32<T>(v.y & 0xffffu);
  x[3] = half_to_f32<T>(v.y >> 16);
}

// Volatile, to stay behind the wait for the kernel before.
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

// y = x / sqrt(mean x^2 + eps) w, then pairs (a, b) turned by positions[r] f_i.
//
// A lane holds 8 channels of a head, both halves of four pairs (channels
// 4l .. 4l + 3 and rot / 2 more), so only the mean crosses lanes, and a warp
// 4, 2 or 1 heads of a row at once.  It walks over the row's heads with the
// row's sines and cosines in registers: 32 heads share 4 of each a lane.
//
// The angle in turns is positions[r] f_i / 2 pi.  Its fraction is exact in
// 64-bit fixed point: F_i = frac(f_i / 2 pi) 2^64 once per CTA, in fp64, and
// the fraction of position times F_i is the low 64 bits of the product of
// whole numbers.  In fp32 a position of 2^17 leaves 7 bits of the turn.
template <typename T, int D>
__global__ void __launch_bounds__(kRotWarps * 32) norm_rotate_kernel(const RotateParams P) {
  constexpr int G = kRotLanes<D>, H = 32 / G;
  __shared__ unsigned long long turn[D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % G, sub = lane / G;
  after_previous();
  for (int i = tid; i < P.rot / 2; i += kRotWarps * 32) {
    double t = (double)P.inv_freq[i] * 0.15915494309189535;  // 1 / 2 pi
    t -= floor(t);
    turn[i] = (unsigned long long)(t * 18446744073709551616.0);
  }
  __syncthreads();
  const bool real = l < D / 8, turns = l < P.rot / 8;
  // this lane's two runs of four channels
  const int o0 = turns && !P.interleaved ? 4 * l : 8 * l;
  const int o1 = turns && !P.interleaved ? P.rot / 2 + 4 * l : 8 * l + 4;
  float w[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const T* src = static_cast<const T*>(P.side[s].weight);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[s][e] = 1.f;
    if (src && real) {
      float a[4], b[4];
      unpack4<T>(load8(src + o0), a);
      unpack4<T>(load8(src + o1), b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[s][e] = a[e];
        w[s][4 + e] = b[e];
      }
    }
  }
  const int steps_q = (P.side[0].heads + H - 1) / H;
  const long long all = (long long)P.rows * P.parts;
  for (long long u = (long long)blockIdx.x * kRotWarps + warp; u < all; u += (long long)gridDim.x * kRotWarps) {
    const int row = (int)(u / P.parts), part = (int)(u - (long long)row * P.parts);
    const int from = (int)((long long)part * P.steps / P.parts), to = (int)((long long)(part + 1) * P.steps / P.parts);
    float cs[4], sn[4];
    if (turns) {
      const unsigned long long pos = (unsigned long long)(long long)P.positions[row];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int frac = (int)((turn[4 * l + e] * pos) >> 32);  // of 2^32 a turn, nearest turn
        sincospif((float)frac * 4.656612873077393e-10f, &sn[e], &cs[e]);
      }
    }
    constexpr int U = 4;  // steps whose loads are in flight at once
    for (int i0 = from; i0 < to; i0 += U) {
      uint2 va[U], vb[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k, s = i >= steps_q, h = (i - (s ? steps_q : 0)) * H + sub;
        va[k] = vb[k] = make_uint2(0u, 0u);
        if (i < to && real && h < P.side[s].heads) {
          const T* src = static_cast<const T*>(P.side[s].x) + (long long)row * P.side[s].sx_row + (long long)h * P.side[s].sx_head;
          va[k] = load8(src + o0);
          vb[k] = load8(src + o1);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k, s = i >= steps_q, h = (i - (s ? steps_q : 0)) * H + sub;
        if (i >= to) break;  // warp-uniform
        float a[4], b[4], sum = 0.f;
        unpack4<T>(va[k], a);
        unpack4<T>(vb[k], b);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = fmaf(a[e], a[e], fmaf(b[e], b[e], sum));
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum * (1.f / D) + P.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] *= r * (s ? w[1][e] : w[0][e]);
          b[e] *= r * (s ? w[1][4 + e] : w[0][4 + e]);
        }
        if (turns) {
          if (!P.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = a[e], y = b[e];
              a[e] = x * cs[e] - y * sn[e];
              b[e] = y * cs[e] + x * sn[e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = a[2 * e], y = a[2 * e + 1], z = b[2 * e], t = b[2 * e + 1];
              a[2 * e] = x * cs[e] - y * sn[e];
              a[2 * e + 1] = y * cs[e] + x * sn[e];
              b[2 * e] = z * cs[2 + e] - t * sn[2 + e];
              b[2 * e + 1] = t * cs[2 + e] + z * sn[2 + e];
            }
          }
        }
        if (real && h < P.side[s].heads) {
          T* dst = static_cast<T*>(P.side[s].y) + (long long)row * P.side[s].sy_row + (long long)h * P.side[s].sy_head;
          *reinterpret_cast<uint2*>(dst + o0) = make_uint2(pack2<T>(a[0], a[1]), pack2<T>(a[2], a[3]));
          *reinterpret_cast<uint2*>(dst + o1) = make_uint2(pack2<T>(b[0], b[1]), pack2<T>(b[2], b[3]));
        }
      }
    }
  }
}

constexpr int kRotCtas = 4;  // per SM

template <typename T, int D>
int launch(RotateParams& P, int num_sms, cudaStream_t s) {
  constexpr int H = 32 / kRotLanes<D>;
  P.steps = (P.side[0].heads + H - 1) / H + (P.side[1].heads + H - 1) / H;
  // A warp for each row where there are as many rows as warps; fewer rows are
  // shared by as many warps as there are, down to a step each.
  const long long warps = (long long)num_sms * kRotCtas * kRotWarps;
  P.parts = (int)max(1ll, min((long long)P.steps, warps / P.rows));
  const long long ctas = ((long long)P.rows * P.parts + kRotWarps - 1) / kRotWarps;
  return launch_kernel(norm_rotate_kernel<T, D>, dim3((unsigned)min(ctas, (long long)num_sms * kRotCtas)), kRotWarps * 32, 0,
                       s, P);
}

template <typename T>
int launch_dim(RotateParams& P, int num_sms, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch<T, 64>(P, num_sms, s);
    case 96: return launch<T, 96>(P, num_sms, s);
    case 128: return launch<T, 128>(P, num_sms, s);
    case 192: return launch<T, 192>(P, num_sms, s);
    case 256: return launch<T, 256>(P, num_sms, s);
    default: return -1;
  }
}

}  // namespace

int launch_norm_rotate(RotateParams& P, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? launch_dim<__nv_bfloat16>(P, num_sms, s) : launch_dim<__half>(P, num_sms, s);
}

}  // namespace sv
