// Norms of the heads of queries and keys, and their rotation to positions.
#include "tree_common.cuh"
#include "serve_internal.h"

namespace sv {
namespace {

constexpr int kRotWarps = 8;

// Lanes of a warp that share a head, 2 CH channels each (some idle where D / 2 CH
// is no power of two).
template <int D, int CH>
constexpr int kRotLanes = (D <= 64 ? 32 : D <= 128 ? 64 : 128) / CH;

// CH channels: 8 or 16 bytes.  Volatile, to stay behind the wait for the kernel
// before.
template <int CH>
struct Run {
  uint32_t v[CH / 2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) v[i] = 0u;
  }
  __device__ __forceinline__ void load(const void* p) {
    if (CH == 8)
      asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[CH / 2 - 2]), "=r"(v[CH / 2 - 1])
                   : "l"(p)
                   : "memory");
    else
      asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void store(void* p) const {
    if (CH == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[CH / 2 - 2], v[CH / 2 - 1]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
  }
  template <typename T>
  __device__ __forceinline__ void unpack(float* x) const {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      x[2 * i] = half_to_f32<T>(v[i] & 0xffffu);
      x[2 * i + 1] = half_to_f32<T>(v[i] >> 16);
    }
  }
  template <typename T>
  __device__ __forceinline__ void pack(const float* x) {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) v[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  }
};

// y = x / sqrt(mean x^2 + eps) w, then pairs (a, b) turned by positions[r] f_i.
//
// A lane holds two runs of CH channels of a head, both halves of CH pairs
// (channels CH l .. and rot / 2 more), so only the mean crosses lanes, and a warp
// up to 8 heads of a row at once.  It walks over the row's heads with the row's
// sines and cosines in registers, which the lanes of the same channels compute
// together.  CH is 8 (16-byte accesses) where rot is a multiple of 16, else 4:
// 16384 rows of 32 heads of 128 take 55 us with 8 and 68 with 4.
//
// The angle in turns is positions[r] f_i / 2 pi.  Its fraction is exact in
// 64-bit fixed point: F_i = frac(f_i / 2 pi) 2^64 once per CTA, in two fp64 parts
// (one would leave 2^-52 of a frequency of several turns, 2^-24 of a turn at a
// position of 2^28), and the fraction of position times F_i is the low 64 bits of
// the product of whole numbers.  In fp32 a position of 2^17 leaves 7 bits of the
// turn.
//
// Its bytes are 2 read and 2 written a channel: 55 us are 4.9 TB/s, 72 % of the
// rate of a plain copy, which reads and writes as much.  The rest is each row's
// start (position, sines, weights, nothing in flight yet) and the last pass: warps
// take whole rows, 16384 of them 7 passes for 6.74.  One row of 16 heads takes 6.8
// us, a launch and two dependent loads.
template <typename T, int D, int CH>
__global__ void __launch_bounds__(kRotWarps * 32) norm_rotate_kernel(const RotateParams P) {
  constexpr int G = kRotLanes<D, CH>, H = 32 / G;
  __shared__ unsigned long long turn[D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % G, sub = lane / G;
  after_previous();
  bool odd = false;  // a frequency that is no number: its pairs are NaN
  for (int i = tid; i < P.rot / 2; i += kRotWarps * 32) {
    const float freq = P.inv_freq[i];
    odd = odd || !isfinite(freq);
    // |f| / 2 pi = t + rest, 1 / 2 pi in two parts and the product's own rounding
    const double f = fabs((double)freq), t = f * 0.15915494309189535;
    const double rest = fma(f, -9.839338337591243e-18, fma(f, 0.15915494309189535, -t));
    const unsigned long long part = (unsigned long long)((t - floor(t)) * 18446744073709551616.0) +
                                    (unsigned long long)(long long)(rest * 18446744073709551616.0);
    turn[i] = freq < 0.f ? 0ull - part : part;
  }
  odd = __syncthreads_or(odd) != 0;
  const bool real = l < D / (2 * CH), turns = l < P.rot / (2 * CH);
  // this lane's two runs
  const int o0 = turns && !P.interleaved ? CH * l : 2 * CH * l;
  const int o1 = turns && !P.interleaved ? P.rot / 2 + CH * l : 2 * CH * l + CH;
  const int steps_q = (P.side[0].heads + H - 1) / H;
  const long long all = (long long)P.rows * P.parts;
  for (long long u = (long long)blockIdx.x * kRotWarps + warp; u < all; u += (long long)gridDim.x * kRotWarps) {
    const int row = (int)div_fast(u, P.parts), part = (int)(u - (long long)row * P.parts);
    const int from = (int)((long long)part * P.steps / P.parts), to = (int)((long long)(part + 1) * P.steps / P.parts);
    float cs[CH], sn[CH];
    if (P.rot > 0) {
      // The H lanes of the same channels each compute every H-th pair (all of
      // them where a head has the whole warp).
      constexpr int OWN = CH / H < 1 ? 1 : CH / H;
      const unsigned long long pos = (unsigned long long)(long long)P.positions[row];
      float c[OWN], s[OWN];
#pragma unroll
      for (int e = 0; e < OWN; ++e) {
        const int i = (e * H + sub) % CH;
        const int frac = turns ? (int)((turn[CH * l + i] * pos) >> 32) : 0;  // of 2^32 a turn, nearest turn
        sincospif((float)frac * 4.656612873077393e-10f, &s[e], &c[e]);
        if (odd && turns && !isfinite(P.inv_freq[CH * l + i])) s[e] = c[e] = NAN;
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        cs[i] = __shfl_sync(0xffffffffu, c[i / H], l + (i % H) * G);
        sn[i] = __shfl_sync(0xffffffffu, s[i / H], l + (i % H) * G);
      }
    }
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {  // queries, then keys
      const int i_from = max(from - (s ? steps_q : 0), 0), i_to = min(to, s ? P.steps : steps_q) - (s ? steps_q : 0);
      if (i_from >= i_to) continue;  // warp-uniform
      const RotateSide& side = P.side[s];
      float w[2 * CH];
#pragma unroll
      for (int e = 0; e < 2 * CH; ++e) w[e] = 1.f;
      const T* weight = static_cast<const T*>(side.weight);
      if (weight && real) {
        Run<CH> x;
        x.load(weight + o0);
        x.template unpack<T>(w);
        x.load(weight + o1);
        x.template unpack<T>(w + CH);
      }
      // this lane's heads: h, h + H, ... of this warp's steps
      int h = i_from * H + sub;
      const int heads = real ? min(side.heads, i_to * H) : 0;
      const T* src = static_cast<const T*>(side.x) + (long long)row * side.sx_row + (long long)h * side.sx_head;
      T* dst = static_cast<T*>(side.y) + (long long)row * side.sy_row + (long long)h * side.sy_head;
      const long long src_step = H * side.sx_head, dst_step = H * side.sy_head;
      // U steps' loads are in flight while the U before are worked on
      constexpr int U = CH == 8 ? 2 : 4;
      Run<CH> va[2][U], vb[2][U];
      int h_load = h;
      auto load = [&](Run<CH>(&a)[U], Run<CH>(&b)[U]) {
#pragma unroll
        for (int k = 0; k < U; ++k, h_load += H, src += src_step) {
          a[k].clear();
          b[k].clear();
          if (h_load < heads) {
            a[k].load(src + o0);
            b[k].load(src + o1);
          }
        }
      };
      auto work = [&](Run<CH>(&va)[U], Run<CH>(&vb)[U]) {
#pragma unroll
        for (int k = 0; k < U; ++k, h += H, dst += dst_step) {
          float a[CH], b[CH], sum = 0.f;
          va[k].template unpack<T>(a);
          vb[k].template unpack<T>(b);
#pragma unroll
          for (int e = 0; e < CH; ++e) sum = fmaf(a[e], a[e], fmaf(b[e], b[e], sum));
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float r = rsqrtf(sum * (1.f / D) + P.eps);
#pragma unroll
          for (int e = 0; e < CH; ++e) {
            a[e] *= r * w[e];
            b[e] *= r * w[CH + e];
          }
          if (turns) {
            if (!P.interleaved) {
#pragma unroll
              for (int e = 0; e < CH; ++e) {
                const float x = a[e], y = b[e];
                a[e] = x * cs[e] - y * sn[e];
                b[e] = y * cs[e] + x * sn[e];
              }
            } else {
#pragma unroll
              for (int e = 0; e < CH / 2; ++e) {
                const float x = a[2 * e], y = a[2 * e + 1], z = b[2 * e], t = b[2 * e + 1];
                a[2 * e] = x * cs[e] - y * sn[e];
                a[2 * e + 1] = y * cs[e] + x * sn[e];
                b[2 * e] = z * cs[CH / 2 + e] - t * sn[CH / 2 + e];
                b[2 * e + 1] = t * cs[CH / 2 + e] + z * sn[CH / 2 + e];
              }
            }
          }
          if (h < heads) {
            va[k].template pack<T>(a);
            vb[k].template pack<T>(b);
            va[k].store(dst + o0);
            vb[k].store(dst + o1);
          }
        }
      };
      load(va[0], vb[0]);
      for (int i = i_from; i < i_to; i += 2 * U) {
        load(va[1], vb[1]);
        work(va[0], vb[0]);
        if (i + U >= i_to) break;
        load(va[0], vb[0]);
        work(va[1], vb[1]);
      }
    }
  }
}

// CTAs per SM: with 1, 2, 3 and 4 the 16384 rows take 82, 55, 66 and 57 us (a row's
// sines are computed once per warp, and 3 do not run at once).
constexpr int kRotCtas = 2;

template <typename T, int D, int CH>
int launch(RotateParams& P, int num_sms, cudaStream_t s) {
  constexpr int H = 32 / kRotLanes<D, CH>;
  P.steps = (P.side[0].heads + H - 1) / H + (P.side[1].heads + H - 1) / H;
  // A warp for each row where there are as many rows as warps; fewer rows are
  // shared by as many warps as there are, down to a step each.
  const long long warps = (long long)num_sms * kRotCtas * kRotWarps;
  P.parts = (int)max(1ll, min((long long)P.steps, warps / P.rows));
  const long long ctas = ((long long)P.rows * P.parts + kRotWarps - 1) / kRotWarps;
  return launch_kernel(norm_rotate_kernel<T, D, CH>, dim3((unsigned)min(ctas, (long long)num_sms * kRotCtas)),
                       kRotWarps * 32, 0, s, P);
}

template <typename T, int CH>
int launch_dim(RotateParams& P, int num_sms, cudaStream_t s) {
  switch (P.dim) {
    case 64: return launch<T, 64, CH>(P, num_sms, s);
    case 96: return launch<T, 96, CH>(P, num_sms, s);
    case 128: return launch<T, 128, CH>(P, num_sms, s);
    case 192: return launch<T, 192, CH>(P, num_sms, s);
    case 256: return launch<T, 256, CH>(P, num_sms, s);
    default: return -1;
  }
}

}  // namespace

int launch_norm_rotate(RotateParams& P, bool bf16, int num_sms, cudaStream_t s) {
  if (P.rot % 16 == 0)
    return bf16 ? launch_dim<__nv_bfloat16, 8>(P, num_sms, s) : launch_dim<__half, 8>(P, num_sms, s);
  return bf16 ? launch_dim<__nv_bfloat16, 4>(P, num_sms, s) : launch_dim<__half, 4>(P, num_sms, s);
}

}  // namespace sv
