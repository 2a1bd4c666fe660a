// Commitment of the accepted path to a cache held in 8 bits.
#include "cache8_common.cuh"

namespace sv {
namespace {

constexpr int kC8Threads = 256;
constexpr int kC8Warps = kC8Threads / 32;
constexpr int kC8Rows = 16;  // tokens of a warp's step

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

// A barrier of the warps that share a unit (constant ids: a barrier that is not
// known reserves all sixteen).
__device__ __forceinline__ void unit_sync(int group, int threads) {
  switch (group) {
    case 0: named_sync(1, threads); break;
    case 1: named_sync(2, threads); break;
    case 2: named_sync(3, threads); break;
    default: named_sync(4, threads); break;
  }
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

// The larger size of each of two values, in the size's bits; NaN against a number
// gives the number (the signs of the result mean nothing).
template <typename T>
__device__ __forceinline__ uint32_t max_size2(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_size2<__half>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <>
__device__ __forceinline__ uint32_t max_size2<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A unit is one block of tokens of one layer and head, keys or values: `warps`
// warps take its rows, 16 a warp and step (a lane 8 channels of every R-th row),
// find the largest size, agree on the scale, and write the bytes.  Bytes bound it:
// 2 read and 1 written for every channel.  So a warp has the rows of its next
// units, or of its next steps, in flight to shared memory while it works on one
// (registers for them would leave too few warps).  A warp with more than 16 rows
// of a unit goes over them twice, for the size and for the bytes.
//
// The CTAs of a request share its units evenly, over all layers, so that each
// looks at the request's lengths and path once for many of them.
//
// CHECKED: the check kernel has run, and a new length of -1 says that the
// request is bad.  Otherwise every CTA checks its request.
template <int D>
struct C8Stage {
  static constexpr int kBytes = kC8Rows * D * 2;               // of a warp's step
  static constexpr int kStages = D <= 128 ? 3 : 2;
  static constexpr int kSmem = kC8Warps * kStages * kBytes;
};

// What a unit's first step brings with its rows.
struct alignas(16) C8Unit {
  float* scale;
  uint8_t* held;  // of the warp's first row
  int q0, q1;     // of the warp's rows, [q0, q1) are new tokens
  int flags;      // 1: a unit, 2: tokens of the block were there
  float old;      // its scale then
};

template <typename T, int D, bool CHECKED>
__global__ void __launch_bounds__(kC8Threads, D <= 128 ? 2 : 1) commit8_kernel(const Commit8Params P) {
  using S = C8Stage<D>;
  constexpr int LR = D / 8;                     // lanes per row
  constexpr int R = 32 / LR;                    // rows of a warp at once
  constexpr int N = kC8Rows / R;                // and how often
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float tops[2][kC8Warps];
  __shared__ C8Unit info[kC8Warps][S::kStages];
  after_previous();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Path8 r;
  if (CHECKED) {
    r.cu = P.cu[b];
    r.m = P.path_len[b];
    const int len = P.new_len[b];
    r.status = len < 0;
    r.ctx = len - r.m;
  } else {
    r = check_path(P, b);
    if (blockIdx.y == 0 && tid == 0) {
      if (P.status) P.status[b] = r.status;
      P.new_len[b] = r.status ? -1 : r.ctx + r.m;
    }
  }
  if (r.status || r.m == 0) return;
  const PageDiv pd(P.page_size), bd(P.block);
  const int32_t* path = P.path + (long long)b * P.ld_path;
  const int32_t* table = P.table + (long long)b * P.ld_table;
  const int W = P.warps, group = warp / W, wsub = warp % W, groups = kC8Warps / W;
  int first_block, last_block, rest;
  bd.split(r.ctx, first_block, rest);
  bd.split(r.ctx + r.m - 1, last_block, rest);
  const int of_layer = (last_block - first_block + 1) * P.heads * 2;  // heads change first: neighbours' rows lie side by side
  const long long units = (long long)of_layer * P.layers;
  const int per = (P.block + W - 1) / W;        // rows of a warp
  const int w_rows = max(0, min(per, P.block - wsub * per));
  const int passes = (per + kC8Rows - 1) / kC8Rows, steps = passes == 1 ? 1 : 2 * passes;  // of a unit
  const int rsub = lane / LR, ch = (lane % LR) * 8;
  const bool lane_on = rsub < R;
  // every warp of a CTA takes the same number of turns
  const long long stride = (long long)gridDim.y * groups, u_base = (long long)blockIdx.y * groups;
  unsigned char* stage = smem + warp * (S::kStages * S::kBytes);
  const uint32_t stage_at = smem_u32(stage) + lane * 16;
  // The copies: of unit after unit, step after step.
  long long base_ahead = u_base;
  int step_ahead = 0, slot_ahead = 0, q0 = 0, q1 = 0, w0 = 0;
  const T* x = nullptr;
  auto copy = [&]() {
    if (base_ahead < units) {
      if (step_ahead == 0) {  // the next unit
        const bool mine = base_ahead + group < units;
        const long long u = mine ? base_ahead + group : 0;
        const int layer = (int)div_fast(u, of_layer), o = (int)(u - (long long)layer * of_layer), kv = o & 1;
        const int j = (int)((uint32_t)(o >> 1) / (uint32_t)P.heads), h = (o >> 1) - j * P.heads;
        const int base = (first_block + j) * P.block;
        w0 = base + wsub * per;
        q0 = max(0, r.ctx - w0);
        q1 = mine ? min(w_rows, r.ctx + r.m - w0) : 0;
        int page, slot, blk, rest2;
        pd.split(base, page, slot);
        bd.split(slot, blk, rest2);
        const int id = table[page];
        float* scale = P.scale[kv] + (long long)layer * P.c_layer + (long long)id * P.c_page + (long long)blk * P.c_block +
                       (long long)h * P.c_head;
        x = static_cast<const T*>(P.x[kv]) + (long long)layer * P.sn_layer + (long long)r.cu * P.sn_node +
            (long long)h * P.sn_head + ch;
        C8Unit& n = info[warp][slot_ahead];
        const bool before = mine && base < r.ctx;
        __syncwarp();  // its last unit has been read
        if (lane == 0) {
          n.scale = scale;
          n.held = P.held[kv] + (long long)layer * P.s_layer + (long long)id * P.s_page +
                   (long long)(slot + wsub * per) * P.s_slot + (long long)h * P.s_head;
          n.q0 = q0;
          n.q1 = q1;
          n.flags = (mine ? 1 : 0) | (before ? 2 : 0);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&n.old)), "l"(scale), "r"(before ? 4 : 0)
                       : "memory");
        }
      }
      const int c = (step_ahead < passes ? step_ahead : step_ahead - passes) * kC8Rows;
      // lane q of the first 16 looks up the node of row c + q
      const int q = c + (lane & 15);
      const int node = q >= q0 && q < q1 ? path[w0 - r.ctx + q] : -1;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = __shfl_sync(0xffffffffu, node, (i * R + rsub) & 31);
        if (lane_on) cp_async16(stage_at + slot_ahead * S::kBytes + i * (R * D * 2), x + (long long)max(at, 0) * P.sn_node, at >= 0);
      }
      if (++step_ahead == steps) {
        step_ahead = 0;
        base_ahead += stride;
      }
      if (++slot_ahead == S::kStages) slot_ahead = 0;
    }
    cp_async_commit();
  };
  const uint32_t em = exp_mask<T>();
  const long long row_step = (long long)R * P.s_slot;
  int turn = 0, slot_now = 0;
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) copy();
  // Waits for the next step's rows and has the copies go on.
  uint4 v[N];
  auto rows = [&]() {
    cp_async_wait<S::kStages - 2>();
    __syncwarp();
    const unsigned char* at = stage + slot_now * S::kBytes + lane * 16;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_on ? *reinterpret_cast<const uint4*>(at + i * (R * D * 2)) : make_uint4(0u, 0u, 0u, 0u);
    if (++slot_now == S::kStages) slot_now = 0;
  };
  for (long long u0 = u_base; u0 < units; u0 += stride, turn ^= 1) {
    C8Unit n;
    float* scale = nullptr;
    uint8_t* held = nullptr;  // row rsub
    bool before = false;
    uint32_t top = 0;  // of two values at once
    bool odd = false;  // infinities
#pragma unroll 1
    for (int c = 0; c < passes; ++c) {
      const int slot = slot_now;
      rows();
      if (c == 0) {
        n = info[warp][slot];
        scale = n.scale;
        held = n.held + (long long)rsub * P.s_slot + ch;
        before = (n.flags & 2) != 0;
      }
      copy();  // into the slot that the step before left
      uint32_t size = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        size = max_size2<T>(max_size2<T>(size, max_size2<T>(v[i].x, v[i].y)), max_size2<T>(v[i].z, v[i].w));
      size &= 0x7fff7fffu;
      // two NaN leave NaN
      if (__any_sync(0xffffffffu, (size & 0xffffu) >= em || (size >> 16) >= em)) {
        odd = true;
        size = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
          size = max_u16x2(size, max_u16x2(max_u16x2(finite_size2(v[i].x, em), finite_size2(v[i].y, em)),
                                           max_u16x2(finite_size2(v[i].z, em), finite_size2(v[i].w, em))));
      }
      top = max_u16x2(top, size);
    }
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    float big = half_to_f32<T>(top);
    if (W > 1) {
      if (lane == 0) tops[turn][warp] = big;
      // the unit's warps; also: every one has read the old scale
      unit_sync(group, W * 32);
      for (int k = 0; k < W; ++k) big = fmaxf(big, tops[turn][group * W + k]);
    } else {
      __syncwarp();
    }
    const float need = scale_for(big);
    const float old = n.old;
    const bool grown = before && need > old;
    const float s = before && !grown ? old : need, inv = s == 0.f ? 0.f : 1.f / s;
    if ((n.flags & 1) && wsub == 0 && lane == 0 && (!before || grown)) *scale = s;
    // eight values under the scale
    auto bytes8 = [&](const uint4& x, bool odd) {
      const uint32_t e[4] = {x.x, x.y, x.z, x.w};
      uint32_t b2[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 f = make_float2(half_to_f32<T>(e[k] & 0xffffu), half_to_f32<T>(e[k] >> 16));
        f = odd ? make_float2(to8_arg(f.x, inv), to8_arg(f.y, inv)) : __fmul2_rn(f, make_float2(inv, inv));
        b2[k] = to_e4m3x2(f.x, f.y);
      }
      return make_uint2(__byte_perm(b2[0], b2[1], 0x5410), __byte_perm(b2[2], b2[3], 0x5410));
    };
#pragma unroll 1
    for (int c = 0; c < passes; ++c) {  // new tokens
      if (passes > 1) {
        rows();
        copy();
      }
      uint8_t* d = held + (long long)(c * kC8Rows) * P.s_slot;
      const int f0 = n.q0 - c * kC8Rows, f1 = n.q1 - c * kC8Rows;
      if (!odd && f0 <= 0 && f1 >= kC8Rows) {
#pragma unroll
        for (int i = 0; i < N; ++i, d += row_step)
          if (lane_on) *reinterpret_cast<uint2*>(d) = bytes8(v[i], false);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i, d += row_step)
          if (lane_on && i * R + rsub >= f0 && i * R + rsub < f1) *reinterpret_cast<uint2*>(d) = bytes8(v[i], true);
      }
    }
    if (grown && lane_on) {  // tokens that were there, under the new scale
      uint8_t* d = held;
      for (int q = rsub; q < min(w_rows, n.q0); q += R, d += row_step) {
        const uint2 w = *reinterpret_cast<const uint2*>(d);
        uint32_t z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t y = k ? w.y : w.x;
          const float2 a = from_e4m3x2(y & 0xffffu), c = from_e4m3x2(y >> 16);
          z[k] = to_e4m3x2(a.x * old * inv, a.y * old * inv) | to_e4m3x2(c.x * old * inv, c.y * old * inv) << 16;
        }
        *reinterpret_cast<uint2*>(d) = make_uint2(z[0], z[1]);
      }
    }
  }
  cp_async_wait<0>();
}

template <typename T, int D, bool CHECKED>
int launch_commit_as(const Commit8Params& P, dim3 grid, cudaStream_t s) {
  constexpr int smem = C8Stage<D>::kSmem;
  if (cudaFuncSetAttribute(commit8_kernel<T, D, CHECKED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(commit8_kernel<T, D, CHECKED>, grid, kC8Threads, smem, s, P);
}

template <typename T, int D>
int launch_commit(const Commit8Params& P, bool checked, dim3 grid, cudaStream_t s) {
  return checked ? launch_commit_as<T, D, true>(P, grid, s) : launch_commit_as<T, D, false>(P, grid, s);
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
constexpr int kC8Waves = 6;       // CTAs for each SM

}  // namespace

int launch_commit8(Commit8Params& P, bool bf16, int num_sms, cudaStream_t s) {
  const int need = (P.block + kC8Rows - 1) / kC8Rows;
  P.warps = 1;
  while (P.warps < kC8Warps && P.warps < need) P.warps *= 2;
  const long long blocks = (P.ld_path + P.block - 2ll) / P.block + 1, units = blocks * P.heads * 2 * P.layers;
  const int groups = kC8Warps / P.warps;
  // As many CTAs as run at once, several times where there is work for them: a
  // request's share depends on its path, which the host does not know.
  const long long turns = (units + groups - 1) / groups, share = (kC8Waves * num_sms + P.B - 1) / P.B;
  const unsigned y = (unsigned)(turns < share ? turns : share < 65535 ? share : 65535);
  const bool checked = P.new_len == P.ctx || P.ld_path > kC8OwnCheck;
  if (checked && launch_kernel(commit8_check_kernel, dim3(P.B), kC8Threads, 0, s, P)) return -1;
  const dim3 grid((unsigned)P.B, y);
  return bf16 ? launch_commit_dim<__nv_bfloat16>(P, checked, grid, s) : launch_commit_dim<__half>(P, checked, grid, s);
}

}  // namespace sv
