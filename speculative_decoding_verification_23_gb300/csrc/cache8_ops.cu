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

// A request's path: its first row and nodes, tokens to write, and the length
// before them.
struct Path8 {
  int cu, n, m, ctx;
};
__device__ __forceinline__ Path8 read_path(const Commit8Params& P, int b) {
  Path8 r;
  r.cu = P.cu[b];
  r.n = P.cu[b + 1] - r.cu;
  r.m = P.path_len[b];
  r.ctx = P.ctx[b];
  return r;
}
__device__ __forceinline__ bool lengths_ok(const Commit8Params& P, const Path8& r) {
  return r.cu >= 0 && r.n >= 0 && (long long)r.cu + r.n <= P.total && r.m >= 0 && r.m <= P.ld_path && r.ctx >= 0 &&
         (long long)r.ctx + r.m <= (long long)P.ld_table * P.page_size;
}
// Bit 0: a node outside the tree, bit 1: a bad page; thread `tid` of `threads`
// looks at every threads-th.
__device__ __forceinline__ int look_path(const Commit8Params& P, const Path8& r, int b, int tid, int threads) {
  int bad = 0;
  const int32_t* path = P.path + (long long)b * P.ld_path;
  for (int i = tid; i < r.m; i += threads) {
    const int node = path[i];
    bad |= node < 0 || node >= r.n ? 1 : 0;
  }
  if (r.m > 0) {
    const PageDiv pd(P.page_size);
    int first, last, slot;
    pd.split(r.ctx, first, slot);
    pd.split(r.ctx + r.m - 1, last, slot);
    for (int p = first + tid; p <= last; p += threads) {
      const int id = P.table[(long long)b * P.ld_table + p];
      bad |= id < 0 || id >= P.num_pages ? 2 : 0;
    }
  }
  return bad;
}
__device__ __forceinline__ int path_status(bool ok, int bad) {
  return (ok && !(bad & 1) ? 0 : kStatusBadLen) | (bad & 2 ? kStatusBadPage : 0);
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
  const Path8 r = read_path(P, b);
  const bool ok = lengths_ok(P, r);
  int bad = ok ? look_path(P, r, b, threadIdx.x, kC8Threads) : 0;
  if (__syncthreads_or(bad)) bad = (__syncthreads_or(bad & 1) ? 1 : 0) | (__syncthreads_or(bad & 2) ? 2 : 0);
  if (threadIdx.x == 0) {
    const int status = path_status(ok, bad);
    if (P.status) P.status[b] = status;
    P.new_len[b] = status ? -1 : r.ctx + r.m;
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
// The groups of warps share the units of all requests evenly, each a run of them
// (over a request's layers, blocks and heads), so that each looks at a request's
// lengths and path once for many.
//
// CHECKED: the check kernel has run, and a new length of -1 says that the
// request is bad.  Otherwise every group checks the requests of its units, and
// the one with a request's first unit tells the caller.
//
// Prompts of up to 4096 tokens, 16 layers of 8 heads, take 416 us (6.1 TB/s, 90 % of
// the copy rate); the paths of 64 requests, 28 layers of 4 heads, 27.5 (2.4 TB/s):
// there the start (lengths, path, table, rows, each after the one before) takes a
// third, and a unit of few rows costs what its lookups and scale cost.  CTAs of one
// request each took 498 and 29.5; three CTAs an SM, whose registers spill, 630 and
// 39.  Every CTA adds up the units of all requests, a thread each: 1024 requests of
// such paths over 4 layers take 61 us, 90 when each warp does so by itself.
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
  __shared__ long long warp_units[kC8Warps];
  long long* before = reinterpret_cast<long long*>(smem);  // of each thread, until rows are copied there
  after_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const PageDiv pd(P.page_size), bd(P.block);
  const int W = P.warps, group = warp / W, wsub = warp % W, groups = kC8Warps / W;
  // Requests: their units, and those before each thread's requests.
  Path8 r;
  int first_block = 0, of_layer = 0;  // heads change first: neighbours' rows lie side by side
  auto request = [&](int b) {         // returns the units
    if (CHECKED) {
      r.cu = P.cu[b];
      r.m = P.path_len[b];
      const int len = P.new_len[b];
      r.ctx = len - r.m;
      if (len < 0) r.m = 0;
    } else {
      r = read_path(P, b);
      if (!lengths_ok(P, r)) r.m = -1;
    }
    if (r.m <= 0) return 0ll;
    int last_block, rest;
    bd.split(r.ctx, first_block, rest);
    bd.split(r.ctx + r.m - 1, last_block, rest);
    of_layer = (last_block - first_block + 1) * P.heads * 2;
    return (long long)of_layer * P.layers;
  };
  const int per_thread = (P.B + kC8Threads - 1) / kC8Threads;
  long long mine = 0;
  for (int b = tid * per_thread; b < min(P.B, (tid + 1) * per_thread); ++b) {
    const long long units = request(b);
    mine += units;
    if (!CHECKED && units == 0 && blockIdx.x == 0) {  // nothing to write, or bad
      const int status = path_status(r.m == 0, 0);
      if (P.status) P.status[b] = status;
      P.new_len[b] = status ? -1 : r.ctx;
    }
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) warp_units[warp] = upto;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kC8Warps; ++w) {
    if (w == warp) before[tid] = total + upto - mine;
    total += warp_units[w];
  }
  __syncthreads();
  const long long all = (long long)gridDim.x * groups, at_group = (long long)blockIdx.x * groups + group;
  const long long u_from = div_fast(at_group * total, all), u_to = div_fast((at_group + 1) * total, all);
  // The request of the first unit.
  int b = 0;
  long long first = 0;
  if (u_from < u_to) {
    int own = -1;  // the thread with it
    for (int i = lane; i < kC8Threads; i += 32)
      if (u_from >= before[i] && u_from < (i + 1 < kC8Threads ? before[i + 1] : total)) own = i;
    if (own >= 0) {
      first = before[own];
      for (b = own * per_thread;; ++b) {
        const long long units = request(b);
        if (u_from < first + units) break;
        first += units;
      }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, own >= 0)) - 1;
    b = __shfl_sync(0xffffffffu, b, src);
    first = __shfl_sync(0xffffffffu, first, src);
  }
  __syncthreads();
  if (u_from == u_to) return;  // every warp of the group
  long long units = request(b);
  const int32_t* path = nullptr;
  const int32_t* table = nullptr;
  bool sound = true;
  auto begin = [&](long long u) {  // a request, whose unit u is the group's first
    path = P.path + (long long)b * P.ld_path;
    table = P.table + (long long)b * P.ld_table;
    if (!CHECKED) {
      const int bad = __reduce_or_sync(0xffffffffu, look_path(P, r, b, lane, 32));
      sound = bad == 0;
      if (u == first && wsub == 0 && lane == 0) {
        if (P.status) P.status[b] = path_status(true, bad);
        P.new_len[b] = bad ? -1 : r.ctx + r.m;
      }
    }
  };
  begin(u_from);
  const int per = (P.block + W - 1) / W;        // rows of a warp
  const int w_rows = max(0, min(per, P.block - wsub * per));
  const int passes = (per + kC8Rows - 1) / kC8Rows, steps = passes == 1 ? 1 : 2 * passes;  // of a unit
  const int rsub = lane / LR, ch = (lane % LR) * 8;
  const bool lane_on = rsub < R;
  unsigned char* stage = smem + warp * (S::kStages * S::kBytes);
  const uint32_t stage_at = smem_u32(stage) + lane * 16;
  // The copies: of unit after unit, step after step.
  long long u_ahead = u_from;
  int step_ahead = 0, slot_ahead = 0, q0 = 0, q1 = 0, w0 = 0;
  const T* x = nullptr;
  auto copy = [&]() {
    if (u_ahead < u_to) {
      if (step_ahead == 0) {  // the next unit
        while (u_ahead >= first + units) {  // ends: some request holds unit u_ahead < total
          first += units;
          units = request(++b);
          if (units > 0) begin(u_ahead);
        }
        const long long u = u_ahead - first;
        const int layer = (int)div_fast(u, of_layer), o = (int)(u - (long long)layer * of_layer), kv = o & 1;
        const int j = (int)((uint32_t)(o >> 1) / (uint32_t)P.heads), h = (o >> 1) - j * P.heads;
        const int base = (first_block + j) * P.block;
        w0 = base + wsub * per;
        q0 = max(0, r.ctx - w0);
        q1 = sound ? min(w_rows, r.ctx + r.m - w0) : 0;
        int page, slot, blk, rest2;
        pd.split(base, page, slot);
        bd.split(slot, blk, rest2);
        const int id = sound ? table[page] : 0;
        float* scale = P.scale[kv] + (long long)layer * P.c_layer + (long long)id * P.c_page + (long long)blk * P.c_block +
                       (long long)h * P.c_head;
        x = static_cast<const T*>(P.x[kv]) + (long long)layer * P.sn_layer + (long long)r.cu * P.sn_node +
            (long long)h * P.sn_head + ch;
        C8Unit& n = info[warp][slot_ahead];
        const bool begun = sound && base < r.ctx;
        __syncwarp();  // its last unit has been read
        if (lane == 0) {
          n.scale = scale;
          n.held = P.held[kv] + (long long)layer * P.s_layer + (long long)id * P.s_page +
                   (long long)(slot + wsub * per) * P.s_slot + (long long)h * P.s_head;
          n.q0 = q0;
          n.q1 = q1;
          n.flags = (sound ? 1 : 0) | (begun ? 2 : 0);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&n.old)), "l"(scale), "r"(begun ? 4 : 0)
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
        ++u_ahead;
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
  for (long long u = u_from; u < u_to; ++u, turn ^= 1) {
    C8Unit n;
    float* scale = nullptr;
    uint8_t* held = nullptr;  // row rsub
    bool begun = false;
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
        begun = (n.flags & 2) != 0;
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
    const bool grown = begun && need > old;
    // Of a scale below 2^-126, which a block only keeps where its new tokens are 0,
    // the inverse may be infinite, and 0 times it NaN.
    const float s = begun && !grown ? old : need, inv = s < 0x1p-126f ? 0.f : 1.f / s;
    if ((n.flags & 1) && wsub == 0 && lane == 0 && (!begun || grown)) *scale = s;
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
      const int end = min(w_rows, n.q0);
      constexpr int U = 4;  // loads in flight
      for (int q = rsub; q < end; q += U * R, d += U * row_step) {
        uint2 w[U];
#pragma unroll
        for (int e = 0; e < U; ++e) w[e] = q + e * R < end ? *reinterpret_cast<const uint2*>(d + e * row_step) : make_uint2(0u, 0u);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          uint32_t z[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t y = k ? w[e].y : w[e].x;
            const float2 a = from_e4m3x2(y & 0xffffu), c = from_e4m3x2(y >> 16);
            z[k] = to_e4m3x2(a.x * old * inv, a.y * old * inv) | to_e4m3x2(c.x * old * inv, c.y * old * inv) << 16;
          }
          if (q + e * R < end) *reinterpret_cast<uint2*>(d + e * row_step) = make_uint2(z[0], z[1]);
        }
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

// Longest path that every group checks by itself.  A launch that checks first costs
// 2.2 us (one request 5.4 to 7.6, the batch 27.5 to 29.0); checking prompts of 4096
// tokens over and over 5 (414 to 419).
constexpr int kC8OwnCheck = 256;

}  // namespace

int launch_commit8(Commit8Params& P, bool bf16, int num_sms, cudaStream_t s) {
  const int need = (P.block + kC8Rows - 1) / kC8Rows;
  P.warps = 1;
  while (P.warps < kC8Warps && P.warps < need) P.warps *= 2;
  const long long blocks = (P.ld_path + P.block - 2ll) / P.block + 1, units = blocks * P.heads * 2 * P.layers * P.B;
  const int groups = kC8Warps / P.warps, room = num_sms * (P.dim <= 128 ? 2 : 1);  // CTAs that run at once
  const unsigned ctas = (unsigned)max(1ll, min((long long)room, (units + groups - 1) / groups));
  const bool checked = P.new_len == P.ctx || P.ld_path > kC8OwnCheck;
  if (checked && launch_kernel(commit8_check_kernel, dim3(P.B), kC8Threads, 0, s, P)) return -1;
  const dim3 grid(ctas);
  return bf16 ? launch_commit_dim<__nv_bfloat16>(P, checked, grid, s) : launch_commit_dim<__half>(P, checked, grid, s);
}

}  // namespace sv
