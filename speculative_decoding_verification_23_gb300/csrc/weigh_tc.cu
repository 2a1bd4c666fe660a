// Attention weights on the 5th-generation tensor cores: keys are the lanes of
// tensor memory, so a thread sums its key's weights over all rows by itself.
#include "tc_common.cuh"

namespace sv {
namespace {

constexpr int kWtRows = 128;  // query rows per block
constexpr int kWtThreads = 192;

template <int D, int RB>
struct WeighShape {
  static constexpr int kQBytes = kWtRows * D * 2;
  static constexpr int kSlot = kTcKeys * D * 2;
  static constexpr int kHalf = kTcKeys * 128;
  // keys in flight: half of the shared memory that the queries leave, or a
  // little more, is enough for the copy rate
  static constexpr int kSlots = (222 * 1024 - RB * kQBytes) / kSlot < 8 ? (222 * 1024 - RB * kQBytes) / kSlot : 8;
  static constexpr int kSmem = RB * kQBytes + kSlots * kSlot + 1024;
};

// The weights of requests without rows, by 128 threads: those of before, or 0.
// Units of kIdle keys of a head, over the CTAs in turn; a warp looks at 32
// requests at once.  16 requests of 8 heads and 16384 tokens, every second one
// without rows, 87 us, 103 with rows in all (units of 4096 keys cost 11 us more,
// of 512 one); 1024 of 500 tokens, one without rows, 331 us, 321 with rows in
// all.  Not inlined, the call costs the batch of the comment below 1.5 us,
// whether made or not.
constexpr int kIdle = 1024;
__device__ __forceinline__ void weigh_idle(const TreeParams& P, const float* before, float* out, int tid) {
  const PageDiv pd(P.page_size);
  const int lane = tid & 31;
  long long u = blockIdx.x;  // this CTA's next unit, counted from the request's first
  for (int b0 = 0; b0 < P.B; b0 += 32) {
    int ctx = 0;
    if (b0 + lane < P.B) {
      const TreeReq r = tree_request(P, b0 + lane);
      if (r.ok && r.n == 0) ctx = r.ctx;
    }
    for (unsigned who = __ballot_sync(0xffffffffu, ctx > 0); who; who &= who - 1) {
      const int b = b0 + __ffs(who) - 1, len = __shfl_sync(0xffffffffu, ctx, b - b0);
      const int parts = (len + kIdle - 1) / kIdle;
      const long long units = (long long)P.heads * parts;
      const int32_t* table = P.table + (long long)b * P.ld_table;
      for (; u < units; u += gridDim.x) {
        const int h = (int)(u / parts), lo = (int)(u - (long long)h * parts) * kIdle, hi = min(len, lo + kIdle);
        const long long at = ((long long)b * P.heads + h) * P.ld;
        for (int j0 = lo + tid; j0 < hi; j0 += 4 * 128) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * 128;
            x[i] = 0.f;
            if (j >= hi) continue;
            int page, slot;
            pd.split(j, page, slot);
            const int id = table[page];
            if (before) x[i] = before[at + j];
            if (id < 0 || id >= P.num_pages) x[i] = NAN;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j0 + i * 128 < hi) out[at + j0 + i * 128] = x[i];
        }
      }
      u -= units;
    }
  }
}

// Every CTA has an even share of all tiles of 128 keys (of all key heads of
// all requests), in order, and keeps a head's query rows, up to RB blocks of
// 128, while its tiles last.  Per tile and block of rows
//   S = K Q^T,  w_j += sum_r 2^(scale log2(e) s_jr - log2(e) lse_r),
// with two score buffers in tensor memory.  Warps 0 - 3: one key a thread;
// warp 4 copies key tiles, warp 5 issues products.
//
// Requests without rows have no tiles: the sums wait for the products by a
// segment's scores alone, so with no scores they could complete q_full twice
// while the products still wait for its first phase, and a parity does not
// tell phases apart that are two away.
//
// A key's sum is one thread's, so there are no atomics and no second pass, and
// nothing but the keys, read once, and a float per key moves: the copies bound
// it.  16 requests of up to 16384 tokens, 8 key heads of 128 channels, 36 rows
// per key head: 322 MB in 62 us, 5.2 TB/s (77 % of the copy rate); with 128
// rows the exponentials take over, 87 us.
template <typename T, int D, int RB>
__global__ void __launch_bounds__(kWtThreads, 1)
    weigh_tc_kernel(const TreeParams P, const float* before, const float* row_lse, float* out,
                    const __grid_constant__ CUtensorMap k_map, int box) {
  using S = WeighShape<D, RB>;
  constexpr int HD = D / 64;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[S::kSlots], empty[S::kSlots], s_full[2], s_free[2], q_full, fin;
  __shared__ __align__(16) float lse2[RB * kWtRows];
  __shared__ int last_key[RB * kWtRows];
  __shared__ bool gaps[RB * kWtRows / 32];  // some of 32 rows add nothing
  __shared__ uint32_t tmem_at;
  __shared__ volatile int dead;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* ring = smem + RB * S::kQBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(&tmem_at))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
    }
    mbar_init(&q_full, 128);
    mbar_init(&fin, 1);
    fence_mbar_init();
    dead = 0;
  }
  if (tid == 128) prefetch_map(&k_map);
  wait_previous();
  const TreeScan scan = tree_scan(P, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  start_next();  // not before this CTA has its tensor memory, which a kernel after it may want too
  const uint32_t tmem = uniform(tmem_at);
  TreeWalk walk;
  walk.begin(P, lane, scan, blockIdx.x);
  TreeSeg g;

  if (warp == 4) {
    // ------------------------------------------------------------ copies
    struct Copy {
      int valid, kvh, page, slot;
      bool any;
    };
    RingFills fills;
    const PageDiv pd(P.page_size);
    const int bx = lane / HD, half = lane % HD;
    int t = 0;
    g.t1 = 0;
    auto ahead = [&]() {  // the tile after, its pages looked up
      Copy c;
      c.any = true;
      c.page = c.slot = 0;
      if (t >= g.t1) {
        c.any = walk.next(P, g);
        t = g.t0;
      }
      if (!c.any) return c;
      const int lo = t++ * kTcKeys;
      c.valid = min(kTcKeys, walk.r.ctx - lo);
      c.kvh = g.kvh;
      if (bx * box < c.valid) {
        int page;
        pd.split(lo + bx * box, page, c.slot);
        c.page = P.table[(long long)g.b * P.ld_table + page];
      }
      return c;
    };
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
    Copy cur = ahead();
    while (ok && cur.any) {
      const Copy next = ahead();
      const int nb = (cur.valid + box - 1) / box;
      if (cur.page < 0 || cur.page >= P.num_pages) cur.page = 0;  // its keys' results become NaN
      ok = warp_wait(&empty[s], ph ^ 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(nb * box * 128 * HD));
      fills.note(s, ph);
      __syncwarp();
      if (bx < nb)
        tma_4d(smem_u32(ring) + s * S::kSlot + half * S::kHalf + bx * box * 128, &k_map, half * 64, cur.slot, cur.kvh,
               cur.page, &full[s]);
      if (++s == S::kSlots) {
        s = 0;
        ph ^= 1;
      }
      cur = next;
    }
    if (!ok) {
      dead = 1;
      fills.drain(full, S::kSlots);
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------- products
    const uint32_t one = elect_one();
    const uint64_t dq = smem_desc(smem_u32(smem), 16, 1024), dk = smem_desc(smem_u32(ring), 16, 1024);
    bool ok = true;
    uint32_t q_ph = 0, f_ph = 3, k_ph = 0;  // f_ph: buffers begin free
    int s = 0, buf = 0;
    while (ok && walk.next(P, g)) {
      const int tiles = uniform(g.t1 - g.t0), rows = uniform(walk.r.n * P.group);
      ok = warp_wait(&q_full, q_ph);
      q_ph ^= 1;
      for (int t = 0; ok && t < tiles; ++t) {
        ok = warp_wait(&full[s], k_ph);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const int n32 = min(kWtRows, (rows - rb * kWtRows + 31) & ~31);
          if (n32 <= 0) break;
          ok = ok && warp_wait(&s_free[buf], (f_ph >> buf) & 1);
          if (!ok) break;
          f_ph ^= 1u << buf;
          tc_fence_after();
          const uint32_t id = inst_desc<T>(n32, false);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks / 4) * S::kHalf + (ks % 4) * 32) >> 4;
            mma_ss(tmem + buf * kWtRows, dk + (uint32_t)(s * (S::kSlot >> 4)) + off,
                   dq + (uint32_t)(rb * (S::kQBytes >> 4)) + off, id, ks > 0, one);
          }
          mma_commit(&s_full[buf], one);
          buf ^= 1;
        }
        mma_commit(&empty[s], one);
        if (++s == S::kSlots) {
          s = 0;
          k_ph ^= 1;
        }
      }
    }
    if (!ok) dead = 1;
    mma_commit(&fin, one);
    __syncwarp();
    mbar_wait(&fin, 0);
  } else {
    // ----------------------------------------------------------- the sums
    const PageDiv pd(P.page_size);
    const float inv_group = 1.f / (float)P.group;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    bool ok = true;
    uint32_t s_ph = 0;
    int buf = 0;
    while (ok && walk.next(P, g)) {
      const TreeReq& r = walk.r;
      const int rows = r.n * P.group;
      // the rows, as in the attention kernel; rows are padded to a multiple of
      // 32 with zeros, whose weight is 0
      constexpr int STEP = 1024 / D, N = 8;
      const int ch = tid % (D / 8);
      const T* src = static_cast<const T*>(P.q) + (long long)r.cu * P.sq_node + ch * 8;
#pragma unroll 1
      for (int r0 = tid / (D / 8); r0 < min(RB * kWtRows, (rows + 31) & ~31); r0 += N * STEP) {
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int R = r0 + i * STEP;
          v[i] = make_uint4(0, 0, 0, 0);
          if (R < rows) {
            const int nd = (int)(((float)R + 0.5f) * inv_group);
            v[i] = load16(src + (long long)nd * P.sq_node +
                          (long long)(g.kvh * P.group + R - nd * P.group) * P.sq_head);
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int R = r0 + i * STEP, rr = R % kWtRows;
          if (R < RB * kWtRows)
            *reinterpret_cast<uint4*>(smem + (R / kWtRows) * S::kQBytes + (ch >> 3) * (kWtRows * 128) + rr * 128 +
                                      (((ch & 7) ^ (rr & 7)) << 4)) = v[i];
        }
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const int R = rb * kWtRows + tid;
        float x = INFINITY;
        int last = -1;  // padding and rows of infinite lse see nothing
        if (R < rows) {
          const int nd = (int)(((float)R + 0.5f) * inv_group);
          x = row_lse[(long long)(r.cu + nd) * P.heads * P.group + g.kvh * P.group + R - nd * P.group];
          if (fabsf(x) != INFINITY) last = r.ctx - r.n + nd;
        }
        lse2[R] = x * 1.4426950408889634f;
        last_key[R] = last;
        const bool gap = __any_sync(0xffffffffu, last < 0);
        if (lane == 0) gaps[R / 32] = gap;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&q_full);
      asm volatile("bar.sync 1, 128;" ::: "memory");  // lse2 and last_key, by these four warps alone
      const float* old = before ? before + ((long long)g.b * P.heads + g.kvh) * P.ld : nullptr;
      float* dst = out + ((long long)g.b * P.heads + g.kvh) * P.ld;
      for (int t = g.t0; ok && t < g.t1; ++t) {
        const int j = t * kTcKeys + tid;
        const bool in = j < r.ctx;
        float w0 = 0.f;
        bool bad = false;
        if (in) {
          int page, slot;
          pd.split(j, page, slot);
          const int id = P.table[(long long)g.b * P.ld_table + page];
          bad = id < 0 || id >= P.num_pages;
          if (old) w0 = old[j];
        }
        const bool late = (t + 1) * kTcKeys > r.ctx - r.n;  // some row does not see all of these keys
        float2 w = make_float2(0.f, 0.f), w1 = w;
        for (int rb = 0; rb * kWtRows < rows; ++rb) {
          ok = warp_wait(&s_full[buf], (s_ph >> buf) & 1);
          s_ph ^= 1u << buf;
          if (!ok) break;
          tc_fence_after();
          const int n32 = min(kWtRows, (rows - rb * kWtRows + 31) & ~31);
#pragma unroll 1
          for (int c = 0; c < n32; c += 32) {
            float z[32];
            tmem_ld32(tmem + lanes + buf * kWtRows + c, z);
            tmem_wait_ld();
            loaded(z);
            const float4* l4 = reinterpret_cast<const float4*>(lse2 + rb * kWtRows + c);
            const float2 sc = make_float2(P.scale_log2, P.scale_log2);
            const int* last = last_key + rb * kWtRows + c;
            // four rows' weights; `pick`: only of the rows that see key j
            auto four = [&](int e, bool pick) {
              const float4 l = l4[e / 4];
              float2 a = __ffma2_rn(make_float2(z[e], z[e + 1]), sc, make_float2(-l.x, -l.y));
              float2 b = __ffma2_rn(make_float2(z[e + 2], z[e + 3]), sc, make_float2(-l.z, -l.w));
              if (pick) {
                a.x = j <= last[e] ? a.x : -INFINITY;
                a.y = j <= last[e + 1] ? a.y : -INFINITY;
                b.x = j <= last[e + 2] ? b.x : -INFINITY;
                b.y = j <= last[e + 3] ? b.y : -INFINITY;
              }
              w = __fadd2_rn(w, make_float2(ex2(a.x), ex2(a.y)));
              w1 = __fadd2_rn(w1, make_float2(ex2(b.x), ex2(b.y)));
            };
            const int left = min(kWtRows, rows - rb * kWtRows) - c;
            if (left >= 32 && !late && !gaps[(rb * kWtRows + c) / 32]) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) four(e, false);
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                if (e < left) four(e, true);
            }
          }
          tc_fence_before();
          mbar_arrive(&s_free[buf]);
          buf ^= 1;
        }
        if (in && ok) dst[j] = bad ? NAN : w0 + ((w.x + w.y) + (w1.x + w1.y));
      }
      // Every thread has read this segment's rows' statistics, and its scores
      // are all computed, before the next segment's rows are written.
      // (A wait that ran out ends all four warps here, together.)
      if (!ok) dead = 1;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      ok = ok && !dead;
    }
    if (__any_sync(0xffffffffu, scan.idle)) weigh_idle(P, before, out, tid);
    // zeros past the lengths, NaN for bad requests, and the statuses
    for (long long i = blockIdx.x; i < (long long)P.B * P.heads; i += gridDim.x) {
      const int b = (int)(i / P.heads), h = (int)(i - (long long)b * P.heads);
      const TreeReq r = tree_request(P, b);
      const float v = r.ok ? 0.f : NAN;
      for (int j = (r.ok ? r.ctx : 0) + tid; j < P.ld; j += 128) out[i * P.ld + j] = v;
      if (h == 0 && warp == 0 && P.status) {
        int bad = 0;
        if (r.ok)
          for (long long p = lane; p < ((long long)r.ctx + P.page_size - 1) / P.page_size; p += 32) {
            const int id = P.table[(long long)b * P.ld_table + p];
            bad |= id < 0 || id >= P.num_pages;
          }
        bad = warp_or(bad);
        if (lane == 0) P.status[b] = r.ok ? (bad ? kStatusBadPage : 0) : kStatusBadLen;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
  // a wait that ran out (not expected) leaves results unwritten: say so
  if (dead && P.status)
    for (int b = tid; b < P.B; b += kWtThreads) atomicOr(&P.status[b], kStatusTimeout);
}

template <typename T, int D, int RB>
int launch_tc(const TreeParams& P, const float* before, const float* lse, float* out, const CUtensorMap& map, int box,
              cudaStream_t s) {
  using S = WeighShape<D, RB>;
  if (cudaFuncSetAttribute(weigh_tc_kernel<T, D, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(weigh_tc_kernel<T, D, RB>, dim3(P.grid), kWtThreads, S::kSmem, s, P, before, lse, out, map, box);
}

template <typename T, int D>
int launch_rows(const TreeParams& P, const float* before, const float* lse, float* out, const CUtensorMap& map, int box,
                cudaStream_t s) {
  const int rows = P.max_nodes * P.group;
  return rows <= kWtRows ? launch_tc<T, D, 1>(P, before, lse, out, map, box, s)
                         : launch_tc<T, D, 2>(P, before, lse, out, map, box, s);
}

}  // namespace

// The rows that stay in shared memory.
int weigh_tc_rows() { return 2 * kWtRows; }

int launch_weigh_tc(const TreeParams& P, const float* before, const float* lse, float* out, bool bf16, cudaStream_t s) {
  CUtensorMap map;
  const int box = page_box(P.page_size);
  const cuuint64_t dims[4] = {(cuuint64_t)P.dim, (cuuint64_t)P.page_size, (cuuint64_t)P.heads, (cuuint64_t)P.num_pages};
  const long long st[3] = {P.s_slot, P.s_head, P.s_page};
  const cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1};
  if (!encode(&map, bf16, 4, P.k, dims, st, bx)) return -1;
  if (P.dim == 64)
    return bf16 ? launch_rows<__nv_bfloat16, 64>(P, before, lse, out, map, box, s)
                : launch_rows<__half, 64>(P, before, lse, out, map, box, s);
  return bf16 ? launch_rows<__nv_bfloat16, 128>(P, before, lse, out, map, box, s)
              : launch_rows<__half, 128>(P, before, lse, out, map, box, s);
}

}  // namespace sv
