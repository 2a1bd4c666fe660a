// Attention of drafted trees over a paged cache on the 5th-generation tensor
// cores: tiles of 128 query rows and 128 keys, scores and outputs in tensor
// memory, keys and values staged by TMA straight from their pages.
#include "tc_common.cuh"

namespace sv {
namespace {

constexpr int kUnit = 64;        // keys per unit of the softmax, half a tile
constexpr int kTcRows = 128;     // query rows per tile (lanes of tensor memory)
constexpr int kNewBox = 16;      // drafted tokens per TMA box
// log2: how far a row's maximum may pass its reference.  0, an exact running
// maximum, rescales outputs all the time: chains of 64 requests 89 us against
// 72, trees 112 against 89, two contexts of 128 K tokens 188 against 157.
constexpr float kLazy = 8.f;

template <int D, int NT>
struct TcShape {
  static constexpr int kQBytes = kTcRows * D * 2;
  static constexpr int kSlot = kTcKeys * D * 2;         // one tile of keys or of values
  static constexpr int kHalf = kTcKeys * 128;           // 64 channels of a tile
  static constexpr int kSlots = D == 64 ? 10 : (NT == 1 ? 6 : 5);
  static constexpr int kSmem = NT * kQBytes + kSlots * kSlot + 1024;  // 1024: alignment
  static constexpr int kWarps = 4 * NT + 1 + NT;
  static constexpr int kThreads = 32 * kWarps;
};

struct TcMaps {
  CUtensorMap k, v;        // (channel, slot, head, page)
  CUtensorMap kn, vn;      // (channel, node, head)
};

// Mask bits of drafted keys base .. base + 31 for node i (as tree_bits16).
__device__ __forceinline__ uint32_t tree_bits32(const TreeParams& P, int cu, int n, int i, int base) {
  uint32_t bits;
  if (P.mask) {
    bits = (base >> 5) < P.mask_words ? P.mask[(long long)(cu + i) * P.mask_words + (base >> 5)] : 0u;
  } else {
    const int k = i - base;
    bits = k < 0 ? 0u : (k >= 31 ? 0xffffffffu : (2u << k) - 1u);
  }
  const int left = n - base;
  return left >= 32 ? bits : (left <= 0 ? 0u : bits & ((1u << left) - 1u));
}

// A tile's keys: [lo, lo + valid) of the cached or of the drafted ones, in
// one or two units.
struct TcTile {
  bool cached;
  int lo, valid, n16;
  __device__ __forceinline__ int unit16(int h) const { return min(kUnit, n16 - h * kUnit); }
};
__device__ __forceinline__ TcTile tc_tile(const TreeReq& r, int t) {
  TcTile x;
  x.cached = t < r.ct;
  x.lo = (x.cached ? t : t - r.ct) * kTcKeys;
  x.valid = min(kTcKeys, (x.cached ? r.ctx : r.n) - x.lo);
  x.n16 = (x.valid + 15) & ~15;
  return x;
}

// Adds the infinities and NaN among the drafted values [lo, hi) that a row
// sees to its result, which was computed with zeros in their places: to the
// written row `dst`, or to its partial result (unnormalised: the weight's
// size does not matter).
template <typename T, int D>
__device__ __noinline__ void add_odd(const TreeParams& P, int cu, int n, int node, int kvh, int lo, int hi, T* dst,
                                     float4* part) {
  const uint32_t em = exp_mask<T>();
  for (int j = lo; j < hi; ++j) {
    if (!((tree_bits32(P, cu, n, node, j & ~31) >> (j & 31)) & 1u)) continue;
    const uint16_t* v = static_cast<const uint16_t*>(P.v_new) + (long long)(cu + j) * P.sn_node + (long long)kvh * P.sn_head;
    for (int d = 0; d < D; ++d) {
      const uint32_t b = v[d];
      if ((b & em) != em) continue;
      if (dst) {
        uint16_t* o = reinterpret_cast<uint16_t*>(dst + d);
        *o = (uint16_t)(pack2<T>(half_to_f32<T>(*o) + half_to_f32<T>(b), 0.f) & 0xffffu);
      } else {
        reinterpret_cast<float*>(part + (long long)(d / 4) * P.rows)[d & 3] += half_to_f32<T>(b);
      }
    }
  }
}

// Warps 0 .. 4 NT - 1: one query row a thread (the softmax); then one warp
// that copies tiles, and for each row tile one that issues its products.
//
// For every staged tile and each of the NT tiles of rows:
//   S = Q K^T (both from shared memory), by 64 keys the softmax by the row's
//   thread, P in 16 bits over the scores read, O += P V (P from tensor
//   memory), so that the products of one half run during the softmax of the
//   other.
// With NT = 1 there are two score buffers, and the next tile's scores are
// computed ahead, 128 keys at once.  With NT = 2 the row tiles share a staged
// tile, and each has one buffer: the next tile's scores take its halves one
// by one.
//
// What bounds it.  With NT = 1 the copies: two contexts of 128 K tokens take
// 157 us in all, 92 % of the copy rate.  64 requests' chains of up to 9 tokens,
// 63 rows per key head, take 72 us, 62 %; of a CTA's 123 thousand cycles (the
// slowest one's 136) 99 go to its 31.5 tiles, near the copy rate, 9 to loading
// the queries of its 2.9 segments, 6 to their ends and 5 to the start, and the
// joining kernel comes after.  With NT = 2, 16 requests' trees of up to 64
// nodes, 89 us, 760 TFLOP/s: of 143 thousand cycles (the slowest 158) 113 go to
// 33 tiles of 256 rows and 128 keys, 1.7 us each, of which 15 wait for scores
// (the copies alone would take 1.5 us a tile), 13 to queries, 8 to segments'
// ends and 4 to the start; the launch and the joining kernel take the rest.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(TcShape<D, NT>::kThreads, 1)
    tree_tc_kernel(const TreeParams P, const __grid_constant__ TcMaps maps, int box) {
  using S = TcShape<D, NT>;
  constexpr int HD = D / 64;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[S::kSlots], empty[S::kSlots], q_full[NT], s_full[4], p_ready[4], o_half[NT], o_done[NT],
      o_last[NT], fin[NT], seg_end;
  __shared__ uint32_t tmem_at;
  // the last segments with a bad page (the copies run at most kSlots / 2
  // segments ahead) and with infinities or NaN among the drafted values
  __shared__ volatile int bad_seg[16], odd_seg[2], dead;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* ring = smem + NT * S::kQBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);

  if (warp == 4 * NT + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_at))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NT);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 128);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&o_half[i], 1);
      mbar_init(&fin[i], 1);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_last[i], 1);
    }
    mbar_init(&seg_end, NT * 128);
    fence_mbar_init();
    for (int i = 0; i < 16; ++i) bad_seg[i] = -1;
    odd_seg[0] = odd_seg[1] = -1;
    dead = 0;
  }
  if (warp == 4 * NT && lane < 4) prefetch_map(lane == 0 ? &maps.k : lane == 1 ? &maps.v : lane == 2 ? &maps.kn : &maps.vn);
  wait_previous();
  const TreeScan scan = tree_scan(P, lane);
  if (blockIdx.x == 0 && warp == 0) tree_store_starts(P, scan, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  start_next();  // not before this CTA has its tensor memory, which a kernel after it may want too
  const uint32_t tmem = uniform(tmem_at);
  TreeWalk walk;
  walk.begin(P, lane, scan, blockIdx.x);
  TreeSeg g;
  int tc = 0;  // tiles so far: the ring holds keys of tile i as fill 2i, values as 2i + 1

  if (warp == 4 * NT) {
    // ------------------------------------------------------------ copies
    // A lane has one box of a tile (at most 16 boxes of 8 slots or more, HD
    // halves each).  The pages of the tile ahead are looked up before this
    // one is copied, also where it is the first of another segment.
    struct Copy {
      TcTile x;
      int kvh, row, seg, page, slot;  // row: of the first drafted token
      bool any;
    };
    RingFills fills;
    const PageDiv pd(P.page_size);
    const int bx = lane / HD, half = lane % HD;
    int seg = -1, t = 0;
    g.t1 = 0;
    auto ahead = [&]() {
      Copy c;
      c.any = true;
      c.page = c.slot = 0;
      if (t >= g.t1) {
        c.any = walk.next(P, g);
        ++seg;
        t = g.t0;
      }
      if (!c.any) return c;
      c.x = tc_tile(walk.r, t++);
      c.kvh = g.kvh;
      c.seg = seg;
      c.row = walk.r.cu + c.x.lo;
      if (c.x.cached && bx * box < c.x.valid) {
        int page;
        pd.split(c.x.lo + bx * box, page, c.slot);
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
      const int rows = cur.x.cached ? box : kNewBox, nb = (cur.x.valid + rows - 1) / rows;
      const uint32_t bytes = (uint32_t)(nb * rows * 128 * HD);
      if (cur.page < 0 || cur.page >= P.num_pages) {
        cur.page = 0;
        bad_seg[cur.seg & 15] = cur.seg;
      }
      __syncwarp();
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        ok = ok && warp_wait(&empty[s], ph ^ 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
        fills.note(s, ph);
        __syncwarp();
        if (bx < nb) {
          const uint32_t at = smem_u32(ring) + s * S::kSlot + half * S::kHalf + bx * rows * 128;
          if (cur.x.cached)
            tma_4d(at, kv ? &maps.v : &maps.k, half * 64, cur.slot, cur.kvh, cur.page, &full[s]);
          else
            tma_3d(at, kv ? &maps.vn : &maps.kn, half * 64, cur.row + bx * rows, cur.kvh, &full[s]);
        }
        if (++s == S::kSlots) {
          s = 0;
          ph ^= 1;
        }
      }
      cur = next;
    }
    if (!ok) {
      dead = 1;
      fills.drain(full, S::kSlots);
    }
  } else if (warp > 4 * NT) {
    // ---------------------------------------------------------- products
    // One warp issues everything of row tile w.  It has little time for a
    // unit of 64 keys, so slots and phases are counted, not computed, and what
    // descriptors depend on is uniform.
    const int w = warp - (4 * NT + 1);
    const uint32_t one = elect_one();
    bool ok = true;
    uint32_t p_ph = 0, q_ph = 0;           // phases (p_ph: a bit per unit buffer)
    int ks_ = 0, vs_ = 1;                  // next slots of keys and of values
    uint32_t k_ph = 0, v_ph = 0;           // and their phases
    const uint64_t da = smem_desc(smem_u32(smem) + w * S::kQBytes, 16, 1024);
    const uint64_t dk = smem_desc(smem_u32(ring), 16, 1024), dv = smem_desc(smem_u32(ring), S::kHalf, 1024);
    const uint32_t o = tmem + 2 * kTcKeys + w * D, id_v = inst_desc<T>(D, true);
    while (ok && walk.next(P, g)) {
      const int t0 = uniform(g.t0), t1 = uniform(g.t1);
      TreeReq r;
      r.ct = uniform(walk.r.ct);
      r.ctx = uniform(walk.r.ctx);
      r.n = uniform(walk.r.n);
      ok = warp_wait(&q_full[w], q_ph);
      q_ph ^= 1;
      // Scores of a tile: with one row tile, 128 keys at once into one of two
      // buffers; with two, 64 keys (half h) as soon as the weights there have
      // been used.
      auto scores = [&](int t, int h) {
        const int n16 = tc_tile(r, t).n16, buf = NT == 1 ? (t - t0) & 1 : w;
        const uint32_t id = inst_desc<T>(NT == 1 ? n16 : min(kUnit, n16 - h * kUnit), false);
        const uint64_t db = dk + (uint32_t)(ks_ * (S::kSlot >> 4) + h * ((kUnit * 128) >> 4));
        if (h == 0) ok = ok && warp_wait(&full[ks_], k_ph);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks / 4) * S::kHalf + (ks % 4) * 32) >> 4;
          mma_ss(tmem + buf * kTcKeys + h * kUnit, da + off, db + off, id, ks > 0, one);
        }
        mma_commit(&s_full[buf * 2 + h], one);
        if (NT == 1 || h == 1 || n16 <= kUnit) {
          mma_commit(&empty[ks_], one);
          ks_ += 2;
          if (ks_ >= S::kSlots) {
            ks_ -= S::kSlots;
            k_ph ^= 1;
          }
        }
      };
      scores(t0, 0);
      if (NT == 1 && t0 + 1 < t1) scores(t0 + 1, 0);
      if (NT == 2 && tc_tile(r, t0).n16 > kUnit) scores(t0, 1);
      for (int t = t0; ok && t < t1; ++t) {
        const int n16 = tc_tile(r, t).n16, buf = NT == 1 ? (t - t0) & 1 : w;
        const uint64_t db = dv + (uint32_t)(vs_ * (S::kSlot >> 4));
        const uint32_t p = tmem + buf * kTcKeys;
        ok = warp_wait(&full[vs_], v_ph) && warp_wait(&p_ready[buf * 2], (p_ph >> (buf * 2)) & 1);
        if (!ok) break;
        tc_fence_after();
        if (n16 >= kUnit) {
#pragma unroll
          for (int ks = 0; ks < kUnit / 16; ++ks)
            mma_ts(o, p + ks * 8, db + ks * (2048 >> 4), id_v, ks > 0 || t > t0, one);
        } else {
          for (int ks = 0; ks < n16 / 16; ++ks) mma_ts(o, p + ks * 8, db + ks * (2048 >> 4), id_v, ks > 0 || t > t0, one);
        }
        mma_commit(&o_half[w], one);
        if (NT == 2 && t + 1 < t1) scores(t + 1, 0);
        p_ph ^= 1u << (buf * 2);
        if (n16 > kUnit) {
          ok = ok && warp_wait(&p_ready[buf * 2 + 1], (p_ph >> (buf * 2 + 1)) & 1);
          if (!ok) break;
          tc_fence_after();
          if (n16 == kTcKeys) {
#pragma unroll
            for (int ks = 4; ks < 8; ++ks) mma_ts(o, p + 32 + ks * 8, db + ks * (2048 >> 4), id_v, true, one);
          } else {
            for (int ks = 4; ks < n16 / 16; ++ks) mma_ts(o, p + 32 + ks * 8, db + ks * (2048 >> 4), id_v, true, one);
          }
          p_ph ^= 2u << (buf * 2);
        }
        mma_commit(&o_done[w], one);  // before the scores that the softmax takes for a sign of it
        mma_commit(&empty[vs_], one);
        if (NT == 1 && t + 2 < t1) scores(t + 2, 0);
        if (NT == 2 && t + 1 < t1 && tc_tile(r, t + 1).n16 > kUnit) scores(t + 1, 1);
        if (t == t1 - 1) mma_commit(&o_last[w], one);
        vs_ += 2;
        if (vs_ >= S::kSlots) {
          vs_ -= S::kSlots;
          v_ph ^= 1;
        }
      }
    }
    if (!ok) dead = 1;
    mma_commit(&fin[w], one);
    __syncwarp();
    mbar_wait(&fin[w], 0);  // every product has ended before tensor memory is freed
  } else if (warp < 4 * NT) {
    // ----------------------------------------------------------- softmax
    const int w = warp >> 2, row = (warp & 3) * 32 + lane, wtid = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_at = tmem + lanes + 2 * kTcKeys + w * D;
    unsigned char* qs = smem + w * S::kQBytes;
    uint32_t s_ph = 0;  // a bit per buffer
    // node of a row: exact, as rows are at most 2^20 and half a row from a multiple
    const float inv_group = 1.f / (float)P.group;
    bool ok = true;
    for (int seg = 0; ok && walk.next(P, g); ++seg) {
      const TreeReq& r = walk.r;
      const int row_lo = g.m * (NT * kTcRows) + w * kTcRows;
      const int nrows = min(kTcRows, r.n * P.group - row_lo);  // may be <= 0
      // This tile's query rows, swizzled as TMA would: 8 rows of 128 bytes a
      // pattern.  A thread copies one 16-byte piece of every (1024 / D)-th
      // row, all its loads in flight at once.
      constexpr int STEP = 1024 / D, N = kTcRows / STEP;
      const int ch = wtid % (D / 8);
      const T* src = static_cast<const T*>(P.q) + (long long)r.cu * P.sq_node + ch * 8;
#pragma unroll 1
      for (int r0 = wtid / (D / 8); r0 < kTcRows; r0 += N * STEP) {
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int rr = r0 + i * STEP, R = row_lo + rr;
          v[i] = make_uint4(0, 0, 0, 0);
          if (rr < nrows) {
            const int nd = (int)(((float)R + 0.5f) * inv_group);
            v[i] = load16(src + (long long)nd * P.sq_node +
                          (long long)(g.kvh * P.group + R - nd * P.group) * P.sq_head);
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int rr = r0 + i * STEP;
          *reinterpret_cast<uint4*>(qs + (ch >> 3) * (kTcRows * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v[i];
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&q_full[w]);
      const bool mine = row < nrows;
      const bool any = (warp & 3) * 32 < nrows;  // warp-uniform
      const int R = row_lo + (mine ? row : 0);
      const int node = mine ? (int)(((float)R + 0.5f) * inv_group) : 0;
      float m = -INFINITY;                 // the row's reference, log2 units
      float2 l2 = make_float2(0.f, 0.f), l3 = l2;  // its sum of 2^(s - m)
      float fix = 0.f;                     // the rounding of the largest weights in it
      for (int t = g.t0; ok && t < g.t1; ++t, ++tc) {
        const TcTile x = tc_tile(r, t);
        uint32_t see[4];
        if (!x.cached && any) {
#pragma unroll
          for (int c = 0; c < 4; ++c) see[c] = tree_bits32(P, r.cu, r.n, node, x.lo + c * 32);
        }
        // Values past the end of a tile's keys, whatever the slots hold, are
        // zero for the product, and so are infinities and NaN among drafted
        // values: a row that does not see them would get 0 times them.
        // Both row tiles' threads see to it before their own weights are ready,
        // writing the same zeros.
        if ((x.valid & 15) || !x.cached) {
          const int f = 2 * tc + 1, s = f % S::kSlots;
          ok = warp_wait(&full[s], (f / S::kSlots) & 1);
          unsigned char* vs = ring + s * S::kSlot;
          const uint32_t em = exp_mask<T>();
          bool odd = false;
          for (int i = (x.cached ? x.valid & ~15 : 0) * (D / 8) + wtid; i < x.n16 * (D / 8); i += 128) {
            const int j = i / (D / 8), ch = i % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(vs + (ch >> 3) * S::kHalf + j * 128 + (((ch & 7) ^ (j & 7)) << 4));
            if (j >= x.valid) {
              *at = make_uint4(0, 0, 0, 0);
            } else if (!x.cached) {
              uint4 v = *at;
              uint32_t* e = reinterpret_cast<uint32_t*>(&v);
              bool hit = false;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if ((e[c] & em) == em) {
                  e[c] &= 0xffff0000u;
                  hit = true;
                }
                if (((e[c] >> 16) & em) == em) {
                  e[c] &= 0xffffu;
                  hit = true;
                }
              }
              if (hit) {
                *at = v;
                odd = true;
              }
            }
          }
          if (odd) odd_seg[seg & 1] = seg;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        const int buf = NT == 1 ? (t - g.t0) & 1 : w;
#pragma unroll 1
        for (int h = 0; h * kUnit < x.n16; ++h) {
          if (NT == 2 || h == 0) {
            ok = ok && warp_wait(&s_full[buf * 2 + h], (s_ph >> (buf * 2 + h)) & 1);
            s_ph ^= 1u << (buf * 2 + h);
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t s_at = tmem + lanes + buf * kTcKeys + h * kUnit;
          if (any) {
            float z[kUnit];
            tmem_ld32(s_at, z);
            tmem_ld32(s_at + 32, z + 32);
            tmem_wait_ld();
            loaded(z);
            loaded(z + 32);
            if (x.valid < kTcKeys || !x.cached) {  // -inf where the row sees nothing
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int left = x.valid - h * kUnit - c * 32;
                const uint32_t old = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
                const uint32_t bits = x.cached ? old : (h == 0 ? see[c] : see[2 + c]);
#pragma unroll
                for (int e = 0; e < 32; ++e) z[c * 32 + e] = (bits >> e) & 1u ? z[c * 32 + e] : -INFINITY;
              }
            }
            float top[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = fmaxf(z[2 * k], z[2 * k + 1]);
#pragma unroll
            for (int e = 8; e < kUnit; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], z[e + 2 * k]), z[e + 2 * k + 1]);
            // the scale is positive
            const float zx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), mx = zx * P.scale_log2;
            // The reference follows the maximum only where it falls more than
            // 2^8 behind (or has none yet): weights up to 2^8 are exact in
            // fp32 sums and in range of both 16-bit types.
            const bool move = mx > m + kLazy || (m == -INFINITY && mx > -INFINITY);
            if (__any_sync(0xffffffffu, move)) {
              const float f = move ? (m == -INFINITY ? 0.f : ex2(m - mx)) : 1.f;
              if (move) {
                m = mx;
                l2.x *= f;
                l2.y *= f;
                l3.x *= f;
                l3.y *= f;
                fix *= f;
              }
              if (t > g.t0 || h > 0) {
                // The unit before is in O.  The scores here came after the
                // products of the tile two before, and o_half follows o_done,
                // so each of these barriers is at most one phase behind, which
                // is all that a parity tells.
                if (tc > 0) ok = warp_wait(&o_done[w], (tc - 1) & 1);
                if (h > 0) ok = ok && warp_wait(&o_half[w], tc & 1);
                if (!ok) break;
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {  // 16 at a time, beside the 64 scores
                  uint32_t o[16];
                  tmem_ld16(o_at + c * 16, o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(o_at + c * 16, o);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const float2 sc = make_float2(P.scale_log2, P.scale_log2), nr = make_float2(-ref, -ref);
            // Where one key takes most of a row, the rounding of its weight
            // for the product is the row's error (with the reference at the
            // maximum it is 1, and exact).  So outputs are divided by a sum
            // that holds each unit's largest weight as rounded; the others'
            // roundings average out.
            const float px = ex2(fmaf(zx, P.scale_log2, -ref));
            fix += half_to_f32<T>(pack2<T>(px, 0.f) & 0xffffu) - px;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float* y = z + c * 32 + e;
                const float2 a = __ffma2_rn(make_float2(y[0], y[1]), sc, nr);
                const float2 b = __ffma2_rn(make_float2(y[2], y[3]), sc, nr);
                const float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
                l2 = __fadd2_rn(l2, ea);
                l3 = __fadd2_rn(l3, eb);
                p[e / 2] = pack2<T>(ea.x, ea.y);
                p[e / 2 + 1] = pack2<T>(eb.x, eb.y);
              }
              tmem_st16(s_at + c * 16, p);
            }
            tc_wait_st();
          }
          tc_fence_before();
          mbar_arrive(&p_ready[buf * 2 + h]);
        }
      }
      if (!ok) break;
      // o_done may be two phases behind here: the segment's last product has a
      // barrier of its own
      ok = warp_wait(&o_last[w], seg & 1);
      if (!ok) break;
      tc_fence_after();
      if (NT > 1) {  // odd_seg may be written by either row tile's threads
        mbar_arrive(&seg_end);
        ok = warp_wait(&seg_end, seg & 1);
        if (!ok) break;
      }
      if (!any) continue;
      const bool poison = bad_seg[seg & 15] == seg, odd = odd_seg[seg & 1] == seg;
      const bool whole = g.t0 == 0 && g.t1 == r.per_item;
      const int slot = 2 * blockIdx.x + tree_slot(g.t0 == 0);
      float l = (l2.x + l2.y) + (l3.x + l3.y);
      if (poison) l = NAN;
      const float inv = l == 0.f ? 0.f : 1.f / (l + fix);
      const int head = g.kvh * P.group + R - node * P.group;
      T* dst = static_cast<T*>(P.out) + (long long)(r.cu + node) * P.so_node + (long long)head * P.so_head;
      const long long prow = (long long)slot * P.rows + w * kTcRows + row;
      float4* part = reinterpret_cast<float4*>(P.part_o) + (long long)slot * P.rows * (D / 4) + w * kTcRows + row;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        __syncwarp();
        tmem_ld32(o_at + c * 32, o);
        tmem_wait_ld();
        loaded(o);
        if (mine && whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 v;
            v.x = pack2<T>(o[e] * inv, o[e + 1] * inv);
            v.y = pack2<T>(o[e + 2] * inv, o[e + 3] * inv);
            v.z = pack2<T>(o[e + 4] * inv, o[e + 5] * inv);
            v.w = pack2<T>(o[e + 6] * inv, o[e + 7] * inv);
            *reinterpret_cast<uint4*>(dst + c * 32 + e) = v;
          }
        } else if (mine) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            part[(c * 8 + e / 4) * P.rows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (mine) {
        if (odd)
          add_odd<T, D>(P, walk.r.cu, walk.r.n, node, g.kvh, max(0, g.t0 - walk.r.ct) * kTcKeys,
                        min(walk.r.n, (g.t1 - walk.r.ct) * kTcKeys), whole ? dst : nullptr, part);
        const float ref = m == -INFINITY ? 0.f : m;
        if (!whole)
          P.part_ml[prow] = make_float4(m, l, l + fix, 0.f);
        else if (P.lse)
          P.lse[(long long)(r.cu + node) * P.heads * P.group + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
      }
      __syncwarp();
      tc_fence_before();
    }
    if (!ok) dead = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) P.failed[blockIdx.x] = dead;
  if (warp == 4 * NT + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <typename T, int D, int NT>
int launch_tc(const TreeParams& P, const TcMaps& maps, int box, cudaStream_t s) {
  using S = TcShape<D, NT>;
  if (cudaFuncSetAttribute(tree_tc_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(tree_tc_kernel<T, D, NT>, dim3(P.grid), S::kThreads, S::kSmem, s, P, maps, box);
}

template <typename T>
int launch_tc_shape(const TreeParams& P, const TcMaps& maps, int box, cudaStream_t s) {
  const int nt = P.rows / kTcRows;
  if (P.dim == 64) return nt == 1 ? launch_tc<T, 64, 1>(P, maps, box, s) : launch_tc<T, 64, 2>(P, maps, box, s);
  return nt == 1 ? launch_tc<T, 128, 1>(P, maps, box, s) : launch_tc<T, 128, 2>(P, maps, box, s);
}

}  // namespace

// Heads of 64 or 128 channels, pages of a multiple of 8 slots (a box of a
// TMA copy fills whole swizzle patterns of 8 rows).
bool tree_tc_fits(int dim, int page_size) { return (dim == 64 || dim == 128) && page_size % 8 == 0; }

TreePlan plan_tree_tc(int rows, int num_sms) {
  TreePlan p;
  p.kernel = 1;
  p.grid = num_sms;
  // Two row tiles where there are more rows than one has: 256 rows of 16
  // requests 89 us against 118 with one (which reads the cache twice), 160
  // rows 76 against 93; 63 rows of 64 requests 76 us against 72 with one.
  p.rows = rows > kTcRows ? 2 * kTcRows : kTcRows;
  p.kt = kTcKeys;
  return p;
}

int launch_tree_tc(const TreeParams& P, bool bf16, cudaStream_t s) {
  TcMaps maps;
  const int box = page_box(P.page_size);
  const cuuint64_t dims[4] = {(cuuint64_t)P.dim, (cuuint64_t)P.page_size, (cuuint64_t)P.heads, (cuuint64_t)P.num_pages};
  const long long st[3] = {P.s_slot, P.s_head, P.s_page};
  const cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1};
  const cuuint64_t ndims[3] = {(cuuint64_t)P.dim, (cuuint64_t)P.total, (cuuint64_t)P.heads};
  const long long nst[2] = {P.sn_node, P.sn_head};
  const cuuint32_t nbx[3] = {64, kNewBox, 1};
  if (!encode(&maps.k, bf16, 4, P.k, dims, st, bx) || !encode(&maps.v, bf16, 4, P.v, dims, st, bx) ||
      !encode(&maps.kn, bf16, 3, P.k_new, ndims, nst, nbx) || !encode(&maps.vn, bf16, 3, P.v_new, ndims, nst, nbx))
    return -1;
  return bf16 ? launch_tc_shape<__nv_bfloat16>(P, maps, box, s) : launch_tc_shape<__half>(P, maps, box, s);
}

}  // namespace sv
