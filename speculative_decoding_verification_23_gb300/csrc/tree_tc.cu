// Attention of drafted trees over a paged cache on the 5th-generation tensor
// cores: tiles of 128 query rows and 128 keys, scores and outputs in tensor
// memory, keys and values staged by TMA straight from their pages.
#include <cuda.h>

#include "tree_common.cuh"

namespace sv {
namespace {

constexpr int kTcKeys = 128;     // keys per tile
constexpr int kTcRows = 128;     // query rows per tile (lanes of tensor memory)
constexpr int kNewBox = 16;      // drafted tokens per TMA box
constexpr float kLazy = 8.f;     // log2: how far a row's maximum may pass its reference

template <int D, int NT>
struct TcShape {
  static constexpr int kQBytes = kTcRows * D * 2;
  static constexpr int kSlot = kTcKeys * D * 2;         // one tile of keys or of values
  static constexpr int kHalf = kTcKeys * 128;           // 64 channels of a tile
  static constexpr int kSlots = D == 64 ? 10 : (NT == 1 ? 6 : 5);
  static constexpr int kSmem = NT * kQBytes + kSlots * kSlot + 1024;  // 1024: alignment
  static constexpr int kWarps = 4 * NT + 2;
  static constexpr int kThreads = 32 * kWarps;
};

struct TcMaps {
  CUtensorMap k, v;        // (channel, slot, head, page)
  CUtensorMap kn, vn;      // (channel, node, head)
};

// --------------------------------------------------------------- tcgen05
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  // 128-byte swizzle (2 at bit 61), descriptor version 1 (bit 46)
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// fp32 accumulation, 16-bit operands; `vmajor`: B's rows are its K axis.
template <typename T>
__device__ __forceinline__ uint32_t inst_desc(int n, bool vmajor);
template <>
__device__ __forceinline__ uint32_t inst_desc<__nv_bfloat16>(int n, bool vmajor) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((vmajor ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
template <>
__device__ __forceinline__ uint32_t inst_desc<__half>(int n, bool vmajor) {
  return (1u << 4) | ((vmajor ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes; the wait is part of the load, so that
// no use of a register can move before it.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
      "%31,%32};" ::"r"(addr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]),
      "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]),
      "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// A bounded wait of a whole warp, with one outcome for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

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

// A tile's keys: [lo, lo + valid) of the cached or of the drafted ones.
struct TcTile {
  bool cached;
  int lo, valid, n16;
};
__device__ __forceinline__ TcTile tc_tile(const TreeReq& r, int t) {
  TcTile x;
  x.cached = t < r.ct;
  x.lo = (x.cached ? t : t - r.ct) * kTcKeys;
  x.valid = min(kTcKeys, (x.cached ? r.ctx : r.n) - x.lo);
  x.n16 = (x.valid + 15) & ~15;
  return x;
}

// Warps 0 .. 4 NT - 1: one query row a thread (the softmax); then one warp
// that copies tiles, one whose first lane issues the products.
//
// The unit of work is a tile of keys for one of the NT tiles of rows.  Units
// alternate between two score buffers in tensor memory:
//   S = Q K^T (both from shared memory), softmax by the row's thread, P in
//   16 bits over S's first columns, O += P V (P from tensor memory).
// With NT = 2 a buffer belongs to a row tile, and both use a staged tile;
// with NT = 1 the scores of the next tile are computed during the softmax.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(TcShape<D, NT>::kThreads, 1)
    tree_tc_kernel(const TreeParams P, const __grid_constant__ TcMaps maps, int box) {
  using S = TcShape<D, NT>;
  constexpr int HD = D / 64;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[S::kSlots], empty[S::kSlots], q_full, s_full[2], p_ready[2], o_done[NT], seg_end, fin;
  __shared__ uint32_t tmem_at;
  // the last segments with a bad page (the copies run at most kSlots / 2
  // segments ahead) and with infinities or NaN among the drafted values
  __shared__ volatile int bad_seg[16], odd_seg[2], dead;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* ring = smem + NT * S::kQBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (warp == 4 * NT + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_at))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&q_full, NT * 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 128);
    }
    for (int i = 0; i < NT; ++i) mbar_init(&o_done[i], 1);
    mbar_init(&seg_end, NT * 128);
    mbar_init(&fin, 1);
    fence_mbar_init();
    for (int i = 0; i < 16; ++i) bad_seg[i] = -1;
    odd_seg[0] = odd_seg[1] = -1;
    dead = 0;
  }
  const TreeScan scan = tree_scan(P, lane);
  if (blockIdx.x == 0 && warp == 0) tree_store_starts(P, scan, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  TreeWalk walk;
  walk.begin(P, lane, scan, blockIdx.x);
  TreeSeg g;
  int tc = 0;  // tiles so far: the ring holds keys of tile i as fill 2i, values as 2i + 1

  if (warp == 4 * NT) {
    // ------------------------------------------------------------ copies
    RingFills fills;
    const PageDiv pd(P.page_size);
    bool ok = true;
    for (int seg = 0; ok && walk.next(P, g); ++seg) {
      for (int t = g.t0; ok && t < g.t1; ++t, ++tc) {
        const TcTile x = tc_tile(g.r, t);
        const int rows = x.cached ? box : kNewBox, nb = (x.valid + rows - 1) / rows;
        const uint32_t bytes = (uint32_t)(nb * rows * 128 * HD);
        // boxes of a tile by lane (at most 16 boxes of 8 slots, HD halves each)
        int page[2], slot[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = e * 32 + lane, bx = i / HD;
          page[e] = slot[e] = 0;
          if (bx < nb && x.cached) {
            pd.split(x.lo + bx * rows, page[e], slot[e]);
            page[e] = P.table[(long long)g.b * P.ld_table + page[e]];
            if (page[e] < 0 || page[e] >= P.num_pages) {
              page[e] = 0;
              bad_seg[seg & 15] = seg;
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int f = 2 * tc + kv, s = f % S::kSlots, ph = (f / S::kSlots) & 1;
          ok = ok && warp_wait(&empty[s], ph ^ 1);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
          fills.note(s, ph);
          __syncwarp();
          const uint32_t dst = smem_u32(ring + s * S::kSlot);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = e * 32 + lane, bx = i / HD, half = i % HD;
            if (bx < nb) {
              const uint32_t at = dst + half * S::kHalf + bx * rows * 128;
              if (x.cached)
                tma_4d(at, kv ? &maps.v : &maps.k, half * 64, slot[e], g.kvh, page[e], &full[s]);
              else
                tma_3d(at, kv ? &maps.vn : &maps.kn, half * 64, g.r.cu + x.lo + bx * rows, g.kvh, &full[s]);
            }
          }
        }
      }
    }
    if (!ok) {
      dead = 1;
      fills.drain(full, S::kSlots);
    }
  } else if (warp == 4 * NT + 1) {
    // ---------------------------------------------------------- products
    bool ok = true;
    uint32_t p_ph[2] = {0, 0}, q_ph = 0;
    const uint32_t q_at = smem_u32(smem), r_at = smem_u32(ring);
    while (ok && walk.next(P, g)) {
      const int tiles = g.t1 - g.t0, units = tiles * NT;
      ok = warp_wait(&q_full, q_ph);
      q_ph ^= 1;
      tc_fence_after();
      auto wait_full = [&](int f) { return warp_wait(&full[f % S::kSlots], (f / S::kSlots) & 1); };
      auto scores = [&](int u) {
        const int i = u / NT, w = NT == 1 ? 0 : u & 1, f = 2 * (tc + i), s = f % S::kSlots;
        if (w == 0) {
          ok = ok && wait_full(f);
          tc_fence_after();
        }
        if (!ok) return;
        if (lane == 0) {
          const TcTile x = tc_tile(g.r, g.t0 + i);
          const uint32_t id = inst_desc<T>(x.n16, false);
          const uint32_t a = q_at + w * S::kQBytes, b = r_at + s * S::kSlot;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks / 4) * S::kHalf + (ks % 4) * 32;
            mma_ss(tmem + (u & 1) * kTcKeys, smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), id, ks > 0);
          }
          mma_commit(&s_full[u & 1]);
          if (w == NT - 1) mma_commit(&empty[s]);
        }
        __syncwarp();
      };
      scores(0);
      if (units > 1) scores(1);
      for (int u = 0; ok && u < units; ++u) {
        const int i = u / NT, w = NT == 1 ? 0 : u & 1, f = 2 * (tc + i) + 1, s = f % S::kSlots;
        ok = warp_wait(&p_ready[u & 1], p_ph[u & 1]);
        p_ph[u & 1] ^= 1;
        if (w == 0) ok = ok && wait_full(f);
        tc_fence_after();
        if (!ok) break;
        if (lane == 0) {
          const TcTile x = tc_tile(g.r, g.t0 + i);
          const uint32_t id = inst_desc<T>(D, true);
          const uint32_t o = tmem + 2 * kTcKeys + w * D, p = tmem + (u & 1) * kTcKeys, v = r_at + s * S::kSlot;
          for (int ks = 0; ks < x.n16 / 16; ++ks)
            mma_ts(o, p + ks * 8, smem_desc(v + ks * 2048, S::kHalf, 1024), id, i > 0 || ks > 0);
          mma_commit(&o_done[w]);
          if (w == NT - 1) mma_commit(&empty[s]);
        }
        __syncwarp();
        if (u + 2 < units) scores(u + 2);
      }
      tc += tiles;
    }
    if (!ok) dead = 1;
    if (lane == 0) mma_commit(&fin);
    __syncwarp();
    mbar_wait(&fin, 0);  // every product has ended before tensor memory is freed
  } else {
    // ----------------------------------------------------------- softmax
    const int w = warp >> 2, row = (warp & 3) * 32 + lane, wtid = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_at = tmem + lanes + 2 * kTcKeys + w * D;
    unsigned char* qs = smem + w * S::kQBytes;
    uint32_t s_ph[2] = {0, 0};
    uint32_t o_n = 0;  // products on this tile's output so far
    bool ok = true;
    for (int seg = 0; ok && walk.next(P, g); ++seg) {
      const TreeReq& r = g.r;
      const int row_lo = g.m * (NT * kTcRows) + w * kTcRows;
      const int nrows = min(kTcRows, r.n * P.group - row_lo);  // may be <= 0
      // this tile's query rows, swizzled as TMA would: 8 rows of 128 bytes a pattern
      for (int i = wtid; i < kTcRows * (D / 8); i += 128) {
        const int rr = i / (D / 8), ch = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (rr < nrows) {
          const int R = row_lo + rr;
          v = *reinterpret_cast<const uint4*>(static_cast<const T*>(P.q) + (long long)(r.cu + R / P.group) * P.sq_node +
                                              (long long)(g.kvh * P.group + R % P.group) * P.sq_head + ch * 8);
        }
        *reinterpret_cast<uint4*>(qs + (ch >> 3) * (kTcRows * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&q_full);
      const bool mine = row < nrows;
      const bool any = (warp & 3) * 32 < nrows;  // warp-uniform
      const int R = row_lo + (mine ? row : 0);
      const int node = mine ? R / P.group : 0;
      float m = -INFINITY;                 // the row's reference, log2 units
      float2 l2 = make_float2(0.f, 0.f);   // its sum of 2^(s - m)
      for (int t = g.t0; ok && t < g.t1; ++t, ++tc) {
        const TcTile x = tc_tile(r, t);
        const int buf = NT == 1 ? (t - g.t0) & 1 : w;
        uint32_t see[4];
        if (!x.cached && any) {
#pragma unroll
          for (int c = 0; c < 4; ++c) see[c] = tree_bits32(P, r.cu, r.n, node, x.lo + c * 32);
        }
        // Values past the end of a tile's keys, whatever the slots hold, are
        // zero for the product, and so are infinities and NaN among drafted
        // values: a row that does not see them would get 0 times them.
        if (w == 0 && ((x.valid & 15) || !x.cached)) {
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
        ok = ok && warp_wait(&s_full[buf], s_ph[buf]);
        s_ph[buf] ^= 1;
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_at = tmem + lanes + buf * kTcKeys;
        if (any) {
          // 32 scores of this row, -inf where it sees nothing; read twice (for
          // the maximum, for the weights) to keep registers for one warp more
          auto chunk = [&](int c, float* z) {
            tmem_ld32(s_at + c * 32, z);
            if (x.valid < kTcKeys || !x.cached) {
              const int left = x.valid - c * 32;
              const uint32_t bits = x.cached ? (left >= 32 ? 0xffffffffu : (1u << left) - 1u) : see[c];
#pragma unroll
              for (int e = 0; e < 32; ++e) z[e] = (bits >> e) & 1u ? z[e] : -INFINITY;
            }
          };
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 32 >= x.valid) break;
            float z[32];
            chunk(c, z);
            float a = fmaxf(z[0], z[1]), b = fmaxf(z[2], z[3]);
#pragma unroll
            for (int e = 4; e < 32; e += 4) {
              a = fmaxf(a, fmaxf(z[e], z[e + 1]));
              b = fmaxf(b, fmaxf(z[e + 2], z[e + 3]));
            }
            mx = fmaxf(mx, fmaxf(a, b));
          }
          mx *= P.scale_log2;  // the scale is positive
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
            }
            if (t > g.t0) {
              ok = warp_wait(&o_done[w], (o_n - 1) & 1);  // the tile before is in O
              if (!ok) break;
              __syncwarp();
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(o_at + c * 32, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(o_at + c * 32, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 sc = make_float2(P.scale_log2, P.scale_log2), nr = make_float2(-ref, -ref);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 32 >= x.valid) break;
            float z[32];
            uint32_t p[16];
            chunk(c, z);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = __ffma2_rn(make_float2(z[e], z[e + 1]), sc, nr);
              const float2 w2 = make_float2(ex2(y.x), ex2(y.y));
              l2 = __fadd2_rn(l2, w2);
              p[e / 2] = pack2<T>(w2.x, w2.y);
            }
            tmem_st16(s_at + c * 16, p);  // over scores that have been read
          }
          tc_wait_st();
        }
        ++o_n;
        tc_fence_before();
        mbar_arrive(&p_ready[buf]);
      }
      if (!ok) break;
      ok = warp_wait(&o_done[w], (o_n - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (NT > 1) {  // odd_seg is written by the first row tile's threads
        mbar_arrive(&seg_end);
        ok = warp_wait(&seg_end, seg & 1);
        if (!ok) break;
      }
      if (!any) continue;
      const bool poison = bad_seg[seg & 15] == seg, odd = odd_seg[seg & 1] == seg;
      const bool whole = g.t0 == 0 && g.t1 == r.per_item;
      const int slot = 2 * blockIdx.x + tree_slot(g.t0 == 0);
      float l = l2.x + l2.y;
      if (poison) l = NAN;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int head = g.kvh * P.group + R % P.group;
      T* dst = static_cast<T*>(P.out) + (long long)(r.cu + node) * P.so_node + (long long)head * P.so_head;
      const long long prow = (long long)slot * P.rows + w * kTcRows + row;
      float* part = P.part_o + prow * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        __syncwarp();
        tmem_ld32(o_at + c * 32, o);
        if (mine && odd) {
          const T* vn = static_cast<const T*>(P.v_new) + (long long)r.cu * P.sn_node + (long long)g.kvh * P.sn_head + c * 32;
          const int lo = max(0, g.t0 - r.ct) * kTcKeys, hi = min(r.n, (g.t1 - r.ct) * kTcKeys);
          for (int j = lo; j < hi; ++j) {
            if (!((tree_bits32(P, r.cu, r.n, node, j & ~31) >> (j & 31)) & 1u)) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t b = *reinterpret_cast<const uint16_t*>(vn + (long long)j * P.sn_node + e);
              if ((b & exp_mask<T>()) == exp_mask<T>()) o[e] += half_to_f32<T>(b);
            }
          }
        }
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
            *reinterpret_cast<float4*>(part + c * 32 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (mine) {
        const float ref = m == -INFINITY ? 0.f : m;
        if (!whole)
          P.part_ml[prow] = make_float2(m, l);
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

// ------------------------------------------------------------------- host
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (EncodeTiled) nullptr;
    }
    return (EncodeTiled)p;
  }();
  return f;
}

// A map of 16-bit elements with rows of 64 channels per box; axes of one
// element get a stride that the encoder takes.
bool encode(CUtensorMap* m, bool bf16, int rank, const void* base, const cuuint64_t* dims, const long long* strides,
            const cuuint32_t* box) {
  EncodeTiled f = encoder();
  if (!f) return false;
  cuuint64_t st[3];
  const cuuint32_t one[4] = {1, 1, 1, 1};
  for (int i = 0; i + 1 < rank; ++i) st[i] = dims[i + 1] == 1 ? 512 : (cuuint64_t)strides[i] * 2;
  return f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void*>(base),
           dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int page_box(int page_size) {
  int a = page_size, b = 64;
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

template <typename T, int D, int NT>
int launch_tc(const TreeParams& P, const TcMaps& maps, int box, cudaStream_t s) {
  using S = TcShape<D, NT>;
  if (cudaFuncSetAttribute(tree_tc_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  tree_tc_kernel<T, D, NT><<<P.grid, S::kThreads, S::kSmem, s>>>(P, maps, box);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
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
