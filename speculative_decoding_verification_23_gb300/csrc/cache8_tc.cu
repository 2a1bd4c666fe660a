// Attention of drafted trees over a paged cache in 8 bits on the 5th-generation
// tensor cores: keys and values staged by TMA straight from their pages as they
// are, brought to fp16 in shared memory by warps of their own, scores and outputs
// in tensor memory.
#include "cache8_common.cuh"
#include "tc_common.cuh"

namespace sv {
namespace {

constexpr int kUnit8 = 64;        // keys per unit of the softmax, half a tile
constexpr int kRows8 = 128;       // query rows per tile (lanes of tensor memory)
// log2: how far a row's largest weight may pass its reference before outputs are
// rescaled, and where the reference lies in fp16: weights stay below 2^15.
constexpr float kLazy8 = 8.f;
constexpr float kTop8 = 7.f;

// PAIR: two row tiles share every staged tile.
template <int D, bool PAIR>
struct C8Shape {
  static constexpr int kQBytes = kRows8 * D * 2;
  static constexpr int kSlot = kTcKeys * D * 2;     // a tile of keys or of values in fp16
  static constexpr int kHalf = kTcKeys * 128;       // 64 channels of it
  static constexpr int kSlots = D == 64 ? (PAIR ? 6 : 8) : (PAIR ? 3 : 4);
  static constexpr int kRaw = kTcKeys * D;          // and in 8 bits
  static constexpr int kRaws = D == 64 ? 8 : 4;
  static constexpr int kQTiles = PAIR ? 2 : 1;
  static constexpr int kSmem = kQTiles * kQBytes + kSlots * kSlot + kRaws * kRaw;
};
constexpr int kC8Tiles = 8;        // tiles that are described ahead
constexpr int kC8Segs = 16;        // segments: more than may be described beside one that is still being written
constexpr int kC8Softmax = 8, kC8Convert = 4;       // warps, then two that copy and two that issue products
constexpr int kC8TcThreads = 32 * (kC8Softmax + kC8Convert + 4);
// Whether values of T need a scale to be exact in fp16.
template <typename T>
constexpr bool kScaled = true;
template <>
constexpr bool kScaled<__half> = false;

// Two columns of this warp's 32 lanes, with the wait.
__device__ __forceinline__ void tmem_st2(uint32_t addr, float a, float b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(addr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b))
               : "memory");
}
__device__ __forceinline__ float2 tmem_ld2(uint32_t addr) {
  uint32_t a, b;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(a), "=r"(b)
               : "r"(addr)
               : "memory");
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// Scores of 16 lanes, 64 columns: of eight columns 8 g .., a thread has columns
// 2 (lane % 4) and the one after of row lane / 4 (r[4 g], r[4 g + 1]) and of the
// row 8 further (r[4 g + 2], r[4 g + 3]).
__device__ __forceinline__ void tmem_ld_pairs(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}
// And weights, two in a word: 32 columns, r[2 g] of the first row and r[2 g + 1]
// of the second.
__device__ __forceinline__ void tmem_st_pairs(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

struct C8Maps {
  CUtensorMap k, v;  // (channel, slot, head, page), bytes
};

struct C8Tile {
  bool cached, some;
  int lo, valid;
};
__device__ __forceinline__ C8Tile c8_tile(const TreeReq& r, int t) {
  C8Tile x;
  const TreeKeys k = tree_keys<true>(r, kTcKeys, t);
  x.cached = k.cached;
  x.lo = k.lo;
  x.valid = min(kTcKeys, k.lim - k.lo);
  x.some = !k.cached || (t >= r.st && k.lo < r.part);
  return x;
}

// What the copying warp tells the others of a tile: its first key, its number of
// keys (bits 0 - 7) and kind, its place in its segment and the tiles from it on
// (0: there are no more).
constexpr int kTileCached = 256, kTileSome = 512;  // some: some rows see a key of it and others do not
struct C8Desc {
  int lo, info, pos, left;
  __device__ __forceinline__ int valid() const { return info & 255; }
  __device__ __forceinline__ int n16() const { return ((info & 255) + 15) & ~15; }
  __device__ __forceinline__ bool cached() const { return (info & kTileCached) != 0; }
  __device__ __forceinline__ bool some() const { return (info & kTileSome) != 0; }
};
// And of a segment: one run of tiles of a key head and block of rows.
struct C8Seg {
  int b, kvh, m;         // request, key/value head, block of rows
  int cu, n, ctx, part;  // as in TreeReq
  int t0, t1, whole;     // its tiles, and whether they are the item's
  int bad, odd;          // a bad page, odd values that were left out
};

// Which of the 32 keys from `base` on a row sees, in a tile that some rows see
// and others do not.  Not inlined: few tiles want it, and the kernel's code is
// large for the instruction cache as it is.
__device__ __noinline__ uint32_t c8_sees(const TreeParams& P, int cu, int n, int ctx, int seen, int lo, int node,
                                         bool cached, int base) {
  if (cached) return tree_window32(base, lo, P.sinks);
  const uint32_t bits = tree_bits16(P, cu, n, node, base) | tree_bits16(P, cu, n, node, base + 16) << 16;
  TreeReq r;
  r.cu = cu;
  r.n = n;
  r.ctx = ctx;
  return tree_window_drafted(P, r, TreeRow{seen, lo}, node, base, bits);
}

// A windowed row, as tree_row.
__device__ __noinline__ int c8_row(const TreeParams& P, int cu, int n, int node) { return tree_seen(P, cu, n, node); }

// Adds the infinities and NaN among the values of a segment's tiles that some
// rows see and others do not, where this row sees them, to channels c0 .. c1 - 1
// of its result, which was computed with zeros in their places: to the written
// row `dst`, or to its partial result (unnormalised: the weight's size does not
// matter).
template <typename T>
__device__ __noinline__ void c8_add_odd(const TreeParams& P, int b, int kvh, int t0, int t1, int seen, int row_lo, int node,
                                        int c0, int c1, T* dst, float4* part) {
  const uint32_t em = exp_mask<T>();
  const PageDiv pd(P.page_size);
  const TreeReq r = tree_request<true>(P, b);
  for (int t = t0; t < t1; ++t) {
    const C8Tile x = c8_tile(r, t);
    if (!x.some) continue;
    for (int e = 0; e < x.valid; ++e) {
      const int j = x.lo + e;
      if (!((c8_sees(P, r.cu, r.n, r.ctx, seen, row_lo, node, x.cached, j & ~31) >> (j & 31)) & 1u)) continue;
      const uint8_t* v8 = nullptr;
      const uint16_t* v16 = nullptr;
      if (x.cached) {
        int page, slot;
        pd.split(j, page, slot);
        const int id = P.table[(long long)b * P.ld_table + page];
        if (id < 0 || id >= P.num_pages) continue;
        v8 = static_cast<const uint8_t*>(P.v) + (long long)id * P.s_page + (long long)slot * P.s_slot +
             (long long)kvh * P.s_head;
      } else {
        v16 = static_cast<const uint16_t*>(P.v_new) + (long long)(r.cu + j) * P.sn_node + (long long)kvh * P.sn_head;
      }
      for (int d = c0; d < c1; ++d) {
        float add;
        if (x.cached) {
          if ((v8[d] & 0x7f) != 0x7f) continue;
          add = NAN;
        } else {
          const uint32_t w = v16[d];
          if ((w & em) != em) continue;
          add = half_to_f32<T>(w);
        }
        if (dst) {
          uint16_t* o = reinterpret_cast<uint16_t*>(dst + d);
          *o = (uint16_t)(pack2<T>(half_to_f32<T>(*o) + add, 0.f) & 0xffffu);
        } else {
          reinterpret_cast<float*>(part + (long long)(d / 4) * P.rows)[d & 3] += add;
        }
      }
    }
  }
}

// A scale's part in the softmax (see cache8_common.cuh): x multiplies scores, y
// is added to their logarithm, z turns a weight back into the softmax's, w says
// that the values count as 0.
__device__ __forceinline__ float4 c8_scale(float ks, float vs) {
  const float v = vs < kLeastScale ? kLeastScale : vs;  // NaN stays, and gives NaN where it is seen
  return make_float4(ks, log2f(v), v == v ? 1.f / v : 0.f, vs < kLeastScale ? 1.f : 0.f);
}

// Warps 0 - 7: the softmax; 8 and 9 convert keys, 10 and 11 values; 12 and 15 copy
// keys and values; 13 and 14 issue the products of each stream.
//
// The copying warps alone walk over the CTA's tiles.  They look up the pages of
// four of them at once, a lane 16 keys, while the four before are copied, and the
// first of them describes each tile and segment to the others.
//
// A tile of 128 keys comes as 8 bits; the conversion writes it in fp16 in the
// swizzled layout that the products read, a thread a key's row in two steps.
// Drafted keys and values are read from where they are, 16 keys a warp, and
// scaled to be exact in fp16.  Per stream and tile:
//   S = Q K^T (shared memory), y = ks S + log2 vs, the softmax by rows,
//   P = 2^(y - m) in fp16 over the scores read, O += P V (P from tensor memory),
//   l += P / vs.
//
// ROWS, the query rows of a key head that a CTA takes at once:
// - 256: two tiles of 128 rows share the staged keys, each a stream of its own, a
//   thread a row, by halves of a tile.
// - 128: one tile of rows, whose tiles of keys two streams take in turn, each with
//   scores, outputs and reference of its own, joined at a segment's end.
// - 64: as 128, with products of 64 rows, which lie in 16 lanes of each warp's
//   32.  A thread then has half of the keys of two rows in the layout of a matrix
//   fragment, so all eight warps are at work where 128 rows would leave half of
//   them idle.
//   The softmax goes by halves of a tile, whose products begin as soon as its
//   weights are there; by whole tiles the chains below took 120 us for 114, the
//   long contexts 132 for 134.
// 16 requests with trees over up to 16384 tokens, 32 / 8 heads, cold: 16 nodes (64
// rows) 109 / 117 / 139 us with ROWS 64 / 128 / 256, 32 nodes 117 and 143 with 128
// and 256, 64 nodes 217 and 166.
//
// 64 ragged requests of up to 9 nodes over up to 8192 tokens take 115 us, trees of
// up to 64 nodes over up to 16384 158, two requests over 128 K tokens 134 (54 % of
// the copy rate).  A tile moves 208 KB through shared memory (32 written by the
// copies, 32 read and 64 written by the conversion, 80 read by the products; 224
// with more than 64 rows), 1650 cycles at 128 bytes a cycle, and takes some 2400:
// the conversion works for 1500 of them and waits for copies and free slots for
// the rest.  Scores on the bytes themselves, with queries in two 8-bit parts (bf16)
// or three (fp16) and values converted as here, took 195, 327 and 183 us where this
// kernel in its first form took 158, 194 and 178.  A segment's end and the next one's queries cost some 20
// thousand cycles, which is what short contexts have besides.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kC8TcThreads, 1)
    cache8_tc_kernel(const Cache8Params C, const __grid_constant__ C8Maps maps, int box) {
  constexpr bool PAIR = ROWS > kRows8, HALF = ROWS < kRows8;
  using S = C8Shape<D, PAIR>;
  const TreeParams& P = C.t;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint64_t raw_full[S::kRaws], raw_empty[S::kRaws], h_full[S::kSlots], h_empty[S::kSlots], d_full[kC8Tiles],
      d_empty[kC8Tiles], sc_full[kC8Tiles], q_full[2], s_full[4], p_ready[4], o_half[2], o_done[2], o_last[2], fin[2],
      seg_end;
  __shared__ float4 scales[kC8Tiles][kTcKeys / 16];
  __shared__ C8Desc tiles[kC8Tiles];
  __shared__ C8Seg segs[kC8Segs];
  __shared__ uint8_t row_scale[S::kQTiles][kRows8];  // powers of two: their exponents and 64
  __shared__ uint32_t tmem_at;
  __shared__ volatile int dead;
  unsigned char* ring = smem + S::kQTiles * S::kQBytes;
  unsigned char* raws = ring + S::kSlots * S::kSlot;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);

  if (warp == kC8Softmax + kC8Convert + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_at))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < S::kRaws; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kC8Convert / 2);
    }
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&h_full[i], kC8Convert / 2);
      mbar_init(&h_empty[i], PAIR ? 2 : 1);
    }
    for (int i = 0; i < kC8Tiles; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&sc_full[i], 1 + kC8Convert);
      mbar_init(&d_empty[i], kC8Convert + 2);  // the products' warps leave a tile when its softmax has ended
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], PAIR ? 128 : 256);
      mbar_init(&o_half[i], 1);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_last[i], 1);
      mbar_init(&fin[i], 1);
    }
    mbar_init(&seg_end, 256);
    fence_mbar_init();
    dead = 0;
  }
  if (warp == kC8Softmax + kC8Convert && lane < 2) prefetch_map(lane == 0 ? &maps.k : &maps.v);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_previous();
  start_next();  // not before this CTA has its tensor memory, which a kernel after it may want too
  const uint32_t tmem = uniform(tmem_at);
  int tc = 0;  // tiles so far: the rings hold keys of tile i as fill 2i, values as 2i + 1

  // The description of tile i; the conversion and the products' warps read it, or
  // pass it by, before it is written over.
  auto wait_tile = [&](int i) { return warp_wait(&d_full[i & (kC8Tiles - 1)], (i / kC8Tiles) & 1); };
  auto leave_tile = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&d_empty[i & (kC8Tiles - 1)]);
  };

  if (warp == kC8Softmax + kC8Convert || warp == kC8Softmax + kC8Convert + 3) {
    // ------------------------------------------------------------ copies
    // One warp copies keys and describes tiles, one copies values.
    const bool values = warp != kC8Softmax + kC8Convert;
    const TreeScan scan = tree_scan<true>(P, lane);
    if (blockIdx.x == 0 && !values) tree_store_starts<true>(P, scan, lane);
    TreeWalkOf<true> walk;
    walk.begin(P, lane, scan, blockIdx.x);
    TreeSeg g;
    g.t1 = 0;
    int t = 0, seg = -1, s = values ? 1 : 0;
    uint32_t ph = 1;
    RingFills fills;
    bool ok = true;
    const PageDiv pd(P.page_size), sd(C.block);
    const CUtensorMap* map = values ? &maps.v : &maps.k;
    const int box_shift = 31 - __clz(box);
    const int sub = lane >> 3, key = (lane & 7) * 16;  // this lane's tile of four, and its keys there
    const uint32_t dst = smem_u32(raws) + key * D;
    struct Batch {
      int count;  // tiles; the rest is of this lane's tile
      C8Desc d;
      C8Seg e;
      int page, slot;
      float ks, vs;
    };
    auto look = [&](Batch& x) {
      x.count = 0;
      x.d.info = x.d.pos = 0;
      x.e.bad = 0;
      // this lane's tile is tile t of the segment
      auto fill = [&](int t) {
        const C8Tile y = c8_tile(walk.r, t);
        x.d.lo = y.lo;
        x.d.info = y.valid | (y.cached ? kTileCached : 0) | (y.some ? kTileSome : 0);
        x.d.pos = t - g.t0;
        x.d.left = g.t1 - t;
        x.e.b = g.b;
        x.e.kvh = g.kvh;
        x.e.m = g.m;
        x.e.cu = walk.r.cu;
        x.e.n = walk.r.n;
        x.e.ctx = walk.r.ctx;
        x.e.part = walk.r.part;
        x.e.t0 = g.t0;
        x.e.t1 = g.t1;
        x.e.whole = g.t0 == 0 && g.t1 == walk.r.per_item;
      };
      if (t + 4 <= g.t1) {  // most often
        fill(t + sub);
        t += 4;
        x.count = 4;
      } else {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          if (t >= g.t1) {
            if (!walk.next(P, g)) break;
            t = g.t0;
          }
          if (sub == i) fill(t);
          ++t;
          ++x.count;
        }
      }
      x.page = x.slot = 0;
      x.ks = x.vs = 0.f;
      if (x.d.cached() && key < x.d.valid()) {
        int page, blk, rest;
        pd.split(x.d.lo + key, page, x.slot);
        x.page = P.table[(long long)x.e.b * P.ld_table + page];
        x.e.bad = x.page < 0 || x.page >= P.num_pages;
        if (x.e.bad) x.page = 0;
        if (!values) {
          sd.split(x.slot, blk, rest);
          const long long at = (long long)x.page * C.c_page + (long long)blk * C.c_block + (long long)x.e.kvh * C.c_head;
          x.ks = C.ks[at];
          x.vs = C.vs[at];
        }
      }
    };
    auto issue = [&](const Batch& x) {
      // a lane's part in its tile's copy: the first of each box's keys
      const bool mine = key < x.d.valid() && (key & (box - 1)) == 0;
      __syncwarp();  // lanes may leave the lookup one by one
      const bool any_bad = !values && __any_sync(0xffffffffu, x.e.bad != 0);
#pragma unroll 1
      for (int i = 0; ok && i < x.count; ++i, ++tc) {
        const int info = __shfl_sync(0xffffffffu, x.d.info, i * 8);
        if (!values) {
          const int at = tc & (kC8Tiles - 1);
          if (__shfl_sync(0xffffffffu, x.d.pos, i * 8) == 0) ++seg;
          ok = warp_wait(&d_empty[at], ((tc / kC8Tiles) & 1) ^ 1);
          if (!ok) break;
          if (sub == i) {
            // of drafted tokens, known once they are read; keys past the end take part with weight 0
            scales[at][lane & 7] = info & kTileCached ? c8_scale(x.ks, x.vs) : make_float4(0.f, 0.f, 0.f, 0.f);
            if ((lane & 7) == 0) {
              tiles[at] = x.d;
              if (x.d.pos == 0) {
                C8Seg e = x.e;
                e.bad = e.odd = 0;
                segs[seg & (kC8Segs - 1)] = e;
              }
            }
          }
          if (any_bad) {
            __syncwarp();
            if (sub == i && x.e.bad) segs[seg & (kC8Segs - 1)].bad = 1;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&d_full[at]);
            mbar_arrive(&sc_full[at]);
          }
        }
        if (!(info & kTileCached)) continue;
        ok = warp_wait(&raw_empty[s], ph);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&raw_full[s], (uint32_t)((((info & 255) + box - 1) >> box_shift << box_shift) * D));
        fills.note(s, ph ^ 1);
        __syncwarp();
        if (sub == i && mine) tma_4d(dst + s * S::kRaw, map, 0, x.slot, x.e.kvh, x.page, &raw_full[s]);
        s += 2;
        if (s >= S::kRaws) {
          s -= S::kRaws;
          ph ^= 1;
        }
      }
    };
    // The next four are looked up before these are copied.
    Batch a;
    look(a);
#pragma unroll 1
    while (ok && a.count > 0) {
      const Batch b = a;
      look(a);
      issue(b);
    }
    if (!values && ok) ok = warp_wait(&d_empty[tc & (kC8Tiles - 1)], ((tc / kC8Tiles) & 1) ^ 1);
    if (ok) {
      if (!values && lane == 0) {
        tiles[tc & (kC8Tiles - 1)].left = 0;
        mbar_arrive(&d_full[tc & (kC8Tiles - 1)]);
      }
    } else {
      dead = 1;
      fills.drain(raw_full, S::kRaws);
    }
  } else if (warp > kC8Softmax + kC8Convert) {
    // ---------------------------------------------------------- products
    // One warp issues everything of stream w.  It has little time for a unit, so
    // slots and phases are counted, not computed: a stream's tiles are every one
    // (two row tiles) or every second one of the CTA, whatever the segments.
    const int w = warp - (kC8Softmax + kC8Convert + 1);
    const uint32_t one = elect_one();
    bool ok = true;
    uint32_t p_ph = 0, q_ph = 0;  // phases (p_ph: a bit per half)
    constexpr int STEP = PAIR ? 1 : 2;
    int k_slot = PAIR ? 0 : 2 * w, v_slot = k_slot + 1;
    uint32_t k_ph = 0, v_ph = 0;
    const uint64_t da = smem_desc(smem_u32(smem) + (PAIR ? w : 0) * S::kQBytes, 16, 1024);
    const uint64_t dk = smem_desc(smem_u32(ring), 16, 1024), dv = smem_desc(smem_u32(ring), S::kHalf, 1024);
    constexpr uint32_t kFewer = HALF ? 4u << 24 : 0u;  // 64 rows: 16 lanes of each warp's 32
    const uint32_t o = tmem + 2 * kTcKeys + w * D, id_v = inst_desc<__half>(D, true) - kFewer, p = tmem + w * kTcKeys;
    auto tile_keys = [&](int i) {  // of tile i, by sixteens
      ok = ok && wait_tile(i);
      return ok ? uniform(tiles[i & (kC8Tiles - 1)].n16()) : 0;
    };
    // Scores: with two row tiles of a half as soon as the weights there have been
    // used; with two streams of 128 keys at once, which reads the queries once.
    auto scores = [&](int n16, int h) {
      const uint32_t id = inst_desc<__half>(PAIR ? min(kUnit8, n16 - h * kUnit8) : n16, false) - kFewer;
      const uint64_t db = dk + (uint32_t)(k_slot * (S::kSlot >> 4) + h * ((kUnit8 * 128) >> 4));
      if (h == 0) ok = ok && warp_wait(&h_full[k_slot], k_ph);
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks / 4) * S::kHalf + (ks % 4) * 32) >> 4;
        mma_ss(p + h * kUnit8, da + off, db + off, id, ks > 0, one);
      }
      mma_commit(&s_full[w * 2 + h], one);
      if (!PAIR || h == 1 || n16 <= kUnit8) {
        mma_commit(&h_empty[k_slot], one);
        k_slot += 2 * STEP;
        if (k_slot >= S::kSlots) {
          k_slot -= S::kSlots;
          k_ph ^= 1;
        }
      }
    };
    while (ok) {
      ok = wait_tile(tc);
      if (!ok) break;
      const int left = uniform(tiles[tc & (kC8Tiles - 1)].left);  // tiles of the segment
      if (left == 0) break;
      ok = warp_wait(&q_full[PAIR ? w : 0], q_ph);
      q_ph ^= 1;
      const int first = PAIR ? 0 : (tc ^ w) & 1;  // this stream's first tile
      if (!PAIR && first == 1) leave_tile(tc);
      int n16 = 0;
      if (first < left) {
        n16 = tile_keys(tc + first);
        if (ok) scores(n16, 0);
        if (PAIR && ok && n16 > kUnit8) scores(n16, 1);
      }
      int next = first + STEP < left ? tile_keys(tc + first + STEP) : 0;
#pragma unroll 1
      for (int i = first; ok && i < left; i += STEP) {
        ok = ok && warp_wait(&h_full[v_slot], v_ph);
#pragma unroll 1
        for (int h = 0; ok && h * kUnit8 < n16; ++h) {
          ok = warp_wait(&p_ready[w * 2 + h], (p_ph >> h) & 1);
          if (!ok) break;
          p_ph ^= 1u << h;
          tc_fence_after();
          const uint64_t db = dv + (uint32_t)(v_slot * (S::kSlot >> 4) + h * (4 * 2048 >> 4));
          const uint32_t at = p + h * kUnit8, begun = h > 0 || i > first;
          const int steps = min(4, n16 / 16 - h * 4);
          if (steps == 4) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) mma_ts(o, at + ks * 8, db + ks * (2048 >> 4), id_v, ks > 0 || begun, one);
          } else {
#pragma unroll 1
            for (int ks = 0; ks < steps; ++ks) mma_ts(o, at + ks * 8, db + ks * (2048 >> 4), id_v, ks > 0 || begun, one);
          }
          if (h == 0) mma_commit(&o_half[w], one);
          if ((h + 1) * kUnit8 >= n16) {
            mma_commit(&o_done[w], one);  // before the scores that the softmax takes for a sign of it
            mma_commit(&h_empty[v_slot], one);
          }
          if (PAIR && next > h * kUnit8 && (next > kUnit8 || n16 <= kUnit8)) scores(next, h);
        }
        if (!ok) break;
        // What the tile had no half for, and the scores of half a tile after a whole
        // one.  Three slots take keys and values in turn, and the conversion of values
        // relies on this order: the slot of a tile's keys is not free before that of
        // the values of the tile before, or a phase of the latter's could be mistaken
        // for the one two further.
        if (PAIR ? (n16 <= kUnit8) == (next > kUnit8) && next > 0 : next > 0) scores(next, PAIR && next > kUnit8 ? 1 : 0);
        v_slot += 2 * STEP;
        if (v_slot >= S::kSlots) {
          v_slot -= S::kSlots;
          v_ph ^= 1;
        }
        if (i + STEP >= left) mma_commit(&o_last[w], one);
        leave_tile(tc + i);
        if (!PAIR && i + 1 < left) {  // the other stream's; not before it is described, or it would count for the one before
          ok = wait_tile(tc + i + 1);
          if (!ok) break;
          leave_tile(tc + i + 1);
        }
        n16 = next;
        next = i + 2 * STEP < left ? tile_keys(tc + i + 2 * STEP) : 0;
      }
      tc += left;
    }
    if (!ok) dead = 1;
    mma_commit(&fin[w], one);
    __syncwarp();
    mbar_wait(&fin[w], 0);  // every product has ended before tensor memory is freed
  } else if (warp >= kC8Softmax) {
    // -------------------------------------------------------- conversion
    // Two warps convert keys and two values, a thread two keys' rows of every tile:
    // each pair waits, fences and arrives once a tile, and neither waits for the
    // other.
    const int kv = (warp - kC8Softmax) >> 1, row0 = ((warp & 1) << 5) + lane;
    const uint32_t em = exp_mask<T>();
    bool ok = true;
    int rs = kv, slot = kv, seg = -1;
    uint32_t rph = 0, hph = 1;
    // where a key's 16-byte pieces lie: swizzled as TMA writes 8 bits (rows of 128
    // or 64 bytes), and as the products want fp16; both repeat every 8 keys
    const uint32_t in_x = D == 64 ? ((row0 >> 1) & 3) << 4 : (row0 & 7) << 4, out_x = (uint32_t)(row0 & 7) << 4;
    for (; ok; ++tc) {
      ok = wait_tile(tc);
      if (!ok) break;
      const C8Desc x = tiles[tc & (kC8Tiles - 1)];
      if (x.left == 0) break;
      if (x.pos == 0) ++seg;
      const bool cached = x.cached(), some = x.some();
      const int valid = x.valid(), n16 = x.n16();
      if (cached) ok = warp_wait(&raw_full[rs], rph);
      ok = ok && warp_wait(&h_empty[slot], hph);
      if (!ok) break;
      bool odd = false;
      if (cached) {
#pragma unroll 1
        for (int row = row0; row - lane < n16; row += 64) {
          unsigned char* dst = ring + slot * S::kSlot + row * 128;
          const unsigned char* src = raws + rs * S::kRaw + row * D;
          // all loads first: only what a warp has in flight by itself hides
          // latencies
          uint4 v[D / 16];
#pragma unroll
          for (int c = 0; c < D / 16; ++c) v[c] = *reinterpret_cast<const uint4*>(src + ((uint32_t)(c << 4) ^ in_x));
          if (kv) {
            // Values past the end of a tile's keys, whatever the slots hold, are
            // zero for the product, and so are those whose scale counts as 0, but
            // for NaN, which a weight of 0 leaves NaN.  Where some rows see a value
            // and others do not, NaN are left out and added to the rows at the end.
            const bool past = row >= valid, zero = scales[tc & (kC8Tiles - 1)][row >> 4].w != 0.f;
            if (__any_sync(0xffffffffu, past || zero || some)) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                uint32_t* e = reinterpret_cast<uint32_t*>(&v[c]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t nan = past ? 0u : __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  odd = odd || (some && nan != 0u);
                  e[k] &= past ? 0u : zero ? (some ? 0u : nan) : some ? ~nan : 0xffffffffu;
                }
              }
            }
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            unsigned char* to = dst + (c >> 2) * S::kHalf;
            const uint32_t at = (uint32_t)((c & 3) << 5);
            *reinterpret_cast<uint4*>(to + (at ^ out_x)) =
                make_uint4(e4m3x2_f16x2(v[c].x & 0xffffu), e4m3x2_f16x2(v[c].x >> 16), e4m3x2_f16x2(v[c].y & 0xffffu),
                           e4m3x2_f16x2(v[c].y >> 16));
            *reinterpret_cast<uint4*>(to + ((at | 16u) ^ out_x)) =
                make_uint4(e4m3x2_f16x2(v[c].z & 0xffffu), e4m3x2_f16x2(v[c].z >> 16), e4m3x2_f16x2(v[c].w & 0xffffu),
                           e4m3x2_f16x2(v[c].w >> 16));
          }
        }
      } else {
        // 16 keys a warp at once: a lane has 8 channels of every (256 / D)-th, copied
        // to where they belong and scaled there.  Little code, as for queries.
        constexpr int PCS = D / 8, RS = 32 / PCS;
        const C8Seg& e = segs[seg & (kC8Segs - 1)];
        const int piece = lane % PCS, r0 = lane / PCS;
        const T* base = static_cast<const T*>(kv ? P.v_new : P.k_new) + (long long)(e.cu + x.lo) * P.sn_node +
                        (long long)e.kvh * P.sn_head + piece * 8;
        auto place = [&](int row) {
          return ring + slot * S::kSlot + (piece >> 3) * S::kHalf + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
        };
#pragma unroll 1
        for (int g = (warp & 1) * 16; g < n16; g += 32) {
#pragma unroll 1
          for (int row = g + r0; row < g + 16; row += RS)
            cp_async16(smem_u32(place(row)), base + (long long)min(row, valid - 1) * P.sn_node, row < valid);
          cp_async_commit();
          cp_async_wait<0>();
          Exact16 s16 = {1.f, 1.f};
          if (kScaled<T>) {
            uint32_t top = 0;
#pragma unroll 1
            for (int row = g + r0; row < g + 16; row += RS) {
              const uint4 v = *reinterpret_cast<const uint4*>(place(row));
              top = max_u16x2(top, max_u16x2(max_u16x2(finite_size2(v.x, em), finite_size2(v.y, em)),
                                             max_u16x2(finite_size2(v.z, em), finite_size2(v.w, em))));
            }
            s16 = exact16<T>(__reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16)));
          }
          if (lane == 0) {
            float4* at = &scales[tc & (kC8Tiles - 1)][g >> 4];
            if (kv == 0) {
              at->x = s16.back;
            } else {
              const float4 y = c8_scale(0.f, s16.back);
              at->y = y.y;
              at->z = y.z;
            }
          }
          if (kScaled<T> || kv) {
#pragma unroll 1
            for (int row = g + r0; row < g + 16; row += RS) {
              uint4 v = *reinterpret_cast<const uint4*>(place(row));
              uint32_t* y = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                if (kv) {  // infinities and NaN are left out
                  if ((y[z] & em) == em) {
                    y[z] &= 0xffff0000u;
                    odd = true;
                  }
                  if (((y[z] >> 16) & em) == em) {
                    y[z] &= 0xffffu;
                    odd = true;
                  }
                }
                y[z] = to_f16x2<T>(y[z], s16.to);
              }
              *reinterpret_cast<uint4*>(place(row)) = v;
            }
          }
        }
      }
      if (odd) segs[seg & (kC8Segs - 1)].odd = 1;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&h_full[slot]);
        if (cached) mbar_arrive(&raw_empty[rs]);
        mbar_arrive(&sc_full[tc & (kC8Tiles - 1)]);  // drafted tokens' scales are known once they are read
        mbar_arrive(&d_empty[tc & (kC8Tiles - 1)]);
      }
      if (cached) {
        rs += 2;
        if (rs >= S::kRaws) {
          rs -= S::kRaws;
          rph ^= 1;
        }
      }
      slot += 2;
      if (slot >= S::kSlots) {
        slot -= S::kSlots;
        hph ^= 1;
      }
    }
    if (!ok) dead = 1;
  } else {
    // ----------------------------------------------------------- softmax
    const int w = warp >> 2, wtid = PAIR ? tid & 127 : tid;
    const int row = HALF ? (warp & 3) * 16 + (lane & 15) : (warp & 3) * 32 + lane;
    const int tile = PAIR ? w : 0;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_at = tmem + lanes + 2 * kTcKeys + w * D;
    unsigned char* qs = smem + tile * S::kQBytes;
    const uint32_t em = exp_mask<T>();
    uint32_t s_ph = 0;  // a bit per half
    int mine_tc = 0;    // this stream's tiles so far
    uint32_t last_ph = 0;
    // node of a row: exact, as rows are at most 2^20 and half a row from a multiple
    const float inv_group = 1.f / (float)P.group;
    // what two rows' threads know, for the row of a lane
    auto of_row = [&](float a, float b) {
      a = __shfl_sync(0xffffffffu, a, (lane & 7) * 4);
      b = __shfl_sync(0xffffffffu, b, (lane & 7) * 4);
      return lane & 8 ? b : a;
    };
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      ok = wait_tile(tc);
      if (!ok) break;
      const int left = tiles[tc & (kC8Tiles - 1)].left;  // tiles of the segment
      if (left == 0) break;
      const C8Seg e = segs[seg & (kC8Segs - 1)];
      const int row_lo = e.m * (S::kQTiles * kRows8) + tile * kRows8;
      const int nrows = min(kRows8, e.n * P.group - row_lo);  // may be <= 0
      // This tile's query rows, scaled to be exact in fp16.  A thread has one
      // 16-byte piece of every (threads / (D / 8))-th row, copied to where it
      // belongs and scaled there.  Little code: it is read anew for every segment.
      constexpr int PER = D / 8, STEP = (PAIR ? 128 : 256) / PER;
      const int ch = wtid % PER;
      const T* src = static_cast<const T*>(P.q) + (long long)e.cu * P.sq_node + (long long)(e.kvh * P.group) * P.sq_head + ch * 8;
      auto place = [&](int rr) {
        return qs + (ch >> 3) * (kRows8 * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
      };
#pragma unroll 1
      for (int rr = wtid / PER; rr < (HALF ? kRows8 / 2 : kRows8); rr += STEP) {
        const int R = row_lo + min(rr, max(nrows - 1, 0)), nd = (int)(((float)R + 0.5f) * inv_group);
        cp_async16(smem_u32(place(rr)), src + (long long)nd * P.sq_node + (long long)(R - nd * P.group) * P.sq_head, rr < nrows);
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (kScaled<T>) {
#pragma unroll 1
        for (int rr = wtid / PER; rr < nrows; rr += STEP) {
          uint4 v = *reinterpret_cast<const uint4*>(place(rr));
          uint32_t top = max_u16x2(max_u16x2(finite_size2(v.x, em), finite_size2(v.y, em)),
                                   max_u16x2(finite_size2(v.z, em), finite_size2(v.w, em)));
          top = max(top & 0xffffu, top >> 16);
          // a row's lanes, which come here together or not at all; other rows' may have left
          const uint32_t peers = ((1u << PER) - 1u) << (lane & ~(PER - 1));
#pragma unroll
          for (int z = PER / 2; z > 0; z >>= 1) top = max(top, __shfl_xor_sync(peers, top, z));
          const Exact16 s16 = exact16<T>(top);
          if (ch == 0) row_scale[tile][rr] = (uint8_t)((__float_as_uint(s16.back) >> 23) - 63);
          *reinterpret_cast<uint4*>(place(rr)) =
              make_uint4(to_f16x2<T>(v.x, s16.to), to_f16x2<T>(v.y, s16.to), to_f16x2<T>(v.z, s16.to), to_f16x2<T>(v.w, s16.to));
        }
        __syncwarp();
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&q_full[tile]);
      ok = warp_wait(&q_full[tile], seg & 1);  // the rows' scales
      if (!ok) break;
      const bool here = row < nrows, mine = here && (!HALF || lane < 16);
      const float rsc = !here ? 0.f : kScaled<T> ? P.scale_log2 * __uint_as_float((uint32_t)(row_scale[tile][row] + 63) << 23) : P.scale_log2;
      const bool any = (warp & 3) * (HALF ? 16 : 32) < nrows;  // warp-uniform
      const int R = row_lo + (here ? row : 0);
      const int node = here ? (int)(((float)R + 0.5f) * inv_group) : 0;
      int seen = 0, see_lo = 0;  // as TreeRow
      if (e.part > 0 && any) {
        seen = c8_row(P, e.cu, e.n, node);
        see_lo = e.ctx + seen - P.window;
      }
      float m = -INFINITY;                         // the row's reference, log2 units
      float2 l2 = make_float2(0.f, 0.f), l3 = l2;  // its sum
      // of half a tile: of the thread's two rows
      float m_b = -INFINITY;
      const int src_a = lane >> 2, src_b = src_a + 8, pair = (lane & 3) * 2;  // their lanes, this thread's keys of eight
      const float rsc_a = HALF ? __shfl_sync(0xffffffffu, rsc, src_a) : 0.f, rsc_b = HALF ? __shfl_sync(0xffffffffu, rsc, src_b) : 0.f;
      constexpr int TSTEP = PAIR ? 1 : 2;
      const int first = PAIR ? 0 : (tc ^ w) & 1;
      for (int i = first; ok && i < left; i += TSTEP, ++mine_tc) {
        const int at = (tc + i) & (kC8Tiles - 1);
        // also says that the tile is described
        ok = wait_tile(tc + i);
        if (!ok) break;
        const C8Desc x = tiles[at];
        const int valid = x.valid(), n16 = x.n16();
        const bool masked = valid < kTcKeys || x.some();
        uint32_t see[4];
        if (x.some() && any) {
          if (x.cached()) {
#pragma unroll
            for (int c = 0; c < 4; ++c) see[c] = tree_window32(x.lo + c * 32, see_lo, P.sinks);
          } else {
            // all words at once; x.lo is a multiple of 32
            const uint32_t* words = P.mask + (long long)(e.cu + node) * P.mask_words;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int wd = (x.lo >> 5) + c, k = node - x.lo - c * 32;
              see[c] = P.mask ? (wd < P.mask_words ? words[wd] : 0u) : k < 0 ? 0u : k >= 31 ? 0xffffffffu : (2u << k) - 1u;
            }
            if (seen > P.window) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const uint32_t left = c8_sees(P, e.cu, e.n, e.ctx, seen, see_lo, node, false, x.lo + c * 32);
                see[0] = c == 0 ? left : see[0];
                see[1] = c == 1 ? left : see[1];
                see[2] = c == 2 ? left : see[2];
                see[3] = c == 3 ? left : see[3];
              }
            }
          }
        }
        // cached keys' scales come with the description; the conversion, which
        // knows drafted ones', may still be waiting for room
        if (!x.cached()) {
          ok = warp_wait(&sc_full[at], ((tc + i) / kC8Tiles) & 1);
          if (!ok) break;
        }
        if constexpr (HALF) {
#pragma unroll 1
          for (int h = 0; h * kUnit8 < n16; ++h) {
            if (h == 0) {  // of both halves
              ok = warp_wait(&s_full[w * 2], s_ph);
              s_ph ^= 1u;
              if (!ok) break;
              tc_fence_after();
            } else {
              __syncwarp();  // one lane arrived for the first half by itself, and loads from tensor memory want all
            }
            if (any) {
              const uint32_t s_at = tmem + lanes + w * kTcKeys + h * kUnit8;
              float z[kUnit8 / 2];  // of eight keys: two of row a, two of row b
              tmem_ld_pairs(s_at, z);
              const float4* sc = &scales[at][h * 4];
              tmem_wait_ld();
              loaded(z);
#pragma unroll
              for (int q = 0; q < kUnit8 / 16; ++q) {
                const float4 e4 = sc[q];
                const float2 ca = make_float2(e4.x * rsc_a, e4.x * rsc_a), cb = make_float2(e4.x * rsc_b, e4.x * rsc_b);
                const float2 b2 = make_float2(e4.y, e4.y);
#pragma unroll
                for (int k = q * 8; k < q * 8 + 8; k += 4) {
                  const float2 a = __ffma2_rn(make_float2(z[k], z[k + 1]), ca, b2), b = __ffma2_rn(make_float2(z[k + 2], z[k + 3]), cb, b2);
                  z[k] = a.x;
                  z[k + 1] = a.y;
                  z[k + 2] = b.x;
                  z[k + 3] = b.y;
                }
              }
              if (masked) {  // -inf where the row sees nothing
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const int rest = valid - h * kUnit8 - c * 32;
                  uint32_t bits = rest >= 32 ? 0xffffffffu : (rest <= 0 ? 0u : (1u << rest) - 1u);
                  if (x.some()) bits &= h == 0 ? see[c] : see[2 + c];
                  const uint32_t ba = __shfl_sync(0xffffffffu, bits, src_a) >> pair, bb = __shfl_sync(0xffffffffu, bits, src_b) >> pair;
#pragma unroll
                  for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                      float* y = z + c * 16 + k * 4 + j;
                      y[0] = (ba >> (k * 8 + j)) & 1u ? y[0] : -INFINITY;
                      y[2] = (bb >> (k * 8 + j)) & 1u ? y[2] : -INFINITY;
                    }
                }
              }
              float ta[2], tb[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                ta[k] = fmaxf(z[4 * k], z[4 * k + 1]);
                tb[k] = fmaxf(z[4 * k + 2], z[4 * k + 3]);
              }
#pragma unroll
              for (int q = 8; q < kUnit8 / 2; q += 8)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  ta[k] = fmaxf(fmaxf(ta[k], z[q + 4 * k]), z[q + 4 * k + 1]);
                  tb[k] = fmaxf(fmaxf(tb[k], z[q + 4 * k + 2]), z[q + 4 * k + 3]);
                }
              float za = fmaxf(ta[0], ta[1]), zb = fmaxf(tb[0], tb[1]);
#pragma unroll
              for (int o = 1; o < 4; o <<= 1) {
                za = fmaxf(za, __shfl_xor_sync(0xffffffffu, za, o));
                zb = fmaxf(zb, __shfl_xor_sync(0xffffffffu, zb, o));
              }
              const bool move_a = za > m + kLazy8 || (m == -INFINITY && za > -INFINITY);
              const bool move_b = zb > m_b + kLazy8 || (m_b == -INFINITY && zb > -INFINITY);
              if (__any_sync(0xffffffffu, move_a || move_b)) {
                const float fa = move_a ? (m == -INFINITY ? 0.f : ex2(m - za)) : 1.f;
                const float fb = move_b ? (m_b == -INFINITY ? 0.f : ex2(m_b - zb)) : 1.f;
                m = move_a ? za : m;
                m_b = move_b ? zb : m_b;
                l2.x *= fa;
                l2.y *= fa;
                l3.x *= fb;
                l3.y *= fb;
                if (i > first || h > 0) {  // as below
                  if (mine_tc > 0) ok = warp_wait(&o_done[w], (mine_tc - 1) & 1);
                  if (h > 0) ok = ok && warp_wait(&o_half[w], mine_tc & 1);
                  if (!ok) break;
                  __syncwarp();
                  tc_fence_after();
                  const float f = of_row(fa, fb);
#pragma unroll 1
                  for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    tmem_ld16(o_at + c * 16, o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st16(o_at + c * 16, o);
                  }
                }
              }
              const float ref_a = m == -INFINITY ? 0.f : m - kTop8, ref_b = m_b == -INFINITY ? 0.f : m_b - kTop8;
              const float2 na = make_float2(-ref_a, -ref_a), nb = make_float2(-ref_b, -ref_b);
              uint32_t p[16];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float iv = sc[k / 2].z;
                const float2 i2 = make_float2(iv, iv);
                const float* y = z + k * 4;
                const float2 a = __fadd2_rn(make_float2(y[0], y[1]), na);
                const float2 b = __fadd2_rn(make_float2(y[2], y[3]), nb);
                const float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
                l2 = __ffma2_rn(ea, i2, l2);
                l3 = __ffma2_rn(eb, i2, l3);
                p[2 * k] = pack2<__half>(ea.x, ea.y);
                p[2 * k + 1] = pack2<__half>(eb.x, eb.y);
              }
              tmem_st_pairs(s_at, p);
              tc_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[w * 2 + h]);
          }
        } else {
#pragma unroll 1
          for (int h = 0; h * kUnit8 < n16; ++h) {
            uint32_t bits[2] = {0xffffffffu, 0xffffffffu};
            if (masked && any) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int rest = valid - h * kUnit8 - c * 32;
                bits[c] = rest >= 32 ? 0xffffffffu : (rest <= 0 ? 0u : (1u << rest) - 1u);
                if (x.some()) bits[c] &= h == 0 ? see[c] : see[2 + c];
              }
            }
            if (PAIR || h == 0) {
              ok = ok && warp_wait(&s_full[w * 2 + h], (s_ph >> h) & 1);
              s_ph ^= 1u << h;
              if (!ok) break;
              tc_fence_after();
            } else {
              __syncwarp();  // as above
            }
            const uint32_t s_at = tmem + lanes + w * kTcKeys + h * kUnit8;
            if (any) {
              float z[kUnit8];
              tmem_ld32(s_at, z);
              tmem_ld32(s_at + 32, z + 32);
              const float4* sc = &scales[at][h * 4];
              tmem_wait_ld();
              loaded(z);
              loaded(z + 32);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 e4 = sc[q];
                const float2 c2 = make_float2(e4.x * rsc, e4.x * rsc), b2 = make_float2(e4.y, e4.y);
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float2 y = __ffma2_rn(make_float2(z[q * 16 + k], z[q * 16 + k + 1]), c2, b2);
                  z[q * 16 + k] = y.x;
                  z[q * 16 + k + 1] = y.y;
                }
              }
              if (masked) {  // -inf where the row sees nothing
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int k = 0; k < 32; ++k) z[c * 32 + k] = (bits[c] >> k) & 1u ? z[c * 32 + k] : -INFINITY;
              }
              float top[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) top[k] = fmaxf(z[2 * k], z[2 * k + 1]);
#pragma unroll
              for (int q = 8; q < kUnit8; q += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], z[q + 2 * k]), z[q + 2 * k + 1]);
              const float zx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
              const bool move = zx > m + kLazy8 || (m == -INFINITY && zx > -INFINITY);
              if (__any_sync(0xffffffffu, move)) {
                const float f = move ? (m == -INFINITY ? 0.f : ex2(m - zx)) : 1.f;
                if (move) {
                  m = zx;
                  l2.x *= f;
                  l2.y *= f;
                  l3.x *= f;
                  l3.y *= f;
                }
                if (i > first || h > 0) {
                  // The unit before is in O.  Each barrier is at most one phase
                  // behind, as the scores here came after the products before.
                  if (mine_tc > 0) ok = warp_wait(&o_done[w], (mine_tc - 1) & 1);
                  if (h > 0) ok = ok && warp_wait(&o_half[w], mine_tc & 1);
                  if (!ok) break;
                  __syncwarp();
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    tmem_ld16(o_at + c * 16, o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st16(o_at + c * 16, o);
                  }
                }
              }
              const float ref = m == -INFINITY ? 0.f : m - kTop8;
              const float2 nr = make_float2(-ref, -ref);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                  const float iv = sc[c * 2 + k / 16].z;
                  const float2 i2 = make_float2(iv, iv);
                  const float* y = z + c * 32 + k;
                  const float2 a = __fadd2_rn(make_float2(y[0], y[1]), nr);
                  const float2 b = __fadd2_rn(make_float2(y[2], y[3]), nr);
                  const float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
                  l2 = __ffma2_rn(ea, i2, l2);
                  l3 = __ffma2_rn(eb, i2, l3);
                  p[k / 2] = pack2<__half>(ea.x, ea.y);
                  p[k / 2 + 1] = pack2<__half>(eb.x, eb.y);
                }
                tmem_st16(s_at + c * 16, p);
              }
              tc_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[w * 2 + h]);
          }
        }
      }
      if (!ok) break;
      const bool had = first < left;  // this stream's part in the segment
      if (had) {
        // o_done may be two phases behind here: the segment's last product has a
        // barrier of its own
        ok = warp_wait(&o_last[w], last_ph);
        last_ph ^= 1;
        if (!ok) break;
      }
      float l = (l2.x + l2.y) + (l3.x + l3.y);
      if (HALF) {
        float la = l2.x + l2.y, lb = l3.x + l3.y;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          la += __shfl_xor_sync(0xffffffffu, la, o);
          lb += __shfl_xor_sync(0xffffffffu, lb, o);
        }
        l = of_row(la, lb);
        m = of_row(m, m_b);
      }
      if (!PAIR && any) tmem_st2(tmem + lanes + w * kTcKeys, m, l);  // where the scores were
      tc_fence_before();
      // both streams are done: with the queries, and with each other's outputs
      mbar_arrive(&seg_end);
      ok = warp_wait(&seg_end, seg & 1);
      if (!ok) break;
      tc_fence_after();
      const int tc0 = tc;
      tc += left;
      if (!any) continue;
      const volatile C8Seg& flags = segs[seg & (kC8Segs - 1)];
      const bool poison = flags.bad != 0, odd = flags.odd != 0, whole = e.whole != 0;
      const int slot = 2 * blockIdx.x + tree_slot(e.t0 == 0);
      const int head = e.kvh * P.group + R - node * P.group;
      T* dst = static_cast<T*>(P.out) + (long long)(e.cu + node) * P.so_node + (long long)head * P.so_head;
      const long long prow = (long long)slot * P.rows + tile * kRows8 + row;
      float4* part = reinterpret_cast<float4*>(P.part_o) + (long long)slot * P.rows * (D / 4) + tile * kRows8 + row;
      // Of a row tile with two streams, each stream's threads join half of the
      // channels.
      float f0 = 1.f, f1 = 0.f;
      bool two = false;
      if (!PAIR) {
        const float2 a = tmem_ld2(tmem + lanes), b = tmem_ld2(tmem + lanes + kTcKeys);
        m = fmaxf(a.x, b.x);
        const float ref = m == -INFINITY ? 0.f : m;
        f0 = ex2(a.x - ref);
        f1 = ex2(b.x - ref);
        l = a.y * f0 + b.y * f1;
        // a stream without a tile has whatever was there before for its outputs
        two = left > 1;
        if (!two && (tc0 & 1)) f0 = f1;
      }
      const float ref = m == -INFINITY ? 0.f : m - kTop8;
      if (poison) l = NAN;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const float g0 = PAIR ? inv : f0 * inv, g1 = f1 * inv;
      const uint32_t at0 = PAIR ? o_at : tmem + lanes + 2 * kTcKeys + (two ? 0 : (tc0 & 1) * D);
      constexpr int CH = PAIR ? D : D / 2;
      const int c0 = PAIR ? 0 : w * CH;
#pragma unroll 1
      for (int c = c0; c < c0 + CH; c += 16) {
        uint32_t o[16];
        __syncwarp();
        tmem_ld16(at0 + c, o);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * g0);
        if (!PAIR && two) {
          uint32_t o1[16];
          tmem_ld16(at0 + D + c, o1);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), g1, __uint_as_float(o[k])));
        }
        if (mine && whole) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(dst + c + k) =
                make_uint4(pack2<T>(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), pack2<T>(__uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])),
                           pack2<T>(__uint_as_float(o[k + 4]), __uint_as_float(o[k + 5])), pack2<T>(__uint_as_float(o[k + 6]), __uint_as_float(o[k + 7])));
        } else if (mine) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<uint4*>(&part[((c + k) / 4) * P.rows]) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      if (mine) {
        if (odd)
          c8_add_odd<T>(P, e.b, e.kvh, e.t0, e.t1, seen, see_lo, node, c0, c0 + CH, whole ? dst : nullptr, part);
        if (PAIR || w == 0) {
          if (!whole)
            P.part_ml[prow] = make_float4(m == -INFINITY ? m : ref, l, l, 0.f);
          else if (P.lse)
            P.lse[(long long)(e.cu + node) * P.heads * P.group + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
        }
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
  if (warp == kC8Softmax + kC8Convert + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// A map of bytes, a head's channels per row of a box.
bool encode8(CUtensorMap* m, const TreeParams& P, const void* base, int box) {
  EncodeTiled f = encoder();
  if (!f) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)P.dim, (cuuint64_t)P.page_size, (cuuint64_t)P.heads, (cuuint64_t)P.num_pages};
  const long long st[3] = {P.s_slot, P.s_head, P.s_page};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) strides[i] = dims[i + 1] == 1 ? 512 : (cuuint64_t)st[i];
  const cuuint32_t bx[4] = {(cuuint32_t)P.dim, (cuuint32_t)box, 1, 1}, one[4] = {1, 1, 1, 1};
  // What a miss brings to L2: not more than a row, unless the rows of a head lie
  // together.  With 256 bytes, 128 K tokens of 8 heads cost 735 MB of DRAM reads
  // for 490.
  const CUtensorMapL2promotion promotion = P.s_slot == P.dim ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : P.dim == 64     ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                             : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, bx, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, P.dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
           promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int ROWS>
int launch_c8(const Cache8Params& C, const C8Maps& maps, int box, cudaStream_t s) {
  using S = C8Shape<D, (ROWS > kRows8)>;
  if (cudaFuncSetAttribute(cache8_tc_kernel<T, D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(cache8_tc_kernel<T, D, ROWS>, dim3(C.t.grid), kC8TcThreads, S::kSmem, s, C, maps, box);
}

template <typename T, int D>
int launch_c8_shape(const Cache8Params& C, const C8Maps& maps, int box, cudaStream_t s) {
  switch (C.t.rows) {
    case kRows8 / 2: return launch_c8<T, D, kRows8 / 2>(C, maps, box, s);
    case kRows8: return launch_c8<T, D, kRows8>(C, maps, box, s);
    default: return launch_c8<T, D, 2 * kRows8>(C, maps, box, s);
  }
}

template <typename T>
int launch_c8_dim(const Cache8Params& C, const C8Maps& maps, int box, cudaStream_t s) {
  return C.t.dim == 64 ? launch_c8_shape<T, 64>(C, maps, box, s) : launch_c8_shape<T, 128>(C, maps, box, s);
}

}  // namespace

// Heads of 64 or 128 channels; pages and blocks of a multiple of 16 tokens, so
// that 16 keys of a tile have one scale and a box of a copy fills whole swizzle
// patterns.
bool cache8_tc_fits(int dim, int page_size, int block) {
  return (dim == 64 || dim == 128) && page_size % 16 == 0 && block % 16 == 0;
}

TreePlan plan_cache8_tc(int rows, int num_sms) {
  TreePlan p;
  p.kernel = 1;
  p.grid = num_sms;
  p.rows = rows > kRows8 ? 2 * kRows8 : rows > kRows8 / 2 ? kRows8 : kRows8 / 2;
  p.kt = kTcKeys;
  return p;
}

int launch_cache8_tc(const Cache8Params& C, bool bf16, cudaStream_t s) {
  C8Maps maps;
  const int box = page_box(C.t.page_size);
  if (!encode8(&maps.k, C.t, C.t.k, box) || !encode8(&maps.v, C.t, C.t.v, box)) return -1;
  return bf16 ? launch_c8_dim<__nv_bfloat16>(C, maps, box, s) : launch_c8_dim<__half>(C, maps, box, s);
}

}  // namespace sv
