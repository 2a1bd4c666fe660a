// Attention of drafted trees over a paged cache in 8 bits: warp tiles on
// mma.sync.
#include "cache8_common.cuh"

namespace sv {
namespace {

constexpr int kW8Warps = 4;
constexpr int kW8Keys = 16 * kW8Warps;  // keys per tile: 16 per warp

template <int D>
struct W8Shape {
  // Bytes per staged row.  Keys are read by 8 bytes, 4 rows of 32 at once:
  // rows an odd number of 32 bytes apart; values by 4, every second row: rows an
  // odd number of 16.
  static constexpr int kKeyPitch = (D / 32) % 2 ? D : D + 32;
  static constexpr int kValPitch = D + 16;
  static constexpr int kScales = 16 * (kKeyPitch + kValPitch);  // 16 of keys, 16 of values
  static constexpr int kWarpStage = kScales + 128;
  static constexpr int kStage = kW8Warps * kWarpStage;
  static constexpr int kStages = D <= 64 ? 8 : (D <= 96 ? 7 : (D <= 128 ? 5 : (D <= 192 ? 6 : 5)));
  static constexpr int kSmem = kStage * kStages + 2 * 16 * kW8Warps * 4;
  static constexpr int kCtas = D <= 128 ? 2 : 1;  // per SM
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

// e4m3 NaN bytes as zero bytes, and whether there were any.
__device__ __forceinline__ uint32_t without_nan8(uint32_t w, bool& any) {
  const uint32_t nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  any = any || nan != 0u;
  return w & ~nan;
}

// As the 16-bit warp tiles (16 rows, 16 keys a warp and tile, asynchronous copies
// in flight per warp, a running maximum per row), on fp16 operands:
//   s_j = scale ks_j (q . k8_j),  w_j = 2^(log2(e) s_j + log2 vs_j - m),
//   O += w_j v8_j,  l += w_j / vs_j,  out = O / l.
// A value's scale goes into its weight's exponent, so the bytes' values are the
// matrix operands as they are (one conversion for two of them).  The order of
// channels is the threads' own: a thread reads 8 bytes of a key for two steps of
// 16 channels, and 4 channels of 4 keys for the values, whose bytes it pairs by
// key before they are converted, so neither needs a transposition.
//
// It serves the calls that the tensor-memory kernel does not take.  64 requests of
// one token over up to 8192 tokens, 28 / 4 heads of 128, would take 160 us (125
// there), and 9 nodes of them, five row tiles that read the keys anew, 467 (115): the
// conversions and products of few rows bound it, not the copies.
template <typename T, int D>
__global__ void __launch_bounds__(kW8Warps * 32, W8Shape<D>::kCtas) cache8_warp_kernel(const Cache8Params C) {
  using S = W8Shape<D>;
  constexpr int B32 = D / 32;   // blocks of 32 channels
  constexpr int CH = D / 16;    // 16-byte pieces per row
  constexpr int NLD = D / 32;   // pieces per lane for 16 rows
  extern __shared__ __align__(128) unsigned char smem[];
  float* ml = reinterpret_cast<float*>(smem + S::kStage * S::kStages);  // [warp][16] m, then l
  const TreeParams& P = C.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = lane >> 2, t4 = lane & 3;
  unsigned char* ring = smem + warp * S::kWarpStage;
  const PageDiv pd(P.page_size), sd(C.block);
  const uint8_t* kc = static_cast<const uint8_t*>(P.k);
  const uint8_t* vc = static_cast<const uint8_t*>(P.v);
  const T* kn = static_cast<const T*>(P.k_new);
  const T* vn = static_cast<const T*>(P.v_new);
  const T* q = static_cast<const T*>(P.q);
  const uint32_t em = exp_mask<T>();

  after_previous();
  const TreeScan scan = tree_scan<true>(P, lane);
  if (blockIdx.x == 0 && warp == 0) tree_store_starts<true>(P, scan, lane);
  TreeWalkOf<true> walk;
  walk.begin(P, lane, scan, blockIdx.x);
  TreeSeg g;
  while (walk.next(P, g)) {
    const TreeReq& r = walk.r;
    const int row_lo = g.m * 16;
    const int nrows = min(16, r.n * P.group - row_lo);
    // Q fragments, rows r0 and r0 + 8: step 2i + s has of this thread the
    // channels 32i + 8 t4 + 4s .. + 3
    uint32_t qf[2 * B32][4];
    int node[2];
    float sc_row[2];
    TreeRow win[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rr = r0 + 8 * h;
      const bool in = rr < nrows;
      node[h] = in ? (row_lo + rr) / P.group : 0;
      const T* src = q + (long long)(r.cu + node[h]) * P.sq_node +
                     (long long)(g.kvh * P.group + (in ? (row_lo + rr) % P.group : 0)) * P.sq_head + 8 * t4;
      uint4 v[B32];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < B32; ++i) {
        v[i] = in ? load16(src + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
        top = max_u16x2(top, max_u16x2(max_u16x2(finite_size2(v[i].x, em), finite_size2(v[i].y, em)),
                                     max_u16x2(finite_size2(v[i].z, em), finite_size2(v[i].w, em))));
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const Exact16 x = exact16<T>(top);
      sc_row[h] = P.scale_log2 * x.back;
#pragma unroll
      for (int i = 0; i < B32; ++i) {
        qf[2 * i][h] = to_f16x2<T>(v[i].x, x.to);
        qf[2 * i][2 + h] = to_f16x2<T>(v[i].y, x.to);
        qf[2 * i + 1][h] = to_f16x2<T>(v[i].z, x.to);
        qf[2 * i + 1][2 + h] = to_f16x2<T>(v[i].w, x.to);
      }
      win[h] = tree_row(P, r, node[h]);
    }
    // O: o[4j + i][2h + e] is channel 32j + 8 t4 + 4e + i of row r0 + 8h
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int bad = 0;
    __syncthreads();  // the last segment's join is done with the ring

    auto load = [&](int t) {
      if (t >= g.t1) return;
      const TreeKeys tk = tree_keys<true>(r, kW8Keys, t);
      const int lo = tk.lo + warp * 16, lim = tk.lim;
      if (!tk.cached || lo >= lim) return;
      const int j = lo + (lane & 15);
      bool real = j < lim;
      long long off = 0, at = 0;
      if (real) {
        int page, slot, blk, rest;
        pd.split(j, page, slot);
        sd.split(slot, blk, rest);
        const int id = P.table[(long long)g.b * P.ld_table + page];
        if (id < 0 || id >= P.num_pages) {
          bad = 1;
          real = false;
        } else {
          off = (long long)id * P.s_page + (long long)slot * P.s_slot + (long long)g.kvh * P.s_head;
          at = (long long)id * C.c_page + (long long)blk * C.c_block + (long long)g.kvh * C.c_head;
        }
      }
      const uint32_t dst = smem_u32(ring + (t % S::kStages) * S::kStage);
      cp_async4(dst + S::kScales + lane * 4, (lane < 16 ? C.ks : C.vs) + at, real);
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int idx = i * 32 + lane, row = idx / CH, ch = idx % CH;
        const long long ro = __shfl_sync(0xffffffffu, off, row);
        const bool rl = __shfl_sync(0xffffffffu, (int)real, row) != 0;
        cp_async16(dst + row * S::kKeyPitch + ch * 16, kc + ro + ch * 16, rl);
        cp_async16(dst + 16 * S::kKeyPitch + row * S::kValPitch + ch * 16, vc + ro + ch * 16, rl);
      }
    };

#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      load(g.t0 + i);
      cp_async_commit();
    }
    for (int t = g.t0; t < g.t1; ++t) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      load(t + S::kStages - 1);  // into the slot that tile t - 1 left
      cp_async_commit();
      const TreeKeys tk = tree_keys<true>(r, kW8Keys, t);
      const bool cached = tk.cached;
      const int lo = tk.lo + warp * 16, lim = tk.lim;
      if (lo >= lim) continue;  // warp-uniform
      // keys that some rows see and others do not: drafted, or at a window's beginning
      const bool some = !cached || (t >= r.st && lo < r.part);
      const unsigned char* kb = ring + (t % S::kStages) * S::kStage;
      const unsigned char* vb = kb + 16 * S::kKeyPitch;
      // this thread's keys of the scores: 8 nt + 2 t4 + e; of keys for the
      // product, 8 nt + r0; of values 2 t4, + 1, + 8, + 9
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float ks[2][2], vs[2][2];
      Exact16 xv = {1.f, 1.f};
      uint32_t odd = 0;
      if (cached) {
        const float* sc = reinterpret_cast<const float*>(kb + S::kScales);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float2 a = *reinterpret_cast<const float2*>(sc + nt * 8 + 2 * t4);
          const float2 b = *reinterpret_cast<const float2*>(sc + 16 + nt * 8 + 2 * t4);
          ks[nt][0] = a.x;
          ks[nt][1] = a.y;
          vs[nt][0] = b.x;
          vs[nt][1] = b.y;
        }
#pragma unroll
        for (int i = 0; i < B32; ++i) {
          const uint2 a = *reinterpret_cast<const uint2*>(kb + r0 * S::kKeyPitch + i * 32 + t4 * 8);
          const uint2 b = *reinterpret_cast<const uint2*>(kb + (8 + r0) * S::kKeyPitch + i * 32 + t4 * 8);
          mma16816<__half>(s[0], qf[2 * i], e4m3x2_f16x2(a.x & 0xffffu), e4m3x2_f16x2(a.x >> 16));
          mma16816<__half>(s[1], qf[2 * i], e4m3x2_f16x2(b.x & 0xffffu), e4m3x2_f16x2(b.x >> 16));
          mma16816<__half>(s[0], qf[2 * i + 1], e4m3x2_f16x2(a.y & 0xffffu), e4m3x2_f16x2(a.y >> 16));
          mma16816<__half>(s[1], qf[2 * i + 1], e4m3x2_f16x2(b.y & 0xffffu), e4m3x2_f16x2(b.y >> 16));
        }
      } else {
        // Drafted keys and values come straight from global memory, twice: their
        // largest sizes first, which scale all 16 of them.
        const long long head = (long long)g.kvh * P.sn_head;
        const long long at0 = (long long)(r.cu + min(lo + r0, lim - 1)) * P.sn_node + head + 8 * t4;
        const long long at1 = (long long)(r.cu + min(lo + 8 + r0, lim - 1)) * P.sn_node + head + 8 * t4;
        const T *k0 = kn + at0, *k1 = kn + at1, *v0 = vn + at0, *v1 = vn + at1;
        uint32_t kt = 0, vt = 0;
#pragma unroll
        for (int i = 0; i < B32; ++i) {
          const uint4 x[2] = {load16(k0 + 32 * i), load16(k1 + 32 * i)};
#pragma unroll
          for (int z = 0; z < 2; ++z)
            kt = max_u16x2(kt, max_u16x2(max_u16x2(finite_size2(x[z].x, em), finite_size2(x[z].y, em)),
                                       max_u16x2(finite_size2(x[z].z, em), finite_size2(x[z].w, em))));
          const uint4 y[2] = {load16(v0 + 32 * i), load16(v1 + 32 * i)};
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t w[4] = {y[z].x, y[z].y, y[z].z, y[z].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              vt = max_u16x2(vt, finite_size2(w[c], em));
              odd |= (uint32_t)((w[c] & em) == em || ((w[c] >> 16) & em) == em);
            }
          }
        }
        kt = max(kt & 0xffffu, kt >> 16);
        vt = max(vt & 0xffffu, vt >> 16);
#pragma unroll
        for (int z = 16; z > 0; z >>= 1) {
          kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, z));
          vt = max(vt, __shfl_xor_sync(0xffffffffu, vt, z));
        }
        const Exact16 xk = exact16<T>(kt);
        xv = exact16<T>(vt);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[nt][e] = xk.back;
            vs[nt][e] = xv.back;
          }
#pragma unroll
        for (int i = 0; i < B32; ++i) {
          const uint4 a = load16(k0 + 32 * i), b = load16(k1 + 32 * i);
          mma16816<__half>(s[0], qf[2 * i], to_f16x2<T>(a.x, xk.to), to_f16x2<T>(a.y, xk.to));
          mma16816<__half>(s[1], qf[2 * i], to_f16x2<T>(b.x, xk.to), to_f16x2<T>(b.y, xk.to));
          mma16816<__half>(s[0], qf[2 * i + 1], to_f16x2<T>(a.z, xk.to), to_f16x2<T>(a.w, xk.to));
          mma16816<__half>(s[1], qf[2 * i + 1], to_f16x2<T>(b.z, xk.to), to_f16x2<T>(b.w, xk.to));
        }
      }
      uint32_t see[2];
      if (cached) {
        const int left = lim - lo;
        see[0] = see[1] = left >= 16 ? 0xffffu : (1u << left) - 1u;
        if (some) {
          see[0] &= tree_window32(lo, win[0].lo, P.sinks);
          see[1] &= tree_window32(lo, win[1].lo, P.sinks);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          see[h] = tree_window_drafted(P, r, win[h], node[h], lo, tree_bits16(P, r.cu, r.n, node[h], lo));
      }
      float mx[2] = {-INFINITY, -INFINITY};
      float iv[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float v = vs[nt][c] < kLeastScale ? kLeastScale : vs[nt][c];  // NaN stays
          const float lv = log2f(v);
          iv[nt][c] = 1.f / v;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& z = s[nt][2 * h + c];
            z = ((see[h] >> (nt * 8 + 2 * t4 + c)) & 1u) ? fmaf(z, sc_row[h] * ks[nt][c], lv) : -INFINITY;
            mx[h] = fmaxf(mx[h], z);
          }
        }
      float sc[2], ref[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        const float mn = fmaxf(m[h], mx[h] - kHead16);
        ref[h] = mn == -INFINITY ? 0.f : mn;
        sc[h] = ex2(m[h] - ref[h]);
        m[h] = mn;
        l[h] *= sc[h];
      }
      uint32_t pf[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(s[nt][e] - ref[e >> 1]);
          l[e >> 1] += p[e] == 0.f ? 0.f : p[e] * iv[nt][e & 1];  // the scale of a hidden key may be NaN
        }
        // the values of a scale that counts as 0
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = vs[nt][e & 1] < kLeastScale ? 0.f : p[e];
        pf[2 * nt] = pack2<__half>(p[0], p[1]);
        pf[2 * nt + 1] = pack2<__half>(p[2], p[3]);
      }
      if (__any_sync(0xffffffffu, sc[0] != 1.f || sc[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= sc[0];
          o[i][1] *= sc[0];
          o[i][2] *= sc[1];
          o[i][3] *= sc[1];
        }
      }
      // A value that some rows do not see must not reach them, but 0 times an
      // infinity or NaN would: such values are zero for the product, and added
      // here to the rows that see them.
      bool any = odd != 0u;
      if (cached && some)
        for (int i = lane; i < 16 * (D / 4); i += 32)
          without_nan8(*reinterpret_cast<const uint32_t*>(vb + i / (D / 4) * S::kValPitch + i % (D / 4) * 4), any);
      const bool strip = some && __any_sync(0xffffffffu, any);
      if (strip)
        for (int key = 0; key < 16 && lo + key < lim; ++key)
#pragma unroll
          for (int j = 0; j < B32; ++j)
#pragma unroll
            for (int c = 0; c < 8; ++c) {  // channel 32j + 8 t4 + c
              float x;
              if (cached) {
                x = (vb[key * S::kValPitch + 32 * j + 8 * t4 + c] & 0x7f) == 0x7f ? NAN : 0.f;
              } else {
                const uint32_t w = reinterpret_cast<const uint16_t*>(vn)[(long long)(r.cu + lo + key) * P.sn_node +
                                                                         (long long)g.kvh * P.sn_head + 32 * j + 8 * t4 + c];
                x = (w & em) == em ? half_to_f32<T>(w) : 0.f;
              }
              if (x != 0.f) {
                if ((see[0] >> key) & 1u) o[4 * j + (c & 3)][c >> 2] += x;
                if ((see[1] >> key) & 1u) o[4 * j + (c & 3)][2 + (c >> 2)] += x;
              }
            }
#pragma unroll
      for (int j = 0; j < B32; ++j) {
        uint32_t b[4][2];  // column i: keys 2 t4 and + 1, and those 8 further, of channel 32j + 4 r0 + i
        if (cached) {
          const unsigned char* at = vb + 2 * t4 * S::kValPitch + 32 * j + 4 * r0;
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = *reinterpret_cast<const uint32_t*>(at + ((k & 1) + (k >> 1) * 8) * S::kValPitch);
            if (strip) {
              bool z = false;
              w[k] = without_nan8(w[k], z);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x = __byte_perm(w[2 * k], w[2 * k + 1], 0x5140), y = __byte_perm(w[2 * k], w[2 * k + 1], 0x7362);
            b[0][k] = e4m3x2_f16x2(x & 0xffffu);
            b[1][k] = e4m3x2_f16x2(x >> 16);
            b[2][k] = e4m3x2_f16x2(y & 0xffffu);
            b[3][k] = e4m3x2_f16x2(y >> 16);
          }
        } else {
          uint2 w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = lo + 2 * t4 + (k & 1) + (k >> 1) * 8;
            w[k] = make_uint2(0u, 0u);
            if (key < lim)
              w[k] = *reinterpret_cast<const uint2*>(vn + (long long)(r.cu + key) * P.sn_node +
                                                     (long long)g.kvh * P.sn_head + 32 * j + 4 * r0);
            if (strip) {
              uint32_t* e = reinterpret_cast<uint32_t*>(&w[k]);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if ((e[c] & em) == em) e[c] &= 0xffff0000u;
                if (((e[c] >> 16) & em) == em) e[c] &= 0xffffu;
              }
            }
            w[k].x = to_f16x2<T>(w[k].x, xv.to);
            w[k].y = to_f16x2<T>(w[k].y, xv.to);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            b[0][k] = __byte_perm(w[2 * k].x, w[2 * k + 1].x, 0x5410);
            b[1][k] = __byte_perm(w[2 * k].x, w[2 * k + 1].x, 0x7632);
            b[2][k] = __byte_perm(w[2 * k].y, w[2 * k + 1].y, 0x5410);
            b[3][k] = __byte_perm(w[2 * k].y, w[2 * k + 1].y, 0x7632);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma16816<__half>(o[4 * j + i], pf, b[i][0], b[i][1]);
      }
      __syncwarp();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    const bool poison = __syncthreads_or(bad) != 0;  // and every warp is done with its ring
    float* so = reinterpret_cast<float*>(smem);  // [warp][16][D]
#pragma unroll
    for (int j = 0; j < B32; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(so + (warp * 16 + r0 + 8 * h) * D + 32 * j + 8 * t4 + 4 * e) =
              make_float4(o[4 * j][2 * h + e], o[4 * j + 1][2 * h + e], o[4 * j + 2][2 * h + e], o[4 * j + 3][2 * h + e]);
    if (t4 == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ml[warp * 16 + r0 + 8 * h] = m[h];
        ml[16 * kW8Warps + warp * 16 + r0 + 8 * h] = l[h];
      }
    }
    __syncthreads();
    const bool whole = g.t0 == 0 && g.t1 == r.per_item;
    const int slot = 2 * blockIdx.x + tree_slot(g.t0 == 0);
    for (int i = tid; i < nrows * (D / 2); i += kW8Warps * 32) {
      const int row = i / (D / 2), d = (i % (D / 2)) * 2;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kW8Warps; ++w) M = fmaxf(M, ml[w * 16 + row]);
      const float R = M == -INFINITY ? 0.f : M;
      float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kW8Warps; ++w) {
        const float f = ex2(ml[w * 16 + row] - R);
        L += ml[16 * kW8Warps + w * 16 + row] * f;
        const float2 v = *reinterpret_cast<const float2*>(so + (w * 16 + row) * D + d);
        x += v.x * f;
        y += v.y * f;
      }
      if (poison) L = x = y = NAN;
      const int R2 = row_lo + row;
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int nd = R2 / P.group, head = g.kvh * P.group + R2 % P.group;
        T* dst = static_cast<T*>(P.out) + (long long)(r.cu + nd) * P.so_node + (long long)head * P.so_head;
        *reinterpret_cast<uint32_t*>(dst + d) = pack2<T>(x * inv, y * inv);
        if (P.lse && d == 0)
          P.lse[(long long)(r.cu + nd) * P.heads * P.group + head] = L == 0.f ? -INFINITY : (R + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float2*>(P.part_o + (((long long)slot * (D / 4) + d / 4) * 16 + row) * 4 + d % 4) = make_float2(x, y);
        if (d == 0) P.part_ml[(long long)slot * 16 + row] = make_float4(M, L, L, 0.f);
      }
    }
  }
}

template <typename T, int D>
int launch_warp8(const Cache8Params& C, cudaStream_t s) {
  using S = W8Shape<D>;
  if (cudaFuncSetAttribute(cache8_warp_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
      cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return launch_kernel(cache8_warp_kernel<T, D>, dim3(C.t.grid), kW8Warps * 32, S::kSmem, s, C);
}

template <typename T>
int launch_warp8_dim(const Cache8Params& C, cudaStream_t s) {
  switch (C.t.dim) {
    case 64: return launch_warp8<T, 64>(C, s);
    case 96: return launch_warp8<T, 96>(C, s);
    case 128: return launch_warp8<T, 128>(C, s);
    case 192: return launch_warp8<T, 192>(C, s);
    case 256: return launch_warp8<T, 256>(C, s);
    default: return -1;
  }
}

}  // namespace

TreePlan plan_cache8_warp(int dim, int num_sms) {
  TreePlan p;
  p.kernel = 0;
  p.rows = 16;
  p.kt = kW8Keys;
  p.grid = num_sms * (dim <= 128 ? 2 : 1);
  return p;
}

int launch_cache8_warp(const Cache8Params& C, bool bf16, cudaStream_t s) {
  return bf16 ? launch_warp8_dim<__nv_bfloat16>(C, s) : launch_warp8_dim<__half>(C, s);
}

}  // namespace sv
