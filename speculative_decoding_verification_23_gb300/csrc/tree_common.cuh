// Device helpers shared by the drafted-tree kernels: the even split of all
// attention tiles over the CTAs, cached-token addresses, 16-bit types.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "tree_internal.h"
#include "tree_launch.cuh"

namespace sv {
namespace {

constexpr float kLn2 = 0.693147180559945309f;

// Two floats to a pair of 16-bit values (the first in the low half).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The bits of a 16-bit type's exponent, all set for infinities and NaN.
template <typename T>
__device__ __forceinline__ uint32_t exp_mask();
template <>
__device__ __forceinline__ uint32_t exp_mask<__nv_bfloat16>() { return 0x7f80u; }
template <>
__device__ __forceinline__ uint32_t exp_mask<__half>() { return 0x7c00u; }

template <typename T>
__device__ __forceinline__ float half_to_f32(uint32_t bits);
template <>
__device__ __forceinline__ float half_to_f32<__nv_bfloat16>(uint32_t bits) { return __uint_as_float(bits << 16); }
template <>
__device__ __forceinline__ float half_to_f32<__half>(uint32_t bits) {
  return __half2float(__ushort_as_half((unsigned short)bits));
}

// ------------------------------------------------ the even split of tiles
struct TreeReq {
  int n, ctx, cu;     // drafted tokens, cached tokens, first row
  int ct, per_item;   // tiles of cached keys, of all keys
  int mb;             // row blocks per head
  bool ok;
  long long tiles;    // of all items
};

__device__ __forceinline__ TreeReq tree_request(const TreeParams& P, int b) {
  TreeReq r;
  r.cu = P.cu[b];
  const int hi = P.cu[b + 1];
  r.n = hi - r.cu;
  r.ctx = P.ctx[b];
  r.ok = r.cu >= 0 && hi <= P.total && r.n >= 0 && r.n <= P.max_nodes && r.ctx >= 0 &&
         (long long)r.ctx <= (long long)P.ld_table * P.page_size;
  // unsigned and by shifts: every role of a CTA does this before it begins
  const int kt_shift = 31 - __clz(P.kt);  // a power of two
  r.ct = (int)(((uint32_t)r.ctx + (uint32_t)P.kt - 1u) >> kt_shift);
  r.per_item = r.ct + (int)(((uint32_t)r.n + (uint32_t)P.kt - 1u) >> kt_shift);
  r.mb = (int)((uint32_t)(r.n * P.group + P.rows - 1) / (uint32_t)P.rows);
  if (P.weigh) {
    r.ok = r.ok && r.n <= r.ctx && r.ctx <= P.ld;
    r.per_item = r.ct;
    r.mb = r.n > 0 ? 1 : 0;  // a request without rows has no tiles
  }
  r.tiles = r.ok ? (long long)r.per_item * r.mb * P.heads : 0;
  return r;
}

// A warp's view of all requests: lane l owns requests [l*per, (l+1)*per).
struct TreeScan {
  long long before, mine, total;
  int per;
  bool idle;  // this lane has a request of cached tokens without rows
};

__device__ __forceinline__ TreeScan tree_scan(const TreeParams& P, int lane) {
  TreeScan s;
  s.per = (P.B + 31) / 32;
  s.mine = 0;
  s.idle = false;
  for (int b = lane * s.per; b < min(P.B, (lane + 1) * s.per); ++b) {
    const TreeReq r = tree_request(P, b);
    s.mine += r.tiles;
    s.idle = s.idle || (r.ok && r.n == 0 && r.ctx > 0);
  }
  long long v = s.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  s.before = v - s.mine;
  s.total = __shfl_sync(0xffffffffu, v, 31);
  return s;
}

// The request that holds tile x (x < total) and its first tile.
__device__ __forceinline__ int tree_locate(const TreeParams& P, const TreeScan& s, int lane, long long x,
                                           long long* first) {
  const bool me = x >= s.before && x < s.before + s.mine;
  int rb = 0;
  long long rs = s.before;
  if (me) {
    for (rb = lane * s.per;; ++rb) {
      const long long t = tree_request(P, rb).tiles;
      if (x < rs + t) break;
      rs += t;
    }
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
  *first = __shfl_sync(0xffffffffu, rs, src);
  return __shfl_sync(0xffffffffu, rb, src);
}

// The first tile of each request, for the kernel that joins split items.
__device__ __forceinline__ void tree_store_starts(const TreeParams& P, const TreeScan& s, int lane) {
  long long at = s.before;
  for (int b = lane * s.per; b < min(P.B, (lane + 1) * s.per); ++b) {
    P.start[b] = at;
    at += tree_request(P, b).tiles;
  }
  if (lane == 0) P.start[P.B] = s.total;
}

// a / b, by 32-bit division (several times faster) where both fit.
__device__ __forceinline__ long long div_fast(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// CTA c of the G in use takes tiles [c*T/G, (c+1)*T/G), at least one each; and
// the CTA that holds tile x.
__device__ __forceinline__ int tree_used(const TreeParams& P, long long T) { return (int)min((long long)P.grid, T); }
__device__ __forceinline__ long long tree_range(long long c, long long T, int G) { return div_fast(c * T, G); }
__device__ __forceinline__ int tree_owner(long long x, long long T, int G) {
  return (int)div_fast((x + 1) * G + T - 1, T) - 1;
}

// A run of tiles of one item inside a CTA's range (of the walk's request).
struct TreeSeg {
  int b, kvh, m;   // request, key/value head, row block
  int t0, t1;      // its tiles
};

// Walks a CTA's range segment by segment; every warp walks by itself.
struct TreeWalk {
  long long x, end, first;
  TreeReq r;
  int b;
  __device__ __forceinline__ void begin(const TreeParams& P, int lane, const TreeScan& s, int cta) {
    const int used = tree_used(P, s.total);
    x = cta < used ? tree_range(cta, s.total, used) : 0;
    end = cta < used ? tree_range(cta + 1, s.total, used) : 0;
    b = 0;
    first = 0;
    if (x < end) {
      b = tree_locate(P, s, lane, x, &first);
      r = tree_request(P, b);
    }
  }
  __device__ __forceinline__ bool next(const TreeParams& P, TreeSeg& g) {
    if (x >= end) return false;
    while (x >= first + r.tiles) {  // ends: some request holds tile x < total
      first += r.tiles;
      r = tree_request(P, ++b);
    }
    const long long off = x - first;
    const int item = (int)div_fast(off, r.per_item);
    g.b = b;
    g.t0 = (int)(off - (long long)item * r.per_item);
    g.t1 = (int)min((long long)r.per_item, g.t0 + (end - x));
    g.kvh = item / r.mb;
    g.m = item - g.kvh * r.mb;
    x += g.t1 - g.t0;
    return true;
  }
};

// Slot of a CTA's partial result: 0 where the item began in an earlier CTA.
__device__ __forceinline__ int tree_slot(bool item_begins_here) { return item_begins_here ? 1 : 0; }

// The 16 mask bits of node `i` for drafted keys base .. base + 15 (base a
// multiple of 16) of a tree of n nodes.
__device__ __forceinline__ uint32_t tree_bits16(const TreeParams& P, int cu, int n, int i, int base) {
  uint32_t bits;
  if (P.mask) {
    bits = (base >> 5) < P.mask_words
               ? P.mask[(long long)(cu + i) * P.mask_words + (base >> 5)] >> (base & 31)
               : 0u;
  } else {
    const int k = i - base;
    bits = k < 0 ? 0u : (k >= 15 ? 0xffffu : (2u << k) - 1u);
  }
  const int left = n - base;
  return left >= 16 ? (bits & 0xffffu) : (left <= 0 ? 0u : bits & ((1u << left) - 1u));
}

// Division of a token's position by the page size: a shift where it is a
// power of two (shift >= 0).
struct PageDiv {
  int size, shift;
  __device__ __forceinline__ explicit PageDiv(int s) {
    size = s;
    shift = (s & (s - 1)) == 0 ? 31 - __clz(s) : -1;
  }
  __device__ __forceinline__ void split(int j, int& page, int& slot) const {
    if (shift >= 0) {
      page = j >> shift;
      slot = j & (size - 1);
    } else {
      page = j / size;
      slot = j - page * size;
    }
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += a b for 16x8 tiles over 16 values.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace
}  // namespace sv
