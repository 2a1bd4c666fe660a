// Device helpers of the 8-bit cache: e4m3 conversions, and exact forms of
// 16-bit values in fp16.
#pragma once

#include "serve_internal.h"
#include "tree_common.cuh"

namespace sv {
namespace {

// Two e4m3 bytes to two fp16 values (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  const uint32_t h = e4m3x2_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two floats to e4m3 bytes, the first in the low one.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// The larger of each of two 16-bit whole numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The sizes of two 16-bit values, infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite_size2(uint32_t two, uint32_t em) {
  const uint32_t lo = two & 0x7fffu, hi = (two >> 16) & 0x7fffu;
  return (lo < em ? lo : 0u) | (hi < em ? hi : 0u) << 16;
}

// ------------------------------------------- 16-bit values exactly in fp16
// bf16 has 8 bits of a value in a range that fp16 does not have.  Scaled so that
// the largest of a set lies in [2^14, 2^15), all that is at least 2^-31 of it is
// exact in fp16, and the rest within 2^-25 of 2^15 (of a set below 2^-46, all
// within 2^-85).  fp16 values stay as they
// are.
struct Exact16 {
  float to, back;  // powers of two, of product 1
};
template <typename T>
__device__ __forceinline__ Exact16 exact16(uint32_t top);  // the largest finite size's bits
template <>
__device__ __forceinline__ Exact16 exact16<__half>(uint32_t) {
  return Exact16{1.f, 1.f};
}
template <>
__device__ __forceinline__ Exact16 exact16<__nv_bfloat16>(uint32_t top) {
  const int e = max((int)(top >> 7), 81);  // exponent + 127; `back` is 2^-60 at least
  return Exact16{__uint_as_float((uint32_t)(127 + 141 - e) << 23), __uint_as_float((uint32_t)(127 + e - 141) << 23)};
}
// Two values of T to fp16 (infinities and NaN stay).
template <typename T>
__device__ __forceinline__ uint32_t to_f16x2(uint32_t two, float to);
template <>
__device__ __forceinline__ uint32_t to_f16x2<__half>(uint32_t two, float) { return two; }
template <>
__device__ __forceinline__ uint32_t to_f16x2<__nv_bfloat16>(uint32_t two, float to) {
  return pack2<__half>(__uint_as_float(two << 16) * to, __uint_as_float(two & 0xffff0000u) * to);
}

// Of a value's scale: what its weights are multiplied by (its logarithm), and
// what turns such a weight back into the softmax's.  Scales below 2^-60, 0
// among them, count as 2^-60 here, and the values as 0.
constexpr float kLeastScale = 8.673617379884035e-19f;  // 2^-60
// The reference of a row lies this far below its largest weight (log2), so that
// fp16 weights keep 24 + this many binary places below it.
constexpr float kHead16 = 14.f;

}  // namespace
}  // namespace sv
