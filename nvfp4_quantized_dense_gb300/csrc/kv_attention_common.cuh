// What both forms of the attention over the NVFP4 cache use.
#pragma once
#include <cstdint>

namespace nvfp4 {

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {   // 2^-22 relative; 2^-inf = 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Pairs of floats in one instruction each (sm_100 and later).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// What a query row is multiplied by: the power of two with exponent field e,
// with the sign of the scores' scale, or that scale itself where it is a NaN:
// the scores that a row sees are NaN then, and the masked ones still -inf.
__device__ __forceinline__ float row_factor(uint32_t e, float qk) {
  return qk == qk ? copysignf(__uint_as_float(e << 23), qk) : qk;
}

// The E4M3 scales of four tokens in a row with those outside [from, to) zeroed
// (places counted from the first of the four): the bytes of a token that no
// query sees may be anything, NaN too, and 0 times NaN would reach every row.
__device__ __forceinline__ uint32_t scales_within(uint32_t four, int from, int to) {
  four = to >= 4 ? four : to <= 0 ? 0u : four & ((1u << (8 * to)) - 1u);
  return from <= 0 ? four : from >= 4 ? 0u : four & (~0u << (8 * from));
}

// The line [0, total) in `parts` equal pieces, the first total % parts of them
// one longer.
struct Line {
  uint32_t size, longer;
  __device__ __forceinline__ Line(int total, int parts)
      : size((uint32_t)total / (uint32_t)parts), longer((uint32_t)total - size * (uint32_t)parts) {}
  __device__ __forceinline__ int at(int p) const { return p * size + min((uint32_t)p, longer); }
  __device__ __forceinline__ int part_of(int x) const {
    const uint32_t k = longer * (size + 1);
    return (uint32_t)x < k ? (uint32_t)x / (size + 1) : longer + ((uint32_t)x - k) / size;
  }
};

}  // namespace nvfp4
