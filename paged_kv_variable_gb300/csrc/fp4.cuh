// Conversions of the 4-bit cache format: e2m1 codes, two a byte (the even dim
// in the low half), one e4m3 scale for every 16 dims of a row.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace pkv {

constexpr int kFp4Block = 16;  // dims that share a scale

// eight codes -> four f16x2, pairs in order (exact: every e2m1 value is an f16 value)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// eight fp32 -> eight codes (round to nearest even, saturate to +-6)
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* f) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// A query row in bf16 as f16 operands: times the power of two that brings its largest magnitude
// to [2^14, 2^15) (2^126 at most), so that any row keeps its bits but for dims that are 2^-31 of
// that or less; its logits take the inverse.
struct RowScale {
  uint32_t up;  // biased exponent
  // most: the largest magnitudes of a row's even and odd dims, as bf16 bits (a row of zeros, or
  // with an infinity or NaN: as it is)
  __device__ __forceinline__ explicit RowScale(uint32_t most) {
    const uint32_t m = max(most & 0xFFFFu, most >> 16), e = m >> 7;
    up = m == 0 || e == 255 ? 127u : min(268u - e, 253u);
  }
  __device__ __forceinline__ float down() const { return __uint_as_float((254u - up) << 23); }
  __device__ __forceinline__ uint32_t times(uint32_t v) const {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(up << 23 | up << 7));
    return r;
  }
};
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_most(uint32_t v, uint32_t most) { return max_u16x2(v & 0x7FFF7FFFu, most); }
// whether each of n pairs of bf16 is a pair of f16 numbers: 0, or from 2^-17 below 2^16
__device__ __forceinline__ bool f16_numbers(const uint32_t* v, int n) {
  uint32_t most = 0, least = 0xFFFFFFFFu;  // (0, less 1, is the largest)
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const uint32_t x = v[i] & 0x7FFF7FFFu;
    uint32_t less;
    asm("add.u16x2 %0, %1, %2;" : "=r"(less) : "r"(x), "r"(0xFFFFFFFFu));
    asm("min.u16x2 %0, %1, %2;" : "=r"(least) : "r"(least), "r"(less));
    most = max_u16x2(most, x);
  }
  return max(most & 0xFFFFu, most >> 16) < 0x4780u && min(least & 0xFFFFu, least >> 16) >= 0x36FFu;
}
// of the four lanes that have a row's dims
__device__ __forceinline__ uint32_t most_of_row(uint32_t most) {
  most = max_u16x2(most, __shfl_xor_sync(0xffffffffu, most, 1));
  return max_u16x2(most, __shfl_xor_sync(0xffffffffu, most, 2));
}

// Quotient of a number below 2^31 by d: (n * mul) >> shift with mul =
// ceil(2^(31 + l) / d), l = ceil(log2 d), shift = 31 + l (the excess of mul, below
// d / 2^l <= 1 units, adds less than 1 / d to the quotient).
struct FastDiv {
  uint32_t mul;
  uint32_t shift;
  int32_t d;
};

inline FastDiv fast_div(int d) {
  FastDiv f{};
  f.d = d;
  uint32_t l = 0;
  while ((1u << l) < (uint32_t)d) ++l;
  f.shift = 31 + l;
  f.mul = (uint32_t)(((1ull << f.shift) + (uint32_t)d - 1) / (uint32_t)d);
  return f;
}

__device__ __forceinline__ int quot(int n, const FastDiv& f) {
  return (int)(((uint64_t)(uint32_t)n * f.mul) >> f.shift);
}

}  // namespace pkv
