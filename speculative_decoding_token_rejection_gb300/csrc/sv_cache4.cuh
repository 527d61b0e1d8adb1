// sv_cache4.cuh -- the 4-bit cache's numbers: nibbles times their group's e4m3
// scale as f16 pairs, exactly.
//
// E2M1 times e4m3 has 2 + 4 significant bits and lies between 2^-10 and 2688: one
// conversion and one f16 product a pair.  For whole numbers, a nibble put into the
// low mantissa bits of 1024 is 1032 + x, and (1032 + x) g - 1032 g takes one fused
// operation, exact if 1032 g is a number of f16: it has 8 + 4 bits, but 129 * 15 <
// 2^11, and g is taken down by 2^4 so that it stays in range.  What a pair of f16
// stands for is unit4 times it; the row's scale takes that factor.
#pragma once

#include <cstdint>

#include "sv_ops.cuh"

namespace sv {

constexpr int kGroup4 = 16;  // elements that share a group scale

template <int FMT>
__host__ __device__ constexpr float unit4() {
  return FMT == SV_CACHE_INT4 ? 16.0f : 1.0f;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// (x & m) ^ c in one operation.
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t m, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "r"(m), "r"(c));
  return r;
}
// The four pairs of f16 of the four bytes of w (E2M1, two to a byte, the low half first).
__device__ __forceinline__ void e2m1_word_to_f16(uint32_t w, uint32_t r[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// What a group's scale (an e4m3 byte) gives the products, twice each: for E2M1 the
// scale; for whole numbers a = g / 16, b = -1032 a, c = a / 16 and d = -72 a.
struct GroupFactors {
  uint32_t a, b, c, d;
};
template <int FMT>
__device__ __forceinline__ GroupFactors group_factors(uint32_t g) {
  GroupFactors f;
  const uint32_t both = e4m3x2_to_f16x2(static_cast<uint16_t>(g | g << 8));
  f.a = FMT == SV_CACHE_INT4 ? hmul2(both, 0x2C002C00u) : both;   // (1/16)
  f.b = FMT == SV_CACHE_INT4 ? hmul2(f.a, 0xE408E408u) : 0u;      // (-1032)
  f.c = FMT == SV_CACHE_INT4 ? hmul2(f.a, 0x2C002C00u) : 0u;
  f.d = FMT == SV_CACHE_INT4 ? hmul2(f.a, 0xD480D480u) : 0u;      // (-72)
  return f;
}

// A group's sixteen elements as pairs (2i, 2i + 1).
template <int FMT>
__device__ __forceinline__ void group_to_f16(uint2 w, GroupFactors f, uint32_t r[8]) {
  if (FMT == SV_CACHE_INT4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = (i ? w.y : w.x) ^ 0x88888888u, low = u & 0x0F0F0F0Fu, high = u >> 4 & 0x0F0F0F0Fu;
      // bytes (low j, 0x64, high j, 0x64)
      r[4 * i] = __byte_perm(low, high, 0x0400) & 0x00FF00FFu | 0x64006400u;
      r[4 * i + 1] = __byte_perm(low, high, 0x0501) & 0x00FF00FFu | 0x64006400u;
      r[4 * i + 2] = __byte_perm(low, high, 0x0602) & 0x00FF00FFu | 0x64006400u;
      r[4 * i + 3] = __byte_perm(low, high, 0x0703) & 0x00FF00FFu | 0x64006400u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = hfma2(r[i], f.a, f.b);
  } else {
    e2m1_word_to_f16(w.x, r);
    e2m1_word_to_f16(w.y, r + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = hmul2(r[i], f.a);
  }
}

// The same with the pairs that take the fewest instructions.  Whole numbers: (0,
// 4), (1, 5), (2, 6), (3, 7) of every eight; a nibble in the second place of a
// byte is 16 x + 1152 in the mantissa of 1024, which c and d undo.
template <int FMT>
__host__ __device__ constexpr bool mixed() {
  return FMT == SV_CACHE_INT4;
}
// The element at place `at` of that order.
__device__ __forceinline__ int mixed_place(int at) { return (at & ~7) | (at >> 1 & 3) | (at & 1) << 2; }
template <int FMT>
__device__ __forceinline__ void group_to_f16_mixed(uint2 w, GroupFactors f, uint32_t r[8]) {
  if (FMT == SV_CACHE_INT4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = i ? w.y : w.x, v = u >> 8;
      r[4 * i] = hfma2(and_xor(u, 0x000F000Fu, 0x64086408u), f.a, f.b);
      r[4 * i + 1] = hfma2(and_xor(u, 0x00F000F0u, 0x64806480u), f.c, f.d);
      r[4 * i + 2] = hfma2(and_xor(v, 0x000F000Fu, 0x64086408u), f.a, f.b);
      r[4 * i + 3] = hfma2(and_xor(v, 0x00F000F0u, 0x64806480u), f.c, f.d);
    }
  } else {
    group_to_f16<FMT>(w, f, r);
  }
}

// Two groups, 32 elements of a row, in that order; the low half of g holds their scales.
template <int FMT>
__device__ __forceinline__ void groups_to_f16_mixed(const uint32_t w[4], uint32_t g, uint32_t r[16]) {
  const uint32_t two = e4m3x2_to_f16x2(static_cast<uint16_t>(g));
  const uint32_t a = FMT == SV_CACHE_INT4 ? hmul2(two, 0x2C002C00u) : two;                         // (1/16)
  const uint32_t b = hmul2(a, 0xE408E408u), c = hmul2(a, 0x2C002C00u), d = hmul2(a, 0xD480D480u);  // (-1032, 1/16, -72)
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t one = q ? 0x3232u : 0x1010u;
    GroupFactors f;
    f.a = __byte_perm(a, 0, one);
    f.b = FMT == SV_CACHE_INT4 ? __byte_perm(b, 0, one) : 0u;
    f.c = FMT == SV_CACHE_INT4 ? __byte_perm(c, 0, one) : 0u;
    f.d = FMT == SV_CACHE_INT4 ? __byte_perm(d, 0, one) : 0u;
    group_to_f16_mixed<FMT>(make_uint2(w[2 * q], w[2 * q + 1]), f, r + 8 * q);
  }
}

// Eight quotients (at most a little more than Q in size) to nibbles, ties to the even code.
template <int FMT>
__device__ __forceinline__ uint32_t pack_nibbles(const float x[8]) {
  uint32_t w = 0;
  if (FMT == SV_CACHE_INT4) {
    // adding 1.5 * 2^23 rounds to the nearest even whole number, whose low bits are the sum's
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w |= (__float_as_uint(fminf(fmaxf(x[e], -7.0f), 7.0f) + 12582912.0f) & 15u) << (4 * e);
  } else {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  }
  return w;
}

}  // namespace sv
