// sv_ops.cuh -- device helpers of the operators around the verifier: the
// ragged request layout, 8-bit cache formats and bf16 packing.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "spec_verify.h"
#include "sv_device.cuh"

namespace sv {

// Draft range of request i: rows s + i .. s + i + g of the verify-token
// layout.  False if cu is not a valid range.
__device__ __forceinline__ bool request_range(const int32_t *cu, int i, int G, int64_t T, int64_t &s, int &g) {
  if (!cu) {
    s = static_cast<int64_t>(i) * G;
    g = G;
    return true;
  }
  s = i ? cu[i - 1] : 0;
  const int64_t e = cu[i];
  if (s < 0 || e < s || e > T || e - s > G) return false;
  g = static_cast<int>(e - s);
  return true;
}

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }
// Two floats rounded to nearest even bf16, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes (low byte first) of floats, round to nearest even, saturating.
__device__ __forceinline__ uint16_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes as two f16 (exact), the low byte in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
  return r;
}
__device__ __forceinline__ float f16_bits_to_float(uint16_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return f;
}
// The four numbers that the four bytes of w stand for (scale aside).
template <int FMT>
__device__ __forceinline__ void cache_word_to_floats(uint32_t w, float f[4]) {
  if (FMT == SV_CACHE_INT8) {
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] = static_cast<float>(static_cast<int8_t>(w >> (8 * c)));
  } else {
    const uint32_t a = e4m3x2_to_f16x2(static_cast<uint16_t>(w)), b = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
    f[0] = f16_bits_to_float(static_cast<uint16_t>(a));
    f[1] = f16_bits_to_float(static_cast<uint16_t>(a >> 16));
    f[2] = f16_bits_to_float(static_cast<uint16_t>(b));
    f[3] = f16_bits_to_float(static_cast<uint16_t>(b >> 16));
  }
}

}  // namespace sv
