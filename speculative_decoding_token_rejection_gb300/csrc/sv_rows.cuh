// sv_rows.cuh -- sixteen elements of a key or value row, fp32 or bf16, to and
// from registers.  VEC: the row starts on a 32-byte boundary.
#pragma once

#include <cstdint>

#include "sv_ops.cuh"

namespace sv {

constexpr int kPer = 16;  // elements of a thread

template <bool BF16, bool VEC>
__device__ __forceinline__ void load_elements(const void *base, int64_t at, float x[kPer]) {
  if (BF16) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    if (VEC) {
      uint32_t w[8];
      ld_stream_32(p, w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[2 * c] = __uint_as_float(w[c] << 16);
        x[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) x[c] = bf16_bits_to_float(p[c]);
    }
  } else {
    const float *p = static_cast<const float *>(base) + at;
    if (VEC) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint32_t w[8];
        ld_stream_32(p + 8 * v, w);
#pragma unroll
        for (int c = 0; c < 8; ++c) x[8 * v + c] = __uint_as_float(w[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) x[c] = p[c];
    }
  }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store_elements(void *base, int64_t at, const float x[kPer]) {
  if (BF16) {
    uint16_t *p = static_cast<uint16_t *>(base) + at;
    if (VEC) {
      uint32_t w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
      st_32(p, w);
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) p[c] = static_cast<uint16_t>(pack_bf16(x[c], 0.0f));
    }
  } else {
    float *p = static_cast<float *>(base) + at;
    if (VEC) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint32_t w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = __float_as_uint(x[8 * v + c]);
        st_32(p + 8 * v, w);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) p[c] = x[c];
    }
  }
}

}  // namespace sv
