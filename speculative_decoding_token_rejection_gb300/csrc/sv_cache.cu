// sv_cache.cu -- tokens quantised into the paged 8-bit KV cache, and read back.
//
// scale = max(max_d |x_d| / Q, 2^-64), byte = rn(x / scale), value = byte *
// scale.  Both divisions are IEEE: the bytes are those of the definition, not
// of a reciprocal's.  Bound by HBM: a row's elements in, head_dim + 4 bytes
// out (and the reverse for reading).  One warp per (token, head) row, so the
// row's maximum is one warp reduction and every load of the row is one
// request; K and V rows of a token are neighbouring warps.
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

// EPL elements of a row per lane, at element lane * EPL.
template <int EPL, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const void *base, int64_t at, int lane, float x[EPL]) {
  if (BF16) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at + lane * EPL;
    if (VEC) {
      uint32_t w[EPL / 2];
      if (EPL == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[EPL / 2 - 1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
      }
#pragma unroll
      for (int c = 0; c < EPL; ++c) x[c] = bf16_bits_to_float((w[c / 2] >> (16 * (c & 1))) & 0xFFFFu);
    } else {
#pragma unroll
      for (int c = 0; c < EPL; ++c) x[c] = bf16_bits_to_float(p[c]);
    }
  } else {
    const float *p = static_cast<const float *>(base) + at + lane * EPL;
    if (VEC && EPL == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(p);
      x[0] = v.x;
      x[1] = v.y;
      x[EPL - 2] = v.z;
      x[EPL - 1] = v.w;
    } else if (VEC) {
      const float2 v = *reinterpret_cast<const float2 *>(p);
      x[0] = v.x;
      x[1] = v.y;
    } else {
#pragma unroll
      for (int c = 0; c < EPL; ++c) x[c] = p[c];
    }
  }
}

template <int EPL, bool BF16, bool VEC>
__device__ __forceinline__ void store_row(void *base, int64_t at, int lane, const float x[EPL]) {
  if (BF16) {
    uint16_t *p = static_cast<uint16_t *>(base) + at + lane * EPL;
    if (VEC && EPL == 4) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[EPL - 2], x[EPL - 1]));
    } else if (VEC) {
      *reinterpret_cast<uint32_t *>(p) = pack_bf16(x[0], x[1]);
    } else {
#pragma unroll
      for (int c = 0; c < EPL; ++c) p[c] = static_cast<uint16_t>(pack_bf16(x[c], 0.0f));
    }
  } else {
    float *p = static_cast<float *>(base) + at + lane * EPL;
    if (VEC && EPL == 4) {
      *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[EPL - 2], x[EPL - 1]);
    } else if (VEC) {
      *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    } else {
#pragma unroll
      for (int c = 0; c < EPL; ++c) p[c] = x[c];
    }
  }
}

// The row of this warp: token t, head h, side 0 (K) or 1 (V); false past the end.
__device__ __forceinline__ bool row_of_warp(const KvParams &P, int64_t &t, int &h, int &side) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const uint32_t per = 2u * P.c.num_kv_heads;
  if (r >= P.T * per) return false;
  t = static_cast<uint32_t>(r) / per;  // (the row count fits 31 bits: checked on the host)
  const int x = static_cast<int>(static_cast<uint32_t>(r) % per);
  side = x & 1;
  h = x >> 1;
  return true;
}

// Slot to offsets of the row's bytes and scale; false for a padding or bad slot.
__device__ __forceinline__ bool place_of(const KvParams &P, int64_t slot, int h, int lane, int64_t &at, int64_t &sat) {
  if (slot < 0 || slot >= P.c.num_blocks * P.c.block_size) {
    if (slot != SV_PADDING_SLOT_ID && lane == 0 && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_SLOT));
    return false;
  }
  const uint32_t b = static_cast<uint32_t>(slot) / static_cast<uint32_t>(P.c.block_size);
  const uint32_t o = static_cast<uint32_t>(slot) % static_cast<uint32_t>(P.c.block_size);
  at = b * P.c.block_stride + h * P.c.head_stride + o * P.c.token_stride;
  sat = b * P.c.scale_block_stride + h * P.c.scale_head_stride + o * P.c.scale_token_stride;
  return true;
}

template <int EPL, bool BF16, bool VEC, int FMT>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvParams P) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  int64_t t, at, sat;
  int h, side;
  if (!row_of_warp(P, t, h, side)) return;
  if (!place_of(P, P.slots[t], h, lane, at, sat)) return;
  float x[EPL];
  load_row<EPL, BF16, VEC>(side ? P.value : P.key,
                           side ? t * P.value_token + h * P.value_head : t * P.key_token + h * P.key_head, lane, x);
  // |x| as bits orders like a number, with infinities and NaN above every finite one
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < EPL; ++c) top = max(top, __float_as_uint(x[c]) & 0x7FFFFFFFu);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  const bool bad = top >= 0x7F800000u;
  const float scale =
      bad ? __uint_as_float(0x7FC00000u)
          : fmaxf(__fdiv_rn(__uint_as_float(top), FMT == SV_CACHE_INT8 ? 127.0f : 448.0f), 0x1p-64f);
  uint32_t w = 0;
  if (!bad) {
#pragma unroll
    for (int c = 0; c < EPL; ++c) x[c] = __fdiv_rn(x[c], scale);
    if (FMT == SV_CACHE_INT8) {
#pragma unroll
      for (int c = 0; c < EPL; ++c)
        w |= (static_cast<uint32_t>(min(127, max(-127, __float2int_rn(x[c])))) & 0xFFu) << (8 * c);
    } else {
#pragma unroll
      for (int c = 0; c < EPL; c += 2) w |= static_cast<uint32_t>(pack_e4m3(x[c], x[c + 1])) << (8 * c);
    }
  }
  uint8_t *dst = static_cast<uint8_t *>(side ? P.c.v : P.c.k) + at + lane * EPL;
  if (EPL == 4)
    *reinterpret_cast<uint32_t *>(dst) = w;
  else
    *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(w);
  if (lane == 0) {
    (side ? P.c.v_scale : P.c.k_scale)[sat] = scale;
    if (bad && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_VALUES));
  }
}

template <int EPL, bool BF16, bool VEC, int FMT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvParams P) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  int64_t t, at, sat;
  int h, side;
  if (!row_of_warp(P, t, h, side)) return;
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (place_of(P, P.slots[t], h, lane, at, sat)) {
    const uint8_t *src = static_cast<const uint8_t *>(side ? P.c.v : P.c.k) + at + lane * EPL;
    const float scale = (side ? P.c.v_scale : P.c.k_scale)[sat];
    const uint32_t w = EPL == 4 ? *reinterpret_cast<const uint32_t *>(src) : *reinterpret_cast<const uint16_t *>(src);
    cache_word_to_floats<FMT>(w, x);
#pragma unroll
    for (int c = 0; c < EPL; ++c) x[c] *= scale;
  }
  store_row<EPL, BF16, VEC>(side ? P.value : P.key,
                            side ? t * P.value_token + h * P.value_head : t * P.key_token + h * P.key_head, lane, x);
}

template <bool WRITE, int EPL, bool BF16, bool VEC, int FMT>
cudaError_t launch(const KvParams &p, cudaStream_t stream) {
  const int64_t rows = p.T * 2 * p.c.num_kv_heads;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  return cudaLaunchKernelEx(&cfg, WRITE ? kv_write_kernel<EPL, BF16, VEC, FMT> : kv_read_kernel<EPL, BF16, VEC, FMT>, p);
}

template <bool WRITE, int EPL>
cudaError_t pick(const KvParams &p, bool bf16, bool vec, cudaStream_t s) {
  const bool i8 = p.c.format == SV_CACHE_INT8;
  if (bf16)
    return vec ? (i8 ? launch<WRITE, EPL, true, true, SV_CACHE_INT8>(p, s) : launch<WRITE, EPL, true, true, SV_CACHE_E4M3>(p, s))
               : (i8 ? launch<WRITE, EPL, true, false, SV_CACHE_INT8>(p, s) : launch<WRITE, EPL, true, false, SV_CACHE_E4M3>(p, s));
  return vec ? (i8 ? launch<WRITE, EPL, false, true, SV_CACHE_INT8>(p, s) : launch<WRITE, EPL, false, true, SV_CACHE_E4M3>(p, s))
             : (i8 ? launch<WRITE, EPL, false, false, SV_CACHE_INT8>(p, s) : launch<WRITE, EPL, false, false, SV_CACHE_E4M3>(p, s));
}

}  // namespace

cudaError_t launch_kv_write(const KvParams &p, bool bf16, bool vec, cudaStream_t s) {
  return p.c.head_dim == 128 ? pick<true, 4>(p, bf16, vec, s) : pick<true, 2>(p, bf16, vec, s);
}
cudaError_t launch_kv_read(const KvParams &p, bool bf16, bool vec, cudaStream_t s) {
  return p.c.head_dim == 128 ? pick<false, 4>(p, bf16, vec, s) : pick<false, 2>(p, bf16, vec, s);
}

}  // namespace sv
