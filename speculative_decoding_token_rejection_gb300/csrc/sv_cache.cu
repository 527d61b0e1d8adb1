// sv_cache.cu -- tokens quantised into the paged 8-bit KV cache, and read back.
//
// scale = max(max_d |x_d| / Q, 2^-64), byte = rn(x / scale), value = byte *
// scale.  Both divisions have IEEE results: the bytes are those of the
// definition, not of a reciprocal's.  Bound by HBM: a row's elements in,
// head_dim + 4 bytes out (and the reverse for reading).
//
// A thread takes 16 elements of a row, 16 bytes of the cache: eight lanes (four
// for head_dim 64) a row, whose maximum takes three (two) shuffles, and
// neighbouring heads of a token side by side in a warp.  With one warp a row
// the places of the rows, not their elements, were most of the instructions:
// 131072 tokens x 8 heads x 128 read back to bf16 took 408 us (issue slots
// 62 % busy, 29 % of the copy rate), this way 141 (85 %).  Keys and values move
// as 32 bytes an access: with 16 every sector went through the memory pipe
// twice, and 50001 x 4 x 64 fp32 written and read back took 52 us for 46.5.
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

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

// The thread's 16 elements: token t, side (0: K), head h, column col of 16.
struct Piece {
  int t, side, h, col;
};
template <int D>
__device__ __forceinline__ bool piece_of_thread(const KvParams &P, const FastDiv &heads, Piece &x) {
  const uint32_t id = blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x;  // (fits: checked on the host)
  x.col = id % (D / kPer);
  const int row = static_cast<int>(id / (D / kPer)), ts = div_by(row, heads);
  x.h = row - ts * P.c.num_kv_heads;
  x.side = ts & 1;
  x.t = ts >> 1;
  return x.t < P.T;
}

// Slot to offsets of the row's bytes and scale; false for a padding or bad slot.
__device__ __forceinline__ bool place_of(const KvParams &P, const FastDiv &page, const Piece &x, int64_t &at,
                                         int64_t &sat) {
  const int64_t slot = P.slots[x.t];
  if (slot < 0 || slot >= P.c.num_blocks * P.c.block_size) {
    if (slot != SV_PADDING_SLOT_ID && x.col == 0 && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_SLOT));
    return false;
  }
  const int b = div_by(static_cast<int>(slot), page), o = static_cast<int>(slot) - b * P.c.block_size;
  at = b * P.c.block_stride + x.h * P.c.head_stride + o * P.c.token_stride + x.col * kPer;
  sat = b * P.c.scale_block_stride + x.h * P.c.scale_head_stride + o * P.c.scale_token_stride;
  return true;
}

template <int D, bool BF16, bool VEC, int FMT>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvParams P, const FastDiv heads, const FastDiv page) {
  pdl_enter();
  Piece p;
  const bool in = piece_of_thread<D>(P, heads, p);
  int64_t at = 0, sat = 0;
  const bool live = in && place_of(P, page, p, at, sat);
  float x[kPer];
  uint32_t top = 0;
  if (live) {
    load_elements<BF16, VEC>(p.side ? P.value : P.key,
                             (p.side ? p.t * P.value_token + p.h * P.value_head : p.t * P.key_token + p.h * P.key_head) +
                                 p.col * kPer,
                             x);
    // |x| as bits orders like a number, with infinities and NaN above every finite one
#pragma unroll
    for (int c = 0; c < kPer; ++c) top = max(top, __float_as_uint(x[c]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int b = D / kPer / 2; b; b >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, b));
  if (!live) return;
  const bool bad = top >= 0x7F800000u;
  const float scale =
      bad ? __uint_as_float(0x7FC00000u)
          : fmaxf(__fdiv_rn(__uint_as_float(top), FMT == SV_CACHE_INT8 ? 127.0f : 448.0f), 0x1p-64f);
  uint32_t w[4] = {0, 0, 0, 0};
  if (!bad) {
    // x / scale: with r the rounded reciprocal, q = x r and one correction by the exact remainder give the rounded
    // quotient (Markstein, 1990).  Quotients too small for that round to a zero byte either way.
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const float q = x[c] * r;
      x[c] = fmaf(fmaf(-q, scale, x[c]), r, q);
    }
    if (FMT == SV_CACHE_INT8) {
      // adding 1.5 * 2^23 rounds to the nearest even whole number, whose low byte is the sum's (|x / scale| <= 127
      // plus an ulp: no clamp is needed)
#pragma unroll
      for (int c = 0; c < kPer; c += 4) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(x[c + e] + 12582912.0f);
        w[c / 4] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kPer; c += 4)
        w[c / 4] = static_cast<uint32_t>(pack_e4m3(x[c], x[c + 1])) | static_cast<uint32_t>(pack_e4m3(x[c + 2], x[c + 3])) << 16;
    }
  }
  *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.side ? P.c.v : P.c.k) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  if (p.col == 0) {
    (p.side ? P.c.v_scale : P.c.k_scale)[sat] = scale;
    if (bad && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_VALUES));
  }
}

// Four bytes' numbers in fp32, exactly.  int8: byte x + 128 in the low mantissa
// bits of 2^23 is 8388736 + x.
template <int FMT>
__device__ __forceinline__ void numbers_of(uint32_t w, float f[4]) {
  if (FMT == SV_CACHE_INT8) {
    w ^= 0x80808080u;
    f[0] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540)) - 8388736.0f;
    f[1] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541)) - 8388736.0f;
    f[2] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7542)) - 8388736.0f;
    f[3] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7543)) - 8388736.0f;
  } else {
    e4m3_word_to_floats(w, f);
  }
}

template <int D, bool BF16, bool VEC, int FMT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvParams P, const FastDiv heads, const FastDiv page) {
  pdl_enter();
  Piece p;
  if (!piece_of_thread<D>(P, heads, p)) return;
  int64_t at, sat;
  float x[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) x[c] = 0.0f;
  if (place_of(P, page, p, at, sat)) {
    const uint4 r = ld_stream_u4(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.side ? P.c.v : P.c.k) + at));
    const float scale = (p.side ? P.c.v_scale : P.c.k_scale)[sat];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      numbers_of<FMT>(w[c], x + 4 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * c + e] *= scale;
    }
  }
  store_elements<BF16, VEC>(p.side ? P.value : P.key,
                            (p.side ? p.t * P.value_token + p.h * P.value_head : p.t * P.key_token + p.h * P.key_head) +
                                p.col * kPer,
                            x);
}

template <bool WRITE, int D, bool BF16, bool VEC, int FMT>
cudaError_t launch(const KvParams &p, cudaStream_t stream) {
  const int64_t threads = p.T * 2 * p.c.num_kv_heads * (D / kPer);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  return cudaLaunchKernelEx(&cfg, WRITE ? kv_write_kernel<D, BF16, VEC, FMT> : kv_read_kernel<D, BF16, VEC, FMT>, p,
                            fast_div(p.c.num_kv_heads), fast_div(p.c.block_size));
}

template <bool WRITE, int D>
cudaError_t pick(const KvParams &p, bool bf16, bool vec, cudaStream_t s) {
  const bool i8 = p.c.format == SV_CACHE_INT8;
  if (bf16)
    return vec ? (i8 ? launch<WRITE, D, true, true, SV_CACHE_INT8>(p, s) : launch<WRITE, D, true, true, SV_CACHE_E4M3>(p, s))
               : (i8 ? launch<WRITE, D, true, false, SV_CACHE_INT8>(p, s) : launch<WRITE, D, true, false, SV_CACHE_E4M3>(p, s));
  return vec ? (i8 ? launch<WRITE, D, false, true, SV_CACHE_INT8>(p, s) : launch<WRITE, D, false, true, SV_CACHE_E4M3>(p, s))
             : (i8 ? launch<WRITE, D, false, false, SV_CACHE_INT8>(p, s) : launch<WRITE, D, false, false, SV_CACHE_E4M3>(p, s));
}

}  // namespace

cudaError_t launch_kv_write(const KvParams &p, bool bf16, bool vec, cudaStream_t s) {
  return p.c.head_dim == 128 ? pick<true, 128>(p, bf16, vec, s) : pick<true, 64>(p, bf16, vec, s);
}
cudaError_t launch_kv_read(const KvParams &p, bool bf16, bool vec, cudaStream_t s) {
  return p.c.head_dim == 128 ? pick<false, 128>(p, bf16, vec, s) : pick<false, 64>(p, bf16, vec, s);
}

}  // namespace sv
