// sv_cache4.cu -- tokens quantised into the paged 4-bit KV cache, and read back.
//
// A row of head_dim elements has a float scale S and an e4m3 scale g for every
// 16 elements:
//   S = max(max_d |x_d| / (448 Q), 2^-64),  g_j = e4m3(max_j |x_d| / (Q S)),
//   nibble = x_d / (g_j S) rounded to E2M1 (Q = 6) or to a whole number (Q = 7).
// All quotients are IEEE ones, so the nibbles are those of the definition.  A
// nibble times g is exact in f16 (2 or 3 bits times 4), and is rounded once, by
// S, on its way out.  Bound by HBM: a row's elements in, head_dim * 9/16 + 4
// bytes out (and the reverse for reading).
//
// A thread takes one group: its maximum needs no neighbour, the row's takes
// three shuffles (two for head_dim 64), and its 16 nibbles are one 8-byte access.
//
// Reading 131072 tokens x 8 heads x 128 as bf16: 142 us, 537 MB written at 3.8
// TB/s beside 151 MB read; filling as much memory alone takes 135 (4.0 TB/s).
// Writing them 194 us as E2M1, 207 as whole numbers (3.5 TB/s), in either order of
// the cache's memory.  Writing and reading 4096 x 8 x 128: 9.8 us, two launches that
// take 8.0 and 6.4 by themselves with cold caches.
#include <cstdint>

#include "sv_cache4.cuh"
#include "sv_internal.h"
#include "sv_rows.cuh"

namespace sv {
namespace {

static_assert(kPer == kGroup4, "a thread takes one group");

// The thread's group: token t, side (0: K), head h, group col of the row.
struct Piece {
  int t, side, h, col;
};
template <int D>
__device__ __forceinline__ bool piece_of_thread(const Kv4Params &P, const FastDiv &heads, Piece &x) {
  const uint32_t id = blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x;  // (fits: checked on the host)
  x.col = id % (D / kGroup4);
  const int row = static_cast<int>(id / (D / kGroup4)), ts = div_by(row, heads);
  x.h = row - ts * P.c.num_kv_heads;
  x.side = ts & 1;
  x.t = ts >> 1;
  return x.t < P.T;
}

// Slot to offsets of the group's nibbles, its scale and the row's; false for a padding or bad slot.
struct Place {
  int64_t data, group, scale;
};
__device__ __forceinline__ bool place_of(const Kv4Params &P, const FastDiv &page, const Piece &x, Place &at) {
  const int64_t slot = P.slots[x.t];
  if (slot < 0 || slot >= P.c.num_blocks * P.c.block_size) {
    if (slot != SV_PADDING_SLOT_ID && x.col == 0 && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_SLOT));
    return false;
  }
  const int b = div_by(static_cast<int>(slot), page), o = static_cast<int>(slot) - b * P.c.block_size;
  at.data = b * P.c.block_stride + x.h * P.c.head_stride + o * P.c.token_stride + x.col * (kGroup4 / 2);
  at.group = b * P.c.group_block_stride + x.h * P.c.group_head_stride + o * P.c.group_token_stride + x.col;
  at.scale = b * P.c.scale_block_stride + x.h * P.c.scale_head_stride + o * P.c.scale_token_stride;
  return true;
}

template <int D, bool BF16, bool VEC, int FMT>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4Params P, const FastDiv heads, const FastDiv page) {
  pdl_enter();
  constexpr float kQ = FMT == SV_CACHE_INT4 ? 7.0f : 6.0f;
  Piece p;
  const bool in = piece_of_thread<D>(P, heads, p);
  Place at{};
  const bool live = in && place_of(P, page, p, at);
  float x[kPer];
  uint32_t most = 0;
  if (live) {
    load_elements<BF16, VEC>(p.side ? P.value : P.key,
                             (p.side ? p.t * P.value_token + p.h * P.value_head : p.t * P.key_token + p.h * P.key_head) +
                                 p.col * kPer,
                             x);
    // |x| as bits orders like a number, with infinities and NaN above every finite one
#pragma unroll
    for (int c = 0; c < kPer; ++c) most = max(most, __float_as_uint(x[c]) & 0x7FFFFFFFu);
  }
  uint32_t top = most;
#pragma unroll
  for (int b = D / kGroup4 / 2; b; b >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, b));
  if (!live) return;
  const bool bad = top >= 0x7F800000u;
  const float scale = bad ? __uint_as_float(0x7FC00000u)
                          : fmaxf(__fdiv_rn(__uint_as_float(top), 448.0f * kQ), 0x1p-64f);
  uint32_t g = 0;
  uint2 w = make_uint2(0, 0);
  if (!bad) {
    g = pack_e4m3(__fdiv_rn(__uint_as_float(most), kQ * scale), 0.0f) & 0xFFu;
    if (g) {
      float gf[4];
      e4m3_word_to_floats(g, gf);
      const float unit = gf[0] * scale;
      // x / unit: with r the rounded reciprocal, q = x r and one correction by the exact remainder give the rounded
      // quotient (Markstein, 1990).  (unit is 2^-73 at least and below 2^126: neither it nor r leaves the normal range.)
      const float r = __frcp_rn(unit);
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const float q = x[c] * r;
        x[c] = fmaf(fmaf(-q, unit, x[c]), r, q);
      }
      w.x = pack_nibbles<FMT>(x);
      w.y = pack_nibbles<FMT>(x + 8);
    }
  }
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.side ? P.c.v : P.c.k) + at.data) = w;
  static_cast<uint8_t *>(p.side ? P.c.v_group : P.c.k_group)[at.group] = static_cast<uint8_t>(g);
  if (p.col == 0) {
    (p.side ? P.c.v_scale : P.c.k_scale)[at.scale] = scale;
    if (bad && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_VALUES));
  }
}

template <int D, bool BF16, bool VEC, int FMT>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Params P, const FastDiv heads, const FastDiv page) {
  pdl_enter();
  Piece p;
  if (!piece_of_thread<D>(P, heads, p)) return;
  Place at;
  float x[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) x[c] = 0.0f;
  if (place_of(P, page, p, at)) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.side ? P.c.v : P.c.k) + at.data));
    const uint32_t g = static_cast<const uint8_t *>(p.side ? P.c.v_group : P.c.k_group)[at.group];
    const float scale = (p.side ? P.c.v_scale : P.c.k_scale)[at.scale];
    uint32_t h[8];
    group_to_f16<FMT>(w, group_factors<FMT>(g), h);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      x[2 * c] = f16_bits_to_float(static_cast<uint16_t>(h[c])) * unit4<FMT>() * scale;
      x[2 * c + 1] = f16_bits_to_float(static_cast<uint16_t>(h[c] >> 16)) * unit4<FMT>() * scale;
    }
  }
  store_elements<BF16, VEC>(p.side ? P.value : P.key,
                            (p.side ? p.t * P.value_token + p.h * P.value_head : p.t * P.key_token + p.h * P.key_head) +
                                p.col * kPer,
                            x);
}

template <bool WRITE, int D, bool BF16, bool VEC, int FMT>
cudaError_t launch(const Kv4Params &p, cudaStream_t stream) {
  const int64_t threads = p.T * 2 * p.c.num_kv_heads * (D / kGroup4);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  return cudaLaunchKernelEx(&cfg, WRITE ? kv4_write_kernel<D, BF16, VEC, FMT> : kv4_read_kernel<D, BF16, VEC, FMT>, p,
                            fast_div(p.c.num_kv_heads), fast_div(p.c.block_size));
}

template <bool WRITE, int D>
cudaError_t pick(const Kv4Params &p, bool bf16, bool vec, cudaStream_t s) {
  const bool i4 = p.c.format == SV_CACHE_INT4;
  if (bf16)
    return vec ? (i4 ? launch<WRITE, D, true, true, SV_CACHE_INT4>(p, s) : launch<WRITE, D, true, true, SV_CACHE_E2M1>(p, s))
               : (i4 ? launch<WRITE, D, true, false, SV_CACHE_INT4>(p, s) : launch<WRITE, D, true, false, SV_CACHE_E2M1>(p, s));
  return vec ? (i4 ? launch<WRITE, D, false, true, SV_CACHE_INT4>(p, s) : launch<WRITE, D, false, true, SV_CACHE_E2M1>(p, s))
             : (i4 ? launch<WRITE, D, false, false, SV_CACHE_INT4>(p, s) : launch<WRITE, D, false, false, SV_CACHE_E2M1>(p, s));
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Params &p, bool bf16, bool vec, cudaStream_t s) {
  return p.c.head_dim == 128 ? pick<true, 128>(p, bf16, vec, s) : pick<true, 64>(p, bf16, vec, s);
}
cudaError_t launch_kv4_read(const Kv4Params &p, bool bf16, bool vec, cudaStream_t s) {
  return p.c.head_dim == 128 ? pick<false, 128>(p, bf16, vec, s) : pick<false, 64>(p, bf16, vec, s);
}

}  // namespace sv
