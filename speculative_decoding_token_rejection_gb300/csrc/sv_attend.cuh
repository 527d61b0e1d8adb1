// sv_attend.cuh -- what the kernels of the verify tokens' attention share: the
// division of the work, the partial results in the workspace, and how value
// scales enter a softmax.
//
// Scores are kept in base 2 with the value's scale inside the exponent:
//   t_k = (q . b_k) * (scale * log2 e * key_scale_k) + log2(value_scale_k),
// with b_k the key's byte numbers.  With M the largest t of a row so far,
//   w_k = 2^(t_k - M),   O = sum w_k c_k  (c_k: the value's byte numbers),
//   l = sum w_k / value_scale_k  ( = 2^-M sum 2^(s_k) ),
// out = O / l and lse = (M + log2 l) ln 2.  So the weights that meet the byte
// numbers in a 16-bit product are at most 1 whatever the sizes of the value
// rows, and a scale costs one addition and one multiplication an element.
// (Zero, negative and other unusual scales: value_scale_terms.)  A key whose
// scale is more than 2^100 below a row's largest may drop out of l.
// Weights are rounded to f16 for that product (11 bits, steps of 2^-24 of the
// largest): the byte numbers have 8 bits and are exact, sums are fp32, and l
// takes the unrounded weights.
#pragma once

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How a call is cut up.  Slot s of a row holds the partial result of prefix
// chunk s, or of private chunk s - prefix_splits.
struct AttendPlan {
  FastDiv page, group;
  int32_t rows;           // (T + N) * group rows for every kv head
  int32_t prefix_splits, prefix_chunk;
  int32_t prefix_tiles, prefix_items;  // prefix row tiles and CTAs of the warp-streaming kernel (0 items: not its work)
  int32_t tensor_tiles;                // prefix row tiles of the tensor-memory kernel (0: not its work)
  // its (kv head, row tile)s, one each `period` units, of which the first image_tiles are key tiles; a CTA's share
  int32_t units, units_cta, period;
  int32_t own_splits, own_chunk, own_tiles;
  int32_t slots;          // partial results of a row
  uint32_t unit_bytes, block_units, token_units;  // a cache row's place in units that divide both strides
  bool ovec;              // output rows allow 8-byte stores
  bool qvec;              // q rows allow 16-byte loads
  int32_t image_tiles;    // tiles of kPrefixKeyTile keys of the prefix
  uint8_t *image;         // the prefix as f16 tiles: [num_kv_heads][image_tiles][K, V]
  float *part_o;          // [rows * num_kv_heads][slots][D], row = token * Hq + query head
  float2 *part_ml;        // [rows * num_kv_heads][slots]: M, l
};

// The prefix on the tensor cores' memory (sv_attend_prefix.cu): tiles of
// kPrefixRowTile rows and kPrefixKeyTile keys.
cudaError_t enable_prefix_kernels();
cudaError_t launch_prefix(const AttendParams &p, const AttendPlan &L, cudaStream_t stream);
constexpr int kPrefixRowTile = 256, kPrefixKeyTile = 128;

// Partial results of the prefix that a row has: of kv head h, row `local` of
// the (T + N) * group.
__device__ __forceinline__ int prefix_slots(const AttendPlan &L, int h, int local) {
  if (L.tensor_tiles == 0) return L.prefix_splits;
  const int first = (h * L.tensor_tiles + local / kPrefixRowTile) * L.period;
  return (first + L.image_tiles - 1) / L.units_cta - first / L.units_cta + 1;
}

// Draft range and length of request i; false (and nothing to write) for a bad
// range.  A bad length counts as 0.
__device__ __forceinline__ bool attend_request(const AttendParams &P, int i, int64_t &first, int &g, int &len,
                                               uint32_t &bits) {
  int64_t s;
  if (!request_range(P.cu, i, P.G, P.T, s, g)) {
    bits |= SV_DATA_BAD_CU;
    return false;
  }
  first = s + i;
  len = P.seq_lens[i];
  if (len < 0 || len > P.max_seq) {
    bits |= SV_DATA_BAD_PARAM;
    len = 0;
  }
  return true;
}

// The request whose range of verify tokens holds `row`, or -1.  The ranges that
// are in order need not be found by a search over all of them, which one bad
// entry misleads: then they are looked through.
__device__ __forceinline__ int request_of_row(const AttendParams &P, int row) {
  if (!P.cu) return row / (P.G + 1);
  const auto holds = [&](int64_t s, int64_t e, int i) {
    return s >= 0 && e >= s && e <= P.T && e - s <= P.G && s + i <= row && row <= e + i;
  };
  int lo = 0, hi = P.N - 1;  // the first request whose last row cu[i] + i is at or behind `row`
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(P.cu[mid]) + mid >= row)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (holds(lo ? P.cu[lo - 1] : 0, P.cu[lo], lo)) return lo;
  int at = -1;
  int32_t s = 0;
#pragma unroll 4
  for (int i = 0; i < P.N; ++i) {
    const int32_t e = P.cu[i];
    if (holds(s, e, i)) at = i;
    s = e;
  }
  return at;
}

// Prefix keys that verify token `row` sees (0 .. P.prefix), or -1 for a row
// that belongs to no request.
__device__ __forceinline__ int prefix_limit(const AttendParams &P, int row) {
  const int i = request_of_row(P, row);
  int64_t first;
  int g, len;
  uint32_t bits = 0;
  if (i < 0 || !attend_request(P, i, first, g, len, bits)) return -1;
  return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(P.prefix), len - g + (row - first))));
}

// A value scale may be any float, and its key counts in l whatever it is.  Its
// size enters a softmax as kLeastScale at least, the smallest that kv_write
// gives; one below that counts as zero, as does one that is no number, and the
// rows that see a key of the latter get NaN outputs.
constexpr float kLeastScale = 0x1p-64f, kLeastLog2 = -64.0f;
__device__ __forceinline__ bool usual_scale(float vs) { return vs >= kLeastScale && vs < INFINITY; }
// log2 of its size, and the size's reciprocal for the sum l.
__device__ __forceinline__ void value_scale_terms(float vs, float &lv, float &inv) {
  const float a = fabsf(vs);
  const bool ok = usual_scale(a);
  lv = ok ? log2f(a) : kLeastLog2;
  inv = ok ? __frcp_rn(a) : 1.0f / kLeastScale;
}

// The exponent of the power of two that a row of q, whose largest finite |q| has
// these bits, is multiplied by on its way to f16: a multiple of 16 that brings
// the largest into [2^-1, 2^15).  bf16 numbers are exact there down to 2^-14
// (2^-13 of the row's largest at least), and off by 2^-25 at most below.  Every
// row has its own, so that nothing of a row (an idle request's, say) reaches
// another; it is 0 for rows from 0.5 to 32767, and the code that puts another
// one right runs only for tiles that hold such a row.
__device__ __forceinline__ int query_shift(uint32_t top_bits) {
  if (top_bits == 0) return 0;
  const int e = static_cast<int>(top_bits >> 23) - 127;
  return max(-120, min(112, -16 * ((e + 1 + 256) / 16 - 16)));  // (both ends and their negatives are in pow2's range)
}
__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace sv
