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
  float *part_rest;       // [rows * num_kv_heads][slots]: what a maximum kept as two numbers is beside M (null where none is)
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

// One partial result of a row: M (and what is beside it), l and the lane's dimensions of O.
template <int D>
struct Part {
  float m, rest, l, o[D / 32];
};
constexpr int kJoinAhead = 4;  // partial results of a row in flight
template <int D>
__device__ __forceinline__ Part<D> load_part(const AttendPlan &L, int64_t row, int s, int lane) {
  Part<D> p;
  const float2 ml = __ldcg(L.part_ml + row * L.slots + s);
  p.m = ml.x;
  p.l = ml.y;
  p.rest = L.part_rest ? __ldcg(L.part_rest + row * L.slots + s) : 0.0f;
  const float *src = L.part_o + (row * L.slots + s) * D;
  if (D == 128) {
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src) + lane);
    p.o[0] = v.x;
    p.o[1] = v.y;
    p.o[D / 32 - 2] = v.z;
    p.o[D / 32 - 1] = v.w;
  } else {
    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src) + lane);
    p.o[0] = v.x;
    p.o[1] = v.y;
  }
  return p;
}
template <int D>
__device__ __forceinline__ void store_part(const AttendPlan &L, int64_t row, int s, int lane, const Part<D> &p) {
  float *dst = L.part_o + (row * L.slots + s) * D;
  if (D == 128)
    reinterpret_cast<float4 *>(dst)[lane] = make_float4(p.o[0], p.o[1], p.o[D / 32 - 2], p.o[D / 32 - 1]);
  else
    reinterpret_cast<float2 *>(dst)[lane] = make_float2(p.o[0], p.o[1]);
  if (lane == 0) {
    L.part_ml[row * L.slots + s] = make_float2(p.m, p.l);
    if (L.part_rest) L.part_rest[row * L.slots + s] = p.rest;
  }
}
// a joined with b: with M the larger maximum, O = sum 2^(M_s - M) O_s and l likewise.  A part without a maximum is
// zeros, or NaN where all its scores are, and is added as it is.
template <int D>
__device__ __forceinline__ void join_part(Part<D> &a, const Part<D> &b) {
  const float m = fmaxf(a.m, b.m), rest = b.m > a.m || (b.m == a.m && b.rest > a.rest) ? b.rest : a.rest;
  const float fa = a.m == -INFINITY ? 1.0f : exp2_approx((a.m - m) + (a.rest - rest));
  const float fb = b.m == -INFINITY ? 1.0f : exp2_approx((b.m - m) + (b.rest - rest));
  a.m = m;
  a.rest = rest;
  a.l = fmaf(a.l, fa, b.l * fb);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) a.o[d] = fmaf(a.o[d], fa, b.o[d] * fb);
}
template <int D>
__device__ __forceinline__ void write_row(const AttendParams &P, const AttendPlan &L, int64_t token, int hq, int lane,
                                          const Part<D> &p) {
  const float r = p.l == 0.0f ? 0.0f : 1.0f / p.l;
  float x[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) x[d] = p.l == 0.0f ? 0.0f : p.o[d] * r;
  uint16_t *dst = P.out + token * P.out_token + hq * P.out_head + lane * (D / 32);
  const uint32_t w0 = pack_bf16(x[0], x[1]), w1 = pack_bf16(x[D / 32 - 2], x[D / 32 - 1]);
  if (L.ovec && D == 128) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(w0, w1);
  } else if (L.ovec) {
    *reinterpret_cast<uint32_t *>(dst) = w0;
  } else {
    dst[0] = static_cast<uint16_t>(w0);
    dst[1] = static_cast<uint16_t>(w0 >> 16);
    if (D == 128) {
      dst[2] = static_cast<uint16_t>(w1);
      dst[3] = static_cast<uint16_t>(w1 >> 16);
    }
  }
  if (P.lse && lane == 0) P.lse[token * P.Hq + hq] = p.l == 0.0f ? -INFINITY : (p.m + (p.rest + log2f(p.l))) * kLn2;
}

// A CTA of the private part: a request's row tile of one kv head over one chunk of its keys.
struct OwnTile {
  int64_t first;        // the request's first row
  int i, h, gam, len;   // the request, the kv head, its drafts and keys
  int r0, rows;         // of the request's (gam + 1) * group rows
  int split, k_begin, k_end;
  bool whole;           // every key that the rows see: the result is the output
};
// False: nothing to do.  `most` rows a tile; the request's groups of 8 rows are dealt evenly to as few tiles as hold them.
__device__ __forceinline__ bool own_tile(const AttendParams &P, const AttendPlan &L, int b, int most, OwnTile &T) {
  const int tile = b % L.own_tiles;
  b /= L.own_tiles;
  T.h = b % P.c.num_kv_heads;
  b /= P.c.num_kv_heads;
  T.split = b % L.own_splits;
  T.i = b / L.own_splits;
  T.k_begin = P.prefix + T.split * L.own_chunk;
  uint32_t bits = 0;
  const bool ok = attend_request(P, T.i, T.first, T.gam, T.len, bits);
  if (bits && tile == 0 && T.h == 0 && T.split == 0 && threadIdx.x == 0 && P.status)
    atomicOr(P.status, static_cast<int>(bits));
  if (!ok) return false;
  const int all = (T.gam + 1) * P.group, groups = (all + 7) / 8, tiles = (groups * 8 + most - 1) / most;
  if (tile >= tiles) return false;
  const int per = (groups + tiles - 1) / tiles * 8;
  T.r0 = tile * per;
  T.rows = min(per, all - T.r0);
  if (T.rows <= 0) return false;
  T.k_end = min(T.len, T.k_begin + L.own_chunk);
  // (a request without a prefix and with one chunk of keys or none needs no joining)
  T.whole = P.prefix == 0 && T.len <= L.own_chunk;
  return T.k_end > T.k_begin || (T.whole && T.split == 0);
}

// The private part over the 4-bit cache (sv_attend4.cu): tiles of 16 rows where every request's rows fit, of 32 where they
// do or most requests' do, else of 64.  256 requests x 4096 keys, 16 rows each: 289 us in tiles of 16, 327 in tiles of 32;
// but ragged ones of 12 rows on average and 20 at most 384 against 361.  Up to 8192 keys, by mean rows, in tiles of 32 and of
// 64: with 36 rows at most 20 428 and 469, 23 461 and 475, 24 474 and 479, 26 496 and 487; with 44 at most 20 440 and 461,
// 23 466 and 468, 24 477 and 468; with 64 at most 20 456 and 468, 22 471 and 471, 23 478 and 472, 24 488 and 474.
constexpr int kOwnRows4 = 64, kOwnRowsMean = 23;
inline int own4_rows(const AttendParams &p) {
  const int64_t most = (p.G + 1) * static_cast<int64_t>(p.group), all = (p.T + p.N) * p.group;
  return most <= 16 ? 16 : most <= 32 || all <= static_cast<int64_t>(p.N) * kOwnRowsMean ? 32 : kOwnRows4;
}
cudaError_t enable_own4_kernels();
cudaError_t launch_own4(const AttendParams &p, const AttendPlan &L, cudaStream_t stream);

}  // namespace sv
