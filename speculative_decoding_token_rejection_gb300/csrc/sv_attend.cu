// sv_attend.cu -- attention of the verify tokens over the paged 8-bit cache:
// the warp-streaming kernel and the joining of its partial results.
//
// A request's rows for one kv head -- (gamma + 1) tokens times the query heads
// of the group -- all read the same keys, so the private part is bound by HBM:
// 2 * head_dim + 8 bytes a key for 4 * head_dim * rows operations.  Each warp
// streams keys on its own, 32 at a time, through shared memory of its own
// (cp.async, two tiles deep), so no warp waits for another in the
// loop.  A copy's eight (D = 64: four) neighbouring lanes take a whole row:
// with the rows dealt to lanes the way the products read them, every 32-byte
// sector was a request of its own, and the requests, not the bytes, set the
// pace (256 private histories: 830 us, waiting for the data or not).  The
// order of the inner dimension of a product is free, so lane (g, c) of a
// 16x8x16 product takes 16-byte columns c, c + 4 of the rows of keys g, g + 8,
// ..., the queries are laid out once in the same order, and no byte is moved
// again; for the second product lane (g, c) takes dimensions [g * D/8,
// (g + 1) * D/8) of the keys whose weights meet them.
//
// Both products are transposed: scores [keys x rows] = K Q^T and outputs
// [dims x rows] = V^T P^T, so the few rows are the 8-wide side of the
// instruction and a tile of 20 rows pays for 24, not 32; the weights turn
// round between the products by 8x8 transposes in registers.  Bytes become
// f16 in registers (exact); sums are fp32.  The running maximum of a row is
// raised only when a weight would pass 2^8, so most tiles neither reduce
// across lanes nor rescale.
//
// The key range of a row tile is cut over CTAs (and over a CTA's four warps)
// when there are few row tiles; the partial results (M, l, O) of a CTA go to
// the workspace and a second kernel joins them.
//
// Measured: 256 requests of 1 to 9 tokens over up to 8192 keys of their own
// (32 heads over 8 of 128, e4m3), 481 us, 4.6 TB/s or 68 % of the copy rate.
// Eight warps an SM cannot hide their own latencies: issue slots are 36 % busy.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kKeys = 32;    // keys of a warp's tile
constexpr float kRaise = 8;  // a row's maximum is raised when a weight would pass 2^kRaise

constexpr int kGroups = 4;   // groups of 8 rows in a row tile
constexpr int kStages = 2;   // tiles in a warp's ring
static_assert(kStages == 2, "the mask of a tile's keys that are left out is that of the copy before it");

// Two CTAs per SM: 255 registers hold four row groups (outputs 128), and 150
// KB of shared memory leave the L1 cache 100 KB.  Three CTAs of up to three
// groups (168 registers), or three stages, were slower -- 256 private
// histories 691 and 675 us against 593 -- although more copies were in flight.
template <int D>
struct Layout {
  static constexpr int kScales = kKeys * 2 * D;  // of a stage: keys, values, then (key scale, value scale) of key `lane`
  static constexpr int kStage = kScales + kKeys * 8;
  static constexpr int kQuery = kGroups * 8 * D * 2;
  static constexpr int kPitch = D + 4;  // floats of an output row while the warps' results are joined
  static constexpr int kRing = kAttendWarps * kStages * kStage;
  static constexpr int kJoin = kAttendWarps * kGroups * 8 * kPitch * 4;
  static constexpr int kBytes = kQuery + (kRing > kJoin ? kRing : kJoin);
};

// Place of 16-byte column `col` of a tile's row.  Columns of a 128-byte line
// change places so that the eight lanes that are served at once meet all
// banks: for K they read columns c, c = 0 .. 3, of rows 2i and 2i + 1; for V
// columns 2i and 2i + 1 of rows 2c (+ 1).
template <int D, bool VALUES>
__device__ __forceinline__ int tile_at(int row, int col) {
  const int line = D == 128 ? row : row >> 1, in = D == 128 ? col : (row & 1) * 4 + col;
  const int turn = VALUES ? (row >> 1 & 3) << 1 : (D == 128 ? (row & 1) << 2 : 0);
  return line * 128 + (in ^ turn) * 16;
}

// The four bytes' numbers with the other sign (int8: -128, which the writer does not give, becomes 127).
template <int FMT>
__device__ __forceinline__ uint32_t negated(uint32_t w) {
  return FMT == SV_CACHE_INT8 ? __vnegss4(w) : w ^ 0x80808080u;
}

struct RowTile {
  int h, k_begin, k_end, slot, r0, rows;
  const int32_t *table;
  int *token;  // [rows] in shared memory: verify token of a row, or -1
  int *limit;  // keys that the row sees are below it
  bool whole;  // every key that the rows see: the result is the output
  int page;    // of the lane's key of its warp's first tile, looked up before the request's length was there
};

// One partial result of a row: M, l and the lane's dimensions of O.
template <int D>
struct Part {
  float m, l, o[D / 32];
};
constexpr int kJoinAhead = 4;  // partial results of a row in flight
template <int D>
__device__ __forceinline__ Part<D> load_part(const AttendPlan &L, int64_t row, int s, int lane) {
  Part<D> p;
  const float2 ml = __ldcg(L.part_ml + row * L.slots + s);
  p.m = ml.x;
  p.l = ml.y;
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
  if (lane == 0) L.part_ml[row * L.slots + s] = make_float2(p.m, p.l);
}
// a joined with b: with M the larger maximum, O = sum 2^(M_s - M) O_s and l likewise.  A part without a maximum is
// zeros, or NaN where all its scores are, and is added as it is.
template <int D>
__device__ __forceinline__ void join_part(Part<D> &a, const Part<D> &b) {
  const float m = fmaxf(a.m, b.m);
  const float fa = a.m == -INFINITY ? 1.0f : exp2_approx(a.m - m), fb = b.m == -INFINITY ? 1.0f : exp2_approx(b.m - m);
  a.m = m;
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
  if (P.lse && lane == 0) P.lse[token * P.Hq + hq] = p.l == 0.0f ? -INFINITY : (p.m + log2f(p.l)) * kLn2;
}

struct JoinSmem {
  float m[kAttendWarps][32], l[kAttendWarps][32];
  uint32_t top[kGroups * 8];  // largest finite |q| of a row
  uint32_t none[kGroups * 8];  // the row sees a value scale that is no number
  int token[kGroups * 8], limit[kGroups * 8];
};

// ANY false: for value scales that kv_write gives to finite rows, and pages inside the cache.  Returns true, with nothing
// written, if the CTA met another one: ANY true then takes any.  (With the rare case in the one loop, as a branch of
// its own in each tile, the values' loads stayed behind it: 256 private histories 526 us against 477.)
template <int D, int FMT, int NT, bool ANY>
__device__ __forceinline__ bool attend_tile(const AttendParams &P, const AttendPlan &L, const RowTile &T, uint8_t *smem,
                                            JoinSmem &J) {
  using Y = Layout<D>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  // ---- the stream of keys ----
  uint8_t *const ring_ptr = smem + Y::kQuery + warp * kStages * Y::kStage;
  const uint32_t ring = smem_addr(ring_ptr);
  const int tiles_all = (max(0, T.k_end - T.k_begin) + kKeys - 1) / kKeys;
  const int ntiles = (tiles_all - warp + kAttendWarps - 1) / kAttendWarps;  // tiles warp, warp + 4, ...
  constexpr int kCols = D / 16;  // 16-byte columns of a row, one lane each in a copy
  const int ccol = lane % kCols;
  const uint8_t *const kcol = static_cast<const uint8_t *>(P.c.k) + T.h * P.c.head_stride + ccol * 16;
  const uint8_t *const vcol = static_cast<const uint8_t *>(P.c.v) + T.h * P.c.head_stride + ccol * 16;
  const float *const kscale = P.c.k_scale + T.h * P.c.scale_head_stride;
  const float *const vscale = P.c.v_scale + T.h * P.c.scale_head_stride;
  uint32_t bits = 0;
  auto page_of = [&](int it) {  // of the lane's key of the warp's tile `it`
    const int k = T.k_begin + (it * kAttendWarps + warp) * kKeys + lane;
    return it < ntiles && k < T.k_end ? (k < P.row0 ? P.tables : T.table)[div_by(k, L.page)] : -1;
  };
  // Copies of a tile: the lane's key first, then the rows, a lane's neighbours taking a whole one, in kCols steps.
  uint32_t unit = 0, dead = 0;  // the row's place in units of L.unit_bytes
  auto copy_keys = [&](int it, int stage, int page) {
    const int k = T.k_begin + (it * kAttendWarps + warp) * kKeys + lane;
    const bool in = k < T.k_end, live = in && page >= 0 && page < P.c.num_blocks;
    if (in && !live) bits = SV_DATA_BAD_SLOT;
    const int off = k - div_by(k, L.page) * P.c.block_size;
    const uint32_t dst = ring + stage * Y::kStage + Y::kScales + lane * 8;
    unit = live ? page * L.block_units + off * L.token_units : 0u;
    const int64_t sat = live ? page * P.c.scale_block_stride + off * P.c.scale_token_stride : 0;
    dead = __ballot_sync(0xFFFFFFFFu, !live);
    copy_async<4>(dst, kscale + sat, live ? 4 : 0);
    copy_async<4>(dst + 4, vscale + sat, live ? 4 : 0);
  };
  auto copy_rows = [&](int stage, int step) {
    const uint32_t dst = ring + stage * Y::kStage;
    const int row = step * (32 / kCols) + lane / kCols;
    const uint32_t u = __shfl_sync(0xFFFFFFFFu, unit, row);
    const uint32_t n = dead >> row & 1u ? 0u : 16u;
    const uint64_t at = static_cast<uint64_t>(u) * L.unit_bytes;
    copy_async<16>(dst + tile_at<D, false>(row, ccol), kcol + at, n);
    copy_async<16>(dst + kKeys * D + tile_at<D, true>(row, ccol), vcol + at, n);
  };

  // (the first copies are on their way before the queries are looked at)
  int page = T.page;
#pragma unroll
  for (int it = 0; it < kStages - 1; ++it) {
    if (it < ntiles) {
      copy_keys(it, it, page);
#pragma unroll
      for (int x = 0; x < kCols; ++x) copy_rows(it, x);
    }
    copy_commit();
    page = page_of(it + 1);
  }

  // ---- the queries as operand fragments: 8 consecutive dimensions for each lane and pair of steps ----
  constexpr int kFrags = (NT * (D / 32) * 32 + kAttendThreads - 1) / kAttendThreads;  // of a thread
  uint4 *const qfrag = reinterpret_cast<uint4 *>(smem);
  const float c_all = P.scale * kLog2e;
  {
    uint4 x[kFrags];
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const int at = f * kAttendThreads + tid, ln = at & 31, s2 = (at >> 5) % (D / 32), nt = (at >> 5) / (D / 32);
      const int r = nt * 8 + (ln >> 2);
      // steps 4q .. 4q + 3 are column q * 4 + c of 16 dimensions; s2 counts pairs of steps
      const int dim = ((s2 >> 1) * 4 + (ln & 3)) * 16 + (s2 & 1) * 8;
      x[f] = make_uint4(0, 0, 0, 0);
      if (nt < NT && r < T.rows && T.token[r] >= 0) {
        const int lr = T.r0 + r, hq = T.h * P.group + lr - div_by(lr, L.group) * P.group;
        const uint16_t *src = P.q + T.token[r] * P.q_token + hq * P.q_head + dim;
        if (L.qvec) {
          x[f] = *reinterpret_cast<const uint4 *>(src);
        } else {
          x[f].x = src[0] | static_cast<uint32_t>(src[1]) << 16;
          x[f].y = src[2] | static_cast<uint32_t>(src[3]) << 16;
          x[f].z = src[4] | static_cast<uint32_t>(src[5]) << 16;
          x[f].w = src[6] | static_cast<uint32_t>(src[7]) << 16;
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const int at = f * kAttendThreads + tid, r = (at >> 5) / (D / 32) * 8 + (lane >> 2);
      const uint32_t w[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = w[e] << 16 & 0x7FFFFFFFu, b = w[e] & 0x7FFF0000u;
        if (a < 0x7F800000u) top = max(top, a);
        if (b < 0x7F800000u) top = max(top, b);
      }
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      if (c == 0 && r < NT * 8) atomicMax(&J.top[r], top);
    }
    __syncthreads();
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const int at = f * kAttendThreads + tid, r = (at >> 5) / (D / 32) * 8 + (lane >> 2);
      const float up = pow2(query_shift(r < NT * 8 ? J.top[r] : 0u));
      uint32_t w[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_f16(bf16_bits_to_float(w[e] & 0xFFFFu) * up, bf16_bits_to_float(w[e] >> 16) * up);
      if (at < NT * (D / 32) * 32) qfrag[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  bool shifted = false;  // some row of the tile was multiplied by a power of two
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) shifted |= query_shift(J.top[nt * 8 + g]) != 0;
  shifted = __any_sync(0xFFFFFFFFu, shifted);
  int limit[NT][2], low = 0x7FFFFFFF;  // of rows nt * 8 + 2c, + 1; low: keys below it are seen by every row of the tile
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * c + e;
      limit[nt][e] = r < T.rows ? T.limit[r] : 0x7FFFFFFF;
      low = min(low, limit[nt][e]);
    }
  low = __reduce_min_sync(0xFFFFFFFFu, low);
  __syncthreads();

  float o[D / 16][NT][4];  // rows nt * 8 + 2c, + 1: dimension g * D/8 + 2t, then dimension g * D/8 + 2t + 1
  Pair l[NT], neg[NT];     // sums over the lane's keys, and the negated maxima
  uint32_t set = 0;        // bit nt * 2 + e: the row has a maximum (without one, weights are taken against 0)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    l[nt] = neg[nt] = pair(0.0f, 0.0f);
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[t][nt][0] = o[t][nt][1] = o[t][nt][2] = o[t][nt][3] = 0.0f;
  }
  int stage = 0, fill = kStages - 1;
  bool strange = false;
  for (int it = 0; it < ntiles; ++it) {
    copy_wait<kStages - 2>();
    __syncwarp();  // the tile is there for every lane, and no lane still reads the one before it
    const uint32_t gone = ANY ? dead : 0u;  // the tile's keys that are left out
    if (it + kStages - 1 < ntiles) {  // (in the place of the one before)
      copy_keys(it + kStages - 1, fill, page);
#pragma unroll
      for (int x = 0; x < kCols; ++x) copy_rows(fill, x);
    }
    copy_commit();
    if (++fill == kStages) fill = 0;
    page = page_of(it + kStages);
    uint8_t *const src = ring_ptr + stage * Y::kStage;
    if (++stage == kStages) stage = 0;
    const float2 sc = *reinterpret_cast<const float2 *>(src + Y::kScales + lane * 8);
    const float kc = sc.x * c_all;
    const int k0 = T.k_begin + (it * kAttendWarps + warp) * kKeys;
    float lv, inv;
    if (ANY) {
      value_scale_terms(sc.y, lv, inv);
    } else {
      lv = log2f(sc.y);
      inv = __frcp_rn(fmaxf(sc.y, kLeastScale));  // (0 behind the range: weight 0 times a number)
      strange |= !usual_scale(sc.y) && k0 + lane < T.k_end;  // (it is 0 for a page outside the cache)
    }
    // scores: keys g, g + 8 of each half mt of the tile, rows 2c, 2c + 1 of each group
    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
      uint4 kb[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) kb[x] = *reinterpret_cast<const uint4 *>(src + tile_at<D, false>(x * 8 + g, q * 4 + c));
#pragma unroll
      for (int s2 = 0; s2 < 2; ++s2) {
        uint4 b[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt] = qfrag[(nt * (D / 32) + q * 2 + s2) * 32 + lane];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint4 &w0 = kb[mt * 2], &w1 = kb[mt * 2 + 1];
            const uint32_t x0 = s2 ? (e ? w0.w : w0.z) : (e ? w0.y : w0.x);
            const uint32_t x1 = s2 ? (e ? w1.w : w1.z) : (e ? w1.y : w1.x);
            uint4 a;
            bytes_to_f16<FMT>(x0, a.x, a.z);
            bytes_to_f16<FMT>(x1, a.y, a.w);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(s[mt][nt], a, e ? b[nt].z : b[nt].x, e ? b[nt].w : b[nt].y);
          }
      }
    }
    const uint32_t odd = ANY ? __ballot_sync(0xFFFFFFFFu, !usual_scale(sc.y)) & ~gone : 0u;
    if (ANY && odd) {  // the lane puts its key's value right in the ring
      if (odd >> lane & 1u) {
#pragma unroll 1
        for (int col = 0; col < kCols; ++col) {
          uint4 &w = *reinterpret_cast<uint4 *>(src + kKeys * D + tile_at<D, true>(lane, col));
          w = usual_scale(-sc.y) ? make_uint4(negated<FMT>(w.x), negated<FMT>(w.y), negated<FMT>(w.z), negated<FMT>(w.w))
                                 : make_uint4(0, 0, 0, 0);
        }
      }
      const uint32_t none = __ballot_sync(0xFFFFFFFFu, !(fabsf(sc.y) < INFINITY)) & odd;
      if (none && lane < T.rows && k0 + __ffs(none) - 1 < T.limit[lane])
        J.none[lane] = 1;  // (the first such key decides which rows see one)
      __syncwarp();
    }
    // weights
    // x: scores without the value's scale.  A product of its own, rounded: subtracting a maximum that equals it gives 0.
    Pair x[4][NT];
    float vw[4];  // log2 of the value scale of keys g, g + 8, g + 16, g + 24
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = __shfl_sync(0xFFFFFFFFu, kc, k * 8 + g);
      vw[k] = __shfl_sync(0xFFFFFFFFu, lv, k * 8 + g);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        x[k][nt] = mul2(pair(s[k >> 1][nt][(k & 1) * 2], s[k >> 1][nt][(k & 1) * 2 + 1]), pair(f, f));
    }
    if (shifted) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Pair back = pair(pow2(-query_shift(J.top[nt * 8 + 2 * c])), pow2(-query_shift(J.top[nt * 8 + 2 * c + 1])));
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k][nt] = mul2(x[k][nt], back);
      }
    }
    if (k0 + kKeys > low || (ANY && gone)) {  // some row does not see all of the tile
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int key = ANY && (gone >> (k * 8 + g) & 1u) ? 0x7FFFFFFF : k0 + k * 8 + g;
          x[k][nt] = pair(key < limit[nt][0] ? lo(x[k][nt]) : -INFINITY, key < limit[nt][1] ? hi(x[k][nt]) : -INFINITY);
        }
    }
    // An exponent is the score less the maximum, and only then the value scale's log (a score too large to hold it
    // would lose it).
    auto exponent = [&](int k, int nt) { return add2(add2(x[k][nt], neg[nt]), pair(vw[k], vw[k])); };
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const Pair y = exponent(k, nt);
        most[0] = fmaxf(most[0], lo(y));
        most[1] = fmaxf(most[1], hi(y));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) raise |= most[e] > (set >> (nt * 2 + e) & 1u ? kRaise : -INFINITY);
    }
    if (__any_sync(0xFFFFFFFFu, raise)) {  // (seldom after the first tiles)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float r[2], up[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const Pair t = add2(x[k][nt], pair(vw[k], vw[k]));
          up[0] = fmaxf(up[0], lo(t));
          up[1] = fmaxf(up[1], hi(t));
        }
        float next[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int b = 4; b <= 16; b <<= 1) up[e] = fmaxf(up[e], __shfl_xor_sync(0xFFFFFFFFu, up[e], b));
          const bool had = set >> (nt * 2 + e) & 1u;
          const float old = -(e ? hi(neg[nt]) : lo(neg[nt]));
          next[e] = had ? fmaxf(old, up[e]) : up[e];
          r[e] = had ? exp2_approx(old - next[e]) : 1.0f;  // (nothing was added up without a maximum but NaN or zeros)
          if (next[e] == -INFINITY) {
            next[e] = old;
            r[e] = 1.0f;
          } else {
            set |= 1u << (nt * 2 + e);
          }
        }
        neg[nt] = pair(-next[0], -next[1]);
        const Pair rr = pair(r[0], r[1]);
        l[nt] = mul2(l[nt], rr);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          const Pair a = mul2(pair(o[t][nt][0], o[t][nt][1]), rr), b = mul2(pair(o[t][nt][2], o[t][nt][3]), rr);
          o[t][nt][0] = lo(a);
          o[t][nt][1] = hi(a);
          o[t][nt][2] = lo(b);
          o[t][nt][3] = hi(b);
        }
      }
    }
    uint32_t p[2][NT][2];  // weights of a half's keys 2c, 2c + 1 (then + 8) for row g
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = __shfl_sync(0xFFFFFFFFu, inv, k * 8 + g);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Pair y = exponent(k, nt);
        const float a = exp2_approx(lo(y)), b = exp2_approx(hi(y));
        l[nt] = fma2(pair(a, b), pair(d, d), l[nt]);
        p[k >> 1][nt][k & 1] = transpose_8x8(pack_f16(a, b));
      }
    }
    // values
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t v[4][D / 32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = j * 16 + (k >> 1) * 8 + 2 * c + (k & 1);
        if (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4 *>(src + kKeys * D + tile_at<D, true>(row, g));
          v[k][0] = w.x;
          v[k][1] = w.y;
          v[k][D / 32 - 2] = w.z;
          v[k][D / 32 - 1] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2 *>(src + kKeys * D + tile_at<D, true>(row, g >> 1) + (g & 1) * 8);
          v[k][0] = w.x;
          v[k][1] = w.y;
        }
      }
#pragma unroll
      for (int wd = 0; wd < D / 32; ++wd)
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          uint4 a;
          bytes_to_f16<FMT>(__byte_perm(v[0][wd], v[1][wd], t2 ? 0x7362 : 0x5140), a.x, a.y);
          bytes_to_f16<FMT>(__byte_perm(v[2][wd], v[3][wd], t2 ? 0x7362 : 0x5140), a.z, a.w);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816(o[wd * 2 + t2][nt], a, p[j][nt][0], p[j][nt][1]);
        }
    }
  }
  copy_wait<0>();
  if (!ANY && __syncthreads_or(strange)) return true;
  if (bits && P.status) atomicOr(P.status, static_cast<int>(bits));

  // ---- the four warps' results joined ----
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = e ? hi(l[nt]) : lo(l[nt]);
#pragma unroll
      for (int b = 4; b <= 16; b <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, b);
      if (g == 0) {
        J.m[warp][nt * 8 + 2 * c + e] = set >> (nt * 2 + e) & 1u ? -(e ? hi(neg[nt]) : lo(neg[nt])) : -INFINITY;
        J.l[warp][nt * 8 + 2 * c + e] = sum;
      }
    }
  __syncthreads();  // (every warp is done with its ring as well)
  float *const acc = reinterpret_cast<float *>(smem + Y::kQuery);  // [warp][row][kPitch]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * c + e;
      float *dst = acc + (warp * NT * 8 + r) * Y::kPitch + g * (D / 8);
#pragma unroll
      for (int t = 0; t < D / 16; t += 2)
        *reinterpret_cast<float4 *>(dst + 2 * t) =
            make_float4(o[t][nt][e], o[t][nt][2 + e], o[t + 1][nt][e], o[t + 1][nt][2 + e]);
    }
  __syncthreads();
  // a lane takes D/32 neighbouring dimensions of a row
  constexpr int kDims = D / 32;
  for (int r = warp; r < T.rows; r += kAttendWarps) {
    const int token = T.token[r];
    if (token < 0) continue;
    const int lr = T.r0 + r, hq = T.h * P.group + lr - div_by(lr, L.group) * P.group;
    Part<D> all;
    all.m = fmaxf(fmaxf(J.m[0][r], J.m[1][r]), fmaxf(J.m[2][r], J.m[3][r]));
    all.l = 0.0f;
#pragma unroll
    for (int d = 0; d < kDims; ++d) all.o[d] = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttendWarps; ++w) {
      // (a warp whose keys the row does not see adds zeros; one with NaN scores alone has no maximum, and adds them)
      const float f = J.m[w][r] == -INFINITY ? 1.0f : exp2_approx(J.m[w][r] - all.m);
      all.l = fmaf(J.l[w][r], f, all.l);
#pragma unroll
      for (int d = 0; d < kDims; ++d) all.o[d] = fmaf(acc[(w * NT * 8 + r) * Y::kPitch + lane * kDims + d], f, all.o[d]);
    }
    if (ANY && J.none[r]) {
#pragma unroll
      for (int d = 0; d < kDims; ++d) all.o[d] = __uint_as_float(0x7FC00000u);
    }
    if (T.whole)
      write_row<D>(P, L, token, hq, lane, all);
    else
      store_part<D>(L, static_cast<int64_t>(token) * P.Hq + hq, T.slot, lane, all);
  }
  return false;
}

template <int D, int FMT, bool ANY>
__device__ __forceinline__ bool attend_block(const AttendParams &P, const AttendPlan &L, JoinSmem &join) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, H = P.c.num_kv_heads;
  RowTile T;
  T.table = P.tables;
  T.token = join.token;
  T.limit = join.limit;
  T.whole = false;
  int64_t first = 0;
  int len = 0, gam = 0;
  const bool shared_part = static_cast<int>(blockIdx.x) < L.prefix_items;
  if (shared_part) {
    int b = blockIdx.x;
    const int tile = b % L.prefix_tiles;
    b /= L.prefix_tiles;
    T.h = b % H;
    T.slot = b / H;
    T.r0 = tile * kGroups * 8;
    T.rows = min(kGroups * 8, L.rows - T.r0);
    T.k_begin = T.slot * L.prefix_chunk;
    T.k_end = min(P.prefix, T.k_begin + L.prefix_chunk);
    const int k = T.k_begin + tid;
    T.page = k < T.k_end ? T.table[div_by(k, L.page)] : -1;
  } else {
    int b = blockIdx.x - L.prefix_items;
    const int tile = b % L.own_tiles;
    b /= L.own_tiles;
    T.h = b % H;
    b /= H;
    const int split = b % L.own_splits;
    const int i = b / L.own_splits;
    T.table += i * P.table_stride;
    T.k_begin = P.prefix + split * L.own_chunk;
    const int k = T.k_begin + tid;
    T.page = k < P.max_seq ? (k < P.row0 ? P.tables : T.table)[div_by(k, L.page)] : -1;  // (tables hold max_seq keys, whatever the length)
    uint32_t bits = 0;
    const bool ok = attend_request(P, i, first, gam, len, bits);
    if (bits && tile == 0 && T.h == 0 && split == 0 && tid == 0 && P.status) atomicOr(P.status, static_cast<int>(bits));
    if (!ok) return false;
    // the request's row groups, dealt evenly to as few tiles as hold them
    const int all = (gam + 1) * P.group, groups = (all + 7) / 8, tiles = (groups + kGroups - 1) / kGroups;
    if (tile >= tiles) return false;
    const int per = (groups + tiles - 1) / tiles * 8;
    T.r0 = tile * per;
    T.rows = min(per, all - T.r0);
    if (T.rows <= 0) return false;
    T.slot = L.prefix_splits + split;
    T.k_end = min(len, T.k_begin + L.own_chunk);
    // (a request without a prefix and with one chunk of keys or none needs no joining)
    T.whole = P.prefix == 0 && len <= L.own_chunk;
    if (T.k_end <= T.k_begin && !(T.whole && split == 0)) return false;
  }
  if (tid < kGroups * 8) join.top[tid] = join.none[tid] = 0;
  if (tid < T.rows) {
    const int t = div_by(T.r0 + tid, L.group);
    int token = t, limit;
    if (shared_part) {
      limit = prefix_limit(P, t);
      if (limit < 0) {  // nobody's row
        token = -1;
        limit = 0x7FFFFFFF;
      }
    } else {
      token = static_cast<int>(first) + t;
      limit = len - gam + t;
    }
    join.token[tid] = token;
    join.limit[tid] = limit;
  }
  __syncthreads();
  if (shared_part) {  // (keys behind every row's are not read: what is there may be no numbers)
    const int r = tid & 31;
    T.k_end = min(T.k_end, __reduce_max_sync(0xFFFFFFFFu, r < T.rows && join.token[r] >= 0 ? join.limit[r] : 0));
  }
  const int groups = (T.rows + 7) / 8;
  if (groups == 1) return attend_tile<D, FMT, 1, ANY>(P, L, T, smem, join);
  if (groups == 2) return attend_tile<D, FMT, 2, ANY>(P, L, T, smem, join);
  if (groups == 3) return attend_tile<D, FMT, 3, ANY>(P, L, T, smem, join);
  return attend_tile<D, FMT, 4, ANY>(P, L, T, smem, join);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kAttendThreads, 2)
    attend_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ AttendPlan L) {
  pdl_enter();
  __shared__ JoinSmem join;
  if (attend_block<D, FMT, false>(P, L, join)) attend_block<D, FMT, true>(P, L, join);
}

// Joins the partial results of a row: one warp a row.
template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const AttendParams P, const AttendPlan L) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x;
  int64_t first;
  int g, len;
  uint32_t bits = 0;
  if (!attend_request(P, i, first, g, len, bits)) return;
  const int own = len > P.prefix ? (len - P.prefix + L.own_chunk - 1) / L.own_chunk : 0;
  if (P.prefix == 0 && own <= 1) return;  // (written already)
  const int rows = (g + 1) * P.Hq;
  for (int r = blockIdx.y * kWarps + warp; r < rows; r += gridDim.y * kWarps) {
    const int64_t row = first * P.Hq + r;
    const int j = r / P.Hq, hq = r - j * P.Hq, h = hq / P.group;
    const int shared = P.prefix ? prefix_slots(L, h, (static_cast<int>(first) + j) * P.group + hq - h * P.group) : 0;
    const int slots = shared + own;
    Part<D> all;
    all.m = -INFINITY;
    all.l = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) all.o[d] = 0.0f;
    for (int s = 0; s < slots; s += kJoinAhead) {
      Part<D> part[kJoinAhead];
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u)
        if (s + u < slots) part[u] = load_part<D>(L, row, s + u < shared ? s + u : s + u - shared + L.prefix_splits, lane);
#pragma unroll
      for (int u = 0; u < kJoinAhead; ++u)
        if (s + u < slots) join_part<D>(all, part[u]);
    }
    write_row<D>(P, L, first + j, hq, lane, all);
  }
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

constexpr int kChunkStep = kAttendWarps * kKeys;  // a CTA's four warps take 32 keys each
constexpr int kTensorRows = 96;  // a shared prefix goes to the tensor-memory kernel from here on
constexpr int kTensorLeast = 4;  // key tiles of a CTA of that kernel, where the prefix has as many
constexpr int kTensorBegin = 7;  // and what beginning another (kv head, row tile) costs it, in key tiles
constexpr int kChunkMost = 8192;                  // so that the longest request is no long tail

// Chunks for `keys` keys when `base` CTAs work on every chunk: enough to give
// each SM two CTAs twice over, none below kChunkStep keys.
// Returns the chunk count before chunks were rounded up to whole steps: no
// fewer than `splits`, and never fewer for more keys, so that a workspace
// sized for longer requests always holds.
int cut(int64_t base, int keys, int num_sms, int &splits, int &chunk) {
  if (keys <= 0) {
    splits = 0;
    chunk = kChunkStep;
    return 0;
  }
  const int64_t want = std::max<int64_t>(1, 4LL * num_sms / std::max<int64_t>(1, base));
  const int most = ceil_div(keys, kChunkStep);
  splits = static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(want, ceil_div(keys, kChunkMost))));
  const int bound = splits;
  chunk = ceil_div(ceil_div(keys, splits), kChunkStep) * kChunkStep;
  splits = ceil_div(keys, chunk);
  return bound;
}

// A short prefix is read by every request for itself (from L2), which saves the
// kernels that would share it, the partial results and the join.  A call's time
// for it, fitted to both sides of 56 calls' sizes at prefixes of 128 to 16384
// keys (head_dim 64 and 128, int8, private ranges of 128 and 1024 keys): read
// by each, a key costs a private CTA 24 ps and 7 for each of its row groups;
// shared on the tensor cores, a key costs a kv head 75 ps and 64 for each row
// tile, and the kernels 31 us and 950 ps a row to begin and end.  So a prefix is
// shared from the length where the two are equal, and always beyond 16384, the
// longest that was measured.  (On the whole table this loses 4 % at most to the
// better side.)  Fewer rows share it in CTAs like the private ones, whose keys cost
// two and a half times as much by the fit, and 0.2 us (5 us at most are lost).
// Measured, us a call, shared | by each request (32 heads over 8 of 128, 128
// private keys): 8 requests x 4 tokens, prefix 2048 57 | 25, 8192 65 | 42; 64 x 5,
// 1024 77 | 50, 2048 84 | 78, 4096 94 | 136; 512 x 8, 512 305 | 257, 1024 335 | 365;
// 512 x 1, 256 118 | 95, 512 120 | 126; 2 x 5 (40 rows), 4096 33 | 29, 16384 48 | 38;
// 16 x 1 (64 rows), 256 17 | 17, 1024 19 | 22.
AttendParams short_prefix(AttendParams p) {
  const int64_t H = p.c.num_kv_heads, own = (p.G + 1) * static_cast<int64_t>(p.group), own_tiles = ceil_div(own, 8 * kGroups);
  // (the rows there may be, so that calls with fewer tokens choose alike)
  const int64_t rows = p.N * own;
  int64_t saved = p.N * H * own_tiles * (24 + 7 * ceil_div(ceil_div(own, 8), own_tiles)), begin, most;  // ps a key; ps; keys
  if (rows >= kTensorRows) {
    saved -= H * (75 + 64 * static_cast<int64_t>(ceil_div(rows, kPrefixRowTile)));
    begin = 31000000 + 950 * rows * H;
    most = 16384 + 1;
  } else {
    saved -= H * 5 * (24 * ceil_div(rows, 8 * kGroups) + 7 * ceil_div(rows, 8)) / 2;
    begin = 200000;
    most = INT64_MAX;
  }
  if (p.prefix < (saved > 0 ? std::min(most, 128 + begin / saved) : most)) {
    p.row0 = p.prefix;
    p.prefix = 0;
  }
  return p;
}

AttendPlan make_plan(const AttendParams &p, int num_sms, int64_t *bytes = nullptr) {
  AttendPlan L{};
  L.page = fast_div(std::max(1, p.c.block_size));
  L.group = fast_div(p.group);
  L.rows = static_cast<int32_t>((p.T + p.N) * p.group);
  L.own_tiles = ceil_div((p.G + 1) * static_cast<int64_t>(p.group), 8 * kGroups);
  L.prefix_tiles = ceil_div(L.rows, 8 * kGroups);
  // (at least one private chunk, though no request may have private keys: its CTAs look at the requests' ranges)
  int bound = std::max(1, cut(static_cast<int64_t>(p.N) * p.c.num_kv_heads * L.own_tiles, p.max_seq - p.prefix, num_sms,
                              L.own_splits, L.own_chunk));
  L.own_splits = std::max(1, L.own_splits);
  const int64_t image_tiles = ceil_div(p.prefix, kPrefixKeyTile), tensor_tiles = ceil_div(L.rows, kPrefixRowTile);
  const int64_t items = tensor_tiles * p.c.num_kv_heads, tiles = items * image_tiles;
  // an item begun costs a CTA about kTensorBegin tiles' time: so many empty units lie between two items where CTAs get
  // more than the least, and one that begins a second item gets fewer tiles (64 requests x 5 tokens over 8192 keys: 123
  // us the whole call, with no empty units 132, with 4 of them 126, with 10 125; 512 x 8 over 16384: 1073 to 1078 all)
  const int64_t gap = tiles > static_cast<int64_t>(num_sms) * kTensorLeast ? kTensorBegin : 0;
  const int64_t units = items * (image_tiles + gap) - gap;
  if (p.prefix > 0 && L.rows >= kTensorRows && units <= 0x3FFFFFFF) {
    L.tensor_tiles = static_cast<int32_t>(tensor_tiles);
    L.image_tiles = static_cast<int32_t>(image_tiles);
    L.period = static_cast<int32_t>(image_tiles + gap);
    L.units = static_cast<int32_t>(units);
    L.units_cta = std::max(ceil_div(units, num_sms), std::min(kTensorLeast, L.image_tiles));
    L.prefix_splits = L.image_tiles == 1 ? 1 : (L.image_tiles - 2) / L.units_cta + 2;  // an item's CTAs at most
    bound += L.prefix_splits;
  } else {
    bound += cut(static_cast<int64_t>(p.c.num_kv_heads) * L.prefix_tiles, p.prefix, num_sms, L.prefix_splits,
                 L.prefix_chunk);
    L.prefix_items = L.prefix_tiles * p.c.num_kv_heads * L.prefix_splits;
  }
  // (Where the private part is one chunk its CTAs could join the prefix's partial results as they end.  Measured, with
  // four rows' results in flight: 203 us for 512 requests x 32 rows, against 147 and a join by itself.)
  L.slots = L.prefix_splits + L.own_splits;
  L.unit_bytes = cache_unit(p.c);
  L.block_units = static_cast<uint32_t>(p.c.block_stride / L.unit_bytes);
  L.token_units = static_cast<uint32_t>(p.c.token_stride / L.unit_bytes);
  L.qvec = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0 && p.q_token % 8 == 0 && p.q_head % 8 == 0;
  L.ovec = (reinterpret_cast<uintptr_t>(p.out) & 7u) == 0 && p.out_token % 4 == 0 && p.out_head % 4 == 0;
  const int64_t rows = static_cast<int64_t>(L.rows) * p.c.num_kv_heads;
  // the workspace: the prefix's tiles, then M and l, then O
  const int64_t image = static_cast<int64_t>(L.image_tiles) * p.c.num_kv_heads * kPrefixKeyTile * p.c.head_dim * 4;
  if (bytes) *bytes = bound <= 1 ? 0 : image + ((rows * bound * 8 + 15) & ~int64_t{15}) + rows * bound * p.c.head_dim * 4;
  L.image = static_cast<uint8_t *>(p.workspace);
  L.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(p.workspace) + image);
  L.part_o = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + image + ((rows * L.slots * 8 + 15) & ~int64_t{15}));
  return L;
}

template <int D, int FMT>
cudaError_t launch(const AttendParams &p, const AttendPlan &L, int num_sms, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const int64_t own = static_cast<int64_t>(p.N) * p.c.num_kv_heads * L.own_tiles * L.own_splits;
  if (own + L.prefix_items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(own + L.prefix_items));
  cfg.blockDim = dim3(kAttendThreads);
  cfg.dynamicSmemBytes = Layout<D>::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  cudaError_t e = L.tensor_tiles ? launch_prefix(p, L, stream) : cudaSuccess;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, attend_kernel<D, FMT>, p, L);
  if (e != cudaSuccess || L.slots == 1) return e;
  // a warp takes two rows where there are rows for more than eight waves of CTAs (512 requests x 256 rows: 1084 us the
  // whole call against 1108 with one row a warp; 64 x 160: 138.5 against 137.4)
  const int64_t rows = (p.G + 1) * static_cast<int64_t>(p.Hq), each = rows * p.N > 320LL * num_sms ? 2 : 1;
  cfg.gridDim = dim3(p.N, std::max(1, std::min(65535, ceil_div(rows, kWarps * each))));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, L);
}

template <int D, int FMT>
cudaError_t enable() {
  return cudaFuncSetAttribute(attend_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
}

}  // namespace

cudaError_t enable_attend_kernels() {
  cudaError_t e;
  if ((e = enable<128, SV_CACHE_INT8>()) != cudaSuccess || (e = enable<128, SV_CACHE_E4M3>()) != cudaSuccess ||
      (e = enable<64, SV_CACHE_INT8>()) != cudaSuccess || (e = enable_prefix_kernels()) != cudaSuccess)
    return e;
  return enable<64, SV_CACHE_E4M3>();
}

int64_t attend_workspace_bytes(const AttendParams &a, int num_sms, bool fewer) {
  AttendParams p = short_prefix(a);
  int64_t most = 0;
  make_plan(p, num_sms, &most);
  if (!fewer || p.prefix == 0) return most;
  // Fewer tokens may have more partial results each.  Calls of one plan need the most with the most rows: 256 a row tile
  // of the tensor-memory kernel, and below kTensorRows 32 a row tile.
  const auto with = [&](int64_t rows) {
    p.T = std::min(a.T, rows / p.group - p.N);
    if (p.T < 0) return;
    int64_t bytes = 0;
    make_plan(p, num_sms, &bytes);
    most = std::max(most, bytes);
  };
  for (const int64_t rows : {8 * kGroups, 16 * kGroups, kTensorRows - 1}) with(rows);
  for (int64_t rows = kPrefixRowTile; rows < (a.T + a.N) * a.group; rows += kPrefixRowTile) with(rows);
  return most;
}

cudaError_t launch_attend(const AttendParams &a, int num_sms, cudaStream_t stream) {
  const AttendParams p = short_prefix(a);
  const AttendPlan L = make_plan(p, num_sms);
  const bool i8 = p.c.format == SV_CACHE_INT8;
  if (p.c.head_dim == 128) return i8 ? launch<128, SV_CACHE_INT8>(p, L, num_sms, stream) : launch<128, SV_CACHE_E4M3>(p, L, num_sms, stream);
  return i8 ? launch<64, SV_CACHE_INT8>(p, L, num_sms, stream) : launch<64, SV_CACHE_E4M3>(p, L, num_sms, stream);
}

}  // namespace sv
