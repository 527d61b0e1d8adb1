// sv_attend.cu -- attention of the verify tokens over the paged 8-bit cache:
// the warp-streaming kernel and the joining of its partial results.
//
// A request's rows for one kv head -- (gamma + 1) tokens times the query heads
// of the group -- are a tile of 16 or 32 rows that all read the same keys, so
// the private part is bound by HBM: 2 * head_dim + 8 bytes a key for 4 *
// head_dim * rows operations.  Each warp streams keys on its own, 32 at a
// time: lane l copies exactly the bytes that lane l will multiply into its own
// shared-memory places (cp.async, three tiles deep), so there is no barrier
// and no wait between warps in the loop.  That works because the order of the
// inner dimension of a product is free: lane (g, c) of a 16x8x16 product takes
// dimensions [c * D/4, (c + 1) * D/4) of key g, contiguous bytes, and the
// queries are laid out once in the same order; for the second product lane
// (g, c) takes dimensions [g * D/8, (g + 1) * D/8) of the keys whose weights it
// computed.  Bytes become f16 in registers (exact); sums are fp32.
//
// The key range of a row tile is cut over CTAs (and over a CTA's four warps)
// when there are few row tiles; the partial results (M, l, O) of a CTA go to
// the workspace and a second kernel joins them.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kStages = 3;
constexpr int kKeys = 32;  // keys of a warp's tile

template <int D>
struct Ring {
  static constexpr int kBytes = kKeys * 2 * D;       // keys, then values
  static constexpr int kScales = kBytes;             // then (key scale, value scale) of key `lane`
  static constexpr int kStage = kBytes + kKeys * 8;
};
template <int D, int MT>
constexpr size_t attend_smem() {
  return static_cast<size_t>(MT) * (D / 16) * 512 + static_cast<size_t>(kAttendWarps) * kStages * Ring<D>::kStage;
}

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(kAttendThreads, 2) attend_kernel(const AttendParams P, const AttendPlan L) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int row_token[MT * 16], row_limit[MT * 16];
  __shared__ uint32_t warp_top[kAttendWarps];
  __shared__ float row_m[kAttendWarps][MT * 16], row_l[kAttendWarps][MT * 16];
  constexpr int R = MT * 16;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int H = P.c.num_kv_heads;

  // ---- which rows and keys ----
  int h, k_begin, k_end, slot, r0, rows;
  int64_t first = 0;
  const int32_t *table = P.tables;
  uint32_t bits = 0;
  int len = 0, gam = 0;
  const bool shared_part = static_cast<int>(blockIdx.x) < L.prefix_items;
  if (shared_part) {
    int b = blockIdx.x;
    const int tile = b % L.prefix_tiles;
    b /= L.prefix_tiles;
    h = b % H;
    slot = b / H;
    r0 = tile * R;
    rows = min(R, L.rows - r0);
    k_begin = slot * L.prefix_chunk;
    k_end = min(P.prefix, k_begin + L.prefix_chunk);
  } else {
    int b = blockIdx.x - L.prefix_items;
    const int tile = b % L.own_tiles;
    b /= L.own_tiles;
    h = b % H;
    b /= H;
    const int split = b % L.own_splits;
    const int i = b / L.own_splits;
    const bool ok = attend_request(P, i, first, gam, len, bits);
    if (bits && tile == 0 && h == 0 && split == 0 && tid == 0 && P.status) atomicOr(P.status, static_cast<int>(bits));
    bits = 0;
    if (!ok) return;
    r0 = tile * R;
    rows = min(R, (gam + 1) * P.group - r0);
    if (rows <= 0) return;
    slot = L.prefix_splits + split;
    k_begin = P.prefix + split * L.own_chunk;
    k_end = min(len, k_begin + L.own_chunk);
    if (k_end <= k_begin && L.slots > 1) return;  // (the joining kernel knows)
    table += i * P.table_stride;
  }
  if (tid < R) {
    int token = -1, limit = 0x7FFFFFFF;
    if (tid < rows) {
      const int t = div_by(r0 + tid, L.group);
      if (shared_part) {
        token = t;
        limit = prefix_limit(P, t);
        if (limit < 0) {  // nobody's row
          token = -1;
          limit = 0x7FFFFFFF;
        }
      } else {
        token = static_cast<int>(first) + t;
        limit = len - gam + t;
      }
    }
    row_token[tid] = token;
    row_limit[tid] = limit;
  }
  __syncthreads();

  // ---- the queries as operand fragments ----
  constexpr int kFrags = MT * (D / 16) * 32 / kAttendThreads;  // of a thread
  uint4 *const qfrag = reinterpret_cast<uint4 *>(smem);
  float c_tile;
  {
    float x[kFrags][8];  // dimensions 0..3 of row g, then of row g + 8
    uint32_t top = 0;
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const int at = f * kAttendThreads + tid, ln = at & 31, kk = (at >> 5) % (D / 16), mt = (at >> 5) / (D / 16);
      const int dim = (ln & 3) * (D / 4) + 4 * kk;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + (ln >> 2);
        const int token = row_token[r];
        uint32_t w[2] = {0, 0};
        if (token >= 0) {
          const int lr = r0 + r, hq = h * P.group + lr - div_by(lr, L.group) * P.group;
          const uint16_t *src = P.q + token * P.q_token + hq * P.q_head + dim;
          if (L.qvec) {
            const uint2 v = *reinterpret_cast<const uint2 *>(src);
            w[0] = v.x;
            w[1] = v.y;
          } else {
            w[0] = src[0] | static_cast<uint32_t>(src[1]) << 16;
            w[1] = src[2] | static_cast<uint32_t>(src[3]) << 16;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = bf16_bits_to_float((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
          x[f][half * 4 + e] = v;
          const uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;
          if (a < 0x7F800000u) top = max(top, a);
        }
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) warp_top[warp] = top;
    __syncthreads();
    top = max(max(warp_top[0], warp_top[1]), max(warp_top[2], warp_top[3]));
    const int shift = query_shift(top);
    const float up = pow2(shift);
    c_tile = P.scale * kLog2e * pow2(-shift);
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
      const float *v = x[f];
      qfrag[f * kAttendThreads + tid] = make_uint4(pack_f16(v[0] * up, v[1] * up), pack_f16(v[4] * up, v[5] * up),
                                                   pack_f16(v[2] * up, v[3] * up), pack_f16(v[6] * up, v[7] * up));
    }
  }
  int limit[MT][2], low = 0x7FFFFFFF;  // low: keys below it are seen by every row of the tile
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      limit[mt][half] = row_limit[mt * 16 + half * 8 + g];
      low = min(low, limit[mt][half]);
    }
  low = __reduce_min_sync(0xFFFFFFFFu, low);
  __syncthreads();

  // ---- the stream of keys ----
  const uint32_t ring = smem_addr(smem) + MT * (D / 16) * 512 + warp * kStages * Ring<D>::kStage;
  const uint8_t *const ring_ptr = smem + MT * (D / 16) * 512 + warp * kStages * Ring<D>::kStage;
  const int tiles_all = (max(0, k_end - k_begin) + kKeys - 1) / kKeys;
  const int ntiles = (tiles_all - warp + kAttendWarps - 1) / kAttendWarps;  // tiles warp, warp + 4, ...
  auto page_of = [&](int it) {  // of the lane's key of the warp's tile `it`
    const int k = k_begin + (it * kAttendWarps + warp) * kKeys + lane;
    return it < ntiles && k < k_end ? table[div_by(k, L.page)] : -1;
  };
  auto issue = [&](int it, int page) {
    if (it < ntiles) {
      const int k = k_begin + (it * kAttendWarps + warp) * kKeys + lane;
      const bool in = k < k_end, live = in && page >= 0 && page < P.c.num_blocks;
      if (in && !live) bits = SV_DATA_BAD_SLOT;
      int64_t at = 0, sat = 0;
      if (live) {
        const int off = k - div_by(k, L.page) * P.c.block_size;
        at = page * P.c.block_stride + h * P.c.head_stride + off * P.c.token_stride;
        sat = page * P.c.scale_block_stride + h * P.c.scale_head_stride + off * P.c.scale_token_stride;
      }
      const uint32_t dst = ring + (it % kStages) * Ring<D>::kStage;
      copy_async<4>(dst + Ring<D>::kScales + lane * 8, P.c.k_scale + sat, live ? 4 : 0);
      copy_async<4>(dst + Ring<D>::kScales + lane * 8 + 4, P.c.v_scale + sat, live ? 4 : 0);
      const uint32_t unit = live ? static_cast<uint32_t>(at >> 4) : 0xFFFFFFFFu;  // (rows are 16-byte aligned)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const uint32_t u = __shfl_sync(0xFFFFFFFFu, unit, nt * 8 + g);
        const uint8_t *src = static_cast<const uint8_t *>(P.c.k) + (u == 0xFFFFFFFFu ? 0 : static_cast<int64_t>(u) * 16 + c * (D / 4));
#pragma unroll
        for (int q = 0; q < D / 64; ++q)
          copy_async<16>(dst + (nt * (D / 64) + q) * 512 + lane * 16, src + (u == 0xFFFFFFFFu ? 0 : q * 16), u == 0xFFFFFFFFu ? 0 : 16);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {  // keys 2c, 2c + 1, 2c + 8, 2c + 9 of each half of the tile
        const uint32_t u = __shfl_sync(0xFFFFFFFFu, unit, (x >> 2) * 16 + ((x >> 1) & 1) * 8 + 2 * c + (x & 1));
        const uint8_t *src = static_cast<const uint8_t *>(P.c.v) + (u == 0xFFFFFFFFu ? 0 : static_cast<int64_t>(u) * 16 + g * (D / 8));
        copy_async<D / 8>(dst + kKeys * D + x * (32 * D / 8) + lane * (D / 8), src, u == 0xFFFFFFFFu ? 0 : D / 8);
      }
    }
    copy_commit();
  };

  float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt][0] = m[mt][1] = -INFINITY;
    l[mt][0] = l[mt][1] = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.0f;
  }
  int page = page_of(0);
#pragma unroll
  for (int it = 0; it < kStages - 1; ++it) {
    issue(it, page);
    page = page_of(it + 1);
  }
  for (int it = 0; it < ntiles; ++it) {
    copy_wait<kStages - 2>();
    const uint8_t *const src = ring_ptr + (it % kStages) * Ring<D>::kStage;
    const float2 sc = *reinterpret_cast<const float2 *>(src + Ring<D>::kScales + lane * 8);
    float kc = sc.x * c_tile, lv, inv;
    value_scale_terms(sc.y, kc, lv, inv);
    // scores
    float s[MT][4][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
      uint4 kb[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) kb[nt] = *reinterpret_cast<const uint4 *>(src + (nt * (D / 64) + q) * 512 + lane * 16);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint4 a[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) a[mt] = qfrag[(mt * (D / 16) + q * 4 + x) * 32 + lane];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint32_t w = x == 0 ? kb[nt].x : x == 1 ? kb[nt].y : x == 2 ? kb[nt].z : kb[nt].w;
          uint32_t b0, b1;
          bytes_to_f16<FMT>(w, b0, b1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma_16816(s[mt][nt], a[mt], b0, b1);
        }
      }
    }
    // weights
    float vw[4][2], iv[4][2];  // of the lane's keys: log2 and reciprocal of the value scale
    const int k0 = k_begin + (it * kAttendWarps + warp) * kKeys;
    const bool cut = k0 + kKeys > low;
    {
      float top[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) top[mt][0] = top[mt][1] = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = nt * 8 + 2 * c + e;
          const float kce = __shfl_sync(0xFFFFFFFFu, kc, key);
          vw[nt][e] = __shfl_sync(0xFFFFFFFFu, lv, key);
          iv[nt][e] = __shfl_sync(0xFFFFFFFFu, inv, key);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // (a product of its own, rounded: subtracting a maximum that equals it gives 0)
              float x = __fmul_rn(s[mt][nt][half * 2 + e], kce);
              if (cut && k0 + key >= limit[mt][half]) x = -INFINITY;
              s[mt][nt][half * 2 + e] = x;
              top[mt][half] = fmaxf(top[mt][half], x + vw[nt][e]);
            }
        }
      bool grew = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float t = top[mt][half];
          t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
          top[mt][half] = fmaxf(t, m[mt][half]);
          grew |= top[mt][half] != m[mt][half];
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {  // (seldom after the first tiles)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float r = m[mt][half] == -INFINITY ? 0.0f : exp2_approx(m[mt][half] - top[mt][half]);
            m[mt][half] = top[mt][half];
            l[mt][half] *= r;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[mt][n][half * 2] *= r;
              o[mt][n][half * 2 + 1] *= r;
            }
          }
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float base = m[mt][half] == -INFINITY ? 0.0f : m[mt][half];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (the score less the maximum first: a score too large to hold the value scale's log keeps it here)
            float w = exp2_approx((s[mt][nt][half * 2 + e] - base) + vw[nt][e]);
            s[mt][nt][half * 2 + e] = w;
            l[mt][half] = fmaf(w, iv[nt][e], l[mt][half]);
          }
      }
    // values
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 a[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float *x = s[mt][half * 2], *y = s[mt][half * 2 + 1];
        a[mt] = make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(y[0], y[1]), pack_f16(y[2], y[3]));
      }
      const uint8_t *vs = src + kKeys * D + half * 4 * (32 * D / 8) + lane * (D / 8);
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {  // eight dimensions of the four keys at a time
        uint2 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = *reinterpret_cast<const uint2 *>(vs + x * (32 * D / 8) + q * 8);
#pragma unroll
        for (int wd = 0; wd < 2; ++wd) {
          const uint32_t v0 = wd ? v[0].y : v[0].x, v1 = wd ? v[1].y : v[1].x, v2 = wd ? v[2].y : v[2].x,
                         v3 = wd ? v[3].y : v[3].x;
          uint32_t b0[4], b1[4];  // (key pair, dimension)
          bytes_to_f16<FMT>(__byte_perm(v0, v1, 0x5140), b0[0], b0[1]);
          bytes_to_f16<FMT>(__byte_perm(v0, v1, 0x7362), b0[2], b0[3]);
          bytes_to_f16<FMT>(__byte_perm(v2, v3, 0x5140), b1[0], b1[1]);
          bytes_to_f16<FMT>(__byte_perm(v2, v3, 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_16816(o[mt][q * 8 + wd * 4 + d], a[mt], b0[d], b1[d]);
        }
      }
    }
    issue(it + kStages - 1, page);
    page = page_of(it + kStages);
  }
  copy_wait<0>();
  if (bits && P.status) atomicOr(P.status, static_cast<int>(bits));

  // ---- the four warps' results joined ----
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x = l[mt][half];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
      if (c == 0) {
        row_m[warp][mt * 16 + half * 8 + g] = m[mt][half];
        row_l[warp][mt * 16 + half * 8 + g] = x;
      }
    }
  __syncthreads();  // (every warp is done with its ring as well)
  float *const acc = reinterpret_cast<float *>(smem);  // [warp][row][D]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = mt * 16 + half * 8 + g;
      const float top = fmaxf(fmaxf(row_m[0][r], row_m[1][r]), fmaxf(row_m[2][r], row_m[3][r]));
      const float f = m[mt][half] == -INFINITY ? (isnan(row_l[warp][r]) ? 1.0f : 0.0f) : exp2_approx(m[mt][half] - top);
      // column n of a product's tile t is dimension n * D/8 + t
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < D / 8; n += 4)
          *reinterpret_cast<float4 *>(acc + (warp * R + r) * D + (2 * c + e) * (D / 8) + n) =
              make_float4(o[mt][n][half * 2 + e] * f, o[mt][n + 1][half * 2 + e] * f, o[mt][n + 2][half * 2 + e] * f,
                          o[mt][n + 3][half * 2 + e] * f);
    }
  __syncthreads();
  for (int r = warp; r < rows; r += kAttendWarps) {
    const int token = row_token[r];
    if (token < 0) continue;
    const int lr = r0 + r, hq = h * P.group + lr - div_by(lr, L.group) * P.group;
    const float top = fmaxf(fmaxf(row_m[0][r], row_m[1][r]), fmaxf(row_m[2][r], row_m[3][r]));
    float sum = 0.0f, x[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) x[d] = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttendWarps; ++w) {
      sum += row_m[w][r] == -INFINITY ? (isnan(row_l[w][r]) ? row_l[w][r] : 0.0f) : row_l[w][r] * exp2_approx(row_m[w][r] - top);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) x[d] += acc[(w * R + r) * D + d * 32 + lane];
    }
    const int64_t row = static_cast<int64_t>(token) * P.Hq + hq;
    if (L.slots > 1) {
      float *dst = L.part_o + (row * L.slots + slot) * D;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) dst[d * 32 + lane] = x[d];
      if (lane == 0) L.part_ml[row * L.slots + slot] = make_float2(top, sum);
    } else {
      uint16_t *dst = P.out + token * P.out_token + hq * P.out_head;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) dst[d * 32 + lane] = static_cast<uint16_t>(pack_bf16(sum == 0.0f ? 0.0f : x[d] * inv, 0.0f));
      if (P.lse && lane == 0) P.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
}

// Joins the partial results of a row: one warp a row.  With M the largest of
// the slots' M_s, out = sum 2^(M_s - M) O_s / sum 2^(M_s - M) l_s.
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
  const int slots = L.prefix_splits + own;
  const int rows = (g + 1) * P.Hq;
  for (int r = blockIdx.y * kWarps + warp; r < rows; r += gridDim.y * kWarps) {
    const int j = r / P.Hq, hq = r % P.Hq;
    const int64_t row = (first + j) * P.Hq + hq;
    const float2 *ml = L.part_ml + row * L.slots;
    float top = -INFINITY;
    bool nan = false;
    for (int s = lane; s < slots; s += 32) {
      const float2 v = ml[s];
      top = fmaxf(top, v.x);
      nan |= isnan(v.y);
    }
    for (int b = 16; b; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, b));
    nan = __any_sync(0xFFFFFFFFu, nan);
    float sum = 0.0f, x[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) x[d] = 0.0f;
    for (int s = 0; s < slots; ++s) {
      const float2 v = ml[s];
      if (v.x == -INFINITY) continue;  // (warp-uniform)
      const float f = exp2_approx(v.x - top);
      sum = fmaf(v.y, f, sum);
      const float *src = L.part_o + (row * L.slots + s) * D;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) x[d] = fmaf(src[d * 32 + lane], f, x[d]);
    }
    if (nan) sum = __uint_as_float(0x7FC00000u);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *dst = P.out + (first + j) * P.out_token + hq * P.out_head;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) dst[d * 32 + lane] = static_cast<uint16_t>(pack_bf16(sum == 0.0f ? 0.0f : x[d] * inv, 0.0f));
    if (P.lse && lane == 0) P.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

constexpr int kChunkStep = kAttendWarps * kKeys;  // a CTA's four warps take 32 keys each
constexpr int kChunkMost = 2048;                  // so that the longest request is no long tail

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

AttendPlan make_plan(const AttendParams &p, int num_sms, int64_t *bytes = nullptr) {
  AttendPlan L{};
  L.page = fast_div(std::max(1, p.c.block_size));
  L.group = fast_div(p.group);
  L.rows = static_cast<int32_t>((p.T + p.N) * p.group);
  const int most = (p.G + 1) * p.group, R = most <= 16 && !p.prefix ? 16 : 32;
  L.own_tiles = ceil_div(most, R);
  L.prefix_tiles = ceil_div(L.rows, R);
  // (at least one private chunk, though no request may have private keys: its CTAs look at the requests' ranges)
  int bound = std::max(1, cut(static_cast<int64_t>(p.N) * p.c.num_kv_heads * L.own_tiles, p.max_seq - p.prefix, num_sms,
                              L.own_splits, L.own_chunk));
  L.own_splits = std::max(1, L.own_splits);
  bound += cut(static_cast<int64_t>(p.c.num_kv_heads) * L.prefix_tiles, p.prefix, num_sms, L.prefix_splits,
               L.prefix_chunk);
  L.prefix_items = L.prefix_tiles * p.c.num_kv_heads * L.prefix_splits;
  L.slots = L.prefix_splits + L.own_splits;
  L.qvec = (reinterpret_cast<uintptr_t>(p.q) & 7u) == 0 && p.q_token % 4 == 0 && p.q_head % 4 == 0;
  const int64_t rows = static_cast<int64_t>(L.rows) * p.c.num_kv_heads;
  if (bytes) *bytes = bound <= 1 ? 0 : ((rows * bound * 8 + 15) & ~int64_t{15}) + rows * bound * p.c.head_dim * 4;
  L.part_ml = static_cast<float2 *>(p.workspace);
  L.part_o = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + ((rows * L.slots * 8 + 15) & ~int64_t{15}));
  return L;
}

template <int D, int FMT, int MT>
cudaError_t launch(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const int64_t own = static_cast<int64_t>(p.N) * p.c.num_kv_heads * L.own_tiles * L.own_splits;
  if (own + L.prefix_items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(own + L.prefix_items));
  cfg.blockDim = dim3(kAttendThreads);
  cfg.dynamicSmemBytes = attend_smem<D, MT>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  cudaError_t e = cudaLaunchKernelEx(&cfg, attend_kernel<D, FMT, MT>, p, L);
  if (e != cudaSuccess || L.slots == 1) return e;
  cfg.gridDim = dim3(p.N, std::max(1, std::min(65535, ceil_div((p.G + 1) * static_cast<int64_t>(p.Hq), kWarps))));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, L);
}

template <int D, int FMT>
cudaError_t pick(const AttendParams &p, const AttendPlan &L, cudaStream_t s) {
  return (p.G + 1) * p.group <= 16 && !p.prefix ? launch<D, FMT, 1>(p, L, s) : launch<D, FMT, 2>(p, L, s);
}

template <int D, int FMT, int MT>
cudaError_t enable() {
  return cudaFuncSetAttribute(attend_kernel<D, FMT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(attend_smem<D, MT>()));
}

}  // namespace

cudaError_t enable_attend_kernels() {
  cudaError_t e;
  if ((e = enable<128, SV_CACHE_INT8, 1>()) != cudaSuccess || (e = enable<128, SV_CACHE_INT8, 2>()) != cudaSuccess ||
      (e = enable<128, SV_CACHE_E4M3, 1>()) != cudaSuccess || (e = enable<128, SV_CACHE_E4M3, 2>()) != cudaSuccess ||
      (e = enable<64, SV_CACHE_INT8, 1>()) != cudaSuccess || (e = enable<64, SV_CACHE_INT8, 2>()) != cudaSuccess ||
      (e = enable<64, SV_CACHE_E4M3, 1>()) != cudaSuccess)
    return e;
  return enable<64, SV_CACHE_E4M3, 2>();
}

int64_t attend_workspace_bytes(const AttendParams &p, int num_sms) {
  int64_t bytes = 0;
  make_plan(p, num_sms, &bytes);
  return bytes;
}

cudaError_t launch_attend(const AttendParams &p, int num_sms, cudaStream_t stream) {
  const AttendPlan L = make_plan(p, num_sms);
  const bool i8 = p.c.format == SV_CACHE_INT8;
  if (p.c.head_dim == 128) return i8 ? pick<128, SV_CACHE_INT8>(p, L, stream) : pick<128, SV_CACHE_E4M3>(p, L, stream);
  return i8 ? pick<64, SV_CACHE_INT8>(p, L, stream) : pick<64, SV_CACHE_E4M3>(p, L, stream);
}

}  // namespace sv
