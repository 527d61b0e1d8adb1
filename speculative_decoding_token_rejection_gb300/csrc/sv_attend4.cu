// sv_attend4.cu -- the private part of the verify tokens' attention over the
// paged 4-bit cache, on the tensor cores' own memory (tcgen05).
//
// A request's rows for one kv head all read the same keys: the part is bound by
// HBM (152 bytes a key for head_dim 128) as long as unpacking a key costs little
// and is done once for all of its rows.  Both products are transposed, keys and
// dimensions on the 128-wide side of the instruction, the few rows on the narrow
// one: S^T [keys x rows] = K Q^T and O^T [dims x rows] += V^T P^T.  A thread takes
// a key, from its bytes to its weights:
//
//   K row    global -> registers -> f16 -> tensor memory (A of the first product)
//   V row    global -> registers -> f16 -> shared memory (A of the second, which
//            wants dimensions outside: 64 of them a 128-byte line per key)
//   scores   tensor memory -> registers: all rows of the thread's key
//   weights  registers -> shared memory (B of the second product)
//
// so no byte is exchanged between threads, and one thread issues the products,
// which run while all unpack: V during the first, the next tile's K during the
// second.  A tile is 128 keys, its bytes are loaded a tile ahead.
//
// Numbers, as in the kernel for the shared prefix: x = (q . n) * (scale * log2 e *
// key_scale), w = 2^(x - m), l = sum w, P = w * value_scale / W, O = W * sum P n_v.
// Any m gives the same quotient O / l; a row's is raised to the largest x +
// log2(value_scale / W) when that passes it by 8, so P stays below 2^8 in f16, and
// W = 2^28 is the middle of the scales that the writer gives.  l takes the
// unrounded weights in fp32.  m is kept as two numbers, a largest x and what the
// value scales add to it: beside a score of 2^28 or more the sum would lose the
// latter, and the weights their place in f16.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_attend.cuh"
#include "sv_cache4.cuh"
#include "sv_tensor.cuh"

namespace sv {
namespace {

constexpr int kOwnThreads = 128, kOwnKeys = 128;  // a thread a key
constexpr float kRaise = 8;
constexpr float kScaleUnit = 0x1p28f;           // W
constexpr float kLeastUnits = kLeastLog2 - 28;  // log2 of the size that a scale counts as at least, in W

struct OwnControl {
  uint64_t s_full, o_full;
  uint32_t tmem, abort;
  uint32_t huge;                       // some |m| is so large that its two parts are subtracted one after the other
  alignas(16) float neg[kOwnRows4];    // negated m, 0 without one
  alignas(16) float negx[kOwnRows4], negu[kOwnRows4];  // its parts, negated
  alignas(16) float back[kOwnRows4];   // what undoes a row's power of two
  alignas(16) int limit[kOwnRows4];    // keys that the row sees are below it
  alignas(16) float factor[kOwnRows4]; // of a raised maximum; at the end, of the outputs
  float mx[kOwnRows4], mu[kOwnRows4];  // m = mx + mu, mx -inf without one
  float part[kOwnThreads / 32][kOwnRows4];
  uint32_t none[kOwnRows4];            // the row sees a value scale that is no number
};

// Shared memory: [D / 64][128 keys][128 bytes] of V, [128 keys][128 bytes] of weights (up to 64 rows), [D / 64][NMAX
// rows][128 bytes] of queries.  16-byte columns of a line are exchanged by line % 8.
template <int D, int NMAX>
struct OwnSmem {
  static constexpr int kLines = kOwnKeys * 128;
  static constexpr int kV = 0, kP = D / 64 * kLines, kQ = kP + kLines, kControl = kQ + D / 64 * NMAX * 128,
                       kBytes = kControl + static_cast<int>(sizeof(OwnControl)) + 1024;  // (the base is rounded up to 1 KB)
};
__device__ __forceinline__ int line_at(int line, int col) { return line * 128 + ((col ^ (line & 7)) << 4); }

__device__ __forceinline__ void tmem_store_row(uint32_t addr, const uint32_t r[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32"
      "};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Sixteen columns of the thread's lane.
__device__ __forceinline__ void tmem_load_row(uint32_t addr, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
      "}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_16(uint32_t addr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
      "};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Eight values of every lane combined over the warp, in nine exchanges: lane 4i
// gets that of value i.
template <bool MAX>
__device__ __forceinline__ float reduce_eight(float v[8], int lane) {
  const auto both = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int n = 4; n; n >>= 1) {
    const bool upper = lane & n * 4;
#pragma unroll
    for (int i = 0; i < n; ++i)
      v[i] = both(upper ? v[i + n] : v[i], __shfl_xor_sync(0xFFFFFFFFu, upper ? v[i] : v[i + n], n * 4));
  }
  v[0] = both(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 2));
  return both(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

// A cache row on its way: nibbles, group scales, the row's scale.
template <int D>
struct RawRow {
  uint32_t w[D / 8], g[D / 64];
  float scale;
};
template <int D>
__device__ __forceinline__ void load_row(RawRow<D> &r, const uint8_t *data, const uint8_t *group, const float *scale) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) ld_stream_32(data + 32 * i, r.w + 8 * i);
  if (D == 128) {
    const uint2 g = __ldg(reinterpret_cast<const uint2 *>(group));
    r.g[0] = g.x;
    r.g[D / 64 - 1] = g.y;
  } else {
    r.g[0] = __ldg(reinterpret_cast<const uint32_t *>(group));
  }
  r.scale = __ldg(scale);
}
template <int D>
__device__ __forceinline__ void zero_row(RawRow<D> &r) {
#pragma unroll
  for (int i = 0; i < D / 8; ++i) r.w[i] = 0;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) r.g[i] = 0;
  r.scale = 0.0f;
}
// Group j of a row as f16 pairs, in the order of mixed_place.
template <int D, int FMT>
__device__ __forceinline__ void unpack_group(const RawRow<D> &r, int j, uint32_t h[8]) {
  group_to_f16_mixed<FMT>(make_uint2(r.w[2 * j], r.w[2 * j + 1]), group_factors<FMT>(r.g[j >> 2] >> (8 * (j & 3)) & 0xFFu), h);
}

template <int D, int FMT, int NMAX>
__global__ void __launch_bounds__(kOwnThreads, NMAX <= 32 ? 3 : 2)
    own4_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ AttendPlan L) {
  pdl_enter();
  OwnTile T;
  if (!own_tile(P, L, blockIdx.x, NMAX, T)) return;
  extern __shared__ uint8_t raw[];
  uint8_t *const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  using Y = OwnSmem<D, NMAX>;
  OwnControl &C = *reinterpret_cast<OwnControl *>(smem + Y::kControl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr uint32_t kS = 64, kO = 64 + NMAX, kCols = NMAX <= 32 ? 128 : 256;  // columns of tensor memory: K, S, O
  const int n16 = (T.rows + 15) / 16, n8 = (T.rows + 7) / 8;

  // ---- the first tile's bytes are on their way before anything else ----
  const int ntiles = (max(0, T.k_end - T.k_begin) + kOwnKeys - 1) / kOwnKeys;
  const int32_t *const table = P.tables + T.i * P.table_stride;
  const uint8_t *const kdata = static_cast<const uint8_t *>(P.c.k) + T.h * P.c.head_stride;
  const uint8_t *const vdata = static_cast<const uint8_t *>(P.c.v) + T.h * P.c.head_stride;
  const uint8_t *const kgroup = P.k_group + T.h * P.group_head, *const vgroup = P.v_group + T.h * P.group_head;
  const float *const kscale = P.c.k_scale + T.h * P.c.scale_head_stride;
  const float *const vscale = P.c.v_scale + T.h * P.c.scale_head_stride;
  uint32_t bits = 0;
  auto page_of = [&](int it) {  // of the thread's key of tile `it`
    const int k = T.k_begin + it * kOwnKeys + tid;
    return k < T.k_end ? (k < P.row0 ? P.tables : table)[div_by(k, L.page)] : -1;
  };
  RawRow<D> kraw, vraw;
  int64_t at_data = 0, at_group = 0, at_scale = 0;
  bool live = false;  // of the key whose bytes are in kraw and vraw (or on their way)
  auto place = [&](int it, int page) {
    const int k = T.k_begin + it * kOwnKeys + tid, off = k - div_by(k, L.page) * P.c.block_size;
    live = k < T.k_end && page >= 0 && page < P.c.num_blocks;
    if (k < T.k_end && !live) bits = SV_DATA_BAD_SLOT;
    at_data = page * P.c.block_stride + off * P.c.token_stride;
    at_group = page * P.group_block + off * P.group_token;
    at_scale = page * P.c.scale_block_stride + off * P.c.scale_token_stride;
  };
  auto load_keys = [&]() {
    if (live)
      load_row<D>(kraw, kdata + at_data, kgroup + at_group, kscale + at_scale);
    else
      zero_row<D>(kraw);
  };
  auto load_values = [&]() {
    if (live)
      load_row<D>(vraw, vdata + at_data, vgroup + at_group, vscale + at_scale);
    else
      zero_row<D>(vraw);
  };
  place(0, page_of(0));
  load_keys();
  load_values();
  int page = page_of(1);

  if (tid == 0) {
    mbar_init(&C.s_full, 1);
    mbar_init(&C.o_full, 1);
    C.abort = C.huge = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&C.tmem, kCols);
  if (tid < kOwnRows4) {
    const int j = div_by(T.r0 + tid, L.group);
    C.limit[tid] = tid < T.rows ? T.len - T.gam + j : 0x7FFFFFFF;
    C.neg[tid] = C.negx[tid] = C.negu[tid] = C.mu[tid] = 0.0f;
    C.mx[tid] = -INFINITY;
    C.none[tid] = 0;
  }
  // ---- the queries: f16, each row with its own power of two, dimensions in the order of the unpacked keys ----
  bool shifted = false;
  {
    constexpr int kCh = D / 8, kRowsPass = kOwnThreads / kCh, kPass = NMAX / kRowsPass;
    const int col = tid % kCh;
    uint4 x[kPass];
#pragma unroll
    for (int f = 0; f < kPass; ++f) {
      const int r = f * kRowsPass + tid / kCh, lr = T.r0 + r, j = div_by(lr, L.group);
      x[f] = make_uint4(0, 0, 0, 0);
      if (r < T.rows) {
        const uint16_t *src = P.q + (T.first + j) * P.q_token + (T.h * P.group + lr - j * P.group) * P.q_head + col * 8;
        if (L.qvec)
          x[f] = *reinterpret_cast<const uint4 *>(src);
        else
          x[f] = make_uint4(src[0] | static_cast<uint32_t>(src[1]) << 16, src[2] | static_cast<uint32_t>(src[3]) << 16,
                            src[4] | static_cast<uint32_t>(src[5]) << 16, src[6] | static_cast<uint32_t>(src[7]) << 16);
      }
    }
#pragma unroll
    for (int f = 0; f < kPass; ++f) {
      const int r = f * kRowsPass + tid / kCh;
      uint32_t w[4] = {x[f].x, x[f].y, x[f].z, x[f].w}, top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = w[e] << 16 & 0x7FFFFFFFu, b = w[e] & 0x7FFF0000u;
        if (a < 0x7F800000u) top = max(top, a);
        if (b < 0x7F800000u) top = max(top, b);
      }
#pragma unroll
      for (int b = kCh / 2; b; b >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, b));
      const int shift = query_shift(top);
      shifted |= shift != 0;
      if (col == 0) C.back[r] = pow2(-shift);
      const float up = pow2(shift);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_f16(bf16_bits_to_float(w[e] & 0xFFFFu) * up, bf16_bits_to_float(w[e] >> 16) * up);
      if (mixed<FMT>()) {  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
        const uint32_t a = __byte_perm(w[0], w[2], 0x5410), b = __byte_perm(w[0], w[2], 0x7632);
        const uint32_t c = __byte_perm(w[1], w[3], 0x5410), d = __byte_perm(w[1], w[3], 0x7632);
        w[0] = a;
        w[1] = b;
        w[2] = c;
        w[3] = d;
      }
      *reinterpret_cast<uint4 *>(smem + Y::kQ + (col >> 3) * (NMAX * 128) + line_at(r, col & 7)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_smem();
  fence_before();
  shifted = __syncthreads_or(shifted);
  fence_after();
  int low = 0x7FFFFFFF;  // keys below it are seen by every row
  for (int r = lane; r < T.rows; r += 32) low = min(low, C.limit[r]);
  low = __reduce_min_sync(0xFFFFFFFFu, low);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, C.tmem, 0), base = smem_addr(smem);
  const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);  // the warp's lanes
  const bool leader = warp == 0 && elected();
  const uint32_t scores = product(n16 * 16, false), outputs = product(n16 * 16, true, D, true);
  const uint64_t queries = operand(base + Y::kQ, 16), values = operand(base + Y::kV, Y::kLines),
                 weights = operand(base + Y::kP, Y::kLines);

  float l[NMAX];  // sums over the thread's keys
#pragma unroll
  for (int r = 0; r < NMAX; ++r) l[r] = 0.0f;
  const float c_all = P.scale * unit4<FMT>() * kLog2e;
  bool force = true;  // some row has no maximum
  bool ok = true;
  int it = 0;
  for (; it < ntiles; ++it) {
    // ---- the tile's keys to tensor memory; scores ----
    const float kc = kraw.scale * c_all;
    const bool dead = !live;
    const int key = T.k_begin + it * kOwnKeys + tid;
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      uint32_t h[32];
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack_group<D, FMT>(kraw, half * 4 + j, h + 8 * j);
      tmem_store_row(mine + half * 32, h);
    }
    tmem_wait_store();
    fence_before();
    __syncthreads();
    if (leader) {
      fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t b = queries + static_cast<uint64_t>((kk >> 2) * (NMAX * 128 >> 4) + (kk & 3) * 2);
        if (kk == 0)
          mma_ts<false>(tmem + kS, tmem, b, scores);
        else
          mma_ts<true>(tmem + kS, tmem + kk * 8, b, scores);
      }
      mma_commit(&C.s_full);
    }
    __syncwarp();
    const bool more = it + 1 < ntiles;
    // (vraw is still this tile's: its place is taken over below)
    const float vs = vraw.scale;
    if (more) place(it + 1, page);
    if (more) load_keys();
    page = page_of(it + 2);
    // ---- the values to shared memory, once the products of the tile before are done with it ----
    if (it > 0) ok = wait(C, &C.o_full, (it - 1) & 1);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t h[8];
      unpack_group<D, FMT>(vraw, j, h);
      uint8_t *const dst = smem + Y::kV + (j >> 2) * Y::kLines;
      *reinterpret_cast<uint4 *>(dst + line_at(tid, (2 * j) & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4 *>(dst + line_at(tid, (2 * j + 1) & 7)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
    if (more) load_values();
    // ---- weights ----
    const bool number = fabsf(vs) < INFINITY;
    const float vr = number && fabsf(vs) >= kLeastScale ? vs * (1.0f / kScaleUnit) : 0.0f;
    const float lv = fmaxf(__log2f(fabsf(vr)), kLeastUnits);
    const bool cut = T.k_begin + (it + 1) * kOwnKeys > low || __any_sync(0xFFFFFFFFu, dead);
    if (!number) {
      for (int r = 0; r < T.rows; ++r)
        if (key < C.limit[r]) C.none[r] = 1;
    }
    float x[NMAX];
    auto load_scores = [&]() {  // a product of its own, rounded: subtracting a maximum that equals it gives 0
#pragma unroll
      for (int c = 0; c < NMAX / 16; ++c)
        if (c < n16) tmem_load_row(mine + kS + c * 16, reinterpret_cast<uint32_t *>(x) + c * 16);
#pragma unroll
      for (int c = 0; c < NMAX / 16; ++c)
        if (c < n16) tmem_wait_load(reinterpret_cast<uint32_t *>(x) + c * 16);
#pragma unroll
      for (int c = 0; c < NMAX / 8; ++c)
        if (c < n8) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const Pair y = mul2(pair(x[c * 8 + e], x[c * 8 + e + 1]), pair(kc, kc));
            x[c * 8 + e] = lo(y);
            x[c * 8 + e + 1] = hi(y);
          }
          if (shifted) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c * 8 + e] *= C.back[c * 8 + e];
          }
          if (cut) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (dead || key >= C.limit[c * 8 + e]) x[c * 8 + e] = -INFINITY;
          }
        }
    };
    ok = wait(C, &C.s_full, it & 1, P.expire) && ok;
    fence_after();
    load_scores();
    auto subtract = [&]() {
      float top = -INFINITY;
      if (C.huge) {
#pragma unroll
        for (int c = 0; c < NMAX / 8; ++c)
          if (c < n8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c * 8 + e] = x[c * 8 + e] + C.negx[c * 8 + e];
          }
      }
      const float *const last = C.huge ? C.negu : C.neg;
#pragma unroll
      for (int c = 0; c < NMAX / 8; ++c)
        if (c < n8) {
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(last + c * 8 + e);
            const Pair a = add2(pair(x[c * 8 + e], x[c * 8 + e + 1]), pair(m.x, m.y));
            const Pair b = add2(pair(x[c * 8 + e + 2], x[c * 8 + e + 3]), pair(m.z, m.w));
            x[c * 8 + e] = lo(a);
            x[c * 8 + e + 1] = hi(a);
            x[c * 8 + e + 2] = lo(b);
            x[c * 8 + e + 3] = hi(b);
            top = fmaxf(fmaxf(top, fmaxf(lo(a), hi(a))), fmaxf(lo(b), hi(b)));
          }
        }
      return top;
    };
    const bool raise = subtract() + lv > kRaise;
    if (__syncthreads_or(raise || force || !ok)) {  // (seldom after the first tile)
      // (whoever gave up did so before the barrier, and nobody waits before the next one)
      if (gave_up(C)) break;
      load_scores();
      // a row's largest x, then the largest of x less that with the value's scale
      auto largest = [&](bool scaled) {
#pragma unroll
        for (int c = 0; c < NMAX / 8; ++c)
          if (c < n8) {
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = scaled ? (x[c * 8 + e] + C.negx[c * 8 + e]) + lv : x[c * 8 + e];
            const float most = reduce_eight<true>(t, lane);
            if ((lane & 3) == 0) C.part[warp][c * 8 + (lane >> 2)] = most;
          }
        __syncthreads();
        return tid < n8 * 8 ? fmaxf(fmaxf(C.part[0][tid], C.part[1][tid]), fmaxf(C.part[2][tid], C.part[3][tid])) : 0.0f;
      };
      const float top_x = largest(false);
      float mx = 0.0f;
      if (tid < n8 * 8) {
        mx = fmaxf(C.mx[tid], top_x);
        C.negx[tid] = mx == -INFINITY ? 0.0f : -mx;
      }
      __syncthreads();
      const float top_u = largest(true);
      bool unset = false;
      if (tid < n8 * 8) {
        const bool had = C.mx[tid] != -INFINITY;
        const float old = had ? (C.mx[tid] - mx) + C.mu[tid] : 0.0f;  // of the sums so far, less mx
        if (!had || top_u > old + kRaise) {
          C.factor[tid] = had ? exp2_approx(old - top_u) : 1.0f;  // (without a maximum O and l are zeros or NaN)
          C.mx[tid] = mx;
          C.mu[tid] = mx == -INFINITY ? 0.0f : top_u;
        } else {
          C.factor[tid] = 1.0f;
        }
        unset = C.mx[tid] == -INFINITY;
        C.negx[tid] = unset ? 0.0f : -C.mx[tid];
        C.negu[tid] = -C.mu[tid];
        C.neg[tid] = C.negx[tid] + C.negu[tid];
        if (fabsf(C.negx[tid]) >= 1048576.0f) C.huge = 1;
      }
      force = __syncthreads_or(unset);
#pragma unroll
      for (int r = 0; r < NMAX; ++r)
        if ((r >> 3) < n8) l[r] *= C.factor[r];
      if (it > 0) {
#pragma unroll
        for (int c = 0; c < NMAX / 16; ++c)
          if (c < n16) {
            uint32_t o[16];
            tmem_load_row(mine + kO + c * 16, o);
            tmem_wait_load(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * C.factor[c * 16 + e]);
            tmem_store_16(mine + kO + c * 16, o);
          }
        tmem_wait_store();
      }
      subtract();
    }
#pragma unroll
    for (int c = 0; c < NMAX / 8; ++c)
      if (c < n8) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const Pair w = pair(exp2_approx(x[c * 8 + e]), exp2_approx(x[c * 8 + e + 1]));
          const Pair s = add2(pair(l[c * 8 + e], l[c * 8 + e + 1]), w), v = mul2(w, pair(vr, vr));
          l[c * 8 + e] = lo(s);
          l[c * 8 + e + 1] = hi(s);
          p[e >> 1] = pack_f16(lo(v), hi(v));
        }
        *reinterpret_cast<uint4 *>(smem + Y::kP + line_at(tid, c)) = make_uint4(p[0], p[1], p[2], p[3]);
      }
    // ---- outputs ----
    fence_proxy_async_smem();
    fence_before();
    __syncthreads();
    if (leader) {
      fence_after();
#pragma unroll
      for (int kk = 0; kk < kOwnKeys / 16; ++kk) {
        const uint64_t step = static_cast<uint64_t>(kk * (2048 >> 4));
        if (kk == 0 && it == 0)
          mma_ss<false>(tmem + kO, values, weights, outputs);
        else
          mma_ss<true>(tmem + kO, values + step, weights + step, outputs);
      }
      mma_commit(&C.o_full);
    }
    __syncwarp();
  }
  // ---- what is in flight ends; sums over the threads ----
  if (ntiles > 0) {
    settle(C, &C.s_full, min(it, ntiles - 1) & 1);
    if (it > 0) settle(C, &C.o_full, (it - 1) & 1);
    fence_after();
  }
#pragma unroll
  for (int c = 0; c < NMAX / 8; ++c)
    if (c < n8) {
      const float sum = reduce_eight<false>(l + c * 8, lane);
      if ((lane & 3) == 0) C.part[warp][c * 8 + (lane >> 2)] = sum;
    }
  __syncthreads();
  const bool lost = gave_up(C);
  const float nan = __uint_as_float(0x7FC00000u);
  if (tid < T.rows) {
    const int lr = T.r0 + tid, j = div_by(lr, L.group), hq = T.h * P.group + lr - j * P.group;
    const float m = lost ? -INFINITY : C.mx[tid] + C.mu[tid];
    const float sum = lost ? nan : (C.part[0][tid] + C.part[1][tid]) + (C.part[2][tid] + C.part[3][tid]);
    const int64_t row = (T.first + j) * P.Hq + hq;
    if (T.whole) {
      if (P.lse) P.lse[row] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
    } else {
      L.part_ml[row * L.slots + L.prefix_splits + T.split] = make_float2(m, sum);
    }
    // (a row without keys that count has the output 0.  Some w was 2^-log2(value_scale / W) at least, so sum is above
    // 2^-101 otherwise, and far below 2^126.)
    C.factor[tid] = lost || C.none[tid] ? nan : !T.whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  __syncthreads();
  // a lane holds a dimension: lane i of the tensor memory for head_dim 128, for 64 the first half of each warp's
  const int at = D == 128 ? tid : warp * 16 + (lane & 15);
  const int dim = mixed<FMT>() ? mixed_place(at) : at;
#pragma unroll
  for (int c = 0; c < NMAX / 16; ++c)
    if (c < n16) {
      uint32_t o[16];
      if (it > 0) {
        tmem_load_row(mine + kO + c * 16, o);
        tmem_wait_load(o);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = c * 16 + e;
        if (r < T.rows && (D == 128 || lane < 16)) {
          const int lr = T.r0 + r, j = div_by(lr, L.group), hq = T.h * P.group + lr - j * P.group;
          const float f = C.factor[r], y = it > 0 ? __uint_as_float(o[e]) * f * (kScaleUnit * unit4<FMT>()) : lost ? nan : 0.0f;
          if (T.whole)
            P.out[(T.first + j) * P.out_token + hq * P.out_head + dim] =
                static_cast<uint16_t>(pack_bf16(f == 0.0f ? 0.0f : y, 0.0f));
          else
            L.part_o[(((T.first + j) * P.Hq + hq) * L.slots + L.prefix_splits + T.split) * D + dim] = y;
        }
      }
    }
  if (P.status) {
    if (lost) bits |= SV_DATA_COPY_TIMEOUT;
    bits = __reduce_or_sync(0xFFFFFFFFu, bits);
    if (lane == 0 && bits) atomicOr(P.status, static_cast<int>(bits));
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) tmem_free(tmem, kCols);
}

template <int D, int FMT, int NMAX>
cudaError_t launch(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const int64_t own = static_cast<int64_t>(p.N) * p.c.num_kv_heads * L.own_tiles * L.own_splits;
  if (own > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(own));
  cfg.blockDim = dim3(kOwnThreads);
  cfg.dynamicSmemBytes = OwnSmem<D, NMAX>::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  return cudaLaunchKernelEx(&cfg, own4_kernel<D, FMT, NMAX>, p, L);
}
template <int D, int FMT>
cudaError_t pick(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  return own4_rows(p) == 32 ? launch<D, FMT, 32>(p, L, stream) : launch<D, FMT, 64>(p, L, stream);
}

template <int D, int FMT>
cudaError_t enable() {
  const cudaError_t e = cudaFuncSetAttribute(own4_kernel<D, FMT, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             OwnSmem<D, 32>::kBytes);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(own4_kernel<D, FMT, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 OwnSmem<D, 64>::kBytes);
}

}  // namespace

cudaError_t enable_own4_kernels() {
  cudaError_t e;
  if ((e = enable<128, SV_CACHE_E2M1>()) != cudaSuccess || (e = enable<128, SV_CACHE_INT4>()) != cudaSuccess ||
      (e = enable<64, SV_CACHE_E2M1>()) != cudaSuccess)
    return e;
  return enable<64, SV_CACHE_INT4>();
}

cudaError_t launch_own4(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  const bool i4 = p.c.format == SV_CACHE_INT4;
  if (p.c.head_dim == 128) return i4 ? pick<128, SV_CACHE_INT4>(p, L, stream) : pick<128, SV_CACHE_E2M1>(p, L, stream);
  return i4 ? pick<64, SV_CACHE_INT4>(p, L, stream) : pick<64, SV_CACHE_E2M1>(p, L, stream);
}

}  // namespace sv
