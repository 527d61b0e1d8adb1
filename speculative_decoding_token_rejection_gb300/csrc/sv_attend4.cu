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
// second.  A tile is 128 keys, its bytes are loaded a tile ahead.  Three to five
// CTAs an SM hide each other's waits.
//
// What bounds it are its warps' waits for their own stages: about 800 instructions
// a warp and tile (unpacking 256 elements a thread, 4 to 6 for a weight, addresses),
// one after another, by 3.5 warps a scheduler, 2.6 in tiles of 64 rows.  They fill 53 %
// and 47 % of the issue slots and no pipe by half: integer operations and conversions
// 46 %, fp32 and f16 arithmetic 29 %, shared memory's data 47 %, tensor cores 13 and 21 %
// (256 ragged requests in tiles of 32 rows; 6 long ones in tiles of 64).  256 requests x
// 4096 keys x 8 heads of 128 (1.28 GB): 4 rows a head 270 us (0.70 of the copy rate), 16
// rows 283, 20 rows 343, 32 rows 352, 64 rows 495; head_dim 64, 4 rows 185 (0.54), 32 rows
// 239.  By CTAs an SM (152 requests x 4 rows, tiles of 32): one 385 us, two 241, three 225,
// four 196.  Lost: 256 threads, two a key, that exchange maxima; K loaded long before V
// (350 us against 331); chunks of 2048 keys (396 against 361); anything that spills in
// the loop (what -Xptxas -v shows lies outside: up to two stores and four loads a warp,
// whatever its tiles).  Gained: bytes prefetched to L2 a tile before they are loaded (350
// to 331 us); places in shared memory.  One tile alone takes 8.9 us, dependent loads
// (length, page, bytes) and code met for the first time.
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
#include <type_traits>

#include "sv_attend.cuh"
#include "sv_cache4.cuh"
#include "sv_tensor.cuh"

namespace sv {
namespace {

constexpr int kOwnKeys = 128, kOwnThreads = kOwnKeys;  // a thread a key
constexpr float kRaise = 8;
constexpr float kHuge = 4096;                   // maxima of this size are two numbers
constexpr float kScaleUnit = 0x1p28f;           // W
constexpr float kLeastUnits = kLeastLog2 - 28;  // log2 of the size that a scale counts as at least, in W

// Where the kv head's rows are, in shared memory: worked out from the arguments for every tile, the multiplications of a
// warp's own registers took 2500 of 8000 cycles a tile.
struct alignas(16) OwnPlaces {
  const uint8_t *k, *v, *k_group, *v_group, *k_scale, *v_scale;
  uint32_t page, token, group_page, group_token, scale_page, scale_token;  // bytes from one to the next
  const int32_t *table, *table0;
};

template <int ROWS>
struct OwnControl {
  OwnPlaces at;
  uint64_t k_empty, s_full, o_full;
  uint32_t tmem, tmem_keys, abort;
  uint32_t huge;                       // some |m| is so large that its two parts are subtracted one after the other
  alignas(16) float neg[ROWS];    // negated m, 0 without one
  alignas(16) float zero[ROWS];
  alignas(16) float negx[ROWS], negu[ROWS];  // its parts, negated
  alignas(16) float back[ROWS];   // what undoes a row's power of two
  alignas(16) int limit[ROWS];    // keys that the row sees are below it
  alignas(16) float factor[ROWS]; // of a raised maximum; at the end, of the outputs
  float mx[ROWS], mu[ROWS];  // m = mx + mu, mx -inf without one
  float part[4][ROWS];            // of the four warps that hold a row
  uint32_t none[ROWS];            // the row sees a value scale that is no number
  alignas(16) int64_t to[ROWS];   // the row's place in the output, or its partial result's
};

// Shared memory: [D / 64][128 keys][128 bytes] of V, weights of up to 64 rows in 128-byte lines, [D / 64][NMAX rows][128
// bytes] of queries.  Two keys of up to 32 rows, four of up to 16, share a line of weights, 64 or 32 keys apart: so four or
// five CTAs' memory fits an SM.  16-byte columns of a line are exchanged by line % 8.
template <int D, int NMAX>
struct OwnSmem {
  static constexpr int kLines = kOwnKeys * 128;
  static constexpr int kV = 0, kP = D / 64 * kLines, kQ = kP + kLines * NMAX / kOwnRows4, kControl = kQ + D / 64 * NMAX * 128,
                       kBytes = kControl + static_cast<int>(sizeof(OwnControl<NMAX>)) + 1024;  // (the base is rounded up to 1 KB)
};
__device__ __forceinline__ int line_at(int line, int col) { return line * 128 + ((col ^ (line & 7)) << 4); }

// Tensor memory is reached by whole warps (.aligned): behind a branch that lanes take apart, and behind a wait, which they
// leave one by one, a __syncwarp() comes first.

// Sixteen columns of the thread's lane.
__device__ __forceinline__ void tmem_store_row(uint32_t addr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
      "};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Eight columns of the thread's lane.
__device__ __forceinline__ void tmem_load_row(uint32_t addr, float r[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(addr)
               : "memory");
}
// Waits for every load so far; the registers go through, so no use of them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_row(float r[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_store_8(uint32_t addr, const float r[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "f"(r[0]),
               "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// A cache row on its way: nibbles and group scales.
template <int D>
struct RawRow {
  uint32_t w[D / 8], g[D / 64];
};
// (Volatile: they stay where they are written, a tile ahead of their use.)
__device__ __forceinline__ uint32_t load_word(const void *p) {
  uint32_t r;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}
template <int D>
__device__ __forceinline__ void load_row(RawRow<D> &r, const uint8_t *data, const uint8_t *group) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) ld_stream_32(data + 32 * i, r.w + 8 * i);
  if (D == 128)
    asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(r.g[0]), "=r"(r.g[D / 64 - 1]) : "l"(group));
  else
    r.g[0] = load_word(group);
}
__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// p + a * x + b * y
__device__ __forceinline__ const uint8_t *step(const uint8_t *p, uint32_t a, uint32_t x, uint32_t b, uint32_t y) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(a), "r"(x), "l"(p));
  asm("mad.wide.u32 %0, %1, %2, %0;" : "+l"(r) : "r"(b), "r"(y));
  return reinterpret_cast<const uint8_t *>(r);
}

// CTAs of an SM: what their registers, shared and tensor memory allow.  (Four of 16 rows and head_dim 128: 96 registers, as
// a fifth would leave, spill in the loop, 406 us against 278 for 256 requests x 4096 keys.  Head_dim 64: five 190, four 205,
// but with 32 rows five 275 against 250.)
constexpr int own4_ctas(int d, int nmax) { return nmax == 64 ? 3 : nmax == 16 && d == 64 ? 5 : 4; }
template <int D, int FMT, int NMAX>
__global__ void __launch_bounds__(kOwnThreads, own4_ctas(D, NMAX))
    own4_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ AttendPlan L) {
  pdl_enter();
  OwnTile T;
  if (!own_tile(P, L, blockIdx.x, NMAX, T)) return;
  extern __shared__ uint8_t raw[];
  uint8_t *const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  using Y = OwnSmem<D, NMAX>;
  OwnControl<NMAX> &C = *reinterpret_cast<OwnControl<NMAX> *>(smem + Y::kControl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Tensor memory: K, S and O.  Where all of them pass 128 columns, which is a quarter of what an SM has, K goes there in
  // two halves of 32 columns, allocated by themselves: three CTAs' 160 columns fit an SM.
  constexpr int kHalves = D == 128 && NMAX > 32 ? 2 : 1;
  constexpr uint32_t kKeyCols = D / 2 / kHalves, kS = 0, kO = NMAX, kOwnCols = 2 * NMAX;
  const int n8 = (T.rows + 7) / 8, n16 = (T.rows + 15) / 16;

  // ---- the first tile's bytes are on their way before anything else ----
  const int ntiles = (max(0, T.k_end - T.k_begin) + kOwnKeys - 1) / kOwnKeys;
  if (tid == 0) {
    OwnPlaces &A = C.at;
    A.k = static_cast<const uint8_t *>(P.c.k) + T.h * P.c.head_stride;
    A.v = static_cast<const uint8_t *>(P.c.v) + T.h * P.c.head_stride;
    A.k_group = P.k_group + T.h * P.group_head;
    A.v_group = P.v_group + T.h * P.group_head;
    A.k_scale = reinterpret_cast<const uint8_t *>(P.c.k_scale + T.h * P.c.scale_head_stride);
    A.v_scale = reinterpret_cast<const uint8_t *>(P.c.v_scale + T.h * P.c.scale_head_stride);
    A.page = static_cast<uint32_t>(P.c.block_stride);
    A.token = static_cast<uint32_t>(P.c.token_stride);
    A.group_page = static_cast<uint32_t>(P.group_block);
    A.group_token = static_cast<uint32_t>(P.group_token);
    A.scale_page = static_cast<uint32_t>(P.c.scale_block_stride * 4);
    A.scale_token = static_cast<uint32_t>(P.c.scale_token_stride * 4);
    A.table = P.tables + T.i * P.table_stride;
    A.table0 = P.tables;
  }
  __syncthreads();
  bool bad = false;  // some page was outside the cache
  // (Nothing here is loaded under a condition: registers that a branch fills otherwise would be waited for at its end.  A
  // key that is not there takes a place that is, and counts for nothing later.)
  auto page_of = [&](int it) {  // of the thread's key of tile `it`
    const int k = max(T.k_begin, min(T.k_begin + it * kOwnKeys + tid, T.k_end - 1));
    return static_cast<int>(load_word((k < P.row0 ? C.at.table0 : C.at.table) + div_by(k, L.page)));
  };
  RawRow<D> krow, vrow;
  uint32_t ks = 0, vs = 0;
  // Whether the key of the rows in krow and vrow (or on their way) is there; the same of the tile behind it, and where
  // that one's key is: its bytes go to the L2 cache a tile before they are loaded.
  bool live = false, next_live = false;
  uint32_t next_page = 0, next_off = 0;
  auto place = [&](int it, int page) {
    const int k = T.k_begin + it * kOwnKeys + tid;
    const bool in = k < T.k_end;
    next_live = in && static_cast<uint32_t>(page) < static_cast<uint32_t>(P.c.num_blocks);
    bad |= in && !next_live;
    next_page = next_live ? page : 0;
    next_off = next_live ? k - div_by(k, L.page) * P.c.block_size : 0;
  };
  auto load = [&]() {
    const OwnPlaces &A = C.at;
    const uint32_t p = next_page, off = next_off;
    live = next_live;
    load_row<D>(krow, step(A.k, A.page, p, A.token, off), step(A.k_group, A.group_page, p, A.group_token, off));
    load_row<D>(vrow, step(A.v, A.page, p, A.token, off), step(A.v_group, A.group_page, p, A.group_token, off));
    ks = load_word(step(A.k_scale, A.scale_page, p, A.scale_token, off));
    vs = load_word(step(A.v_scale, A.scale_page, p, A.scale_token, off));
  };
  auto prefetch = [&]() {
    const OwnPlaces &A = C.at;
    const uint32_t p = next_page, off = next_off;
    prefetch_line(step(A.k, A.page, p, A.token, off));
    prefetch_line(step(A.v, A.page, p, A.token, off));
    prefetch_line(step(A.k_group, A.group_page, p, A.group_token, off));
    prefetch_line(step(A.v_group, A.group_page, p, A.group_token, off));
    prefetch_line(step(A.k_scale, A.scale_page, p, A.scale_token, off));
    prefetch_line(step(A.v_scale, A.scale_page, p, A.scale_token, off));
  };
  int page = 0;
  if (ntiles > 0) {
    place(0, page_of(0));
    load();
    place(1, page_of(1));
    page = page_of(2);
  }

  if (tid == 0) {
    mbar_init(&C.k_empty, 1);
    mbar_init(&C.s_full, 1);
    mbar_init(&C.o_full, 1);
    C.abort = C.huge = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_get(&C.tmem, kOwnCols);
    tmem_get(&C.tmem_keys, kKeyCols);
    tmem_no_more();
  }
  if (tid < NMAX) {
    const int j = div_by(T.r0 + tid, L.group);
    C.limit[tid] = tid < T.rows ? T.len - T.gam + j : 0x7FFFFFFF;
    C.zero[tid] = C.neg[tid] = C.negx[tid] = C.negu[tid] = C.mu[tid] = 0.0f;
    C.mx[tid] = -INFINITY;
    C.none[tid] = 0;
  }
  // ---- the queries: f16, each row with its own power of two, dimensions in the order of the unpacked keys ----
  bool shifted = false;
  {
    constexpr int kCh = D / 8, kRowsPass = kOwnThreads / kCh, kPass = (NMAX + kRowsPass - 1) / kRowsPass;
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
      if (r < NMAX) {
        if (col == 0) C.back[r] = pow2(-shift);
        *reinterpret_cast<uint4 *>(smem + Y::kQ + (col >> 3) * (NMAX * 128) + line_at(r, col & 7)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  fence_proxy_async_smem();
  fence_before();
  shifted = __syncthreads_or(shifted);
  fence_after();
  int low = 0x7FFFFFFF;  // keys below it are seen by every row
  for (int r = lane; r < T.rows; r += 32) low = min(low, C.limit[r]);
  low = __reduce_min_sync(0xFFFFFFFFu, low);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, C.tmem, 0), tmem_keys = __shfl_sync(0xFFFFFFFFu, C.tmem_keys, 0);
  const uint32_t base = smem_addr(smem), lanes = static_cast<uint32_t>(warp * 32) << 16;  // the warp's part of tensor memory
  const bool leader = elected();

  float l[NMAX];  // sums over the thread's keys
#pragma unroll
  for (int r = 0; r < NMAX; ++r) l[r] = 0.0f;
  const float c_all = P.scale * unit4<FMT>() * kLog2e;
  // Half (or all) of the keys in krow to tensor memory, and their part of the scores.
  constexpr int kTwos = D / 32 / kHalves;  // pairs of groups in it
  auto unpack_keys = [&](int half) {
    if (half) __syncwarp();  // (before the first half the loop's)
#pragma unroll
    for (int two = 0; two < kTwos; ++two) {
      const int at = half * kTwos + two;
      uint32_t h[16];
      groups_to_f16_mixed<FMT>(krow.w + 4 * at, live ? krow.g[at >> 1] >> (16 * (at & 1)) : 0u, h);
      tmem_store_row(tmem_keys + lanes + two * 16, h);
    }
    tmem_wait_store();
    fence_before();
    __syncthreads();
    if (warp == 0) {
      fence_after();
      const uint64_t queries = operand(base + Y::kQ, 16);
      const uint32_t shape = product(n16 * 16, false);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 2 * kTwos; ++kk) {
          const int at = half * 2 * kTwos + kk;
          const uint64_t b = queries + static_cast<uint64_t>((at >> 2) * (NMAX * 128 >> 4) + (at & 3) * 2);
          if (at == 0)
            mma_ts<false>(tmem + kS, tmem_keys, b, shape);
          else
            mma_ts<true>(tmem + kS, tmem_keys + kk * 8, b, shape);
        }
        mma_commit(half == kHalves - 1 ? &C.s_full : &C.k_empty);
      }
    }
  };
  // Half (or all) of the values in vrow to shared memory.
  // (kShare keys to a line of weights, kShareLines apart)
  constexpr int kShare = 64 / NMAX, kShareLines = kOwnKeys / kShare;
  const uint32_t p_line = base + Y::kP + tid % kShareLines * 128 + (((tid / kShareLines * (NMAX / 8)) ^ (tid & 7)) << 4);
  const uint32_t v_line = base + Y::kV + tid * 128 + ((tid & 7) << 4);
  auto unpack_values = [&](int half) {
#pragma unroll
    for (int two = half * kTwos; two < (half + 1) * kTwos; ++two) {
      uint32_t h[16];
      groups_to_f16_mixed<FMT>(vrow.w + 4 * two, live ? vrow.g[two >> 1] >> (16 * (two & 1)) : 0u, h);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"((v_line ^ ((two & 1) * 64 + c * 16)) + (two >> 1) * Y::kLines),
                     "r"(h[4 * c]), "r"(h[4 * c + 1]), "r"(h[4 * c + 2]), "r"(h[4 * c + 3])
                     : "memory");
    }
  };
  bool force = true;  // some row has no maximum
  bool ok = true;
  int it = 0;
  __syncwarp();
  for (; it < ntiles; ++it) {
    const bool dead = !live;
    const float kc = __uint_as_float(ks) * c_all, v_scale = dead ? 0.0f : __uint_as_float(vs);
    const int key = T.k_begin + it * kOwnKeys + tid;
    const bool more = it + 1 < ntiles;
    unpack_keys(0);
    if (it > 0) ok = wait(C, &C.o_full, (it - 1) & 1) && ok;  // (the values' and weights' place is free, and O is there)
    unpack_values(0);
    if (kHalves == 2) {
      ok = wait(C, &C.k_empty, it & 1) && ok;
      fence_after();
      unpack_keys(1);
      unpack_values(1);
    }
    if (more) {
      load();
      place(it + 2, page);
      prefetch();
      page = page_of(it + 3);
    }
    ok = wait(C, &C.s_full, it & 1, P.expire) && ok;
    fence_after();
    // ---- weights ----
    const bool number = fabsf(v_scale) < INFINITY;
    const float vr = number && fabsf(v_scale) >= kLeastScale ? v_scale * (1.0f / kScaleUnit) : 0.0f;
    const float lv = fmaxf(__log2f(fabsf(vr)), kLeastUnits);
    const uint32_t s_mine = tmem + lanes + kS;
    if (!number) {
      for (int r = 0; r < T.rows; ++r)
        if (key < C.limit[r]) C.none[r] = 1;
    }
    __syncwarp();
    // Two eights of rows at a time: columns 16 g .. (the first eight again where there is one).
    auto load_scores = [&](int g, float x[16]) {
      const uint32_t at = s_mine + g * 16;
      tmem_load_row(at, x);
      tmem_load_row(2 * g + 1 < n8 ? at + 8 : at, x + 8);
      tmem_wait_row(x);
      tmem_wait_row(x + 8);
    };
    auto store_scores = [&](int g, const float x[16]) {
      tmem_store_8(s_mine + g * 16, x);
      if (2 * g + 1 < n8) tmem_store_8(s_mine + g * 16 + 8, x + 8);
    };
    // x * by - m
    float by = kc;
    auto exponents = [&](int g, float x[16], const float *neg) {
      load_scores(g, x);
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(neg + g * 16 + e);
        const Pair a = fma2(pair(x[e], x[e + 1]), pair(by, by), pair(m.x, m.y));
        const Pair b = fma2(pair(x[e + 2], x[e + 3]), pair(by, by), pair(m.z, m.w));
        x[e] = lo(a);
        x[e + 1] = hi(a);
        x[e + 2] = lo(b);
        x[e + 3] = hi(b);
      }
    };
    const float *neg = C.neg;
    // Rows that do not see every key, or have a power of two: their scores in base 2 take the place of the products.
    if (T.k_begin + (it + 1) * kOwnKeys > low || shifted || __any_sync(0xFFFFFFFFu, dead)) {
#pragma unroll 1
      for (int g = 0; 2 * g < n8; ++g) {
        float x[16];
        load_scores(g, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = g * 16 + e;
          const float back = C.back[r];  // (no branches: their loads would come one after another, 160 cycles each)
          x[e] = static_cast<int>(dead) | static_cast<int>(key >= C.limit[r]) ? -INFINITY : x[e] * kc * back;
        }
        store_scores(g, x);
      }
      tmem_wait_store();
      by = 1.0f;
    }
    // Weights with the m there is; in the first tile, or where a weight passes 2^8 with it (seldom), with a new one.
    // (Below kHuge a fused operation's exact product differs from a rounded one by 2^-12 at most.  Beyond, that would part
    // equal scores, and from 2^28 on send weights out of range: there every product is rounded first.)
    bool fresh = force || C.huge, stop = false;
    for (;;) {
      if (fresh) {
        const bool huge = C.huge;
        // The rows' largest (x + part) + add, to the threads that keep the rows' m.
        auto largest = [&](const float *part, float add) {
#pragma unroll 1
          for (int c = 0; c < n8; ++c) {
            float x[8];
            tmem_load_row(s_mine + c * 8, x);
            tmem_wait_row(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (__fmul_rn(x[e], by) + part[c * 8 + e]) + add;
            const float most = reduce_eight<true>(x, lane);
            if ((lane & 3) == 0) C.part[warp][c * 8 + (lane >> 2)] = most;
            __syncwarp();
          }
          __syncthreads();
          return tid < n8 * 8 ? fmaxf(fmaxf(C.part[0][tid], C.part[1][tid]), fmaxf(C.part[2][tid], C.part[3][tid])) : 0.0f;
        };
        float mx = 0.0f, mu = 0.0f;
        // first with m in one number, then, where one is too large for that, its two parts one after the other
#pragma unroll 1
        for (int round = huge ? 1 : 0; round < 3; ++round) {
          const float most = largest(round == 2 ? C.negx : C.zero, round == 1 ? 0.0f : lv);
          if (tid < n8 * 8) {
            if (round == 2) {
              mu = most;
            } else {
              mx = round == 0 ? most : fmaxf(C.mx[tid], most);
              if (round == 0 && fabsf(mx) >= kHuge && fabsf(mx) < INFINITY) C.huge = 1;
              if (round == 1) C.negx[tid] = mx == -INFINITY ? 0.0f : -mx;
            }
          }
          __syncthreads();
          if (round == 0 && !C.huge) break;
        }
        bool unset = false, raised = false;
        if (tid < n8 * 8) {
          const bool had = C.mx[tid] != -INFINITY;
          const float old = had ? (C.mx[tid] - mx) + C.mu[tid] : 0.0f;  // of the sums so far, less mx
          raised = !had || mu > old + kRaise;
          C.factor[tid] = had && raised ? exp2_approx(old - mu) : 1.0f;  // (without a maximum O and l are zeros or NaN)
          if (raised) {
            C.mx[tid] = mx;
            C.mu[tid] = mx == -INFINITY ? 0.0f : mu;
          }
          unset = C.mx[tid] == -INFINITY;
          C.negx[tid] = unset ? 0.0f : -C.mx[tid];
          C.negu[tid] = -C.mu[tid];
          C.neg[tid] = C.negx[tid] + C.negu[tid];
        }
        force = __syncthreads_or(unset);
        if (it > 0) {
          ok = wait(C, &C.o_full, (it - 1) & 1) && ok;
          __syncwarp();
          fence_after();
#pragma unroll
          for (int c = 0; c < NMAX / 8; ++c)
            if (c < n8) {
#pragma unroll
              for (int e = 0; e < 8; ++e) l[c * 8 + e] *= C.factor[c * 8 + e];
            }
#pragma unroll 1
          for (int c = 0; c < n8; ++c) {
            float o[8];
            tmem_load_row(tmem + lanes + kO + c * 8, o);
            tmem_wait_row(o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= C.factor[c * 8 + e];
            tmem_store_8(tmem + lanes + kO + c * 8, o);
          }
        }
        if (C.huge) {  // the exponents take the scores' place
#pragma unroll 1
          for (int c = 0; c < n8; ++c) {
            float x[8];
            tmem_load_row(s_mine + c * 8, x);
            tmem_wait_row(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (__fmul_rn(x[e], by) + C.negx[c * 8 + e]) + C.negu[c * 8 + e];
            tmem_store_8(s_mine + c * 8, x);
          }
          by = 1.0f;
          neg = C.zero;
        }
        tmem_wait_store();
      }
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < NMAX / 16; ++g)
        if (2 * g < n8) {
          float x[16];
          exponents(g, x, neg);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (2 * g + c < n8) {
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                top = max3(top, x[c * 8 + e], x[c * 8 + e + 1]);
                const Pair w = pair(exp2_approx(x[c * 8 + e]), exp2_approx(x[c * 8 + e + 1]));
                float *const sum = l + g * 16 + c * 8 + e;
                const Pair s = add2(pair(sum[0], sum[1]), w), v = mul2(w, pair(vr, vr));
                sum[0] = lo(s);
                sum[1] = hi(s);
                p[e >> 1] = pack_f16(lo(v), hi(v));
              }
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_line ^ ((g << 5) + (c << 4))), "r"(p[0]),
                           "r"(p[1]), "r"(p[2]), "r"(p[3])
                           : "memory");
            }
        }
      fence_proxy_async_smem();
      fence_before();
      if (!__syncthreads_or((!fresh && top + lv > kRaise) || !ok)) break;
      // (whoever gave up did so before the barrier, and nobody waits before the next one)
      stop = gave_up(C);
      if (stop) break;
      // The sums as they were.  (What the subtraction loses is 2^-24 of a weight that comes again; beside one that is no
      // number of fp32 the sums so far, below 2^106, are nothing.  A NaN of a key before stays.)
#pragma unroll
      for (int g = 0; g < NMAX / 16; ++g)
        if (2 * g < n8) {
          float x[16];
          exponents(g, x, neg);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float w = exp2_approx(x[e]);
            float &sum = l[g * 16 + e];
            if (2 * g + (e >> 3) < n8) sum = x[e] < 127.0f || sum != sum ? sum - w : 0.0f;
          }
        }
      fresh = true;
    }
    if (stop) break;
    // ---- outputs ----
    if (warp == 0) {
      fence_after();
      const uint64_t v_operand = operand(base + Y::kV, Y::kLines), p_operand = operand(base + Y::kP, Y::kLines);
      const uint32_t output_shape = product(n16 * 16, true, D, true);
      if (leader) {
        if (it == 0)
          mma_ss<false>(tmem + kO, v_operand, p_operand, output_shape);
        else
          mma_ss<true>(tmem + kO, v_operand, p_operand, output_shape);
#pragma unroll
        for (int kk = 1; kk < kOwnKeys / 16; ++kk)
          mma_ss<true>(tmem + kO, v_operand + kk * (2048 >> 4),
                       p_operand + kk % (8 / kShare) * (2048 >> 4) + kk / (8 / kShare) * (2 * NMAX >> 4),
                       output_shape);
        mma_commit(&C.o_full);
      }
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
    // (the sums are those of both parts where they were subtracted one after the other)
    const float rest = C.huge && fabsf(m) < INFINITY ? (C.mx[tid] - m) + C.mu[tid] : 0.0f;
    const float sum = lost ? nan : (C.part[0][tid] + C.part[1][tid]) + (C.part[2][tid] + C.part[3][tid]);
    const int64_t at = (T.first + j) * P.Hq + hq;
    const int64_t slot = at * L.slots + L.prefix_splits + T.split;
    if (T.whole) {
      if (P.lse) P.lse[at] = sum == 0.0f ? -INFINITY : (m + (rest + log2f(sum))) * kLn2;
    } else {
      L.part_ml[slot] = make_float2(m, sum);
      L.part_rest[slot] = rest;
    }
    C.to[tid] = T.whole ? (T.first + j) * P.out_token + hq * P.out_head : slot * D;
    // (a row without keys that count has the output 0.  Some w was 2^-log2(value_scale / W) at least, so sum is above
    // 2^-101 otherwise, and far below 2^126.)
    C.factor[tid] = lost || C.none[tid] ? nan : !T.whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  __syncthreads();
  // a lane holds a dimension: lane i of the tensor memory for head_dim 128, for 64 the first half of each warp's
  const int at = D == 128 ? tid : warp * 16 + (lane & 15);
  const int dim = mixed<FMT>() ? mixed_place(at) : at;
  const float scale = it > 0 ? kScaleUnit * unit4<FMT>() : lost ? nan : 0.0f;
#pragma unroll 1
  for (int c = 0; c < n8; ++c) {
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 1.0f;
    if (it > 0) {
      tmem_load_row(tmem + lanes + kO + c * 8, o);
      tmem_wait_row(o);
    }
    if (D == 128 || lane < 16) {
      float f[8];
      int64_t to[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] = C.factor[c * 8 + e];
        to[e] = C.to[c * 8 + e] + dim;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = f[e] == 0.0f ? 0.0f : o[e] * f[e] * scale;
        if (c * 8 + e < T.rows) {
          if (T.whole)
            P.out[to[e]] = static_cast<uint16_t>(pack_bf16(y, 0.0f));
          else
            L.part_o[to[e]] = y;
        }
      }
    }
    __syncwarp();
  }
  if (P.status) {
    const uint32_t bits = __reduce_or_sync(0xFFFFFFFFu, (bad ? static_cast<uint32_t>(SV_DATA_BAD_SLOT) : 0u) |
                                                            (lost ? static_cast<uint32_t>(SV_DATA_COPY_TIMEOUT) : 0u));
    if (lane == 0 && bits) atomicOr(P.status, static_cast<int>(bits));
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) {
    tmem_free(tmem, kOwnCols);
    tmem_free(tmem_keys, kKeyCols);
  }
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
  const int rows = own4_rows(p);
  return rows == 16   ? launch<D, FMT, 16>(p, L, stream)
         : rows == 32 ? launch<D, FMT, 32>(p, L, stream)
                      : launch<D, FMT, 64>(p, L, stream);
}

template <int D, int FMT>
cudaError_t enable() {
  cudaError_t e = cudaFuncSetAttribute(own4_kernel<D, FMT, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       OwnSmem<D, 16>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(own4_kernel<D, FMT, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize, OwnSmem<D, 32>::kBytes);
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
