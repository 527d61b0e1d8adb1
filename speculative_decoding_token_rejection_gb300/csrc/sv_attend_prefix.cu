// sv_attend_prefix.cu -- the shared prefix of the verify tokens' attention on
// the tensor cores' own memory (tcgen05).
//
// All requests' rows of a kv head meet the same prefix keys, so the work is two
// matrix products of thousands of rows and is bound by the tensor cores and
// what feeds them: 4 * head_dim operations a (row, key) pair, one exponential
// each.  The prefix's bytes become f16 (exact) once for the whole call: a small
// kernel writes the K and V tiles of 128 keys to the workspace in the very
// order the products want them in shared memory, so a tile is one bulk copy.
// (Turned into f16 by every CTA for itself, the tiles took three warps 6000
// cycles each, most of it page look-ups and shared-memory stores, against 2050
// of the products: 64 requests x 5 tokens over 8192 keys 100 us.)
// An item is 256 rows (two accumulator tiles of 128) of one kv head; the units
// of work, its key tiles, are dealt over as many CTAs as there are SMs, item
// after item, so an item's keys are cut only where one CTA's share ends; empty
// units between the items stand for the time that beginning another one takes.
// In a CTA:
//
//   warps 0-3, 4-7  softmax of a row tile, 32 rows a warp: reads S from tensor
//                   memory, writes the weights back over it as f16
//   warps 8, 9      the keys' factors, four tiles ahead
//   warp 10         copies K and V tiles, two deep
//   warp 11         issues S = Q K^T and O += P V (P from tensor memory)
//
// While one row tile's softmax runs, the tensor cores work for the other:
// S0 S1 | P0 V, S0' | P1 V, S1' | ...  The products run in the order they are
// issued, so S0' may overwrite P0, and "S0' is done" tells the softmax that
// P0 V is too: the output may be rescaled then.
//
// A softmax lane holds four rows' scores of 32 keys each, the accumulator shape
// of a small product, not one row's 128: the keys' factors are read from shared
// memory once for four rows.  (A thread a row, those reads alone kept the
// shared-memory path busy for 2000 cycles a tile, as long as the products:
// 1.28 ms for 512 requests x 8 tokens over 16384 keys.)
//
// Numbers.  x = (q . b) * (scale * log2 e * key_scale) as in sv_attend.cuh, but
// the value scales are kept out of the exponent: w = 2^(x - m), l = sum w,
// P = w * value_scale / W, O = W * sum P b.  Any m gives the same quotient O / l;
// it is raised to the largest x + log2(value_scale / W) when that passes it by
// 8, so P stays below 2^8.  Whether it may have is seen from max x and the
// tile's largest value scale alone.  W is 2^28, the middle of the scales that
// kv_write gives (2^-64 to 2^121): w and l stay within fp32 for any of them.
// (One near the first tile's scales sent later ones out of range.)
//
// Measured: 512 requests x 8 tokens over 16384 keys, 805 us of the call's 1.03
// ms: 1.37 PFLOP/s, 72 % of a plain matrix product's rate.  A key tile takes a
// CTA about 3300 cycles, of which a softmax warp works for 1800 and waits for its row
// tile's products for 1250; a segment adds 25000 (queries in, results out).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_attend.cuh"

namespace sv {
namespace {

constexpr int kRowsTile = kPrefixRowTile / 2;  // rows of an accumulator tile
constexpr int kKeyTile = kPrefixKeyTile;
constexpr int kSoftmaxThreads = 256;
constexpr int kVectorThreads = 64;
constexpr int kPrefixThreads = kSoftmaxThreads + kVectorThreads + 64;
constexpr int kVectorSlots = 4;
constexpr uint32_t kWaitPolls = 1u << 24;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kRaise = 8;
constexpr float kScaleUnit = 0x1p28f;  // W
constexpr float kLeastUnits = kLeastLog2 - 28;  // log2 of the size that a scale counts as at least, in W

struct alignas(16) Vectors {  // of one key tile
  float2 kc[kKeyTile / 2], vr[kKeyTile / 2];  // of two keys: their factors; their value scales / W
  uint32_t dead[4];  // keys left out, a bit each
  uint32_t none[4];  // keys whose value scale is no number
  float top[2];      // log2 of the largest value scale / W, of keys 0-31 and 64-95, and of the others
};

struct Control {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], vec_full[kVectorSlots], vec_empty[kVectorSlots], s_full[2], p_full[2], q_full, done;
  uint32_t tmem, abort;
  float back[2 * kRowsTile];  // what undoes a row's power of two
};

static_assert(sizeof(Vectors) % 16 == 0, "every slot starts on a 16-byte boundary");

template <int D>
struct Smem {
  static constexpr int kTile = kKeyTile * D * 2;  // a K, V or Q tile in f16
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kVec = 6 * kTile,
                       kControl = kVec + kVectorSlots * static_cast<int>(sizeof(Vectors)),
                       kBytes = kControl + static_cast<int>(sizeof(Control)) + 1024;  // (the base is rounded up to 1 KB)
};

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D (tensor memory) = A B (+ D), both operands in shared memory.
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
// The same with A in tensor memory.
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Arrives on `bar` once every product issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Tensor memory in the shape of a 16x8 product's accumulator, N of them side by
// side, for 16 of the warp's 32 lanes: register 4j, 4j + 1 of lane (g, c) are
// columns 8j + 2c, + 1 of row g, the next two of row g + 8.
__device__ __forceinline__ void tmem_load_128(uint32_t addr, uint32_t r[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
      "}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_32(uint32_t addr, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
      "}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// Waits for every load so far; the registers go through, so no use of them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_load(uint32_t r[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_store_32(uint32_t addr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
      "};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 columns of 16-bit pairs: register 2j of lane (g, c) is column 4j + c of row g, the next one of row g + 8.
__device__ __forceinline__ void tmem_store_pairs(uint32_t addr, const uint32_t r[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand with rows of 128 bytes (64 f16), 8-row groups of 1 KB,
// 16-byte columns exchanged within a group (column ^ row % 8).  `next64`:
// bytes from 64 elements to the next 64 where those run along the operand's
// outer dimension.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t next64) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | static_cast<uint64_t>((next64 >> 4) & 0x3FFF) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// f16 operands, fp32 sums, 128 x n; B's outer dimension contiguous or its inner one.
constexpr uint32_t product(int n, bool b_outer_contiguous) {
  return 1u << 4 | (b_outer_contiguous ? 1u << 16 : 0u) | static_cast<uint32_t>(n / 8) << 17 | (128u / 16) << 24;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// The CTA gives up: no wait begins anew, rows that are not done become NaN, and
// the status word says so at the end.
__device__ __forceinline__ void give_up(Control &C) {
  *const_cast<volatile uint32_t *>(&C.abort) = 1;
  __threadfence_block();
}
__device__ __forceinline__ bool gave_up(const Control &C) { return *const_cast<const volatile uint32_t *>(&C.abort) != 0; }
// Waits for phase `parity` of a barrier; false when the CTA gives up (a wait
// of two seconds, `expire`, or another thread that did).
__device__ __forceinline__ bool wait(Control &C, uint64_t *bar, uint32_t parity, bool expire = false) {
  if (!expire) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t began = now_ns();
    for (uint32_t it = 0; it < kWaitPolls; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if (gave_up(C)) return false;
      if ((it & 15u) == 15u && now_ns() - began > kWaitNs) break;
    }
  }
  give_up(C);
  return false;
}
// The same for all lanes of a warp together.
__device__ __forceinline__ bool wait_warp(Control &C, uint64_t *bar, uint32_t parity, bool expire = false) {
  return __all_sync(0xFFFFFFFFu, wait(C, bar, parity, expire));
}
// Waits for what is in flight, also in a CTA that has given up: shared and
// tensor memory must not go before it.
__device__ __forceinline__ void settle(Control &C, uint64_t *bar, uint32_t parity) {
  const uint64_t began = now_ns();
  while (!mbar_try_wait(bar, parity))
    if (now_ns() - began > kWaitNs) {
      give_up(C);
      return;
    }
}

// The prefix's K and V as f16 tiles of 128 keys, each in the order of its
// shared memory: 64 dimensions after 64, rows of 128 bytes, 16-byte columns
// exchanged by row % 8.  Keys that are not there are zeros, and so are e4m3
// values that are no numbers: they lie behind every request's length, and a
// weight of 0 times one would be NaN.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const AttendParams P, const AttendPlan L) {
  pdl_enter();
  // a thread takes eight bytes of a row and gives one 16-byte column: neighbouring lanes fill whole lines
  constexpr int kCols = D / 8, kPieces = kKeyTile * kCols / kThreads;
  const int tile = blockIdx.x, h = blockIdx.y, side = blockIdx.z, col = threadIdx.x % kCols;
  const uint8_t *const base = static_cast<const uint8_t *>(side ? P.c.v : P.c.k) + h * P.c.head_stride + col * 8;
  uint8_t *const out = L.image + ((static_cast<int64_t>(h) * L.image_tiles + tile) * 2 + side) * (kKeyTile * D * 2);
  uint2 raw[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int r = p * (kThreads / kCols) + threadIdx.x / kCols, k = tile * kKeyTile + r;
    raw[p] = make_uint2(0, 0);
    if (k < P.prefix) {
      const int x = div_by(k, L.page), page = P.tables[x];
      if (page >= 0 && page < P.c.num_blocks)
        raw[p] = __ldg(reinterpret_cast<const uint2 *>(
            base + page * P.c.block_stride + (k - x * P.c.block_size) * P.c.token_stride));
      if (FMT == SV_CACHE_E4M3 && side) {
        raw[p].x &= ~__vcmpeq4(raw[p].x & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        raw[p].y &= ~__vcmpeq4(raw[p].y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int r = p * (kThreads / kCols) + threadIdx.x / kCols;
    uint32_t w[4];
    bytes_to_f16<FMT>(raw[p].x, w[0], w[1]);
    bytes_to_f16<FMT>(raw[p].y, w[2], w[3]);
    *reinterpret_cast<uint4 *>(out + (col >> 3) * (kKeyTile * 128) + r * 128 + (((col & 7) ^ (r & 7)) << 4)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A CTA's consecutive key tiles of one item: a kv head's 256 rows.
struct Segment {
  int h, r0, tiles, n, k_begin, k_end, slot;
};

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1) prefix_kernel(const AttendParams P, const AttendPlan L) {
  pdl_enter();
  extern __shared__ uint8_t raw[];
  uint8_t *const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  using Y = Smem<D>;
  Control &C = *reinterpret_cast<Control *>(smem + Y::kControl);
  Vectors *const vec = reinterpret_cast<Vectors *>(smem + Y::kVec);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = L.image_tiles, u_end = min(L.units, static_cast<int>(blockIdx.x + 1) * L.units_cta);
  auto segment = [&](int u) {  // the CTA's work from unit u on: key tiles of one item (kv head, 256 rows)
    const int item = u / L.period, t0 = u - item * L.period;
    Segment s;
    s.h = item / L.tensor_tiles;
    s.r0 = (item - s.h * L.tensor_tiles) * 2 * kRowsTile;
    s.tiles = L.rows - s.r0 > kRowsTile ? 2 : 1;
    s.n = min(T - t0, u_end - u);
    s.k_begin = t0 * kKeyTile;
    s.k_end = min(P.prefix, s.k_begin + s.n * kKeyTile);
    s.slot = static_cast<int>(blockIdx.x) - item * L.period / L.units_cta;
    return s;
  };
  auto tile_from = [&](int u) {  // the first key tile's unit from u on
    const int t = u % L.period;
    return t < T ? u : u + L.period - t;
  };
  const int u_begin = tile_from(blockIdx.x * L.units_cta);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&C.k_full[i], 1);
      mbar_init(&C.k_empty[i], 1);
      mbar_init(&C.v_full[i], 1);
      mbar_init(&C.v_empty[i], 1);
      mbar_init(&C.s_full[i], 1);
      mbar_init(&C.p_full[i], kRowsTile);
    }
    for (int i = 0; i < kVectorSlots; ++i) {
      mbar_init(&C.vec_full[i], kVectorThreads);
      mbar_init(&C.vec_empty[i], 8);
    }
    mbar_init(&C.q_full, kSoftmaxThreads);
    mbar_init(&C.done, 1);
    C.abort = 0;
    fence_mbar_init();
  }
  if (warp == 11) tmem_alloc(&C.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();

  // Roles pass from one segment to the next on their own: the copies and the factors run ahead as far as their rings
  // allow, the products wait for the queries, and the softmax warps, which write those, have seen the products end.
  int done_tiles = 0, done_segments = 0;  // (barrier phases run on from one segment to the next)

  // The softmax warps' scores need more registers than the others do: 256 * 208 + 128 * 88 = 384 * 168, what the CTA
  // was launched with.
  if (warp >= 8)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  if (warp < 8) {
    // -------------------------------------------------------------------
    // softmax of row tile `t`
    // -------------------------------------------------------------------
    const int t = warp >> 2, w4 = warp & 3;
    int mine = 0;  // key tiles of this row tile so far
    bool ok = true;
    for (int u = u_begin; u < u_end;) {
      const Segment S = segment(u);
      const int h = S.h, r0 = S.r0, tiles = S.tiles, n = S.n, k_begin = S.k_begin, slot = S.slot;
      bool shifted = false;  // some row of the warp was multiplied by a power of two
      {  // the tile's queries: f16, each row with its own power of two
        uint4 x[D / 8];  // warp w4 takes rows 32 * w4 ..; a row is D/8 lanes
        constexpr int kLanes = D / 8, kRowsPass = 32 / kLanes, kQ = 32 / kRowsPass;
        auto source = [&](int f) {  // null: no such row
          const int r = r0 + t * kRowsTile + w4 * 32 + f * kRowsPass + lane / kLanes;
          const int token = div_by(r, L.group), hq = h * P.group + r - token * P.group;
          return r < L.rows ? P.q + token * P.q_token + hq * P.q_head + lane % kLanes * 8 : nullptr;
        };
#pragma unroll
        for (int f = 0; f < kQ; ++f) x[f] = make_uint4(0, 0, 0, 0);
        if (L.qvec) {  // (all loads before the first use)
#pragma unroll
          for (int f = 0; f < kQ; ++f)
            if (const uint16_t *src = source(f)) x[f] = *reinterpret_cast<const uint4 *>(src);
        } else {
#pragma unroll
          for (int f = 0; f < kQ; ++f)
            if (const uint16_t *src = source(f))
              x[f] = make_uint4(src[0] | static_cast<uint32_t>(src[1]) << 16, src[2] | static_cast<uint32_t>(src[3]) << 16,
                                src[4] | static_cast<uint32_t>(src[5]) << 16, src[6] | static_cast<uint32_t>(src[7]) << 16);
        }
#pragma unroll
        for (int f = 0; f < kQ; ++f) {
          uint32_t w[4] = {x[f].x, x[f].y, x[f].z, x[f].w}, top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo_ = w[e] << 16 & 0x7FFFFFFFu, hi_ = w[e] & 0x7FFF0000u;
            if (lo_ < 0x7F800000u) top = max(top, lo_);
            if (hi_ < 0x7F800000u) top = max(top, hi_);
          }
#pragma unroll
          for (int b = kLanes / 2; b; b >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, b));
          const int shift = query_shift(top), r = w4 * 32 + f * kRowsPass + lane / kLanes, col = lane % kLanes;
          shifted |= shift != 0;
          if (col == 0) C.back[t * kRowsTile + r] = pow2(-shift);
          const float up = pow2(shift);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_f16(bf16_bits_to_float(w[e] & 0xFFFFu) * up, bf16_bits_to_float(w[e] >> 16) * up);
          *reinterpret_cast<uint4 *>(smem + Y::kQ + t * Y::kTile + (col >> 3) * (kRowsTile * 128) + r * 128 +
                                     (((col & 7) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        fence_before();
        mbar_arrive(&C.q_full);
      }
      shifted = __any_sync(0xFFFFFFFFu, shifted);  // (and the warp's entries of C.back are there)
      __syncwarp();
      // row `lane` of the warp's 32, then the lane's own four: g, g + 8, g + 16, g + 24
      const int g = lane >> 2, c = lane & 3;
      int my_token = -1, my_limit = 0x7FFFFFFF;
      {
        const int row = r0 + t * kRowsTile + w4 * 32 + lane;
        if (row < L.rows) {
          my_token = div_by(row, L.group);
          my_limit = prefix_limit(P, my_token);
          if (my_limit < 0) {  // nobody's row
            my_token = -1;
            my_limit = 0x7FFFFFFF;
          }
        }
      }
      const int low = __reduce_min_sync(0xFFFFFFFFu, my_limit);  // keys below it are seen by all rows of the warp
      const uint32_t s_addr = C.tmem + (static_cast<uint32_t>(w4 * 32) << 16) + t * 128;
      const uint32_t o_addr = s_addr + 256;
      constexpr uint32_t kHalf = 16u << 16;  // the warp's second 16 rows
      float m[4];
      Pair l[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        m[x] = -INFINITY;
        l[x] = pair(0.0f, 0.0f);
      }
      uint32_t nan_rows = 0;  // bit x: the row sees a value scale that is no number
      for (int i = 0; ok && i < n; ++i) {
        const int it = done_tiles + i;
        const Vectors &V = vec[it % kVectorSlots];
        ok = wait_warp(C, &C.vec_full[it % kVectorSlots], it / kVectorSlots & 1);
        if (t >= tiles) {  // (no rows: the factors' slot is handed back)
          if (ok && lane == 0) mbar_arrive(&C.vec_empty[it % kVectorSlots]);
          continue;
        }
        ok = ok && wait_warp(C, &C.s_full[t], (mine + i) & 1);
        if (!ok) break;
        fence_after();
        const int k0 = k_begin + i * kKeyTile;
        const uint32_t any_dead = V.dead[0] | V.dead[1] | V.dead[2] | V.dead[3];
        const uint32_t any_none = V.none[0] | V.none[1] | V.none[2] | V.none[3];
        const bool cut = any_dead || any_none || k0 + kKeyTile > low || shifted;
        const float over = fmaxf(V.top[0], V.top[1]);
        uint32_t s[2][64];  // rows g and g + 8 of each half of the warp's 32: the scores, then the exponents
        auto load_scores = [&]() {
          tmem_load_128(s_addr, s[0]);
          tmem_load_128(s_addr + kHalf, s[1]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_wait_load(s[0] + 16 * q);
            tmem_wait_load(s[1] + 16 * q);
          }
        };
        auto get = [&](int x, int j) {  // columns 8j + 2c, + 1 of row x
          return pair(__uint_as_float(s[x >> 1][j * 4 + (x & 1) * 2]), __uint_as_float(s[x >> 1][j * 4 + (x & 1) * 2 + 1]));
        };
        auto put = [&](int x, int j, float a, float b) {
          s[x >> 1][j * 4 + (x & 1) * 2] = __float_as_uint(a);
          s[x >> 1][j * 4 + (x & 1) * 2 + 1] = __float_as_uint(b);
        };
        load_scores();
        // Most tiles: every row sees all keys and has a maximum that holds.  One fused operation an exponent then (below
        // 2^24 its exact product differs from a rounded one by less than the 2^8 that a weight may grow).
        bool plain = !cut;
#pragma unroll
        for (int x = 0; x < 4; ++x) plain = plain && fabsf(m[x]) < 16777216.0f;
        plain = __all_sync(0xFFFFFFFFu, plain);
        if (plain) {
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 f = V.kc[j * 4 + c];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const Pair y = fma2(get(x, j), pair(f.x, f.y), pair(-m[x], -m[x]));
              put(x, j, lo(y), hi(y));
              top[x] = fmaxf(top[x], fmaxf(lo(y), hi(y)));
            }
          }
          plain = __all_sync(0xFFFFFFFFu, !(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) + over > kRaise));
          if (!plain) load_scores();  // (they are still there)
        }
        if (!plain) {
          // x, and its largest.  A product of its own, rounded: subtracting a maximum that equals it gives 0.
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          int limit[4];
          Pair back[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            limit[x] = __shfl_sync(0xFFFFFFFFu, my_limit, x * 8 + g);
            const float f = C.back[t * kRowsTile + w4 * 32 + x * 8 + g];
            back[x] = pair(f, f);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 f = V.kc[j * 4 + c];
            const uint32_t dead = V.dead[j >> 2] >> ((j & 3) * 8 + 2 * c);
            const int key = k0 + j * 8 + 2 * c;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const Pair y = mul2(mul2(get(x, j), pair(f.x, f.y)), back[x]);  // (the key's scale may keep it finite)
              const float a_ = key >= limit[x] || (dead & 1u) ? -INFINITY : lo(y);
              const float b_ = key + 1 >= limit[x] || (dead & 2u) ? -INFINITY : hi(y);
              put(x, j, a_, b_);
              top[x] = fmaxf(top[x], fmaxf(a_, b_));
            }
          }
          if (any_none) {  // the first such key decides which rows see one
            const int key = k0 + (V.none[0]   ? __ffs(V.none[0])
                                  : V.none[1] ? 32 + __ffs(V.none[1])
                                  : V.none[2] ? 64 + __ffs(V.none[2])
                                              : 96 + __ffs(V.none[3])) - 1;
#pragma unroll
            for (int x = 0; x < 4; ++x) nan_rows |= key < limit[x] ? 1u << x : 0u;
          }
          bool raise = false;
#pragma unroll
          for (int x = 0; x < 4; ++x) raise |= top[x] + over > m[x] + kRaise || (m[x] == -INFINITY && top[x] > -INFINITY);
          if (__any_sync(0xFFFFFFFFu, raise)) {  // (seldom after the first tiles)
            float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, r[4];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 f = V.vr[j * 4 + c];
              const Pair lv = pair(fmaxf(__log2f(fabsf(f.x)), kLeastUnits), fmaxf(__log2f(fabsf(f.y)), kLeastUnits));
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const Pair y = add2(get(x, j), lv);
                most[x] = fmaxf(most[x], fmaxf(lo(y), hi(y)));
              }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              most[x] = fmaxf(most[x], __shfl_xor_sync(0xFFFFFFFFu, most[x], 1));
              most[x] = fmaxf(most[x], __shfl_xor_sync(0xFFFFFFFFu, most[x], 2));
              const float next = most[x] > m[x] + kRaise || m[x] == -INFINITY ? most[x] : m[x];
              r[x] = m[x] == -INFINITY ? 1.0f : exp2_approx(m[x] - next);  // (without a maximum O and l are zeros or NaN)
              m[x] = next;
              l[x] = mul2(l[x], pair(r[x], r[x]));
            }
            if (i > 0) {
#pragma unroll
              for (int q = 0; q < D / 32; ++q)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  uint32_t o[16];
                  tmem_load_32(o_addr + half * kHalf + q * 32, o);
                  tmem_wait_load(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r[half * 2 + (e >> 1 & 1)]);
                  tmem_store_32(o_addr + half * kHalf + q * 32, o);
                }
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const Pair neg = m[x] == -INFINITY ? pair(0.0f, 0.0f) : pair(-m[x], -m[x]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const Pair y = add2(get(x, j), neg);
              put(x, j, lo(y), hi(y));
            }
          }
        }
        // the weights, sixteen columns of a half at a time
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[2][8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = V.vr[(q * 4 + j) * 4 + c];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const Pair y = get(x, q * 4 + j), w = pair(exp2_approx(lo(y)), exp2_approx(hi(y)));
              l[x] = add2(l[x], w);
              const Pair v = mul2(w, pair(f.x, f.y));
              p[x >> 1][j * 2 + (x & 1)] = pack_f16(lo(v), hi(v));
            }
          }
          tmem_store_pairs(s_addr + q * 16, p[0]);
          tmem_store_pairs(s_addr + kHalf + q * 16, p[1]);
        }
        tmem_wait_store();
        fence_before();
        mbar_arrive(&C.p_full[t]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.vec_empty[it % kVectorSlots]);
      }
      // the partial result: NaN from a CTA that has given up (its products may have ended early)
      if (ok) ok = wait_warp(C, &C.done, done_segments & 1) && !__any_sync(0xFFFFFFFFu, gave_up(C));
      fence_after();
      if (t < tiles) {
        int64_t at[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = r0 + t * kRowsTile + w4 * 32 + x * 8 + g;
          const int token = __shfl_sync(0xFFFFFFFFu, my_token, x * 8 + g);
          at[x] = token < 0 ? -1 : (static_cast<int64_t>(token) * P.Hq + h * P.group + row - token * P.group) * L.slots + slot;
          float sum = lo(l[x]) + hi(l[x]);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          if (c == 0 && at[x] >= 0)
            L.part_ml[at[x]] = ok ? make_float2(m[x], sum) : make_float2(-INFINITY, __uint_as_float(0x7FC00000u));
        }
#pragma unroll
        for (int q = 0; ok && q < D / 32; ++q)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[16];
            tmem_load_32(o_addr + half * kHalf + q * 32, o);
            tmem_wait_load(o);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int x = half * 2 + (e >> 1 & 1);
              const float by = nan_rows >> x & 1u ? __uint_as_float(0x7FC00000u) : kScaleUnit;
              if (at[x] >= 0)
                *reinterpret_cast<float2 *>(L.part_o + at[x] * D + q * 32 + (e >> 2) * 8 + 2 * c) =
                    make_float2(__uint_as_float(o[e]) * by, __uint_as_float(o[e + 1]) * by);
            }
          }
      }
      fence_before();
      done_tiles += n;
      ++done_segments;
      if (t < tiles) mine += n;
      u = tile_from(u + n);
    }
  } else if (warp < 10) {
    // -------------------------------------------------------------------
    // the keys' factors: keys lt and lt + 64 of every tile
    // -------------------------------------------------------------------
    const int lt = tid - kSoftmaxThreads;
    uint32_t bad = 0;
    bool ok = true;
    for (int u = u_begin; u < u_end;) {
      const Segment S = segment(u);
      const int h = S.h, n = S.n, k_begin = S.k_begin, k_end = S.k_end;
      const float *const kscale = P.c.k_scale + h * P.c.scale_head_stride;
      const float *const vscale = P.c.v_scale + h * P.c.scale_head_stride;
      float ks[2], vs[2];
      bool out[2];  // a key of the range whose page is outside the cache (those behind the range are no row's)
      int page[2];
      auto key_of = [&](int i, int e) { return k_begin + i * kKeyTile + lt + e * kVectorThreads; };
      auto pages = [&](int i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) page[e] = i < n && key_of(i, e) < k_end ? P.tables[div_by(key_of(i, e), L.page)] : -1;
      };
      auto scales = [&](int i) {  // of the tile whose pages are there
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = key_of(i, e);
          const bool in = i < n && k < k_end;
          out[e] = false;
          ks[e] = vs[e] = 0.0f;
          if (in && page[e] >= 0 && page[e] < P.c.num_blocks) {
            const int64_t at = page[e] * P.c.scale_block_stride +
                               (k - div_by(k, L.page) * P.c.block_size) * P.c.scale_token_stride;
            ks[e] = kscale[at];
            vs[e] = vscale[at];
          } else if (in) {
            out[e] = true;
            bad = SV_DATA_BAD_SLOT;
          }
        }
      };
      pages(0);
      scales(0);
      pages(1);
      const float c_all = P.scale * kLog2e;
      for (int i = 0; ok && i < n; ++i) {
        const int it = done_tiles + i, slot_v = it % kVectorSlots;
        ok = wait_warp(C, &C.vec_empty[slot_v], (it / kVectorSlots & 1) ^ 1);
        if (!ok) break;
        Vectors &V = vec[slot_v];
        float most = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = lt + e * kVectorThreads;
          const float v = vs[e];
          const bool number = fabsf(v) < INFINITY;
          if (number) most = fmaxf(most, fabsf(v));
          (r & 1 ? V.kc[r >> 1].y : V.kc[r >> 1].x) = ks[e] * c_all;
          (r & 1 ? V.vr[r >> 1].y : V.vr[r >> 1].x) = number && fabsf(v) >= kLeastScale ? v * (1.0f / kScaleUnit) : 0.0f;
          const uint32_t dead = __ballot_sync(0xFFFFFFFFu, out[e]), none = __ballot_sync(0xFFFFFFFFu, !number);
          if (lane == 0) {
            V.dead[r >> 5] = dead;
            V.none[r >> 5] = none;
          }
        }
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
        if (lane == 0) V.top[warp - 8] = log2f(fmaxf(__uint_as_float(top), kLeastScale) * (1.0f / kScaleUnit));
        mbar_arrive(&C.vec_full[slot_v]);
        scales(i + 1);
        pages(i + 2);
      }
      done_tiles += n;
      u = tile_from(u + n);
    }
    if (P.status && bad) atomicOr(P.status, static_cast<int>(bad));
  } else if (warp == 10) {
    // -------------------------------------------------------------------
    // copies
    // -------------------------------------------------------------------
    if (lane == 0) {
      bool ok = true;
      int issued = 0;  // K and V tiles alternate
      for (int u = u_begin; ok && u < u_end; u = tile_from(u + 1)) {
        const int item = u / L.period, h = item / L.tensor_tiles;
        const uint8_t *const image = L.image + (static_cast<int64_t>(h) * T + u - item * L.period) * 2 * Y::kTile;
        for (int v = 0; v < 2; ++v) {
          const int it = issued >> 1, st = it & 1;
          ok = wait(C, v ? &C.v_empty[st] : &C.k_empty[st], (it >> 1 & 1) ^ 1);
          if (!ok) break;
          uint64_t *full = v ? &C.v_full[st] : &C.k_full[st];
          mbar_arrive_expect_tx(full, Y::kTile);
          bulk_g2s(smem + (v ? Y::kV : Y::kK) + st * Y::kTile, image + v * Y::kTile, Y::kTile, full);
          ++issued;
        }
      }
      // (nobody else may wait for the last ones)
      for (int j = max(0, issued - 4); j < issued; ++j) {
        const int it = j >> 1;
        settle(C, j & 1 ? &C.v_full[it & 1] : &C.k_full[it & 1], it >> 1 & 1);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------------
    // the products
    // -------------------------------------------------------------------
    // The whole warp runs the loop, so addresses stay warp-uniform (one thread's own cost it 3700 cycles a tile to issue
    // 2050 cycles of products); one elected lane issues.
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, C.tmem, 0), base = smem_addr(smem);
    constexpr uint32_t kScores = product(kKeyTile, false), kOutputs = product(D, true);
    const uint64_t queries = operand(base + Y::kQ, 16), keys = operand(base + Y::kK, 16),
                   values = operand(base + Y::kV, kKeyTile * 128);
    const bool leader = elected();
    auto scores = [&](int t, int st) {
      const uint64_t a = queries + static_cast<uint64_t>(t * (Y::kTile >> 4)), b = keys + static_cast<uint64_t>(st * (Y::kTile >> 4));
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr int kBlock = (kRowsTile * 128) >> 4;
          const int at = (kk >> 2) * kBlock + (kk & 3) * 2;
          if (kk == 0)
            mma_ss<false>(tmem + t * 128, a + at, b + at, kScores);
          else
            mma_ss<true>(tmem + t * 128, a + at, b + at, kScores);
        }
        mma_commit(&C.s_full[t]);
      }
    };
    auto outputs = [&](int t, int st, bool add) {
      const uint64_t b = values + static_cast<uint64_t>(st * (Y::kTile >> 4));
      if (leader) {
        if (add)
          mma_ts<true>(tmem + 256 + t * 128, tmem + t * 128, b, kOutputs);
        else
          mma_ts<false>(tmem + 256 + t * 128, tmem + t * 128, b, kOutputs);
#pragma unroll
        for (int kk = 1; kk < kKeyTile / 16; ++kk)
          mma_ts<true>(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, b + kk * (2048 >> 4), kOutputs);
      }
    };
    auto commit = [&](uint64_t *bar) {
      if (leader) mma_commit(bar);
    };
    bool ok = true;
    int second = 0;  // key tiles of the second row tile so far
    for (int u = u_begin; u < u_end;) {
      const Segment S = segment(u);
      const int n = S.n, tiles = S.tiles;
      ok = ok && wait_warp(C, &C.q_full, done_segments & 1) &&
           wait_warp(C, &C.k_full[done_tiles & 1], done_tiles >> 1 & 1);
      if (ok) {
        fence_after();
        for (int t = 0; t < tiles; ++t) scores(t, done_tiles & 1);
        commit(&C.k_empty[done_tiles & 1]);
      }
      for (int i = 0; ok && i < n; ++i) {
        const int it = done_tiles + i, st = it & 1, sn = st ^ 1;
        ok = wait_warp(C, &C.v_full[st], it >> 1 & 1);
        for (int t = 0; ok && t < tiles; ++t) {
          ok = wait_warp(C, &C.p_full[t], (t ? second + i : it) & 1, P.expire);
          if (!ok) break;
          fence_after();
          outputs(t, st, i > 0);
          if (t == tiles - 1) commit(&C.v_empty[st]);
          if (i + 1 < n) {
            if (t == 0) {
              ok = wait_warp(C, &C.k_full[sn], (it + 1) >> 1 & 1);
              if (!ok) break;
              fence_after();
            }
            scores(t, sn);
            if (t == tiles - 1) commit(&C.k_empty[sn]);
          }
        }
      }
      commit(&C.done);
      settle(C, &C.done, done_segments & 1);
      __syncwarp();
      done_tiles += n;
      ++done_segments;
      if (tiles == 2) second += n;
      u = tile_from(u + n);
    }
    __syncwarp();
    fence_before();
  }
  __syncthreads();
  fence_after();
  if (warp == 11) {
    tmem_free(C.tmem, 512);
    if (lane == 0 && gave_up(C) && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_COPY_TIMEOUT));
  }
}

template <int D, int FMT>
cudaError_t launch(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(L.image_tiles), static_cast<unsigned>(p.c.num_kv_heads), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, unpack_kernel<D, FMT>, p, L);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((L.units + L.units_cta - 1) / L.units_cta));
  cfg.blockDim = dim3(kPrefixThreads);
  cfg.dynamicSmemBytes = Smem<D>::kBytes;
  return cudaLaunchKernelEx(&cfg, prefix_kernel<D>, p, L);
}
template <int D>
cudaError_t enable() {
  return cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
}

}  // namespace

cudaError_t enable_prefix_kernels() {
  const cudaError_t e = enable<128>();
  return e != cudaSuccess ? e : enable<64>();
}

cudaError_t launch_prefix(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  const bool i8 = p.c.format == SV_CACHE_INT8;
  if (p.c.head_dim == 128) return i8 ? launch<128, SV_CACHE_INT8>(p, L, stream) : launch<128, SV_CACHE_E4M3>(p, L, stream);
  return i8 ? launch<64, SV_CACHE_INT8>(p, L, stream) : launch<64, SV_CACHE_E4M3>(p, L, stream);
}

}  // namespace sv
