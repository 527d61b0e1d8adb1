// sv_logprobs.cu -- log-probabilities of the committed tokens, with rank,
// entropy and the largest alternatives.
//
// One CTA (or, for few tokens, a cluster of up to eight) per token place
// (i, m), one pass over the row.  With d = (logit - reference) * (log2 e / T) a
// thread sums z = sum 2^d and zx = sum 2^d d and counts the logits above the
// token's; the reference is raised when a value passes it by 2^16, so the loop
// neither rescales nor waits for another thread.  Then
//   log p = (logit - reference) / T - ln z,   entropy = ln z - ln 2 zx / z.
//
// The K largest come from block maxima: a block is 2 KB of the row, four
// 16-byte vectors a lane, and its largest key takes one warp reduction.  Order
// blocks by (largest key, lower block first).  Every element of a block that
// is not among the first K has K elements before it in the order (larger
// value, lower index first) -- the K blocks' maxima -- so the K largest
// elements lie in those K blocks, whatever ties there are.  They are read
// again (from L2, K * 2 KB a row); elements that reach the last chosen block's
// maximum -- a few more than K, unless there are many ties -- are ranked by
// counting.  A CTA with fewer than K blocks (short rows, or a row cut over a
// cluster) takes the K-th largest maximum of parts of blocks instead: no
// element below it is among the K largest, and the CTA's few blocks are all
// read again.  (With every element a candidate, 64 tokens of V = 151936 with 20
// alternatives took 82 us, now 21; two of V = 92471 with 32 40, now 17.)
//
// Bound by HBM: the row is read once, 512 requests' committed tokens (2641
// rows of 151936 bf16 logits) are 0.80 GB and take 161 us with 20 alternatives,
// 5.0 TB/s or 74 % of the copy rate; without alternatives 130 us.  Fetching
// instructions stalled it most: ragged vectors, candidates and a second copy of
// the loop's body in line cost 25 us together, so the loop is kept short.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

constexpr int kUnroll = 4;        // vectors of a lane in a group: a group is 2 KB, and a block one group
constexpr int kGroup = 32 * kUnroll;
constexpr int kMaxBlocks = 2048;  // block maxima that a CTA keeps; above 4 MB of row a CTA, blocks are several groups
constexpr int kCandidates = 256;  // ranked by counting, one a thread; more (ties) are sorted into lists
constexpr int kMaxCluster = 8;
constexpr float kRaiseBy = 16.0f;
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

struct Sums {
  float ref, z, zx;  // reference logit, sum 2^d, sum 2^d d
  uint32_t above, bad;
};

struct LogprobsSmem {
  unsigned long long lists[kWarps][SV_MAX_TOP_LOGPROBS];  // the warps' largest (key, lower index first)
  unsigned long long best[SV_MAX_TOP_LOGPROBS];           // the CTA's, read by the cluster's first
  unsigned long long candidates[kCandidates];
  Sums warp_sums[kWarps], sums;
  alignas(16) uint32_t block_key[kMaxBlocks];
  int chosen[SV_MAX_TOP_LOGPROBS];
  float floor;         // largest element of the last chosen block
  int count;           // candidates
};

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 1.0 in each half where a > b.
__device__ __forceinline__ uint32_t above_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The number that an ordered key stands for (-0 comes back as +0).
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Sums with another reference; c = log2 e / T.
__device__ __forceinline__ void rebase(Sums &s, float ref, float c) {
  if (s.ref == ref) return;
  if (s.ref == -INFINITY) {
    s.ref = ref;
    return;  // (nothing summed yet)
  }
  const float by = (s.ref - ref) * c, r = exp2_approx(by);
  s.zx = r * fmaf(by, s.z, s.zx);
  if (!(r > 0.0f)) s.zx = 0.0f;
  s.z *= r;
  s.ref = ref;
}
__device__ __forceinline__ void merge(Sums &a, Sums b, float c) {
  const float ref = fmaxf(a.ref, b.ref);
  rebase(a, ref, c);
  rebase(b, ref, c);
  a.z += b.z;
  a.zx += b.zx;
  a.above += b.above;
  a.bad |= b.bad;
}

// A warp's sums together, in every lane: the common reference first, so that a lane changes its own once.
__device__ __forceinline__ void merge_warp(Sums &s, float c) {
  rebase(s, logit_of(__reduce_max_sync(0xFFFFFFFFu, ordered_bits(s.ref))), c);
#pragma unroll
  for (int b = 16; b; b >>= 1) {
    s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, b);
    s.zx += __shfl_xor_sync(0xFFFFFFFFu, s.zx, b);
  }
  s.above = __reduce_add_sync(0xFFFFFFFFu, s.above);
  s.bad = __reduce_or_sync(0xFFFFFFFFu, s.bad);
}

__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
  const uint32_t h = static_cast<uint32_t>(v >> 32), top = __reduce_max_sync(0xFFFFFFFFu, h);
  const uint32_t l = __reduce_max_sync(0xFFFFFFFFu, h == top ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(top) << 32 | l;
}

// A vector that the row does not fill, from its elements x .. ; the rest is -inf.  (Not inlined: four of them at each of
// the loop's loads were most of the kernel's instructions, and fetching those stalled it.)
template <bool BF16>
__device__ __noinline__ uint4 edge_vector(const uint8_t *at, int x, int V) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (BF16) {
      const uint16_t *p = reinterpret_cast<const uint16_t *>(at) + 2 * e;
      const int y = x + 2 * e;
      w[e] = (y >= 0 && y < V ? p[0] : 0xFF80u) | static_cast<uint32_t>(y + 1 >= 0 && y + 1 < V ? p[1] : 0xFF80u) << 16;
    } else {
      const uint32_t *p = reinterpret_cast<const uint32_t *>(at) + e;
      const int y = x + e;
      w[e] = y >= 0 && y < V ? *p : 0xFF800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The row as 16-byte vectors: vector v holds elements v * kPer - shift ..
template <bool BF16>
struct Row {
  static constexpr int kPer = BF16 ? 8 : 4;
  const uint8_t *base;  // of vector 0 (the 16-byte boundary at or below the row)
  int shift, V;
  __device__ __forceinline__ int vectors() const { return (V + shift + kPer - 1) / kPer; }
  __device__ __forceinline__ uint4 load(int v) const {
    const int x = v * kPer - shift;
    const uint8_t *at = base + static_cast<int64_t>(v) * 16;
    if (x >= 0 && x + kPer <= V) return ld_stream_u4(reinterpret_cast<const uint4 *>(at));
    return edge_vector<BF16>(at, x, V);
  }
};

__device__ __forceinline__ float word_of(const uint4 &r, int e) {
  return __uint_as_float(e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w);
}
template <bool BF16>
__device__ __forceinline__ float element(const uint4 &r, int e) {
  if (!BF16) return word_of(r, e);
  const uint32_t w = __float_as_uint(word_of(r, e >> 1));
  return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
}

template <bool BF16>
__device__ __forceinline__ float largest(const uint4 &r) {
  if (!BF16) return max_nan(max_nan(word_of(r, 0), word_of(r, 1)), max_nan(word_of(r, 2), word_of(r, 3)));
  const uint32_t t = max_nan_bf16x2(max_nan_bf16x2(r.x, r.y), max_nan_bf16x2(r.z, r.w));
  return max_nan(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u));
}

// A block maximum's place in the order (largest key, lower block first).  A
// bf16's key has 16 bits: the block's number goes below them, and one
// comparison decides; an fp32's needs the block as well where keys are equal.
template <bool BF16>
__device__ __forceinline__ uint32_t block_order(uint32_t key, int block) {
  return BF16 ? (key & 0xFFFF0000u) | static_cast<uint32_t>(0xFFFF - block) : key;
}
static_assert(kMaxBlocks <= 0x10000, "a block's number fits 16 bits");
template <bool BF16>
__device__ __forceinline__ bool block_before(uint32_t key, int block, uint32_t other, int other_block) {
  return BF16 ? key > other : key > other || (key == other && block < other_block);
}

// The elements of a vector at x0 .. that are the row's and reach the floor, among the candidates.  (Not inlined: there
// are a few calls a row, from four places.)
template <bool BF16>
__device__ __noinline__ void take_candidates(LogprobsSmem &sm, uint4 r, int x0, int V, float floor) {
  for (int e = 0; e < Row<BF16>::kPer; ++e) {
    const float v = element<BF16>(r, e);
    if (x0 + e < 0 || x0 + e >= V || !(v >= floor)) continue;
    const int to = atomicAdd(&sm.count, 1);
    if (to < kCandidates) sm.candidates[to] = pack_key(v, static_cast<uint32_t>(x0 + e));
  }
}

// The maxima of a group's parts: of each lane's vectors, or of each four lanes'.
template <bool BF16>
__device__ __noinline__ void part_maxima(LogprobsSmem &sm, uint32_t key, int gi, int parts) {
  const int lane = threadIdx.x & 31;
  if (parts == 8) {
    key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, 1));
    key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, 2));
    if (lane & 3) return;
  }
  const int b = gi * parts + lane * parts / 32;
  sm.block_key[b] = block_order<BF16>(key, b);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 3) logprobs_kernel(const LogprobsParams P) {
  pdl_enter();
  __shared__ LogprobsSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int64_t place = blockIdx.x / C;
  const int i = static_cast<int>(place / (P.G + 1)), m = static_cast<int>(place % (P.G + 1));
  const int32_t tok = P.tokens[place];
  uint32_t bits = 0;
  int64_t s;
  int g;
  const float temp = P.temperature ? P.temperature[i] : 1.0f;
  if (!request_range(P.cu, i, P.G, P.T, s, g) || (tok != -1 && m > g)) {
    bits = SV_DATA_BAD_CU;
  } else if (tok != -1) {
    if (tok < 0 || tok >= P.V) bits |= SV_DATA_BAD_DRAFT_ID;
    if (!temperature_ok(temp)) bits |= SV_DATA_BAD_PARAM;
  }
  if (tok == -1 || bits) {  // (the same for the whole cluster)
    if (rank == 0) {
      const bool skip = tok == -1 || (bits & SV_DATA_BAD_CU);
      const float none = skip ? 0.0f : __uint_as_float(0x7FC00000u);
      if (tid == 0) {
        P.logprobs[place] = none;
        if (P.entropy) P.entropy[place] = none;
        if (P.ranks) P.ranks[place] = -1;
        if (bits && P.status) atomicOr(P.status, static_cast<int>(bits));
      }
      if (tid < P.K) {
        P.top_ids[place * P.K + tid] = -1;
        P.top_logprobs[place * P.K + tid] = none;
      }
    }
    return;
  }
  const int64_t at = (s + i + m) * P.row_stride * (BF16 ? 2 : 4);
  const uint8_t *const row_ptr = static_cast<const uint8_t *>(P.logits) + at;
  Row<BF16> row;
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row_ptr) & 15u);
  row.base = row_ptr - off;
  row.shift = static_cast<int>(off) / (BF16 ? 2 : 4);
  row.V = P.V;
  const float mine = BF16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t *>(row_ptr)[tok])
                          : reinterpret_cast<const float *>(row_ptr)[tok];
  const uint32_t mine2 = (__float_as_uint(mine) >> 16) * 0x10001u;  // (bf16 rows)
  const float t = temp == 0.0f ? 1.0f : temp, c = kLog2E / t;

  // ---- the pass over this CTA's vectors ----
  const int nv = row.vectors();
  const int chunk = (nv + C - 1) / C + kGroup - 1 & ~(kGroup - 1);
  const int v0 = static_cast<int>(min(static_cast<int64_t>(nv), static_cast<int64_t>(rank) * chunk));
  const int v1 = min(nv, v0 + chunk);
  const int groups = (v1 - v0 + kGroup - 1) / kGroup;
  const int per_block = max(1, (groups + kMaxBlocks - 1) / kMaxBlocks);
  // fewer blocks than alternatives: parts of them, 32 or 8 of a group, give the floor
  const int parts = P.K <= groups ? 0 : groups <= kThreads / 32 ? 32 : 8;
  const int blocks = parts ? groups * parts : (groups + per_block - 1) / per_block;
  if (P.K) {
    if (per_block > 1)
      for (int b = tid; b < blocks; b += kThreads) sm.block_key[b] = 0;
    if (tid < 4 && blocks + tid < kMaxBlocks) sm.block_key[blocks + tid] = 0;  // (read four at a time)
    if (tid == 0) sm.count = 0;
    if (per_block > 1) __syncthreads();
  }
  // groups [g_lo, g_hi) hold full vectors only
  const int g_lo = row.shift && rank == 0 ? 1 : 0;
  const int g_hi = (min(v1, (P.V + row.shift) / Row<BF16>::kPer) - v0) / kGroup;
  const uint4 *const mine_v = reinterpret_cast<const uint4 *>(row.base) + v0 + lane;
  constexpr uint32_t kNone = BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  auto fetch = [&](int gi, uint4 raw[kUnroll]) {
    if (gi >= g_lo && gi < g_hi) {
      const uint4 *p = mine_v + static_cast<int64_t>(gi) * kGroup;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) raw[u] = ld_stream_u4(p + u * 32);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = v0 + gi * kGroup + u * 32 + lane;
        raw[u] = make_uint4(kNone, kNone, kNone, kNone);
        if (gi < groups && v < v1) raw[u] = row.load(v);
      }
    }
  };
  Sums sum{-INFINITY, 0.0f, 0.0f, 0u, 0u};
  Pair z = pair(0.0f, 0.0f), zx = z;
  bool bad = false;
  auto take = [&](int gi, const uint4 raw[kUnroll]) {
    float top;
    if (BF16) {
      uint32_t t2 = raw[0].x, n2 = 0;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint4 &v = raw[u];
        t2 = max_nan_bf16x2(t2, max_nan_bf16x2(max_nan_bf16x2(v.x, v.y), max_nan_bf16x2(v.z, v.w)));
        n2 = add_bf16x2(n2, add_bf16x2(add_bf16x2(above_bf16x2(v.x, mine2), above_bf16x2(v.y, mine2)),
                                       add_bf16x2(above_bf16x2(v.z, mine2), above_bf16x2(v.w, mine2))));
      }
      top = max_nan(__uint_as_float(t2 << 16), __uint_as_float(t2 & 0xFFFF0000u));
      // (counts of up to 16 a half, exact)
      sum.above += static_cast<uint32_t>(__uint_as_float(n2 << 16) + __uint_as_float(n2 & 0xFFFF0000u));
    } else {
      top = word_of(raw[0], 0);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          top = max_nan(top, word_of(raw[u], e));
          sum.above += word_of(raw[u], e) > mine ? 1u : 0u;
        }
    }
    const uint32_t key = ordered_bits(top);
    bad |= !(top < INFINITY);  // +inf, or NaN, which the maxima hand on (and which no key orders)
    if (parts) {
      part_maxima<BF16>(sm, key, gi, parts);
    } else if (P.K) {
      const uint32_t k = __reduce_max_sync(0xFFFFFFFFu, key);
      if (lane == 0) {
        if (per_block == 1)
          sm.block_key[gi] = block_order<BF16>(k, gi);
        else
          atomicMax(&sm.block_key[gi / per_block], block_order<BF16>(k, gi / per_block));
      }
    }
    if ((top - sum.ref) * c > kRaiseBy && top > -INFINITY) {  // (seldom after the first)
      sum.z = lo(z) + hi(z);
      sum.zx = lo(zx) + hi(zx);
      rebase(sum, top, c);
      z = pair(sum.z, 0.0f);
      zx = pair(sum.zx, 0.0f);
    }
    if (sum.ref > -INFINITY) {
      const Pair neg = pair(-sum.ref, -sum.ref), cc = pair(c, c);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int e = 0; e < Row<BF16>::kPer; e += 2) {
          Pair d = mul2(add2(pair(element<BF16>(raw[u], e), element<BF16>(raw[u], e + 1)), neg), cc);
          // (a masked entry: its 2^d is 0, and so is 0 * d)
          d = pair(fmaxf(lo(d), -200.0f), fmaxf(hi(d), -200.0f));
          const Pair w = pair(exp2_approx(lo(d)), exp2_approx(hi(d)));
          z = add2(z, w);
          zx = fma2(w, d, zx);
        }
    }
  };
  // a group is fetched while the one before it is taken (one copy of the code: two in turn, without the moves, are twice
  // the instructions to fetch)
  uint4 now[kUnroll], next[kUnroll];
  fetch(warp, now);
#pragma unroll 1
  for (int gi = warp; gi < groups; gi += kWarps) {
    fetch(gi + kWarps, next);
    take(gi, now);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) now[u] = next[u];
  }
  sum.bad = bad;
  sum.z = lo(z) + hi(z);
  sum.zx = lo(zx) + hi(zx);
  merge_warp(sum, c);
  if (lane == 0) sm.warp_sums[warp] = sum;
  __syncthreads();

  // ---- the K blocks with the largest maxima, then their K largest elements ----
  const int K = P.K, kb = min(K, blocks);
  if (warp == 0) {  // (lanes 8 and up hold nothing)
    Sums a = lane < kWarps ? sm.warp_sums[lane] : Sums{-INFINITY, 0.0f, 0.0f, 0u, 0u};
    merge_warp(a, c);
    if (lane == 0) sm.sums = a;
  }
  if (K) {
    for (int b = tid; b < blocks; b += kThreads) {
      const uint32_t key = sm.block_key[b];
      int before = 0;
      for (int j = 0; j < blocks; j += 4) {
        const uint4 k = *reinterpret_cast<const uint4 *>(&sm.block_key[j]);
        before += block_before<BF16>(k.x, j, key, b) + block_before<BF16>(k.y, j + 1, key, b) +
                  block_before<BF16>(k.z, j + 2, key, b) + block_before<BF16>(k.w, j + 3, key, b);
      }
      if (before < kb) sm.chosen[before] = b;
      // (a negative bf16's key has ones in its lower half)
      if (before == K - 1) sm.floor = logit_of(!BF16 ? key : key & 0x80000000u ? key & 0xFFFF0000u : key | 0xFFFFu);
    }
    __syncthreads();
    const float floor = kb == K ? sm.floor : -INFINITY;
    // elements that reach the floor
    auto fetch_again = [&](int gi, int u) {
      const int v = v0 + gi * kGroup + u * 32 + lane;
      return gi < groups && v < v1 ? row.load(v) : make_uint4(kNone, kNone, kNone, kNone);
    };
    auto reaching = [&](int gi, int u, const uint4 &r) {  // bit e: element e of the vector is the row's and reaches it
      const int v = v0 + gi * kGroup + u * 32 + lane, x0 = v * Row<BF16>::kPer - row.shift;
      uint32_t left = 0;
      if (gi < groups && v < v1 && largest<BF16>(r) >= floor) {  // (for one lane in dozens)
#pragma unroll
        for (int e = 0; e < Row<BF16>::kPer; ++e)
          if (x0 + e >= 0 && x0 + e < P.V && element<BF16>(r, e) >= floor) left |= 1u << e;
      }
      return left;
    };
    const int again = parts ? groups : kb;  // (parts cross in index order: all groups are looked at)
    for (int k = warp; k < again; k += kWarps)
      for (int p = 0; p < per_block; ++p) {
        const int gi = parts ? k : sm.chosen[k] * per_block + p;
        uint4 r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) r[u] = fetch_again(gi, u);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (gi < groups && largest<BF16>(r[u]) >= floor)  // (for one lane in dozens)
            take_candidates<BF16>(sm, r[u], (v0 + gi * kGroup + u * 32 + lane) * Row<BF16>::kPer - row.shift, P.V, floor);
      }
    if (tid < SV_MAX_TOP_LOGPROBS) sm.best[tid] = 0;
    __syncthreads();
    const int count = sm.count;
    if (count <= kCandidates) {  // (their order in the array does not matter: keys are all different)
      if (tid < count) {
        const unsigned long long key = sm.candidates[tid];
        int before = 0;
        for (int j = 0; j < count; ++j) before += sm.candidates[j] > key;
        if (before < K) sm.best[before] = key;
      }
    } else {
      // many ties: every warp sorts its blocks' elements into a list of K (lane k holds the k-th), the lists are merged
      unsigned long long list = 0;
      for (int k = warp; k < again; k += kWarps)
        for (int p = 0; p < per_block; ++p)
          for (int u = 0; u < kUnroll; ++u) {
            const int gi = parts ? k : sm.chosen[k] * per_block + p;
            const uint4 r = fetch_again(gi, u);
            uint32_t left = reaching(gi, u, r);
            const int x0 = (v0 + gi * kGroup + u * 32 + lane) * Row<BF16>::kPer - row.shift;
            for (;;) {
              unsigned long long best = 0;
              int at_e = 0;
#pragma unroll
              for (int e = 0; e < Row<BF16>::kPer; ++e) {
                const unsigned long long key = pack_key(element<BF16>(r, e), static_cast<uint32_t>(x0 + e));
                if ((left >> e & 1u) && key > best) {
                  best = key;
                  at_e = e;
                }
              }
              const unsigned long long top = warp_max64(best);
              if (top <= __shfl_sync(0xFFFFFFFFu, list, K - 1)) break;  // (0 too: nothing left)
              if (best == top) left &= ~(1u << at_e);
              const int pos = __popc(__ballot_sync(0xFFFFFFFFu, list > top));
              const unsigned long long before = __shfl_up_sync(0xFFFFFFFFu, list, 1);
              list = lane > pos ? before : lane == pos ? top : list;
            }
          }
      if (lane < K) sm.lists[warp][lane] = list;
      __syncthreads();
      if (warp == 0) {
        // lane l takes list l % 8 from its (l / 8)-th entry on, every fourth: K rounds pick the largest head
        int at_l = lane >> 3;
        const unsigned long long *mine_l = sm.lists[lane & 7];
        unsigned long long head = at_l < K ? mine_l[at_l] : 0ull;
        for (int k = 0; k < K; ++k) {
          const unsigned long long top = warp_max64(head);
          if (lane == 0) sm.best[k] = top;
          if (head == top && top) {
            at_l += 4;
            head = at_l < K ? mine_l[at_l] : 0ull;
          }
        }
      }
    }
  }
  __syncthreads();

  // ---- the cluster's first CTA joins and writes ----
  if (C > 1) cluster_sync();
  if (rank == 0 && warp == 0) {
    Sums a = sm.sums;
    for (int r = 1; r < C; ++r) {
      Sums b;
      const uint32_t src = map_to_rank(smem_addr(&sm.sums), r);
      b.ref = __uint_as_float(ld_dsmem_u32(src));
      b.z = __uint_as_float(ld_dsmem_u32(src + 4));
      b.zx = __uint_as_float(ld_dsmem_u32(src + 8));
      b.above = ld_dsmem_u32(src + 12);
      b.bad = ld_dsmem_u32(src + 16);
      merge(a, b, c);
    }
    bad = a.bad || a.ref == -INFINITY;
    const float nan = __uint_as_float(0x7FC00000u), lnz = logf(a.z);
    // the k-th largest of the CTAs' lists (each in order): lane l takes CTA l % C from entry l / C on, every (32 / C)-th
    unsigned long long taken = 0;
    if (C == 1) {
      if (lane < K) taken = sm.best[lane];
    } else if (K) {
      const int step = 32 / C, who = lane % C;
      int next = lane / C;
      const uint32_t list = map_to_rank(smem_addr(sm.best), who);
      unsigned long long head = next < K ? ld_dsmem_u64(list + next * 8) : 0ull;
      for (int k = 0; k < K; ++k) {
        const unsigned long long top = warp_max64(head);
        if (lane == k) taken = top;
        if (head == top && top) {
          next += step;
          head = next < K ? ld_dsmem_u64(list + next * 8) : 0ull;
        }
      }
    }
    if (lane < K) {
      const uint32_t x = key_index(taken);
      const float v = bad ? 0.0f : logit_of(static_cast<uint32_t>(taken >> 32));
      P.top_ids[place * K + lane] = bad ? -1 : static_cast<int32_t>(x);
      P.top_logprobs[place * K + lane] = bad ? nan : (v - a.ref) / t - lnz;
    }
    if (lane == 0) {
      P.logprobs[place] = bad ? nan : (mine - a.ref) / t - lnz;
      if (P.entropy) P.entropy[place] = bad ? nan : lnz - a.zx / a.z * kLn2F;
      if (P.ranks) P.ranks[place] = bad ? -1 : 1 + static_cast<int32_t>(a.above);
      if (bad && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_VALUES));
    }
  }
  if (C > 1) cluster_sync();  // (the first CTA has read the others' shared memory)
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams &p, bool bf16, int num_sms, cudaStream_t stream) {
  const int64_t places = static_cast<int64_t>(p.N) * (p.G + 1);
  // Rows are split over a cluster while the call has fewer than two CTAs per
  // SM and a CTA would keep at least 8 KB of the row.
  int cluster = 1;
  while (cluster < kMaxCluster && places * cluster < 2LL * num_sms &&
         static_cast<int64_t>(p.V) * (bf16 ? 2 : 4) / (2 * cluster) >= 8192)
    cluster *= 2;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(places * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, static_cast<unsigned>(cluster), p.pdl);
  return cudaLaunchKernelEx(&cfg, bf16 ? logprobs_kernel<true> : logprobs_kernel<false>, p);
}

}  // namespace sv
