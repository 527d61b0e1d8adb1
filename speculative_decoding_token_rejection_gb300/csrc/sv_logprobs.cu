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
// The K largest come from block maxima: a block is 512 bytes of the row, one
// 16-byte vector a lane, and its largest key takes one warp reduction.  Order
// blocks by (largest key, lower block first).  Every element of a block that
// is not among the first K has K elements before it in the order (larger
// value, lower index first) -- the K blocks' maxima -- so the K largest
// elements lie in those K blocks, whatever ties there are.  They are read
// again (from L2), K * 512 bytes a row.
//
// Bound by HBM: the row is read once, 512 requests' committed tokens (2641
// rows of 151936 bf16 logits) are 0.80 GB.  About seven instructions an element, one
// of them an exponential.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

constexpr int kMaxBlocks = 2048;  // block maxima that a CTA keeps; longer chunks have longer blocks
constexpr int kUnroll = 4;        // vectors in flight per thread
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
  Sums warp_sums[kWarps], sums;
  uint32_t block_key[kMaxBlocks];
  int chosen[SV_MAX_TOP_LOGPROBS];
  uint32_t floor_key;  // key of the last chosen block
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

__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
  const uint32_t h = static_cast<uint32_t>(v >> 32), top = __reduce_max_sync(0xFFFFFFFFu, h);
  const uint32_t l = __reduce_max_sync(0xFFFFFFFFu, h == top ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(top) << 32 | l;
}

// The row as 16-byte vectors: vector v holds elements v * kPer - shift ..
template <bool BF16>
struct Row {
  static constexpr int kPer = BF16 ? 8 : 4;
  const uint8_t *base;  // of vector 0 (the 16-byte boundary at or below the row)
  int shift, V;
  __device__ __forceinline__ int vectors() const { return (V + shift + kPer - 1) / kPer; }
  // A vector that the row does not fill is put together from its elements; the rest is -inf.
  __device__ __forceinline__ uint4 load(int v) const {
    const int x = v * kPer - shift;
    if (x >= 0 && x + kPer <= V) return ld_stream_u4(reinterpret_cast<const uint4 *>(base) + v);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (BF16) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + static_cast<int64_t>(v) * kPer + 2 * e;
        const int y = x + 2 * e;
        w[e] = (y >= 0 && y < V ? p[0] : 0xFF80u) | static_cast<uint32_t>(y + 1 >= 0 && y + 1 < V ? p[1] : 0xFF80u) << 16;
      } else {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(base) + static_cast<int64_t>(v) * kPer + e;
        const int y = x + e;
        w[e] = y >= 0 && y < V ? *p : 0xFF800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobsParams P) {
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
  const int chunk = ((nv + C - 1) / C + 31) & ~31;  // whole warps' worth
  const int v0 = rank * chunk, v1 = min(nv, v0 + chunk);
  const int steps = v1 > v0 ? (v1 - v0 + 31) / 32 : 0;                 // of 32 vectors
  const int per_block = (steps + kMaxBlocks - 1) / kMaxBlocks;         // steps a block (1 for all but huge rows)
  const int blocks = steps ? (steps + per_block - 1) / per_block : 0;
  Sums sum{-INFINITY, 0.0f, 0.0f, 0u, 0u};
  Pair z = pair(0.0f, 0.0f), zx = z;
  float above_f = 0.0f;
  for (int b0 = warp; b0 < blocks; b0 += kWarps * kUnroll) {
    uint32_t key[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) key[u] = 0;
    for (int p = 0; p < per_block; ++p) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int b = b0 + u * kWarps, v = v0 + (b * per_block + p) * 32 + lane;
        raw[u] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
        if (!BF16) raw[u] = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
        if (b < blocks && v < v1) raw[u] = row.load(v);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint4 &r = raw[u];
        float top;
        if (BF16) {
          const uint32_t t2 = max_nan_bf16x2(max_nan_bf16x2(r.x, r.y), max_nan_bf16x2(r.z, r.w));
          top = max_nan(__uint_as_float(t2 << 16), __uint_as_float(t2 & 0xFFFF0000u));
          const uint32_t n2 = add_bf16x2(add_bf16x2(above_bf16x2(r.x, mine2), above_bf16x2(r.y, mine2)),
                                         add_bf16x2(above_bf16x2(r.z, mine2), above_bf16x2(r.w, mine2)));
          above_f += __uint_as_float(n2 << 16) + __uint_as_float(n2 & 0xFFFF0000u);
        } else {
          top = max_nan(max_nan(word_of(r, 0), word_of(r, 1)), max_nan(word_of(r, 2), word_of(r, 3)));
#pragma unroll
          for (int e = 0; e < 4; ++e) above_f += word_of(r, e) > mine ? 1.0f : 0.0f;
        }
        if (!(top < INFINITY)) sum.bad = 1;  // NaN or +inf
        key[u] = max(key[u], ordered_bits(top));
        if ((top - sum.ref) * c > kRaiseBy) {  // (seldom after the first)
          if (top > -INFINITY) {
            sum.z = lo(z) + hi(z);
            sum.zx = lo(zx) + hi(zx);
            rebase(sum, top, c);
            z = pair(sum.z, 0.0f);
            zx = pair(sum.zx, 0.0f);
          }
        }
        const Pair neg = pair(-sum.ref, -sum.ref), cc = pair(c, c);
        if (sum.ref > -INFINITY) {
#pragma unroll
          for (int e = 0; e < Row<BF16>::kPer; e += 2) {
            Pair d = mul2(add2(pair(element<BF16>(r, e), element<BF16>(r, e + 1)), neg), cc);
            // (a masked entry: its 2^d is 0, and so is 0 * d)
            d = pair(fmaxf(lo(d), -200.0f), fmaxf(hi(d), -200.0f));
            const Pair w = pair(exp2_approx(lo(d)), exp2_approx(hi(d)));
            z = add2(z, w);
            zx = fma2(w, d, zx);
          }
        }
      }
    }
    if (P.K) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t k = __reduce_max_sync(0xFFFFFFFFu, key[u]);
        if (lane == 0 && b0 + u * kWarps < blocks) sm.block_key[b0 + u * kWarps] = k;
      }
    }
    sum.above += static_cast<uint32_t>(above_f);
    above_f = 0.0f;
  }
  sum.z = lo(z) + hi(z);
  sum.zx = lo(zx) + hi(zx);
#pragma unroll
  for (int b = 16; b; b >>= 1) {
    Sums o;
    o.ref = __shfl_xor_sync(0xFFFFFFFFu, sum.ref, b);
    o.z = __shfl_xor_sync(0xFFFFFFFFu, sum.z, b);
    o.zx = __shfl_xor_sync(0xFFFFFFFFu, sum.zx, b);
    o.above = __shfl_xor_sync(0xFFFFFFFFu, sum.above, b);
    o.bad = __shfl_xor_sync(0xFFFFFFFFu, sum.bad, b);
    merge(sum, o, c);
  }
  if (lane == 0) sm.warp_sums[warp] = sum;
  __syncthreads();

  // ---- the K blocks with the largest maxima, then their K largest elements ----
  const int K = P.K, kb = min(K, blocks);
  if (warp == 0) {
    if (lane == 0) {
      Sums a = sm.warp_sums[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) merge(a, sm.warp_sums[w], c);
      sm.sums = a;
    }
    if (K) {
      // a lane keeps blocks lane, lane + 32, ...; its best is found again when it has been taken
      auto lane_best = [&](uint32_t &key, uint32_t &block) {
        key = 0;
        block = 0xFFFFFFFFu;
        for (int b = lane; b < blocks; b += 32)
          if (sm.block_key[b] > key) {  // (the lower block stays among equal keys)
            key = sm.block_key[b];
            block = b;
          }
      };
      uint32_t key, block;
      lane_best(key, block);
      for (int k = 0; k < kb; ++k) {
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key);
        const uint32_t first = __reduce_min_sync(0xFFFFFFFFu, key == top ? block : 0xFFFFFFFFu);
        if (block == first && key == top) {
          sm.chosen[k] = static_cast<int>(first);
          if (k == kb - 1) sm.floor_key = top;
          sm.block_key[first] = 0;
          lane_best(key, block);
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();
  if (K) {
    unsigned long long mineL = 0;  // lane k: the warp's k-th largest
    const uint32_t floor_key = kb == K ? sm.floor_key : 0u;
    for (int k = warp; k < kb; k += kWarps) {
      const int b = sm.chosen[k];
      for (int p = 0; p < per_block; ++p) {
        const int v = v0 + (b * per_block + p) * 32 + lane;
        const uint4 r = v < v1 ? row.load(v) : make_uint4(0, 0, 0, 0);
        const int x0 = v * Row<BF16>::kPer - row.shift;
        uint32_t left = 0;  // elements that may still be taken
#pragma unroll
        for (int e = 0; e < Row<BF16>::kPer; ++e)
          if (v < v1 && x0 + e >= 0 && x0 + e < P.V && ordered_bits(element<BF16>(r, e)) >= floor_key) left |= 1u << e;
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
          if (top <= __shfl_sync(0xFFFFFFFFu, mineL, K - 1)) break;  // (0 too: nothing left)
          if (best == top) left &= ~(1u << at_e);
          const int pos = __popc(__ballot_sync(0xFFFFFFFFu, mineL > top));
          const unsigned long long before = __shfl_up_sync(0xFFFFFFFFu, mineL, 1);
          mineL = lane > pos ? before : lane == pos ? top : mineL;
        }
      }
    }
    if (lane < K) sm.lists[warp][lane] = mineL;
    __syncthreads();
    if (warp == 0) {
      // lane l takes list l % 8 from its (l / 8)-th entry on, every fourth: K rounds pick the largest head
      int next = lane >> 3;
      const unsigned long long *list = sm.lists[lane & 7];
      unsigned long long head = next < K ? list[next] : 0ull;
      for (int k = 0; k < K; ++k) {
        const unsigned long long top = warp_max64(head);
        if (lane == 0) sm.best[k] = top;
        if (head == top && top) {
          next += 4;
          head = next < K ? list[next] : 0ull;
        }
      }
    }
    __syncthreads();
  }

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
    const bool bad = a.bad || a.ref == -INFINITY;
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
      const float v = bad ? 0.0f : BF16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t *>(row_ptr)[x])
                                        : reinterpret_cast<const float *>(row_ptr)[x];
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

cudaError_t enable_logprobs_kernels() { return cudaSuccess; }

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
