// sv_rotate.cu -- rotary positions of queries and keys, with a norm of each head
// in the same pass.
//
// Bound by HBM: every row is read and written once.  An angle is
// position * turns modulo 2^64, a fraction of a turn exact to 2^-64 a position:
// one integer product, no table of angles, no loss at far positions.  Its sine
// and cosine cost some forty instructions, so a thread keeps those of its pairs
// in registers and walks the heads of its token.
#include <algorithm>
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

// sin and cos of position * turns / 2^64 turns, times m.  The angle is reduced to an eighth of a turn before it is
// rounded to fp32, so its error is 2^-24 of at most pi / 4.
__device__ __forceinline__ void angle(int32_t position, uint64_t turns, float m, float &s, float &c) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns + (1ull << 31);
  const uint32_t h = static_cast<uint32_t>(t >> 32), q = (h + (1u << 29)) >> 30;
  float a, b;
  sincospif(static_cast<float>(static_cast<int32_t>(h - (q << 30))) * 0x1p-31f, &a, &b);
  if (q & 1u) {
    const float x = a;
    a = b;
    b = -x;
  }
  if (q & 2u) {
    a = -a;
    b = -b;
  }
  s = a * m;
  c = b * m;
}

template <bool BF16>
__device__ __forceinline__ float load_one(const void *p, int64_t at) {
  return BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p)[at]) : static_cast<const float *>(p)[at];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void *p, int64_t at, float x) {
  if (BF16)
    static_cast<uint16_t *>(p)[at] = static_cast<uint16_t>(pack_bf16(x, 0.0f));
  else
    static_cast<float *>(p)[at] = x;
}

// Any head size, alignment and rotated part: a warp a token, a pair (or an element that stays) a lane and step.  Sines
// and cosines are worked out for every head: 4096 tokens x 40 heads x 80 bf16 of which 20 turn 82 us (637 GB/s), with norms
// 112; heads of 128 that are not aligned 89.
constexpr int kMostPerLane = SV_MAX_ROTATE_HEAD_DIM / 32;
template <bool BF16>
__global__ void __launch_bounds__(kThreads) rotate_any_kernel(const RotateParams P) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (token >= P.T) return;
  const int32_t position = P.positions[token];
  if (position < 0) return;
  const int half = P.rotary / 2;
  for (int head = blockIdx.y; head < P.Hq + P.Hk; head += gridDim.y) {
    const bool key = head >= P.Hq;
    const RotateSide &S = key ? P.k : P.q;
    const int h = key ? head - P.Hq : head;
    const int64_t from = token * S.in_token + h * S.in_head, to = token * S.out_token + h * S.out_head;
    float x[kMostPerLane];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kMostPerLane; ++k) {
      const int d = k * 32 + lane;
      x[k] = d < P.D ? load_one<BF16>(S.in, from + d) : 0.0f;
      sum = fmaf(x[k], x[k], sum);
    }
    if (S.weight) {
#pragma unroll
      for (int b = 16; b; b >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, b);
      const float r = __frsqrt_rn(sum / static_cast<float>(P.D) + P.eps);
#pragma unroll
      for (int k = 0; k < kMostPerLane; ++k) {
        const int d = k * 32 + lane;
        if (d < P.D) x[k] = x[k] * r * load_one<BF16>(S.weight, d);
      }
    }
    __shared__ float row[kWarps][SV_MAX_ROTATE_HEAD_DIM];
    float *const mine = row[threadIdx.x >> 5];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kMostPerLane; ++k)
      if (k * 32 + lane < P.D) mine[k * 32 + lane] = x[k];
    __syncwarp();
    for (int i = lane; i < half; i += 32) {
      const int at = P.interleaved ? 2 * i : i, bt = P.interleaved ? 2 * i + 1 : i + half;
      float s, c;
      angle(position, P.turns[i], P.magnitude, s, c);
      const float a = mine[at], b = mine[bt];
      store_one<BF16>(S.out, to + at, a * c - b * s);
      store_one<BF16>(S.out, to + bt, b * c + a * s);
    }
    for (int d = P.rotary + lane; d < P.D; d += 32) store_one<BF16>(S.out, to + d, mine[d]);
  }
}

// Sixteen bytes of a row.
template <bool BF16>
constexpr int vector_elements() {
  return BF16 ? 8 : 4;
}
template <bool BF16>
__device__ __forceinline__ uint4 load_vector(const void *p, int64_t at) {
  return *reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + at * (BF16 ? 2 : 4));
}
// The elements of two vectors, first and second ones of the pairs apart: i of
// either vector, or neighbours (those of the first vector first).
template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void split(const uint4 v[2], float *a, float *b) {
  constexpr int VE = vector_elements<BF16>();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float x[VE];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[(2 * i + 1) % VE] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (INTERLEAVED)
        (i & 1 ? b : a)[k * (VE / 2) + (i >> 1)] = x[i];
      else
        (k ? b : a)[i] = x[i];
    }
  }
}
template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void store_split(void *p, int64_t at, int k, const float *a, const float *b) {
  constexpr int VE = vector_elements<BF16>();
  float x[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) x[i] = INTERLEAVED ? (i & 1 ? b : a)[k * (VE / 2) + (i >> 1)] : (k ? b : a)[i];
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = BF16 ? pack_bf16(x[2 * i], x[(2 * i + 1) % VE]) : __float_as_uint(x[i]);
  *reinterpret_cast<uint4 *>(static_cast<char *>(p) + at * (BF16 ? 2 : 4)) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of whole 16-byte vectors.  A lane takes two vectors of a row (UNITS
// times), whose pairs lie in them: elements i .. and i + rotary / 2 .., or
// neighbouring ones, or such as stay.  `lanes` neighbouring lanes share a row,
// and walk `heads` heads of one token, kAhead rows' loads in flight.
//
// 50001 fp32 tokens x 10 heads x 128: 80 us (94 % of the copy rate).  4096 tokens x
// 40 heads x 128 bf16 that lie in L2: 13.7 us, with norms 17.0 (20.6 from HBM);
// 32768 tokens with norms 126 (79 %).  A row's norm is a chain (load, sum,
// shuffles, root) that more rows in flight hide: four of bf16 rows with norms on
// two CTAs an SM, where two rows on three CTAs took a quarter longer.  Without
// norms, or in fp32 (whose rows are twice the registers), more CTAs are better:
// 15.3 us with four rows, and 90 for the fp32 tokens.  What bounds rows with norms is
// that chain, step after step, for 3.3 warps a scheduler: half of the issue slots are
// filled, no pipe beyond 38 %.  Two forms spill in the loop: neighbours paired with norms in
// bf16 (19.1 us for 4096 tokens, 131 for 32768) and fp32 rows above 256 with norms (16384
// tokens x 10 heads x 512: 138 us, 102 without norms).
constexpr int rows_ahead(bool bf16, bool norm) { return bf16 && norm ? 4 : 2; }
constexpr int rotate_ctas(bool bf16, bool norm) { return bf16 && norm ? 2 : 3; }  // of an SM
template <bool BF16, bool INTERLEAVED, bool NORM, int UNITS>
__global__ void __launch_bounds__(kThreads, rotate_ctas(BF16, NORM))
    rotate_kernel(const __grid_constant__ RotateParams P, const int lanes, const int heads, const FastDiv parts) {
  pdl_enter();
  constexpr int VE = vector_elements<BF16>(), kAhead = rows_ahead(BF16, NORM);
  const int lane = threadIdx.x & 31, col = lane & (lanes - 1);
  const uint32_t group = lanes == 32 ? 0xFFFFFFFFu : ((1u << lanes) - 1u) << (lane & ~(lanes - 1));
  const int item = static_cast<int>((blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x) / lanes);
  const int token = div_by(item, parts), first = (item - token * parts.d) * heads;
  if (token >= P.T) return;
  const int32_t position = P.positions[token];
  if (position < 0) return;
  const int last = min(first + heads, P.Hq + P.Hk);
  const float mean = 1.0f / static_cast<float>(P.D);

  int at[UNITS][2];     // where the lane's vectors begin, -1 for none
  bool turns[UNITS][2]; // their pairs are turned (in the half layout both vectors' are or none)
  float c[UNITS][VE], s[UNITS][VE];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int unit = u * lanes + col, turned = P.rotary / (2 * VE);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int rest = P.rotary + (unit - turned) * 2 * VE + v * VE, pair = (2 * unit + v) * VE;
      if (INTERLEAVED) {
        at[u][v] = pair < P.D ? pair : -1;
        turns[u][v] = pair < P.rotary;
      } else {
        at[u][v] = unit < turned ? unit * VE + v * (P.rotary / 2) : rest < P.D ? rest : -1;
        turns[u][v] = unit < turned;
      }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      s[u][e] = 0.0f;
      c[u][e] = 1.0f;
      if (turns[u][INTERLEAVED ? e / (VE / 2) : 0]) angle(position, P.turns[unit * VE + e], P.magnitude, s[u][e], c[u][e]);
    }
  }
  float wa[NORM ? UNITS : 1][VE], wb[NORM ? UNITS : 1][VE];
  const void *held = nullptr;  // the weights in wa and wb
  for (int h = first; h < last; h += kAhead) {
    uint4 raw[kAhead][UNITS][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool key = h + k >= P.Hq;
      const RotateSide &S = key ? P.k : P.q;
      const int64_t from = token * S.in_token + (h + k - (key ? P.Hq : 0)) * S.in_head;
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          raw[k][u][v] = make_uint4(0, 0, 0, 0);
          if (h + k < last && at[u][v] >= 0) raw[k][u][v] = load_vector<BF16>(S.in, from + at[u][v]);
        }
    }
    float r[kAhead];
    if (NORM) {  // all rows' sums before the first is needed
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        Pair sum = pair(0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          float a[VE], b[VE];
          split<BF16, INTERLEAVED>(raw[k][u], a, b);
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            sum = fma2(pair(a[e], a[e + 1]), pair(a[e], a[e + 1]), sum);
            sum = fma2(pair(b[e], b[e + 1]), pair(b[e], b[e + 1]), sum);
          }
        }
        r[k] = lo(sum) + hi(sum);
      }
      for (int i = lanes >> 1; i; i >>= 1)
#pragma unroll
        for (int k = 0; k < kAhead; ++k) r[k] += __shfl_xor_sync(group, r[k], i);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) r[k] = rsqrtf(fmaf(r[k], mean, P.eps));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (h + k >= last) break;
      const bool key = h + k >= P.Hq;
      const RotateSide &S = key ? P.k : P.q;
      const int64_t to = token * S.out_token + (h + k - (key ? P.Hq : 0)) * S.out_head;
      const bool norm = NORM && S.weight;
      float a[UNITS][VE], b[UNITS][VE];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) split<BF16, INTERLEAVED>(raw[k][u], a[u], b[u]);
      if (norm && S.weight != held) {
        held = S.weight;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          uint4 w[2];
#pragma unroll
          for (int v = 0; v < 2; ++v)
            w[v] = at[u][v] >= 0 ? load_vector<BF16>(held, at[u][v]) : make_uint4(0, 0, 0, 0);
          split<BF16, INTERLEAVED>(w, wa[u], wb[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        float p[VE], q[VE];
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
          Pair x = pair(a[u][e], a[u][e + 1]), y = pair(b[u][e], b[u][e + 1]);
          if (norm) {
            x = mul2(x, mul2(pair(wa[u][e], wa[u][e + 1]), pair(r[k], r[k])));
            y = mul2(y, mul2(pair(wb[u][e], wb[u][e + 1]), pair(r[k], r[k])));
          }
          // (what stays keeps clear of its neighbours: an infinity times a sine of zero is no number)
          if (turns[u][INTERLEAVED ? e / (VE / 2) : 0]) {
            const Pair cc = pair(c[u][e], c[u][e + 1]), ss = pair(s[u][e], s[u][e + 1]);
            const Pair t = fma2(y, pair(-lo(ss), -hi(ss)), mul2(x, cc));
            y = fma2(y, cc, mul2(x, ss));
            x = t;
          }
          p[e] = lo(x);
          p[e + 1] = hi(x);
          q[e] = lo(y);
          q[e + 1] = hi(y);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (at[u][v] >= 0) store_split<BF16, INTERLEAVED>(S.out, to + at[u][v], v, p, q);
      }
    }
  }
}

template <bool BF16, bool INTERLEAVED, bool NORM>
cudaError_t launch_vectors(const cudaLaunchConfig_t &cfg, const RotateParams &p, int lanes, int heads, int parts, int units) {
  // (two bytes an element: 512 of them are 32 lanes' vectors)
  return cudaLaunchKernelEx(&cfg, BF16 || units == 1 ? rotate_kernel<BF16, INTERLEAVED, NORM, 1>
                                                     : rotate_kernel<BF16, INTERLEAVED, NORM, BF16 ? 1 : 2>,
                            p, lanes, heads, fast_div(parts));
}
template <bool BF16>
cudaError_t pick(const cudaLaunchConfig_t &cfg, const RotateParams &p, int lanes, int heads, int parts, int units) {
  const bool norm = p.q.weight || p.k.weight;
  if (p.interleaved)
    return norm ? launch_vectors<BF16, true, true>(cfg, p, lanes, heads, parts, units)
                : launch_vectors<BF16, true, false>(cfg, p, lanes, heads, parts, units);
  return norm ? launch_vectors<BF16, false, true>(cfg, p, lanes, heads, parts, units)
              : launch_vectors<BF16, false, false>(cfg, p, lanes, heads, parts, units);
}

bool whole_vectors(const RotateSide &s, int heads, int ve) {
  if (heads == 0) return true;
  const auto aligned = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  return aligned(s.in) && aligned(s.out) && aligned(s.weight) && s.in_token % ve == 0 && s.in_head % ve == 0 &&
         s.out_token % ve == 0 && s.out_head % ve == 0;
}

}  // namespace

cudaError_t launch_rotate(const RotateParams &p, bool bf16, int num_sms, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  const int all = p.Hq + p.Hk, ve = bf16 ? 8 : 4, half = p.interleaved ? p.rotary : p.rotary / 2;
  if (p.D % ve || half % ve || !whole_vectors(p.q, p.Hq, ve) || !whole_vectors(p.k, p.Hk, ve)) {
    cfg.gridDim = dim3(static_cast<unsigned>((p.T + kWarps - 1) / kWarps), static_cast<unsigned>(all < 64 ? all : 64));
    return cudaLaunchKernelEx(&cfg, bf16 ? rotate_any_kernel<true> : rotate_any_kernel<false>, p);
  }
  const int turned = p.interleaved ? 0 : p.rotary / (2 * ve);
  const int need = turned + (p.D - turned * 2 * ve + 2 * ve - 1) / (2 * ve);  // pairs of vectors in a row
  int lanes = 1;
  while (lanes < need && lanes < 32) lanes *= 2;
  const int units = (need + lanes - 1) / lanes;
  // A token's heads are cut into parts, no finer than a step's rows: without norms until 1024 threads an SM are there,
  // with them, and with fewer CTAs on an SM, where the waves of CTAs times a CTA's steps (and the angles, about one more)
  // are the fewest: 4096 tokens x 40 heads in 0.8 waves of 5 steps 17.0 us, in 2.1 waves of 2 steps 20.3.
  const bool norm = p.q.weight || p.k.weight;
  const int step = rows_ahead(bf16, norm), most = (all + step - 1) / step;
  int parts = static_cast<int>(std::min<int64_t>(most, (num_sms * 1024LL + p.T * lanes - 1) / (p.T * lanes)));
  if (norm) {
    int64_t least = INT64_MAX;
    for (int steps = 1; steps <= most; steps += 1 + steps / 64) {
      const int n = (most + steps - 1) / steps;
      if (n > 1 && p.T * n * lanes > INT32_MAX) continue;  // (a thread's number is an int)
      const int64_t ctas = (p.T * n * lanes + kThreads - 1) / kThreads, at_once = num_sms * rotate_ctas(bf16, norm);
      const int64_t time = (ctas + at_once - 1) / at_once * (steps + 1);
      if (time < least) {
        least = time;
        parts = n;
      }
    }
  }
  const int heads = (all + parts - 1) / parts;
  parts = (all + heads - 1) / heads;
  cfg.gridDim = dim3(static_cast<unsigned>((p.T * parts * lanes + kThreads - 1) / kThreads));
  return bf16 ? pick<true>(cfg, p, lanes, heads, parts, units) : pick<false>(cfg, p, lanes, heads, parts, units);
}

}  // namespace sv
