// sv_rotate.cu -- rotary positions of queries and keys, with a norm of each head
// in the same pass.
//
// Bound by HBM: every row is read and written once.  An angle is
// position * turns modulo 2^64, a fraction of a turn exact to 2^-64 a position:
// one integer product, no table of angles, no loss at far positions.  Its sine
// and cosine cost some forty instructions, so a thread keeps those of its pairs
// in registers and walks the heads of its token.
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

// Any head size, alignment and rotated part: a warp a token, a pair (or an element that stays) a lane and step.
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

// Sixteen bytes of a row: VE elements.
template <bool BF16>
struct Vector {
  static constexpr int kElements = BF16 ? 8 : 4;
};
template <bool BF16>
__device__ __forceinline__ uint4 load_vector(const void *p, int64_t at) {
  return *reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + at * (BF16 ? 2 : 4));
}
template <bool BF16>
__device__ __forceinline__ void numbers(const uint4 &v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store_vector(void *p, int64_t at, const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : __float_as_uint(x[i]);
  *reinterpret_cast<uint4 *>(static_cast<char *>(p) + at * (BF16 ? 2 : 4)) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of whole 16-byte vectors.  A lane takes two vectors of a row (UNITS
// times), whose pairs lie in them: elements i .. and i + rotary / 2 .., or
// neighbouring ones, or such as stay.  `lanes` neighbouring lanes share a row,
// and walk `heads` heads of one token, kAhead rows' loads in flight.
constexpr int kAhead = 4;
template <bool BF16, bool INTERLEAVED, bool NORM, int UNITS>
__global__ void __launch_bounds__(kThreads, 2) rotate_kernel(const __grid_constant__ RotateParams P, const int lanes,
                                                            const int heads, const FastDiv parts) {
  pdl_enter();
  constexpr int VE = Vector<BF16>::kElements;
  const int lane = threadIdx.x & 31, col = lane & (lanes - 1);
  const uint32_t group = lanes == 32 ? 0xFFFFFFFFu : ((1u << lanes) - 1u) << (lane & ~(lanes - 1));
  const int item = static_cast<int>((blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x) / lanes);
  const int token = div_by(item, parts), first = (item - token * parts.d) * heads;
  if (token >= P.T) return;
  const int32_t position = P.positions[token];
  if (position < 0) return;
  const int last = min(first + heads, P.Hq + P.Hk);

  int at[UNITS][2];  // where the lane's vectors begin, -1 for none
  float c[UNITS][VE], s[UNITS][VE];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int unit = u * lanes + col, turned = P.rotary / (2 * VE);
    if (INTERLEAVED) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        at[u][v] = (2 * unit + v) * VE < P.D ? (2 * unit + v) * VE : -1;
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
          const int i = (2 * unit + v) * (VE / 2) + e;
          s[u][v * (VE / 2) + e] = 0.0f;
          c[u][v * (VE / 2) + e] = 1.0f;
          if (2 * i < P.rotary) angle(position, P.turns[i], P.magnitude, s[u][v * (VE / 2) + e], c[u][v * (VE / 2) + e]);
        }
      }
    } else {
      const int rest = P.rotary + (unit - turned) * 2 * VE;
      at[u][0] = unit < turned ? unit * VE : rest < P.D ? rest : -1;
      at[u][1] = unit < turned ? unit * VE + P.rotary / 2 : rest + VE < P.D ? rest + VE : -1;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        s[u][e] = 0.0f;
        c[u][e] = 1.0f;
        if (unit < turned) angle(position, P.turns[unit * VE + e], P.magnitude, s[u][e], c[u][e]);
      }
    }
  }
  float w[NORM ? UNITS : 1][2][VE];
  const void *held = nullptr;  // the weights in w
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
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (h + k >= last) break;
      const bool key = h + k >= P.Hq;
      const RotateSide &S = key ? P.k : P.q;
      const int64_t to = token * S.out_token + (h + k - (key ? P.Hq : 0)) * S.out_head;
      float x[UNITS][2][VE];
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) numbers<BF16>(raw[k][u][v], x[u][v]);
      if (NORM && S.weight) {
        if (S.weight != held) {
          held = S.weight;
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int v = 0; v < 2; ++v)
              if (at[u][v] >= 0) numbers<BF16>(load_vector<BF16>(held, at[u][v]), w[u][v]);
        }
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
          for (int e = 0; e < VE; ++e) sum = fmaf(x[u][0][e], x[u][0][e], fmaf(x[u][1][e], x[u][1][e], sum));
        for (int b = lanes >> 1; b; b >>= 1) sum += __shfl_xor_sync(group, sum, b);
        const float r = __frsqrt_rn(sum / static_cast<float>(P.D) + P.eps);
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            x[u][0][e] = x[u][0][e] * r * w[u][0][e];
            x[u][1][e] = x[u][1][e] * r * w[u][1][e];
          }
      }
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        float y[2][VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          // (pairs side by side lie in one vector, the first VE / 2 of them in the first one)
          float &a = INTERLEAVED ? x[u][e / (VE / 2)][2 * (e % (VE / 2))] : x[u][0][e];
          float &b = INTERLEAVED ? x[u][e / (VE / 2)][2 * (e % (VE / 2)) + 1] : x[u][1][e];
          float &p = INTERLEAVED ? y[e / (VE / 2)][2 * (e % (VE / 2))] : y[0][e];
          float &q = INTERLEAVED ? y[e / (VE / 2)][2 * (e % (VE / 2)) + 1] : y[1][e];
          p = a * c[u][e] - b * s[u][e];
          q = b * c[u][e] + a * s[u][e];
        }
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (at[u][v] >= 0) store_vector<BF16>(S.out, to + at[u][v], y[v]);
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
  // a token's heads are cut over more lanes while that fills the SMs (1024 threads each), no finer than kAhead heads
  int parts = static_cast<int>((num_sms * 1024LL + p.T * lanes - 1) / (p.T * lanes));
  if (parts > (all + kAhead - 1) / kAhead) parts = (all + kAhead - 1) / kAhead;
  const int heads = (all + parts - 1) / parts;
  parts = (all + heads - 1) / heads;
  cfg.gridDim = dim3(static_cast<unsigned>((p.T * parts * lanes + kThreads - 1) / kThreads));
  return bf16 ? pick<true>(cfg, p, lanes, heads, parts, units) : pick<false>(cfg, p, lanes, heads, parts, units);
}

}  // namespace sv
