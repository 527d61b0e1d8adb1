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

}  // namespace

cudaError_t launch_rotate(const RotateParams &p, bool bf16, int num_sms, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const int64_t tokens = (p.T + kWarps - 1) / kWarps;
  cfg.gridDim = dim3(static_cast<unsigned>(tokens), static_cast<unsigned>(p.Hq + p.Hk < 64 ? p.Hq + p.Hk : 64));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  (void)num_sms;
  return cudaLaunchKernelEx(&cfg, bf16 ? rotate_any_kernel<true> : rotate_any_kernel<false>, p);
}

}  // namespace sv
