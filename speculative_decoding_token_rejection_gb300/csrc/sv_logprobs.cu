// sv_logprobs.cu -- log-probabilities of the committed tokens, with rank,
// entropy and the largest alternatives.
//
// One CTA per token place (i, m).  A first pass finds the row's maximum, a
// second the sums, and each alternative is one more pass that looks for the
// largest entry behind the last one found.
#include <cmath>
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

template <bool BF16>
__device__ __forceinline__ float logit_at(const void *row, int x) {
  return BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(row)[x]) : static_cast<const float *>(row)[x];
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobsParams P) {
  pdl_enter();
  __shared__ ReduceSmem red;
  __shared__ float sums[3][kWarps];
  const int i = blockIdx.x / (P.G + 1), m = blockIdx.x % (P.G + 1), tid = threadIdx.x;
  const int64_t place = blockIdx.x;
  int32_t tok = P.tokens[place];
  uint32_t bits = 0;
  int64_t s;
  int g;
  const bool range = request_range(P.cu, i, P.G, P.T, s, g) && (tok < 0 || m <= g);
  if (!range) bits |= SV_DATA_BAD_CU;
  const float temp = P.temperature ? P.temperature[i] : 1.0f;
  if (range && tok != -1 && (tok < 0 || tok >= P.V)) bits |= SV_DATA_BAD_DRAFT_ID;
  if (range && tok != -1 && !temperature_ok(temp)) bits |= SV_DATA_BAD_PARAM;
  const bool skip = !range || tok == -1;
  float lse = 0.0f, logp = 0.0f, ent = 0.0f, top = 0.0f, inv = 1.0f;
  int rank = -1;
  const void *row = nullptr;
  if (!skip && !bits) {
    const int64_t r = s + i + m;
    row = BF16 ? static_cast<const void *>(static_cast<const uint16_t *>(P.logits) + r * P.row_stride)
               : static_cast<const void *>(static_cast<const float *>(P.logits) + r * P.row_stride);
    KeyFlags k{0ull, 0u};
    for (int x = tid; x < P.V; x += kThreads) {
      const float v = logit_at<BF16>(row, x);
      if (!(v < INFINITY)) k.flags = 1;
      k.key = umax64(k.key, pack_key(v, x));
    }
    k = cluster_reduce(k, red, 0, 1);
    top = logit_at<BF16>(row, key_index(k.key));
    if (k.flags || top == -INFINITY) bits |= SV_DATA_BAD_VALUES;
    inv = temp == 0.0f ? 1.0f : temp;
  }
  if (!skip && !bits) {
    const float mine = logit_at<BF16>(row, tok);
    float z = 0.0f, zx = 0.0f, n = 0.0f;
    for (int x = tid; x < P.V; x += kThreads) {
      const float v = logit_at<BF16>(row, x), d = v / inv - top / inv, e = expf(d);
      z += e;
      if (e > 0.0f) zx += e * d;
      n += v > mine ? 1.0f : 0.0f;
    }
    for (int b = 16; b; b >>= 1) {
      z += __shfl_xor_sync(0xFFFFFFFFu, z, b);
      zx += __shfl_xor_sync(0xFFFFFFFFu, zx, b);
      n += __shfl_xor_sync(0xFFFFFFFFu, n, b);
    }
    if ((tid & 31) == 0) {
      sums[0][tid >> 5] = z;
      sums[1][tid >> 5] = zx;
      sums[2][tid >> 5] = n;
    }
    __syncthreads();
    z = zx = n = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      z += sums[0][w];
      zx += sums[1][w];
      n += sums[2][w];
    }
    lse = logf(z);
    logp = (mine / inv - top / inv) - lse;
    ent = lse - zx / z;
    rank = 1 + static_cast<int>(n);
  } else if (!skip) {
    logp = ent = __uint_as_float(0x7FC00000u);
  }
  if (tid == 0) {
    P.logprobs[place] = logp;
    if (P.entropy) P.entropy[place] = ent;
    if (P.ranks) P.ranks[place] = rank;
    if (bits && P.status) atomicOr(P.status, static_cast<int>(bits));
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < P.K; ++k) {
    int id = -1;
    float lp = skip ? 0.0f : __uint_as_float(0x7FC00000u);
    if (!skip && !bits) {
      KeyFlags b{0ull, 0u};
      for (int x = tid; x < P.V; x += kThreads) {
        const unsigned long long key = pack_key(logit_at<BF16>(row, x), x);
        if (key < last) b.key = umax64(b.key, key);
      }
      b = cluster_reduce(b, red, k + 1, 1);
      last = b.key;
      id = key_index(last);
      lp = (logit_at<BF16>(row, id) / inv - top / inv) - lse;
    }
    if (tid == 0) {
      P.top_ids[place * P.K + k] = id;
      P.top_logprobs[place * P.K + k] = lp;
    }
  }
}

}  // namespace

cudaError_t enable_logprobs_kernels() { return cudaSuccess; }

cudaError_t launch_logprobs(const LogprobsParams &p, bool bf16, int, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.N * (p.G + 1)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 1, p.pdl);
  return cudaLaunchKernelEx(&cfg, bf16 ? logprobs_kernel<true> : logprobs_kernel<false>, p);
}

}  // namespace sv
