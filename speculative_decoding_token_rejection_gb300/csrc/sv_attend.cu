// sv_attend.cu -- attention of the verify tokens over the paged 8-bit cache.
//
// One CTA per (request, verify token, query head): its threads score a tile of
// keys each, a running maximum and sum rescale the output row, and every
// thread then gathers one output dimension over the tile's values.
#include <cmath>
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;  // keys of a tile, and threads of a CTA

template <int D, int FMT>
__global__ void __launch_bounds__(kTile) attend_kernel(const AttendParams P) {
  pdl_enter();
  __shared__ float q[D];
  __shared__ float w[kTile];
  __shared__ int64_t at[kTile], sat[kTile];
  __shared__ float red[kTile / 32];
  const int i = blockIdx.x, j = blockIdx.y / P.Hq, hq = blockIdx.y % P.Hq, hk = hq / P.group;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t s;
  int g;
  if (!request_range(P.cu, i, P.G, P.T, s, g)) {
    if (tid == 0 && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_CU));
    return;
  }
  if (j > g) return;
  const int64_t row = s + i + j;
  int len = P.seq_lens[i];
  if (len < 0 || len > P.max_seq) {
    if (tid == 0 && P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_PARAM));
    len = 0;
  }
  const int see = min(len, max(0, len - g + j));  // keys 0 .. see - 1
  for (int d = tid; d < D; d += kTile) q[d] = bf16_bits_to_float(P.q[row * P.q_token + hq * P.q_head + d]);
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int k0 = 0; k0 < see; k0 += kTile) {
    const int k = k0 + tid;
    float sc = -INFINITY;
    bool live = k < see;
    if (live) {
      const int32_t *table = P.tables + (k < P.prefix ? 0 : i) * P.table_stride;
      const int page = table[k / P.c.block_size], off = k % P.c.block_size;
      if (page < 0 || page >= P.c.num_blocks) {
        if (P.status) atomicOr(P.status, static_cast<int>(SV_DATA_BAD_SLOT));
        live = false;
      } else {
        at[tid] = page * P.c.block_stride + hk * P.c.head_stride + off * P.c.token_stride;
        sat[tid] = page * P.c.scale_block_stride + hk * P.c.scale_head_stride + off * P.c.scale_token_stride;
      }
    }
    if (!live) at[tid] = -1;
    __syncthreads();
    if (live) {
      const uint32_t *kr = reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(P.c.k) + at[tid]);
      float dot = 0.0f;
      for (int d = 0; d < D; d += 4) {
        float x[4];
        cache_word_to_floats<FMT>(kr[d / 4], x);
        dot += q[d] * x[0] + q[d + 1] * x[1] + q[d + 2] * x[2] + q[d + 3] * x[3];
      }
      sc = dot * P.c.k_scale[sat[tid]] * P.scale;
    }
    float top = sc;
    for (int b = 16; b; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, b));
    if (lane == 0) red[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m1 = fmaxf(m, top);
    const float e = live && m1 != -INFINITY ? expf(sc - m1) : (live && isnan(sc) ? sc : 0.0f);
    w[tid] = e;
    const float r = m == -INFINITY ? 0.0f : expf(m - m1);
    o *= r;
    l *= r;
    m = m1;
    __syncthreads();
    const int n = min(kTile, see - k0);
    for (int x = 0; x < n; ++x) {
      l += w[x];
      if (tid < D && at[x] >= 0) {
        float v[4];
        const uint32_t word = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(P.c.v) + at[x] + (tid & ~3));
        cache_word_to_floats<FMT>(word, v);
        const float y = (tid & 3) == 0 ? v[0] : (tid & 3) == 1 ? v[1] : (tid & 3) == 2 ? v[2] : v[3];
        o += w[x] * (y * P.c.v_scale[sat[x]]);
      }
    }
    __syncthreads();
  }
  if (tid < D)
    P.out[row * P.out_token + hq * P.out_head + tid] =
        static_cast<uint16_t>(pack_bf16(l == 0.0f ? 0.0f : o / l, 0.0f));
  if (P.lse && tid == 0) P.lse[row * P.Hq + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int D, int FMT>
cudaError_t launch(const AttendParams &p, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.N, (p.G + 1) * p.Hq);
  cfg.blockDim = dim3(kTile);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  return cudaLaunchKernelEx(&cfg, attend_kernel<D, FMT>, p);
}

}  // namespace

cudaError_t enable_attend_kernels() { return cudaSuccess; }

int64_t attend_workspace_bytes(const AttendParams &, int) { return 0; }

cudaError_t launch_attend(const AttendParams &p, int, cudaStream_t stream) {
  const bool i8 = p.c.format == SV_CACHE_INT8;
  if (p.c.head_dim == 128) return i8 ? launch<128, SV_CACHE_INT8>(p, stream) : launch<128, SV_CACHE_E4M3>(p, stream);
  return i8 ? launch<64, SV_CACHE_INT8>(p, stream) : launch<64, SV_CACHE_E4M3>(p, stream);
}

}  // namespace sv
