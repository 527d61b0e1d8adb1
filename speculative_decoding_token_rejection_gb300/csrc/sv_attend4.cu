// sv_attend4.cu -- the private part of the verify tokens' attention over the
// paged 4-bit cache.
//
// With x = (q . n) * (scale * log2 e * key_scale) for a key's numbers n (nibble
// times group scale) and m the largest x of a row so far,
//   w = 2^(x - m),  l = sum w,  O = sum w * value_scale * n_v,
// out = O / l and lse = (m + log2 l) ln 2.  Any m gives the same quotient.
// Everything here is fp32; tiles of 32 keys are unpacked to shared memory.
#include <cmath>
#include <cstdint>

#include "sv_attend.cuh"
#include "sv_cache4.cuh"

namespace sv {
namespace {

constexpr int kOwnThreads = 128, kTileKeys = 32;

template <int D>
struct OwnSmem {
  float q[kOwnRows4][D + 1];
  float k[kTileKeys][D + 1], v[kTileKeys][D + 1];
  float x[kOwnRows4][kTileKeys + 1];
  float kscale[kTileKeys], vscale[kTileKeys];
  int live[kTileKeys];
  uint32_t top[kOwnRows4];  // largest finite |q| of a row
};

template <int D, int FMT>
__global__ void __launch_bounds__(kOwnThreads) own4_kernel(const AttendParams P, const AttendPlan L) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t raw[];
  OwnSmem<D> &S = *reinterpret_cast<OwnSmem<D> *>(raw);
  OwnTile T;
  if (!own_tile(P, L, blockIdx.x, kOwnRows4, T)) return;
  const int tid = threadIdx.x, r = tid >> 1, part = tid & 1;  // two threads a row, every second dimension
  const int32_t *const table = P.tables + T.i * P.table_stride;
  if (tid < kOwnRows4) S.top[tid] = 0;
  __syncthreads();
  for (int at = tid; at < kOwnRows4 * D; at += kOwnThreads) {
    const int row = at / D, d = at - row * D, lr = T.r0 + row, j = div_by(lr, L.group);
    float x = 0.0f;
    if (row < T.rows)
      x = bf16_bits_to_float(P.q[(T.first + j) * P.q_token + (T.h * P.group + lr - j * P.group) * P.q_head + d]);
    S.q[row][d] = x;
    const uint32_t size = __float_as_uint(x) & 0x7FFFFFFFu;
    if (size < 0x7F800000u) atomicMax(&S.top[row], size);
  }
  __syncthreads();
  // (sums of a row's products stay in range: its own power of two goes in before them, and out behind the key's scale)
  const int shift = query_shift(S.top[r]);
  for (int d = part; d < D; d += 2) S.q[r][d] *= pow2(shift);
  const float back = pow2(-shift);
  const int j = div_by(T.r0 + r, L.group);
  const int limit = r < T.rows ? T.len - T.gam + j : 0;  // keys that the row sees are below it
  const float c_all = P.scale * kLog2e * unit4<FMT>();
  float m = -INFINITY, l = 0.0f, o[D / 2];
#pragma unroll
  for (int d = 0; d < D / 2; ++d) o[d] = 0.0f;
  uint32_t bits = 0;
  for (int k0 = T.k_begin; k0 < T.k_end; k0 += kTileKeys) {
    __syncthreads();
    for (int at = tid; at < 2 * kTileKeys * (D / kGroup4); at += kOwnThreads) {
      const int col = at % (D / kGroup4), key = at / (D / kGroup4) % kTileKeys, side = at / (D / kGroup4) / kTileKeys;
      const int k = k0 + key;
      uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      float scale = 0.0f;
      bool live = false;
      if (k < T.k_end) {
        const int x = div_by(k, L.page), off = k - x * P.c.block_size, page = (k < P.row0 ? P.tables : table)[x];
        live = page >= 0 && page < P.c.num_blocks;
        if (live) {
          const uint8_t *const src = static_cast<const uint8_t *>(side ? P.c.v : P.c.k) + page * P.c.block_stride +
                                     T.h * P.c.head_stride + off * P.c.token_stride + col * 8;
          const uint32_t g = (side ? P.v_group : P.k_group)[page * P.group_block + T.h * P.group_head +
                                                            off * P.group_token + col];
          group_to_f16<FMT>(__ldg(reinterpret_cast<const uint2 *>(src)), group_factors<FMT>(g), w);
          scale = (side ? P.c.v_scale : P.c.k_scale)[page * P.c.scale_block_stride + T.h * P.c.scale_head_stride +
                                                     off * P.c.scale_token_stride];
        } else {
          bits = SV_DATA_BAD_SLOT;
        }
      }
      float *const dst = (side ? S.v : S.k)[key] + col * kGroup4;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dst[2 * e] = f16_bits_to_float(static_cast<uint16_t>(w[e]));
        dst[2 * e + 1] = f16_bits_to_float(static_cast<uint16_t>(w[e] >> 16));
      }
      if (col == 0) {
        if (side)
          S.vscale[key] = fabsf(scale) < kLeastScale ? 0.0f : fabsf(scale) < INFINITY ? scale : __uint_as_float(0x7FC00000u);
        else
          S.kscale[key] = scale;
        S.live[key] = live;
      }
    }
    __syncthreads();
    float top = m;
    for (int key = part; key < kTileKeys; key += 2) {
      float s = 0.0f;
      for (int d = 0; d < D; ++d) s = fmaf(S.q[r][d], S.k[key][d], s);
      s = s * (S.kscale[key] * c_all) * back;
      if (!S.live[key] || k0 + key >= limit) s = -INFINITY;
      S.x[r][key] = s;
      top = fmaxf(top, s);
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    __syncwarp();
    const float f = m == -INFINITY ? 1.0f : exp2f(m - top);
    if (top > -INFINITY) m = top;
    l *= f;
#pragma unroll
    for (int d = 0; d < D / 2; ++d) o[d] *= f;
    for (int key = 0; key < kTileKeys; ++key) {
      if (!S.live[key] || k0 + key >= limit) continue;
      const float w = exp2f(S.x[r][key] - (m == -INFINITY ? 0.0f : m)), wv = w * S.vscale[key];
      l += w;
#pragma unroll
      for (int d = 0; d < D / 2; ++d) o[d] = fmaf(wv, S.v[key][2 * d + part], o[d]);
    }
  }
  if (bits && P.status) atomicOr(P.status, static_cast<int>(bits));
  // rows to shared memory, then a warp a row
  __syncthreads();
#pragma unroll
  for (int d = 0; d < D / 2; ++d) S.q[r][2 * d + part] = o[d] * unit4<FMT>();
  if (part == 0) {
    S.x[r][0] = m;
    S.x[r][1] = l;
  }
  __syncthreads();
  const int lane = tid & 31;
  for (int row = tid >> 5; row < T.rows; row += kOwnThreads / 32) {
    const int lr = T.r0 + row, tok = div_by(lr, L.group), hq = T.h * P.group + lr - tok * P.group;
    Part<D> p;
    p.m = S.x[row][0];
    p.l = S.x[row][1];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) p.o[d] = S.q[row][lane * (D / 32) + d];
    if (T.whole)
      write_row<D>(P, L, T.first + tok, hq, lane, p);
    else
      store_part<D>(L, (T.first + tok) * P.Hq + hq, L.prefix_splits + T.split, lane, p);
  }
}

template <int D, int FMT>
cudaError_t launch(const AttendParams &p, const AttendPlan &L, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const int64_t own = static_cast<int64_t>(p.N) * p.c.num_kv_heads * L.own_tiles * L.own_splits;
  if (own > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(own));
  cfg.blockDim = dim3(kOwnThreads);
  cfg.dynamicSmemBytes = sizeof(OwnSmem<D>);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  return cudaLaunchKernelEx(&cfg, own4_kernel<D, FMT>, p, L);
}

template <int D, int FMT>
cudaError_t enable() {
  return cudaFuncSetAttribute(own4_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(OwnSmem<D>));
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
  if (p.c.head_dim == 128) return i4 ? launch<128, SV_CACHE_INT4>(p, L, stream) : launch<128, SV_CACHE_E2M1>(p, L, stream);
  return i4 ? launch<64, SV_CACHE_INT4>(p, L, stream) : launch<64, SV_CACHE_E2M1>(p, L, stream);
}

}  // namespace sv
