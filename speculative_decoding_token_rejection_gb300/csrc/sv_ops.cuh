// sv_ops.cuh -- device helpers of the operators around the verifier: the
// ragged request layout, 8-bit cache formats and bf16 packing.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

// Draft range of request i: rows s + i .. s + i + g of the verify-token
// layout.  False if cu is not a valid range.
__device__ __forceinline__ bool request_range(const int32_t *cu, int i, int G, int64_t T, int64_t &s, int &g) {
  if (!cu) {
    s = static_cast<int64_t>(i) * G;
    g = G;
    return true;
  }
  s = i ? cu[i - 1] : 0;
  const int64_t e = cu[i];
  if (s < 0 || e < s || e > T || e - s > G) return false;
  g = static_cast<int>(e - s);
  return true;
}

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }
// Two floats rounded to nearest even bf16, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes (low byte first) of floats, round to nearest even, saturating.
__device__ __forceinline__ uint16_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes as two f16 (exact), the low byte in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
  return r;
}
__device__ __forceinline__ float f16_bits_to_float(uint16_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return f;
}
// The four numbers of the four e4m3 bytes of w.
__device__ __forceinline__ void e4m3_word_to_floats(uint32_t w, float f[4]) {
  const uint32_t a = e4m3x2_to_f16x2(static_cast<uint16_t>(w)), b = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
  f[0] = f16_bits_to_float(static_cast<uint16_t>(a));
  f[1] = f16_bits_to_float(static_cast<uint16_t>(a >> 16));
  f[2] = f16_bits_to_float(static_cast<uint16_t>(b));
  f[3] = f16_bits_to_float(static_cast<uint16_t>(b >> 16));
}

}  // namespace sv

namespace sv {

// ---------------------------------------------------------------------------
// 8-bit numbers to pairs of f16, exactly
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Bytes 0, 1 (lo) and 2, 3 (hi) of w as f16 pairs.  int8: a byte x + 128 put
// into the low mantissa bits of 1024 is the number 1152 + x; subtracting 1152
// is exact.
template <int FMT>
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (FMT == SV_CACHE_INT8) {
    w ^= 0x80808080u;
    lo = hadd2(__byte_perm(w, 0x64646464u, 0x4140), 0xE480E480u);  // (-1152, -1152)
    hi = hadd2(__byte_perm(w, 0x64646464u, 0x4342), 0xE480E480u);
  } else {
    lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w));
    hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------------------
// asynchronous copies to shared memory; the bytes behind `n` are zeros.  (No
// memory clobber: other loads may move across them.  What they write is read
// behind copy_wait only.)
// ---------------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t n) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(BYTES));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D[16x8] += A[16x16] B[16x8], f16 with fp32 sums.
__device__ __forceinline__ void mma_16816(float d[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// n / d by the factors of fast_div.
__device__ __forceinline__ int div_by(int n, const FastDiv &f) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(n)) * f.mul) >> f.shift);
}

}  // namespace sv

namespace sv {

// 32 bytes at once, from and to 32-byte boundaries: a whole sector a lane, where
// two 16-byte accesses would touch every sector twice.
__device__ __forceinline__ void ld_stream_32(const void *p, uint32_t r[8]) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void st_32(void *p, const uint32_t r[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Two fp32 numbers in one register pair, one instruction for both.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ float lo(Pair p) {
  return __uint_as_float(static_cast<uint32_t>(p.v));
}
__device__ __forceinline__ float hi(Pair p) {
  return __uint_as_float(static_cast<uint32_t>(p.v >> 32));
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// An 8x8 tile of 16-bit numbers transposed across the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

}  // namespace sv
