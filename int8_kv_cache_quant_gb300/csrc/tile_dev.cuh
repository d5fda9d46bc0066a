// tile_dev.cuh — device helpers shared by the kernels that stream operand tiles to the 5th-generation
// tensor core (prefill.cu, chunk_weights.cu, prefill_window.cu): packed fp32 pairs, widening of int8 codes, power-of-two
// row scales, and bounded waits that give up together.
#pragma once

#include <cuda_bf16.h>

#include "kvq_dev.cuh"
#include "tcgen05.cuh"

namespace kvq {

// One operand piece in shared memory: 128 rows x 64 16-bit values, 128-byte swizzle, K-major.
constexpr int kPieceBytes = 16384;

// Packed fp32 pairs (add / mul / fma .rn.f32x2): each lane is rounded exactly like the scalar
// operation, so these give the same bits as __fadd_rn / __fmul_rn / __fmaf_rn per element with
// half the instructions.
struct f2 {
  unsigned long long v;
};
__device__ __forceinline__ f2 mk2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
// one half of a pair: the unpacking mov names both halves and the other one is dropped
#pragma nv_diag_suppress 550
__device__ __forceinline__ float lo2(f2 a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
  return x;
}
__device__ __forceinline__ float hi2(f2 a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
  return y;
}
#pragma nv_diag_default 550
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) {
  f2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// 16 int8 codes (one int4) -> two 16-byte chunks of 8 fp16 (exact integer values).
__device__ __forceinline__ void widen16(const int4 raw, uint4& c0, uint4& c1) {
  uint32_t lo, hi;
  i8x4_to_h2x2(static_cast<uint32_t>(raw.x), kSelB01, kSelB23, lo, hi);
  c0.x = lo;
  c0.y = hi;
  i8x4_to_h2x2(static_cast<uint32_t>(raw.y), kSelB01, kSelB23, lo, hi);
  c0.z = lo;
  c0.w = hi;
  i8x4_to_h2x2(static_cast<uint32_t>(raw.z), kSelB01, kSelB23, lo, hi);
  c1.x = lo;
  c1.y = hi;
  i8x4_to_h2x2(static_cast<uint32_t>(raw.w), kSelB01, kSelB23, lo, hi);
  c1.z = lo;
  c1.w = hi;
}

// 16 int8 codes -> eight words of two bf16 each.  With 0x43 above it, the low seven bits of a code are
// the bf16 number 128 + (code & 127), and its sign bit alone is 128 or 256: their difference is
// the code, exactly.
__device__ __forceinline__ void widen16_bf16(const uint4& raw, uint32_t* out) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = __byte_perm(w[i >> 1], 0x43434343u, (i & 1) ? kSelB23 : kSelB01);
    const uint32_t lo = v & 0xFF7FFF7Fu, hi = v & 0xFF80FF80u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi));
    out[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

__device__ __forceinline__ void sts128(uint8_t* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  const uint32_t s = smem_u32(p);
  return p + (((s + 1023u) & ~1023u) - s);
}

// 2^(e - 14) and its inverse for a row maximum amax (1 for amax = 0), exponents clamped.
__device__ __forceinline__ void pow2_scales(float amax, float& to_f16, float& back) {
  int e = amax > 0.f ? static_cast<int>((__float_as_uint(amax) >> 23) & 0xFF) - 127 : 14;
  e = max(-100, min(e, 100));
  to_f16 = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
  back = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23);
}

// Bounded wait that also gives up as soon as another thread of the CTA has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, unsigned int* status,
                                              volatile int* abort_flag, long long budget) {
  if (mbar_try_wait(bar, parity)) return true;
  long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > budget) {
      set_status(status, KVQ_DEV_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace kvq
