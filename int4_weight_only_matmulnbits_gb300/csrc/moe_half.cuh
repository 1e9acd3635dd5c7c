// fp16 forms of codes and activations, and asynchronous copies, shared by the
// kernels of the expert layer.
#pragma once

#include <cuda_fp16.h>

#include "mnb_common.cuh"

namespace mnb {

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight codes: pairs of 1024 + q (rows g: r[0], r[2]) and of 1024 + 16 q
// (rows g + 8: r[1], r[3]).
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, kMagic = 0x64006400u;
  r[0] = lop3_and_or(w, kLow, kMagic);
  r[1] = lop3_and_or(w, kHigh, kMagic);
  w >>= 8;
  r[2] = lop3_and_or(w, kLow, kMagic);
  r[3] = lop3_and_or(w, kHigh, kMagic);
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The power of two that brings a row whose largest magnitude has the bits
// `top` into 2^14 .. 2^15 (1 for rows of zeros and rows that are not finite;
// at most 2^126), as an exponent.
__device__ __forceinline__ int row_shift(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  if (top == 0u || e == 255) return 0;
  return min(14 - (e - 127), 126);
}
__device__ __forceinline__ float exp2i(int k) {  // 2^k, |k| <= 126
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

// Eight consecutive activations from element k of a row, zeros past K.
__device__ __forceinline__ void load8(const void *A, bool f32, bool vec, int64_t row, int k,
                                      int K, float (&v)[8]) {
  if (vec && k + 8 <= K) {
    if (f32) {
      const float4 *a = reinterpret_cast<const float4 *>(static_cast<const float *>(A) + row + k);
      const float4 x = a[0], y = a[1];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
      const uint4 x =
          *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(A) + row + k);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = 0.f;
      if (k + q < K)
        v[q] = f32 ? static_cast<const float *>(A)[row + k + q]
                   : bf16_bits_to_f32(static_cast<const uint16_t *>(A)[row + k + q]);
    }
  }
}

}  // namespace mnb
