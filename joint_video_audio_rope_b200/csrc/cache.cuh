// What the kernels over the paged 8-bit cache share (cache.cu, cache_attn*.cu): e4m3 codes as
// fp16, powers of two, asynchronous copies.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"

namespace mmdit {

// 1 / f of a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse_pow2(float f) {
  return __int_as_float((254 << 23) - __float_as_int(f));
}
// Four e4m3 codes as two pairs of fp16 (as one 32-bit register each: through the 16-bit
// halves of the type's C++ interface this took three times the operations).
__device__ __forceinline__ void halves_of(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ float2 unpack_half2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 16 bytes to shared memory, asynchronously.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

}  // namespace mmdit
