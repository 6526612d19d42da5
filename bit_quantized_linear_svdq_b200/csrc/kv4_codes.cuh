// kv4_codes.cuh -- device helpers shared by the kernels of the 4-bit cache.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

namespace svdq {

// Four bytes of packed E2M1 codes (eight values) -> four fp16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t* d) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}

// Two e4m3 bytes (bits 7:0 and 15:8) -> fp16 pair (low, high), exact.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return *reinterpret_cast<const __half2*>(&h);
}

}  // namespace svdq
