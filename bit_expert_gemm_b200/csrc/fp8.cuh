// FP8 E4M3 with one FP32 scale per block of 128: helpers shared by the
// quantiser, the grouped GEMM and the one-kernel decode layer.
//
//   a = max(amax of the block, 2^-80),  s = fl32(a / 448),  r = fl32(448 / a)
//   code = e4m3_rn_sat(fl32(v * r)),    value = e4m3(code) * s
//
// Every step is one FP32 IEEE operation, so the codes are the same wherever
// they are formed.  The floor keeps s normal and r finite for an all-zero
// block.  A block that holds an infinity gets s = +inf and decodes as NaN; a
// NaN takes no part in the maximum and has the E4M3 NaN code itself.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;
constexpr float kFp8AmaxFloor = 8.271806125530277e-25f;  // 2^-80

__host__ __device__ constexpr int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

struct Fp8Scale {
  float s, r;  // dequantisation scale, quantisation multiplier
};
__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
  const float a = fmaxf(amax, kFp8AmaxFloor);
  return {__fdiv_rn(a, kFp8Max), __fdiv_rn(kFp8Max, a)};
}

// Four FP32 values -> four E4M3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}
__device__ __forceinline__ uint32_t fp8_quant4(float a, float b, float c, float d, float r) {
  return f32x4_to_e4m3(__fmul_rn(a, r), __fmul_rn(b, r), __fmul_rn(c, r), __fmul_rn(d, r));
}

}  // namespace moe
