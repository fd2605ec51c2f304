// The 8-bit activation checkpoint's values (act8.cu has the format).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "device_ops.cuh"
#include "layout.cuh"

namespace any4 {

// K as the weights' (a multiple of 64), groups of 64 .. 1024 columns.
inline bool act_shape_ok(int m, int k, int group) {
  return m >= 1 && m <= kMaxTokens && k <= (1 << 20) && shape_ok(kTileRows, k, group);
}

// 2^121: from this step on a code's value may round to an infinity (-128 times
// any smaller step is a bf16 number yet).
constexpr uint32_t kHugeStep = 0x7C00u;

// Four codes (a 32-bit word) times a step (in both halves of step2): two bf16
// pairs. Byte c = 128 s + m (s its sign bit) stands for m - 128 s; as bf16
// bits, 0x4300 | m is 128 + m and 0x4300 | 128 s is 128 + 128 s, both exact,
// and so is their difference. The product rounds once.
__device__ __forceinline__ uint32_t act8_pair(uint32_t spread, uint32_t step2) {
  const uint32_t up = (spread & 0x007F007Fu) | 0x43004300u, down = (spread & 0x00800080u) | 0x43004300u;
  __nv_bfloat162 u, d;
  u = *reinterpret_cast<const __nv_bfloat162*>(&up);
  d = *reinterpret_cast<const __nv_bfloat162*>(&down);
  const __nv_bfloat162 c = __hsub2(u, d);
  return fma_bf16x2(*reinterpret_cast<const uint32_t*>(&c), step2, 0x80008000u);   // + -0: the product alone
}
__device__ __forceinline__ void act8_values4(uint32_t codes, uint32_t step2, uint32_t& p0, uint32_t& p1) {
  p0 = act8_pair(prmt(codes, 0u, 0x4140u), step2);
  p1 = act8_pair(prmt(codes, 0u, 0x4342u), step2);
}

}  // namespace any4
