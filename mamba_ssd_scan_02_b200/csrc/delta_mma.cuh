// delta_mma.cuh -- what the front end and the chunk kernel of the delta rule share: the layout of an
// operand tile, the two-part fp16 operands, the base-2 exponential.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace delta {

// 16-byte chunk c of row r of a tile of 128-byte rows with the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return (uint32_t)row * 128u + ((uint32_t)(chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
// fp16 pairs: hi, and lo = what hi leaves
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __float22half2_rn(v);
  hi = h2(h);
  lo = h2(__float22half2_rn(__ffma2_rn(__half22float2(h), make_float2(-1.f, -1.f), v)));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace delta
}  // namespace ssd
