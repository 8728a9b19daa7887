// state_cache.cu -- fp32 recurrent states to and from a cache in 8 bits.
//
// A block of 32 elements shares the scale 2^e, the smallest power of two that brings the block's
// largest magnitude to at most 448 (e4m3) or 127 (int8).  Multiplying by a power of two is exact,
// so the stored element is the correctly rounded x 2^-e and reading back x = q 2^e is exact: the
// result does not depend on the order or the width of any arithmetic.  e comes from the bits of
// the largest magnitude m 2^f with m in [1/2, 1): 448 = 7/8 2^9 and 127 = 127/128 2^7.
//
// Bound by HBM: 4 bytes read and 33/32 written per element (store), the reverse (load).  A warp
// takes 128 elements (four blocks) per step: eight lanes per block with 16 bytes each, so every
// access is a full line, and kUnroll consecutive steps are in flight, whose scales are a full sector.
// 64 states of 128 heads x 64 x 128: store 55.6 us (65 with the scales written step by step), load 54 us,
// 0.93 and 0.96 of a copy's rate.
#include <cuda_fp8.h>

#include "common.cuh"
#include "delta_plan.h"
#include "plan.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;
constexpr int kRow = 128;                               // elements of a warp's step
constexpr int kPerCta = kThreads / 32 * kUnroll * kRow; // elements of a CTA

// Entry i's slots; false if the entry is skipped.  A destination that an earlier entry has is
// skipped (so no two CTAs write the same place) and latched, like a slot outside its array.
__device__ __forceinline__ bool entry(const StateCachePlan &p, bool store, int i, long long *state, long long *cache) {
  const int ss = p.state_slots ? p.state_slots[i] : i, cs = p.cache_slots ? p.cache_slots[i] : i;
  const int *src = store ? p.state_slots : p.cache_slots, *dst = store ? p.cache_slots : p.state_slots;
  const int own = store ? cs : ss;
  bool twice = false;
  if (dst) {  // an earlier entry that is not skipped itself
    for (int j = threadIdx.x; j < i; j += kThreads) twice |= dst[j] == own && (!src || src[j] >= 0);
    twice = __syncthreads_or(twice);
  }
  if (ss < 0 || cs < 0) return false;
  if (twice || ss >= p.n_states || cs >= p.n_cache) {
    if (threadIdx.x == 0) latch_error(p.err, (int)SSD_ERR_DEVICE_BOUNDS);
    return false;
  }
  *state = ss;
  *cache = cs;
  return true;
}

template <bool kE4m3>
__device__ __forceinline__ uint32_t block_scale(uint32_t top) {  // bits of the largest magnitude -> scale byte
  const uint32_t f = top >> 23, frac = top & 0x7fffffu;
  if (f == 255) return 255;
  // top = (1 + frac 2^-23) 2^(f-127); e + 127 = f - 8 or one more (e4m3), f - 6 or one more (int8)
  const int e = kE4m3 ? (int)f - 8 + (frac > 0x600000u ? 1 : 0) : (int)f - 6 + (frac > 0x7e0000u ? 1 : 0);
  return e < 0 ? 0u : (uint32_t)e;
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) state_store_kernel(const StateCachePlan p) {
  long long state, cache;
  if (!entry(p, true, blockIdx.y, &state, &cache)) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long at0 = (long long)blockIdx.x * kPerCta + warp * kUnroll * kRow;
  const float *src = p.states + state * p.elems + 4 * lane;
  float4 x[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i)  // (steps past the end read the last one: no branch between the loads)
    x[i] = __ldcs(reinterpret_cast<const float4 *>(src + min(at0 + i * kRow, p.elems - kRow)));
  uint32_t scales = 0;  // lane i: the four scale bytes of step i
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long at = at0 + i * kRow;
    // the largest magnitude as an integer: a NaN ranks above infinity, which ranks above the rest
    const uint32_t a = __float_as_uint(x[i].x) & 0x7fffffffu, b = __float_as_uint(x[i].y) & 0x7fffffffu;
    const uint32_t c = __float_as_uint(x[i].z) & 0x7fffffffu, d = __float_as_uint(x[i].w) & 0x7fffffffu;
    uint32_t top = max(max(a, b), max(c, d));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = block_scale<kE4m3>(top);
    uint32_t bits = 0;
    if (byte != 255) {
      const float f = __uint_as_float((254u - byte) << 23);  // 2^-e
      if (kE4m3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[i].x * f, x[i].y * f), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[i].z * f, x[i].w * f), __NV_SATFINITE, __NV_E4M3);
        bits = lo | (hi << 16);
      } else {
        bits = (uint32_t)(__float2int_rn(x[i].x * f) & 255) | ((uint32_t)(__float2int_rn(x[i].y * f) & 255) << 8) |
               ((uint32_t)(__float2int_rn(x[i].z * f) & 255) << 16) | ((uint32_t)__float2int_rn(x[i].w * f) << 24);
      }
    }
    // the row's four scale bytes leave as one word
    uint32_t word = byte << (lane & 24);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 16);
    if (lane == i) scales = word;
    const long long out = cache * p.elems + at;
    if (at < p.elems && in_bounds(out + kRow - 1, p.cache_extent, p.err))
      *reinterpret_cast<uint32_t *>(p.cache + out + 4 * lane) = bits;
  }
  const long long at = at0 + lane * kRow, out = cache * p.elems + at;
  if (lane < kUnroll && at < p.elems && in_bounds(out + kRow - 1, p.cache_extent, p.err))
    *reinterpret_cast<uint32_t *>(p.scales + out / 32) = scales;
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) state_load_kernel(const StateCachePlan p) {
  long long state, cache;
  if (!entry(p, false, blockIdx.y, &state, &cache)) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long at0 = (long long)blockIdx.x * kPerCta + warp * kUnroll * kRow;
  uint32_t x[kUnroll], sc[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long in = cache * p.elems + min(at0 + i * kRow, p.elems - kRow);
    x[i] = __ldcs(reinterpret_cast<const uint32_t *>(p.cache + in + 4 * lane));
    sc[i] = *(p.scales + in / 32 + lane / 8);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long at = at0 + i * kRow;
    if (at >= p.elems) break;
    // 2^e: byte 0 is the subnormal 2^-127; 255 is NaN
    const float f = __uint_as_float(sc[i] == 255 ? 0x7fffffffu : sc[i] == 0 ? 0x400000u : sc[i] << 23);
    float4 v;
    if (kE4m3) {
      const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[i] & 0xffffu), __NV_E4M3);
      const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[i] >> 16), __NV_E4M3);
      const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
      v = make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
    } else {
      v = make_float4((float)(int8_t)(x[i] & 255) * f, (float)(int8_t)((x[i] >> 8) & 255) * f,
                      (float)(int8_t)((x[i] >> 16) & 255) * f, (float)(int8_t)(x[i] >> 24) * f);
    }
    const long long out = state * p.elems + at + 4 * lane;
    if (in_bounds(out + 3, p.states_extent, p.err))
      __stcs(reinterpret_cast<float4 *>(p.states + out), v);
  }
}

}  // namespace

cudaError_t launch_state_store(const StateCachePlan &p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.elems + kPerCta - 1) / kPerCta), p.count);
  if (p.format == SSD_STATE_E4M3) state_store_kernel<true><<<grid, kThreads, 0, s>>>(p);
  else state_store_kernel<false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_state_load(const StateCachePlan &p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.elems + kPerCta - 1) / kPerCta), p.count);
  if (p.format == SSD_STATE_E4M3) state_load_kernel<true><<<grid, kThreads, 0, s>>>(p);
  else state_load_kernel<false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssd
