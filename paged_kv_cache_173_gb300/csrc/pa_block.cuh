// pa_block.cuh -- device helpers shared by the kernels that keep side data
// per (block, KV head): power-of-two exponents of block scales and bounds.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

namespace {

constexpr int kMinScaleExp = -64;   // smallest block scale the writer makes: 2^-64
constexpr int kMinBoundExp = -100;  // smallest exponent of the key bounds and whole-number queries
constexpr float kFloatMax = 3.402823466e38f;

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// The smallest e >= floor with amax <= top * 2^e, where top = (1 + TOP_FRAC / 2^23) * 2^TOP_EXP
// and amax >= 0 is finite.  A float is (1 + frac / 2^23) * 2^x, so e is x - TOP_EXP
// unless its fraction is above top's.
template <int TOP_EXP, int TOP_FRAC>
__device__ __forceinline__ int least_exp(float amax, int floor) {
  const int bits = __float_as_int(amax);
  const int x = (bits >> 23) - 127;
  const int e = x - TOP_EXP + ((bits & 0x7fffff) > TOP_FRAC ? 1 : 0);
  return e > floor ? e : floor;
}

// 448 = 1.75 * 2^8: the largest E4M3 value.
__device__ __forceinline__ int scale_exp(float amax) { return least_exp<8, 0x600000>(amax, kMinScaleExp); }
// 127 = 1.984375 * 2^6: the largest bound code.
__device__ __forceinline__ int bound_exp(float amax) { return least_exp<6, 0x7e0000>(amax, kMinBoundExp); }
// 255 = 1.9921875 * 2^7: the largest whole-number query element.
__device__ __forceinline__ int query_exp(float amax) { return least_exp<7, 0x7f0000>(amax, kMinBoundExp); }

// |x| where x is finite, else 0: non-finite elements set no scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= kFloatMax ? a : 0.f;
}

// Two to four units in the last place of x above it: a maximum that has room for the roundings of
// what is taken off it before it is the largest weight's exponent, which float16 bounds.
__device__ __forceinline__ float rounded_up(float x) { return fmaf(fabsf(x), 2.384185791015625e-7f, x); }

}  // namespace

}  // namespace pa
