// mp_gate.cuh -- what the gated activation's kernels share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mp_common.cuh"

namespace mp {

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}

// 1 / (1 + exp(-x)) of two channels from the fast exponential and reciprocal.  The
// exponential's argument is rounded to fp32, so for negative x the error grows with
// |x|: 2e-7 at -4, 8e-7 at -15, 3.4e-6 at -84, and the two functions' few ulps.  That
// is far below the rounding to e4m3 or bf16 that follows; in the row weight's gradient,
// which is not rounded so, such gates' terms are small.  Below -87.3 the result is
// subnormal and loses bits, and from -88.8 on exp(-x) is infinite and the result 0.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float2 t = mul2(x, make_float2(-kLog2e, -kLog2e));
  float2 e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = add2(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return r;
}

// The same in two factors, the result and `k`, for channels below kFarGate too: there
// both are exp(x / 2) = 1 / (1 + exp(-x / 2)) (to fp32), which is a normal number down to
// -174 and 0 from -177.4 on; elsewhere k is 1 and the result as above, to the bit.  What
// is to be multiplied by the sigmoid takes the one factor first and `k` last, so that a
// large value in between brings the product back into range.
constexpr float kFarGate = -80.0f;
__device__ __forceinline__ float2 sigmoid2_far(float2 x, float2& k) {
  const bool fx = x.x < kFarGate, fy = x.y < kFarGate;
  // (half of a float is exact: the exponential's argument is half of what it was)
  const float2 r = sigmoid2(make_float2(fx ? 0.5f * x.x : x.x, fy ? 0.5f * x.y : x.y));
  k = make_float2(fx ? r.x : 1.0f, fy ? r.y : 1.0f);
  return r;
}

}  // namespace mp
