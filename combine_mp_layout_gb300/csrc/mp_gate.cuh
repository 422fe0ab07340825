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
// which is not rounded so, such gates' terms are small.
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

}  // namespace mp
