// mp_swiglu.cu -- the gated activation between an expert's two products,
// quantised for the second one, and its gradient, quantised for the gradient
// products.
//
//   z_i = w_r * g_i / (1 + exp(-g_i)) * u_i      (w_r: the row's routing weight, or 1)
//   dg_i = w_r dz_i u_i sig_i (1 + g_i (1 - sig_i)),  du_i = w_r dz_i g_i sig_i,
//   dw_r = sum_i dz_i g_i sig_i u_i,                   sig_i = 1 / (1 + exp(-g_i))
// Quantisation as on dispatch: per 128 channels scale = amax / 448, codes
// e4m3(value / scale) (scale 1, all codes 0, for a block whose scale would be
// below 2^-126).
//
// Both kernels are bound by memory: they read bf16 once and write one byte per
// value.  A lane holds 16 channels (one 32-byte load per operand), eight lanes
// a scale block, a warp four blocks at a time.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_internal.h"

namespace mp {

namespace {

constexpr int kSwWarps = 4;
constexpr int kCPL = 16;                  // channels per lane
constexpr int kSpan = kCPL * kWarp;       // channels per warp and step

struct SwigluArgs {
  int rows, I;
  const uint16_t* gate_up;   // bf16 [rows][2I]
  const float* row_weights;  // or NULL
  const int32_t* num_rows;   // or NULL
  const uint16_t* d_out;     // bf16 [rows][I] (gradient)
  unsigned char* out;        // e4m3 [rows][I], gradient: [rows][2I]
  float* out_scales;
  float* d_row_weights;      // [rows] or NULL
};

// 16 bf16 channels of one lane (32-byte loads where the base allows).
template <bool A32>
__device__ __forceinline__ void load16(const uint16_t* p, float (&f)[kCPL]) {
  uint32_t w[8];
  if constexpr (A32) {
    const Words<8> v = ld_stream_w<8>(reinterpret_cast<const Words<8>*>(p));
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v.w[i];
  } else {
    const Words<4> a = ld_stream_w<4>(reinterpret_cast<const Words<4>*>(p));
    const Words<4> b = ld_stream_w<4>(reinterpret_cast<const Words<4>*>(p) + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = a.w[i];
      w[4 + i] = b.w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

// 1 / (1 + exp(-x)) from the fast exponential and reciprocal: a few fp32 ulps,
// far below the e4m3 rounding that follows.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// Quantises the lane's 16 values (its block's other values in the seven lanes
// beside it) and stores codes and scale.  Every lane of the warp calls it.
__device__ __forceinline__ void quantise_store(const float (&z)[kCPL], bool valid,
                                               unsigned char* codes, float* scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kCPL; ++i) amax = fmaxf(amax, fabsf(z[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  float sc = amax * (1.0f / 448.0f);
  if (!(sc >= 0x1p-126f)) sc = 1.0f;
  const float inv = sc < INFINITY ? __fdiv_rn(1.0f, sc) : 0.0f;
  if (!valid) return;
  Words<4> q;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q.w[i] = e4m3x4(z[4 * i] * inv, z[4 * i + 1] * inv, z[4 * i + 2] * inv, z[4 * i + 3] * inv);
  st_stream_w<4>(reinterpret_cast<Words<4>*>(codes), q);
  if ((threadIdx.x & 7) == 0) *scale = sc;
}

__device__ __forceinline__ int live_rows(const SwigluArgs& p) {
  if (p.num_rows == nullptr) return p.rows;
  return min(max(__ldg(p.num_rows), 0), p.rows);
}

// A warp per (row, span of 512 channels).
template <bool A32>
__global__ void __launch_bounds__(kSwWarps * kWarp)
mp_k_swiglu(const SwigluArgs p) {
  const int lane = threadIdx.x & 31;
  const int spans = (p.I + kSpan - 1) / kSpan;
  const int64_t units = int64_t(live_rows(p)) * spans;
  const int64_t nw = int64_t(gridDim.x) * kSwWarps;
  for (int64_t unit = int64_t(blockIdx.x) * kSwWarps + (threadIdx.x >> 5); unit < units;
       unit += nw) {
    const int64_t row = unit / spans;
    const int ch = int(unit - row * spans) * kSpan + lane * kCPL;
    const bool valid = ch < p.I;
    float g[kCPL], u[kCPL];
    if (valid) {
      const uint16_t* src = p.gate_up + row * 2 * p.I + ch;
      load16<A32>(src, g);
      load16<A32>(src + p.I, u);
    } else {
#pragma unroll
      for (int i = 0; i < kCPL; ++i) g[i] = u[i] = 0.0f;
    }
    const float w = p.row_weights != nullptr ? __ldg(p.row_weights + row) : 1.0f;
#pragma unroll
    for (int i = 0; i < kCPL; ++i) g[i] = g[i] * sigmoid_fast(g[i]) * u[i] * w;
    quantise_store(g, valid, p.out + row * p.I + ch, p.out_scales + row * (p.I / 128) + ch / 128);
  }
}

// A block per row: its warps take the row's spans in turn, and the row weight's
// gradient is added up in a fixed order (lanes, then warps).
template <bool A32>
__global__ void __launch_bounds__(kSwWarps * kWarp)
mp_k_swiglu_backward(const SwigluArgs p) {
  __shared__ float red[2][kSwWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = live_rows(p);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, flip ^= 1) {
    const float w = p.row_weights != nullptr ? __ldg(p.row_weights + row) : 1.0f;
    float dw = 0.0f;
    for (int c0 = warp * kSpan; c0 < p.I; c0 += kSwWarps * kSpan) {
      const int ch = c0 + lane * kCPL;
      const bool valid = ch < p.I;
      float g[kCPL], u[kCPL], d[kCPL];
      if (valid) {
        const uint16_t* src = p.gate_up + row * 2 * p.I + ch;
        load16<A32>(src, g);
        load16<A32>(src + p.I, u);
        load16<A32>(p.d_out + row * p.I + ch, d);
      } else {
#pragma unroll
        for (int i = 0; i < kCPL; ++i) g[i] = u[i] = d[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kCPL; ++i) {
        const float sig = sigmoid_fast(g[i]);
        const float act = g[i] * sig;
        dw += d[i] * act * u[i];
        const float dd = d[i] * w;
        const float du = dd * act;
        g[i] = dd * u[i] * sig * (1.0f + g[i] * (1.0f - sig));
        u[i] = du;
      }
      unsigned char* codes = p.out + row * 2 * p.I + ch;
      float* scales = p.out_scales + row * (p.I / 64) + ch / 128;
      quantise_store(g, valid, codes, scales);
      quantise_store(u, valid, codes + p.I, scales + p.I / 128);
    }
    if (p.d_row_weights != nullptr) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dw += __shfl_xor_sync(kFull, dw, o);
      if (lane == 0) red[flip][warp] = dw;
      __syncthreads();  // (two buffers: one barrier per row is enough)
      if (threadIdx.x == 0) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < kSwWarps; ++i) all += red[flip][i];
        p.d_row_weights[row] = all;
      }
    }
  }
}

}  // namespace

cudaError_t launch_swiglu(int rows, int I, const void* gate_up, const float* row_weights,
                          const int32_t* num_rows, void* out, float* out_scales, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  SwigluArgs p = {};
  p.rows = rows; p.I = I;
  p.gate_up = static_cast<const uint16_t*>(gate_up);
  p.row_weights = row_weights; p.num_rows = num_rows;
  p.out = static_cast<unsigned char*>(out); p.out_scales = out_scales;
  const int64_t units = int64_t(rows) * ((I + kSpan - 1) / kSpan);
  const int64_t blocks = std::min<int64_t>((units + kSwWarps - 1) / kSwWarps, 0x7fffffff);
  const bool a32 = (reinterpret_cast<uintptr_t>(gate_up) & 31u) == 0;
  if (a32)
    mp_k_swiglu<true><<<unsigned(blocks), kSwWarps * kWarp, 0, st>>>(p);
  else
    mp_k_swiglu<false><<<unsigned(blocks), kSwWarps * kWarp, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_backward(int rows, int I, const void* gate_up, const float* row_weights,
                                   const void* d_out, const int32_t* num_rows, void* d_gate_up,
                                   float* d_gate_up_scales, float* d_row_weights,
                                   cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  SwigluArgs p = {};
  p.rows = rows; p.I = I;
  p.gate_up = static_cast<const uint16_t*>(gate_up);
  p.row_weights = row_weights; p.num_rows = num_rows;
  p.d_out = static_cast<const uint16_t*>(d_out);
  p.out = static_cast<unsigned char*>(d_gate_up); p.out_scales = d_gate_up_scales;
  p.d_row_weights = d_row_weights;
  const bool a32 = ((reinterpret_cast<uintptr_t>(gate_up) | reinterpret_cast<uintptr_t>(d_out)) &
                    31u) == 0;
  if (a32)
    mp_k_swiglu_backward<true><<<unsigned(rows), kSwWarps * kWarp, 0, st>>>(p);
  else
    mp_k_swiglu_backward<false><<<unsigned(rows), kSwWarps * kWarp, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace mp
