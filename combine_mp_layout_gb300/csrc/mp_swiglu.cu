// mp_swiglu.cu -- the gated activation between an expert's two products,
// quantised for the second one, and its gradient, quantised for the gradient
// products.
//
//   z_i = w_r * g_i / (1 + exp(-g_i)) * u_i      (w_r: the row's routing weight, or 1)
//   dg_i = w_r dz_i u_i sig_i (1 + g_i (1 - sig_i)),  du_i = w_r dz_i g_i sig_i,
//   dw_r = sum_i dz_i g_i sig_i u_i,                   sig_i = 1 / (1 + exp(-g_i))
// Quantisation: per 128 channels scale = amax * (1 / 448), codes e4m3(value * (1 /
// scale)) (scale 1, all codes 0, for a block whose scale would be below 2^-126).
// Both products are with a rounded reciprocal: the scale is within one fp32 ulp of
// amax / 448 and the value that is rounded to a code within 1.5 ulp of value / scale.
// The dispatch rounds the quotients themselves, so for the same values its scales can
// differ in the last bit, and a code where the quotient lies that near the middle of
// two.  (With the codes' quotients the gradient takes 102 us instead of 91.)
//
// Both kernels are bound by memory: they read bf16 once and write one byte per
// value.  A lane holds 16 channels (one 32-byte load per operand), eight lanes
// a scale block, a warp four blocks at a time; the arithmetic is in packed fp32
// pairs, and the gradient's registers are held to 64 so that eight blocks share
// an SM (104 us with 93 registers, 92 us with 64).
// Measured at 32,768 rows of 2,048 channels with row weights: forward 58.5 us (5.8
// TB/s), gradient 92 us (5.9 TB/s); 64 rows: 2.7 us.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_gate.cuh"
#include "mp_internal.h"

namespace mp {

namespace {

constexpr int kSwWarps = 4;
constexpr int kCPL = 16;                  // channels per lane
constexpr int kSpan = kCPL * kWarp;       // channels per warp and step
constexpr int kBlocksPerSM = 64;          // of a full grid; larger problems loop

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

// 16 bf16 channels of one lane, as their eight words (32-byte loads where the
// base allows).
template <bool A32>
__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[8]) {
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
}
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// Quantises the lane's 16 values (its block's other values in the seven lanes
// beside it) and stores codes and scale.  Every lane of the warp calls it.
__device__ __forceinline__ void quantise_store(const float2 (&z)[kCPL / 2], bool valid,
                                               unsigned char* codes, float* scale) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kCPL / 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(z[i].x), fabsf(z[i].y)));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  float sc = amax * (1.0f / 448.0f);
  if (!(sc >= 0x1p-126f)) sc = 1.0f;
  const float inv = sc < INFINITY ? __fdiv_rn(1.0f, sc) : 0.0f;
  if (!valid) return;
  const float2 inv2 = make_float2(inv, inv);
  Words<4> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q.w[i] = e4m3x4(mul2(z[2 * i], inv2), mul2(z[2 * i + 1], inv2));
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
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int spans = (p.I - 1) / kSpan + 1;
  const int64_t units = int64_t(live_rows(p)) * spans;
  const int64_t nw = int64_t(gridDim.x) * kSwWarps;
  for (int64_t unit = int64_t(blockIdx.x) * kSwWarps + (threadIdx.x >> 5); unit < units;
       unit += nw) {
    const int64_t row = unit / spans;
    // (unsigned, here and below: the channels after a row's last may lie past 2^31)
    const uint32_t ch = uint32_t(unit - row * spans) * kSpan + lane * kCPL;
    const bool valid = ch < uint32_t(p.I);
    uint32_t g[kCPL / 2] = {}, u[kCPL / 2] = {};
    if (valid) {
      const uint16_t* src = p.gate_up + row * 2 * p.I + ch;
      load16<A32>(src, g);
      load16<A32>(src + p.I, u);
    }
    const float w = p.row_weights != nullptr ? __ldg(p.row_weights + row) : 1.0f;
    const float2 w2 = make_float2(w, w);
    float2 z[kCPL / 2];
#pragma unroll
    for (int i = 0; i < kCPL / 2; ++i) {
      const float2 gate = unpack2(g[i]);
      z[i] = mul2(mul2(mul2(gate, sigmoid2(gate)), unpack2(u[i])), w2);
    }
    quantise_store(z, valid, p.out + row * p.I + ch, p.out_scales + row * (p.I / 128) + ch / 128);
  }
}

// WPR warps (1, 2 or 4) per row take the row's spans in turn; the row weight's
// gradient is added up in a fixed order (lanes, then warps).
template <bool A32, int WPR>
__global__ void __launch_bounds__(kSwWarps * kWarp, 8)
mp_k_swiglu_backward(const SwigluArgs p) {
  pdl_wait_prior_grid();
  __shared__ float red[2][kSwWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kRows = kSwWarps / WPR;
  const int rows = live_rows(p);
  int flip = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < rows;
       r0 += int64_t(gridDim.x) * kRows, flip ^= 1) {
    const int64_t row = r0 + warp / WPR;
    const bool live = row < rows;
    const float w = live && p.row_weights != nullptr ? __ldg(p.row_weights + row) : 1.0f;
    const float2 w2 = make_float2(w, w), one = make_float2(1.0f, 1.0f);
    float2 dw = make_float2(0.0f, 0.0f);
    for (uint32_t c0 = (warp % WPR) * kSpan; live && c0 < uint32_t(p.I); c0 += WPR * kSpan) {
      const uint32_t ch = c0 + lane * kCPL;
      const bool valid = ch < uint32_t(p.I);
      uint32_t g[kCPL / 2] = {}, u[kCPL / 2] = {}, d[kCPL / 2] = {};
      if (valid) {
        const uint16_t* src = p.gate_up + row * 2 * p.I + ch;
        load16<A32>(src, g);
        load16<A32>(src + p.I, u);
        load16<A32>(p.d_out + row * p.I + ch, d);
      }
      float2 dg[kCPL / 2], du[kCPL / 2];
#pragma unroll
      for (int i = 0; i < kCPL / 2; ++i) {
        const float2 gate = unpack2(g[i]), up = unpack2(u[i]), dz = unpack2(d[i]);
        const float2 sig = sigmoid2(gate);
        const float2 act = mul2(gate, sig);
        dw = fma2(mul2(dz, act), up, dw);
        const float2 dd = mul2(dz, w2);
        du[i] = mul2(dd, act);
        // sig (1 + gate (1 - sig)) = sig + act (1 - sig)
        const float2 slope = fma2(act, fma2(sig, make_float2(-1.0f, -1.0f), one), sig);
        dg[i] = mul2(mul2(dd, up), slope);
      }
      unsigned char* codes = p.out + row * 2 * p.I + ch;
      float* scales = p.out_scales + row * (p.I / 64) + ch / 128;
      quantise_store(dg, valid, codes, scales);
      quantise_store(du, valid, codes + p.I, scales + p.I / 128);
    }
    if (p.d_row_weights != nullptr) {
      float sum = dw.x + dw.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if constexpr (WPR == 1) {
        if (live && lane == 0) p.d_row_weights[row] = sum;
      } else {
        if (lane == 0) red[flip][warp] = sum;
        __syncthreads();  // (two buffers: one barrier per turn is enough)
        if (live && lane == 0 && warp % WPR == 0) {
          float all = 0.0f;
#pragma unroll
          for (int i = 0; i < WPR; ++i) all += red[flip][warp + i];
          p.d_row_weights[row] = all;
        }
      }
    }
  }
}

// A thread per (token, slot): its weight to the row that the slot was given, or
// (BACK) the row's gradient back to the slot.
template <bool BACK>
__global__ void __launch_bounds__(256)
mp_k_ll_row_weights(int64_t slots, int64_t rows, const int32_t* __restrict__ slot_row,
                    const float* __restrict__ in, float* __restrict__ out) {
  pdl_wait_prior_grid();
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= slots) return;
  const int row = __ldg(slot_row + i);
  const bool placed = row >= 0 && row < rows;
  if constexpr (BACK)
    out[i] = placed ? __ldg(in + row) : 0.0f;
  else if (placed)
    out[row] = __ldg(in + i);
}

unsigned grid_for(int64_t blocks) {
  return unsigned(std::min<int64_t>(blocks, int64_t(sm_count()) * kBlocksPerSM));
}

template <bool A32>
cudaError_t launch_backward(const SwigluArgs& p, cudaStream_t st) {
  const int spans = (p.I - 1) / kSpan + 1;
  const int64_t rows = p.rows;
  const dim3 block(kSwWarps * kWarp);
  if (spans == 1)
    return launch_waiting(mp_k_swiglu_backward<A32, 1>, dim3(grid_for((rows + 3) / 4)), block, 0,
                          st, 0, p);
  if (spans == 2)
    return launch_waiting(mp_k_swiglu_backward<A32, 2>, dim3(grid_for((rows + 1) / 2)), block, 0,
                          st, 0, p);
  return launch_waiting(mp_k_swiglu_backward<A32, 4>, dim3(grid_for(rows)), block, 0, st, 0, p);
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
  const int64_t units = int64_t(rows) * ((I - 1) / kSpan + 1);
  const unsigned blocks = grid_for((units + kSwWarps - 1) / kSwWarps);
  const bool a32 = (reinterpret_cast<uintptr_t>(gate_up) & 31u) == 0;
  return launch_waiting(a32 ? mp_k_swiglu<true> : mp_k_swiglu<false>, dim3(blocks),
                        dim3(kSwWarps * kWarp), 0, st, 0, p);
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
  return a32 ? launch_backward<true>(p, st) : launch_backward<false>(p, st);
}

cudaError_t launch_ll_row_weights(int64_t slots, int64_t rows, bool back, const int32_t* slot_row,
                                  const float* in, float* out, cudaStream_t st) {
  if (slots == 0) return cudaSuccess;
  const unsigned blocks = unsigned((slots + 255) / 256);
  return launch_waiting(back ? mp_k_ll_row_weights<true> : mp_k_ll_row_weights<false>,
                        dim3(blocks), dim3(256), 0, st, 0, slots, rows, slot_row, in, out);
}

}  // namespace mp
