// mp_swiglu_bf16.cu -- the gated activation between an expert's two bf16 products,
// and its gradient.
//
//   z_i = w_r * g_i / (1 + exp(-g_i)) * u_i      (w_r: the row's routing weight, or 1)
//   dg_i = w_r dz_i u_i sig_i (1 + g_i (1 - sig_i)),  du_i = w_r dz_i g_i sig_i,
//   dw_r = sum_i dz_i g_i sig_i u_i,                   sig_i = 1 / (1 + exp(-g_i))
// in fp32 pairs, one rounding to bf16 per output; dw_r is summed in fp32 in a fixed
// order (a lane's channels, lanes, warps).
//
// Both are bound by memory: 6 bytes per channel forward, 10 in the gradient, read or
// written once, in 32-byte vectors (16 channels of a lane) where the rows allow it and
// 16-byte ones otherwise.  Measured at 32,768 rows of 2,048 channels with row weights:
// forward 60.0 us (6.7 TB/s), gradient 101 us (6.6 TB/s); 64 rows: 1.8 us.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_gate.cuh"
#include "mp_internal.h"

namespace mp {

namespace {

constexpr int kThreads = 128;
constexpr int kBlocksPerSM = 64;  // of a full grid; larger problems loop

struct GateArgs {
  int rows, I;
  const uint16_t* gate_up;   // bf16 [rows][2I]
  const float* row_weights;  // or NULL
  const int32_t* num_rows;   // or NULL
  const uint16_t* d_out;     // bf16 [rows][I] (gradient)
  uint16_t* out;             // bf16 [rows][I], gradient: [rows][2I]
  float* d_row_weights;      // [rows] or NULL
};

__device__ __forceinline__ int live_rows(const GateArgs& p) {
  if (p.num_rows == nullptr) return p.rows;
  return min(max(__ldg(p.num_rows), 0), p.rows);
}

// CPL channels (8 or 16) of one lane.
template <int CPL>
__device__ __forceinline__ Words<CPL / 2> load_ch(const uint16_t* p) {
  return ld_stream_w<CPL / 2>(reinterpret_cast<const Words<CPL / 2>*>(p));
}
template <int CPL>
__device__ __forceinline__ void store_ch(uint16_t* p, const float2 (&z)[CPL / 2]) {
  Words<CPL / 2> o;
#pragma unroll
  for (int i = 0; i < CPL / 2; ++i) o.w[i] = pack_bf16x2_rn(z[i].x, z[i].y);
  st_stream_w<CPL / 2>(reinterpret_cast<Words<CPL / 2>*>(p), o);
}

// Whether one of a lane's gates is below kFarGate.  Those lanes take a form of their own
// (FAR), which takes the sigmoid in two factors; the others' sums and roundings are
// what they are without it.  (The look at the gates costs nothing that shows: both
// kernels wait for memory.)
template <int W>
__device__ __forceinline__ bool any_far(const Words<W>& g) {
  uint32_t least = g.w[0];
#pragma unroll
  for (int i = 1; i < W; ++i)
    asm("min.bf16x2 %0, %0, %1;" : "+r"(least) : "r"(g.w[i]));
  return fminf(bf16_lo(least), bf16_hi(least)) < kFarGate;  // (NaN is never the least)
}

template <bool FAR, int CPL>
__device__ __forceinline__ void gated(const Words<CPL / 2>& g, const Words<CPL / 2>& u, float2 w2,
                                      float2 (&z)[CPL / 2]) {
#pragma unroll
  for (int j = 0; j < CPL / 2; ++j) {
    const float2 gate = unpack2(g.w[j]);
    float2 k;
    const float2 sig = FAR ? sigmoid2_far(gate, k) : sigmoid2(gate);
    z[j] = mul2(mul2(mul2(gate, sig), unpack2(u.w[j])), w2);
    if (FAR) z[j] = mul2(z[j], k);
  }
}

// One lane's channels of the gradient; their terms of the row weight's are added to dw.
template <bool FAR, int CPL>
__device__ __forceinline__ void gated_backward(const Words<CPL / 2>& g, const Words<CPL / 2>& u,
                                               const Words<CPL / 2>& d, float2 w2,
                                               float2 (&dg)[CPL / 2], float2 (&du)[CPL / 2],
                                               float2& dw) {
  const float2 one = make_float2(1.0f, 1.0f);
#pragma unroll
  for (int j = 0; j < CPL / 2; ++j) {
    const float2 gate = unpack2(g.w[j]), up = unpack2(u.w[j]), dz = unpack2(d.w[j]);
    float2 k;
    const float2 sig = FAR ? sigmoid2_far(gate, k) : sigmoid2(gate);
    const float2 act = mul2(gate, sig);
    dw = fma2(mul2(dz, act), FAR ? mul2(up, k) : up, dw);
    const float2 dd = mul2(dz, w2);
    du[j] = mul2(dd, act);
    // sig (1 + gate (1 - sig)) = sig + act (1 - sig)
    const float2 slope = fma2(act, fma2(sig, make_float2(-1.0f, -1.0f), one), sig);
    dg[j] = mul2(mul2(dd, up), slope);
    if (FAR) {  // (1 - sig, with half of the exponent, is 1 in fp32 all the same)
      du[j] = mul2(du[j], k);
      dg[j] = mul2(dg[j], k);
    }
  }
}

// A thread per vector of CPL channels.  Index: uint32_t while all vectors' numbers
// (and one grid more) fit, which makes the division to the row a short one.
template <int CPL, typename Index>
__global__ void __launch_bounds__(kThreads)
mp_k_swiglu_bf16(const GateArgs p) {
  pdl_wait_prior_grid();
  const Index per = Index(p.I / CPL);
  const Index all = Index(live_rows(p)) * per, step = Index(gridDim.x) * kThreads;
  for (Index i = Index(blockIdx.x) * kThreads + threadIdx.x; i < all; i += step) {
    const Index row = i / per;
    const int64_t ch = int64_t(i - row * per) * CPL;
    const uint16_t* src = p.gate_up + int64_t(row) * 2 * p.I + ch;
    const Words<CPL / 2> g = load_ch<CPL>(src), u = load_ch<CPL>(src + p.I);
    const float w = p.row_weights != nullptr ? __ldg(p.row_weights + row) : 1.0f;
    const float2 w2 = make_float2(w, w);
    float2 z[CPL / 2];
    if (any_far(g))
      gated<true, CPL>(g, u, w2, z);
    else
      gated<false, CPL>(g, u, w2, z);
    store_ch<CPL>(p.out + int64_t(row) * p.I + ch, z);
  }
}

// LPR lanes (8 to 128) per row take the row's vectors in turn.
template <int CPL, int LPR>
__global__ void __launch_bounds__(kThreads, 8)
mp_k_swiglu_backward_bf16(const GateArgs p) {
  pdl_wait_prior_grid();
  __shared__ float red[2][kThreads / kWarp];
  constexpr int kRows = kThreads / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = threadIdx.x % LPR;
  const int rows = live_rows(p);
  int flip = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < rows;
       r0 += int64_t(gridDim.x) * kRows, flip ^= 1) {
    const int64_t row = r0 + threadIdx.x / LPR;
    const bool live = row < rows;
    const float w = live && p.row_weights != nullptr ? __ldg(p.row_weights + row) : 1.0f;
    const float2 w2 = make_float2(w, w);
    float2 dw = make_float2(0.0f, 0.0f);
    for (uint32_t ch = at * CPL; live && ch < uint32_t(p.I); ch += LPR * CPL) {
      const uint16_t* src = p.gate_up + row * 2 * p.I + ch;
      const Words<CPL / 2> g = load_ch<CPL>(src), u = load_ch<CPL>(src + p.I);
      const Words<CPL / 2> d = load_ch<CPL>(p.d_out + row * p.I + ch);
      float2 dg[CPL / 2], du[CPL / 2];
      if (any_far(g))
        gated_backward<true, CPL>(g, u, d, w2, dg, du, dw);
      else
        gated_backward<false, CPL>(g, u, d, w2, dg, du, dw);
      uint16_t* dst = p.out + row * 2 * p.I + ch;
      store_ch<CPL>(dst, dg);
      store_ch<CPL>(dst + p.I, du);
    }
    if (p.d_row_weights != nullptr) {
      float sum = dw.x + dw.y;
#pragma unroll
      for (int o = (LPR < kWarp ? LPR : kWarp) / 2; o > 0; o >>= 1)
        sum += __shfl_xor_sync(kFull, sum, o);
      if constexpr (LPR <= kWarp) {
        if (live && at == 0) p.d_row_weights[row] = sum;
      } else {
        if (lane == 0) red[flip][warp] = sum;
        __syncthreads();  // (two buffers: one barrier per turn is enough)
        if (live && at == 0) {
          float all = 0.0f;
#pragma unroll
          for (int i = 0; i < LPR / kWarp; ++i) all += red[flip][warp + i];
          p.d_row_weights[row] = all;
        }
      }
    }
  }
}

unsigned grid_for(int64_t blocks) {
  return unsigned(std::min<int64_t>(blocks, int64_t(sm_count()) * kBlocksPerSM));
}

template <int CPL, int LPR>
cudaError_t launch_backward_as(const GateArgs& p, cudaStream_t st) {
  constexpr int kRows = kThreads / LPR;
  return launch_waiting(mp_k_swiglu_backward_bf16<CPL, LPR>,
                        dim3(grid_for((int64_t(p.rows) + kRows - 1) / kRows)), dim3(kThreads), 0,
                        st, 0, p);
}

// Lanes per row: what the row's vectors fill once, between 8 lanes and a block.
template <int CPL>
cudaError_t launch_backward(const GateArgs& p, cudaStream_t st) {
  const int per = p.I / CPL;
  if (per <= 8) return launch_backward_as<CPL, 8>(p, st);
  if (per <= 32) return launch_backward_as<CPL, 32>(p, st);
  return launch_backward_as<CPL, 128>(p, st);
}

template <int CPL>
cudaError_t launch_forward(const GateArgs& p, cudaStream_t st) {
  const int64_t all = int64_t(p.rows) * (p.I / CPL);
  const unsigned blocks = grid_for((all + kThreads - 1) / kThreads);
  const bool small = all + int64_t(blocks) * kThreads < (int64_t(1) << 32);
  return launch_waiting(small ? mp_k_swiglu_bf16<CPL, uint32_t> : mp_k_swiglu_bf16<CPL, uint64_t>,
                        dim3(blocks), dim3(kThreads), 0, st, 0, p);
}

bool wide(int I, uintptr_t pointers) { return I % 16 == 0 && (pointers & 31u) == 0; }

}  // namespace

cudaError_t launch_swiglu_bf16(int rows, int I, const void* gate_up, const float* row_weights,
                               const int32_t* num_rows, void* out, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  GateArgs p = {};
  p.rows = rows; p.I = I;
  p.gate_up = static_cast<const uint16_t*>(gate_up);
  p.row_weights = row_weights; p.num_rows = num_rows;
  p.out = static_cast<uint16_t*>(out);
  return wide(I, reinterpret_cast<uintptr_t>(gate_up) | reinterpret_cast<uintptr_t>(out))
             ? launch_forward<16>(p, st)
             : launch_forward<8>(p, st);
}

cudaError_t launch_swiglu_backward_bf16(int rows, int I, const void* gate_up,
                                        const float* row_weights, const void* d_out,
                                        const int32_t* num_rows, void* d_gate_up,
                                        float* d_row_weights, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  GateArgs p = {};
  p.rows = rows; p.I = I;
  p.gate_up = static_cast<const uint16_t*>(gate_up);
  p.row_weights = row_weights; p.num_rows = num_rows;
  p.d_out = static_cast<const uint16_t*>(d_out);
  p.out = static_cast<uint16_t*>(d_gate_up);
  p.d_row_weights = d_row_weights;
  return wide(I, reinterpret_cast<uintptr_t>(gate_up) | reinterpret_cast<uintptr_t>(d_out) |
                     reinterpret_cast<uintptr_t>(d_gate_up))
             ? launch_backward<16>(p, st)
             : launch_backward<8>(p, st);
}

}  // namespace mp
