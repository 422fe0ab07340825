// mp_expert_abi.cu -- the C ABI of the expert layer's operators (router, block-
// scaled products, gated activation) declared in include/mp_layout.h: argument
// checks, then one launch per call.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_internal.h"

namespace {

using namespace mp;

bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
constexpr int64_t k31 = int64_t(1) << 31;
int status_of(cudaError_t e) { return e == cudaSuccess ? MP_OK : MP_ERR_CUDA; }

bool route_shape_ok(int R, int N, int K, int E) {
  return R >= 1 && R <= MP_MAX_RANKS && N >= 0 && K >= 1 && K <= MP_MAX_TOPK && E >= K &&
         E <= MP_MAX_EXPERTS && int64_t(R) * N * K < k31;
}

// Checks common to the router and its gradient.
bool route_args_ok(int R, int N, int K, int E, int scoring, int dtype, const void* logits,
                   const int32_t* topk_idx, const int32_t* counts, const int32_t* routed) {
  if (!route_shape_ok(R, N, K, E)) return false;
  if (scoring != MP_SOFTMAX && scoring != MP_SIGMOID) return false;
  if (dtype != MP_FP32 && dtype != MP_BF16) return false;
  if (!counts || !routed || (N > 0 && (!logits || !topk_idx))) return false;
  return aligned_to(logits, dtype == MP_FP32 ? 4 : 2) && aligned_to(topk_idx, 4) &&
         aligned_to(counts, 4) && aligned_to(routed, 4);
}

// Checks common to the three products: rows with their scales on one side (and
// on the other, for the weights' gradient).
bool matmul_args_ok(int E, int rows, int N, int K, const void* a, const float* a_scales,
                    const void* w, const float* w_scales, bool w_always,
                    const int32_t* expert_offsets, const void* out, bool out_always,
                    const int32_t* dev_err) {
  if (E < 1 || E > MP_MAX_EXPERTS || rows < 0 || N < 1 || K < 1) return false;
  if (K % MP_SCALE_BLOCK != 0 || int64_t(E) * N >= k31) return false;
  if (rows > INT32_MAX - 1024) return false;  // a tile's last row index stays an int
  if (!dev_err || (!expert_offsets && E != 1)) return false;
  if (rows > 0 && (!a || !a_scales)) return false;
  if ((rows > 0 || w_always) && (!w || !w_scales)) return false;
  if ((rows > 0 || out_always) && !out) return false;
  return aligned_to(a, 16) && aligned_to(w, 16) && aligned_to(out, 16) &&
         aligned_to(a_scales, 4) && aligned_to(w_scales, 4) && aligned_to(expert_offsets, 4) &&
         aligned_to(dev_err, 4);
}

// Row tiles of 64 rows or more, at most one short one per expert, times column
// tiles of 256 channels.
bool tiles_ok(int E, int rows, int cols) {
  return (int64_t(rows) / 64 + E) * ((int64_t(cols) + 255) / 256) < k31;
}

}  // namespace

extern "C" {

size_t mp_route_workspace_size(int R, int N, int E) {
  if (!route_shape_ok(R, N, 1, E)) return 0;
  return route_workspace_bytes(R, E);
}

int mp_route(int R, int N, int K, int E, int scoring, int dtype, const void* logits,
             const float* bias, const uint8_t* active, int normalize, float scale,
             float loss_coef, int32_t* topk_idx, float* topk_weights,
             int32_t* num_tokens_per_expert, int32_t* num_routed, float* balance_loss,
             int32_t* dev_err, void* workspace, mp_stream_t stream) {
  if (!route_args_ok(R, N, K, E, scoring, dtype, logits, topk_idx, num_tokens_per_expert,
                     num_routed))
    return MP_ERR_INVALID_ARG;
  if (bias && scoring != MP_SIGMOID) return MP_ERR_INVALID_ARG;
  if (!balance_loss || !dev_err || !workspace || (N > 0 && !topk_weights))
    return MP_ERR_INVALID_ARG;
  if (!aligned_to(bias, 4) || !aligned_to(topk_weights, 4) || !aligned_to(balance_loss, 4) ||
      !aligned_to(dev_err, 4) || !aligned_to(workspace, 16))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_route(R, N, K, E, scoring, dtype, logits, bias, active, normalize,
                                scale, loss_coef, topk_idx, topk_weights, num_tokens_per_expert,
                                num_routed, balance_loss, dev_err,
                                static_cast<unsigned char*>(workspace),
                                reinterpret_cast<cudaStream_t>(stream)));
}

int mp_route_backward(int R, int N, int K, int E, int scoring, int dtype, const void* logits,
                      const uint8_t* active, int normalize, float scale, float loss_coef,
                      const int32_t* topk_idx, const float* d_topk_weights,
                      const int32_t* num_tokens_per_expert, const int32_t* num_routed,
                      const float* d_balance_loss, void* d_logits, mp_stream_t stream) {
  if (!route_args_ok(R, N, K, E, scoring, dtype, logits, topk_idx, num_tokens_per_expert,
                     num_routed))
    return MP_ERR_INVALID_ARG;
  if (N > 0 && !d_logits) return MP_ERR_INVALID_ARG;
  if (!aligned_to(d_logits, dtype == MP_FP32 ? 4 : 2) || !aligned_to(d_topk_weights, 4) ||
      !aligned_to(d_balance_loss, 4))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_route_backward(R, N, K, E, scoring, dtype, logits, active, normalize,
                                         scale, loss_coef, topk_idx, d_topk_weights,
                                         num_tokens_per_expert, num_routed, d_balance_loss,
                                         d_logits, reinterpret_cast<cudaStream_t>(stream)));
}

int mp_expert_matmul_e4m3(int E, int rows, int N, int K, const void* a, const float* a_scales,
                          const void* w, const float* w_scales, const int32_t* expert_offsets,
                          void* out, int32_t* dev_err, mp_stream_t stream) {
  if (!matmul_args_ok(E, rows, N, K, a, a_scales, w, w_scales, true, expert_offsets, out, false,
                      dev_err) ||
      N % 16 != 0 || !tiles_ok(E, rows, N))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_matmul(E, rows, N, K, false, a, a_scales, w, w_scales,
                                        expert_offsets, out, dev_err,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int mp_expert_matmul_dgrad_e4m3(int E, int rows, int N, int K, const void* dy,
                                const float* dy_scales, const void* w, const float* w_scales,
                                const int32_t* expert_offsets, void* dx, int32_t* dev_err,
                                mp_stream_t stream) {
  if (!matmul_args_ok(E, rows, N, K, dy, dy_scales, w, w_scales, true, expert_offsets, dx, false,
                      dev_err) ||
      N % MP_SCALE_BLOCK != 0 || !tiles_ok(E, rows, K))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_matmul(E, rows, N, K, true, dy, dy_scales, w, w_scales,
                                        expert_offsets, dx, dev_err,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int mp_expert_matmul_wgrad_e4m3(int E, int rows, int N, int K, const void* dy,
                                const float* dy_scales, const void* a, const float* a_scales,
                                const int32_t* expert_offsets, void* dw, int32_t* dev_err,
                                mp_stream_t stream) {
  if (!matmul_args_ok(E, rows, N, K, dy, dy_scales, a, a_scales, false, expert_offsets, dw, true,
                      dev_err) ||
      N % MP_SCALE_BLOCK != 0 ||
      int64_t(E) * (N / 128) * ((int64_t(K) + 255) / 256) >= k31)
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_wgrad(E, rows, N, K, dy, dy_scales, a, a_scales, expert_offsets,
                                       dw, dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

int mp_swiglu_e4m3(int rows, int I, const void* gate_up, const float* row_weights,
                   const int32_t* num_rows, void* out, float* out_scales, mp_stream_t stream) {
  if (rows < 0 || I < 1 || I % MP_SCALE_BLOCK != 0) return MP_ERR_INVALID_ARG;
  if (rows > 0 && (!gate_up || !out || !out_scales)) return MP_ERR_INVALID_ARG;
  if (!aligned_to(gate_up, 16) || !aligned_to(out, 16) || !aligned_to(out_scales, 4) ||
      !aligned_to(row_weights, 4) || !aligned_to(num_rows, 4))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_swiglu(rows, I, gate_up, row_weights, num_rows, out, out_scales,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

int mp_swiglu_backward_e4m3(int rows, int I, const void* gate_up, const float* row_weights,
                            const void* d_out, const int32_t* num_rows, void* d_gate_up,
                            float* d_gate_up_scales, float* d_row_weights, mp_stream_t stream) {
  if (rows < 0 || I < 1 || I % MP_SCALE_BLOCK != 0) return MP_ERR_INVALID_ARG;
  if (rows > 0 && (!gate_up || !d_out || !d_gate_up || !d_gate_up_scales))
    return MP_ERR_INVALID_ARG;
  if (!aligned_to(gate_up, 16) || !aligned_to(d_out, 16) || !aligned_to(d_gate_up, 16) ||
      !aligned_to(d_gate_up_scales, 4) || !aligned_to(row_weights, 4) ||
      !aligned_to(num_rows, 4) || !aligned_to(d_row_weights, 4))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_swiglu_backward(rows, I, gate_up, row_weights, d_out, num_rows,
                                          d_gate_up, d_gate_up_scales, d_row_weights,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

int ll_row_weights(int R, int N, int K, const int32_t* slot_row, int64_t rows, bool back,
                   const float* in, const float* in_slots, float* out, const float* out_slots,
                   mp_stream_t stream) {
  if (R < 1 || R > MP_MAX_RANKS || N < 0 || K < 1 || K > MP_MAX_TOPK || rows < 0 ||
      int64_t(R) * N * K >= k31)
    return MP_ERR_INVALID_ARG;
  if (N > 0 && (!slot_row || !(back ? out_slots : in_slots))) return MP_ERR_INVALID_ARG;
  if (rows > 0 && !(back ? in : out)) return MP_ERR_INVALID_ARG;
  if (!aligned_to(slot_row, 4) || !aligned_to(in, 4) || !aligned_to(out, 4))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_ll_row_weights(int64_t(R) * N * K, rows, back, slot_row, in, out,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

int mp_ll_row_weights(int R, int N, int K, const float* topk_weights, const int32_t* slot_row,
                      int64_t recv_capacity, float* row_weights, mp_stream_t stream) {
  return ll_row_weights(R, N, K, slot_row, recv_capacity, false, topk_weights, topk_weights,
                        row_weights, nullptr, stream);
}

int mp_ll_row_weights_backward(int R, int N, int K, const float* d_row_weights, int64_t rows,
                               const int32_t* slot_row, float* d_topk_weights,
                               mp_stream_t stream) {
  return ll_row_weights(R, N, K, slot_row, rows, true, d_row_weights, nullptr, d_topk_weights,
                        d_topk_weights, stream);
}

}  // extern "C"
