// mp_expert_bf16_abi.cu -- the C ABI of the expert layer's operators on bf16 rows
// (products with bf16 and 4-bit weights, gated activation) declared in include/mp_layout.h:
// argument checks, then one launch per call.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_internal.h"

namespace {

using namespace mp;

bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
constexpr int64_t k31 = int64_t(1) << 31, k40 = int64_t(1) << 40;
int status_of(cudaError_t e) { return e == cudaSuccess ? MP_OK : MP_ERR_CUDA; }

// Checks common to the products: `w` stands for the second operand (weights, or
// rows for the weights' gradient).
bool product_args_ok(int E, int rows, int N, int K, const void* a, const void* w, bool w_always,
                     const int32_t* expert_offsets, const void* out, bool out_always,
                     const int32_t* dev_err) {
  if (E < 1 || E > MP_MAX_EXPERTS || rows < 0 || N < 1 || K < 1) return false;
  if (N % 8 != 0 || K % 8 != 0 || N > INT32_MAX - 1024 || K > INT32_MAX - 1024) return false;
  if (rows > INT32_MAX - 1024) return false;  // a tile's last row index stays an int
  if (int64_t(N) * K >= k40 / 4) return false;  // a tensor map's stride, in bytes (fp32)
  if (!dev_err || (!expert_offsets && E != 1)) return false;
  if (rows > 0 && !a) return false;
  if ((rows > 0 || w_always) && !w) return false;
  if ((rows > 0 || out_always) && !out) return false;
  return aligned_to(a, 16) && aligned_to(w, 16) && aligned_to(out, 16) &&
         aligned_to(expert_offsets, 4) && aligned_to(dev_err, 4);
}

// Row tiles of `most` rows, at most one short one per expert, times column tiles of
// 256 channels; and as many more as there can be blocks, so that a loop over tiles
// ends before its counter does.
bool tiles_ok(int E, int rows, int cols, int most) {
  return (int64_t(rows) / most + E) * ((int64_t(cols) + 255) / 256) < k31 - 4096;
}

bool gate_args_ok(int rows, int I) {
  return rows >= 0 && I >= 1 && I % 8 == 0 && I <= INT32_MAX - 4096;
}

}  // namespace

extern "C" {

int mp_expert_matmul_bf16(int E, int rows, int N, int K, const void* a, const void* w,
                          const int32_t* expert_offsets, void* out, int32_t* dev_err,
                          mp_stream_t stream) {
  if (!product_args_ok(E, rows, N, K, a, w, true, expert_offsets, out, false, dev_err) ||
      !tiles_ok(E, rows, N, 256))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_matmul_bf16(E, rows, N, K, false, a, w, expert_offsets, out,
                                             dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

int mp_expert_matmul_dgrad_bf16(int E, int rows, int N, int K, const void* dy, const void* w,
                                const int32_t* expert_offsets, void* dx, int32_t* dev_err,
                                mp_stream_t stream) {
  if (!product_args_ok(E, rows, N, K, dy, w, true, expert_offsets, dx, false, dev_err) ||
      !tiles_ok(E, rows, K, 256))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_matmul_bf16(E, rows, N, K, true, dy, w, expert_offsets, dx,
                                             dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

int mp_expert_matmul_wgrad_bf16(int E, int rows, int N, int K, const void* dy, const void* a,
                                const int32_t* expert_offsets, int dw_dtype, int accumulate,
                                void* dw, int32_t* dev_err, mp_stream_t stream) {
  if (!product_args_ok(E, rows, N, K, dy, a, false, expert_offsets, dw, true, dev_err) ||
      (dw_dtype != MP_BF16 && dw_dtype != MP_FP32) || (accumulate && dw_dtype != MP_FP32) ||
      int64_t(E) * ((int64_t(N) + 255) / 256) * ((int64_t(K) + 255) / 256) >= k31 - 4096)
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_wgrad_bf16(E, rows, N, K, dy, a, expert_offsets,
                                            dw_dtype == MP_FP32, accumulate != 0, dw, dev_err,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

int mp_expert_matmul_mxfp4(int E, int rows, int N, int K, const void* a, const void* w,
                           const uint8_t* w_scales, const int32_t* expert_offsets, void* out,
                           int32_t* dev_err, mp_stream_t stream) {
  if (!product_args_ok(E, rows, N, K, a, w, true, expert_offsets, out, false, dev_err) ||
      K % MP_MX_BLOCK != 0 || !w_scales || !tiles_ok(E, rows, N, 160))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_expert_matmul_mxfp4(E, rows, N, K, a, w, w_scales, expert_offsets, out,
                                              dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

int mp_swiglu_bf16(int rows, int I, const void* gate_up, const float* row_weights,
                   const int32_t* num_rows, void* out, mp_stream_t stream) {
  if (!gate_args_ok(rows, I) || (rows > 0 && (!gate_up || !out))) return MP_ERR_INVALID_ARG;
  if (!aligned_to(gate_up, 16) || !aligned_to(out, 16) || !aligned_to(row_weights, 4) ||
      !aligned_to(num_rows, 4))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_swiglu_bf16(rows, I, gate_up, row_weights, num_rows, out,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int mp_swiglu_backward_bf16(int rows, int I, const void* gate_up, const float* row_weights,
                            const void* d_out, const int32_t* num_rows, void* d_gate_up,
                            float* d_row_weights, mp_stream_t stream) {
  if (!gate_args_ok(rows, I) || (rows > 0 && (!gate_up || !d_out || !d_gate_up)))
    return MP_ERR_INVALID_ARG;
  if (!aligned_to(gate_up, 16) || !aligned_to(d_out, 16) || !aligned_to(d_gate_up, 16) ||
      !aligned_to(row_weights, 4) || !aligned_to(num_rows, 4) || !aligned_to(d_row_weights, 4))
    return MP_ERR_INVALID_ARG;
  return status_of(launch_swiglu_backward_bf16(rows, I, gate_up, row_weights, d_out, num_rows,
                                               d_gate_up, d_row_weights,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
