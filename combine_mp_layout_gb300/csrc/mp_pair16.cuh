// mp_pair16.cuh -- what the bf16 products of the experts share: tensor maps of
// bf16 arrays, loads and arrivals within a pair of blocks, and where a tile of
// the ragged rows lies.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_internal.h"
#include "mp_tcgen05.cuh"

namespace mp {

constexpr int kMaxBlockSmem = 232448;  // bytes of shared memory a block may have

// ---------------------------------------------------------------------------
// Host: tensor maps with the 128-byte swizzle over [depth][rows][cols].
// ---------------------------------------------------------------------------
inline bool make_map_3d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int elem,
                        uint64_t cols, uint64_t rows, uint64_t depth, uint32_t box_cols,
                        uint32_t box_rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cols, rows, depth};
  const cuuint64_t strides[2] = {cols * uint64_t(elem), cols * rows * uint64_t(elem)};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool make_map_bf16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                          uint32_t box_cols, uint32_t box_rows) {
  return encode_map_2d(map, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, cols, rows, box_cols,
                       box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Raises a kernel's shared-memory limit to the most that a block may have, once
// per device and thread.  The limit belongs to the function on the device, and so
// to all threads: always the same value, so that none lowers another's.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kernel, bool (&configured)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && configured[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBlockSmem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) configured[dev] = true;
  return e;
}

// ---------------------------------------------------------------------------
// Device: a pair of blocks is an even rank of a cluster and the one after it.
// The even one issues the pair's MMAs, so the barriers of operands that have
// arrived are its.
// ---------------------------------------------------------------------------
__host__ __device__ constexpr uint32_t mma_idesc_bf16(int m, int n, bool a_mn, bool b_mn) {
  return mma_idesc(m, n, 1u, 1u, a_mn, b_mn);  // bf16 x bf16 (kind::f16)
}

// TMA loads into this block's shared memory whose bytes are counted on a barrier
// of this block or of the other one of its pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int x, int y,
                                                 int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
// An arrival (with bytes to come) on a barrier at a shared::cluster address.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// The barrier of both blocks of the pair gets one arrival when every MMA issued
// so far by this thread is done; `even` is the cluster rank of the first.
__device__ __forceinline__ void commit_to_pair(uint64_t* bar, int even) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(uint16_t(3u << even))
      : "memory");
}

// A position in a ring of n slots: the slot and how often the ring went round.
struct RingAt {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      ++round;
    }
  }
};

// First and one-past-last row of expert e, forced into [0, rows].
__device__ __forceinline__ void rows_of(const int32_t* offsets, int rows, int e, int& lo,
                                        int& hi) {
  if (offsets == nullptr) {
    lo = 0;
    hi = rows;
    return;
  }
  lo = min(max(__ldg(offsets + e), 0), rows);
  hi = max(lo, min(__ldg(offsets + e + 1), rows));
}

// What is wrong with offsets e and e + 1.
__device__ __forceinline__ int offset_errors(const int32_t* offsets, int rows, int e) {
  if (offsets == nullptr) return 0;
  const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
  return (lo < 0 || hi < lo ? MP_ERR_INVALID_ARG : 0) | (hi > rows ? MP_ERR_CAPACITY : 0);
}

}  // namespace mp
