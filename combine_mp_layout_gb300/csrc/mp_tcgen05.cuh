// mp_tcgen05.cuh -- inline PTX for the tensor-core kernels: tensor maps and
// TMA tile loads, shared-memory matrix descriptors, tcgen05 MMA / TMEM.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_common.cuh"

namespace mp {

// ---------------------------------------------------------------------------
// Host: a 2-D tensor map over a dense row-major array (inner extent `cols`
// elements of `elem` bytes), loaded in boxes of box_cols x box_rows.  Elements
// outside the array read as zero.
// ---------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

inline bool encode_map_2d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int elem,
                          uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows,
                          CUtensorMapSwizzle swizzle) {
  const EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * uint64_t(elem)};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t step[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Bytes (e4m3 codes), with the 128-byte swizzle.
inline bool make_map_bytes(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                           uint32_t box_cols, uint32_t box_rows) {
  return encode_map_2d(map, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, cols, rows, box_cols, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}
// fp32 values (scales), as they are.
inline bool make_map_f32(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                         uint32_t box_cols, uint32_t box_rows) {
  return encode_map_2d(map, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, cols, rows, box_cols,
                       box_rows, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// ---------------------------------------------------------------------------
// Device
// ---------------------------------------------------------------------------
// True for one lane of the (whole, converged) warp.  tcgen05 and TMA
// instructions stand in branches on this and on warp_index(), which tell the
// compiler that one thread of a uniform warp issues them: in a branch on a lane
// number each MMA cost about 120 clocks to issue, here less than 64 (128 x 64 x
// 128 e4m3 products back to back: 480 clocks per four MMAs against 264).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(p)::"memory");
  return p != 0;
}
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(kFull, int(threadIdx.x >> 5), 0);
}

// A TMA load of one box; its bytes are counted on the mbarrier.
__device__ __forceinline__ void tma_load_2d(void* smem_dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait on an mbarrier phase by one thread (2^26 attempts of some 20
// clocks, about a second); false, with the failure noted in the block's flag,
// when it gives up.  Every role of a block that waits for another one gives up
// by itself.  The loop is three instructions: whatever else it does is added
// to the time from one role to the next, which the products wait for.
// `patience`, here and below: how many times as long, where what is waited for
// takes longer the larger the problem is.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity,
                                             volatile int* failed, int patience = 1) {
  uint32_t ok;
  do {
    asm volatile(
        "{\n .reg .pred p;\n .reg .u32 n;\n mov.u32 n, 0;\n"
        "$MP_TRY_%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " @p bra $MP_END_%=;\n add.u32 n, n, 1;\n setp.lt.u32 p, n, 67108864;\n"
        " @p bra $MP_TRY_%=;\n setp.ne.u32 p, n, n;\n"
        "$MP_END_%=:\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
  } while (!ok && --patience > 0);
  if (!ok) *failed = 1;
  return ok != 0;
}
// The same for roles that are ahead of the others and have time: suspended
// between attempts (up to 1 us each), so that they take no issue slots and no
// turns at the barrier unit from those that are waited for.
__device__ __forceinline__ bool bounded_wait_idle(uint64_t* bar, uint32_t parity,
                                                  volatile int* failed, int patience = 1) {
  do {
    for (uint32_t n = 0; n < kSpinLimit; ++n)
      if (mbar_try_wait(bar, parity)) return true;
  } while (--patience > 0);
  *failed = 1;
  return false;
}
__device__ __forceinline__ bool bounded_wait_idle_warp(uint64_t* bar, uint32_t parity,
                                                       volatile int* failed, int patience = 1) {
  return __all_sync(kFull, bounded_wait_idle(bar, parity, failed, patience));
}
// The first form for a whole warp.  The vote in the loop makes the answer, and
// so the loop itself, the same for all lanes in the compiler's eyes too: the
// branches after it need no reconvergence.
__device__ __forceinline__ bool bounded_wait_warp(uint64_t* bar, uint32_t parity,
                                                  volatile int* failed, int patience = 1) {
  do {
    for (uint32_t n = 0; n < (1u << 25); ++n)
      if (__all_sync(kFull, try_wait(bar, parity))) return true;
  } while (--patience > 0);
  *failed = 1;
  return false;
}

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One whole warp (of each block of the pair, for PAIR) allocates and later frees
// TMEM columns: a power of two >= 32.  A kernel uses one group size throughout.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_dst, uint32_t cols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(smem_dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(smem_dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem, uint32_t cols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

// ---------------------------------------------------------------------------
// Clusters.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
// Every thread of every block of the cluster, each warp together.
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared::cluster address of a shared variable in the block of that rank.
__device__ __forceinline__ uint32_t map_to_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
// An arrival on the mbarrier at this place in the first block of the pair.  It
// orders nothing in global memory: what it publishes is shared memory that a
// proxy fence has made visible to the tensor core, or TMEM that has been read.
// (With a release at cluster scope every arrival waits for a memory fence, and
// for the loads in flight.)
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar, int rank) {
  if (rank == 0)
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, 0))
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: 8 rows of 128 bytes form
// an atom of 1 KB.  K-major operand: sbo = bytes between groups of 8 rows (lbo
// unused).  MN-major operand: sbo = bytes between groups of 8 reduction steps,
// lbo = bytes between 128-byte chunks of the M or N extent.
__host__ __device__ constexpr uint64_t smem_desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr & 0x3ffffu) >> 4) | (uint64_t(lbo >> 4) << 16) |
         (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Instruction descriptor: fp32 accumulator, M x N tile, operand majors.
__host__ __device__ constexpr uint32_t mma_idesc(int m, int n, uint32_t a_fmt, uint32_t b_fmt,
                                                 bool a_mn, bool b_mn) {
  return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t mma_idesc_f8(int m, int n, bool a_mn, bool b_mn) {
  return mma_idesc(m, n, 0u, 0u, a_mn, b_mn);  // e4m3 x e4m3
}
__host__ __device__ constexpr uint32_t mma_idesc_f16(int m, int n, bool a_mn, bool b_mn) {
  return mma_idesc(m, n, 0u, 0u, a_mn, b_mn);  // f16 x f16 (kind::f16)
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// Pair only: M = 256 rows in two blocks.
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// The mbarrier (of both blocks, for PAIR) gets one arrival when every MMA
// issued so far by this thread is done.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}

// 16 columns of this warp's 32 TMEM lanes: v[j] = columns 2j, 2j + 1 of lane.
__device__ __forceinline__ void tmem_ld_x16(uint32_t src, float2 (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y),
        "=f"(v[3].x), "=f"(v[3].y), "=f"(v[4].x), "=f"(v[4].y), "=f"(v[5].x), "=f"(v[5].y),
        "=f"(v[6].x), "=f"(v[6].y), "=f"(v[7].x), "=f"(v[7].y)
      : "r"(src));
}
// Waits for this thread's TMEM loads.  The loaded values pass through, so that
// no use of them can be moved ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(float2 (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0].x), "+f"(v[0].y), "+f"(v[1].x), "+f"(v[1].y), "+f"(v[2].x),
                 "+f"(v[2].y), "+f"(v[3].x), "+f"(v[3].y), "+f"(v[4].x), "+f"(v[4].y),
                 "+f"(v[5].x), "+f"(v[5].y), "+f"(v[6].x), "+f"(v[6].y), "+f"(v[7].x),
                 "+f"(v[7].y)::"memory");
}

}  // namespace mp
