// mp_pair16.cuh -- what the bf16 products of the experts share: tensor maps of
// bf16 arrays, loads and arrivals within a pair of blocks, 4-bit codes as bf16, and
// where a tile of the ragged rows lies.
#pragma once

#include <algorithm>
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
// Host: tensor maps over [depth][rows][cols], with the 128-byte swizzle.
// ---------------------------------------------------------------------------
inline bool make_map_3d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int elem,
                        uint64_t cols, uint64_t rows, uint64_t depth, uint32_t box_cols,
                        uint32_t box_rows,
                        CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cols, rows, depth};
  const cuuint64_t strides[2] = {cols * uint64_t(elem), cols * rows * uint64_t(elem)};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
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
// (dst: a shared address.  What a loading thread does per stage is kept short: its
// instructions wait their turn among the other warps'.)
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
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
// A box from shared memory to the array, in the current bulk async-group; what
// lies outside the array is not written.  The lines leave L2 first: nothing here
// reads them again (weights' gradient of 4,095 rows, 64 experts x 4096 x 2048, fp32:
// 362 us, 379 without the hint).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z,
                                             const void* src) {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint "
      "[%0, {%1, %2, %3}], [%4], %5;" ::"l"(map),
      "r"(x), "r"(y), "r"(z), "r"(smem_addr(src)), "l"(policy)
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight e2m1 codes as bf16 pairs in order, 2^-126 times their value: sign to bit
// 15, the two exponent bits and the mantissa bit to bits 8 to 6 (both shifts are
// one product).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // code 2i to bits 0-3, code 2i+1 to bits 16-19 (selector 8: a byte's sign bit, here 0)
    uint32_t two;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(two) : "r"(even), "r"(odd), "r"(0x8480 + i * 0x1111));
    o[i] = (two * 0x1040u) & 0x81c081c0u;
  }
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

// ---------------------------------------------------------------------------
// Tiles of the products on ragged rows: 256 output channels (the MMA's M side,
// 128 per block) by up to 256 rows (its N side), 64 reduction steps per stage.
// ---------------------------------------------------------------------------
constexpr int kBC = 128;                  // channels per block: 256 per pair
constexpr int kBR = 256;                  // most rows per tile
constexpr int kUnit = 32;                 // rows that a tile is a multiple of
constexpr int kBK = 64;                   // reduction steps per stage: 128 bytes
constexpr int kStageC = kBC * kBK * 2;    // bytes of a stage: channels, then rows
constexpr int kStageR = kBR / 2 * kBK * 2;
constexpr int kStage = kStageC + kStageR;
constexpr int kMaxParts = 4;              // pairs that share a tile's reduction: one cluster
constexpr int kBandTiles = 8;             // row tiles per band of the tile order
constexpr int kTurned = 16 * 32 * 2;      // bytes of 16 rows x 32 channels

struct RaggedArgs {
  int E, rows, out_cols, red;             // out_cols, red: N and K, or K and N
  int stages;
  int out32;                              // rows of out are 32-byte aligned
  int patience;                           // of the waits for whole tiles
  const int32_t* expert_offsets;          // [E + 1], or NULL: one expert with all rows
  uint16_t* out;                          // bf16 [rows][out_cols]
  int32_t* dev_err;
};

// Adds up a value of every thread; all threads get the sum.
template <int THREADS>
__device__ __forceinline__ int block_sum(int v, int* scan) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) scan[threadIdx.x >> 5] = v;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) sum += scan[w];
  __syncthreads();
  return sum;
}

// Exclusive prefix over experts of their number of tiles of `most` rows, into
// pre[0 .. E].  Offsets that are negative or decrease leave no tiles at all
// (overlapping experts could make more of them than the launcher's check allows
// for).
template <int THREADS>
__device__ void tile_prefix(const RaggedArgs& p, int most, int* pre, int* scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.E + THREADS - 1) / THREADS;
  const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
  int sum = 0, bad = 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    rows_of(p.expert_offsets, p.rows, e, lo, hi);
    pre[e] = (hi - lo + most - 1) / most;
    sum += pre[e];
    bad |= offset_errors(p.expert_offsets, p.rows, e);
  }
  if (bad && blockIdx.x == 0) raise_error(p.dev_err, bad);
  bad = __syncthreads_or(bad & MP_ERR_INVALID_ARG);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += scan[w];
  int at = base + incl - sum;
  for (int e = e0; e < e1; ++e) {
    const int n = pre[e];
    pre[e] = at;
    at += n;
  }
  if (tid == THREADS - 1) pre[p.E] = bad ? 0 : base + incl;
  __syncthreads();
}

// The most rows of a tile: `most`, or 32 or 64 fewer where their tiles fill the
// pairs' turns better.  A turn takes about as long as its tiles' units of 32 rows on
// average and 1.25 more (measured with bf16 weights, 4096 x 7168: 38.4 us with 256
// rows, 34.3 with 224, 32.7 with 211), so a smaller tile has to save whole turns.
// (32 experts of about 1,024 rows, 2,048 channels from 7168: 17 turns of 6.5 units
// take 535 us, 16 of 7.2 units 550.)  `least_turn`: what one takes whatever its rows.
template <int THREADS>
__device__ int tile_rows(const RaggedArgs& p, int most, float least_turn, int ncol, int pairs,
                         int* scan) {
  const int full = most / kUnit;
  int units = 0, tiles[3] = {0, 0, 0};
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    int lo, hi;
    rows_of(p.expert_offsets, p.rows, e, lo, hi);
    const int u = (hi - lo + kUnit - 1) / kUnit;
    units += u;
#pragma unroll
    for (int i = 0; i < 3; ++i) tiles[i] += (u + full - i - 1) / (full - i);
  }
  units = block_sum<THREADS>(units, scan);
  int best = full;
  float least = INFINITY;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float t = float(block_sum<THREADS>(tiles[i], scan));
    if (i > 0 && t * ncol >= 0x1p30f) break;  // (their number stays an int)
    const float turn = fmaxf(units / fmaxf(t, 1.0f) + 1.25f, least_turn);
    const float cost = ceilf(t * ncol / pairs) * turn;
    if (cost < least) {
      least = cost;
      best = full - i;
    }
  }
  return best * kUnit;
}

struct Tile {
  int e, row0, nrows, n, col0;  // n: nrows rounded up to whole units
};

// The expert that tile t belongs to: pre[e] * ncol <= t < pre[e + 1] * ncol.
__device__ __forceinline__ int expert_of(const int* pre, int E, int ncol, int t) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * ncol <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Tile t in the order: experts ascending; within an expert, bands of kBandTiles
// row tiles, in a band channels slowest, so that the tiles running at one time
// share few weight channels and a band's rows.
__device__ __forceinline__ Tile tile_at(const RaggedArgs& p, const int* pre, int ncol, int t) {
  const int lo = expert_of(pre, p.E, ncol, t);
  const int mt = pre[lo + 1] - pre[lo];
  const int local = t - pre[lo] * ncol;
  const int band = local / (kBandTiles * ncol);
  const int rem = local - band * kBandTiles * ncol;
  const int mb = min(kBandTiles, mt - band * kBandTiles);
  const int nt = rem / mb, m = band * kBandTiles + rem - nt * mb;
  int r0, r1;
  rows_of(p.expert_offsets, p.rows, lo, r0, r1);
  // the expert's rows in whole units, spread evenly over its tiles: the first `rest` of
  // them have one unit more.  (Every role finds its tiles by itself, in the time that
  // the products of a short reduction wait for: no long divisions.)
  const int units = (r1 - r0 + kUnit - 1) / kUnit;
  const int each = units / mt, rest = units - each * mt;
  Tile tile;
  tile.e = lo;
  tile.row0 = r0 + (m * each + min(m, rest)) * kUnit;
  tile.n = (each + (m < rest ? 1 : 0)) * kUnit;
  tile.nrows = min(tile.n, r1 - tile.row0);
  tile.col0 = nt * 2 * kBC;
  return tile;
}

// Every warp's end: nothing of the cluster is in use after it.
__device__ __forceinline__ void cluster_end() {
  __syncwarp();
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
}

// A tile's rows, half of them per block: a multiple of 16 (up to 128), loaded as one
// or two boxes of 16, 32, 64 or 128 rows (112 as 128: the stage has the room).
struct RowMaps {
  CUtensorMap m[4];
};
inline bool make_row_maps(RowMaps* r, const void* a, int red, int rows) {
  for (int i = 0; i < 4; ++i)
    if (!make_map_bf16(&r->m[i], a, uint64_t(red), uint64_t(rows), kBK, 16u << i)) return false;
  return true;
}
struct RowBoxes {
  const CUtensorMap *one, *two;  // two: NULL if one box is all
  int row, row2;                 // their first rows
  uint32_t at2, bytes;           // of the second box in the stage; of both
  __device__ __forceinline__ RowBoxes(const RowMaps& maps, int row0, int n, int rank) {
    int half = n / 2;
    row = row2 = row0 + rank * half;
    if (half == 112) half = 128;
    const int big = half >= 128 ? 3 : half >= 64 ? 2 : half >= 32 ? 1 : 0;
    const int rest = half - (16 << big);  // 0, 16 or 32
    one = &maps.m[big];
    two = rest == 0 ? nullptr : &maps.m[rest == 32 ? 1 : 0];
    row2 += 16 << big;
    at2 = uint32_t(16 << big) * kBK * 2;
    bytes = uint32_t(half) * kBK * 2;
  }
  __device__ __forceinline__ void load(uint32_t dst, int k, uint32_t bar) const {
    tma_load_2d_pair(dst, one, k, row, bar);
    if (two != nullptr) tma_load_2d_pair(dst + at2, two, k, row2, bar);
  }
};

// The products of one stage: four K = 16 steps.
template <bool C_MN>
__device__ __forceinline__ void stage_products(const unsigned char* stage, uint32_t acc,
                                               uint32_t idesc, bool first) {
  const uint32_t sc = smem_addr(stage);
  const uint64_t dc = smem_desc_sw128(sc, C_MN ? kStageC / 2 : 16, 1024);
  const uint64_t dr = smem_desc_sw128(sc + kStageC, 16, 1024);
#pragma unroll
  for (int k = 0; k < kBK / 16; ++k)
    mma_f16_pair(acc, dc + (C_MN ? ((k * 16 * 128) >> 4) : ((k * 32) >> 4)),
                 dr + ((k * 32) >> 4), idesc, !first || k > 0);
}

// A finished accumulator, this warp's 32 channels from `ch` on and every SHARE-th 32
// rows from the `mine`-th on, to bf16 rows.  `src`: its TMEM lanes and first column;
// `turned`: 2 * kTurned bytes of its own, in which 16 rows x 32 channels at a time are
// turned around.
template <int SHARE>
__device__ __forceinline__ void write_tile(const RaggedArgs& p, const Tile& tl, int ch,
                                           uint32_t src, int mine, unsigned char* turned) {
  if (mine * 32 >= tl.n) return;
  const int lane = threadIdx.x & 31;
  const int r = lane >> 1, h = (lane & 1) * 16;  // the row and channels that it stores
  const int left = p.out_cols - (ch + h);        // a multiple of 8 (or <= 0)
  uint16_t* dst = p.out + int64_t(tl.row0 + r) * p.out_cols + ch + h;
  float2 v[2][8];
  tmem_ld_x16(src + mine * 32, v[0]);
  tmem_wait_ld(v[0]);
  for (int c0 = mine * 32; c0 < tl.n; c0 += SHARE * 32) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {  // 16 rows; the next 16 on their way from TMEM
      const int c = c0 + b * 16, next = b == 0 ? c + 16 : c0 + SHARE * 32;
      if (next < tl.n) tmem_ld_x16(src + next, v[b ^ 1]);
      uint16_t* tw = reinterpret_cast<uint16_t*>(turned + b * kTurned) + lane;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t two = pack_bf16x2_rn(v[b][j].x, v[b][j].y);
        tw[(2 * j) * 32] = uint16_t(two);
        tw[(2 * j + 1) * 32] = uint16_t(two >> 16);
      }
      __syncwarp();
      if (c + r < tl.nrows) {
        const uint4* tr = reinterpret_cast<const uint4*>(turned + b * kTurned + r * 64 + h * 2);
        const uint4 x = tr[0], y = tr[1];
        if (p.out32 && left >= 16) {
          const Words<8> o = {{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
          st_stream_w<8>(reinterpret_cast<Words<8>*>(dst + int64_t(c) * p.out_cols), o);
        } else {
          uint4* d = reinterpret_cast<uint4*>(dst + int64_t(c) * p.out_cols);
          if (left >= 8) d[0] = x;
          if (left >= 16) d[1] = y;
        }
      }
      if (next < tl.n) tmem_wait_ld(v[b ^ 1]);
    }
  }
}

// fp32 sums of a part of the reduction into shared memory, [row][channel]; rows shared
// among warps as above.
template <int SHARE>
__device__ __forceinline__ void store_part(const Tile& tl, int q, uint32_t src, int mine,
                                           void* stages) {
  float* to = reinterpret_cast<float*>(stages) + q * 32 + (threadIdx.x & 31);
  for (int c = mine * 16; c < tl.n; c += SHARE * 16) {
    float2 v[8];
    tmem_ld_x16(src + c, v);
    tmem_wait_ld(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      to[(c + 2 * j) * kBC] = v[j].x;
      to[(c + 2 * j + 1) * kBC] = v[j].y;
    }
  }
}

// The parts' sums in ascending order, rounded once: four channels of a row per
// thread and turn, the rows spread over the blocks that hold the same channels.
template <int THREADS>
__device__ __forceinline__ void join_parts(const RaggedArgs& p, const Tile& tl, int rank, int part,
                                           int parts, const void* stages) {
  const int ch0 = tl.col0 + rank * kBC;
  for (int i = part * THREADS + int(threadIdx.x); i < tl.nrows * (kBC / 4);
       i += parts * THREADS) {
    const int row = i / (kBC / 4), c4 = i % (kBC / 4) * 4;
    const float* at = reinterpret_cast<const float*>(stages) + row * kBC + c4;
    float4 v[kMaxParts];  // all on their way before the first is needed
#pragma unroll
    for (int z = 0; z < kMaxParts; ++z)
      v[z] = z < parts ? ld_cluster_f4(map_to_rank(at, uint32_t(2 * z + rank)))
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 sum = v[0];
#pragma unroll
    for (int z = 1; z < kMaxParts; ++z) {
      sum.x += v[z].x;
      sum.y += v[z].y;
      sum.z += v[z].z;
      sum.w += v[z].w;
    }
    if (ch0 + c4 < p.out_cols) {
      uint2 o;
      o.x = pack_bf16x2_rn(sum.x, sum.y);
      o.y = pack_bf16x2_rn(sum.z, sum.w);
      *reinterpret_cast<uint2*>(p.out + int64_t(tl.row0 + row) * p.out_cols + ch0 + c4) = o;
    }
  }
}

// How many clusters of `size` blocks of a kernel, with as much shared memory as there
// is, run at once; asked once per kind of kernel, device and thread.  (On 152 SMs 76 of two
// blocks, 36 of four, 23 of six, 15 of eight.)
template <typename Kernel>
inline int clusters_at_once(Kernel kernel, int threads, int size) {
  struct Known { int dev[64][9] = {}; };
  static thread_local Known known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || size > 8) return 0;
  if (dev >= 0 && dev < 64 && known.dev[dev][size] > 0) return known.dev[dev][size] - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(size * 16));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = kMaxBlockSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(size);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();  // (not this call's to report)
    n = 0;
  }
  if (dev >= 0 && dev < 64) known.dev[dev][size] = n + 1;
  return n;
}

// The most parts, up to `most`, that a reduction can be shared in by clusters of
// `per` blocks a part so that all of `tiles` clusters run at once and each part has
// `least` of the reduction's stages.
template <typename Kernel>
inline int parts_for(Kernel kernel, int threads, int64_t tiles, int per, int most, int stages,
                     int least) {
  for (int parts = most; parts > 1; --parts)
    if (stages >= parts * least && tiles * per * parts <= sm_count() &&
        tiles <= clusters_at_once(kernel, threads, per * parts))
      return parts;
  return 1;
}
// Tiles of `most` rows, at most: every expert's first row starts one.
inline int64_t most_row_tiles(int E, int rows, int most) {
  const int used = std::min(E, rows);
  return used + (int64_t(rows) - used) / most;
}

}  // namespace mp
