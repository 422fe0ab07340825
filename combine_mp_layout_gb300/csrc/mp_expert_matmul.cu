// mp_expert_matmul.cu -- products of the experts on e4m3 rows with one fp32
// scale per block of 128, grouped by expert (sm_103a: TMA, tcgen05, TMEM).
//
// Forward   y[r][n]  = sum_kb sa[r][kb] * sw[e][n/128][kb] * P(r, n, kb),
//           P(r, n, kb) = sum over the 128 channels k of block kb of a[r][k] * w[e][n][k]
// Gradient of the rows (TB = true: the same weights, read along the other axis)
//           dx[r][k] = sum_nb sd[r][nb] * sw[e][nb][k/128] * sum_{n in nb} dy[r][n] * w[e][n][k]
// for every row r of expert e (rows expert_offsets[e] .. expert_offsets[e+1]).
//
// The scales change every 128 channels of the reduction, so the tensor core
// sums one block (four K = 32 steps of kind::f8f6f4, exact products, fp32
// accumulation in TMEM) and the block sums are added up in fp32 registers with
// their scale: one packed FMA per two outputs and block.  A thread owns one
// output row (one TMEM lane), so the product of the two scales is one register.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_internal.h"
#include "mp_tcgen05.cuh"

namespace mp {

namespace {

constexpr int kBM = 128;             // rows per tile: the M of one MMA
constexpr int kBK = 128;             // reduction channels per stage: one scale block
constexpr int kABox = 32;            // rows per TMA box of the A tile: a short last tile of an
                                     // expert loads only the boxes that hold rows
constexpr int kEpiWarps = 8;         // two warpgroups, each BN / 2 columns of all 128 rows
constexpr int kMMThreads = 128 + kEpiWarps * 32;
constexpr int kBand = 16;            // m-tiles per band of the tile order

struct MMArgs {
  int E, rows, out_cols, red_blocks;  // out_cols: N (forward) or K (dgrad)
  int w_rows;                         // weight rows per expert (N)
  const float* a_scales;              // [rows][red_blocks]
  const float* w_scales;              // [E][ceil(N/128)][K/128]
  int64_t ws_expert;                  // strides of w_scales, in floats
  int ws_out, ws_red;
  const int32_t* expert_offsets;      // [E + 1], or NULL: one expert with all rows
  uint16_t* out;                      // bf16 [rows][out_cols]
  int32_t* dev_err;
};

// Where a tile lies.
struct Tile {
  int e, row0, nrows, col0;
};

template <int BN>
struct MMShape {
  static constexpr int kStageA = kBM * kBK;
  static constexpr int kStageB = BN * kBK;
  static constexpr int kStage = kStageA + kStageB;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kTmemCols = 2 * BN;
};

// Shared memory after the 1024-byte aligned stages.
template <int BN>
struct MMTail {
  uint64_t full[MMShape<BN>::kStages], empty[MMShape<BN>::kStages];
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int failed;
  int scan[kMMThreads / 32];
};

template <int BN>
size_t mm_smem_bytes(int E) {
  return 1024 + size_t(MMShape<BN>::kStages) * MMShape<BN>::kStage + sizeof(MMTail<BN>) +
         size_t(E + 1) * 4;
}

// First and one-past-last row of expert e, forced into [0, rows].
__device__ __forceinline__ void expert_range(const MMArgs& p, int e, int& lo, int& hi) {
  if (p.expert_offsets == nullptr) {
    lo = 0;
    hi = p.rows;
    return;
  }
  lo = min(max(__ldg(p.expert_offsets + e), 0), p.rows);
  hi = max(lo, min(__ldg(p.expert_offsets + e + 1), p.rows));
}

// Exclusive prefix over experts of their number of m-tiles, into pre[0 .. E].
// Offsets that are negative or decrease leave no tiles at all (overlapping
// experts could make more of them than the launcher's check allows for).
__device__ void tile_prefix(const MMArgs& p, int* pre, int* scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.E + kMMThreads - 1) / kMMThreads;
  const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
  int sum = 0, bad = 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    expert_range(p, e, lo, hi);
    sum += (hi - lo + kBM - 1) / kBM;
    if (p.expert_offsets != nullptr) {
      const int a = __ldg(p.expert_offsets + e), b = __ldg(p.expert_offsets + e + 1);
      if (a < 0 || b < a) bad |= MP_ERR_INVALID_ARG;
      if (b > p.rows) bad |= MP_ERR_CAPACITY;
    }
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
    int lo, hi;
    expert_range(p, e, lo, hi);
    pre[e] = at;
    at += (hi - lo + kBM - 1) / kBM;
  }
  if (tid == kMMThreads - 1) pre[p.E] = bad ? 0 : base + incl;
  __syncthreads();
}

// Tile t in the order: experts ascending; within an expert, bands of kBand
// m-tiles, in a band columns slowest, so that the tiles running at one time
// share few weight columns and a band's rows.
template <int BN>
__device__ __forceinline__ Tile tile_at(const MMArgs& p, const int* pre, int ncol, int t) {
  int lo = 0, hi = p.E;  // pre[lo] * ncol <= t < pre[hi] * ncol
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * ncol <= t) lo = mid; else hi = mid;
  }
  const int mt = pre[lo + 1] - pre[lo];
  const int local = t - pre[lo] * ncol;
  const int band = local / (kBand * ncol);
  const int rem = local - band * kBand * ncol;
  const int mb = min(kBand, mt - band * kBand);
  const int nt = rem / mb, m = band * kBand + rem % mb;
  int r0, r1;
  expert_range(p, lo, r0, r1);
  Tile tile;
  tile.e = lo;
  tile.row0 = r0 + m * kBM;
  tile.nrows = min(kBM, r1 - tile.row0);
  tile.col0 = nt * BN;
  return tile;
}

template <int BN, bool TB>
__global__ void __launch_bounds__(kMMThreads, 1)
mp_k_expert_matmul(const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_w, const MMArgs p) {
  using S = MMShape<BN>;
  constexpr int kHalf = BN / 2;  // columns per epilogue warpgroup
  extern __shared__ unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  MMTail<BN>* tail = reinterpret_cast<MMTail<BN>*>(stages + size_t(S::kStages) * S::kStage);
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&tail->full[i], 1);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->tfull[i], 1);
      mbar_init(&tail->tempty[i], kEpiWarps);
    }
    tail->failed = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(&tail->tmem, S::kTmemCols);
  tile_prefix(p, pre, tail->scan);  // (its barriers also publish the mbarriers and the TMEM base)
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int ncol = (p.out_cols + BN - 1) / BN;
  const int tiles = pre[p.E] * ncol;  // below 2^31: the launcher checks
  volatile int* failed = &tail->failed;

  // The accumulators of BN = 256 need more registers than a twelfth of the
  // file: the four warps that only issue give theirs up (128 * 72 + 256 * 216
  // = the launch's 384 * 168).
  if (warp < 4) {
  if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // ---- loads: one lane keeps the ring of stages full
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const Tile tl = tile_at<BN>(p, pre, ncol, t);
        const int boxes = (tl.nrows + kABox - 1) / kABox;
        const uint32_t bytes = uint32_t(boxes) * kABox * kBK + S::kStageB;
        for (int kb = 0; kb < p.red_blocks; ++kb, ++it) {
          const uint32_t st = it % S::kStages, use = it / S::kStages;
          if (use > 0 && !bounded_wait(&tail->empty[st], (use - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          unsigned char* sa = stages + size_t(st) * S::kStage;
          unsigned char* sb = sa + S::kStageA;
          mbar_arrive_expect_tx(&tail->full[st], bytes);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sa + b * kABox * kBK, &map_a, kb * kBK, tl.row0 + b * kABox,
                        &tail->full[st]);
          if constexpr (TB) {
#pragma unroll
            for (int c = 0; c < BN / 128; ++c)
              tma_load_2d(sb + c * 128 * kBK, &map_w, tl.col0 + c * 128,
                          tl.e * p.w_rows + kb * kBK, &tail->full[st]);
          } else {
            tma_load_2d(sb, &map_w, kb * kBK, tl.e * p.w_rows + tl.col0, &tail->full[st]);
          }
        }
      }
      // every load that was issued lands before the block may end
      for (uint32_t i = it > uint32_t(S::kStages) ? it - S::kStages : 0; i < it; ++i) {
        uint32_t n = 0;
        while (!mbar_try_wait(&tail->full[i % S::kStages], (i / S::kStages) & 1u) &&
               ++n < kSpinLimit) {
        }
      }
    }
  } else if (warp == 1) {
    // ---- products: one lane issues the MMAs of a stage into one of two accumulators
    if (elect_one()) {
      constexpr uint32_t idesc = mma_idesc_f8(kBM, BN, /*a_mn=*/false, /*b_mn=*/TB);
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int kb = 0; kb < p.red_blocks; ++kb, ++it) {
          const uint32_t st = it % S::kStages, buf = it & 1u;
          if (!bounded_wait(&tail->full[st], (it / S::kStages) & 1u, failed) ||
              (it >= 2 && !bounded_wait(&tail->tempty[buf], ((it >> 1) - 1) & 1u, failed))) {
            ok = false;
            break;
          }
          tcgen05_fence_after();
          const uint32_t sa = smem_addr(stages + size_t(st) * S::kStage);
          const uint32_t sb = sa + S::kStageA;
          const uint64_t da = smem_desc_sw128(sa, 16, 1024);
          const uint64_t db = smem_desc_sw128(sb, TB ? 128 * kBK : 16, 1024);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_f8(tmem + buf * BN, da + ((k * 32) >> 4),
                   db + (TB ? ((k * 32 * 128) >> 4) : ((k * 32) >> 4)), idesc, k > 0);
          mma_commit(&tail->empty[st]);
          mma_commit(&tail->tfull[buf]);
        }
      }
      if (it >= 1) {  // the last products finish before TMEM is given back
        const uint32_t last = it - 1;
        uint32_t n = 0;
        while (!mbar_try_wait(&tail->tfull[last & 1u], (last >> 1) & 1u) && ++n < kSpinLimit) {
        }
      }
    }
  }
  } else {
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- block sums from TMEM into fp32 registers, then bf16 rows
    const int ew = warp - 4;
    const int half = ew >> 2;                // which half of the columns
    const int lrow = (ew & 3) * 32 + lane;   // row of the tile = TMEM lane
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile tl = tile_at<BN>(p, pre, ncol, t);
      const bool warp_has_rows = (ew & 3) * 32 < tl.nrows;
      const bool has_row = lrow < tl.nrows;
      const int64_t row = tl.row0 + (has_row ? lrow : 0);
      const float* sa = p.a_scales + row * p.red_blocks;
      const int cb = min((tl.col0 + half * kHalf) >> 7, (p.out_cols - 1) >> 7);
      const float* sw = p.w_scales + tl.e * p.ws_expert + int64_t(cb) * p.ws_out;
      float2 acc[kHalf / 2];
#pragma unroll
      for (int j = 0; j < kHalf / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      float s_next = __ldg(sa) * __ldg(sw);
      for (int kb = 0; kb < p.red_blocks; ++kb, ++it) {
        const float s = s_next;
        if (kb + 1 < p.red_blocks) s_next = __ldg(sa + kb + 1) * __ldg(sw + int64_t(kb + 1) * p.ws_red);
        const uint32_t buf = it & 1u;
        if (!bounded_wait_warp(&tail->tfull[buf], (it >> 1) & 1u, failed)) {
          ok = false;
          break;
        }
        tcgen05_fence_after();
        if (warp_has_rows) {
          const uint32_t src = tmem + buf * BN + half * kHalf + (uint32_t(ew & 3) << 21);
          const float2 s2 = make_float2(s, s);
#pragma unroll
          for (int c = 0; c < kHalf / 32; ++c) {
            float2 v[16];
            tmem_ld_x32(src + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c * 16 + j] = fma2(v[j], s2, acc[c * 16 + j]);
          }
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->tempty[buf]);
      }
      if (ok && has_row) {
        uint16_t* dst = p.out + row * p.out_cols + tl.col0 + half * kHalf;
        const int left = p.out_cols - (tl.col0 + half * kHalf);  // a multiple of 16 (or <= 0)
#pragma unroll
        for (int c = 0; c < kHalf / 8; ++c) {
          if (c * 8 < left) {
            int4 o;
            o.x = int(pack_bf16x2_rn(acc[c * 4].x, acc[c * 4].y));
            o.y = int(pack_bf16x2_rn(acc[c * 4 + 1].x, acc[c * 4 + 1].y));
            o.z = int(pack_bf16x2_rn(acc[c * 4 + 2].x, acc[c * 4 + 2].y));
            o.w = int(pack_bf16x2_rn(acc[c * 4 + 3].x, acc[c * 4 + 3].y));
            *reinterpret_cast<int4*>(dst + c * 8) = o;
          }
        }
      }
    }
  }

  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::kTmemCols);
  if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
}

template <int BN, bool TB>
cudaError_t launch_mm(const MMArgs& p, const CUtensorMap& ma, const CUtensorMap& mw,
                      cudaStream_t st) {
  static thread_local int configured_smem[64] = {0};
  const int smem = int(mm_smem_bytes<BN>(p.E));
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || configured_smem[dev] < smem) {
    e = cudaFuncSetAttribute(mp_k_expert_matmul<BN, TB>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured_smem[dev] = smem;
  }
  // at most one tile per row block and expert
  const int64_t mt = (int64_t(p.rows) + kBM - 1) / kBM + (p.E - 1);
  const int64_t tiles = mt * ((p.out_cols + BN - 1) / BN);
  if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const int grid = int(tiles < sm_count() ? tiles : sm_count());
  mp_k_expert_matmul<BN, TB><<<grid, kMMThreads, size_t(smem), st>>>(ma, mw, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_matmul(int E, int rows, int N, int K, bool dgrad, const void* a,
                                 const float* a_scales, const void* w, const float* w_scales,
                                 const int32_t* expert_offsets, void* out, int32_t* dev_err,
                                 cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int red = dgrad ? N : K, cols = dgrad ? K : N;
  const int kb = K / MP_SCALE_BLOCK, nb = (N + MP_SCALE_BLOCK - 1) / MP_SCALE_BLOCK;
  MMArgs p;
  p.E = E;
  p.rows = rows;
  p.out_cols = cols;
  p.red_blocks = red / kBK;
  p.w_rows = N;
  p.a_scales = a_scales;
  p.w_scales = w_scales;
  p.ws_expert = int64_t(nb) * kb;
  p.ws_out = dgrad ? 1 : kb;
  p.ws_red = dgrad ? kb : 1;
  p.expert_offsets = expert_offsets;
  p.out = static_cast<uint16_t*>(out);
  p.dev_err = dev_err;
  const int BN = 256;
  CUtensorMap ma, mw;
  if (!make_map_2d(&ma, a, 1, uint64_t(red), uint64_t(rows), kBK, kABox) ||
      !make_map_2d(&mw, w, 1, uint64_t(K), uint64_t(E) * N, kBK, dgrad ? kBK : BN))
    return cudaErrorInvalidValue;
  return dgrad ? launch_mm<256, true>(p, ma, mw, st) : launch_mm<256, false>(p, ma, mw, st);
}

}  // namespace mp
