// mp_expert_matmul.cu -- products of the experts on e4m3 rows with one fp32
// scale per block of 128, grouped by expert (sm_103a: TMA, tcgen05, TMEM).
//
// Forward   y[r][n]  = sum_kb sa[r][kb] * sw[e][n/128][kb] * P(r, n, kb),
//           P(r, n, kb) = sum over the 128 channels k of block kb of a[r][k] * w[e][n][k]
// Gradient of the rows (DGRAD: the same weights, read along the other axis)
//           dx[r][k] = sum_nb sd[r][nb] * sw[e][nb][k/128] * sum_{n in nb} dy[r][n] * w[e][n][k]
// for every row r of expert e (rows expert_offsets[e] .. expert_offsets[e+1]).
//
// The scales change every 128 channels of the reduction, so the tensor core
// sums one block (four K = 32 steps of kind::f8f6f4: exact products, fp32 sums
// in TMEM) and the block sums are added up in fp32 registers with their scale,
// a packed FMA per two outputs and block.
//
// Layout.  A tile is 128 rows by 256 output channels.  The rows are the M side
// (one TMEM lane each), so the scale of a row is one register of the thread that
// owns the lane: with the weights there and the rows as columns, reading a scale
// per column from shared memory took as long as the products.
//
// Warps of a block: one loads (TMA, a ring of stages), one issues the MMAs, two
// work out the scales of the next steps, the others add up the block sums.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_internal.h"
#include "mp_tcgen05.cuh"

namespace mp {

namespace {

constexpr int kBM = 128;             // rows per block
constexpr int kBN = 256;             // output channels per tile
constexpr int kBK = 128;             // reduction channels per stage: one scale block
constexpr int kShortBox = 32;        // rows per TMA box of a tile that is not full
constexpr int kEpiWarps = 8;         // two warpgroups, half of the channels each
constexpr int kEpiFirst = 4;         // warps before them: loads, products, scales (2)
constexpr int kMMThreads = (kEpiFirst + kEpiWarps) * 32;
constexpr int kCols = kBN * 4 / kEpiWarps;  // channels per warp, of 32 rows
constexpr int kTileRing = 8;         // tiles whose place is kept for the epilogue
constexpr int kBandRows = 2048;      // rows per band of the tile order
constexpr int kMaxStages = 4;
constexpr int kMaxParts = 4;         // blocks that share a tile's reduction: one cluster (of
                                     // eight, too few fit beside each other: 25 us against
                                     // 14.5 us for 32 rows x 4096 x 7168)
constexpr int kMaxSmem = 232448;     // bytes of shared memory a block may have

struct MMArgs {
  int E, rows, out_cols, red_blocks;  // out_cols: N (forward) or K (dgrad)
  int w_rows;                         // weight rows per expert (N)
  int stages;
  int out32;                          // out is 32-byte aligned
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

constexpr int kStageR = kBM * kBK;
constexpr int kStageW = kBN * kBK;
constexpr int kStage = kStageR + kStageW;

// Shared memory after the stages (1024-byte aligned, as the swizzle wants them).
// ready[slot]: the loads of a step have landed, its scales are in place and its
// accumulator is free.
// done[slot]: its products are finished, so the stage may be loaded again and
// the accumulator read.  One barrier each way per step: the thread that issues
// the products needs about 260 clocks for one wait, four MMAs and one commit,
// and with two waits and two commits it could not keep up with the products.
struct MMTail {
  uint64_t ready[kMaxStages], done[kMaxStages];
  float scale[kMaxStages][2][kBM];            // [half of the channels][row]
  int4 tile[kTileRing];                       // first row, rows, first channel
  uint32_t tmem;
  int failed;
  int scan[kMMThreads / 32];
};

size_t mm_smem_bytes(int E, int stages) {
  return size_t(stages) * kStage + sizeof(MMTail) + size_t(E + 1) * 4;
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

// Exclusive prefix over experts of their number of row tiles, into pre[0 .. E].
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

// Tile t in the order: experts ascending; within an expert, bands of kBandRows
// rows, in a band channels slowest, so that the tiles running at one time share
// few weight channels and a band's rows.
__device__ __forceinline__ Tile tile_at(const MMArgs& p, const int* pre, int ncol, int t) {
  constexpr int kBand = kBandRows / kBM;
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
  tile.col0 = nt * kBN;
  return tile;
}

// A position in a ring of n slots: the slot and how often the ring went round.
struct Ring {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      ++round;
    }
  }
};

// Every warp's end: nothing of the block (or cluster) is in use after it.
template <bool SPLIT>
__device__ __forceinline__ void block_end() {
  __syncwarp();
  tcgen05_fence_before();
  if constexpr (SPLIT) cluster_sync_all(); else __syncthreads();
  tcgen05_fence_after();
}

// SPLIT: one tile per cluster, each of its blocks a part of the reduction.
template <bool DGRAD, bool SPLIT>
__global__ void __launch_bounds__(kMMThreads, 1)
mp_k_expert_matmul(const __grid_constant__ CUtensorMap map_rows,
                   const __grid_constant__ CUtensorMap map_short,
                   const __grid_constant__ CUtensorMap map_w, const MMArgs p) {
  // (aligned by its declaration: a pointer rounded up by hand is no longer known
  // to be shared memory, and generic loads of the scales cost the epilogue time)
  extern __shared__ __align__(1024) unsigned char stages[];
  MMTail* tail = reinterpret_cast<MMTail*>(stages + size_t(p.stages) * kStage);
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&tail->ready[i], 1 + 2 + kEpiWarps);
      mbar_init(&tail->done[i], 1);
    }
    tail->failed = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<false>(&tail->tmem, 2 * kBN);
  pdl_wait_prior_grid();  // (nothing of the above touches global memory)
  tile_prefix(p, pre, tail->scan);
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int ncol = ceil_div(p.out_cols, kBN);
  const int tiles = pre[p.E] * ncol;  // below 2^31: the C ABI checks
  const int parts = SPLIT ? int(cluster_size()) : 1, part = SPLIT ? int(cluster_rank()) : 0;
  const int first = blockIdx.x / parts, step = SPLIT ? tiles : gridDim.x;
  // the reduction blocks of this block's tiles
  const int kb_lo = SPLIT ? p.red_blocks * part / parts : 0;
  const int kb_hi = SPLIT ? p.red_blocks * (part + 1) / parts : p.red_blocks;
  // steps of this block: every tile's reduction blocks, one after the other
  const int64_t count = tiles > first ? (tiles - first + step - 1) / step : 0;
  const int64_t steps = count * (kb_hi - kb_lo);
  volatile int* failed = &tail->failed;

  // The sums need more registers than a twelfth of the file: the four warps
  // before them give theirs up (128 * 96 + 256 * 200 is less than the launch's
  // 384 * 168).  Each side has its own end, which keeps the two budgets apart.
  if (warp < kEpiFirst) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 0) {
      // ---- loads: one lane keeps the ring of stages full
      if (elect_one()) {
        Ring s;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          const Tile tl = tile_at(p, pre, ncol, t);
          const int boxes = (tl.nrows + kShortBox - 1) / kShortBox;
          const uint32_t bytes = uint32_t(boxes) * kShortBox * kBK + kStageW;
          for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(p.stages)) {
            if (s.round > 0 &&
                !bounded_wait_idle(&tail->done[s.slot], (s.round - 1) & 1u, failed)) {
              ok = false;
              break;
            }
            unsigned char* sr = stages + size_t(s.slot) * kStage;
            unsigned char* sw = sr + kStageR;
            uint64_t* ready = &tail->ready[s.slot];
            mbar_arrive_expect_tx(ready, bytes);
            if (boxes == kBM / kShortBox) {
              tma_load_2d(sr, &map_rows, kb * kBK, tl.row0, ready);
            } else {
              for (int i = 0; i < boxes; ++i)
                tma_load_2d(sr + i * kShortBox * kBK, &map_short, kb * kBK,
                            tl.row0 + i * kShortBox, ready);
            }
            if constexpr (DGRAD) {
#pragma unroll
              for (int c = 0; c < kBN / 128; ++c)
                tma_load_2d(sw + c * 128 * kBK, &map_w, tl.col0 + c * 128,
                            tl.e * p.w_rows + kb * kBK, ready);
            } else {
              tma_load_2d(sw, &map_w, kb * kBK, tl.e * p.w_rows + tl.col0, ready);
            }
          }
        }
        // every load has landed and been used before the block may end
        for (int i = 0; i < p.stages; ++i, s.next(p.stages))
          if (s.round > 0) bounded_wait(&tail->done[s.slot], (s.round - 1) & 1u, failed);
      }
    } else if (warp == 1) {
      // ---- products: one lane issues the MMAs of a stage into one of two accumulators
      if (elect_one()) {
        constexpr uint32_t idesc = mma_idesc_f8(kBM, kBN, /*a_mn=*/false, /*b_mn=*/DGRAD);
        Ring s;
        uint32_t acc = tmem;
        for (int64_t i = 0; i < steps; ++i, s.next(p.stages), acc ^= kBN) {
          if (!bounded_wait(&tail->ready[s.slot], s.round & 1u, failed)) break;
          tcgen05_fence_after();
          const uint32_t sr = smem_addr(stages + size_t(s.slot) * kStage);
          const uint64_t dr = smem_desc_sw128(sr, 16, 1024);
          const uint64_t dw = smem_desc_sw128(sr + kStageR, DGRAD ? 128 * kBK : 16, 1024);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_f8(acc, dr + ((k * 32) >> 4),
                   dw + (DGRAD ? ((k * 32 * 128) >> 4) : ((k * 32) >> 4)), idesc, k > 0);
          mma_commit<false>(&tail->done[s.slot]);
        }
      }
    } else {
      // ---- scales of the next steps: row times weight scale, this warp for one
      // half of the channels.  Four steps are loaded at a time, one such group
      // ahead of the one in use: a row's scales lie red_blocks apart, so every
      // load is a trip to L2.
      const int half = warp - 2;
      const bool vec = p.red_blocks % 4 == 0 && kb_lo % 4 == 0 && kb_hi % 4 == 0 &&
                       (reinterpret_cast<uintptr_t>(p.a_scales) & 15) == 0;
      Ring s;
      // a slot's old scales are used up when the step two after theirs, which took
      // their accumulator over, is done: `behind` is that step
      Ring behind;
      behind.slot = 2;
      int made = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++made) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const float* src[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          src[i] = p.a_scales + int64_t(tl.row0 + min(lane + i * 32, tl.nrows - 1)) * p.red_blocks;
        const int cb = min((tl.col0 >> 7) + half, (p.out_cols - 1) >> 7);
        const float* sw = p.w_scales + tl.e * p.ws_expert + int64_t(cb) * p.ws_out;
        float ahead[4][4], wahead[4];
        auto load4 = [&](int kb) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            wahead[u] = kb + u < kb_hi ? __ldg(sw + int64_t(kb + u) * p.ws_red) : 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (vec) {
              const float4 v = __ldg(reinterpret_cast<const float4*>(src[i] + kb));
              ahead[i][0] = v.x;
              ahead[i][1] = v.y;
              ahead[i][2] = v.z;
              ahead[i][3] = v.w;
            } else {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                ahead[i][u] = kb + u < kb_hi ? __ldg(src[i] + kb + u) : 0.0f;
            }
          }
        };
        load4(kb_lo);
        for (int kb0 = kb_lo; kb0 < kb_hi && ok; kb0 += 4) {
          float v[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][i] = ahead[i][u] * wahead[u];
          if (kb0 + 4 < kb_hi) load4(kb0 + 4);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (kb0 + u < kb_hi && ok) {
              if (s.round > 0) {
                ok = bounded_wait_idle_warp(&tail->done[behind.slot], behind.round & 1u, failed);
                behind.next(p.stages);
              }
              if (ok) {
                // (a tile's place is overwritten kTileRing tiles later, and at most
                // as many steps as there are stages are prepared ahead)
                if (kb0 + u == kb_lo && half == 0 && lane == 0)
                  tail->tile[made % kTileRing] = make_int4(tl.row0, tl.nrows, tl.col0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) tail->scale[s.slot][half][lane + i * 32] = v[u][i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&tail->ready[s.slot]);
                s.next(p.stages);
              }
            }
          }
        }
      }
    }
    if constexpr (SPLIT) cluster_sync_all();  // (the parts are being joined)
    block_end<SPLIT>();
    if (warp == 1) tmem_dealloc<false>(tmem, 2 * kBN);
    if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- block sums from TMEM into fp32 registers, then bf16 rows
    const int q = warp & 3;                        // the TMEM lanes this warp may read: 32 q ..
    const int col = ((warp - kEpiFirst) >> 2) * kCols;  // its columns of the accumulator
    const int lrow = q * 32 + lane;
    Ring s;
    int free_slot = 0;  // the step that gets this step's accumulator next
    auto hand_back = [&] {
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->ready[free_slot]);
      if (++free_slot == p.stages) free_slot = 0;
    };
    hand_back();  // both accumulators are free at the start
    hand_back();
    uint32_t src = tmem + col + (uint32_t(q) << 21);
    int4 tl = make_int4(0, 0, 0, 0);
    for (int64_t i = 0; i < count; ++i) {
      float2 acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      bool ok = true, some = false;
      for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(p.stages), src ^= kBN) {
        ok = bounded_wait_warp(&tail->done[s.slot], s.round & 1u, failed);
        if (!ok) break;
        tcgen05_fence_after();
        if (kb == kb_lo) some = q * 32 < tail->tile[i % kTileRing].y;
        if (some) {
          const float sc = tail->scale[s.slot][col >> 7][lrow];
          const float2 s2 = make_float2(sc, sc);
          // groups of 16 channels: one on its way from TMEM while the one before
          // is added up
          float2 v[2][8];
          tmem_ld_x16(src, v[0]);
          tmem_wait_ld(v[0]);
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            if (c + 1 < kCols / 16)
              tmem_ld_x16(src + (c + 1) * 16, v[(c + 1) & 1]);
            else
              hand_back();  // the last group is in registers
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[c * 8 + j] = fma2(v[c & 1][j], s2, acc[c * 8 + j]);
            if (c + 1 < kCols / 16) tmem_wait_ld(v[(c + 1) & 1]);
          }
        } else {
          hand_back();
        }
      }
      if (!ok) break;
      tl = tail->tile[i % kTileRing];
      if (SPLIT) {
        // fp32 sums into the stages, which are done with: [4 channels][row]
        float4* mine = reinterpret_cast<float4*>(stages) + (col >> 2) * kBM + lrow;
        if (lrow < tl.y) {
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c)
            mine[c * kBM] = make_float4(acc[2 * c].x, acc[2 * c].y, acc[2 * c + 1].x,
                                        acc[2 * c + 1].y);
        }
      } else if (lrow < tl.y) {
        uint16_t* dst =
            p.out + int64_t(tl.x + lrow) * p.out_cols + tl.z + col;
        const int left = p.out_cols - (tl.z + col);  // a multiple of 16 (or <= 0)
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {  // 16 channels: one 32-byte sector
          if (c * 16 < left) {
            Words<8> o;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o.w[j] = pack_bf16x2_rn(acc[c * 8 + j].x, acc[c * 8 + j].y);
            if (p.out32) {
              st_stream_w<8>(reinterpret_cast<Words<8>*>(dst + c * 16), o);
            } else {
              int4* d = reinterpret_cast<int4*>(dst + c * 16);
              d[0] = make_int4(o.w[0], o.w[1], o.w[2], o.w[3]);
              d[1] = make_int4(o.w[4], o.w[5], o.w[6], o.w[7]);
            }
          }
        }
      }
    }
    if constexpr (SPLIT) {
      cluster_sync_all();
      // the parts in ascending order: four channels of a row per thread and turn
      const int quads = tl.y * (kBN / 4);
      for (int i = part * kEpiWarps * 32 + int(threadIdx.x) - kEpiFirst * 32; i < quads;
           i += parts * kEpiWarps * 32) {
        const int row = i / (kBN / 4), c4 = i % (kBN / 4);
        const float4* at = reinterpret_cast<const float4*>(stages) + c4 * kBM + row;
        float4 v[kMaxParts];  // all on their way before the first is needed
#pragma unroll
        for (int z = 0; z < kMaxParts; ++z)
          v[z] = z < parts ? ld_cluster_f4(map_to_rank(at, z))
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float4 sum = v[0];
#pragma unroll
        for (int z = 1; z < kMaxParts; ++z) {
          sum.x += v[z].x;
          sum.y += v[z].y;
          sum.z += v[z].z;
          sum.w += v[z].w;
        }
        if (tl.z + c4 * 4 < p.out_cols) {
          uint2 o;
          o.x = pack_bf16x2_rn(sum.x, sum.y);
          o.y = pack_bf16x2_rn(sum.z, sum.w);
          *reinterpret_cast<uint2*>(p.out + int64_t(tl.x + row) * p.out_cols + tl.z + c4 * 4) = o;
        }
      }
    }
    block_end<SPLIT>();
  }
}

// ---------------------------------------------------------------------------
// A few rows in all (one token, or one token's experts): the weights' bytes are
// the whole cost, and the tiles above spend longer on their pipeline's start
// than on the bytes.  A block takes 16 channels of one expert and up to eight
// rows (the MMA's columns), its warps every eighth scale block of the reduction.  The products are
// mma.m16n8k32 on registers: which channels of a scale block meet in one MMA is
// free, as long as both operands agree, so a thread's operands are the 16 bytes
// that it loads.  Each block sum (fp32) is scaled and added up in fp32, the
// warps' sums are joined in a fixed order.  One row of 4096 x 7168: 6.4 to 8.0 us from
// run to run, 3.7 to 4.6 TB/s of weights.
// ---------------------------------------------------------------------------
constexpr int kVecRows = 8;   // columns of the MMA, rows that the launcher gives it
constexpr int kVecWarps = 8;

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&c)[4], uint32_t a0, uint32_t a1,
                                                 uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// grid (channels / 16, rows): the block of row r works if r is its expert's first.
__global__ void __launch_bounds__(kVecWarps * 32)
mp_k_expert_matvec(const MMArgs p, const unsigned char* __restrict__ a,
                   const unsigned char* __restrict__ w) {
  __shared__ float part[kVecWarps][kVecRows][16];
  __shared__ int mine[2];  // expert, rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.y;
  int e = 0, nrows = p.rows;
  pdl_wait_prior_grid();
  if (p.expert_offsets != nullptr) {
    if (threadIdx.x == 0) mine[1] = 0;
    __syncthreads();
    int bad = 0;
    for (int i = threadIdx.x; i < p.E; i += kVecWarps * 32) {
      const int lo = __ldg(p.expert_offsets + i), hi = __ldg(p.expert_offsets + i + 1);
      if (lo < 0 || hi < lo) bad |= MP_ERR_INVALID_ARG;
      if (hi > p.rows) bad |= MP_ERR_CAPACITY;
      if (lo == row0 && hi > lo) {
        mine[0] = i;
        mine[1] = min(hi, p.rows) - lo;
      }
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) raise_error(p.dev_err, bad);
    if (__syncthreads_or(bad & MP_ERR_INVALID_ARG)) return;
    e = mine[0];
    nrows = mine[1];
  } else if (row0 != 0) {
    return;
  }
  if (nrows <= 0) return;
  const int n0 = blockIdx.x * 16;
  const int g = lane >> 2, t = lane & 3;
  const int64_t K = int64_t(p.red_blocks) * kBK;
  const unsigned char* w0 = w + (int64_t(e) * p.w_rows + n0 + g) * K + t * 16;
  const unsigned char* w1 = w0 + 8 * K;
  const unsigned char* x = a + (row0 + min(g, nrows - 1)) * K + t * 16;
  const float* sw = p.w_scales + e * p.ws_expert + int64_t(n0 >> 7) * p.ws_out;
  const float* sa0 = p.a_scales + int64_t(row0 + min(2 * t, nrows - 1)) * p.red_blocks;
  const float* sa1 = p.a_scales + int64_t(row0 + min(2 * t + 1, nrows - 1)) * p.red_blocks;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  // (one scale block at a time: with four in flight per warp the registers leave an
  // SM one block, and one row takes 9.4 us)
  for (int kb = warp; kb < p.red_blocks; kb += kVecWarps) {
    const int64_t at = int64_t(kb) * kBK;
    Words<4> va[2], vb[2];
    uint4 vx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      va[h] = ld_stream_w<4>(reinterpret_cast<const Words<4>*>(w0 + at + h * 64));
      vb[h] = ld_stream_w<4>(reinterpret_cast<const Words<4>*>(w1 + at + h * 64));
      vx[h] = __ldg(reinterpret_cast<const uint4*>(x + at + h * 64));
    }
    const float s = __ldg(sw + int64_t(kb) * p.ws_red);
    const float s0 = s * __ldg(sa0 + kb), s1 = s * __ldg(sa1 + kb);
    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mma_e4m3_16x8x32(c, va[h].w[0], vb[h].w[0], va[h].w[1], vb[h].w[1], vx[h].x, vx[h].y);
      mma_e4m3_16x8x32(c, va[h].w[2], vb[h].w[2], va[h].w[3], vb[h].w[3], vx[h].z, vx[h].w);
    }
    sum[0] = fmaf(c[0], s0, sum[0]);
    sum[1] = fmaf(c[1], s1, sum[1]);
    sum[2] = fmaf(c[2], s0, sum[2]);
    sum[3] = fmaf(c[3], s1, sum[3]);
  }
  part[warp][2 * t][g] = sum[0];
  part[warp][2 * t + 1][g] = sum[1];
  part[warp][2 * t][g + 8] = sum[2];
  part[warp][2 * t + 1][g + 8] = sum[3];
  __syncthreads();
  const int row = threadIdx.x >> 4, ch = threadIdx.x & 15;
  if (row < nrows) {
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecWarps; ++i) all += part[i][row][ch];
    p.out[int64_t(row0 + row) * p.out_cols + n0 + ch] = uint16_t(pack_bf16x2_rn(all, 0.0f));
  }
}

template <bool DGRAD, bool SPLIT>
cudaError_t launch_mm_as(MMArgs p, const CUtensorMap& mr, const CUtensorMap& ms,
                         const CUtensorMap& mw, int blocks, int parts, cudaStream_t st) {
  p.stages = kMaxStages;
  while (mm_smem_bytes(p.E, p.stages) > size_t(kMaxSmem)) --p.stages;
  const int smem = int(mm_smem_bytes(p.E, p.stages));
  // The limit belongs to the function on the device, and so to all threads: always the
  // most that a block may have, whatever this call needs, so that none lowers another's.
  static thread_local bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(mp_k_expert_matmul<DGRAD, SPLIT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  return launch_waiting(mp_k_expert_matmul<DGRAD, SPLIT>, dim3(unsigned(blocks)), dim3(kMMThreads),
                        size_t(smem), st, SPLIT ? unsigned(parts) : 0u, mr, ms, mw, p);
}

template <bool DGRAD>
cudaError_t launch_mm(const MMArgs& p, const void* a, const void* w, int K, int red,
                      cudaStream_t st) {
  CUtensorMap mr, ms, mw;
  if (!make_map_bytes(&mr, a, uint64_t(red), uint64_t(p.rows), kBK, kBM) ||
      !make_map_bytes(&ms, a, uint64_t(red), uint64_t(p.rows), kBK, kShortBox) ||
      !make_map_bytes(&mw, w, uint64_t(K), uint64_t(p.E) * p.w_rows, kBK, DGRAD ? kBK : kBN))
    return cudaErrorInvalidValue;
  // at most one short tile per expert
  const int64_t row_tiles = std::min<int64_t>(p.rows, int64_t(p.rows) / kBM + p.E);
  const int64_t tiles = row_tiles * ceil_div(p.out_cols, kBN);
  const int sms = sm_count();
  // too few tiles for the GPU: up to four blocks (one cluster) share each (nine
  // rows x 4096 x 7168: 12.5 us, 25.8 us with a block per tile)
  int parts = 1;
  while (parts < kMaxParts && tiles * parts * 2 <= sms && p.red_blocks >= parts * 4) parts *= 2;
  if (parts > 1)
    return launch_mm_as<DGRAD, true>(p, mr, ms, mw, int(tiles) * parts, parts, st);
  return launch_mm_as<DGRAD, false>(p, mr, ms, mw, int(std::min<int64_t>(tiles, sms)), 1, st);
}

}  // namespace

cudaError_t launch_expert_matmul(int E, int rows, int N, int K, bool dgrad, const void* a,
                                 const float* a_scales, const void* w, const float* w_scales,
                                 const int32_t* expert_offsets, void* out, int32_t* dev_err,
                                 cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int red = dgrad ? N : K, cols = dgrad ? K : N;
  const int kb = K / MP_SCALE_BLOCK, nb = ceil_div(N, MP_SCALE_BLOCK);
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
  p.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.dev_err = dev_err;
  // one expert's few rows (4096 x 7168 in this form, and as tiles, in one run: one row
  // 7.5 and 11.5 us, eight 8.5 and 12.4 us; but eight rows of seven experts 49 and 38 us)
  if (!dgrad && rows <= kVecRows && (E == 1 || rows == 1)) {
    return launch_waiting(mp_k_expert_matvec,
                          dim3(unsigned(N / 16), unsigned(expert_offsets ? rows : 1)),
                          dim3(kVecWarps * 32), 0, st, 0, p, static_cast<const unsigned char*>(a),
                          static_cast<const unsigned char*>(w));
  }
  return dgrad ? launch_mm<true>(p, a, w, K, red, st) : launch_mm<false>(p, a, w, K, red, st);
}

}  // namespace mp
