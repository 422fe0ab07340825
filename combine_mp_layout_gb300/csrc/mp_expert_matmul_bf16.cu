// mp_expert_matmul_bf16.cu -- products of the experts on bf16 rows, grouped by
// expert (sm_103a: TMA, tcgen05 on pairs of blocks, TMEM).
//
// Forward   y[r][n]  = sum over k of a[r][k] * w[e][n][k]
// Gradient of the rows (DGRAD: the same weights, read along the other axis)
//           dx[r][k] = sum over n of dy[r][n] * w[e][n][k]
// for every row r of expert e (rows expert_offsets[e] .. expert_offsets[e+1]).
// Products are exact, sums fp32 in TMEM, one rounding to bf16.
//
// Layout.  A pair of blocks (cta_group::2) works on 256 output channels by up to
// 256 rows.  The weights are the MMA's M side and the rows its N side, because N
// can be any multiple of 32: an expert's rows are cut into equal tiles of whole
// 32s, so what its last tile wastes is less than 32 rows (with rows on the M side
// it was half a tile of 256 per expert: of 32 experts with about 1,024 rows each a
// ninth of all products).  Each block loads its 128 channels and half of the rows,
// 64 of the reduction per stage: 32 KB a stage and block for 512 clocks of MMA.
// The accumulator has a channel per TMEM lane and a row per column; the epilogue
// turns 16 rows x 32 channels at a time around in shared memory, so that a warp
// writes whole 64-byte pieces of the output's rows.
//
// Warps of a block: one loads, one (of the pair's first block) issues the MMAs,
// four write finished tiles while the next one's products run into the second
// accumulator.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

constexpr int kBC = 128;                  // channels per block: 256 per pair
constexpr int kBR = 256;                  // most rows per tile
constexpr int kUnit = 32;                 // rows that a tile is a multiple of
constexpr int kBK = 64;                   // reduction steps per stage: 128 bytes
constexpr int kStageC = kBC * kBK * 2;    // bytes of a stage: channels, then rows
constexpr int kStageR = kBR / 2 * kBK * 2;
constexpr int kStage = kStageC + kStageR;
constexpr int kMaxStages = 6;
constexpr int kMaxParts = 4;              // pairs that share a tile's reduction: one cluster
constexpr int kBandTiles = 8;             // row tiles per band of the tile order
constexpr int kEpiWarps = 4;
constexpr int kEpiFirst = 2;
constexpr int kThreads = (kEpiFirst + kEpiWarps) * 32;
constexpr int kTurn = 16 * 32 * 2;        // bytes of 16 rows x 32 channels

struct Args {
  int E, rows, out_cols, red;             // out_cols, red: N and K, or K and N
  int stages;
  int out32;                              // rows of out are 32-byte aligned
  int patience;                           // of the waits for whole tiles
  const int32_t* expert_offsets;          // [E + 1], or NULL: one expert with all rows
  uint16_t* out;                          // bf16 [rows][out_cols]
  int32_t* dev_err;
};

// Shared memory after the stages (1024-byte aligned, as the swizzle wants them).
struct Tail {
  uint64_t full[kMaxStages], empty[kMaxStages];  // full: of the pair's first block
  uint64_t tfull[2], tempty[2];
  alignas(16) unsigned char turn[kEpiWarps][2][kTurn];
  uint32_t tmem;
  int failed;
  int scan[kThreads / 32];
};

size_t smem_bytes(int E, int stages) {
  return size_t(stages) * kStage + sizeof(Tail) + size_t(E + 1) * 4;
}

// Exclusive prefix over experts of their number of row tiles, into pre[0 .. E].
// Offsets that are negative or decrease leave no tiles at all (overlapping
// experts could make more of them than the launcher's check allows for).
__device__ void tile_prefix(const Args& p, int* pre, int* scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.E + kThreads - 1) / kThreads;
  const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
  int sum = 0, bad = 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    rows_of(p.expert_offsets, p.rows, e, lo, hi);
    pre[e] = (hi - lo + kBR - 1) / kBR;
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
  if (tid == kThreads - 1) pre[p.E] = bad ? 0 : base + incl;
  __syncthreads();
}

struct Tile {
  int e, row0, nrows, n, col0;  // n: nrows rounded up to whole units
};

// Tile t in the order: experts ascending; within an expert, bands of kBandTiles
// row tiles, in a band channels slowest, so that the tiles running at one time
// share few weight channels and a band's rows.
__device__ __forceinline__ Tile tile_at(const Args& p, const int* pre, int ncol, int t) {
  int lo = 0, hi = p.E;  // pre[lo] * ncol <= t < pre[hi] * ncol
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * ncol <= t) lo = mid; else hi = mid;
  }
  const int mt = pre[lo + 1] - pre[lo];
  const int local = t - pre[lo] * ncol;
  const int band = local / (kBandTiles * ncol);
  const int rem = local - band * kBandTiles * ncol;
  const int mb = min(kBandTiles, mt - band * kBandTiles);
  const int m = band * kBandTiles + rem % mb;
  int r0, r1;
  rows_of(p.expert_offsets, p.rows, lo, r0, r1);
  // the expert's rows in whole units, spread evenly over its tiles
  const int units = (r1 - r0 + kUnit - 1) / kUnit;
  const int u0 = int(int64_t(units) * m / mt), u1 = int(int64_t(units) * (m + 1) / mt);
  Tile tile;
  tile.e = lo;
  tile.row0 = r0 + u0 * kUnit;
  tile.n = (u1 - u0) * kUnit;
  tile.nrows = min(tile.n, r1 - tile.row0);
  tile.col0 = rem / mb * 2 * kBC;
  return tile;
}

// Every warp's end: nothing of the cluster is in use after it.
__device__ __forceinline__ void cluster_end() {
  __syncwarp();
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
}

// SPLIT: one tile per cluster, each of its pairs a part of the reduction.
template <bool DGRAD, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mp_k_expert_matmul_bf16(const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ CUtensorMap map_r16,
                        const __grid_constant__ CUtensorMap map_r32,
                        const __grid_constant__ CUtensorMap map_r64,
                        const __grid_constant__ CUtensorMap map_r128, const Args p) {
  extern __shared__ __align__(1024) unsigned char stages[];
  Tail* tail = reinterpret_cast<Tail*>(stages + size_t(p.stages) * kStage);
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int crank = int(cluster_rank()), rank = crank & 1, even = crank & ~1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&tail->full[i], 2);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->tfull[i], 1);
      mbar_init(&tail->tempty[i], 2 * kEpiWarps);
    }
    tail->failed = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<true>(&tail->tmem, 512);
  pdl_wait_prior_grid();  // (nothing of the above touches global memory)
  tile_prefix(p, pre, tail->scan);
  cluster_sync_all();  // the barriers and TMEM of all blocks are ready
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int ncol = ceil_div(p.out_cols, 2 * kBC);
  const int tiles = pre[p.E] * ncol;  // below 2^31: the C ABI checks
  const int parts = SPLIT ? int(cluster_size()) / 2 : 1, part = SPLIT ? crank / 2 : 0;
  const int first = blockIdx.x / (2 * parts), step = SPLIT ? max(tiles, 1) : int(gridDim.x) / 2;
  const int nk = ceil_div(p.red, kBK);
  const int kb_lo = SPLIT ? int(int64_t(nk) * part / parts) : 0;
  const int kb_hi = SPLIT ? int(int64_t(nk) * (part + 1) / parts) : nk;
  volatile int* failed = &tail->failed;

  if (warp == 0) {
    // ---- loads: one lane keeps the ring of stages full
    if (elect_one()) {
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const int half = tl.n / 2, row = tl.row0 + rank * half;
        const CUtensorMap* map_r = half > 64   ? &map_r128
                                   : half > 32 ? &map_r64
                                   : half > 16 ? &map_r32
                                               : &map_r16;
        const int box = half > 64 ? 128 : half > 32 ? 64 : half > 16 ? 32 : 16;
        const uint32_t bytes = uint32_t(kStageC + box * kBK * 2);
        const int ch = tl.col0 + rank * kBC;
        for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(p.stages)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          unsigned char* sc = stages + size_t(s.slot) * kStage;
          const uint32_t bar = map_to_rank(&tail->full[s.slot], even);
          arrive_expect_at(bar, bytes);
          if constexpr (DGRAD) {
            tma_load_3d_pair(sc, &map_w, ch, kb * kBK, tl.e, bar);
            tma_load_3d_pair(sc + kStageC / 2, &map_w, ch + 64, kb * kBK, tl.e, bar);
          } else {
            tma_load_3d_pair(sc, &map_w, kb * kBK, ch, tl.e, bar);
          }
          tma_load_2d_pair(sc + kStageC, map_r, kb * kBK, row, bar);
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < p.stages; ++i, s.next(p.stages))
        if (s.round > 0) bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed);
    }
  } else if (warp == 1) {
    // ---- products: four K = 16 MMAs a stage into the tile's accumulator
    if (rank == 0 && elect_one()) {
      RingAt s;
      uint32_t nt = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++nt) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const uint32_t idesc = mma_idesc_bf16(2 * kBC, tl.n, DGRAD, false);
        const uint32_t buf = nt & 1u;
        if (nt >= 2)
          ok = bounded_wait(&tail->tempty[buf], ((nt >> 1) - 1) & 1u, failed, p.patience);
        for (int kb = kb_lo; kb < kb_hi && ok; ++kb) {
          ok = bounded_wait(&tail->full[s.slot], s.round & 1u, failed);
          if (!ok) break;
          tcgen05_fence_after();
          const uint32_t sc = smem_addr(stages + size_t(s.slot) * kStage);
          const uint64_t dc = smem_desc_sw128(sc, DGRAD ? kStageC / 2 : 16, 1024);
          const uint64_t dr = smem_desc_sw128(sc + kStageC, 16, 1024);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_f16_pair(tmem + buf * kBR, dc + (DGRAD ? ((k * 16 * 128) >> 4) : ((k * 32) >> 4)),
                         dr + ((k * 32) >> 4), idesc, kb > kb_lo || k > 0);
          commit_to_pair(&tail->empty[s.slot], even);
          s.next(p.stages);
        }
        if (ok) commit_to_pair(&tail->tfull[buf], even);
      }
    }
  } else {
    // ---- accumulators to bf16 rows
    const int q = warp & 3;  // the TMEM lanes this warp may read: 32 q ..
    unsigned char* turn = tail->turn[warp - kEpiFirst][0];
    uint32_t nt = 0;
    for (int t = first; t < tiles; t += step, ++nt) {
      const Tile tl = tile_at(p, pre, ncol, t);
      const uint32_t buf = nt & 1u;
      if (!bounded_wait_idle_warp(&tail->tfull[buf], (nt >> 1) & 1u, failed, p.patience)) break;
      tcgen05_fence_after();
      const uint32_t src = tmem + buf * kBR + (uint32_t(q) << 21);
      const int ch = tl.col0 + rank * kBC + q * 32;
      if (SPLIT) {
        // fp32 sums into the stages, which are done with: [row][channel]
        float* mine = reinterpret_cast<float*>(stages) + q * 32 + lane;
        for (int c = 0; c < tl.n; c += 16) {
          float2 v[8];
          tmem_ld_x16(src + c, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mine[(c + 2 * j) * kBC] = v[j].x;
            mine[(c + 2 * j + 1) * kBC] = v[j].y;
          }
        }
      } else if (ch < p.out_cols) {
        const int r = lane >> 1, h = (lane & 1) * 16;  // the row and channels that it stores
        const int left = p.out_cols - (ch + h);        // a multiple of 8 (or <= 0)
        uint16_t* dst = p.out + int64_t(tl.row0 + r) * p.out_cols + ch + h;
        float2 v[2][8];
        tmem_ld_x16(src, v[0]);
        tmem_wait_ld(v[0]);
        for (int c0 = 0; c0 < tl.n; c0 += 32) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // 16 rows; the next 16 on their way from TMEM
            const int c = c0 + b * 16;
            if (c + 16 < tl.n) tmem_ld_x16(src + c + 16, v[b ^ 1]);
            uint16_t* tw = reinterpret_cast<uint16_t*>(turn + b * kTurn) + lane;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t two = pack_bf16x2_rn(v[b][j].x, v[b][j].y);
              tw[(2 * j) * 32] = uint16_t(two);
              tw[(2 * j + 1) * 32] = uint16_t(two >> 16);
            }
            __syncwarp();
            if (c + r < tl.nrows) {
              const uint4* tr = reinterpret_cast<const uint4*>(turn + b * kTurn + r * 64 + h * 2);
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
            if (c + 16 < tl.n) tmem_wait_ld(v[b ^ 1]);
          }
        }
      }
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(map_to_rank(&tail->tempty[buf], even));
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    // the parts in ascending order: four channels of a row per thread and turn
    if (first < tiles) {
      const Tile tl = tile_at(p, pre, ncol, first);
      const int ch0 = tl.col0 + rank * kBC;
      for (int i = part * kThreads + int(threadIdx.x); i < tl.nrows * (kBC / 4);
           i += parts * kThreads) {
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
  }
  cluster_end();
  if (warp == 1) tmem_dealloc<true>(tmem, 512);
  if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
}

template <bool DGRAD, bool SPLIT>
cudaError_t launch_as(Args p, const CUtensorMap& mw, const CUtensorMap (&mr)[4], int blocks,
                      int parts, cudaStream_t st) {
  p.stages = kMaxStages;
  while (smem_bytes(p.E, p.stages) > size_t(kMaxBlockSmem)) --p.stages;
  static thread_local bool configured[64] = {};
  const cudaError_t e = allow_smem(mp_k_expert_matmul_bf16<DGRAD, SPLIT>, configured);
  if (e != cudaSuccess) return e;
  return launch_waiting(mp_k_expert_matmul_bf16<DGRAD, SPLIT>, dim3(unsigned(blocks)),
                        dim3(kThreads), smem_bytes(p.E, p.stages), st, unsigned(2 * parts), mw,
                        mr[0], mr[1], mr[2], mr[3], p);
}

template <bool DGRAD>
cudaError_t launch_mm(const Args& p, const void* a, const void* w, int N, int K,
                      cudaStream_t st) {
  CUtensorMap mw, mr[4];
  if (!make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, uint64_t(K), uint64_t(N),
                   uint64_t(p.E), 64, DGRAD ? kBK : kBC))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 4; ++i)
    if (!make_map_bf16(&mr[i], a, uint64_t(p.red), uint64_t(p.rows), kBK, 16u << i))
      return cudaErrorInvalidValue;
  // at most one short tile per expert
  const int64_t row_tiles = std::min<int64_t>(p.rows, int64_t(p.rows) / kBR + p.E);
  const int64_t tiles = row_tiles * ceil_div(p.out_cols, 2 * kBC);
  const int pairs = sm_count() / 2, nk = ceil_div(p.red, kBK);
  // Few tiles: clusters of two or four pairs share a tile's reduction, while all
  // of them run at once.
  int parts = 1;
  while (parts < kMaxParts && tiles * 2 * parts <= pairs && nk >= 4 * parts) parts *= 2;
  if (parts > 1) return launch_as<DGRAD, true>(p, mw, mr, int(tiles) * 2 * parts, parts, st);
  return launch_as<DGRAD, false>(p, mw, mr, 2 * int(std::min<int64_t>(tiles, pairs)), 1, st);
}

}  // namespace

cudaError_t launch_expert_matmul_bf16(int E, int rows, int N, int K, bool dgrad, const void* a,
                                      const void* w, const int32_t* expert_offsets, void* out,
                                      int32_t* dev_err, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  Args p = {};
  p.E = E;
  p.rows = rows;
  p.out_cols = dgrad ? K : N;
  p.red = dgrad ? N : K;
  p.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && p.out_cols % 16 == 0;
  p.patience = 1 + p.red / (1 << 20);
  p.expert_offsets = expert_offsets;
  p.out = static_cast<uint16_t*>(out);
  p.dev_err = dev_err;
  return dgrad ? launch_mm<true>(p, a, w, N, K, st) : launch_mm<false>(p, a, w, N, K, st);
}

}  // namespace mp
