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
// With few tiles, clusters of two to four pairs share a tile's reduction and join
// their sums through shared memory in a fixed order (SPLIT).
//
// Measured, 32,768 rows over 32 experts: 4096 x 7168 1.07 ms cool (1.80 PFLOP/s, 0.95 of
// the cuBLAS burst rate) and 1.24 ms at the card's power limit, where the pipe of the
// products is active 94% of the time and the clock is what gives; its gradient through
// 7168 x 2048 0.54 and 0.63 ms.  One expert with all rows: 0.97 and 1.14 ms (cuBLAS 0.95
// and 1.12): an eighth more tiles and 1.9 GB of weights are the difference.
//
// Warps of a block: one loads, one (of the pair's first block) issues the MMAs,
// eight write finished tiles while the next one's products run into the second
// accumulator (with four the writing set the pace of short reductions).
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

constexpr int kMaxStages = 6;
constexpr int kEpiWarps = 8, kEpiFirst = 2;
constexpr int kShare = kEpiWarps / 4;           // warps that share a quarter of the channels
constexpr int kThreads = (kEpiFirst + kEpiWarps) * 32;

// Shared memory after the stages (1024-byte aligned, as the swizzle wants them).
struct Tail {
  uint64_t full[kMaxStages], empty[kMaxStages];  // full: of the pair's first block
  uint64_t tfull[2], tempty[2];
  alignas(16) unsigned char turned[kEpiWarps][2][kTurned];
  uint32_t tmem;
  int failed;
  int scan[kThreads / 32];
};

size_t smem_bytes(int E, int stages) {
  return size_t(stages) * kStage + sizeof(Tail) + size_t(E + 1) * 4;
}

// SPLIT: one tile per cluster, each of its pairs a part of the reduction.
template <bool DGRAD, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mp_k_expert_matmul_bf16(const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ RowMaps map_r, const RaggedArgs p) {
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
  const int ncol = ceil_div(p.out_cols, 2 * kBC);
  const int pairs = SPLIT ? 1 : int(gridDim.x) / 2;
  tile_prefix<kThreads>(p, SPLIT ? kBR : tile_rows<kThreads>(p, kBR, 0.0f, ncol, pairs, tail->scan), pre,
                        tail->scan);
  cluster_sync_all();  // the barriers and TMEM of all blocks are ready
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int tiles = pre[p.E] * ncol;  // below 2^31: the C ABI checks
  const int parts = SPLIT ? int(cluster_size()) / 2 : 1, part = SPLIT ? crank / 2 : 0;
  const int first = blockIdx.x / (2 * parts), step = SPLIT ? max(tiles, 1) : pairs;
  const int nk = ceil_div(p.red, kBK);
  const int kb_lo = SPLIT ? int(int64_t(nk) * part / parts) : 0;
  const int kb_hi = SPLIT ? int(int64_t(nk) * (part + 1) / parts) : nk;
  volatile int* failed = &tail->failed;

  if (warp == 0) {
    // ---- loads: one lane keeps the ring of stages full
    if (elect_one()) {
      const uint32_t stage0 = smem_addr(stages), full0 = map_to_rank(&tail->full[0], even);
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const RowBoxes rows(map_r, tl.row0, tl.n, rank);
        const uint32_t bytes = kStageC + rows.bytes;
        const int ch = tl.col0 + rank * kBC;
        for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(p.stages)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          const uint32_t sc = stage0 + uint32_t(s.slot) * kStage, bar = full0 + s.slot * 8;
          arrive_expect_at(bar, bytes);
          if constexpr (DGRAD) {
            tma_load_3d_pair(sc, &map_w, ch, kb * kBK, tl.e, bar);
            tma_load_3d_pair(sc + kStageC / 2, &map_w, ch + 64, kb * kBK, tl.e, bar);
          } else {
            tma_load_3d_pair(sc, &map_w, kb * kBK, ch, tl.e, bar);
          }
          rows.load(sc + kStageC, kb * kBK, bar);
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
      // (the next tile is looked up while this one's last products run)
      int n = first < tiles ? tile_at(p, pre, ncol, first).n : 0, next = 0;
      for (int t = first; t < tiles && ok; t += step, ++nt, n = next) {
        const uint32_t idesc = mma_idesc_bf16(2 * kBC, n, DGRAD, false);
        const uint32_t buf = nt & 1u;
        if (nt >= 2)
          ok = bounded_wait(&tail->tempty[buf], ((nt >> 1) - 1) & 1u, failed, p.patience);
        for (int kb = kb_lo; kb < kb_hi && ok; ++kb) {
          ok = bounded_wait(&tail->full[s.slot], s.round & 1u, failed);
          if (!ok) break;
          tcgen05_fence_after();
          stage_products<DGRAD>(stages + size_t(s.slot) * kStage, tmem + buf * kBR, idesc,
                                kb == kb_lo);
          commit_to_pair(&tail->empty[s.slot], even);
          s.next(p.stages);
        }
        if (ok) commit_to_pair(&tail->tfull[buf], even);
        if (t + step < tiles) next = tile_at(p, pre, ncol, t + step).n;
      }
    }
  } else {
    // ---- accumulators to bf16 rows
    const int q = warp & 3;  // the TMEM lanes this warp may read: 32 q ..
    const int mine = (warp - kEpiFirst) >> 2;
    unsigned char* turned = tail->turned[warp - kEpiFirst][0];
    uint32_t nt = 0;
    for (int t = first; t < tiles; t += step, ++nt) {
      const Tile tl = tile_at(p, pre, ncol, t);
      const uint32_t buf = nt & 1u;
      if (!bounded_wait_idle_warp(&tail->tfull[buf], (nt >> 1) & 1u, failed, p.patience)) break;
      tcgen05_fence_after();
      const uint32_t src = tmem + buf * kBR + (uint32_t(q) << 21);
      const int ch = tl.col0 + rank * kBC + q * 32;
      if (SPLIT)
        store_part<kShare>(tl, q, src, mine, stages);  // (the stages are done with)
      else if (ch < p.out_cols)
        write_tile<kShare>(p, tl, ch, src, mine, turned);
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(map_to_rank(&tail->tempty[buf], even));
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (first < tiles)
      join_parts<kThreads>(p, tile_at(p, pre, ncol, first), rank, part, parts, stages);
  }
  cluster_end();
  if (warp == 1) tmem_dealloc<true>(tmem, 512);
  if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
}

template <bool DGRAD, bool SPLIT>
cudaError_t launch_as(RaggedArgs p, const CUtensorMap& mw, const RowMaps& mr, int blocks,
                      int parts, cudaStream_t st) {
  p.stages = kMaxStages;
  while (smem_bytes(p.E, p.stages) > size_t(kMaxBlockSmem)) --p.stages;
  return launch_waiting(mp_k_expert_matmul_bf16<DGRAD, SPLIT>, dim3(unsigned(blocks)),
                        dim3(kThreads), smem_bytes(p.E, p.stages), st, unsigned(2 * parts), mw,
                        mr, p);
}

template <bool DGRAD>
cudaError_t launch_mm(const RaggedArgs& p, const void* a, const void* w, int N, int K,
                      cudaStream_t st) {
  static thread_local bool whole[64] = {}, split[64] = {};
  cudaError_t e = allow_smem(mp_k_expert_matmul_bf16<DGRAD, false>, whole);
  if (e == cudaSuccess) e = allow_smem(mp_k_expert_matmul_bf16<DGRAD, true>, split);
  if (e != cudaSuccess) return e;
  CUtensorMap mw;
  RowMaps mr;
  if (!make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, uint64_t(K), uint64_t(N),
                   uint64_t(p.E), 64, DGRAD ? kBK : kBC) ||
      !make_row_maps(&mr, a, p.red, p.rows))
    return cudaErrorInvalidValue;
  const int64_t tiles = most_row_tiles(p.E, p.rows, kBR) * ceil_div(p.out_cols, 2 * kBC);
  const int parts = parts_for(mp_k_expert_matmul_bf16<DGRAD, true>, kThreads, tiles, 2, kMaxParts,
                              ceil_div(p.red, kBK), 4);
  if (parts > 1) return launch_as<DGRAD, true>(p, mw, mr, int(tiles) * 2 * parts, parts, st);
  const int pairs = int(std::min<int64_t>(tiles, sm_count() / 2));
  return launch_as<DGRAD, false>(p, mw, mr, 2 * pairs, 1, st);
}

}  // namespace

cudaError_t launch_expert_matmul_bf16(int E, int rows, int N, int K, bool dgrad, const void* a,
                                      const void* w, const int32_t* expert_offsets, void* out,
                                      int32_t* dev_err, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  // The form for few rows: the crossing was measured with equal numbers of rows over 32
  // experts (4096 x 7168, four each: 282 us, tiles 277).  How the rows lie is not known
  // here: 256 rows all on one of 64 experts take 139 us, 39 in tiles, and spread over the 64
  // 573 and 578.
  if (!dgrad && (rows <= 16 || rows / 4 <= E)) {
    const cudaError_t e =
        launch_expert_rows(E, rows, N, K, a, w, nullptr, expert_offsets, out, dev_err, st);
    if (e != cudaErrorNotSupported) return e;
  }
  RaggedArgs p = {};
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
