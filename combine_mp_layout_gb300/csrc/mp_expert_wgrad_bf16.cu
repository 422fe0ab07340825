// mp_expert_wgrad_bf16.cu -- the gradient of the experts' weights from bf16 rows
// (sm_103a: TMA, tcgen05 on pairs of blocks, TMEM).
//
//   dw[e][n][k] (+)= sum over the rows r of expert e of dy[r][n] * a[r][k]
//
// Products are exact, sums over the rows fp32 in TMEM; then one rounding to bf16,
// or none (fp32, optionally added to what stands there: one fp32 addition).
//
// A pair of blocks (cta_group::2) works on 256 x 256 weights, 64 rows per stage:
// each block loads its 128 dy channels (M) and its half of the a channels (N), 32
// KB for 512 clocks of MMA.  Both operands are MN-major: a row of channels stays a
// row in shared memory, nothing is transposed.
//
// An expert's last stage may reach into the next expert's rows (or past the array,
// where the loads give zeros).  These rows must not count, whatever they hold, so
// a warp of each block overwrites them with zeros in shared memory, up to the next
// multiple of 16; steps of 16 rows behind that are not issued.
//
// With few tiles, clusters of two to four pairs share a tile's rows and join their
// sums through shared memory in a fixed order (SPLIT).
//
// Measured: 32,768 rows over 32 experts, 4096 x 7168, to bf16 1.05 ms cool (1.83
// PFLOP/s), 1.22 ms at the card's power limit; without the stores of 1.9 GB 0.96 ms.
// 4,095 rows, skewed, over 64 experts of 4096 x 2048, to fp32: 363 us, 5.9 TB/s written.
//
// Warps of a block: one loads, one (of the pair's first block) issues the MMAs,
// one clears, four write finished tiles while the next one's products run.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

constexpr int kWC = 128;                      // dy and a channels per block
constexpr int kWRows = 64;                    // rows per stage: four K = 16 steps
constexpr int kWOperand = kWRows * kWC * 2;
constexpr int kWStage = 2 * kWOperand;
constexpr int kChunk = kWRows * 128;          // 64 channels (128 bytes) of a stage's rows
constexpr int kWStages = 6;
constexpr int kSlab = 32 * 128;               // 128 bytes of 32 finished rows
constexpr int kEpiWarps = 4;
constexpr int kClearWarp = 2, kEpiFirst = 3;
constexpr int kWThreads = (kEpiFirst + kEpiWarps) * 32;

struct WArgs {
  int E, rows, N, K;
  const int32_t* expert_offsets;
  void* dw;
  int32_t* dev_err;
  int accumulate;  // fp32: add to dw
  int patience;    // of the waits for whole tiles
};

struct WTail {
  uint64_t full[kWStages], empty[kWStages];  // full: of the pair's first block
  uint64_t last[kWStages];                   // this block's loads of a stage to be cleared
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int failed;
};
constexpr size_t kWSmem = size_t(kWStages) * kWStage + kEpiWarps * 2 * kSlab + sizeof(WTail);
static_assert(kWSmem <= size_t(kMaxBlockSmem));

struct WTile {
  int e, lo, hi, n0, k0;  // n0, k0: of the pair
  __device__ __forceinline__ int steps() const { return (hi - lo + kWRows - 1) / kWRows; }
  // rows of the last stage, 0 if it is a whole one
  __device__ __forceinline__ int rest() const { return (hi - lo) % kWRows; }
};

// Experts ascending, then n, with k fastest: the tiles running at one time
// share the rows of an expert.
__device__ __forceinline__ WTile wtile_at(const WArgs& p, int t) {
  const int kt = ceil_div(p.K, 2 * kWC), nt = ceil_div(p.N, 2 * kWC);
  WTile w;
  w.e = t / (kt * nt);
  const int rem = t - w.e * (kt * nt);
  w.n0 = (rem / kt) * 2 * kWC;
  w.k0 = (rem % kt) * 2 * kWC;
  rows_of(p.expert_offsets, p.rows, w.e, w.lo, w.hi);
  return w;
}

// The stages of a pair's part of the tile's rows.
struct Steps {
  int lo, hi;
  bool cleared;  // the last one has rows of another expert
  __device__ __forceinline__ Steps(const WTile& w, int part, int parts) {
    const int all = w.steps();
    lo = int(int64_t(all) * part / parts);
    hi = int(int64_t(all) * (part + 1) / parts);
    cleared = hi == all && hi > lo && w.rest() != 0;
  }
};

// Half of a tile's a channels: whole MMA steps of 32 for the pair.
__device__ __forceinline__ int half_cols(const WArgs& p, const WTile& w) {
  return min(2 * kWC, (p.K - w.k0 + 31) & ~31) / 2;
}

// The parts' sums in ascending order: four columns of a row per thread and turn, the
// rows spread over the blocks that hold the same ones.
template <bool F32>
__device__ __forceinline__ void join_sums(const WArgs& p, const WTile& w, int rank, int part,
                                          int parts, const void* stages) {
  if (F32 && p.accumulate && w.lo == w.hi) return;
  constexpr int kQuads = 2 * kWC / 4;
  for (int i = part * kWThreads + int(threadIdx.x); i < kWC * kQuads; i += parts * kWThreads) {
    const int r = i / kQuads, c = i % kQuads, n = w.n0 + rank * kWC + r, k = w.k0 + c * 4;
    if (n >= p.N || k >= p.K) continue;
    const float4* at = reinterpret_cast<const float4*>(stages) + r * kQuads + (c ^ (r & 7));
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
    const int64_t to = (int64_t(w.e) * p.N + n) * p.K + k;
    if constexpr (F32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.dw) + to);
      if (p.accumulate) {
        const float4 o = *dst;
        sum = make_float4(o.x + sum.x, o.y + sum.y, o.z + sum.z, o.w + sum.w);
      }
      *dst = sum;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dw) + to) =
          make_uint2(pack_bf16x2_rn(sum.x, sum.y), pack_bf16x2_rn(sum.z, sum.w));
    }
  }
}

// SPLIT: one tile per cluster, each of its pairs a part of the rows.
template <bool F32, bool SPLIT>
__global__ void __launch_bounds__(kWThreads, 1)
mp_k_expert_wgrad_bf16(const __grid_constant__ CUtensorMap map_dy,
                       const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_dw, const WArgs p) {
  extern __shared__ __align__(1024) unsigned char stages[];
  WTail* tail = reinterpret_cast<WTail*>(stages + size_t(kWStages) * kWStage +
                                         kEpiWarps * 2 * kSlab);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int crank = int(cluster_rank()), rank = crank & 1, even = crank & ~1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&tail->full[i], 2);
      mbar_init(&tail->empty[i], 1);
      mbar_init(&tail->last[i], 1);
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
  if (blockIdx.x == 0) {
    int bad = 0;
    for (int e = threadIdx.x; e < p.E; e += kWThreads)
      bad |= offset_errors(p.expert_offsets, p.rows, e);
    if (bad) raise_error(p.dev_err, bad);
  }
  __syncthreads();
  cluster_sync_all();  // both blocks' barriers and TMEM are ready
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int tiles = p.E * ceil_div(p.N, 2 * kWC) * ceil_div(p.K, 2 * kWC);
  const int parts = SPLIT ? int(cluster_size()) / 2 : 1, part = SPLIT ? crank / 2 : 0;
  const int first = blockIdx.x / (2 * parts), stride = SPLIT ? tiles : int(gridDim.x) / 2;
  volatile int* failed = &tail->failed;

  if (warp == 0) {
    // ---- loads: one lane keeps the ring of stages full
    if (elect_one()) {
      const uint32_t stage0 = smem_addr(stages), full0 = map_to_rank(&tail->full[0], even);
      const uint32_t last0 = map_to_rank(&tail->last[0], uint32_t(crank));
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const WTile w = wtile_at(p, t);
        const int half = half_cols(p, w);
        const int n = w.n0 + rank * kWC, k = w.k0 + rank * half;
        const uint32_t bytes = uint32_t(kWOperand + (half > 64 ? kWOperand : kChunk));
        const Steps steps(w, part, parts);
        for (int i = steps.lo; i < steps.hi; ++i, s.next(kWStages)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          const uint32_t dst = stage0 + uint32_t(s.slot) * kWStage;
          const int row = w.lo + i * kWRows;
          // a stage to be cleared goes to this block's clearing warp first
          const uint32_t bar = (steps.cleared && i + 1 == steps.hi ? last0 : full0) + s.slot * 8;
          arrive_expect_at(bar, bytes);
          tma_load_2d_pair(dst, &map_dy, n, row, bar);
          tma_load_2d_pair(dst + kChunk, &map_dy, n + 64, row, bar);
          tma_load_2d_pair(dst + kWOperand, &map_a, k, row, bar);
          if (half > 64) tma_load_2d_pair(dst + kWOperand + kChunk, &map_a, k + 64, row, bar);
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < kWStages; ++i, s.next(kWStages))
        if (s.round > 0) bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed);
    }
  } else if (warp == 1) {
    // ---- products
    if (rank == 0 && elect_one()) {
      RingAt s;
      uint32_t nt = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const WTile w = wtile_at(p, t);
        const Steps steps(w, part, parts);
        if (steps.lo == steps.hi) continue;
        const uint32_t idesc = mma_idesc_bf16(2 * kWC, 2 * half_cols(p, w), true, true);
        const uint32_t buf = nt & 1u;
        if (nt >= 2)
          ok = bounded_wait(&tail->tempty[buf], ((nt >> 1) - 1) & 1u, failed, p.patience);
        for (int i = steps.lo; i < steps.hi && ok; ++i) {
          ok = bounded_wait(&tail->full[s.slot], s.round & 1u, failed);
          if (!ok) break;
          tcgen05_fence_after();
          const uint32_t sd = smem_addr(stages + size_t(s.slot) * kWStage);
          const uint64_t dd = smem_desc_sw128(sd, kChunk, 1024);
          const uint64_t da = smem_desc_sw128(sd + kWOperand, kChunk, 1024);
          const int rows = steps.cleared && i + 1 == steps.hi ? w.rest() : kWRows;
#pragma unroll
          for (int k = 0; k < kWRows / 16; ++k)
            if (k * 16 < rows)
              mma_f16_pair(tmem + buf * 256, dd + ((k * 16 * 128) >> 4),
                           da + ((k * 16 * 128) >> 4), idesc, i > steps.lo || k > 0);
          commit_to_pair(&tail->empty[s.slot], even);
          s.next(kWStages);
        }
        if (ok) commit_to_pair(&tail->tfull[buf], even);
        ++nt;
      }
    }
  } else if (warp == kClearWarp) {
    // ---- rows of another expert behind a tile's last one, to zeros
    int slot = 0;
    uint32_t phase = 0;  // bit i: parity of the next wait for last[i]
    for (int t = first; t < tiles; t += stride) {
      const WTile w = wtile_at(p, t);
      const Steps steps(w, part, parts);
      const int n = steps.hi - steps.lo, rest = w.rest();
      const int at = (slot + n + kWStages - 1) % kWStages;
      slot = (slot + n) % kWStages;
      if (!steps.cleared) continue;
      if (!bounded_wait_idle_warp(&tail->last[at], (phase >> at) & 1u, failed, p.patience)) break;
      phase ^= 1u << at;
      unsigned char* dst = stages + size_t(at) * kWStage;
      const int some = (-rest) & 15;  // rows to clear: 128 bytes of each of four chunks
      for (int i = lane; i < some * 32; i += 32)
        *reinterpret_cast<uint4*>(dst + (i & 3) * kChunk + (rest + (i >> 5)) * 128 +
                                  ((i >> 2) & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_at(map_to_rank(&tail->full[at], even));
    }
  } else {
    // ---- accumulators to weights' gradients; an expert without rows gets zeros.  A
    // warp's 32 rows go out in slabs 128 bytes wide, through shared memory (a lane its
    // row, swizzled) and TMA, so that the weights' rows are written in whole lines.
    constexpr int kCols = F32 ? 32 : 64;  // of a slab
    const int q = warp & 3;  // the TMEM lanes this warp may read: 32 q ..
    unsigned char* slabs = stages + size_t(kWStages) * kWStage + q * 2 * kSlab;
    uint32_t nt = 0;  // tiles with products so far
    int at = 0;       // the slab buffer in turn
    for (int t = first; t < tiles; t += stride) {
      const WTile w = wtile_at(p, t);
      const Steps steps(w, part, parts);
      const bool some = steps.hi > steps.lo;
      if (!SPLIT && !some && F32 && p.accumulate) continue;
      const uint32_t buf = nt & 1u;
      if (some && !bounded_wait_idle_warp(&tail->tfull[buf], (nt >> 1) & 1u, failed, p.patience))
        break;
      tcgen05_fence_after();
      const int n0 = w.n0 + rank * kWC + q * 32;
      const uint32_t src = tmem + buf * 256 + (uint32_t(q) << 21);
      if (SPLIT) {
        // fp32 sums into the stages, which are done with: [row][column], swizzled
        float4* row = reinterpret_cast<float4*>(stages) + (q * 32 + lane) * (2 * kWC / 4);
        for (int c = 0; c < 2 * kWC; c += 16) {
          float2 v[8] = {};
          if (some) {
            tmem_ld_x16(src + c, v);
            tmem_wait_ld(v);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            row[(c / 4 + j) ^ (lane & 7)] =
                make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
        }
      } else if (n0 < p.N) {
        const float* before =
            F32 ? static_cast<const float*>(p.dw) +
                      (int64_t(w.e) * p.N + min(n0 + lane, p.N - 1)) * p.K + w.k0
                : nullptr;
        for (int c = 0; c < 2 * kWC && w.k0 + c < p.K; c += kCols, at ^= 1) {
          unsigned char* slab = slabs + at * kSlab;
          if (lane == 0) bulk_wait_read<1>();  // what went out of this buffer has
          __syncwarp();
#pragma unroll
          for (int h = 0; h < kCols / 16; ++h) {  // 16 columns: 64 or 32 bytes of a row
            float2 v[8];
            if (some) {
              tmem_ld_x16(src + c + h * 16, v);
              tmem_wait_ld(v);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = make_float2(0.0f, 0.0f);
            }
            uint4* row = reinterpret_cast<uint4*>(slab + lane * 128);
            if constexpr (F32) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (p.accumulate) {
                  const int col = c + h * 16 + j * 4;
                  const float4 o = w.k0 + col < p.K
                                       ? *reinterpret_cast<const float4*>(before + col)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  v[2 * j] = add2(make_float2(o.x, o.y), v[2 * j]);
                  v[2 * j + 1] = add2(make_float2(o.z, o.w), v[2 * j + 1]);
                }
                row[(h * 4 + j) ^ (lane & 7)] =
                    make_uint4(__float_as_uint(v[2 * j].x), __float_as_uint(v[2 * j].y),
                               __float_as_uint(v[2 * j + 1].x), __float_as_uint(v[2 * j + 1].y));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j)
                row[(h * 2 + j) ^ (lane & 7)] = make_uint4(
                    pack_bf16x2_rn(v[4 * j].x, v[4 * j].y),
                    pack_bf16x2_rn(v[4 * j + 1].x, v[4 * j + 1].y),
                    pack_bf16x2_rn(v[4 * j + 2].x, v[4 * j + 2].y),
                    pack_bf16x2_rn(v[4 * j + 3].x, v[4 * j + 3].y));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {  // (what lies past N or K is not written)
            tma_store_3d(&map_dw, w.k0 + c, n0, w.e, slab);
            bulk_commit();
          }
        }
      }
      if (some) {
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(map_to_rank(&tail->tempty[buf], even));
        ++nt;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (first < tiles) join_sums<F32>(p, wtile_at(p, first), rank, part, parts, stages);
  }
  cluster_end();  // nothing of the cluster is in use any more
  if (warp == 1) tmem_dealloc<true>(tmem, 512);
  if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
}

template <bool F32>
cudaError_t launch_wgrad(const WArgs& p, const CUtensorMap& mdy, const CUtensorMap& ma,
                         cudaStream_t st) {
  CUtensorMap mdw;
  if (!make_map_3d(&mdw, p.dw,
                   F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   F32 ? 4 : 2, uint64_t(p.K), uint64_t(p.N), uint64_t(p.E), F32 ? 32 : 64, 32))
    return cudaErrorInvalidValue;
  static thread_local bool whole[64] = {}, split[64] = {};
  cudaError_t e = allow_smem(mp_k_expert_wgrad_bf16<F32, false>, whole);
  if (e == cudaSuccess) e = allow_smem(mp_k_expert_wgrad_bf16<F32, true>, split);
  if (e != cudaSuccess) return e;
  const int64_t tiles = int64_t(p.E) * ceil_div(p.N, 2 * kWC) * ceil_div(p.K, 2 * kWC);
  // (an expert's stages on average)
  const int parts = parts_for(mp_k_expert_wgrad_bf16<F32, true>, kWThreads, tiles, 2, kMaxParts,
                              p.rows / p.E / kWRows, 16);
  if (parts > 1)
    return launch_waiting(mp_k_expert_wgrad_bf16<F32, true>, dim3(unsigned(tiles) * 2 * parts),
                          dim3(kWThreads), kWSmem, st, unsigned(2 * parts), mdy, ma, mdw, p);
  const int pairs = int(std::min<int64_t>(tiles, sm_count() / 2));
  return launch_waiting(mp_k_expert_wgrad_bf16<F32, false>, dim3(unsigned(2 * pairs)),
                        dim3(kWThreads), kWSmem, st, 2u, mdy, ma, mdw, p);
}

}  // namespace

cudaError_t launch_expert_wgrad_bf16(int E, int rows, int N, int K, const void* dy, const void* a,
                                     const int32_t* expert_offsets, bool f32, bool accumulate,
                                     void* dw, int32_t* dev_err, cudaStream_t st) {
  WArgs p = {};
  p.E = E; p.rows = rows; p.N = N; p.K = K;
  p.expert_offsets = expert_offsets;
  p.dw = dw;
  p.dev_err = dev_err;
  p.accumulate = accumulate;
  p.patience = 1 + rows / (1 << 20);
  CUtensorMap mdy = {}, ma = {};
  if (rows > 0 && (!make_map_bf16(&mdy, dy, uint64_t(N), uint64_t(rows), 64, kWRows) ||
                   !make_map_bf16(&ma, a, uint64_t(K), uint64_t(rows), 64, kWRows)))
    return cudaErrorInvalidValue;
  return f32 ? launch_wgrad<true>(p, mdy, ma, st) : launch_wgrad<false>(p, mdy, ma, st);
}

}  // namespace mp
