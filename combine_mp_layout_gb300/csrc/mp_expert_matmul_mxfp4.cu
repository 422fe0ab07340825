// mp_expert_matmul_mxfp4.cu -- products of the experts on bf16 rows with 4-bit
// weights (MXFP4: e2m1 codes, one UE8M0 scale per 32 channels), grouped by expert
// (sm_103a: TMA, tcgen05 on pairs of blocks, TMEM).
//
//   out[r][n] = sum over k of a[r][k] * 2^(s[e][n][k/32] - 127) * c[e][n][k]
//
// A code times its scale is a bf16 number (exactly: two significant bits, and the
// smallest scale leaves 2^-128), so the weights are turned into bf16 on their way
// into shared memory and the products are exact; sums are fp32, rounded once.
//
// Layout: that of the bf16 products, a tile of 256 channels by up to 256 rows per
// pair of blocks.  The codes come by TMA into a ring of raw stages (128 channels x
// 256 reduction steps, 16 KB); eight warps, in two groups that take alternate
// stages of 64 steps, turn them into the MMA's operand, a thread a channel's 64
// codes; one warp hands finished stages over to the tensor core's proxy (a proxy
// fence waits for the loads that its thread has in flight, and the converting
// warps have the scales' underway).
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

constexpr int kMaxStages = 4;
constexpr int kRaw = 4;                        // raw stages
constexpr int kRawSteps = 4;                   // stages of 64 in a raw stage of 256
constexpr int kRawStage = kBC * kRawSteps * kBK / 2;
constexpr int kGroupWarps = kBC / 32;          // a thread per channel
constexpr int kEpiFirst = 2, kRawWarp = kEpiFirst + kEpiWarps, kHandWarp = kRawWarp + 1,
              kConvFirst = kHandWarp + 1;
constexpr int kThreads = (kConvFirst + 2 * kGroupWarps) * 32;

struct Fp4Weights {
  const unsigned char* scales;                 // [E][N][K/32]
  int vec;                                     // 8 scales of 256 steps are one aligned word
};

struct Tail {
  uint64_t full[kMaxStages], empty[kMaxStages];  // full: of the pair's first block
  uint64_t conv[kMaxStages];                     // this block's weights of a stage are written
  uint64_t raw[kRaw], rawfree[kRaw];
  uint64_t tfull[2], tempty[2];
  alignas(16) unsigned char turned[kEpiWarps][2][kTurned];
  uint32_t tmem;
  int failed;
  int scan[kThreads / 32];
};

size_t smem_bytes(int E, int stages) {
  return size_t(stages) * kStage + size_t(kRaw) * kRawStage + sizeof(Tail) + size_t(E + 1) * 4;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The bf16 multiplier (twice) that belongs to a scale for codes as `codes8` leaves
// them, 2^-126 times their value: 2^126 * 2^(s-127) up to s = 128.
__device__ __forceinline__ uint32_t multiplier(uint32_t s) {
  return (s + 126u) * 0x00800080u;
}
// Above that the two factors are put on one after the other; 255 is NaN.
__device__ __forceinline__ uint32_t large_multiplier(uint32_t s) {
  return s == 255u ? 0x7fc07fc0u : s * 0x00800080u;
}

// Eight e2m1 codes as bf16 pairs in order, 2^-126 times their value: sign to bit
// 15, the two exponent bits and the mantissa bit to bits 8 to 6.
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

// 32 codes (16 bytes) with their scale, to four 16-byte chunks.
template <bool LARGE>
__device__ __forceinline__ void convert32(const uint4& codes, uint32_t s, uint4 (&out)[4]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const uint32_t m = LARGE ? 0x7e807e80u : multiplier(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o[4];
    codes8(w[i], o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = mul_bf16x2(o[j], m);
      if (LARGE) o[j] = mul_bf16x2(o[j], large_multiplier(s));
    }
    out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// SPLIT: one tile per cluster, each of its pairs a part of the reduction.
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mp_k_expert_matmul_mxfp4(const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ RowMaps map_r, const RaggedArgs p,
                         const Fp4Weights fw) {
  extern __shared__ __align__(1024) unsigned char stages[];
  unsigned char* raws = stages + size_t(p.stages) * kStage;
  Tail* tail = reinterpret_cast<Tail*>(raws + size_t(kRaw) * kRawStage);
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int crank = int(cluster_rank()), rank = crank & 1, even = crank & ~1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&tail->full[i], 4);
      mbar_init(&tail->empty[i], 1);
      mbar_init(&tail->conv[i], kGroupWarps);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&tail->raw[i], 1);
      mbar_init(&tail->rawfree[i], 2 * kGroupWarps);
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
  tile_prefix<kThreads>(p, SPLIT ? kBR : tile_rows<kThreads>(p, ncol, pairs, tail->scan), pre,
                        tail->scan);
  cluster_sync_all();  // the barriers and TMEM of all blocks are ready
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int tiles = pre[p.E] * ncol;  // below 2^31: the C ABI checks
  const int parts = SPLIT ? int(cluster_size()) / 2 : 1, part = SPLIT ? crank / 2 : 0;
  const int first = blockIdx.x / (2 * parts), step = SPLIT ? max(tiles, 1) : pairs;
  // raw stages of this pair's part of the reduction, and stages
  const int nk = ceil_div(p.red, kBK), nr = ceil_div(p.red, kRawSteps * kBK);
  const int rb_lo = SPLIT ? int(int64_t(nr) * part / parts) : 0;
  const int rb_hi = SPLIT ? int(int64_t(nr) * (part + 1) / parts) : nr;
  const int kb_lo = rb_lo * kRawSteps, kb_hi = min(rb_hi * kRawSteps, nk);
  volatile int* failed = &tail->failed;

  if (warp == 0) {
    // ---- rows: one lane keeps the ring of stages full
    if (elect_one()) {
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const int half = tl.n / 2, row = tl.row0 + rank * half;
        for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(p.stages)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          const uint32_t bar = map_to_rank(&tail->full[s.slot], even);
          arrive_expect_at(bar, uint32_t(half * kBK * 2));
          load_rows(stages + size_t(s.slot) * kStage + kStageC, map_r, kb * kBK, row, half, bar);
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < p.stages; ++i, s.next(p.stages))
        if (s.round > 0) bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed);
    }
  } else if (warp == 1) {
    // ---- products
    if (rank == 0 && elect_one()) {
      RingAt s;
      uint32_t nt = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++nt) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const uint32_t idesc = mma_idesc_bf16(2 * kBC, tl.n, false, false);
        const uint32_t buf = nt & 1u;
        if (nt >= 2)
          ok = bounded_wait(&tail->tempty[buf], ((nt >> 1) - 1) & 1u, failed, p.patience);
        for (int kb = kb_lo; kb < kb_hi && ok; ++kb) {
          ok = bounded_wait(&tail->full[s.slot], s.round & 1u, failed);
          if (!ok) break;
          tcgen05_fence_after();
          stage_products<false>(stages + size_t(s.slot) * kStage, tmem + buf * kBR, idesc,
                                kb == kb_lo);
          commit_to_pair(&tail->empty[s.slot], even);
          s.next(p.stages);
        }
        if (ok) commit_to_pair(&tail->tfull[buf], even);
      }
    }
  } else if (warp < kRawWarp) {
    // ---- accumulators to bf16 rows
    const int q = warp & 3;  // the TMEM lanes this warp may read: 32 q ..
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
        store_part(tl, q, src, stages);  // (the stages are done with)
      else if (ch < p.out_cols)
        write_tile(p, tl, ch, src, turned);
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(map_to_rank(&tail->tempty[buf], even));
    }
  } else if (warp == kRawWarp) {
    // ---- codes as they are, some stages ahead of the conversion
    if (elect_one()) {
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile tl = tile_at(p, pre, ncol, t);
        const int ch = tl.col0 + rank * kBC;
        for (int rb = rb_lo; rb < rb_hi; ++rb, s.next(kRaw)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->rawfree[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&tail->raw[s.slot], kRawStage);
          tma_load_3d(raws + s.slot * kRawStage, &map_w, rb * (kRawSteps * kBK / 2), ch, tl.e,
                      &tail->raw[s.slot]);
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < kRaw; ++i, s.next(kRaw))
        if (s.round > 0) bounded_wait_idle(&tail->rawfree[s.slot], (s.round - 1) & 1u, failed);
    }
  } else if (warp == kHandWarp) {
    // ---- each stage that this block's warps have written, on to the products
    if (elect_one()) {
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(p.stages)) {
          ok = bounded_wait(&tail->conv[s.slot], s.round & 1u, failed);
          if (!ok) break;
          fence_proxy_async_smem();
          arrive_at(map_to_rank(&tail->full[s.slot], even));
        }
      }
    }
  } else {
    // ---- codes to bf16: a thread 64 codes of channel r in every other stage
    const int group = (warp - kConvFirst) / kGroupWarps;
    const int r = ((warp - kConvFirst) % kGroupWarps) * 32 + lane;
    const int groups = p.red / 32;
    RingAt s, rs;
    int group_of = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile tl = tile_at(p, pre, ncol, t);
      // (channels past the last one: codes are zeros, any scale will do)
      const int ch = min(tl.col0 + rank * kBC + r, p.out_cols - 1);
      const unsigned char* sc = fw.scales + (int64_t(tl.e) * p.out_cols + ch) * groups;
      // the scales of a raw stage, one stage ahead of their use
      auto scales8 = [&](int rb) -> uint2 {
        const int g = rb * 8;
        if (fw.vec) return __ldg(reinterpret_cast<const uint2*>(sc + g));
        uint32_t v[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i >> 2] |= uint32_t(__ldg(sc + min(g + i, groups - 1))) << (8 * (i & 3));
        return make_uint2(v[0], v[1]);
      };
      uint2 ahead = scales8(rb_lo);
      for (int rb = rb_lo; rb < rb_hi && ok; ++rb, rs.next(kRaw)) {
        const uint2 now = ahead;
        if (rb + 1 < rb_hi) ahead = scales8(rb + 1);
        ok = bounded_wait_warp(&tail->raw[rs.slot], rs.round & 1u, failed);
        if (!ok) break;
        const unsigned char* src = raws + rs.slot * kRawStage + r * 128;
        const int steps = min(kRawSteps, kb_hi - rb * kRawSteps);
        for (int i = 0; i < steps; ++i, group_of ^= 1, s.next(p.stages)) {
          if (group_of != group) continue;
          const uint4 c0 = *reinterpret_cast<const uint4*>(src + (((2 * i) ^ (r & 7)) << 4));
          const uint4 c1 = *reinterpret_cast<const uint4*>(src + (((2 * i + 1) ^ (r & 7)) << 4));
          const uint32_t two = (i < 2 ? now.x : now.y) >> (16 * (i & 1));
          const uint32_t s0 = two & 255u, s1 = (two >> 8) & 255u;
          uint4 o[2][4];
          if (__any_sync(kFull, s0 > 128u || s1 > 128u)) {
            convert32<true>(c0, s0, o[0]);
            convert32<true>(c1, s1, o[1]);
          } else {
            convert32<false>(c0, s0, o[0]);
            convert32<false>(c1, s1, o[1]);
          }
          if (s.round > 0) ok = bounded_wait_warp(&tail->empty[s.slot], (s.round - 1) & 1u, failed);
          if (!ok) break;
          unsigned char* dst = stages + size_t(s.slot) * kStage + r * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(dst + ((j ^ (r & 7)) << 4)) = o[j >> 2][j & 3];
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->conv[s.slot]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->rawfree[rs.slot]);
      }
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

template <bool SPLIT>
cudaError_t launch_as(RaggedArgs p, const Fp4Weights& fw, const CUtensorMap& mw,
                      const RowMaps& mr, int blocks, int parts, cudaStream_t st) {
  p.stages = kMaxStages;
  while (smem_bytes(p.E, p.stages) > size_t(kMaxBlockSmem)) --p.stages;
  static thread_local bool configured[64] = {};
  const cudaError_t e = allow_smem(mp_k_expert_matmul_mxfp4<SPLIT>, configured);
  if (e != cudaSuccess) return e;
  return launch_waiting(mp_k_expert_matmul_mxfp4<SPLIT>, dim3(unsigned(blocks)), dim3(kThreads),
                        smem_bytes(p.E, p.stages), st, unsigned(2 * parts), mw, mr, p, fw);
}

}  // namespace

cudaError_t launch_expert_matmul_mxfp4(int E, int rows, int N, int K, const void* a,
                                       const void* w, const unsigned char* w_scales,
                                       const int32_t* expert_offsets, void* out, int32_t* dev_err,
                                       cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  if (rows <= 8 || rows / 4 <= E) {
    const cudaError_t e =
        launch_expert_rows(E, rows, N, K, a, w, w_scales, expert_offsets, out, dev_err, st);
    if (e != cudaErrorNotSupported) return e;
  }
  RaggedArgs p = {};
  p.E = E;
  p.rows = rows;
  p.out_cols = N;
  p.red = K;
  p.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && N % 16 == 0;
  p.patience = 1 + K / (1 << 20);
  p.expert_offsets = expert_offsets;
  p.out = static_cast<uint16_t*>(out);
  p.dev_err = dev_err;
  Fp4Weights fw;
  fw.scales = w_scales;
  fw.vec = K % (kRawSteps * kBK) == 0 && (reinterpret_cast<uintptr_t>(w_scales) & 7u) == 0;
  CUtensorMap mw;
  RowMaps mr;
  if (!make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(K) / 2, uint64_t(N),
                   uint64_t(E), kRawSteps * kBK / 2, kBC) ||
      !make_row_maps(&mr, a, K, rows))
    return cudaErrorInvalidValue;
  const int64_t tiles = most_row_tiles(p.E, p.rows, kBR) * ceil_div(p.out_cols, 2 * kBC);
  const int parts = parts_for(tiles, ceil_div(K, kBK), 2 * kRawSteps);
  if (parts > 1) return launch_as<true>(p, fw, mw, mr, int(tiles) * 2 * parts, parts, st);
  const int pairs = int(std::min<int64_t>(tiles, sm_count() / 2));
  return launch_as<false>(p, fw, mw, mr, 2 * pairs, 1, st);
}

}  // namespace mp
