// mp_expert_matmul_mxfp4.cu -- products of the experts on bf16 rows with 4-bit
// weights (MXFP4: e2m1 codes, one UE8M0 scale per 32 channels), grouped by expert
// (sm_103a: TMA, tcgen05 on pairs of blocks, TMEM).
//
//   out[r][n] = sum over k of a[r][k] * 2^(s[e][n][k/32] - 127) * c[e][n][k]
//
// A code times its scale is a bf16 number (exactly: two significant bits, and the
// smallest scale leaves 2^-128), so the weights are turned into bf16 on their way to
// the tensor core and the products are exact; sums are fp32, rounded once.
//
// Layout: that of the bf16 products, a tile of 256 channels by a number of rows per
// pair of blocks, but the weights' operand (the MMA's M side) lies in TMEM, in four or
// six stages of 64 steps, 32 columns each, beside the accumulators.  In shared memory
// each stage would have to be written and read there, 32 KB beside the 40 KB of the
// codes and rows, more than the products' time allows for (512 rows over 32 experts,
// 4096 x 7168: 240 us, so 180).  The codes come by TMA into a ring of raw stages (128
// channels x 256 reduction steps, 16 KB); sixteen warps, in four groups that take the
// stages in turn, turn them into bf16, a thread a channel's 64 codes.
//
// A stage's conversion takes as long as the products of some 200 rows, so what counts
// is how seldom a weight is converted: tiles are of up to 288 rows with one
// accumulator, or, where that saves no tiles, of up to 192 or 160 with two (and the
// write of a tile under the next one's products).  8,191 rows over 32 experts, 7168 x
// 2048: 169 us (1.42 PFLOP/s), 204 with 192 rows; 32,768 rows, 4096 x 7168: 1.05 ms
// (1.83 PFLOP/s).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

// TMEM is one or two accumulators of MOST columns (a tile's most rows) and stages of
// 64 steps of weights in the rest.
constexpr int kWeightCols = kBK / 2;           // TMEM columns of a stage of weights
template <int MOST>
struct Form {
  static constexpr int kAccs = MOST > 224 ? 1 : 2;
  static constexpr int kStages = MOST > 224 ? 6 : (512 - 2 * MOST) / kWeightCols;
  static constexpr int kRowStage = MOST / 2 * kBK * 2;
  static constexpr int kRaw = MOST > 224 ? 5 : 6;  // raw stages
  static_assert(kAccs * MOST + kStages * kWeightCols <= 512);
};
constexpr int kMaxStages = 6, kMaxRaw = 6;
constexpr float kLeastTurn = 6.5f;             // a stage's conversion, in units of 32 rows
constexpr int kRawSteps = 4;                   // stages of 64 in a raw stage of 256
constexpr int kRawStage = kBC * kRawSteps * kBK / 2;
constexpr int kGroupWarps = kBC / 32;          // a thread per channel
constexpr int kGroups = 4;                     // that take the stages in turn
constexpr int kConvWarps = kGroups * kGroupWarps;
constexpr int kEpiWarps = 4, kShare = kEpiWarps / 4;  // (eight take time from the converting ones)
constexpr int kEpiFirst = 2, kRawWarp = kEpiFirst + kEpiWarps, kConvFirst = kRawWarp + 1;
constexpr int kThreads = (kConvFirst + kConvWarps) * 32;

struct Fp4Weights {
  const unsigned char* scales;                 // [E][N][K/32]
  int vec;                                     // two scales of 64 steps are one aligned word
};

struct Tail {
  uint64_t full[kMaxStages], empty[kMaxStages];  // full: of the pair's first block
  uint64_t raw[kMaxRaw], rawfree[kMaxRaw];
  uint64_t tfull[2], tempty[2];
  alignas(16) unsigned char turned[kEpiWarps][2][kTurned];
  uint32_t tmem;
  int failed;
  int scan[kThreads / 32];
};

template <int MOST>
__host__ __device__ constexpr size_t ring_bytes() {
  return size_t(Form<MOST>::kRaw) * kRawStage +
         size_t(Form<MOST>::kStages) * Form<MOST>::kRowStage;
}
template <int MOST>
size_t smem_bytes(int E) {
  return ring_bytes<MOST>() + sizeof(Tail) + size_t(E + 1) * 4;
}

// The bf16 multiplier (twice) that belongs to a scale for codes as `codes8` leaves
// them, 2^-126 times their value: 2^126 * 2^(s-127) up to s = 128.
__device__ __forceinline__ uint32_t multiplier(uint32_t s) {
  return (s + 126u) * 0x00800080u;
}
// Where a warp meets a scale above that, its two factors are put on one after the other,
// and those of all the other scales too: 2^126, then 2^(s-127) for any s (at 0 that is a
// subnormal number); 255 is NaN.
__device__ __forceinline__ uint32_t large_multiplier(uint32_t s) {
  return s == 255u ? 0x7fc07fc0u : s == 0u ? 0x00400040u : s * 0x00800080u;
}

// 32 codes (16 bytes) with their scale, to 16 pairs.
template <bool LARGE>
__device__ __forceinline__ void convert32(const uint4& codes, uint32_t s, uint32_t* out) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const uint32_t m = LARGE ? 0x7e807e80u : multiplier(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o[4];
    codes8(w[i], o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[4 * i + j] = mul_bf16x2(o[j], m);
      if (LARGE) out[4 * i + j] = mul_bf16x2(out[4 * i + j], large_multiplier(s));
    }
  }
}

// 32 words of each lane to 32 columns of this warp's TMEM lanes.
__device__ __forceinline__ void tmem_st_x32(uint32_t dst, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(dst),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Pair only: M = 256 channels from both blocks' TMEM.
__device__ __forceinline__ void mma_pair_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                              bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}

// Of a tile's rows those that one MMA takes: all, or 160 of 288.
__device__ __forceinline__ int first_rows(int n) { return n <= kBR ? n : 160; }

// SPLIT: one tile per cluster, each of its pairs a part of the reduction.
template <int MOST, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mp_k_expert_matmul_mxfp4(const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ RowMaps map_r, const RaggedArgs p,
                         const Fp4Weights fw) {
  constexpr int kStages = Form<MOST>::kStages, kRowStage = Form<MOST>::kRowStage;
  constexpr int kRaw = Form<MOST>::kRaw, kAccs = Form<MOST>::kAccs;
  static_assert(kStages <= kMaxStages && kRaw <= kMaxRaw);
  static_assert(ring_bytes<MOST>() >= size_t(MOST) * kBC * 4);  // holds a part's sums
  extern __shared__ __align__(1024) unsigned char raws[];
  unsigned char* stages = raws + size_t(kRaw) * kRawStage;
  Tail* tail = reinterpret_cast<Tail*>(raws + ring_bytes<MOST>());
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int crank = int(cluster_rank()), rank = crank & 1, even = crank & ~1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&tail->full[i], 2 + 2 * kGroupWarps);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&tail->raw[i], 1);
      mbar_init(&tail->rawfree[i], kConvWarps);
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
  tile_prefix<kThreads>(p, SPLIT ? MOST : tile_rows<kThreads>(p, MOST, kLeastTurn, ncol, pairs, tail->scan), pre,
                        tail->scan);
  cluster_sync_all();  // the barriers and TMEM of all blocks are ready
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem, weights = tmem + kAccs * MOST;
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
      const uint32_t stage0 = smem_addr(stages), full0 = map_to_rank(&tail->full[0], even);
      RingAt s;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile tl = tile_at(p, pre, ncol, t);
        // (rows past the first 256 are another MMA's)
        const int n1 = first_rows(tl.n), n2 = tl.n - n1;
        const RowBoxes rows(map_r, tl.row0, n1, rank);
        const RowBoxes more(map_r, tl.row0 + n1, max(n2, kUnit), rank);
        const uint32_t bytes = rows.bytes + (n2 > 0 ? more.bytes : 0);
        for (int kb = kb_lo; kb < kb_hi; ++kb, s.next(kStages)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          const uint32_t bar = full0 + s.slot * 8;
          arrive_expect_at(bar, bytes);
          rows.load(stage0 + s.slot * kRowStage, kb * kBK, bar);
          if (MOST > kBR && n2 > 0)
            more.load(stage0 + s.slot * kRowStage + n1 / 2 * kBK * 2, kb * kBK, bar);
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < kStages; ++i, s.next(kStages))
        if (s.round > 0) bounded_wait_idle(&tail->empty[s.slot], (s.round - 1) & 1u, failed);
    }
  } else if (warp == 1) {
    // ---- products
    if (rank == 0 && elect_one()) {
      RingAt s;
      uint32_t nt = 0;
      bool ok = true;
      // (the next tile is looked up while this one's last products run; in the loop over
      // the stages it costs MXFP4 weights up to a tenth)
      int n = first < tiles ? tile_at(p, pre, ncol, first).n : 0, next = 0;
      for (int t = first; t < tiles && ok; t += step, ++nt, n = next) {
        const int n1 = first_rows(n), n2 = n - n1;
        const uint32_t idesc = mma_idesc_bf16(2 * kBC, n1, false, false);
        const uint32_t idesc2 = mma_idesc_bf16(2 * kBC, max(n2, kUnit), false, false);
        const uint32_t buf = nt % kAccs;
        if (nt >= kAccs)
          ok = bounded_wait(&tail->tempty[buf], (nt / kAccs - 1) & 1u, failed, p.patience);
        for (int kb = kb_lo; kb < kb_hi && ok; ++kb) {
          ok = bounded_wait(&tail->full[s.slot], s.round & 1u, failed);
          if (!ok) break;
          tcgen05_fence_after();
          const uint64_t dr = smem_desc_sw128(smem_addr(stages + s.slot * kRowStage), 16, 1024);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_pair_tmem(tmem + buf * MOST, weights + s.slot * kWeightCols + k * 8,
                          dr + ((k * 32) >> 4), idesc, kb > kb_lo || k > 0);
          if (MOST > kBR && n2 > 0) {
            const uint64_t dm = dr + ((n1 / 2 * kBK * 2) >> 4);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              mma_pair_tmem(tmem + n1, weights + s.slot * kWeightCols + k * 8,
                            dm + ((k * 32) >> 4), idesc2, kb > kb_lo || k > 0);
          }
          commit_to_pair(&tail->empty[s.slot], even);
          s.next(kStages);
        }
        if (ok) commit_to_pair(&tail->tfull[buf], even);
        if (t + step < tiles) next = tile_at(p, pre, ncol, t + step).n;
      }
    }
  } else if (warp < kRawWarp) {
    // ---- accumulators to bf16 rows
    const int q = warp & 3;  // the TMEM lanes this warp may read: 32 q ..
    const int share = (warp - kEpiFirst) >> 2;
    unsigned char* turned = tail->turned[warp - kEpiFirst][0];
    uint32_t nt = 0;
    for (int t = first; t < tiles; t += step, ++nt) {
      const Tile tl = tile_at(p, pre, ncol, t);
      const uint32_t buf = nt % kAccs;
      if (!bounded_wait_idle_warp(&tail->tfull[buf], (nt / kAccs) & 1u, failed, p.patience)) break;
      tcgen05_fence_after();
      const uint32_t src = tmem + buf * MOST + (uint32_t(q) << 21);
      const int ch = tl.col0 + rank * kBC + q * 32;
      if (SPLIT)
        store_part<kShare>(tl, q, src, share, raws);  // (the rings are done with)
      else if (ch < p.out_cols)
        write_tile<kShare>(p, tl, ch, src, share, turned);
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
  } else {
    // ---- codes to bf16: a thread 64 codes of channel r in every fourth stage, for the
    // TMEM lanes 32 q .. that its warp may write.  (A group skips stages, but none of
    // their slots can be a phase behind: it has waited for the use of a slot not four
    // stages before.)
    const int group = (warp - kConvFirst) / kGroupWarps, q = warp & 3;
    const int r = q * 32 + lane;
    const int groups = p.red / 32;
    RingAt rs;
    uint32_t count = 0;  // stages before the raw stage at hand
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile tl = tile_at(p, pre, ncol, t);
      // (channels past the last one: codes are zeros, any scale will do)
      const int ch = min(tl.col0 + rank * kBC + r, p.out_cols - 1);
      const unsigned char* sc = fw.scales + (int64_t(tl.e) * p.out_cols + ch) * groups;
      auto scales2 = [&](int kb) -> uint32_t {  // of the stage's two groups of 32
        if (fw.vec) return __ldg(reinterpret_cast<const uint16_t*>(sc + 2 * min(kb, nk - 1)));
        return __ldg(sc + min(2 * kb, groups - 1)) |
               uint32_t(__ldg(sc + min(2 * kb + 1, groups - 1))) << 8;
      };
      // this group's first stage of the tile; its next scales are loaded one ahead
      int mine = kb_lo + ((group - int(count)) & (kGroups - 1));
      uint32_t ahead = scales2(mine);
      for (int rb = rb_lo; rb < rb_hi && ok; ++rb, rs.next(kRaw)) {
        ok = bounded_wait_warp(&tail->raw[rs.slot], rs.round & 1u, failed);
        if (!ok) break;
        const int end = min((rb + 1) * kRawSteps, kb_hi);
        if (mine < end) {
          const int i = mine - rb * kRawSteps;
          const unsigned char* src = raws + rs.slot * kRawStage + r * 128;
          const uint4 c0 = *reinterpret_cast<const uint4*>(src + (((2 * i) ^ (r & 7)) << 4));
          const uint4 c1 = *reinterpret_cast<const uint4*>(src + (((2 * i + 1) ^ (r & 7)) << 4));
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->rawfree[rs.slot]);
          const uint32_t s0 = ahead & 255u, s1 = ahead >> 8;
          mine += kGroups;
          ahead = scales2(mine);
          uint32_t o[32];
          if (__any_sync(kFull, s0 > 128u || s1 > 128u)) {
            convert32<true>(c0, s0, o);
            convert32<true>(c1, s1, o + 16);
          } else {
            convert32<false>(c0, s0, o);
            convert32<false>(c1, s1, o + 16);
          }
          const uint32_t at = count + i, slot = at % kStages, round = at / kStages;
          if (round > 0) ok = bounded_wait_warp(&tail->empty[slot], (round - 1) & 1u, failed);
          if (!ok) break;
          tcgen05_fence_after();
          tmem_st_x32(weights + slot * kWeightCols + (uint32_t(q) << 21), o);
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(map_to_rank(&tail->full[slot], even));
        } else if (lane == 0) {  // (a short last raw stage)
          mbar_arrive(&tail->rawfree[rs.slot]);
        }
        count += end - rb * kRawSteps;
      }
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (first < tiles)
      join_parts<kThreads>(p, tile_at(p, pre, ncol, first), rank, part, parts, raws);
  }
  cluster_end();
  if (warp == 1) tmem_dealloc<true>(tmem, 512);
  if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
}

template <int MOST, bool SPLIT>
cudaError_t launch_as(const RaggedArgs& p, const Fp4Weights& fw, const CUtensorMap& mw,
                      const RowMaps& mr, int blocks, int parts, cudaStream_t st) {
  return launch_waiting(mp_k_expert_matmul_mxfp4<MOST, SPLIT>, dim3(unsigned(blocks)),
                        dim3(kThreads), smem_bytes<MOST>(p.E), st, unsigned(2 * parts), mw, mr, p,
                        fw);
}

// About how long tiles of up to MOST rows take, for experts with equal numbers of rows
// (and a spread of their root): the pairs' turns times what a turn of this form was
// measured to take, in us for 2,048 steps.  (32 experts, 7168 x 2048, with 160 / 192 /
// 288 rows: 140 rows each 111 / 125 / 124 us, 256: 201 / 208 / 162, 320: 247 / 217 / 236,
// 512: 379 / 340 / 308, 700: 475 / 409 / 411.)
template <int MOST>
float tiles_time(const RaggedArgs& p) {
  const int used = std::min(p.E, p.rows);
  const float each = float(p.rows) / float(used);
  const float tiles = std::ceil((each + (used > 1 ? std::sqrt(each) : 0.0f)) / MOST);
  const float turns =
      std::ceil(tiles * used * ceil_div(p.out_cols, 2 * kBC) / float(sm_count() / 2));
  const float turn = MOST == 160 ? 8.2f
                     : MOST == 192 ? 8.6f
                                   : 10.7f + 0.035f * std::max(each / tiles - 200.0f, -28.0f);
  return turns * turn;
}

template <int MOST>
cudaError_t launch_tiles(const RaggedArgs& p, const Fp4Weights& fw, const CUtensorMap& mw,
                         const RowMaps& mr, cudaStream_t st) {
  static thread_local bool whole[64] = {}, split[64] = {};
  cudaError_t e = allow_smem(mp_k_expert_matmul_mxfp4<MOST, false>, whole);
  if (e == cudaSuccess) e = allow_smem(mp_k_expert_matmul_mxfp4<MOST, true>, split);
  if (e != cudaSuccess) return e;
  const int64_t tiles = most_row_tiles(p.E, p.rows, MOST) * ceil_div(p.out_cols, 2 * kBC);
  const int parts = parts_for(mp_k_expert_matmul_mxfp4<MOST, true>, kThreads, tiles, 2, kMaxParts,
                              ceil_div(p.red, kRawSteps * kBK), 4);
  if (parts > 1)
    return launch_as<MOST, true>(p, fw, mw, mr, int(tiles) * 2 * parts, parts, st);
  const int pairs = int(std::min<int64_t>(tiles, sm_count() / 2));
  return launch_as<MOST, false>(p, fw, mw, mr, 2 * pairs, 1, st);
}

}  // namespace

cudaError_t launch_expert_matmul_mxfp4(int E, int rows, int N, int K, const void* a,
                                       const void* w, const unsigned char* w_scales,
                                       const int32_t* expert_offsets, void* out, int32_t* dev_err,
                                       cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  // The form for few rows: the crossing was measured with equal numbers of rows over 32
  // experts (4096 x 7168, eight each: 164 us, tiles 180).  How the rows lie is not known
  // here: 2,047 rows over 256 experts of 4096 x 2048 take 258 us spread evenly (tiles 416),
  // 463 with all but one each on the first (436), and 252 all on one (35).
  if (rows <= 16 || rows / 8 <= E) {
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
  fw.vec = K % kBK == 0 && (reinterpret_cast<uintptr_t>(w_scales) & 1u) == 0;
  CUtensorMap mw;
  RowMaps mr;
  if (!make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(K) / 2, uint64_t(N),
                   uint64_t(E), kRawSteps * kBK / 2, kBC) ||
      !make_row_maps(&mr, a, K, rows))
    return cudaErrorInvalidValue;
  const float t160 = tiles_time<160>(p), t192 = tiles_time<192>(p);
  if (smem_bytes<288>(E) <= size_t(kMaxBlockSmem) && tiles_time<288>(p) < std::min(t160, t192))
    return launch_tiles<288>(p, fw, mw, mr, st);
  return t160 <= t192 ? launch_tiles<160>(p, fw, mw, mr, st)
                      : launch_tiles<192>(p, fw, mw, mr, st);
}

}  // namespace mp
