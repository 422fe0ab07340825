// mp_expert_wgrad.cu -- the gradient of the experts' weights from e4m3 rows
// with one fp32 scale per 128 channels (sm_103a: tcgen05, TMEM).
//
//   dw[e][n][k] = sum over the rows r of expert e of
//                 (sd[r][n/128] * dy[r][n]) * (sa[r][k/128] * a[r][k])
//
// Here the scales change with every step of the reduction, so they cannot be
// taken out of the tensor core's sum: the rows are dequantised to f16 on their
// way into shared memory.  A code is exact in f16; its scale is divided by a
// power of two near the largest scale that its channel block has in the expert
// and rounded to f16, and so is their product: 2^-11 each, where the code itself
// carries up to 2^-4.  That holds within f16's normal range: for every code at
// scales down to 2^-10 of the largest, for codes from 1 up down to 2^-19; below it
// the error is half a step of f16's subnormals, 2^-30 of the largest scale.
// Blocks whose codes are all zero do not count for the largest: quantisers give
// them scale 1, which beside a gradient's small scales would leave these no bits.
// Products are exact, sums over the rows fp32 in TMEM; the powers of two are put
// back in fp32 before the one rounding to bf16.  (Against dequantising in fp32 and
// rounding to bf16 this is eight times as exact and two instructions per pair of
// values instead of five.)
//
// A pair of blocks (cta_group::2) works on 256 x 256 weights: each block
// dequantises the 128 dy channels of its half of M and the 128 a channels of
// its half of N, 64 rows per stage.  Per stage and block that is 16,384 values
// to convert and 32 KB to write to and 32 KB to read from shared memory per 512
// clocks of MMA; one block alone on 128 x 256 has to convert and move half as
// much again for the same products.  Both operands are MN-major: a row of
// channels stays a row in shared memory, nothing is transposed.
//
// Measured: 32,768 rows over 32 experts, 4096 x 7168: 1.7 ms (1.13 PFLOP/s, 0.60 of
// the cuBLAS bf16 burst rate); bound by the converting warps (a stage about 1,000
// clocks, its products 512; tensor pipe 48% active).
//
// Warps of a block: one loads rows and scales as they are (TMA, a ring of raw
// stages: with loads to registers the lines that an SM can have on their way,
// half of them for a scale each, set the pace), sixteen convert from there,
// four write finished tiles, one (in the first block) issues the MMAs, three
// look up the largest scales of
// the tiles to come, and one hands each converted stage over to the tensor
// core's proxy.  The hand-over is its own because a proxy
// fence waits for the loads that its thread has in flight: in the converting
// warps it made every stage as long as a load.
#include <algorithm>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_internal.h"
#include "mp_tcgen05.cuh"

namespace mp {

namespace {

constexpr int kWC = 128;            // dy and a channels per block: one scale block each
constexpr int kWRows = 64;          // rows per stage: four K = 16 steps of kind::f16
constexpr int kWStages = 4;
constexpr int kWOperand = kWRows * kWC * 2;
constexpr int kWStage = 2 * kWOperand;
constexpr int kConvWarps = 16;
constexpr int kRaw = 5;             // raw stages: dy and a codes, then their scales
constexpr int kRawCodes = kWRows * kWC;
constexpr int kRawScales = kWRows * 16;  // four scales of a row: one TMA box is 16 bytes wide
constexpr int kRawStage = 2 * (kRawCodes + kRawScales);
constexpr int kMmaWarp = kConvWarps + 4, kHandWarp = kMmaWarp + 1, kNormWarp = kMmaWarp + 2,
              kLoadWarp = kNormWarp + 3;
constexpr int kWThreads = (kLoadWarp + 1) * 32;
constexpr int kNorms = 4;           // tiles whose powers of two are kept
constexpr int kLbo = kWRows * 128;  // 64 f16 channels (128 bytes) of all of a stage's rows

struct WgradArgs {
  int E, rows, N, K;
  const unsigned char* dy;
  const float* dy_scales;
  const unsigned char* a;
  const float* a_scales;
  const int32_t* expert_offsets;
  uint16_t* dw;
  int32_t* dev_err;
  int out32;                        // dw is 32-byte aligned
  int tma_scales;                   // both scale arrays can be loaded by TMA
  int patience;                     // of the waits
};

struct WgradTail {
  uint64_t raw[kRaw], rawfree[kRaw];
  uint64_t conv[kWStages];          // a block's half of a stage is written
  uint64_t nfull[kNorms], nempty[kNorms];
  // powers of two of this block's dy and a channels, and the limits of their scales
  // times these
  struct __align__(16) Norm { float dy, a; __half most_dy, most_a; } norm[kNorms];
  int back[kNorms][3];              // exponents to put back: dy's, and both blocks' a's
  int2 queue[3][2 * kWarp];         // rows whose codes are to be looked at, their scales
  uint64_t full[kWStages], empty[kWStages], tfull[2], tempty[2];
  uint32_t tmem;
  int failed;
};
constexpr size_t kWSmem =
    size_t(kWStages) * kWStage + size_t(kRaw) * kRawStage + sizeof(WgradTail);

struct WTile {
  int e, lo, hi, n0, k0;  // n0, k0: of the pair
};

// Experts ascending, then n, with k fastest: the tiles running at one time
// share the rows of an expert.
__device__ __forceinline__ WTile wtile_at(const WgradArgs& p, int t) {
  const int kt = ceil_div(p.K, 2 * kWC), nt = ceil_div(p.N, 2 * kWC);
  WTile w;
  w.e = t / (kt * nt);
  const int rem = t - w.e * (kt * nt);
  w.n0 = (rem / kt) * 2 * kWC;
  w.k0 = (rem % kt) * 2 * kWC;
  if (p.expert_offsets == nullptr) {
    w.lo = 0;
    w.hi = p.rows;
  } else {
    w.lo = min(max(__ldg(p.expert_offsets + w.e), 0), p.rows);
    w.hi = max(w.lo, min(__ldg(p.expert_offsets + w.e + 1), p.rows));
  }
  return w;
}

// 16 e4m3 values times the scale s2 (twice the same) in f16: 8 words.
__device__ __forceinline__ void dequant16(const uint4& v, __half2 s2, uint32_t (&o)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h0, h1;  // f16 pairs: every e4m3 value is exact in f16
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}"
        : "=r"(h0), "=r"(h1)
        : "r"(w[i]));
    const __half2 p0 = __hmul2(*reinterpret_cast<__half2*>(&h0), s2);
    const __half2 p1 = __hmul2(*reinterpret_cast<__half2*>(&h1), s2);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&p0);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&p1);
  }
}

// The 16 channels 16c .. 16c+15 of stage row r, at the 128-byte swizzle of the
// MN-major tile.  (Eight neighbouring lanes have four chunks of two rows, whose
// swizzles differ in the lowest bit: eight different 16-byte banks.)
__device__ __forceinline__ void store16(unsigned char* tile, int r, int c, const uint32_t (&o)[8]) {
  unsigned char* row = tile + (c >> 2) * kLbo + r * 128;
  const int u = (c & 3) * 2, sw = r & 7;
  *reinterpret_cast<uint4*>(row + ((u ^ sw) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(row + (((u + 1) ^ sw) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
}

// Two scales to f16, each within its limit; NaN stays.  Past the limit only the
// scales of blocks of zeros are, which may be anything finite beside the others'.
__device__ __forceinline__ __half2 limited(float lo, float hi, __half2 most) {
  const __half2 s = __floats2half2_rn(lo, hi);
  uint32_t r;
  asm("min.NaN.xorsign.abs.f16x2 %0, %1, %2;"
      : "=r"(r)
      : "r"(*reinterpret_cast<const uint32_t*>(&s)),
        "r"(*reinterpret_cast<const uint32_t*>(&most)));
  return *reinterpret_cast<const __half2*>(&r);
}

// The scales of one channel block in an expert's rows, with its codes.
struct ScaleColumn {
  const float* scale;           // of the rows' block, `ld` floats apart
  int64_t ld;
  const unsigned char* codes;   // its 128 codes in each row, `pitch` bytes apart
  int64_t pitch;
  int lo, hi;                   // rows
};
__device__ __forceinline__ bool not_zero(uint32_t codes4) { return (codes4 & 0x7f7f7f7fu) != 0; }

constexpr int kLook = 4;            // 16-byte loads of codes per lane in flight

// Raises top to the largest scale among the first n (1 to 32) queued rows whose
// codes are not all zero: eight lanes per row, all rows on their way together.
__device__ __forceinline__ float top_of_queued(const ScaleColumn& c, const int2* queue, int n,
                                               int lane, float top) {
  unsigned mine = 0;  // of the four rows that this lane's queue place is among
#pragma unroll
  for (int s0 = 0; s0 < 8; s0 += kLook) {
    uint4 v[kLook];
#pragma unroll
    for (int s = 0; s < kLook; ++s) {
      const int row = queue[min((s0 + s) * 4 + (lane >> 3), n - 1)].x;
      v[s] = __ldg(reinterpret_cast<const uint4*>(c.codes + row * c.pitch) + (lane & 7));
    }
#pragma unroll
    for (int s = 0; s < kLook; ++s) {
      const unsigned b = __ballot_sync(kFull, not_zero(v[s].x | v[s].y | v[s].z | v[s].w));
      if (lane >> 2 == s0 + s) mine = b;
    }
  }
  const bool counts = lane < n && (mine >> ((lane & 3) * 8) & 0xffu) != 0;
  float x = counts ? __int_as_float(queue[lane].y) : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return fmaxf(top, x);
}

// The largest finite scale of the rows whose codes are not all zero.  Only rows
// above the largest found so far are looked at: a few, and those of zeros.
// (32,768 rows over 32 experts, 4096 x 7168, gradients of scale 2^-30: without
// rows of zeros 1.70 ms and not called, a tenth of them zeros 2.5 ms, half 4.6 ms.)
__device__ float top_of_used(const ScaleColumn& c, int2* queue, int lane) {
  float top = 0.0f;
  int queued = 0;
  for (int r0 = c.lo; r0 < c.hi; r0 += 256) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = r0 + i * 32 + lane;
      x[i] = row < c.hi ? fabsf(__ldg(c.scale + row * c.ld)) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool look = x[i] > top && x[i] < INFINITY;
      const unsigned b = __ballot_sync(kFull, look);
      if (look)
        queue[queued + __popc(b & ((1u << lane) - 1u))] =
            make_int2(r0 + i * 32 + lane, __float_as_int(x[i]));
      queued += __popc(b);
      __syncwarp();
      if (queued >= kWarp) {
        top = top_of_queued(c, queue, kWarp, lane, top);
        queued -= kWarp;
        const int2 rest = queue[kWarp + lane];
        __syncwarp();
        if (lane < queued) queue[lane] = rest;
        __syncwarp();
      }
    }
  }
  return queued > 0 ? top_of_queued(c, queue, queued, lane, top) : top;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWThreads, 1)
mp_k_expert_wgrad(const __grid_constant__ CUtensorMap map_dy,
                  const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_sd,
                  const __grid_constant__ CUtensorMap map_sa, const WgradArgs p) {
  extern __shared__ __align__(1024) unsigned char stages[];
  unsigned char* raws = stages + size_t(kWStages) * kWStage;
  WgradTail* tail = reinterpret_cast<WgradTail*>(raws + size_t(kRaw) * kRawStage);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = int(cluster_rank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&tail->conv[i], kConvWarps / 2);
      mbar_init(&tail->full[i], 2);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&tail->raw[i], 1);
      mbar_init(&tail->rawfree[i], kConvWarps / 2);
    }
    for (int i = 0; i < kNorms; ++i) {
      mbar_init(&tail->nfull[i], 3);
      mbar_init(&tail->nempty[i], 4 + kConvWarps);  // every warp that reads the slot
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->tfull[i], 1);
      mbar_init(&tail->tempty[i], 2 * 4);
    }
    tail->failed = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) tmem_alloc<true>(&tail->tmem, 512);
  pdl_wait_prior_grid();  // (nothing of the above touches global memory)
  if (p.expert_offsets != nullptr && blockIdx.x == 0) {
    int bad = 0;
    for (int e = threadIdx.x; e < p.E; e += kWThreads) {
      const int lo = __ldg(p.expert_offsets + e), hi = __ldg(p.expert_offsets + e + 1);
      if (lo < 0 || hi < lo) bad |= MP_ERR_INVALID_ARG;
      if (hi > p.rows) bad |= MP_ERR_CAPACITY;
    }
    if (bad) raise_error(p.dev_err, bad);
  }
  __syncthreads();
  cluster_sync_all();  // both blocks' mbarriers and TMEM are ready
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int tiles = p.E * ceil_div(p.N, 2 * kWC) * ceil_div(p.K, 2 * kWC);
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  volatile int* failed = &tail->failed;

  if (warp < kConvWarps) {
    // ---- raw rows, dequantised, into the ring of stages.  The warps are two
    // groups that take alternate stages, a thread with 16 channels of rows r and
    // r + 32 of each operand: what a stage costs in waits and arrivals is spread
    // over two stages' time.  Rows past the expert's last one (of another expert)
    // count as zeros.  Eight neighbouring lanes have four chunks of rows r and
    // r ^ 5, whose places differ by both swizzles: no two of them read or write
    // the same 16-byte bank.
    const int group = warp & 1, gw = warp >> 1;
    const int c = (lane & 3) | ((lane >> 1) & 4);
    const int r = (gw >> 1) * 8 + (((gw & 1) + ((lane >> 3) & 2)) ^ (((lane >> 2) & 1) * 5));
    const int nb = p.N / 128, kb = p.K / 128;
    uint32_t seen = 0;  // tiles with rows so far
    int slot = 0, rs = 0, turn = 0;
    uint32_t round = 0, rround = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += stride) {
      const WTile w = wtile_at(p, t);
      if (w.lo == w.hi) continue;
      const int nblk = min(w.n0 + rank * kWC, p.N - kWC) / 128;
      const int kblk = min(w.k0 + rank * kWC, p.K - kWC) / 128;
      const int norm = seen % kNorms;
      ok = bounded_wait_warp(&tail->nfull[norm], (seen / kNorms) & 1u, failed, p.patience);
      if (!ok) break;
      ++seen;
      for (int row0 = w.lo; row0 < w.hi; row0 += kWRows, turn ^= 1) {
        if (turn == group) {
          ok = bounded_wait_warp(&tail->raw[rs], rround & 1u, failed, p.patience);
          if (!ok) break;
          const unsigned char* src = raws + rs * kRawStage;
          uint4 vd[2], va[2];
          float sd[2], sa[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = (r + 32 * i) * 128 + ((c ^ (r & 7)) << 4);
            vd[i] = *reinterpret_cast<const uint4*>(src + at);
            va[i] = *reinterpret_cast<const uint4*>(src + kRawCodes + at);
            const int row = row0 + r + 32 * i;
            if (p.tma_scales) {
              const float* sc =
                  reinterpret_cast<const float*>(src + 2 * kRawCodes) + (r + 32 * i) * 4;
              sd[i] = sc[nblk & 3];
              sa[i] = sc[kWRows * 4 + (kblk & 3)];
            } else {
              const int64_t in = min(row, w.hi - 1);
              sd[i] = __ldg(p.dy_scales + in * nb + nblk);
              sa[i] = __ldg(p.a_scales + in * kb + kblk);
            }
            if (row0 + kWRows > w.hi && row >= w.hi) {
              vd[i] = va[i] = make_uint4(0, 0, 0, 0);
              sd[i] = sa[i] = 0.0f;
            }
          }
          if (round > 0)
            ok = bounded_wait_warp(&tail->empty[slot], (round - 1) & 1u, failed, p.patience);
          if (!ok) break;
          unsigned char* dst = stages + slot * kWStage;
          uint32_t o[8];
          // (read in every stage: kept over the loop it costs spills)
          const WgradTail::Norm nm = tail->norm[norm];
          const __half2 most = __halves2half2(nm.most_dy, nm.most_a);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 s2 = limited(sd[i] * nm.dy, sa[i] * nm.a, most);
            dequant16(vd[i], __low2half2(s2), o);
            store16(dst, r + 32 * i, c, o);
            dequant16(va[i], __high2half2(s2), o);
            store16(dst + kWOperand, r + 32 * i, c, o);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&tail->rawfree[rs]);
            mbar_arrive(&tail->conv[slot]);
          }
        }
        if (++rs == kRaw) {
          rs = 0;
          ++rround;
        }
        if (++slot == kWStages) {
          slot = 0;
          ++round;
        }
      }
      // Given back by either group: one without a stage in this tile is waited for by
      // nothing else, and would find the barrier a phase further.
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->nempty[norm]);
    }
  } else if (warp < kConvWarps + 4) {
    // ---- accumulators to bf16 weights' gradients; an expert without rows gets zeros
    const int q = warp & 3;
    uint32_t nt = 0;  // tiles with products so far
    for (int t = first; t < tiles; t += stride) {
      const WTile w = wtile_at(p, t);
      const bool some = w.hi > w.lo;
      const uint32_t buf = nt & 1u;
      if (some && !bounded_wait_idle_warp(&tail->tfull[buf], (nt >> 1) & 1u, failed, p.patience))
        break;
      tcgen05_fence_after();
      // The powers of two to put back, in two factors of the same sign of exponent: one
      // after the other, dy's and a's could leave fp32's range on the way to a sum that
      // lies within it.
      float2 back[2][2] = {};
      if (some) {
        const int norm = nt % kNorms;
        if (!bounded_wait_warp(&tail->nfull[norm], (nt / kNorms) & 1u, failed, p.patience)) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ex = tail->back[norm][0] + tail->back[norm][1 + h];  // -252 to 244
          const float f = __uint_as_float(uint32_t(127 + (ex >> 1)) << 23);
          const float g = __uint_as_float(uint32_t(127 + ex - (ex >> 1)) << 23);
          back[h][0] = make_float2(f, f);
          back[h][1] = make_float2(g, g);
        }
      }
      const int n = w.n0 + rank * kWC + q * 32 + lane;
      uint16_t* dst = p.dw + (int64_t(w.e) * p.N + n) * p.K + w.k0;
#pragma unroll
      for (int c = 0; c < 2 * kWC / 16; ++c) {
        float2 v[8];
        if (some) {
          tmem_ld_x16(tmem + buf * 256 + c * 16 + (uint32_t(q) << 21), v);
          tmem_wait_ld(v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = make_float2(0.0f, 0.0f);
        }
        if (n < p.N && w.k0 + c * 16 < p.K) {
          Words<8> o;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 t2 = mul2(mul2(v[j], back[c / (kWC / 16)][0]), back[c / (kWC / 16)][1]);
            o.w[j] = pack_bf16x2_rn(t2.x, t2.y);
          }
          if (p.out32) {
            st_stream_w<8>(reinterpret_cast<Words<8>*>(dst + c * 16), o);
          } else {
            uint4* d = reinterpret_cast<uint4*>(dst + c * 16);
            d[0] = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
            d[1] = make_uint4(o.w[4], o.w[5], o.w[6], o.w[7]);
          }
        }
      }
      if (some) {
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_first(&tail->tempty[buf], rank);
          mbar_arrive(&tail->nempty[nt % kNorms]);
        }
        ++nt;
      }
    }
  } else if (warp == kHandWarp) {
    // ---- each stage that this block's warps have written, on to the products
    if (elect_one()) {
      int slot = 0;
      uint32_t round = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const WTile w = wtile_at(p, t);
        const int steps = (w.hi - w.lo + kWRows - 1) / kWRows;
        for (int step = 0; step < steps; ++step) {
          ok = bounded_wait(&tail->conv[slot], round & 1u, failed, p.patience);
          if (!ok) break;
          fence_proxy_async_smem();
          mbar_arrive_first(&tail->full[slot], rank);
          if (++slot == kWStages) {
            slot = 0;
            ++round;
          }
        }
      }
    }
  } else if (warp == kLoadWarp) {
    // ---- rows and scales as they are, some stages ahead of the conversion
    if (elect_one()) {
      int rs = 0;
      uint32_t rround = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const WTile w = wtile_at(p, t);
        const int n = min(w.n0 + rank * kWC, p.N - kWC), k = min(w.k0 + rank * kWC, p.K - kWC);
        for (int row0 = w.lo; row0 < w.hi; row0 += kWRows) {
          if (rround > 0)
            ok = bounded_wait_idle(&tail->rawfree[rs], (rround - 1) & 1u, failed, p.patience);
          if (!ok) break;
          unsigned char* dst = raws + rs * kRawStage;
          uint64_t* bar = &tail->raw[rs];
          mbar_arrive_expect_tx(bar, p.tma_scales ? kRawStage : 2 * kRawCodes);
          tma_load_2d(dst, &map_dy, n, row0, bar);
          tma_load_2d(dst + kRawCodes, &map_a, k, row0, bar);
          if (p.tma_scales) {
            tma_load_2d(dst + 2 * kRawCodes, &map_sd, (n / 128) & ~3, row0, bar);
            tma_load_2d(dst + 2 * kRawCodes + kRawScales, &map_sa, (k / 128) & ~3, row0, bar);
          }
          if (++rs == kRaw) {
            rs = 0;
            ++rround;
          }
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < kRaw; ++i) {
        if (rround > 0)
          bounded_wait_idle(&tail->rawfree[rs], (rround - 1) & 1u, failed, p.patience);
        if (++rs == kRaw) {
          rs = 0;
          ++rround;
        }
      }
    }
  } else if (warp >= kNormWarp) {
    // ---- the power of two of a channel block in the tiles to come: of dy's, or
    // of one of the two of a.  Scaled by it the block's largest finite scale of
    // the expert's rows lies in [2^5, 2^6): times 448 it is within f16.
    const int which = warp - kNormWarp;
    uint32_t seen = 0;
    for (int t = first; t < tiles; t += stride) {
      const WTile w = wtile_at(p, t);
      if (w.lo == w.hi) continue;
      const int slot = seen % kNorms;
      const int ch = which == 0 ? min(w.n0 + rank * kWC, p.N - kWC)
                                : min(w.k0 + (which - 1) * kWC, p.K - kWC);
      ScaleColumn col;
      col.scale = (which == 0 ? p.dy_scales : p.a_scales) + ch / 128;
      col.ld = (which == 0 ? p.N : p.K) / 128;
      col.codes = (which == 0 ? p.dy : p.a) + ch;
      col.pitch = which == 0 ? p.N : p.K;
      col.lo = w.lo;
      col.hi = w.hi;
      float top = 0.0f, least = INFINITY;  // of the finite scales, of those above zero
      int top_row = w.lo;
      bool odd = false;  // a scale is not finite
      for (int r0 = w.lo; r0 < w.hi; r0 += 256) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = fabsf(__ldg(col.scale + min(r0 + i * 32 + lane, w.hi - 1) * col.ld));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          odd |= !(x[i] < INFINITY);
          if (x[i] > top && x[i] < INFINITY) {
            top = x[i];
            top_row = min(r0 + i * 32 + lane, w.hi - 1);
          }
          least = fminf(least, x[i] > 0.0f ? x[i] : INFINITY);
        }
      }
      const float own = top;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        least = fminf(least, __shfl_xor_sync(kFull, least, o));
      }
      odd = __any_sync(kFull, odd);
      // Within 2^10 of the largest every product with a code is a normal f16 number,
      // whichever blocks are zeros.  Otherwise the largest has to be one that counts.
      if (top > least * 0x1p10f) {
        const int row =
            __shfl_sync(kFull, top_row, __ffs(__ballot_sync(kFull, own == top)) - 1);
        const uint32_t v =
            __ldg(reinterpret_cast<const uint32_t*>(col.codes + row * col.pitch) + lane);
        if (!__any_sync(kFull, not_zero(v))) top = top_of_used(col, tail->queue[which], lane);
      }
      const int ex = max(int(__float_as_uint(top) >> 23) - 127, -121);
      if (seen >= kNorms &&
          !bounded_wait_idle_warp(&tail->nempty[slot], (seen / kNorms - 1) & 1u, failed,
                                  p.patience))
        break;
      if (lane == 0) {
        const float mul = __uint_as_float(uint32_t(132 - ex) << 23);          // 2^(5 - ex)
        // (an infinite scale stays one: its channel block is lost to all rows anyway)
        const __half most = __float2half_rn(odd ? INFINITY : 64.0f);
        if (which == 0) {
          tail->norm[slot].dy = mul;
          tail->norm[slot].most_dy = most;
        } else if (which == 1 + rank) {
          tail->norm[slot].a = mul;
          tail->norm[slot].most_a = most;
        }
        tail->back[slot][which] = ex - 5;
        mbar_arrive(&tail->nfull[slot]);
      }
      __syncwarp();
      ++seen;
    }
  } else if (rank == 0 && elect_one()) {
    // ---- products: four K = 16 MMAs a stage into the tile's accumulator
    constexpr uint32_t idesc = mma_idesc_f16(2 * kWC, 2 * kWC, true, true);
    uint32_t nt = 0;
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += stride) {
      const WTile w = wtile_at(p, t);
      const int steps = (w.hi - w.lo + kWRows - 1) / kWRows;
      if (steps == 0) continue;
      const uint32_t buf = nt & 1u;
      if (nt >= 2) ok = bounded_wait(&tail->tempty[buf], ((nt >> 1) - 1) & 1u, failed, p.patience);
      for (int step = 0; step < steps && ok; ++step) {
        ok = bounded_wait(&tail->full[slot], round & 1u, failed, p.patience);
        if (!ok) break;
        tcgen05_fence_after();
        const uint32_t sd = smem_addr(stages + slot * kWStage);
        const uint64_t dd = smem_desc_sw128(sd, kLbo, 1024);
        const uint64_t da = smem_desc_sw128(sd + kWOperand, kLbo, 1024);
#pragma unroll
        for (int k = 0; k < kWRows / 16; ++k)
          mma_f16_pair(tmem + buf * 256, dd + ((k * 16 * 128) >> 4), da + ((k * 16 * 128) >> 4),
                        idesc, step > 0 || k > 0);
        mma_commit<true>(&tail->empty[slot]);
        if (++slot == kWStages) {
          slot = 0;
          ++round;
        }
      }
      if (ok) mma_commit<true>(&tail->tfull[buf]);
      ++nt;
    }
    // the last products finish before TMEM is given back
    const int last = slot > 0 ? slot - 1 : kWStages - 1;
    if (slot > 0 || round > 0)
      bounded_wait(&tail->empty[last], (slot > 0 ? round : round - 1) & 1u, failed, p.patience);
  }

  __syncwarp();
  tcgen05_fence_before();
  cluster_sync_all();  // nothing of either block is in use any more
  tcgen05_fence_after();
  if (warp == kMmaWarp) tmem_dealloc<true>(tmem, 512);
  if (threadIdx.x == 0 && tail->failed) raise_error(p.dev_err, MP_ERR_TIMEOUT);
}

}  // namespace

cudaError_t launch_expert_wgrad(int E, int rows, int N, int K, const void* dy,
                                const float* dy_scales, const void* a, const float* a_scales,
                                const int32_t* expert_offsets, void* dw, int32_t* dev_err,
                                cudaStream_t st) {
  WgradArgs p;
  p.E = E; p.rows = rows; p.N = N; p.K = K;
  p.dy = static_cast<const unsigned char*>(dy);
  p.dy_scales = dy_scales;
  p.a = static_cast<const unsigned char*>(a);
  p.a_scales = a_scales;
  p.expert_offsets = expert_offsets;
  p.dw = static_cast<uint16_t*>(dw);
  p.dev_err = dev_err;
  p.tma_scales = 0;
  // Roles wait for whole tiles and for the look over a whole expert's scales: 2^21 rows
  // take 20 ms of products and, if all of them are zeros to look at, about 0.1 s.
  p.patience = 1 + rows / (1 << 21);
  static thread_local int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(mp_k_expert_wgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(kWSmem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  p.out32 = (reinterpret_cast<uintptr_t>(dw) & 31u) == 0;
  // below 2^31: the C ABI checks
  const int64_t tiles = int64_t(E) * ceil_div(N, 2 * kWC) * ceil_div(K, 2 * kWC);
  const int pairs = int(std::min<int64_t>(tiles, sm_count() / 2));
  CUtensorMap mdy = {}, ma = {}, msd = {}, msa = {};
  if (rows > 0) {
    const int nb = N / 128, kb = K / 128;
    // TMA wants rows of whole 16 bytes, and a base aligned to them
    p.tma_scales = nb % 4 == 0 && kb % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(dy_scales) |
                     reinterpret_cast<uintptr_t>(a_scales)) & 15u) == 0;
    if (!make_map_bytes(&mdy, dy, uint64_t(N), uint64_t(rows), kWC, kWRows) ||
        !make_map_bytes(&ma, a, uint64_t(K), uint64_t(rows), kWC, kWRows))
      return cudaErrorInvalidValue;
    if (p.tma_scales && (!make_map_f32(&msd, dy_scales, uint64_t(nb), uint64_t(rows), 4, kWRows) ||
                         !make_map_f32(&msa, a_scales, uint64_t(kb), uint64_t(rows), 4, kWRows)))
      return cudaErrorInvalidValue;
  }
  return launch_waiting(mp_k_expert_wgrad, dim3(unsigned(2 * pairs)), dim3(kWThreads), kWSmem, st,
                        0, mdy, ma, msd, msa, p);
}

}  // namespace mp
