// mp_expert_wgrad.cu -- the gradient of the experts' weights from e4m3 rows
// with one fp32 scale per 128 channels (sm_103a: tcgen05, TMEM).
//
//   dw[e][n][k] = sum over the rows r of expert e of
//                 (sd[r][n/128] * dy[r][n]) * (sa[r][k/128] * a[r][k])
//
// Here the scales change with every step of the reduction, so they cannot be
// taken out of the tensor core's sum: the rows are dequantised on their way
// into shared memory.  Each value (e4m3, 4 significant bits, times its fp32
// scale) is rounded once to bf16 (8 significant bits: an error of at most
// 2^-8 of the value, where e4m3 itself carries up to 2^-4), the products are
// exact and summed in fp32 in TMEM over all rows of the expert.
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

constexpr int kWM = 128;            // dy channels per tile (one scale block): the M of the MMA
constexpr int kWN = 256;            // a channels per tile (two scale blocks): its N
constexpr int kWRows = 64;          // rows per stage: four K = 16 steps of kind::f16
constexpr int kWStages = 4;
constexpr int kWStageA = kWRows * kWM * 2;
constexpr int kWStageB = kWRows * kWN * 2;
constexpr int kWStage = kWStageA + kWStageB;
constexpr int kConvWarps = 8;       // global -> registers -> bf16 -> shared memory
constexpr int kWThreads = (kConvWarps + 4 + 1) * 32;  // 4 epilogue warps, 1 MMA warp
constexpr int kLbo = kWRows * 128;  // 64 bf16 channels (128 bytes) of all of a stage's rows

struct WgradArgs {
  int E, rows, N, K;
  const unsigned char* dy;
  const float* dy_scales;
  const unsigned char* a;
  const float* a_scales;
  const int32_t* expert_offsets;
  uint16_t* dw;
  int32_t* dev_err;
};

struct WgradTail {
  uint64_t full[kWStages], empty[kWStages], tfull[2], tempty[2];
  uint32_t tmem;
  int failed;
};
constexpr size_t kWSmem = 1024 + size_t(kWStages) * kWStage + sizeof(WgradTail);

struct WTile {
  int e, lo, hi, n0, k0;
};

// Experts ascending, then n, with k fastest: the tiles running at one time
// share the rows of an expert.
__device__ __forceinline__ WTile wtile_at(const WgradArgs& p, int t) {
  const int kt = (p.K + kWN - 1) / kWN, nt = p.N / kWM;
  WTile w;
  w.e = t / (kt * nt);
  const int rem = t - w.e * (kt * nt);
  w.n0 = (rem / kt) * kWM;
  w.k0 = (rem % kt) * kWN;
  if (p.expert_offsets == nullptr) {
    w.lo = 0;
    w.hi = p.rows;
  } else {
    w.lo = min(max(__ldg(p.expert_offsets + w.e), 0), p.rows);
    w.hi = max(w.lo, min(__ldg(p.expert_offsets + w.e + 1), p.rows));
  }
  return w;
}

// 16 e4m3 values times s, rounded to bf16: 8 words.
__device__ __forceinline__ void dequant16(const uint4& v, float s, uint32_t (&o)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h0, h1;  // f16 pairs: every e4m3 value is exact in f16
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}"
        : "=r"(h0), "=r"(h1)
        : "r"(w[i]));
    const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&h0));
    const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&h1));
    o[2 * i] = pack_bf16x2_rn(f0.x * s, f0.y * s);
    o[2 * i + 1] = pack_bf16x2_rn(f1.x * s, f1.y * s);
  }
}

// The 16 channels 16c .. 16c+15 of stage row r, at the 128-byte swizzle of the
// MN-major tile.  Lanes with an odd 64-channel group store their second half
// first, so that eight neighbouring lanes hit eight different 16-byte banks.
__device__ __forceinline__ void store16(unsigned char* tile, int r, int c, const uint32_t (&o)[8]) {
  unsigned char* row = tile + (c >> 2) * kLbo + r * 128;
  const int u = (c & 3) * 2, sw = r & 7;
  const uint4 x = make_uint4(o[0], o[1], o[2], o[3]), y = make_uint4(o[4], o[5], o[6], o[7]);
  const bool odd = (c >> 2) & 1;
  *reinterpret_cast<uint4*>(row + (((odd ? u + 1 : u) ^ sw) << 4)) = odd ? y : x;
  *reinterpret_cast<uint4*>(row + (((odd ? u : u + 1) ^ sw) << 4)) = odd ? x : y;
}

__global__ void __launch_bounds__(kWThreads, 1)
mp_k_expert_wgrad(const WgradArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WgradTail* tail = reinterpret_cast<WgradTail*>(stages + size_t(kWStages) * kWStage);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&tail->full[i], kConvWarps);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->tfull[i], 1);
      mbar_init(&tail->tempty[i], 4);
    }
    tail->failed = 0;
    mbar_init_fence();
  }
  if (warp == kConvWarps + 4) tmem_alloc(&tail->tmem, 512);
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
  tcgen05_fence_after();
  const uint32_t tmem = tail->tmem;
  const int tiles = p.E * (p.N / kWM) * ((p.K + kWN - 1) / kWN);
  volatile int* failed = &tail->failed;

  if (warp < kConvWarps) {
    // ---- rows from global memory, dequantised, into the ring of stages
    const int nb = p.N / 128, kb = p.K / 128;
    const int ra = threadIdx.x >> 3, ca = threadIdx.x & 7;    // dy: 8 lanes a row, 2 x 32 rows
    const int rb = threadIdx.x >> 4, cbk = threadIdx.x & 15;  // a: 16 lanes a row, 4 x 16 rows
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const WTile w = wtile_at(p, t);
      const int steps = (w.hi - w.lo + kWRows - 1) / kWRows;
      const bool b_in = w.k0 + cbk * 16 < p.K;
      uint4 va[2], vb[4];
      float sa[2], sb[4];
      auto load = [&](int step) {
        const int r0 = w.lo + step * kWRows;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t r = r0 + ra + i * 32;
          const bool in = r < w.hi;
          va[i] = in ? __ldg(reinterpret_cast<const uint4*>(p.dy + r * p.N + w.n0) + ca)
                     : make_uint4(0, 0, 0, 0);
          sa[i] = in ? __ldg(p.dy_scales + r * nb + w.n0 / 128) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t r = r0 + rb + i * 16;
          const bool in = r < w.hi && b_in;
          vb[i] = in ? __ldg(reinterpret_cast<const uint4*>(p.a + r * p.K + w.k0) + cbk)
                     : make_uint4(0, 0, 0, 0);
          sb[i] = in ? __ldg(p.a_scales + r * kb + (w.k0 + cbk * 16) / 128) : 0.0f;
        }
      };
      if (steps > 0) load(0);
      for (int step = 0; step < steps; ++step, ++it) {
        const uint32_t st = it % kWStages, use = it / kWStages;
        if (use > 0 && !bounded_wait_warp(&tail->empty[st], (use - 1) & 1u, failed)) {
          ok = false;
          break;
        }
        unsigned char* ta = stages + size_t(st) * kWStage;
        unsigned char* tb = ta + kWStageA;
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          dequant16(va[i], sa[i], o);
          store16(ta, ra + i * 32, ca, o);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dequant16(vb[i], sb[i], o);
          store16(tb, rb + i * 16, cbk, o);
        }
        if (step + 1 < steps) load(step + 1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->full[st]);
      }
    }
  } else if (warp < kConvWarps + 4) {
    // ---- accumulators to bf16 weights' gradients; an expert without rows gets zeros
    const int q = warp & 3;
    uint32_t nt = 0;  // tiles with products so far
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const WTile w = wtile_at(p, t);
      const bool some = w.hi > w.lo;
      const uint32_t buf = nt & 1u;
      if (some && !bounded_wait_warp(&tail->tfull[buf], (nt >> 1) & 1u, failed)) {
        ok = false;
        break;
      }
      tcgen05_fence_after();
      uint16_t* dst = p.dw + (int64_t(w.e) * p.N + w.n0 + q * 32 + lane) * p.K + w.k0;
#pragma unroll
      for (int c = 0; c < kWN / 16; ++c) {
        float2 v[8];
        if (some) {
          tmem_ld_x16(tmem + buf * kWN + c * 16 + (uint32_t(q) << 21), v);
          tmem_wait_ld(v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = make_float2(0.0f, 0.0f);
        }
        if (w.k0 + c * 16 < p.K) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint4 o;
            o.x = pack_bf16x2_rn(v[4 * j].x, v[4 * j].y);
            o.y = pack_bf16x2_rn(v[4 * j + 1].x, v[4 * j + 1].y);
            o.z = pack_bf16x2_rn(v[4 * j + 2].x, v[4 * j + 2].y);
            o.w = pack_bf16x2_rn(v[4 * j + 3].x, v[4 * j + 3].y);
            reinterpret_cast<uint4*>(dst + c * 16)[j] = o;
          }
        }
      }
      if (some) {
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->tempty[buf]);
        ++nt;
      }
    }
  } else if (elect_one()) {
    // ---- products: four K = 16 MMAs a stage into the tile's accumulator
    constexpr uint32_t idesc = mma_idesc_bf16(kWM, kWN, true, true);
    uint32_t it = 0, nt = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const WTile w = wtile_at(p, t);
      const int steps = (w.hi - w.lo + kWRows - 1) / kWRows;
      if (steps == 0) continue;
      const uint32_t buf = nt & 1u;
      if (nt >= 2 && !bounded_wait(&tail->tempty[buf], ((nt >> 1) - 1) & 1u, failed)) break;
      for (int step = 0; step < steps; ++step, ++it) {
        const uint32_t st = it % kWStages;
        if (!bounded_wait(&tail->full[st], (it / kWStages) & 1u, failed)) {
          ok = false;
          break;
        }
        tcgen05_fence_after();
        const uint32_t sa = smem_addr(stages + size_t(st) * kWStage);
        const uint64_t da = smem_desc_sw128(sa, kLbo, 1024);
        const uint64_t db = smem_desc_sw128(sa + kWStageA, kLbo, 1024);
#pragma unroll
        for (int k = 0; k < kWRows / 16; ++k)
          mma_bf16(tmem + buf * kWN, da + ((k * 16 * 128) >> 4), db + ((k * 16 * 128) >> 4), idesc,
                   step > 0 || k > 0);
        mma_commit(&tail->empty[st]);
      }
      if (!ok) break;
      mma_commit(&tail->tfull[buf]);
      ++nt;
    }
    if (it >= 1) {  // the last products finish before TMEM is given back
      const uint32_t last = it - 1;
      uint32_t n = 0;
      while (!mbar_try_wait(&tail->empty[last % kWStages], (last / kWStages) & 1u) &&
             ++n < kSpinLimit) {
      }
    }
  }

  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == kConvWarps + 4) tmem_dealloc(tmem, 512);
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
  const int64_t tiles = int64_t(E) * (N / kWM) * ((K + kWN - 1) / kWN);
  if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const int grid = int(std::min<int64_t>(tiles, sm_count()));
  mp_k_expert_wgrad<<<grid, kWThreads, kWSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace mp
