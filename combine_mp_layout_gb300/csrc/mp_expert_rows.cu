// mp_expert_rows.cu -- products of the experts for few rows each (decoding): bf16
// rows with bf16 or MXFP4 weights.
//
// The weights' bytes are the whole cost, so the kernel is a stream of weights: a
// block takes 128 output channels of one expert and up to eight of its rows, a warp
// of its own keeps a ring of 16 KB pieces (128 channels x 128 bytes) full by TMA,
// and sixteen warps multiply from there with mma.m16n8k16 (the channels are the M
// side, the rows the N side): a warp 16 channels and one half of each piece's
// reduction.  A tensor-core tile of 256 x 32 would spend longer on its pipeline's
// start, and for 4-bit weights on writing the converted weights to shared memory.
// With few blocks, clusters share a reduction; sums are joined in a fixed order.
//
// bf16 weights: products exact, sums fp32.
//
// MXFP4 weights: one instruction turns two codes into f16, several fewer than bf16
// takes (83 against 34 codes per clock and SM with the products), so here the rows
// become f16 as well.  That is exact in all that matters: per row and 32 channels
// they are divided by a power of two that brings the largest into [2^15, 2^16), so
// values down to 2^-32 of it keep all their eight bits, and what is lost of smaller
// ones is at most 2^-40 of it; rows of very small values (below 2^-93) are divided
// by less, and lose nothing.  The products of 32 channels are summed by the tensor
// core, then multiplied by both powers of two and added up in fp32.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

constexpr int kVR = 8;                     // rows of a block: the MMA's columns
constexpr int kHalfWarps = kBC / 16;       // warps that cover the channels once
constexpr int kMulWarps = 2 * kHalfWarps;
constexpr int kThreads = (kMulWarps + 1) * 32;
constexpr int kPiece = kBC * 128;          // bytes of a piece of weights
constexpr int kMaxPieces = 8;              // in the ring
constexpr int kMaxVecParts = 8;            // blocks that share a reduction: one cluster

template <bool FP4>
struct Form {
  static constexpr int kSteps = FP4 ? 256 : 64;  // reduction steps of a piece
  // a row's bytes: eight rows' 16-byte reads fall into different banks
  static constexpr int kPad = FP4 ? 64 : 16;
};

struct VecArgs {
  int E, rows, N, K;
  int pieces;                    // of the ring
  int steps;                     // most reduction steps of a block, whole pieces
  const uint16_t* a;             // bf16 [rows][K]
  const unsigned char* scales;   // MXFP4: [E][N][K/32]
  int vec;                       // four scales are one aligned word
  RaggedArgs r;                  // for the tiles' prefix
};

struct VecTail {
  uint64_t raw[kMaxPieces], rawfree[kMaxPieces];
  alignas(16) float part[2][kVR][kBC];  // sums of the two halves: [row][channel]
  int failed;
  int scan[kThreads / 32];
};

template <bool FP4>
__host__ __device__ constexpr int row_stride(int steps) { return steps * 2 + Form<FP4>::kPad; }

template <bool FP4>
size_t vec_smem_bytes(int E, int steps, int pieces) {
  return size_t(pieces) * kPiece + size_t(kVR) * row_stride<FP4>(steps) +
         (FP4 ? size_t(steps / 32) * kVR * 4 : 0) + sizeof(VecTail) + size_t(E + 1) * 4;
}

template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight e2m1 codes as f16 pairs in order.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// The codes that the scale 2^(e - 127) takes past bf16's largest number (from 2^128)
// count as infinite, as they do where the weights become bf16.
__device__ __forceinline__ void overflow(uint32_t e, uint32_t (&o)[4]) {
  if (e < 253u || e == 255u) return;
  const uint32_t from = e == 254u ? 0x4000u : 0x4400u;  // 2 or 4 in f16
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((o[i] & 0x7fffu) >= from) o[i] = (o[i] & 0xffff8000u) | 0x7c00u;
    if (((o[i] >> 16) & 0x7fffu) >= from) o[i] = (o[i] & 0x8000ffffu) | 0x7c000000u;
  }
}

// 16 bytes of a row from reduction step k on, zeros past its end (K % 8 == 0).
__device__ __forceinline__ uint4 row16(const uint16_t* row, int k, int K) {
  return k < K ? __ldg(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
}

// The largest finite magnitude's bits of eight bf16 values, and that of `top`.
__device__ __forceinline__ uint32_t largest(uint32_t top, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) top = max(top, lo);
    if (hi < 0x7f80u) top = max(top, hi);
  }
  return top;
}

__device__ __forceinline__ uint4 to_f16(const uint4& v, float by) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(bf16_hi(w[i]) * by), "f"(bf16_lo(w[i]) * by));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The rows of a block into shared memory: for bf16 weights as they are, for MXFP4
// ones as f16 with a power of two per row and 32 channels (2^-10 of it is stored:
// a sum of products times that stays within fp32, and the scale it is multiplied by
// next gets the 2^10 back).
template <bool FP4>
__device__ __forceinline__ void stage_rows(const VecArgs& p, int row0, int nrows, int k0, int steps,
                                           unsigned char* xs, float* sx) {
  const int stride = row_stride<FP4>(p.steps);
  if constexpr (FP4) {
    const int groups = steps / 32;
    for (int i = threadIdx.x; i < nrows * groups; i += kMulWarps * 32) {
      const int r = i / groups, g = i - r * groups, k = k0 + g * 32;
      const uint16_t* src = p.a + int64_t(row0 + r) * p.K;
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = row16(src, k + 8 * j, p.K);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = largest(top, v[j]);
      const int ex = max(int(top >> 7) - 127 - 15, -109);
      const float by = __uint_as_float(uint32_t(127 - ex) << 23);
      uint4* dst = reinterpret_cast<uint4*>(xs + r * stride + g * 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[j] = to_f16(v[j], by);
      sx[g * kVR + r] = __uint_as_float(uint32_t(127 + ex - 10) << 23);
    }
  } else {
    const int vecs = steps / 8;
    for (int i = threadIdx.x; i < nrows * vecs; i += kMulWarps * 32) {
      const int r = i / vecs, k = (i - r * vecs) * 8;
      *reinterpret_cast<uint4*>(xs + r * stride + k * 2) =
          row16(p.a + int64_t(row0 + r) * p.K, k0 + k, p.K);
    }
  }
}

// This warp's half of a piece of bf16 weights: 32 steps.  Which reduction steps
// meet in an MMA is free as long as both operands agree: a lane's are one of the
// chunks of 16 bytes 2t and 2t + 1, which no two lanes read from the same banks.
__device__ __forceinline__ void multiply_bf16(const unsigned char* piece, const unsigned char* x,
                                              int half, int ch, int g, int t, float (&acc)[4]) {
  const unsigned char* w0 = piece + (ch + g) * 128;
  const int c = 2 * t + half;
  const uint4 lo = *reinterpret_cast<const uint4*>(w0 + ((c ^ g) << 4));
  const uint4 hi = *reinterpret_cast<const uint4*>(w0 + 8 * 128 + ((c ^ g) << 4));
  const uint4 b = *reinterpret_cast<const uint4*>(x + c * 16);
  mma_16x8x16<false>(acc, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma_16x8x16<false>(acc, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// This warp's half of a piece of MXFP4 weights: four groups of 32 steps.  s0, s1:
// the four scale bytes of channels g and g + 8.
template <bool LARGE>
__device__ __forceinline__ void multiply_fp4(const unsigned char* piece, const unsigned char* x,
                                             const float* sx, int half, int ch, int g, int t,
                                             uint32_t s0, uint32_t s1, float2 (&acc)[2]) {
  const unsigned char* w0 = piece + (ch + g) * 128 + t * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = half * 4 + i;
    uint32_t lo[4], hi[4];
    codes_to_f16(*reinterpret_cast<const uint32_t*>(w0 + ((c ^ g) << 4)), lo);
    codes_to_f16(*reinterpret_cast<const uint32_t*>(w0 + 8 * 128 + ((c ^ g) << 4)), hi);
    const uint32_t e0 = (s0 >> (8 * i)) & 255u, e1 = (s1 >> (8 * i)) & 255u;
    if constexpr (LARGE) {
      overflow(e0, lo);
      overflow(e1, hi);
    }
    const uint4 b = *reinterpret_cast<const uint4*>(x + c * 64 + t * 16);
    float2 sx2 = *reinterpret_cast<const float2*>(sx + c * kVR + 2 * t);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    mma_16x8x16<true>(v, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
    mma_16x8x16<true>(v, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
    float f0, f1;  // 2^(s - 127 + 10)
    if constexpr (LARGE) {  // some scale is past 2^117: without the 2^10
      sx2 = mul2(sx2, make_float2(1024.0f, 1024.0f));
      f0 = e0 == 0 ? 0x1p-127f : __uint_as_float(e0 == 255u ? 0x7fc00000u : e0 << 23);
      f1 = e1 == 0 ? 0x1p-127f : __uint_as_float(e1 == 255u ? 0x7fc00000u : e1 << 23);
    } else {
      f0 = __uint_as_float((e0 + 10u) << 23);
      f1 = __uint_as_float((e1 + 10u) << 23);
    }
    acc[0] = fma2(mul2(make_float2(v[0], v[1]), sx2), make_float2(f0, f0), acc[0]);
    acc[1] = fma2(mul2(make_float2(v[2], v[3]), sx2), make_float2(f1, f1), acc[1]);
  }
}

__device__ __forceinline__ void mul_warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kMulWarps * 32) : "memory");
}

// SPLIT: one unit (expert's rows, channels) per cluster, each block a part of the
// reduction; else blocks take units in turn.
template <bool FP4, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mp_k_expert_rows(const __grid_constant__ CUtensorMap map_w, const VecArgs p) {
  constexpr int kSteps = Form<FP4>::kSteps;
  extern __shared__ __align__(1024) unsigned char pieces[];
  unsigned char* xs = pieces + size_t(p.pieces) * kPiece;
  float* sx = reinterpret_cast<float*>(xs + kVR * row_stride<FP4>(p.steps));
  VecTail* tail = reinterpret_cast<VecTail*>(sx + (FP4 ? p.steps / 32 * kVR : 0));
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.pieces; ++i) {
      mbar_init(&tail->raw[i], 1);
      mbar_init(&tail->rawfree[i], kMulWarps);
    }
    tail->failed = 0;
    mbar_init_fence();
  }
  pdl_wait_prior_grid();  // (nothing of the above touches global memory)
  tile_prefix<kThreads, kVR>(p.r, pre, tail->scan);
  const int parts = SPLIT ? int(cluster_size()) : 1, part = SPLIT ? int(cluster_rank()) : 0;
  const int ncol = ceil_div(p.N, kBC);
  const int units = pre[p.E] * ncol;  // below 2^30: the launcher checks
  const int first = blockIdx.x / parts, stride = SPLIT ? max(units, 1) : int(gridDim.x);
  const int np = ceil_div(p.K, kSteps);
  const int lo = np * part / parts, hi = np * (part + 1) / parts;  // pieces of this block
  volatile int* failed = &tail->failed;

  if (warp == kMulWarps) {
    // ---- weights: one lane keeps the ring full
    if (elect_one()) {
      RingAt s;
      bool ok = true;
      for (int u = first; u < units && ok; u += stride) {
        const int e = expert_of(pre, p.E, ncol, u);
        const int ch = (u - pre[e] * ncol) / (pre[e + 1] - pre[e]) * kBC;
        for (int i = lo; i < hi; ++i, s.next(p.pieces)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->rawfree[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&tail->raw[s.slot], kPiece);
          tma_load_3d(pieces + s.slot * kPiece, &map_w, i * (FP4 ? 128 : kSteps), ch, e,
                      &tail->raw[s.slot]);
        }
      }
      // every load has landed and been used before the block may end
      for (int i = 0; i < p.pieces; ++i, s.next(p.pieces))
        if (s.round > 0) bounded_wait_idle(&tail->rawfree[s.slot], (s.round - 1) & 1u, failed);
    }
    __syncwarp();
    if constexpr (SPLIT) {
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    const int half = warp / kHalfWarps, ch = warp % kHalfWarps * 16;
    const int g = lane >> 2, t = lane & 3;
    const int groups = p.K / 32;
    RingAt s;
    bool ok = true;
    // (SPLIT: blocks without a unit meet the others at the cluster's barriers)
    for (int u = first; u < units || (SPLIT && u == first); u += stride) {
      const bool live = u < units;
      int e = 0, row0 = 0, nrows = 0, col0 = 0;
      if (live) {
        e = expert_of(pre, p.E, ncol, u);
        const int mt = pre[e + 1] - pre[e], local = u - pre[e] * ncol;
        int r0, r1;
        rows_of(p.r.expert_offsets, p.rows, e, r0, r1);
        col0 = local / mt * kBC;
        row0 = r0 + local % mt * kVR;
        nrows = min(kVR, r1 - row0);
        stage_rows<FP4>(p, row0, nrows, lo * kSteps, (hi - lo) * kSteps, xs, sx);
      }
      mul_warps_sync();
      if (live && ok) {
        const unsigned char* x = xs + g * row_stride<FP4>(p.steps);
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (FP4) {
          float2 acc2[2] = {};
          // (channels past the last one: codes are zeros, any scale will do)
          const unsigned char* sc0 =
              p.scales + (int64_t(e) * p.N + min(col0 + ch + g, p.N - 1)) * groups;
          const unsigned char* sc1 =
              p.scales + (int64_t(e) * p.N + min(col0 + ch + g + 8, p.N - 1)) * groups;
          auto scales4 = [&](const unsigned char* sc, int i) -> uint32_t {
            const int at = i * 8 + half * 4;
            if (p.vec) return __ldg(reinterpret_cast<const uint32_t*>(sc + min(at, groups - 4)));
            uint32_t v = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v |= uint32_t(__ldg(sc + min(at + j, groups - 1))) << (8 * j);
            return v;
          };
          // the scales of a piece, one piece ahead of their use
          uint32_t a0 = scales4(sc0, lo), a1 = scales4(sc1, lo);
          for (int i = lo; i < hi; ++i, s.next(p.pieces)) {
            const uint32_t s0 = a0, s1 = a1;
            if (i + 1 < hi) {
              a0 = scales4(sc0, i + 1);
              a1 = scales4(sc1, i + 1);
            }
            ok = bounded_wait_warp(&tail->raw[s.slot], s.round & 1u, failed);
            if (!ok) break;
            const unsigned char* piece = pieces + s.slot * kPiece;
            const unsigned char* xp = x + (i - lo) * kSteps * 2;
            const float* sp = sx + (i - lo) * (kSteps / 32) * kVR;
            const bool large = (__vcmpgtu4(s0, 0xf4f4f4f4u) | __vcmpgtu4(s1, 0xf4f4f4f4u)) != 0;
            if (__any_sync(kFull, large))
              multiply_fp4<true>(piece, xp, sp, half, ch, g, t, s0, s1, acc2);
            else
              multiply_fp4<false>(piece, xp, sp, half, ch, g, t, s0, s1, acc2);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail->rawfree[s.slot]);
          }
          acc[0] = acc2[0].x;
          acc[1] = acc2[0].y;
          acc[2] = acc2[1].x;
          acc[3] = acc2[1].y;
        } else {
          for (int i = lo; i < hi; ++i, s.next(p.pieces)) {
            ok = bounded_wait_warp(&tail->raw[s.slot], s.round & 1u, failed);
            if (!ok) break;
            multiply_bf16(pieces + s.slot * kPiece, x + (i - lo) * kSteps * 2, half, ch, g, t,
                          acc);
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail->rawfree[s.slot]);
          }
        }
        tail->part[half][2 * t][ch + g] = acc[0];
        tail->part[half][2 * t + 1][ch + g] = acc[1];
        tail->part[half][2 * t][ch + g + 8] = acc[2];
        tail->part[half][2 * t + 1][ch + g + 8] = acc[3];
      }
      if constexpr (SPLIT) cluster_sync_all(); else mul_warps_sync();
      // two channels of a row per thread; halves, then parts, in ascending order
      for (int i = part * kMulWarps * 32 + int(threadIdx.x); live && i < nrows * (kBC / 2);
           i += parts * kMulWarps * 32) {
        const int r = i / (kBC / 2), c = i % (kBC / 2) * 2;
        float2 sum = make_float2(0.0f, 0.0f);
        if constexpr (SPLIT) {
          for (int z = 0; z < parts; ++z)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 v;
              asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                           : "=f"(v.x), "=f"(v.y)
                           : "r"(map_to_rank(&tail->part[h][r][c], uint32_t(z)))
                           : "memory");
              sum = add2(sum, v);
            }
        } else {
          sum = add2(*reinterpret_cast<const float2*>(&tail->part[0][r][c]),
                     *reinterpret_cast<const float2*>(&tail->part[1][r][c]));
        }
        if (col0 + c < p.N)
          *reinterpret_cast<uint32_t*>(p.r.out + int64_t(row0 + r) * p.N + col0 + c) =
              pack_bf16x2_rn(sum.x, sum.y);
      }
      if constexpr (SPLIT) {
        cluster_sync_all();  // the other blocks have read this one's sums
        break;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && tail->failed) raise_error(p.r.dev_err, MP_ERR_TIMEOUT);
}

template <bool FP4, bool SPLIT>
cudaError_t launch_as(const VecArgs& p, const CUtensorMap& mw, int blocks, int parts,
                      cudaStream_t st) {
  static thread_local bool configured[64] = {};
  const cudaError_t e = allow_smem(mp_k_expert_rows<FP4, SPLIT>, configured);
  if (e != cudaSuccess) return e;
  return launch_waiting(mp_k_expert_rows<FP4, SPLIT>, dim3(unsigned(blocks)), dim3(kThreads),
                        vec_smem_bytes<FP4>(p.E, p.steps, p.pieces), st,
                        SPLIT ? unsigned(parts) : 0u, mw, p);
}

// cudaErrorNotSupported, with nothing launched, where this form is not meant for it.
template <bool FP4>
cudaError_t launch_rows(VecArgs p, const void* w, cudaStream_t st) {
  constexpr int kSteps = Form<FP4>::kSteps;
  const int64_t chunks = std::min<int64_t>(p.rows, int64_t(p.rows) / kVR + p.E);
  const int64_t units = chunks * ceil_div(p.N, kBC);
  const int np = ceil_div(p.K, kSteps);
  int parts = 1;
  while (parts < kMaxVecParts && units * 2 * parts <= sm_count() && np >= 4 * parts) parts *= 2;
  p.steps = ceil_div(np, parts) * kSteps;
  p.pieces = kMaxPieces;
  while (p.pieces > 2 && vec_smem_bytes<FP4>(p.E, p.steps, p.pieces) > size_t(kMaxBlockSmem))
    --p.pieces;
  if (units >= (int64_t(1) << 30) ||
      vec_smem_bytes<FP4>(p.E, p.steps, p.pieces) > size_t(kMaxBlockSmem))
    return cudaErrorNotSupported;
  CUtensorMap mw;
  const bool map_ok =
      FP4 ? make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(p.K) / 2,
                        uint64_t(p.N), uint64_t(p.E), 128, kBC)
          : make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, uint64_t(p.K),
                        uint64_t(p.N), uint64_t(p.E), kSteps, kBC);
  if (!map_ok) return cudaErrorInvalidValue;
  if (parts > 1) return launch_as<FP4, true>(p, mw, int(units) * parts, parts, st);
  return launch_as<FP4, false>(p, mw, int(std::min<int64_t>(units, sm_count())), 1, st);
}

}  // namespace

cudaError_t launch_expert_rows(int E, int rows, int N, int K, const void* a, const void* w,
                               const unsigned char* w_scales, const int32_t* expert_offsets,
                               void* out, int32_t* dev_err, cudaStream_t st) {
  VecArgs p = {};
  p.E = p.r.E = E;
  p.rows = p.r.rows = rows;
  p.N = N;
  p.K = K;
  p.a = static_cast<const uint16_t*>(a);
  p.scales = w_scales;
  p.vec = K % 128 == 0 && (reinterpret_cast<uintptr_t>(w_scales) & 3u) == 0;
  p.r.expert_offsets = expert_offsets;
  p.r.out = static_cast<uint16_t*>(out);
  p.r.dev_err = dev_err;
  return w_scales != nullptr ? launch_rows<true>(p, w, st) : launch_rows<false>(p, w, st);
}

}  // namespace mp
