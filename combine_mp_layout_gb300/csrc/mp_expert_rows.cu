// mp_expert_rows.cu -- products of the experts for few rows each (decoding): bf16
// rows with bf16 or MXFP4 weights.
//
// The weights' bytes are the whole cost, so the kernel is a stream of weights: a
// block takes 128 output channels of one expert and up to eight of its rows, a warp
// of its own keeps a ring of 16 KB pieces (128 channels x 128 bytes) full by TMA,
// and sixteen warps multiply from there with mma.m16n8k16 (the channels are the M
// side, the rows the N side): a warp 32 channels of a piece or half of one.  A tile of
// the tensor core's (256 x 32) would spend longer on its pipeline's start, and for
// 4-bit weights on writing the converted weights to shared memory.  With few blocks,
// clusters share a reduction; sums are joined in a fixed order: a block's own first, so
// that the first block of a cluster fetches one of each other block, all at once (eight
// MXFP4 rows 10.2 -> 9.3 us; every block fetching a share of all sums before).
//
// bf16 weights: products exact, sums fp32.
//
// MXFP4 weights: one instruction turns two codes into f16, several fewer than bf16
// takes (83 against 34 codes per clock and SM with the products), so here the rows
// become f16 as well: per row and 32 channels they are divided by a power of two that
// brings the largest into [2^15, 2^16), so values down to 2^-32 of it keep all their
// eight bits.  Where a row that a block takes has a value below that, the block's rows
// stay bf16 and the codes become bf16 too (WIDE): then the power of two leaves the
// largest at 2^101 at most, and only values below 2^-99 beside one of 2^100 or more can
// lose bits.  The products of 32 channels are summed by the tensor core, then multiplied
// by both powers of two and added up in fp32.
//
// Measured, 4096 x 7168: one bf16 row 13.3 us (4.4 TB/s of weights; 8.2 us with the
// weights in L2), one MXFP4 row 8.1; MXFP4 rows over 32 experts, one each 95 us (5.2 TB/s),
// two each 106 (59% of the issue slots; 70 us without the products), 61 drawn at random 88
// to 100 by how many experts have none.  (The look for values that f16 cannot hold is 1 to
// 2% of these.)
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mp_pair16.cuh"

namespace mp {

namespace {

constexpr int kVR = 8;                     // most rows of a block: the MMA's columns
// Warps take the pieces in sets.  A slot of the ring belongs to one set (the ring is a
// multiple of their number): a warp that met a slot after a piece of another set could
// find that piece still on its way, and its wait for the next one already over.  Four
// sets of four warps, a piece each, where the ring has eight pieces; with fewer, two
// sets whose warps share a piece (61 rows over 32 experts: 98 us with four sets, 102
// with two; where four pieces are all there are, 121 and 109).
constexpr int kChWarps = kBC / 32;         // warps that cover the channels: 32 each
constexpr int kMulWarps = 4 * kChWarps;
constexpr int kSums = 4;                   // sets times halves
constexpr int kThreads = (kMulWarps + 1) * 32;
constexpr int kPiece = kBC * 128;          // bytes of a piece of weights
constexpr int kScales = kBC * 16;          // and of its MXFP4 scales: 16 bytes per channel
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
  int room;                      // rows of a block that there is room for: 4 or 8
  int pieces;                    // of the ring: 8, 6, 4 or 2
  int steps;                     // most reduction steps of a block, whole pieces
  const uint16_t* a;             // bf16 [rows][K]
  const unsigned char* scales;   // MXFP4: [E][N][K/32]
  int tma_scales;                // these can be loaded by TMA
  RaggedArgs r;                  // for the tiles' prefix
};

struct VecTail {
  uint64_t raw[kMaxPieces], rawfree[kMaxPieces];
  alignas(16) float part[kSums][kVR][kBC];  // sums of set and half: [row][channel]
  int failed;
  int wide;                      // the first row of those that f16 cannot hold
  int scan[kThreads / 32];
};

template <bool FP4>
__host__ __device__ constexpr int row_stride(int steps) { return steps * 2 + Form<FP4>::kPad; }

template <bool FP4>
size_t vec_smem_bytes(int E, int room, int steps, int pieces) {
  return size_t(pieces) * (kPiece + (FP4 ? kScales : 0)) +
         size_t(room) * row_stride<FP4>(steps) +
         (FP4 ? size_t(steps / 32) * room * 4 : 0) + sizeof(VecTail) + size_t(E + 1) * 4;
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

// The same as bf16 pairs.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t (&o)[4]) {
  codes8(w, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], 0x7e807e80u);  // (2^126)
}

// The codes (f16, or bf16 where WIDE) that the scale 2^(e - 127) takes past bf16's
// largest number (from 2^128) count as infinite, as they do in the tiles' weights.
template <bool WIDE>
__device__ __forceinline__ void overflow(uint32_t e, uint32_t (&o)[4]) {
  if (e < 253u || e == 255u) return;
  constexpr uint32_t kInf = WIDE ? 0x7f80u : 0x7c00u;
  const uint32_t from = e == 254u ? 0x4000u : WIDE ? 0x4080u : 0x4400u;  // 2 or 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((o[i] & 0x7fffu) >= from) o[i] = (o[i] & 0xffff8000u) | kInf;
    if (((o[i] >> 16) & 0x7fffu) >= from) o[i] = (o[i] & 0x8000ffffu) | kInf << 16;
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

// The least magnitudes' bits but zero's, less one, of eight bf16 values and `least`, for
// even and odd values apart.
__device__ __forceinline__ uint32_t smallest2(uint32_t least, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n .reg .b32 t;\n add.u16x2 t, %1, %2;\n min.u16x2 %0, %0, t;\n}"
        : "+r"(least)
        : "r"(w[i] & 0x7fff7fffu), "r"(~0u));
  return least;
}

// Eight bf16 values times a power of two, as bf16 or f16.
__device__ __forceinline__ uint4 times_bf16(const uint4& v, float by) {
  return make_uint4(pack_bf16x2_rn(bf16_lo(v.x) * by, bf16_hi(v.x) * by),
                    pack_bf16x2_rn(bf16_lo(v.y) * by, bf16_hi(v.y) * by),
                    pack_bf16x2_rn(bf16_lo(v.z) * by, bf16_hi(v.z) * by),
                    pack_bf16x2_rn(bf16_lo(v.w) * by, bf16_hi(v.w) * by));
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
// ones as f16, or bf16 where WIDE, with a power of two per row and 32 channels (2^-10 of
// it is stored: a sum of products times that stays within fp32, and the scale it is
// multiplied by next gets the 2^10 back).  `wide` becomes row0 where f16 has lost bits.
template <bool FP4, bool WIDE>
__device__ __forceinline__ void stage_rows(const VecArgs& p, int row0, int nrows, int k0, int steps,
                                           unsigned char* xs, float* sx, volatile int* wide) {
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
      const int ex = max(int(top >> 7) - 127 - (WIDE ? 100 : 15), -109);
      const float by = __uint_as_float(uint32_t(127 - ex) << 23);
      uint4* dst = reinterpret_cast<uint4*>(xs + r * stride + g * 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[j] = WIDE ? times_bf16(v[j], by) : to_f16(v[j], by);
      if (!WIDE && ex > -109) {  // (at -109 the rows' least value is f16's least)
        uint32_t least = ~0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) least = smallest2(least, v[j]);
        if (min(least & 0xffffu, least >> 16) < (uint32_t(ex + 110) << 7) - 1u)
          *wide = row0;  // below 2^(ex - 17)
      }
      sx[g * p.room + r] = __uint_as_float(uint32_t(127 + ex - 10) << 23);
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

// A warp's 32 channels and half of a piece of bf16 weights.  Which reduction steps
// meet in an MMA is free as long as both operands agree: a lane's are one of the
// chunks of 16 bytes 2t and 2t + 1, which no two lanes read from the same banks.
__device__ __forceinline__ void multiply_bf16(const unsigned char* w0, const unsigned char* x,
                                              int half, int g, int t, float (&acc)[2][4]) {
  const int c = 2 * t + half;
  const uint4 b = *reinterpret_cast<const uint4*>(x + c * 16);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const unsigned char* wm = w0 + m * 16 * 128 + ((c ^ g) << 4);
    const uint4 lo = *reinterpret_cast<const uint4*>(wm);
    const uint4 hi = *reinterpret_cast<const uint4*>(wm + 8 * 128);
    mma_16x8x16<false>(acc[m], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma_16x8x16<false>(acc[m], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
  }
}

// Byte j of four scale bytes as the exponent of an fp32 number.
__device__ __forceinline__ float exponent_of(uint32_t s4, int j) {
  const uint32_t v = j == 3 ? s4 >> 1 : s4 << (23 - 8 * j);
  return __uint_as_float(v & 0x7f800000u);
}
// The same whatever the byte is (`more` is not in it): 2^(s - 127 + 10), or from 245
// on 2^(s - 127), and `by` the 2^10 that is put on the sum instead.
__device__ __forceinline__ float any_exponent_of(uint32_t s4, int j, float& by) {
  const uint32_t e = (s4 >> (8 * j)) & 255u;
  by = e > 244u ? 1024.0f : 1.0f;
  return __uint_as_float(e == 255u ? 0x7fc00000u : (e > 244u ? e : e + 10u) << 23);
}

// A warp's 32 channels and half of a piece of MXFP4 weights: four groups of 32
// steps, a lane 8 of them for channels g, g + 8, g + 16 and g + 24, whose scale
// bytes are s.  sx: the rows' powers of two, `room` for each group.
template <bool LARGE, bool WIDE>
__device__ __forceinline__ void multiply_fp4(const unsigned char* from, const unsigned char* x,
                                             const float* sx, int room, int half, int g, int t,
                                             const uint32_t (&s)[4], float (&acc)[2][4]) {
  from += t * 4;
  x += t * 16;
  // 2^10 more, which the rows' powers of two lack (below 192: no carry between bytes)
  const uint32_t more = LARGE ? 0u : 0x0a0a0a0au;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = half * 4 + i;
    const uint4 b = *reinterpret_cast<const uint4*>(x + c * 64);
    const float2 sx2 = *reinterpret_cast<const float2*>(sx + c * room);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const unsigned char* wm = from + m * 16 * 128 + ((c ^ g) << 4);
      const uint32_t e0 = s[2 * m] + more, e1 = s[2 * m + 1] + more;
      uint32_t lo[4], hi[4];
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wm);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wm + 8 * 128);
      if constexpr (WIDE) {
        codes_to_bf16(w0, lo);
        codes_to_bf16(w1, hi);
      } else {
        codes_to_f16(w0, lo);
        codes_to_f16(w1, hi);
      }
      if constexpr (LARGE) {
        overflow<WIDE>((e0 >> (8 * i)) & 255u, lo);
        overflow<WIDE>((e1 >> (8 * i)) & 255u, hi);
      }
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma_16x8x16<!WIDE>(v, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
      mma_16x8x16<!WIDE>(v, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
      float f0, f1;
      if constexpr (LARGE) {
        float by0, by1;
        f0 = any_exponent_of(e0, i, by0);
        f1 = any_exponent_of(e1, i, by1);
        v[0] *= by0;
        v[1] *= by0;
        v[2] *= by1;
        v[3] *= by1;
      } else {
        f0 = exponent_of(e0, i);
        f1 = exponent_of(e1, i);
      }
      const float2 v0 = mul2(make_float2(v[0], v[1]), sx2), v1 = mul2(make_float2(v[2], v[3]), sx2);
      acc[m][0] = fmaf(v0.x, f0, acc[m][0]);
      acc[m][1] = fmaf(v0.y, f0, acc[m][1]);
      acc[m][2] = fmaf(v1.x, f1, acc[m][2]);
      acc[m][3] = fmaf(v1.y, f1, acc[m][3]);
    }
  }
}

__device__ __forceinline__ void mul_warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kMulWarps * 32) : "memory");
}

// Unit u: four or eight rows (at most) of an expert by 128 channels, channels fastest.
struct Unit {
  int e, row0, nrows, col0;
};
__device__ __forceinline__ Unit unit_at(const VecArgs& p, const int* pre, int ncol, int u) {
  Unit n;
  n.e = expert_of(pre, p.E, ncol, u);
  const int local = u - pre[n.e] * ncol;
  int r0, r1;
  rows_of(p.r.expert_offsets, p.rows, n.e, r0, r1);
  n.row0 = r0 + local / ncol * p.room;
  n.nrows = min(p.room, r1 - n.row0);
  n.col0 = local % ncol * kBC;
  return n;
}

// MXFP4 scales that TMA cannot load: those of half of piece i, of a lane's four channels
// from c0 on, from where they are.
__device__ __forceinline__ void fetch_scales(const VecArgs& p, const Unit& n, int c0, int i,
                                             int half, uint32_t (&sc)[4]) {
  const int groups = p.K / 32;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    // (past the last channel or step: codes are zeros, any scale will do)
    const unsigned char* from =
        p.scales + (int64_t(n.e) * p.N + min(n.col0 + c0 + 8 * c, p.N - 1)) * groups;
    sc[c] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sc[c] |= uint32_t(__ldg(from + min(i * 8 + half * 4 + j, groups - 1))) << (8 * j);
  }
}

// Rows that f16 cannot hold: staged as bf16, and a warp's share of a unit's products.
// Functions of their own, called where they are needed: as a branch in the kernel's loop,
// or as a second loop beside it, they cost all other rows up to 7%, as calls 1 to 2%.
// (4096 x 7168, one row each over 32 experts: 217 us with such rows, 95 without; one row of
// one expert 14.6 and 8.9.)
__device__ __noinline__ void stage_wide(const VecArgs& p, const Unit n, int lo, int hi,
                                        unsigned char* xs, float* sx) {
  constexpr int kSteps = Form<true>::kSteps;
  stage_rows<true, true>(p, n.row0, n.nrows, lo * kSteps, (hi - lo) * kSteps, xs, sx, nullptr);
}

struct WideSums {
  float acc[8];
  RingAt s;
  bool ok;
};
template <int SETS>
__device__ __noinline__ WideSums wide_products(const VecArgs& p, const Unit n,
                                               const unsigned char* pieces, const unsigned char* x,
                                               const float* sx, VecTail* tail, int lo, int hi,
                                               RingAt s, bool ok) {
  constexpr int kSteps = Form<true>::kSteps;
  constexpr int kHalves = 4 / SETS, kSetWarps = kHalves * kChWarps;
  const unsigned char* scales = pieces + size_t(p.pieces) * kPiece;
  const int warp = warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int set = warp / kSetWarps, half0 = kHalves > 1 ? warp % kSetWarps / kChWarps : 0;
  const int ch = warp % kChWarps * 32;
  float acc[2][4] = {};
  for (int i = lo; i < hi; ++i, s.next(p.pieces)) {
    if (s.slot % SETS != set) continue;
    ok = ok && bounded_wait_warp(&tail->raw[s.slot], s.round & 1u, &tail->failed);
    if (!ok) break;
    const unsigned char* from = pieces + s.slot * kPiece + (ch + g) * 128;
    const float* sp = sx + (i - lo) * (kSteps / 32) * p.room + ((2 * t) & (p.room - 1));
#pragma unroll 1
    for (int half = half0; half < 2; half += kHalves) {
      uint32_t sc[4];
      if (p.tma_scales) {
        const unsigned char* at =
            scales + s.slot * kScales + (ch + g) * 16 + (i & 1) * 8 + half * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[c] = *reinterpret_cast<const uint32_t*>(at + c * 8 * 16);
      } else {
        fetch_scales(p, n, ch + g, i, half, sc);
      }
      multiply_fp4<true, true>(from, x + (i - lo) * kSteps * 2, sp, p.room, half, g, t, sc, acc);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&tail->rawfree[s.slot]);
  }
  WideSums r;
#pragma unroll
  for (int m = 0; m < 8; ++m) r.acc[m] = acc[m / 4][m % 4];
  r.s = s;
  r.ok = ok;
  return r;
}

// SPLIT: one unit per cluster, each block a part of the reduction; else each block
// takes a run of units, so that it seldom has other rows to fetch.
template <bool FP4, bool SPLIT, int SETS>
__global__ void __launch_bounds__(kThreads, 1)
mp_k_expert_rows(const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_s, const __grid_constant__ VecArgs p) {
  constexpr int kSteps = Form<FP4>::kSteps;
  constexpr int kHalves = 4 / SETS;  // of a piece's reduction that go to other warps
  constexpr int kSetWarps = kHalves * kChWarps;
  extern __shared__ __align__(1024) unsigned char pieces[];
  unsigned char* scales = pieces + size_t(p.pieces) * kPiece;
  unsigned char* xs = scales + (FP4 ? size_t(p.pieces) * kScales : 0);
  float* sx = reinterpret_cast<float*>(xs + p.room * row_stride<FP4>(p.steps));
  VecTail* tail = reinterpret_cast<VecTail*>(sx + (FP4 ? p.steps / 32 * p.room : 0));
  int* pre = reinterpret_cast<int*>(tail + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.pieces; ++i) {
      mbar_init(&tail->raw[i], 1);
      mbar_init(&tail->rawfree[i], kSetWarps);
    }
    tail->failed = 0;
    tail->wide = -1;
    mbar_init_fence();
  }
  pdl_wait_prior_grid();  // (nothing of the above touches global memory)
  tile_prefix<kThreads>(p.r, p.room, pre, tail->scan);
  const int parts = SPLIT ? int(cluster_size()) : 1, part = SPLIT ? int(cluster_rank()) : 0;
  const int ncol = ceil_div(p.N, kBC);
  const int units = pre[p.E] * ncol;  // below 2^30: the launcher checks
  const int64_t blocks = gridDim.x / parts, block = blockIdx.x / parts;
  const int first = SPLIT ? int(block) : int(units * block / blocks);
  const int last = SPLIT ? min(first + 1, units) : int(units * (block + 1) / blocks);
  const int np = ceil_div(p.K, kSteps);
  const int lo = np * part / parts, hi = np * (part + 1) / parts;  // pieces of this block
  volatile int* failed = &tail->failed;

  if (warp == kMulWarps) {
    // ---- weights: one lane keeps the ring full
    if (elect_one()) {
      RingAt s;
      bool ok = true;
      for (int u = first; u < last && ok; ++u) {
        const Unit n = unit_at(p, pre, ncol, u);
        for (int i = lo; i < hi; ++i, s.next(p.pieces)) {
          if (s.round > 0 &&
              !bounded_wait_idle(&tail->rawfree[s.slot], (s.round - 1) & 1u, failed)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&tail->raw[s.slot],
                                kPiece + (FP4 && p.tma_scales ? kScales : 0));
          tma_load_3d(pieces + s.slot * kPiece, &map_w, i * (FP4 ? 128 : kSteps), n.col0, n.e,
                      &tail->raw[s.slot]);
          if (FP4 && p.tma_scales)  // (x in whole 16 bytes: two pieces' scales)
            tma_load_3d(scales + s.slot * kScales, &map_s, i * 8 & ~15, n.col0, n.e,
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
    const int set = warp / kSetWarps, half0 = kHalves > 1 ? warp % kSetWarps / kChWarps : 0;
    const int ch = warp % kChWarps * 32;
    const int g = lane >> 2, t = lane & 3;
    RingAt s;
    bool ok = true;
    Unit n = {};
    if (first < last) n = unit_at(p, pre, ncol, first);
    int staged = -1;  // the first row of those in shared memory
    // (SPLIT: blocks without a unit meet the others at the cluster's barriers)
    for (int u = first; u < last || (SPLIT && u == first); ++u) {
      const bool live = u < last;
      const bool fresh = live && staged != n.row0;
      if (fresh) {
        stage_rows<FP4, false>(p, n.row0, n.nrows, lo * kSteps, (hi - lo) * kSteps, xs, sx,
                               &tail->wide);
        staged = n.row0;
      }
      mul_warps_sync();  // the rows are there, and the sums of the unit before are used up
      const bool wide = FP4 && live && *static_cast<volatile const int*>(&tail->wide) == n.row0;
      if (wide && fresh) {
        stage_wide(p, n, lo, hi, xs, sx);
        mul_warps_sync();
      }
      if (live) {
        const unsigned char* x = xs + (g & (p.room - 1)) * row_stride<FP4>(p.steps);
        float acc[2][4] = {};
        if (wide) {
          const WideSums ws = wide_products<SETS>(p, n, pieces, x, sx, tail, lo, hi, s, ok);
#pragma unroll
          for (int m = 0; m < 8; ++m) acc[m / 4][m % 4] = ws.acc[m];
          s = ws.s;
          ok = ws.ok;
        }
        for (int i = wide ? hi : lo; i < hi; ++i, s.next(p.pieces)) {
          if (s.slot % SETS != set) continue;
          // (scales that are fetched are on their way during the wait)
          uint32_t sc[2 / kHalves][4];
#pragma unroll
          for (int h = 0; h < 2 / kHalves; ++h)
            if (FP4 && !p.tma_scales) fetch_scales(p, n, ch + g, i, half0 + h, sc[h]);
          ok = ok && bounded_wait_warp(&tail->raw[s.slot], s.round & 1u, failed);
          if (!ok) break;
          const unsigned char* w0 = pieces + s.slot * kPiece + (ch + g) * 128;
          const unsigned char* xp = x + (i - lo) * kSteps * 2;
          if constexpr (FP4) {
            const float* sp = sx + (i - lo) * (kSteps / 32) * p.room + ((2 * t) & (p.room - 1));
            uint32_t large = 0;  // scales from 2^65 on (192): the careful form
#pragma unroll
            for (int h = 0; h < 2 / kHalves; ++h) {
              if (p.tma_scales) {
                const unsigned char* from = scales + s.slot * kScales + (ch + g) * 16 +
                                            (i & 1) * 8 + (half0 + h) * 4;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  sc[h][c] = *reinterpret_cast<const uint32_t*>(from + c * 8 * 16);
              }
#pragma unroll
              for (int c = 0; c < 4; ++c) large |= sc[h][c] & (sc[h][c] << 1);
            }
            if (__any_sync(kFull, (large & 0x80808080u) != 0)) {
#pragma unroll
              for (int h = 0; h < 2 / kHalves; ++h)
                multiply_fp4<true, false>(w0, xp, sp, p.room, half0 + h, g, t, sc[h], acc);
            } else {
#pragma unroll
              for (int h = 0; h < 2 / kHalves; ++h)
                multiply_fp4<false, false>(w0, xp, sp, p.room, half0 + h, g, t, sc[h], acc);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2 / kHalves; ++h) multiply_bf16(w0, xp, half0 + h, g, t, acc);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->rawfree[s.slot]);
        }
        const int sum = set * kHalves + half0;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          tail->part[sum][2 * t][ch + m * 16 + g] = acc[m][0];
          tail->part[sum][2 * t + 1][ch + m * 16 + g] = acc[m][1];
          tail->part[sum][2 * t][ch + m * 16 + g + 8] = acc[m][2];
          tail->part[sum][2 * t + 1][ch + m * 16 + g + 8] = acc[m][3];
        }
      }
      mul_warps_sync();
      // two channels of a row per thread: sets and halves in ascending order, then parts
      static_assert(kMulWarps * 32 == kVR * (kBC / 2));
      const int r = int(threadIdx.x) / (kBC / 2), c = int(threadIdx.x) % (kBC / 2) * 2;
      const bool mine = live && r < n.nrows;
      float2 sum = make_float2(0.0f, 0.0f);
      if (mine) {
#pragma unroll
        for (int h = 0; h < kSums; ++h)
          sum = add2(sum, *reinterpret_cast<const float2*>(&tail->part[h][r][c]));
      }
      if constexpr (SPLIT) {
        // the first block adds up the parts, all on their way before the first is needed
        if (mine) *reinterpret_cast<float2*>(&tail->part[0][r][c]) = sum;
        cluster_sync_all();
        if (mine && part == 0) {
          float2 v[kMaxVecParts];
#pragma unroll
          for (int z = 1; z < kMaxVecParts; ++z)
            if (z < parts)
              asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                           : "=f"(v[z].x), "=f"(v[z].y)
                           : "r"(map_to_rank(&tail->part[0][r][c], uint32_t(z)))
                           : "memory");
#pragma unroll
          for (int z = 1; z < kMaxVecParts; ++z)
            if (z < parts) sum = add2(sum, v[z]);
        }
      }
      if (mine && part == 0 && n.col0 + c < p.N)
        *reinterpret_cast<uint32_t*>(p.r.out + int64_t(n.row0 + r) * p.N + n.col0 + c) =
            pack_bf16x2_rn(sum.x, sum.y);
      if (u + 1 < last) n = unit_at(p, pre, ncol, u + 1);
      if constexpr (SPLIT) {
        cluster_sync_all();  // the other blocks have read this one's sums
        break;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && tail->failed) raise_error(p.r.dev_err, MP_ERR_TIMEOUT);
}

template <bool FP4, bool SPLIT, int SETS>
cudaError_t launch_as(const VecArgs& p, const CUtensorMap& mw, const CUtensorMap& ms, int blocks,
                      int parts, cudaStream_t st) {
  static thread_local bool configured[64] = {};
  const cudaError_t e = allow_smem(mp_k_expert_rows<FP4, SPLIT, SETS>, configured);
  if (e != cudaSuccess) return e;
  return launch_waiting(mp_k_expert_rows<FP4, SPLIT, SETS>, dim3(unsigned(blocks)), dim3(kThreads),
                        vec_smem_bytes<FP4>(p.E, p.room, p.steps, p.pieces), st,
                        SPLIT ? unsigned(parts) : 0u, mw, ms, p);
}

// cudaErrorNotSupported, with nothing launched, where this form is not meant for it.
template <bool FP4>
cudaError_t launch_rows(VecArgs p, const void* w, cudaStream_t st) {
  constexpr int kSteps = Form<FP4>::kSteps;
  static thread_local bool configured[64] = {};
  const cudaError_t e = allow_smem(mp_k_expert_rows<FP4, true, 4>, configured);
  if (e != cudaSuccess) return e;
  // Room for four rows while the experts have two on average: the rows' place is the
  // ring's (7168 steps: eight pieces instead of four).
  p.room = p.rows <= 4 || p.rows / 2 < p.E ? 4 : kVR;
  const int64_t units = most_row_tiles(p.E, p.rows, p.room) * ceil_div(p.N, kBC);
  const int np = ceil_div(p.K, kSteps);
  const int parts =
      parts_for(mp_k_expert_rows<FP4, true, 4>, kThreads, units, 1, kMaxVecParts, np, 2);
  p.steps = ceil_div(np, parts) * kSteps;
  if (p.steps > (1 << 16)) return cudaErrorNotSupported;  // (no room for the rows)
  p.pieces = kMaxPieces;
  while (p.pieces > 2 &&
         vec_smem_bytes<FP4>(p.E, p.room, p.steps, p.pieces) > size_t(kMaxBlockSmem))
    p.pieces -= 2;
  if (units >= (int64_t(1) << 30) ||
      vec_smem_bytes<FP4>(p.E, p.room, p.steps, p.pieces) > size_t(kMaxBlockSmem))
    return cudaErrorNotSupported;
  CUtensorMap mw, ms = {};
  const bool map_ok =
      FP4 ? make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(p.K) / 2,
                        uint64_t(p.N), uint64_t(p.E), 128, kBC)
          : make_map_3d(&mw, w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, uint64_t(p.K),
                        uint64_t(p.N), uint64_t(p.E), kSteps, kBC);
  if (!map_ok) return cudaErrorInvalidValue;
  if (p.tma_scales &&
      !make_map_3d(&ms, p.scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(p.K) / 32,
                   uint64_t(p.N), uint64_t(p.E), 16, kBC, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const bool four = p.pieces == kMaxPieces;
  if (parts > 1)
    return four ? launch_as<FP4, true, 4>(p, mw, ms, int(units) * parts, parts, st)
                : launch_as<FP4, true, 2>(p, mw, ms, int(units) * parts, parts, st);
  const int blocks = int(std::min<int64_t>(units, sm_count()));
  return four ? launch_as<FP4, false, 4>(p, mw, ms, blocks, 1, st)
              : launch_as<FP4, false, 2>(p, mw, ms, blocks, 1, st);
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
  // TMA wants rows of whole 16 bytes, and a base aligned to them
  p.tma_scales =
      w_scales != nullptr && K % 512 == 0 && (reinterpret_cast<uintptr_t>(w_scales) & 15u) == 0;
  p.r.expert_offsets = expert_offsets;
  p.r.out = static_cast<uint16_t*>(out);
  p.r.dev_err = dev_err;
  return w_scales != nullptr ? launch_rows<true>(p, w, st) : launch_rows<false>(p, w, st);
}

}  // namespace mp
