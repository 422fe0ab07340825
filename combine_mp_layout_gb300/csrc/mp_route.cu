// mp_route.cu -- the router: scores, top-K experts, weights, per-expert counts
// and the balance loss in one pass over the logits, and the gradient of the
// weights and the loss with respect to the logits.
//
// Per token, over the experts e whose logit is not -inf:
//   score  s_e = softmax(l)_e  or  1 / (1 + exp(-l_e))
//   key        = l_e (softmax), s_e + bias_e (sigmoid): the K largest keys are
//                chosen, ties going to the lower expert
//   weight w_k = scale * s_k, or scale * s_k / sum of the chosen s
//   share  p_e = s_e / sum of all s
// Per source rank, T its tokens with a chosen expert, c_e its counts:
//   loss = coef * E / (K * T^2) * sum_e c_e * sum_t p_{t,e}
//
// A warp (up to 1,024 experts) or a block of eight warps (beyond) holds one
// token's logits in registers, V per thread, so they are read once.
//
// Measured at 8 x 4,096 tokens, 256 experts, top-8, sigmoid: forward 31.6 us, gradient
// 25.6 us (10 and 14 us of memory traffic are in them at most); 8 tokens of 64 experts
// 5.3 us; with a block per token, 2,048, 4,096 and 8,192 experts, forward 510, 673 and
// 1,585 us, gradient 308, 419 and 1,099 us.  The forward pass is bound by
// instructions, about 770 per token and warp (71% of the issue slots taken):
// exponential and reciprocal of every score, the candidates' compares and ballots;
// about 8 us are launch, block sums and the ranks' ends.
//
// The sums over tokens are order-free and so the same on every run: counts are
// integers, and each block's share sums (fp32, added in a fixed order) enter
// the global sums as fixed-point integers with as many fraction bits as 2^63 /
// (N + 1) leaves.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "../../include/mp_layout.h"
#include "mp_common.cuh"
#include "mp_internal.h"

namespace mp {

namespace {

constexpr int kRouteWarps = 8;
constexpr int kRouteThreads = kRouteWarps * kWarp;
// Up to how many choices candidates are tried first.  8 x 4,096 tokens of 256
// experts, both ways side by side: 8 choices 34 us against 44 us by rounds, 16 38 and
// 55, 20 50 and 60, but 32 choices 87 and 76 us (nearly all lanes' largest count, and
// more than 32 keys reach the least of them).  Later steps shortened what both share:
// 8 choices take 31.6 us now.
constexpr int kCandidateTopk = 20;

struct RouteArgs {
  int R, N, K, E;
  int normalize;
  float scale, loss_coef;
  const void* logits;
  const float* bias;        // or NULL
  const uint8_t* active;    // or NULL
  int32_t* topk_idx;
  float* topk_weights;
  int32_t* counts;          // [R][E]
  int32_t* routed;          // [R]
  float* loss;              // [R]
  int32_t* dev_err;
  // workspace: done counters and routed sums [MP_MAX_RANKS], then [R][E] sums and counts
  uint32_t* ws_done;
  int32_t* ws_routed;
  unsigned long long* ws_mass;
  int32_t* ws_count;
  float fix;                // 2^fraction bits of ws_mass
  // gradient
  const float* d_weights;   // [R][N][K] or NULL
  const float* d_loss;      // [R] or NULL
  void* d_logits;
};

// Reductions over the W warps that share a token; every thread gets the result.
// `red` holds kRouteWarps words (unused for W = 1).
template <int W, typename T, typename Op>
__device__ __forceinline__ T team_reduce(T v, T* red, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(kFull, v, o));
  if constexpr (W > 1) {
    __syncthreads();  // the words of the reduction before are free
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = op(v, red[w]);
  }
  return v;
}
struct OpSum {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct OpMax {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
template <int W>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(kFull, v);
  if constexpr (W > 1) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = max(v, red[w]);
  }
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t team_min(uint32_t v, uint32_t* red) {
  return ~team_max<W>(~v, red);
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Exchanges of a sorting network: the larger key (with its 4-bit tag) to place a.
__device__ __forceinline__ void order2(uint32_t& ka, uint32_t& ta, uint32_t& kb, uint32_t& tb) {
  const bool swap = kb > ka;  // equal keys stay: they are in order of their tags
  const uint32_t k0 = max(ka, kb), k1 = min(ka, kb);
  const uint32_t t0 = swap ? tb : ta, t1 = swap ? ta : tb;
  ka = k0;
  kb = k1;
  ta = t0;
  tb = t1;
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  if constexpr (std::is_same<T, float>::value)
    return __ldg(p);
  else
    return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p))) << 16);
}

template <typename T>
__device__ __forceinline__ void store_grad(T* p, float v) {
  if constexpr (std::is_same<T, float>::value)
    *p = v;
  else
    *p = __float2bfloat16_rn(v);
}

// 1 / (1 + exp(-x)), with a correctly rounded reciprocal: it is part of the
// selection key, so its last bit can decide.
__device__ __forceinline__ float sigmoid_exact(float x) { return __frcp_rn(1.0f + expf(-x)); }
// The same without the reciprocal's branch for extreme exponents, for 1 <= y <
// 2^126: an approximation within an ulp and one correction with the exact
// remainder give the correctly rounded reciprocal (Markstein, "IA-64 and
// Elementary Functions"; compared with __frcp_rn for every float of that range).
__device__ __forceinline__ float rcp_mid(float y) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(y));
  return __fmaf_rn(r, __fmaf_rn(-y, r, 1.0f), r);
}

// Floats to integers with the same order (-0 and +0 alike); 0 means "cannot be chosen".
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A token's logits and scores, V experts per thread: expert j * (W * 32) + t.
template <typename T, int V, int W, bool SIG>
struct TokenScores {
  float s[V];   // scores, 0 where the expert is not allowed
  float inv;    // share = s * inv
  bool live;    // finite or -inf everywhere, and active
  float m, inv_total;  // softmax: s = exp(l - m) * inv_total

  // the score of one more logit of the same token
  __device__ __forceinline__ float score_of(float x) const {
    if constexpr (SIG) return x > -INFINITY ? sigmoid_exact(x) : 0.0f;
    return x > -INFINITY ? expf(x - m) * inv_total : 0.0f;
  }

  // x: the token's logits, -inf past the last expert.  LEFT_OUT: the caller leaves a
  // token out that is not live; its scores are not to be used.
  template <bool LEFT_OUT>
  __device__ __forceinline__ void compute(float (&x)[V], bool active, float* red) {
    bool bad = false;
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      bad |= !(x[j] < INFINITY);  // NaN or +inf
      mx = fmaxf(mx, x[j]);
    }
    if (SIG && W == 1) {
      bad = __any_sync(kFull, bad);
      live = active && !bad;
      m = 0.0f;
    } else {
      // one reduction for both: a bad value makes the maximum +inf
      mx = bad ? INFINITY : mx;
      if constexpr (W == 1)
        mx = warp_max(mx);
      else
        mx = team_reduce<W>(mx, red, OpMax());
      live = active && mx < INFINITY;
      m = mx > -INFINITY ? mx : 0.0f;
    }
    float total = 0.0f;
    if constexpr (SIG) {
      bool far = false;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!LEFT_OUT && !live) x[j] = -INFINITY;
        const float y = 1.0f + expf(-x[j]);  // +inf: the score is 0
        s[j] = y < 0x1p126f ? rcp_mid(y) : 0.0f;
        far |= y >= 0x1p126f && y < INFINITY;
      }
      if (far) {  // logits below about -87
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = x[j] > -INFINITY ? sigmoid_exact(x[j]) : 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!LEFT_OUT && !live) x[j] = -INFINITY;
        s[j] = x[j] > -INFINITY ? expf(x[j] - m) : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) total += s[j];
    total = team_reduce<W>(total, red, OpSum());
    inv_total = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
    inv = SIG ? inv_total : 1.0f;
    if constexpr (!SIG) {
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] *= inv_total;
    }
  }
};

template <typename T, int V, int W>
__device__ __forceinline__ void load_token(const T* row, int E, int t, float (&x)[V]) {
  if (E == V * W * kWarp) {  // (no comparison per logit then)
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = load_logit(row + j * (W * kWarp) + t);
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * (W * kWarp) + t;
    x[j] = e < E ? load_logit(row + e) : -INFINITY;
  }
}

// Choosing the K largest keys, among equal ones the lowest expert.  A key of -inf
// is never chosen; the choices are fewer than K if there are no more.
//
// A warp per token.  The K-th of the lanes' largest keys is no larger than the K-th
// of all keys, so the choices are among those that reach it, a few more than K when
// few lanes hold two of them.  Each of these goes to a lane, in the experts' order,
// and counts those before it.  A choice is an expert and its score.  Returns the
// number of choices, or -1 if there are more than 32 candidates.
template <int V>
__device__ __forceinline__ int choose_candidates(const float (&key)[V],
                                                 const float (&score)[V], int K, int lane,
                                                 float* sm_key, int2* sm_choice, int2* chosen) {
  float m = key[0];
#pragma unroll
  for (int j = 1; j < V; ++j) m = fmaxf(m, key[j]);
  float least = -INFINITY;
  for (int k = 0; k < K; ++k) {  // (equal ones leave together: the bound is lower then)
    least = warp_max(m);
    m = m == least ? -INFINITY : m;
  }
  least = fmaxf(least, -FLT_MAX);  // -inf is no candidate
  sm_key[lane] = -INFINITY;
  __syncwarp();
  const unsigned below = (1u << lane) - 1u;
  int c = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool in = key[j] >= least;
    const unsigned b = __ballot_sync(kFull, in);
    const int at = c + __popc(b & below);
    if (in && at < kWarp) {
      sm_key[at] = key[j];
      sm_choice[at] = make_int2(j * kWarp + lane, __float_as_int(score[j]));
    }
    c += __popc(b);
  }
  __syncwarp();
  if (c > kWarp) return -1;
  const float k = sm_key[lane];
  int place = 0;
  for (int q = 0; q < c; q += 4) {  // (keys past c are -inf)
    const float4 o = *reinterpret_cast<const float4*>(sm_key + q);
    place += int(o.x > k) + int(o.y > k) + int(o.z > k) + int(o.w > k);
  }
  const unsigned taken = __reduce_or_sync(kFull, lane < c ? 1u << place : 0u);
  if (__popc(taken) != c) {  // equal keys share a place: the lower expert first
    for (int q = 0; q < c; ++q) place += int(q < lane && sm_key[q] == k);
  }
  if (lane < c && place < K) chosen[place] = sm_choice[lane];
  return min(c, K);
}

// The largest of a team's keys that are left (0: none), searched again in the lane
// that lost one.
template <int V, int W>
struct Searched {
  uint32_t (&key)[V];
  const int t;
  uint32_t best = 0;
  int bestj = 0;
  __device__ __forceinline__ Searched(uint32_t (&k)[V], int thread) : key(k), t(thread) {
    search(-1);
  }
  __device__ __forceinline__ void search(int gone) {
    best = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j == gone) key[j] = 0;
      if (key[j] > best) { best = key[j]; bestj = j; }
    }
  }
  // the expert, or -1; the same in every thread
  __device__ __forceinline__ int next(uint32_t* red) {
    const uint32_t top = team_max<W>(best, red);
    if (top == 0) return -1;
    const uint32_t own = uint32_t(bestj * (W * kWarp) + t);
    const uint32_t e = team_min<W>(best == top ? own : 0xffffffffu, red);
    if (best == top && own == e) search(bestj);
    return int(e);
  }
};

// A warp per token, in K rounds: for any K and any ties.  The experts alone.
template <int V>
__device__ __forceinline__ int choose_rounds(const float (&value)[V], int K, int lane,
                                             int2* chosen) {
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = value[j] > -INFINITY ? order_key(value[j]) : 0u;
  int k = 0;
  if constexpr (V <= 8) {
    // Each lane sorts its keys once (odd-even transposition: neighbours only, so
    // equal keys keep their order), then K rounds take the largest head.  Against
    // searching each lane's keys again in every round this is fewer instructions.
    uint32_t tag[V];
#pragma unroll
    for (int j = 0; j < V; ++j) tag[j] = j;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = i & 1; j + 1 < V; j += 2) order2(key[j], tag[j], key[j + 1], tag[j + 1]);
    uint32_t tags = 0;  // 4 bits each, the head's lowest
#pragma unroll
    for (int j = 0; j < V; ++j) tags |= tag[j] << (4 * j);
    for (; k < K; ++k) {
      const uint32_t top = __reduce_max_sync(kFull, key[0]);
      if (top == 0) break;
      bool won = key[0] == top;
      const uint32_t e = (tags & 15u) * kWarp + lane;
      const unsigned heads = __ballot_sync(kFull, won);
      if (heads & (heads - 1)) {  // (the whole warp is here: the ballot is the same for all)
        const uint32_t lowest = __reduce_min_sync(kFull, won ? e : 0xffffffffu);
        won = won && e == lowest;
      }
      if (won) chosen[k].x = int(e);
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) key[j] = won ? key[j + 1] : key[j];
      key[V - 1] = won ? 0u : key[V - 1];
      tags = won ? tags >> 4 : tags;
    }
  } else {
    Searched<V, 1> rest(key, lane);
    for (; k < K; ++k) {
      const int e = rest.next(nullptr);
      if (e < 0) break;
      if (lane == 0) chosen[k].x = e;
    }
  }
  return k;
}

// A block per token: thread k of the first warp gets the k-th choice.
template <int V, int W>
__device__ __forceinline__ bool choose_in_block(const float (&value)[V], int K, int t,
                                                uint32_t* red, int& mine) {
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = value[j] > -INFINITY ? order_key(value[j]) : 0u;
  Searched<V, W> rest(key, t);
  int k = 0;
  for (; k < K; ++k) {
    const int e = rest.next(red);
    if (e < 0) break;
    if (t == k) mine = e;
  }
  return k > 0;
}

// Blocks per SM that the registers are to allow.  With a warp per token of 1,024
// experts two blocks and a few spilled registers (forward 96 us for 8 x 4,096 tokens,
// top-8, sigmoid, gradient 87 us) beat one block without (147 and 144 us); with up to
// 256 experts four (80 registers and three blocks: forward 39 us against 31).
constexpr int route_blocks(int V, int W) { return V <= 8 ? 4 : V == 16 || W == 1 ? 2 : 1; }

// grid (blocks per rank, R).  W = 1: a warp per token; W = 8: a block per token.
template <typename T, int V, int W, bool SIG>
__global__ void __launch_bounds__(kRouteThreads, route_blocks(V, W))
mp_k_route(const RouteArgs p) {
  constexpr int kTeam = W * kWarp;
  constexpr int kTeams = kRouteWarps / W;
  extern __shared__ int sm_count_[];  // [E] counts
  __shared__ float red[kRouteWarps];
  __shared__ uint32_t redu[kRouteWarps];
  __shared__ float stage[W == 1 ? kRouteWarps * 256 : 1];
  __shared__ int2 sm_chosen[W == 1 ? kRouteWarps : 1][MP_MAX_TOPK];
  __shared__ __align__(16) float sm_key[W == 1 ? kRouteWarps : 1][kWarp];
  __shared__ int2 sm_choice[W == 1 ? kRouteWarps : 1][kWarp];
  __shared__ float sm_bias[W == 1 && SIG ? V * kWarp : 1];
  __shared__ int s_routed;
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % kTeam;   // thread within the token's team
  const int team = threadIdx.x / kTeam;
  const int rank = blockIdx.y;
  const int E = p.E, K = p.K;
  pdl_wait_prior_grid();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) sm_count_[e] = 0;
  if constexpr (W == 1 && SIG) {
    for (int e = threadIdx.x; e < V * kWarp; e += kRouteThreads)
      sm_bias[e] = p.bias != nullptr && e < E ? __ldg(p.bias + e) : 0.0f;
  }
  if (threadIdx.x == 0) s_routed = 0;
  __syncthreads();

  float mass[V];  // this thread's experts: sum of shares over the team's tokens
#pragma unroll
  for (int j = 0; j < V; ++j) mass[j] = 0.0f;
  int routed = 0;

  // (unsigned: the index after the last token may lie past 2^31)
  for (uint32_t n = blockIdx.x * kTeams + team; n < uint32_t(p.N); n += gridDim.x * kTeams) {
    const int64_t tok = int64_t(rank) * p.N + n;
    const T* row = static_cast<const T*>(p.logits) + tok * E;
    float x[V];
    load_token<T, V, W>(row, E, t, x);
    TokenScores<T, V, W, SIG> sc;
    const bool active = p.active == nullptr || p.active[tok] != 0;
    sc.template compute<W == 1>(x, active, red);
    if (active && !sc.live && t == 0) raise_error(p.dev_err, MP_ERR_BAD_VALUE);
    if (W == 1 && !sc.live) {
      if (lane < K) {
        p.topk_idx[tok * K + lane] = -1;
        p.topk_weights[tok * K + lane] = 0.0f;
      }
      continue;
    }

    float key[V];  // -inf where the expert cannot be chosen
#pragma unroll
    for (int j = 0; j < V; ++j) {
      key[j] = x[j];
      if constexpr (SIG) {
        const int e = j * kTeam + t;
        const float b = W == 1 ? sm_bias[W == 1 ? e : 0]
                               : p.bias != nullptr && e < E ? __ldg(p.bias + e) : 0.0f;
        const float k = sc.s[j] + b;
        key[j] = x[j] > -INFINITY && k > -INFINITY ? k : -INFINITY;
      }
    }
    int mine = -1;  // lane k of the (first) warp: the k-th choice
    float w = 0.0f;  // its score
    bool any;
    if constexpr (W == 1) {
      int2* chosen = sm_chosen[warp];
      int n = -1;
      if (V > 1 && K <= kCandidateTopk)
        n = choose_candidates<V>(key, sc.s, K, lane, sm_key[warp], sm_choice[warp], chosen);
      const bool scored = n >= 0;
      if (!scored) n = choose_rounds<V>(key, K, lane, chosen);
      __syncwarp();
      if (lane < n) {
        mine = chosen[lane].x;
        w = scored ? __int_as_float(chosen[lane].y) : sc.score_of(load_logit(row + mine));
      }
      __syncwarp();
      any = n > 0;
    } else {
      any = choose_in_block<V, W>(key, K, t, redu, mine);
      if (warp == 0 && mine >= 0) w = sc.score_of(load_logit(row + mine));
    }
    if (W == 1 || warp == 0) {
      if (p.normalize) {
        float total = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
        w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
      }
      w *= p.scale;
      if (lane < K) {
        p.topk_idx[tok * K + lane] = mine;
        p.topk_weights[tok * K + lane] = w;
        if (mine >= 0) atomicAdd(&sm_count_[mine], 1);
      }
    }
    if (any) {
      ++routed;
#pragma unroll
      for (int j = 0; j < V; ++j) mass[j] += sc.s[j] * sc.inv;
    }
  }

  // the block's sums into the rank's
  if (t == 0 && routed) atomicAdd(&s_routed, routed);
  unsigned long long* gm = p.ws_mass + int64_t(rank) * E;
  int32_t* gc = p.ws_count + int64_t(rank) * E;
  if constexpr (W == 1) {
    constexpr int kChunk = V < 8 ? V : 8;  // 256 experts at a time
#pragma unroll
    for (int c = 0; c < V; c += kChunk) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kChunk; ++j) stage[warp * 256 + j * kWarp + lane] = mass[c + j];
      __syncthreads();
      const int e = c * kWarp + int(threadIdx.x);
      if (threadIdx.x < kChunk * kWarp && e < E) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) sum += stage[w * 256 + threadIdx.x];
        if (sum != 0.0f) atomicAdd(gm + e, (unsigned long long)(sum * p.fix));
      }
    }
  } else {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * kTeam + t;
      if (e < E && mass[j] != 0.0f) atomicAdd(gm + e, (unsigned long long)(mass[j] * p.fix));
    }
  }
  for (int e = threadIdx.x; e < E; e += kRouteThreads)
    if (sm_count_[e]) atomicAdd(gc + e, sm_count_[e]);
  if (threadIdx.x == 0 && s_routed) atomicAdd(p.ws_routed + rank, s_routed);

  // the rank's last block writes its counts and loss and clears the workspace
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = atom_add_acq_rel_u32(p.ws_done + rank, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int T_ = __ldcg(p.ws_routed + rank);
  const float unfix = 1.0f / p.fix;
  float sum = 0.0f;  // a fixed order again: thread, warp, block
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    const int c = __ldcg(gc + e);
    const unsigned long long f = __ldcg(gm + e);
    p.counts[int64_t(rank) * E + e] = c;
    sum += float(c) * (float(f) * unfix);
    gc[e] = 0;
    gm[e] = 0;
  }
  sum = team_reduce<kRouteWarps>(sum, red, OpSum());
  if (threadIdx.x == 0) {
    const float tokens = float(T_ > 0 ? T_ : 1);
    p.routed[rank] = T_;
    p.loss[rank] = p.loss_coef * float(E) / float(K) * (sum / tokens / tokens);
    p.ws_routed[rank] = 0;
    p.ws_done[rank] = 0;
  }
}

// Gradient.  With c_e = d_loss * coef * E * counts_e / (K T^2) (the share's
// gradient; the counts are constants) and g_k the chosen scores' gradient,
//   softmax: dl_e = p_e (h_e - sum_j p_j h_j),  h = c + g at the chosen
//   sigmoid: dl_e = s_e (1 - s_e) ((c_e - sum_j p_j c_j) / sum_j s_j + g_e)
//   g_k = scale * dw_k, or scale / S * (dw_k - sum_j dw_j s_j / S), S = sum of the chosen s.
template <typename T, int V, int W, bool SIG>
__global__ void __launch_bounds__(kRouteThreads, route_blocks(V, W))
mp_k_route_backward(const RouteArgs p) {
  constexpr int kTeam = W * kWarp;
  constexpr int kTeams = kRouteWarps / W;
  extern __shared__ float sm_g[];  // [kTeams][E]: the chosen scores' gradients
  __shared__ float red[kRouteWarps];
  __shared__ int s_any;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % kTeam;
  const int team = threadIdx.x / kTeam;
  const int rank = blockIdx.y;
  const int E = p.E, K = p.K;
  float* g = sm_g + team * E;
  pdl_wait_prior_grid();
  for (int e = t; e < E; e += kTeam) g[e] = 0.0f;
  float c[V];  // the share's gradient, the same for every routed token of the rank
  {
    const int routed = __ldg(p.routed + rank);
    const float T_ = float(routed > 0 ? routed : 1);
    const float f = p.d_loss != nullptr
        ? __ldg(p.d_loss + rank) * p.loss_coef * float(E) / (float(K) * T_ * T_) : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * kTeam + t;
      c[j] = e < E && p.d_loss != nullptr ? f * float(__ldg(p.counts + int64_t(rank) * E + e))
                                           : 0.0f;
    }
  }
  if constexpr (W > 1) __syncthreads(); else __syncwarp();

  for (uint32_t n = blockIdx.x * kTeams + team; n < uint32_t(p.N); n += gridDim.x * kTeams) {
    const int64_t tok = int64_t(rank) * p.N + n;
    const T* row = static_cast<const T*>(p.logits) + tok * E;
    T* row_out = static_cast<T*>(p.d_logits) + tok * E;
    float x[V];
    load_token<T, V, W>(row, E, t, x);
    TokenScores<T, V, W, SIG> sc;
    const bool active = p.active == nullptr || p.active[tok] != 0;
    // what the chosen ones' gradients need is on its way while the scores are computed
    int id = -1;
    float d = 0.0f, chosen_x = -INFINITY;
    if ((W == 1 || warp == 0) && lane < K) {
      id = __ldg(p.topk_idx + tok * K + lane);
      if (p.d_weights != nullptr) d = __ldg(p.d_weights + tok * K + lane) * p.scale;
      if (uint32_t(id) >= uint32_t(E)) id = -1;
      if (id >= 0) chosen_x = load_logit(row + id);
    }
    sc.template compute<false>(x, active, red);

    bool any;
    if (W == 1 || warp == 0) {
      any = __any_sync(kFull, id >= 0);
      float s = 0.0f;
      if (id >= 0 && sc.live)
        s = sc.score_of(chosen_x);
      else
        d = 0.0f;
      if (p.normalize) {
        float total = s, dot = d * s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          total += __shfl_xor_sync(kFull, total, o);
          dot += __shfl_xor_sync(kFull, dot, o);
        }
        const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
        d = (d - dot * inv) * inv;
      }
      if (id >= 0) g[id] = d;
      if (W > 1 && lane == 0) s_any = any;
    }
    if constexpr (W > 1) {
      __syncthreads();
      any = s_any;
    } else {
      __syncwarp();
    }
    float h[V];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * kTeam + t;
      const float gj = e < E ? g[e] : 0.0f;
      const float cj = any ? c[j] : 0.0f;
      if constexpr (SIG) {
        h[j] = gj;
        dot += sc.s[j] * sc.inv * cj;
      } else {
        h[j] = gj + cj;
        dot += sc.s[j] * h[j];
      }
    }
    dot = team_reduce<W>(dot, red, OpSum());  // (for W > 1 its barriers follow every read of g)
    if constexpr (W == 1) __syncwarp();
    if ((W == 1 || warp == 0) && id >= 0) g[id] = 0.0f;  // cleared for the next token
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * kTeam + t;
      float d;
      if constexpr (SIG)
        d = sc.s[j] * (1.0f - sc.s[j]) * (h[j] + ((any ? c[j] : 0.0f) - dot) * sc.inv);
      else
        d = sc.s[j] * (h[j] - dot);
      if (e < E) store_grad(row_out + e, d);
    }
    if constexpr (W == 1) __syncwarp(); else __syncthreads();
  }
}

template <typename T, int V, int W, bool SIG>
cudaError_t launch_route_as(const RouteArgs& p, bool backward, cudaStream_t st) {
  constexpr int kTeams = kRouteWarps / W;
  // As many blocks as are resident at a time, spread over the ranks.  (Up to 256
  // experts, forward: four per SM 19 us for 8 x 4,096 tokens of 64, three 20, six 23: a
  // block's sums at its end cost more than the tokens that it takes over.)
  const int64_t need = (int64_t(p.N) + kTeams - 1) / kTeams;
  const int64_t most = std::max<int64_t>(1, int64_t(sm_count()) * (W > 1 || V == 32 ? 2 : 4) / p.R);
  const dim3 grid(unsigned(std::max<int64_t>(1, std::min(need, most))), unsigned(p.R));
  if (backward)
    return launch_waiting(mp_k_route_backward<T, V, W, SIG>, grid, dim3(kRouteThreads),
                          size_t(kTeams) * p.E * 4, st, 0, p);
  return launch_waiting(mp_k_route<T, V, W, SIG>, grid, dim3(kRouteThreads), size_t(p.E) * 4, st,
                        0, p);
}

template <typename T, bool SIG>
cudaError_t launch_route_v(const RouteArgs& p, bool backward, cudaStream_t st) {
  const int E = p.E;
  if (E <= 32) return launch_route_as<T, 1, 1, SIG>(p, backward, st);
  if (E <= 64) return launch_route_as<T, 2, 1, SIG>(p, backward, st);
  if (E <= 128) return launch_route_as<T, 4, 1, SIG>(p, backward, st);
  if (E <= 256) return launch_route_as<T, 8, 1, SIG>(p, backward, st);
  if (E <= 512) return launch_route_as<T, 16, 1, SIG>(p, backward, st);
  if (E <= 1024) return launch_route_as<T, 32, 1, SIG>(p, backward, st);
  if (E <= 2048) return launch_route_as<T, 8, 8, SIG>(p, backward, st);
  if (E <= 4096) return launch_route_as<T, 16, 8, SIG>(p, backward, st);
  return launch_route_as<T, 32, 8, SIG>(p, backward, st);
}

cudaError_t launch_route_t(const RouteArgs& p, int scoring, int dtype, bool backward,
                           cudaStream_t st) {
  if (dtype == MP_FP32)
    return scoring == MP_SIGMOID ? launch_route_v<float, true>(p, backward, st)
                                 : launch_route_v<float, false>(p, backward, st);
  return scoring == MP_SIGMOID ? launch_route_v<__nv_bfloat16, true>(p, backward, st)
                               : launch_route_v<__nv_bfloat16, false>(p, backward, st);
}

}  // namespace

size_t route_workspace_bytes(int R, int E) {
  return size_t(MP_MAX_RANKS) * 8 + size_t(R) * E * 12;
}

cudaError_t launch_route(int R, int N, int K, int E, int scoring, int dtype, const void* logits,
                         const float* bias, const uint8_t* active, int normalize, float scale,
                         float loss_coef, int32_t* topk_idx, float* topk_weights,
                         int32_t* num_tokens_per_expert, int32_t* num_routed, float* balance_loss,
                         int32_t* dev_err, unsigned char* workspace, cudaStream_t st) {
  RouteArgs p = {};
  p.R = R; p.N = N; p.K = K; p.E = E;
  p.normalize = normalize; p.scale = scale; p.loss_coef = loss_coef;
  p.logits = logits; p.bias = bias; p.active = active;
  p.topk_idx = topk_idx; p.topk_weights = topk_weights;
  p.counts = num_tokens_per_expert; p.routed = num_routed; p.loss = balance_loss;
  p.dev_err = dev_err;
  p.ws_done = reinterpret_cast<uint32_t*>(workspace);
  p.ws_routed = reinterpret_cast<int32_t*>(workspace + size_t(MP_MAX_RANKS) * 4);
  p.ws_mass = reinterpret_cast<unsigned long long*>(workspace + size_t(MP_MAX_RANKS) * 8);
  p.ws_count = reinterpret_cast<int32_t*>(workspace + size_t(MP_MAX_RANKS) * 8 + size_t(R) * E * 8);
  int bits = 62;  // the largest sum, N, stays below 2^63
  for (int64_t n = N; n > 0; n >>= 1) --bits;
  p.fix = ldexpf(1.0f, bits);
  return launch_route_t(p, scoring, dtype, false, st);
}

cudaError_t launch_route_backward(int R, int N, int K, int E, int scoring, int dtype,
                                  const void* logits, const uint8_t* active, int normalize,
                                  float scale, float loss_coef, const int32_t* topk_idx,
                                  const float* d_topk_weights,
                                  const int32_t* num_tokens_per_expert, const int32_t* num_routed,
                                  const float* d_balance_loss, void* d_logits, cudaStream_t st) {
  if (N == 0) return cudaSuccess;
  RouteArgs p = {};
  p.R = R; p.N = N; p.K = K; p.E = E;
  p.normalize = normalize; p.scale = scale; p.loss_coef = loss_coef;
  p.logits = logits; p.active = active;
  p.topk_idx = const_cast<int32_t*>(topk_idx);
  p.counts = const_cast<int32_t*>(num_tokens_per_expert);
  p.routed = const_cast<int32_t*>(num_routed);
  p.d_weights = d_topk_weights; p.d_loss = d_balance_loss; p.d_logits = d_logits;
  return launch_route_t(p, scoring, dtype, true, st);
}

}  // namespace mp
