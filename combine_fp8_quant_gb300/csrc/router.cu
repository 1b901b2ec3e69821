// router.cu -- the router of an MoE block: each token's experts and weights from
// its logits, the batch's balance and z losses, and the gradient of the logits.
//
//   score     s_e = exp(l_e) / sum_j exp(l_j)   or   1 / (1 + exp(-l_e))
//   choice    the K largest of l_e, or of s_e + b_e with a bias, lowest index first
//             among equals; weights scale * s_k, or scale * s_k / sum over the chosen
//   balance   over groups q of n_q tokens:  1/Q sum_q E / (K n_q^2) sum_e c[q,e] P[q,e],
//             c the chosen slots, P the sums of p (the scores normalised over the experts)
//   z         mean over the tokens of logsumexp(l)^2
//
// One warp works on a token with its logits in registers (lane i holds the vectors i,
// 32 + i, ... of the row), so a row is read once and everything about it is a few warp
// reductions.
#include <cfloat>
#include <climits>
#include <type_traits>

#include "elem.cuh"
#include "kernels.h"

namespace moeperm {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kNegInf = -INFINITY;

template <int TYPE>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (TYPE == kF32) {
    return __ldg(static_cast<const float*>(p) + i);
  } else {
    const uint32_t w = __ldg(static_cast<const uint16_t*>(p) + i);
    return TYPE == kBF16 ? __uint_as_float(w << 16) : f16x2_to_float2(w).x;
  }
}
template <int TYPE>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (TYPE == kF32) {
    static_cast<float*>(p)[i] = v;
  } else {
    static_cast<uint16_t*>(p)[i] = (uint16_t)(TYPE == kBF16 ? pack_bf16x2(v, 0.0f) : pack_f16x2(v, 0.0f));
  }
}

// Expert of a lane's i-th logit: vectors of V logits, the warp's 32 side by side.
template <int V>
__device__ __forceinline__ int expert_of(int i, int lane) {
  return (i / V) * 32 * V + lane * V + i % V;
}
// Logits of a token; -inf past the last expert. V > 1: the rows are whole aligned
// vectors of V (two, four or eight to 16 bytes or less).
template <int TYPE, int N, int V>
__device__ __forceinline__ void load_row(float (&v)[N], const void* p, int64_t at, int E, int lane) {
  if constexpr (V == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i * 32 + lane < E ? load_elem<TYPE>(p, at + i * 32 + lane) : kNegInf;
  } else {
    constexpr int kBytes = V * (TYPE == kF32 ? 4 : 2), kWords = kBytes / 4;
    const uint8_t* row = static_cast<const uint8_t*>(p) + at * (kBytes / V) + lane * kBytes;
#pragma unroll
    for (int j = 0; j < N / V; ++j) {
      uint32_t w[kWords];
      if (j * 32 * V + lane * V < E) {
        const uint8_t* q = row + j * 32 * kBytes;
        if constexpr (kWords == 4) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(q));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else if constexpr (kWords == 2) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(q));
          w[0] = x.x; w[1] = x.y;
        } else {
          w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          if constexpr (TYPE == kF32) {
            v[j * V + i] = __uint_as_float(w[i]);
          } else {
            const float2 f = TYPE == kBF16 ? make_float2(bf16_lo(w[i]), bf16_hi(w[i])) : f16x2_to_float2(w[i]);
            v[j * V + 2 * i] = f.x;
            v[j * V + 2 * i + 1] = f.y;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[j * V + i] = kNegInf;
      }
    }
  }
}
// The same way back, rounded to the type.
template <int TYPE, int N, int V>
__device__ __forceinline__ void store_row(void* p, int64_t at, int E, int lane, const float (&v)[N]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * 32 + lane < E) store_elem<TYPE>(p, at + i * 32 + lane, v[i]);
  } else {
    constexpr int kBytes = V * (TYPE == kF32 ? 4 : 2), kWords = kBytes / 4;
    uint8_t* row = static_cast<uint8_t*>(p) + at * (kBytes / V) + lane * kBytes;
#pragma unroll
    for (int j = 0; j < N / V; ++j) {
      if (j * 32 * V + lane * V >= E) break;
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = TYPE == kF32 ? __float_as_uint(v[j * V + i])
               : TYPE == kBF16 ? pack_bf16x2(v[j * V + 2 * i], v[j * V + 2 * i + 1])
                               : pack_f16x2(v[j * V + 2 * i], v[j * V + 2 * i + 1]);
      uint8_t* q = row + j * 32 * kBytes;
      if constexpr (kWords == 4) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (kWords == 2) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(q) = w[0];
    }
  }
}

// Floats as unsigned integers of the same order. 0: never chosen (NaN and -inf).
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // both zeros are one key
  return f > kNegInf ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;
}

// e^x and 1 / x by the approximating instructions, results below 2^-126 as 0 (e^x to about
// 2 + 1.2 |x| steps, 1 / x to one). The functions that keep such numbers take three to
// four times the instructions, which are the bound here: the choice for 16384 tokens of
// 256 experts takes 25.1 us with expf and a division and 21.5 with these (without a bias 13.8
// and 12.7).
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // a NaN is left out
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// CTAs an SM that a kernel with N logits a lane is compiled for.
__host__ __device__ constexpr int min_blocks(int N) { return N <= 8 ? 4 : N <= 16 ? 2 : 1; }

// 1 / (1 + e^-l) and 1 minus that, neither with cancellation.
__device__ __forceinline__ float sigmoid(float l) {
  const float x = fast_exp(-fabsf(l));
  return (l < 0.0f ? x : 1.0f) * fast_rcp(1.0f + x);
}
__device__ __forceinline__ float sigmoid_rest(float l) {
  const float x = fast_exp(-fabsf(l));
  return (l < 0.0f ? 1.0f : x) * fast_rcp(1.0f + x);
}

// Where every logit of a set is below this, its sigmoids are exponentials (to 2^-28, less than
// fp32 rounds by) that may leave the range of a float, and their ratios are those of a
// softmax. Above it a ratio is lost where its sigmoid is below 2^-126: one below 2^-97.
constexpr float kFarBelow = -20.0f;

// Normalised scores of a token over all experts: softmax, or sigmoids over their
// sum. m: the largest logit (-inf: a row without any, whose scores are 0). rest: 1
// minus the sigmoids, where they are asked for.
template <bool kRest, int N>
__device__ __forceinline__ void scores(const float (&l)[N], float m, bool sig, float (&p)[N], float (&rest)[N]) {
  if (m == kNegInf) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = isnan(l[i]) ? l[i] : 0.0f;
      if (kRest) rest[i] = 1.0f;
    }
    return;
  }
  float z = 0.0f;
  if (!sig || m < kFarBelow) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = fast_exp(l[i] - m);
      if (kRest) rest[i] = 1.0f;
      z += p[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = fast_exp(-fabsf(l[i])), r = fast_rcp(1.0f + x), xr = x * r;
      p[i] = l[i] < 0.0f ? xr : r;
      if (kRest) rest[i] = l[i] < 0.0f ? r : xr;
      z += p[i];
    }
  }
  const float r = fast_rcp(warp_sum(z));
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] *= r;
}

// ---------------------------------------------------------------------------
// The choice of experts
// ---------------------------------------------------------------------------

// The choice by K rounds of the largest key left, for a token that the quick way does
// not settle: keys of KEY (uint32_t: ordered logits; double: scores with bias in 64
// bits). Lane k gets the k-th id (-1: none).
template <typename KEY, int TYPE, int N>
__device__ __forceinline__ int choose_by_rounds(const RouteArgs& a, int64_t at, int lane) {
  KEY key[N];
  const KEY none = std::is_same<KEY, double>::value ? (KEY)-INFINITY : (KEY)0;
  if constexpr (std::is_same<KEY, double>::value) {
    double z = 0.0, m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      key[i] = i * 32 + lane < a.E ? (double)load_elem<TYPE>(a.logits, at + i * 32 + lane) : -INFINITY;
      m = fmax(m, key[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      key[i] = a.sigmoid ? 1.0 / (1.0 + exp(-key[i])) : exp(key[i] - m);
      z += key[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int e = i * 32 + lane;
      const bool may = e < a.E && load_elem<TYPE>(a.logits, at + (e < a.E ? e : 0)) > kNegInf;
      key[i] = may ? (a.sigmoid ? key[i] : key[i] / z) + (double)__ldg(a.bias + e) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = i * 32 + lane < a.E ? ordered(load_elem<TYPE>(a.logits, at + i * 32 + lane)) : 0u;
  }
  int mine = -1;
  for (int k = 0; k < a.K; ++k) {
    KEY best = none;
    int id = INT_MAX;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > best) {
        best = key[i];
        id = i * 32 + lane;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const KEY ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oi = __shfl_xor_sync(0xffffffffu, id, o);
      if (ob > best || (ob == best && oi < id)) {
        best = ob;
        id = oi;
      }
    }
    if (id == INT_MAX) break;
    if (lane == k) mine = id;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * 32 + lane == id) key[i] = none;
  }
  return mine;
}

// One token with logits l. The quick way: at least K + 2 keys are no less than the
// (K + 2)-th largest of the 32 lanes' largest, and seldom many more (ten or eleven of 256
// for K = 8). They go to shared memory, one for each lane, which counts those that come
// before its own. Returns false, with nothing written, where that does not settle the
// choice: more candidates than lanes, or, with a bias, keys too near each other for 32
// bits. EXACT settles it: such candidates by keys in 64 bits, else rounds over all keys.
template <bool EXACT, int TYPE, int N, int V>
__device__ __forceinline__ bool route_token(const RouteArgs& a, int64_t t, const float (&l)[N], uint2* cand,
                                            const float* s_bias, int lane) {
  const bool biased = a.bias != nullptr;
  float key[N], m = kNegInf, z = 1.0f;
  if (!a.sigmoid && (biased || !a.renorm)) {  // the sum over all experts
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) z += fast_exp(l[i] - m);
    z = warp_sum(z);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = l[i];
  if (biased) {
    const float r = a.sigmoid ? 0.0f : fast_rcp(z);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = expert_of<V>(i, lane);
      const float s = a.sigmoid ? sigmoid(l[i]) : fast_exp(l[i] - m) * r;
      key[i] = l[i] > kNegInf ? s + s_bias[e < a.E ? e : 0] : kNegInf;
    }
  }
  // a key that at least K + 2 reach (or every one that may be chosen, where there are fewer)
  float top = kNegInf, floor = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, key[i]);
  for (int have = 0; have < a.K + 2;) {
    const float best = warp_max(top);
    floor = fmaxf(best, -FLT_MAX);
    if (best == kNegInf) break;
    const bool is = top == best;
    have += __popc(__ballot_sync(0xffffffffu, is));
    if (is) top = kNegInf;
  }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) mine += key[i] >= floor;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int below = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += below;
  }
  const int n = __shfl_sync(0xffffffffu, upto, 31);
  if (!EXACT && n > 32) return false;
  int id = -1, rank = 32, got = min(n, a.K);
  float lk = kNegInf;
  bool rounds = n > 32;
  if (!rounds) {
    uint2* at = cand + (upto - mine);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] >= floor) *at++ = make_uint2(__float_as_uint(key[i]), (uint32_t)expert_of<V>(i, lane));
    if (lane < 3) cand[n + lane] = make_uint2(0xFF800000u, 0);  // up to a whole four
    __syncwarp();
    float k = kNegInf;
    if (lane < n) {
      k = __uint_as_float(cand[lane].x);
      id = (int)cand[lane].y;
      lk = load_elem<TYPE>(a.logits, t * a.ld + id);
      rank = 0;
    }
    // Keys in 32 bits are off by 2^-21 (sigmoid), or by (N + 12) 2^-24 (a sum of 32 N
    // exponentials), and half a step of the sum with the bias. Two of them nearer than
    // twice that, and not equal from equal parts, are told apart in 64 bits.
    const float eps = (a.sigmoid ? 0x1p-19f : (N + 24) * 0x1p-23f) + fabsf(k) * 0x1p-22f;
    int near = 0;  // (its own among them)
    for (int j = 0; j < n; j += 4) {
      const uint4 p0 = *reinterpret_cast<const uint4*>(cand + j), p1 = *reinterpret_cast<const uint4*>(cand + j + 2);
      const uint2 o[4] = {make_uint2(p0.x, p0.y), make_uint2(p0.z, p0.w), make_uint2(p1.x, p1.y), make_uint2(p1.z, p1.w)};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float ok = __uint_as_float(o[u].x);
        rank += ok > k || (ok == k && (int)o[u].y < id);
        if (biased) near += !(fabsf(ok - k) > eps);
      }
    }
    __syncwarp();
    if (biased) {
      // A key that is no candidate may be as near to the last chosen one only if that one
      // is as near to the least candidate.
      const bool in = lane < n && rank < a.K;
      const bool open = __any_sync(0xffffffffu, in && n >= a.K + 2 && floor > -FLT_MAX && !(k - floor > 2.0f * eps));
      if (open || __any_sync(0xffffffffu, in && near > 1)) {
        const float bk = lane < n ? s_bias[id] : 0.0f;
        bool unlike = false;  // a candidate near a chosen one, and not of equal parts
        for (int j = 0; j < n; ++j) {
          const float ok = __shfl_sync(0xffffffffu, k, j), ol = __shfl_sync(0xffffffffu, lk, j);
          const float ob = __shfl_sync(0xffffffffu, bk, j);
          unlike |= !(fabsf(ok - k) > eps) && (ol != lk || ob != bk);
        }
        unlike = __any_sync(0xffffffffu, unlike && in);
        if (!EXACT && (open || unlike)) return false;
        if (EXACT) {
          rounds = open || !a.sigmoid;
          if (!rounds) {
            const double k64 = lane < n ? 1.0 / (1.0 + exp(-(double)lk)) + (double)bk : 0.0;
            rank = lane < n ? 0 : 32;
            for (int j = 0; j < n; ++j) {
              const double o = __shfl_sync(0xffffffffu, k64, j);
              const int oid = __shfl_sync(0xffffffffu, id, j);
              rank += o > k64 || (o == k64 && oid < id);
            }
          }
        }
      }
    }
  }
  if (EXACT && rounds) {
    id = biased ? choose_by_rounds<double, TYPE, N>(a, t * a.ld, lane) : choose_by_rounds<uint32_t, TYPE, N>(a, t * a.ld, lane);
    rank = id >= 0 ? lane : 32;
    lk = id >= 0 ? load_elem<TYPE>(a.logits, t * a.ld + id) : kNegInf;
    got = __popc(__ballot_sync(0xffffffffu, id >= 0));
  }
  const bool chosen = rank < a.K;
  float s = 0.0f;
  if (a.renorm) {
    const float mk = warp_max(chosen ? lk : kNegInf);
    const bool soft = !a.sigmoid || mk < kFarBelow;
    if (chosen) s = soft ? fast_exp(lk - mk) : sigmoid(lk);
    s *= fast_rcp(warp_sum(s));
  } else if (chosen) {
    s = a.sigmoid ? sigmoid(lk) : fast_exp(lk - m) * fast_rcp(z);
  }
  if (chosen) {
    a.ids[t * a.K + rank] = id;
    a.weights[t * a.K + rank] = a.scale * s;
  }
  if (lane >= got && lane < a.K) {
    a.ids[t * a.K + lane] = -1;
    a.weights[t * a.K + lane] = 0.0f;
  }
  return true;
}

// Tokens that the quick way does not settle wait until the warp's others are done (at
// most 64 at a time): as calls in the loop they cost every token 40% (registers). Bound by
// instructions, 947 a token of 256 experts with biased sigmoids of logits with a deviation of
// 1.5, where one token in a thousand waits. How many wait, and so the time, depends on the
// data. 16384 tokens of 256 experts, K = 8, in us:
//   logits' deviation        1.5        0.1        0.02       all equal
//   sigmoid, bias of 0.1     22         22         22         17
//   sigmoid, bias of zeros   22         22         27         394
//   softmax, bias of 0.1     38         17         17         17
//   softmax, bias of zeros   39         267        420        408
//   no bias                  13         13         13         29
// (near keys of softmax scores are computed again over all experts). With many slots most
// tokens have more than 32 candidates, with K of 30 and more all: K = 16, 20 and 32 take 73,
// 429 and 851 us with biased sigmoids and 23, 60 and 98 without a bias; of 64 experts 23, 66
// and 482, and 15, 24 and 69.
template <int TYPE, int N, int V>
__global__ void __launch_bounds__(kThreads, min_blocks(N)) route_kernel(RouteArgs a) {
  __shared__ __align__(16) uint2 s_cand[kWarps][36];  // key, expert; in fours
  __shared__ float s_bias[32 * N];
  const int lane = threadIdx.x & 31;
  uint2* cand = s_cand[threadIdx.x >> 5];
  const int64_t nwarps = (int64_t)gridDim.x * kWarps;
  const int n_live = live_count(a.d_num_tokens, a.T, a.status, blockIdx.x == 0 && threadIdx.x == 0);
  int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  float next[N];
  if (t < n_live) load_row<TYPE, N, V>(next, a.logits, t * a.ld, a.E, lane);
  if (a.bias != nullptr) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) s_bias[e] = __ldg(a.bias + e);
    __syncthreads();
  }
  while (t < n_live) {
    const int64_t first = t;
    uint64_t open = 0;  // bit i: token first + i * nwarps
    for (int i = 0; i < 64 && t < n_live; ++i, t += nwarps) {
      float l[N];
#pragma unroll
      for (int j = 0; j < N; ++j) l[j] = next[j];
      if (t + nwarps < n_live) load_row<TYPE, N, V>(next, a.logits, (t + nwarps) * a.ld, a.E, lane);
      if (!route_token<false, TYPE, N, V>(a, t, l, cand, s_bias, lane)) open |= 1ull << i;
    }
    while (open != 0) {
      const int64_t late = first + (__ffsll((long long)open) - 1) * nwarps;
      open &= open - 1;
      float l[N];
      load_row<TYPE, N, V>(l, a.logits, late * a.ld, a.E, lane);
      route_token<true, TYPE, N, V>(a, late, l, cand, s_bias, lane);
    }
  }
}

// ---------------------------------------------------------------------------
// Groups of tokens
// ---------------------------------------------------------------------------

// Sizes and first flattened tokens of the groups in shared memory: cnt, st [Q] (and 33
// ints of scratch). Groups lie one after the other inside the live tokens; if any does
// not, the call has none (and flags it). In the flattened order a group is followed by
// `pad` places without a token. Returns the places of all groups.
__device__ __forceinline__ int plan_groups(const GroupArgs& g, int n_live, int pad, int32_t* cnt, int32_t* st,
                                           int32_t* scratch, int32_t* status, int& nonempty) {
  if (g.begin == nullptr) {
    if (threadIdx.x == 0) {
      cnt[0] = n_live;
      st[0] = 0;
    }
    __syncthreads();
    nonempty = n_live > 0;
    return n_live > 0 ? n_live + pad : 0;
  }
  bool ok = true;
  for (int q = threadIdx.x; q < g.Q; q += blockDim.x) {
    const int b = __ldg(g.begin + q), e = __ldg(g.end + q);
    const int before = q > 0 ? __ldg(g.end + q - 1) : 0;
    ok &= before <= b && b >= 0 && b <= e && e <= n_live;
    cnt[q] = e > b ? e - b + pad : 0;
  }
  int some = 0;
  ok = __syncthreads_and(ok);
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(status, kStBadLayout);
  for (int q = threadIdx.x; q < g.Q; q += blockDim.x) {
    if (!ok) cnt[q] = 0;
    some += cnt[q] > 0;
  }
  __syncthreads();
  const int total = aligned_starts(cnt, st, g.Q, 1, INT_MAX, scratch);
  some = __reduce_add_sync(0xffffffffu, some);
  if (threadIdx.x == 0) scratch[0] = 0;
  __syncthreads();
  if ((threadIdx.x & 31) == 0 && some > 0) atomicAdd(scratch, some);
  __syncthreads();
  nonempty = scratch[0];
  if (pad > 0) {
    for (int q = threadIdx.x; q < g.Q; q += blockDim.x)
      if (cnt[q] > 0) cnt[q] -= pad;
    __syncthreads();
  }
  return total;
}

// ---------------------------------------------------------------------------
// The losses
// ---------------------------------------------------------------------------

// Workspace: sums of the parts [slots][E] and their counts [slots][E], z [slots], each
// group's share of the losses, and what the second launch has to know. A CTA takes a
// run of the flattened tokens; its part of group q has slot blockIdx.x + q, which no
// other part has, since along the tokens the two only grow.
struct BalanceWs {
  float* P;
  int32_t* c;
  float* z;
  float* share;      // [Q][slices] balance
  float* zshare;     // [Q]
  int32_t* meta;     // [Q][3]: first slot, slots, tokens; then groups with tokens, tokens, ticket
};
__host__ __device__ inline int64_t balance_slots(int Q) { return kBalanceParts + Q; }
__device__ __forceinline__ BalanceWs balance_ws(const BalanceArgs& a) {
  const int64_t slots = balance_slots(a.g.Q), slices = (a.E + 31) / 32;
  BalanceWs w;
  w.P = a.ws;
  w.c = reinterpret_cast<int32_t*>(w.P + slots * a.E);
  w.z = reinterpret_cast<float*>(w.c + slots * a.E);
  w.share = w.z + slots;
  w.zshare = w.share + a.g.Q * slices;
  w.meta = reinterpret_cast<int32_t*>(w.zshare + a.g.Q);
  return w;
}

// Square of the logsumexp of a row whose largest logit but for NaN is infinite (warp_max leaves
// NaN out): NaN with one, 0 where all are -inf (such a token has no part in the loss).
template <int N>
__device__ __forceinline__ float odd_row(const float (&l)[N], float m) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) bad |= isnan(l[i]);
  return __any_sync(0xffffffffu, bad) ? __uint_as_float(0x7FC00000u) : m > 0.0f ? INFINITY : 0.0f;
}

// Sums over a run of tokens, one warp a token, four at a time. Joining the warps' sums
// for a group costs a CTA about as much as kGroupCost tokens, so a run of short groups
// counts for more. Bound by latencies: a batch of 65536 tokens leaves a warp about a
// dozen.
constexpr int kGroupCost = 32;
template <int TYPE, int N, int V>
__global__ void __launch_bounds__(kThreads) balance_parts_kernel(BalanceArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t s_scratch[33];
  __shared__ float s_z[kWarps];
  pdl_launch_dependents();  // the second launch waits for this one's end on the device
  int32_t* cnt = sm;
  int32_t* st = cnt + a.g.Q;
  int32_t* hist = st + a.g.Q;                               // [E]
  float* s_acc = reinterpret_cast<float*>(hist + a.E);      // [kWarps][E]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = a.E;
  const int n_live = live_count(a.d_num_tokens, a.T, a.status, blockIdx.x == 0 && tid == 0);
  int nonempty;
  const int total = plan_groups(a.g, n_live, kGroupCost, cnt, st, s_scratch, a.status, nonempty);
  const int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  const BalanceWs w = balance_ws(a);
  if (blockIdx.x == 0) {
    for (int q = tid; q < a.g.Q; q += kThreads) {
      const int b0 = cnt[q] > 0 ? st[q] / per : 0;
      w.meta[3 * q] = b0 + q;
      w.meta[3 * q + 1] = cnt[q] > 0 ? (st[q] + cnt[q] - 1) / per - b0 + 1 : 0;
      w.meta[3 * q + 2] = cnt[q];
    }
    if (tid == 0) {
      w.meta[3 * a.g.Q] = nonempty;
      w.meta[3 * a.g.Q + 1] = total - nonempty * kGroupCost;
      w.meta[3 * a.g.Q + 2] = 0;
    }
  }
  int at = (int)min((int64_t)blockIdx.x * per, (int64_t)total);
  const int stop = (int)min((int64_t)at + per, (int64_t)total);
  if (at >= stop) return;
  int q = 0;
  for (int hi = a.g.Q - 1; q < hi;) {  // the last group that starts at or before `at`
    const int mid = (q + hi + 1) >> 1;
    if (st[mid] <= at) q = mid; else hi = mid - 1;
  }
  for (; at < stop; ++q) {
    const int upto = min(stop, st[q] + cnt[q]);
    if (upto <= at) {  // past the group's tokens
      if (cnt[q] > 0) at = max(at, min(stop, st[q] + cnt[q] + kGroupCost));
      continue;
    }
    for (int e = tid; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int64_t first = (a.g.begin != nullptr ? __ldg(a.g.begin + q) : 0) + (at - st[q]);
    const int n = upto - at;
    for (int64_t i = tid; i < (int64_t)n * a.K; i += kThreads) {
      const int id = __ldg(a.ids + first * a.K + i);
      if (id >= 0 && id < E) atomicAdd(hist + id, 1);
    }
    float acc[N], z = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    constexpr int kAhead = N <= 8 ? 4 : N <= 16 ? 2 : 1;  // tokens of a warp in flight
    for (int j = warp; j < n; j += kAhead * kWarps) {
      float l[kAhead][N];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j + u * kWarps < n) load_row<TYPE, N, V>(l[u], a.logits, (first + j + u * kWarps) * a.ld, E, lane);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (j + u * kWarps >= n) break;
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, l[u][i]);
        m = warp_max(m);
        float p[N], zs = 0.0f;
        const bool odd = !(fabsf(m) < INFINITY);
        if (!odd) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            p[i] = fast_exp(l[u][i] - m);
            zs += p[i];
          }
          zs = warp_sum(zs);
          const float lse = m + __logf(zs);
          z = fmaf(lse, lse, z);
          const float r = fast_rcp(zs);
#pragma unroll
          for (int i = 0; i < N; ++i) p[i] *= r;
        } else {
          z += odd_row(l[u], m);
        }
        if (a.sigmoid || odd) scores<false>(l[u], m, a.sigmoid, p, p);  // (the z loss is of the softmax's sum)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += p[i];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (expert_of<V>(i, lane) < E) s_acc[warp * E + expert_of<V>(i, lane)] = acc[i];
    if (lane == 0) s_z[warp] = z;
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + q;
    for (int e = tid; e < E; e += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += s_acc[i * E + e];
      w.P[slot * E + e] = v;
      w.c[slot * E + e] = hist[e];
    }
    if (tid == 0) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += s_z[i];
      w.z[slot] = v;
    }
    __syncthreads();
    at = min(stop, st[q] + cnt[q] + kGroupCost);  // (upto, where the run ends inside)
  }
}

// Joins the parts of group blockIdx.y for 32 experts; the last to finish joins the groups.
// All latency: what it reads is in L2. With few groups (of many parts each) a CTA joins
// them, a row of threads for every 32nd part; with many, a warp.
constexpr int kFewGroups = 8;
template <bool FEW>
__global__ void __launch_bounds__(FEW ? 1024 : 128) balance_join_kernel(BalanceArgs a) {
  __shared__ float s_p[32][33];
  __shared__ int32_t s_c[32][33];
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int q = blockIdx.y, E = a.E, slices = (E + 31) / 32, slice = FEW ? blockIdx.x : blockIdx.x * 4 + row;
  if (slice >= slices) return;
  const int e0 = slice * 32, e = e0 + lane;
  const BalanceWs w = balance_ws(a);
  const int first = __ldcg(w.meta + 3 * q), parts = __ldcg(w.meta + 3 * q + 1), n = __ldcg(w.meta + 3 * q + 2);
  float p = 0.0f;
  int c = 0;
  if (e < E) {
#pragma unroll 8
    for (int i = FEW ? row : 0; i < parts; i += FEW ? 32 : 1) {
      p += __ldcg(w.P + (int64_t)(first + i) * E + e);
      c += __ldcg(w.c + (int64_t)(first + i) * E + e);
    }
  }
  if (slice == 0 && (!FEW || row == 31)) {
    float z = 0.0f;
    for (int i = lane; i < parts; i += 32) z += __ldcg(w.z + first + i);
    z = warp_sum(z);
    if (lane == 0) w.zshare[q] = z;
  }
  if (FEW) {  // warp k joins the parts of expert e0 + k
    s_p[row][lane] = p;
    s_c[row][lane] = c;
    __syncthreads();
    p = warp_sum(s_p[lane][row]);
    c = __reduce_add_sync(0xffffffffu, s_c[lane][row]);
    __syncthreads();
    if (lane == 0) {
      s_p[0][row] = p;
      s_c[0][row] = c;
    }
    __syncthreads();
    if (row > 0) return;
    p = s_p[0][lane];
    c = s_c[0][lane];
  }
  if (e < E) {
    a.counts[(int64_t)q * E + e] = c;
    a.prob_sums[(int64_t)q * E + e] = p;
  }
  const float dot = warp_sum(e < E ? (float)c * p : 0.0f);
  int last = 0;
  if (lane == 0) {
    w.share[(int64_t)q * slices + slice] = n > 0 ? dot / n / n * E / a.K : 0.0f;
    __threadfence();
    last = atomicAdd(reinterpret_cast<unsigned*>(w.meta + 3 * a.g.Q + 2), 1u) == (unsigned)(slices * a.g.Q - 1);
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  float b = 0.0f, z = 0.0f;
#pragma unroll 8
  for (int64_t i = lane; i < (int64_t)slices * a.g.Q; i += 32) b += __ldcg(w.share + i);
#pragma unroll 4
  for (int i = lane; i < a.g.Q; i += 32) z += __ldcg(w.zshare + i);
  b = warp_sum(b);
  z = warp_sum(z);
  if (lane == 0) {
    const int some = __ldcg(w.meta + 3 * a.g.Q), total = __ldcg(w.meta + 3 * a.g.Q + 1);
    a.loss[0] = some > 0 ? b / some : 0.0f;
    a.loss[1] = total > 0 ? z / total : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// The gradient of the logits
// ---------------------------------------------------------------------------

// One warp a token; a warp takes runs of kRun tokens, so that a group's counts stay in
// registers for some while the runs of a group are spread over the SMs (tokens of no group
// cost half as much). What the chosen experts add is spread over the row through a line of
// shared memory. Bound by latencies and issue: about 400 instructions a token of 256
// experts, against 2 KB of traffic.
constexpr int kRun = 4;
template <int TYPE, int N, int V>
__global__ void __launch_bounds__(kThreads, min_blocks(N)) route_grad_kernel(RouteGradArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t s_scratch[33];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = a.E, K = a.K, Q = a.g.Q;
  int32_t* cnt = sm;       // tokens of each group
  int32_t* st = cnt + Q;   // its first token
  float* add = reinterpret_cast<float*>(st + Q) + warp * E;
  for (int e = lane; e < E; e += 32) add[e] = 0.0f;
  const int n_live = live_count(a.d_num_tokens, a.T, a.status, blockIdx.x == 0 && tid == 0);
  float db = 0.0f, dz = 0.0f;
  if (a.dloss != nullptr) {  // uniform over the grid
    int nonempty;
    const int total = plan_groups(a.g, n_live, 0, cnt, st, s_scratch, a.status, nonempty);
    if (nonempty > 0) {
      db = __ldg(a.dloss) * (float)E / ((float)K * (float)nonempty);
      dz = 2.0f * __ldg(a.dloss + 1) / (float)total;
    }
    if (a.g.begin != nullptr) {
      for (int q = tid; q < Q; q += kThreads) st[q] = __ldg(a.g.begin + q);
      __syncthreads();
    }
  }
  __syncwarp();
  const int64_t nwarps = (int64_t)gridDim.x * kWarps;
  int64_t t = ((int64_t)blockIdx.x * kWarps + warp) * kRun;
  auto following = [&](int64_t at) { return ++at % kRun ? at : at + (nwarps - 1) * kRun; };
  int q = 0, have = -1;             // group that holds token t or comes next; the group of g
  float g[N];                       // its gradient of the sums of p
  float l[N], next[N], dw = 0.0f, ndw = 0.0f, lk, nlk = kNegInf;
  int id = -1, nid = -1;
  auto load = [&](int64_t at, float (&row)[N], int& i, float& d) {
    load_row<TYPE, N, V>(row, a.logits, at * a.ld, E, lane);
    i = -1;
    d = 0.0f;
    if (a.dweights != nullptr && lane < K) {
      i = __ldg(a.ids + at * K + lane);
      d = __ldg(a.dweights + at * K + lane);
      if (i < 0 || i >= E) {
        i = -1;
        d = 0.0f;
      }
    }
  };
  if (t < n_live) {
    load(t, next, nid, ndw);
    if (nid >= 0) nlk = load_elem<TYPE>(a.logits, t * a.ld + nid);
  }
  for (int64_t after; t < a.T; t = after) {
    after = following(t);
    if (t >= n_live) {
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] = 0.0f;
      store_row<TYPE, N, V>(a.dlogits, t * a.ldd, E, lane, l);
      continue;
    }
    id = nid;
    dw = ndw;
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = next[i];
    lk = nlk;
    const bool more = after < n_live;
    if (more) load(after, next, nid, ndw);
    float r[N], m = kNegInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r[i] = 0.0f;
      m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
    if (db != 0.0f || dz != 0.0f) {
      if (t % kRun == 0) {  // the first group that ends behind t
        int lo = q;
        for (int hi = Q; lo < hi;) {
          const int mid = (lo + hi) >> 1;
          if (st[mid] + cnt[mid] <= t) lo = mid + 1; else hi = mid;
        }
        q = lo;
      } else {
        while (q < Q && st[q] + cnt[q] <= t) ++q;
      }
      if (q < Q && t >= st[q]) {
        if (have != q) {
          have = q;
          const float n = (float)cnt[q], scale = db / n / n;
#pragma unroll
          for (int i = 0; i < N; ++i)
            g[i] = expert_of<V>(i, lane) < E ? scale * (float)__ldg(a.counts + (int64_t)q * E + expert_of<V>(i, lane)) : 0.0f;
        }
        float p[N], rest[N], dot = 0.0f;
        scores<true>(l, m, a.sigmoid, p, rest);
#pragma unroll
        for (int i = 0; i < N; ++i) dot = fmaf(p[i], g[i], dot);
        dot = warp_sum(dot);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          r[i] = p[i] * (g[i] - dot);
          if (a.sigmoid) r[i] *= rest[i];
        }
        if (dz != 0.0f && m != kNegInf) {
          float z = 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            p[i] = fast_exp(l[i] - m);
            z += p[i];
          }
          z = warp_sum(z);
          const float c = dz * (m + __logf(z)) * fast_rcp(z);
#pragma unroll
          for (int i = 0; i < N; ++i) r[i] = fmaf(c, p[i], r[i]);
        }
      }
    }
    if (a.dweights != nullptr) {
      float dk;
      if (a.renorm) {
        const float mk = warp_max(lk);
        const bool soft = !a.sigmoid || mk < kFarBelow;
        const float s = id >= 0 && mk != kNegInf ? (soft ? fast_exp(lk - mk) : sigmoid(lk)) : 0.0f;
        const float sum = warp_sum(s);
        const float u = id >= 0 && mk != kNegInf ? s * fast_rcp(sum) : 0.0f;
        dk = a.scale * u * (dw - warp_sum(u * dw));
        if (a.sigmoid) dk *= sigmoid_rest(lk);
      } else if (a.sigmoid) {
        dk = id >= 0 ? a.scale * dw * sigmoid(lk) * sigmoid_rest(lk) : 0.0f;
      } else {
        float z = 0.0f, p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          p[i] = fast_exp(l[i] - m);
          z += p[i];
        }
        z = warp_sum(z);
        dk = id >= 0 && m != kNegInf ? a.scale * dw * fast_exp(lk - m) * fast_rcp(z) : 0.0f;
        const float c = m == kNegInf ? 0.0f : warp_sum(dk) * fast_rcp(z);
        if (m != kNegInf) {
#pragma unroll
          for (int i = 0; i < N; ++i) r[i] = fmaf(-c, p[i], r[i]);
        }
      }
      // an expert twice in a token: one after the other, in the order of the slots
      const unsigned same = __match_any_sync(0xffffffffu, id >= 0 ? id : -1 - lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
        for (int k = 0; k < K; ++k) {
          if (lane == k && id >= 0) add[id] += dk;
          __syncwarp();
        }
      } else if (id >= 0) {
        add[id] = dk;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (expert_of<V>(i, lane) < E) r[i] += add[expert_of<V>(i, lane)];
      __syncwarp();
      if (id >= 0) add[id] = 0.0f;
      __syncwarp();
    }
    nlk = more && nid >= 0 ? load_elem<TYPE>(a.logits, after * a.ld + nid) : kNegInf;
    store_row<TYPE, N, V>(a.dlogits, t * a.ldd, E, lane, r);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

// Calls f with the element type, the logits a lane holds and its vectors' length as
// constants. Vectors where every row is made of whole aligned ones, of 16 bytes or what
// a lane holds.
template <typename F>
cudaError_t by_shape(int type, int E, bool whole, F f) {
  auto by_v = [&](auto ty, auto n) -> cudaError_t {
    constexpr int kMost = decltype(ty)::value == kF32 ? 4 : 8, kN = decltype(n)::value, kV = kN < kMost ? kN : kMost;
    if constexpr (kV > 1)
      if (whole && E % kV == 0) return f(ty, n, std::integral_constant<int, kV>{});
    return f(ty, n, std::integral_constant<int, 1>{});
  };
  auto by_n = [&](auto ty) -> cudaError_t {
    if (E <= 32) return by_v(ty, std::integral_constant<int, 1>{});
    if (E <= 64) return by_v(ty, std::integral_constant<int, 2>{});
    if (E <= 128) return by_v(ty, std::integral_constant<int, 4>{});
    if (E <= 256) return by_v(ty, std::integral_constant<int, 8>{});
    if (E <= 512) return by_v(ty, std::integral_constant<int, 16>{});
    return by_v(ty, std::integral_constant<int, 32>{});
  };
  if (type == kBF16) return by_n(std::integral_constant<int, kBF16>{});
  if (type == kF16) return by_n(std::integral_constant<int, kF16>{});
  return by_n(std::integral_constant<int, kF32>{});
}
// Rows that start on 16 bytes each.
bool whole_rows(const void* p, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (type == kF32 ? 4 : 2) % 16 == 0;
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int type, int num_sms, cudaStream_t s) {
  return by_shape(type, a.E, whole_rows(a.logits, a.ld, type), [&](auto ty, auto n, auto v) {
    auto kernel = route_kernel<decltype(ty)::value, decltype(n)::value, decltype(v)::value>;
    int per_sm = 0;
    cudaError_t err = occupancy(kernel, kThreads, 0, &per_sm);
    if (err != cudaSuccess) return err;
    const int64_t need = ((int64_t)a.T + kWarps - 1) / kWarps, most = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
    kernel<<<(unsigned)(need < most ? need : most), kThreads, 0, s>>>(a);
    return cudaGetLastError();
  });
}

size_t balance_ws_bytes(int E, int Q) {
  const int64_t slots = balance_slots(Q), slices = (E + 31) / 32;
  return (size_t)(slots * (2 * (int64_t)E + 1) + Q * (slices + 4) + 3) * 4;
}

cudaError_t launch_balance(const BalanceArgs& a, int type, int num_sms, cudaStream_t s) {
  cudaError_t err = by_shape(type, a.E, whole_rows(a.logits, a.ld, type), [&](auto ty, auto n, auto v) {
    auto kernel = balance_parts_kernel<decltype(ty)::value, decltype(n)::value, decltype(v)::value>;
    const size_t smem = (2 * (size_t)a.g.Q + (1 + kWarps) * (size_t)a.E) * 4;
    cudaError_t e = opt_in_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (a.T + 2 * kWarps - 1) / (2 * kWarps);  // two tokens a warp at least
    if (grid > kBalanceParts) grid = kBalanceParts;
    if (grid < 1) grid = 1;
    kernel<<<(unsigned)grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
  });
  if (err != cudaSuccess) return err;
  const bool few = a.g.Q <= kFewGroups;
  const unsigned slices = (unsigned)((a.E + 31) / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(few ? slices : (slices + 3) / 4, (unsigned)a.g.Q);
  cfg.blockDim = dim3(few ? 1024 : 128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? balance_join_kernel<true> : balance_join_kernel<false>, a);
}

cudaError_t launch_route_grad(const RouteGradArgs& a, int type, int num_sms, cudaStream_t s) {
  const bool whole = whole_rows(a.logits, a.ld, type) && whole_rows(a.dlogits, a.ldd, type);
  return by_shape(type, a.E, whole, [&](auto ty, auto n, auto v) {
    auto kernel = route_grad_kernel<decltype(ty)::value, decltype(n)::value, decltype(v)::value>;
    const size_t smem = (2 * (size_t)a.g.Q + kWarps * (size_t)a.E) * 4;
    cudaError_t err = opt_in_smem(kernel, smem);
    if (err != cudaSuccess) return err;
    int per_sm = 0;
    err = occupancy(kernel, kThreads, smem, &per_sm);
    if (err != cudaSuccess) return err;
    const int64_t need = ((int64_t)a.T + kWarps * kRun - 1) / (kWarps * kRun), most = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
    kernel<<<(unsigned)(need < most ? need : most), kThreads, smem, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace moeperm
