// Expert selection from router logits: softmax or sigmoid scores s, keys s + bias, groups of experts, top-k by
// key (ties to the lower expert), weights from the scores; and its gradient with the selection held.
//
// A token is held by G lanes (8, 16 or 32) of a warp, NV consecutive experts a lane, from one read of its
// logits.  The top-k goes by candidates: of the largest keys of both halves of the lanes' experts, sorted over the lanes, the
// k + 1st is a bound that at least k + 1 keys reach and few more do (11 of 256 for k = 8); these are put one after the other in
// shared memory and ranked by counting.  Cross-lane work, which bounds the kernel (with the exponentials), so does not
// grow with k.  The rounds of a maximum over the lanes remain for what the bound does not serve: k + 1 beyond the lanes,
// fewer experts left than that, more than 32 candidates.  The slots' weights are then formed one slot a lane, from
// the logits themselves.
//
// Measured: 65536 tokens of 256 experts, k = 8, 4 of 8 groups, sigmoid, bias, fp32 58 us, 10.6 of them to read and write
// (91 with rounds alone, 136 with every doubt settled for the whole token): issue of ~650 instructions a token, two
// thirds on the ALU, and at the end of the kernel the last tokens in doubt; 8192 of 8, k = 2, 2.4 us; 65536 of 256 in bf16
// without groups and without a bias 25 to 28 us, with one 41 to 59 (sigmoid, renormalised: 44; biases of 0, where many
// keys are equal, 43), and with all logits equal 134 (200 in groups).  16 lanes a token of 256 experts rather than 32: 56
// and 71 us when that was tried.  The gradient of the first 13.3 us where dlogits stay in L2, 5.5 TB/s, 19.8 where they
// do not, 10.9 to read and write.
//
// Which expert wins must not hang on the rounding of a score, so the order is that of the keys in 64 bits:
//   - without a bias and without sums of keys (groups scored by two) the order of the keys is the order of the
//     logits, which are compared as they are (scores that round to the same number have an order, too);
//   - else the keys are formed in 32 bits, and a token in which two keys that follow each other (or the two
//     group scores at the border) are nearer than their error can bridge is done again in 64 bits.
// The second way is rare where logits are spread (about one token in 500 at 256 experts), and the first
// costs nothing, so that no token pays for 64-bit exponentials, of which an SM does few.
//
// The error of a 32-bit key.  exp's approximation is off by 2^-22 and its argument's product by |x| 2^-24,
// relatively; of a sigmoid, s (1 - s) |x| <= 0.23 of that counts, so s is off by less than 2^-21.6 and the sum
// with the bias by 2^-24 of itself: two keys differ wrongly by less than 2^-20.5 + 2^-23 |key|, and
// 2^-19 max(1, |key|) is what is asked for.  A softmax's sum of at most 32 + 5 rounded additions is
// 2^-18.7 off in one direction for all experts, so twice as much is asked for there.  A sum of two keys is off by as much as
// both together and its own rounding, 2^-20.5 + 2^-22 times the larger magnitude of the two, however small it is itself.
// The kernels are built once for fp32 logits (select_fp32.cu) and once for 16-bit ones (select_16.cu), which look up which
// of the two types they have: types looked up in one build cost 10% when that was tried (51 : 57 us, gradient 4.1 : 4.6), a build
// for each of three types most of the time to compile.
#pragma once

#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "grouped.cuh"

namespace moe {

namespace {

constexpr bool kFp32 = MOE_SELECT_FP32;   // set before this file is included
constexpr int kWarps = 4;          // of a block
constexpr int kMaxExpertGroups = 64;

struct SelParams {
  const void* logits;
  const float* bias;               // nullable
  int32_t* idx;
  float* w;
  const float* dw;                 // backward
  void* dl;
  int64_t T;
  int E, k;
  int n, per, top, sum;            // expert groups, experts of one, groups kept, keys summed (1 or 2)
  bool sigmoid, renorm;
  float scale;
  int dtype;                       // of logits and dl
};

// ---- lanes of a token ----------------------------------------------------------------------------

template <int G>
__device__ __forceinline__ uint32_t group_mask(int lane) {
  return G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane & ~(G - 1));
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t mask) {
  if constexpr (G == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(mask, v, o));
    return v;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

template <int G>
__device__ __forceinline__ float group_fmax(float v, uint32_t mask) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
  return v;
}

// Order of floats as order of integers; finite values and infinities lie above 1.
constexpr uint32_t kTaken = 0, kMasked = 1;
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);   // (-0 is 0)
  return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) != 0 ? u ^ 0x80000000u : ~u);
}

// ---- logits --------------------------------------------------------------------------------------

__device__ __forceinline__ float logit(const SelParams& p, int64_t at) {
  if (kFp32) return static_cast<const float*>(p.logits)[at];
  const uint16_t v = static_cast<const uint16_t*>(p.logits)[at];
  return p.dtype == MOE_BF16 ? bf16_lo(v) : __half2float(__ushort_as_half(v));
}

__device__ __forceinline__ uint16_t narrow16(const SelParams& p, float v) {
  return p.dtype == MOE_BF16 ? (uint16_t)pack_bf16(v, 0.f) : __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ void put(const SelParams& p, int64_t at, float v) {
  if (kFp32) static_cast<float*>(p.dl)[at] = v;
  else static_cast<uint16_t*>(p.dl)[at] = narrow16(p, v);
}

template <class T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };
template <class T, int NV> constexpr int vec_of() { return NV * (int)sizeof(T) <= 16 ? NV : 16 / (int)sizeof(T); }

// This lane's experts e0 .. e0 + NV - 1 of the row at `row`; -inf past the last.  Rows start on V elements where E is
// a multiple of V (the array on 16 bytes).
template <class T, int NV, class F>
__device__ __forceinline__ void load_as(const T* row, int e0, int E, float (&x)[NV], F widen) {
  constexpr int V = vec_of<T, NV>();
  if (E % V == 0 && e0 + NV <= E) {
#pragma unroll
    for (int i = 0; i < NV; i += V) {
      const Vec<T, V> r = *reinterpret_cast<const Vec<T, V>*>(row + e0 + i);
#pragma unroll
      for (int j = 0; j < V; ++j) x[i + j] = widen(r.v[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = e0 + i < E ? widen(row[e0 + i]) : -INFINITY;
  }
}

template <int NV>
__device__ __forceinline__ void load_row(const SelParams& p, int64_t row, int e0, float (&x)[NV]) {
  if constexpr (kFp32) {
    load_as(static_cast<const float*>(p.logits) + row, e0, p.E, x, [](float v) { return v; });
  } else {
    uint16_t const* at = static_cast<const uint16_t*>(p.logits) + row;
    const bool bf16 = p.dtype == MOE_BF16;
    load_as(at, e0, p.E, x, [bf16](uint16_t v) { return bf16 ? bf16_lo(v) : __half2float(__ushort_as_half(v)); });
  }
}

template <class T, int NV, class F>
__device__ __forceinline__ void store_as(T* row, int e0, int E, const float (&x)[NV], F narrow) {
  constexpr int V = vec_of<T, NV>();
  if (E % V == 0) {
#pragma unroll
    for (int i = 0; i < NV; i += V) {
      Vec<T, V> r;
#pragma unroll
      for (int j = 0; j < V; ++j) r.v[j] = narrow(x[i + j]);
      if (e0 + i < E) *reinterpret_cast<Vec<T, V>*>(row + e0 + i) = r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < E) row[e0 + i] = narrow(x[i]);
  }
}

template <int NV>
__device__ __forceinline__ void store_row(const SelParams& p, int64_t row, int e0, const float (&x)[NV]) {
  if constexpr (kFp32) store_as(static_cast<float*>(p.dl) + row, e0, p.E, x, [](float v) { return v; });
  else store_as(static_cast<uint16_t*>(p.dl) + row, e0, p.E, x, [&p](float v) { return narrow16(p, v); });
}

template <int NV>
__device__ __forceinline__ void load_bias(const float* bias, int e0, int E, float (&b)[NV]) {
  if (NV % 4 == 0 && E % 4 == 0 && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0) {
#pragma unroll
    for (int i = 0; i < NV; i += 4)
      if (e0 + i < E) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(bias + e0 + i));
        b[i] = v.x;
        b[i + 1] = v.y;
        b[i + 2] = v.z;
        b[i + 3] = v.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < E) b[i] = __ldg(bias + e0 + i);
  }
}

// A warp: n zeros of dl from `at` on, whole rows.
__device__ __forceinline__ void fill_zero(const SelParams& p, int64_t at, int n, int lane) {
  constexpr int size = kFp32 ? 4 : 2;
  uint8_t* to = static_cast<uint8_t*>(p.dl) + at * size;
  if (p.E * size % 16 == 0) {
    for (int i = lane * 16; i < n * size; i += 512) *reinterpret_cast<uint4*>(to + i) = make_uint4(0u, 0u, 0u, 0u);
  } else {
    for (int i = lane; i < n; i += 32) put(p, at + i, 0.f);
  }
}

// (a logit that is -inf masks its expert; NaN too, as far as the selection goes)
__device__ __forceinline__ bool masked(float x) { return !(x > -INFINITY); }

// e^v for keys: a result below 2^-126 is 0.
__device__ __forceinline__ float exp_fast(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * 1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float rcp_fast(float v) {   // of 1 and more
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float sigmoid32(float x) { return __fdiv_rn(1.f, 1.f + expf(-x)); }
// A sigmoid over e^low, low the smaller of 0 and the largest x of a sum: ratios that do not underflow with the sigmoids.
__device__ __forceinline__ float sigmoid_over(float x, float low) {
  return x >= 0.f ? sigmoid32(x) : __fdiv_rn(expf(x - low), 1.f + expf(x));
}

// ---- the same in 64 bits, for a token whose order is in doubt ---------------------------------------

__device__ __forceinline__ void top2_merge(double& a, double& b, double oa, double ob) {
  if (oa > a) {
    b = fmax(a, ob);
    a = oa;
  } else {
    b = fmax(b, oa);
  }
}

// An expert's key in 64 bits; top and sum as of softmax64.
__device__ __noinline__ double key64(const SelParams& p, int64_t row, int e, double top, double sum) {
  const double x = fminf(logit(p, row + e), FLT_MAX);
  const double s = p.sigmoid ? 1. / (1. + exp(-x)) : exp(x - top) / sum;
  return p.bias != nullptr ? s + (double)p.bias[e] : s;
}

// The sum of a token's exponentials, over its lanes (1 with sigmoids).
template <int G, int NV>
__device__ __noinline__ double softmax64(const SelParams& p, int64_t row, int e0, double top, uint32_t lanes) {
  if (p.sigmoid) return 1.;
  double sum = 0.;
  for (int i = 0; i < NV && e0 + i < p.E; ++i) {
    const float x = logit(p, row + e0 + i);
    if (!masked(x)) sum += exp((double)fminf(x, FLT_MAX) - top);
  }
  for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
  return sum;
}

// One token by its G lanes, the slots' experts to who.
template <int G, int NV>
__device__ __noinline__ void select64(const SelParams& p, int64_t t, int lane, int* who) {
  const uint32_t mask = group_mask<G>(lane);
  const int li = lane & (G - 1), e0 = li * NV;
  const int64_t row = t * p.E;
  double key[NV];
  uint32_t out = 0;   // masked experts of this lane, and taken or absent ones
  uint32_t gone = 0;
  double m = -INFINITY, z = 0.;
  for (int i = 0; i < NV; ++i) {
    const float x = e0 + i < p.E ? logit(p, row + e0 + i) : -INFINITY;
    if (e0 + i >= p.E) gone |= 1u << i;
    if (masked(x)) out |= 1u << i;
    key[i] = masked(x) ? -INFINITY : (double)fminf(x, FLT_MAX);
    m = fmax(m, key[i]);
  }
  if (p.sigmoid) {
    for (int i = 0; i < NV; ++i) key[i] = 1. / (1. + exp(-key[i]));
  } else {
    for (int o = G / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(mask, m, o));
    for (int i = 0; i < NV; ++i) {
      key[i] = (out >> i & 1u) != 0 ? 0. : exp(key[i] - m);
      z += key[i];
    }
    for (int o = G / 2; o > 0; o >>= 1) z += __shfl_xor_sync(mask, z, o);
    for (int i = 0; i < NV; ++i) key[i] /= z;
  }
  for (int i = 0; i < NV; ++i) {
    if (p.bias != nullptr && e0 + i < p.E) key[i] += (double)p.bias[e0 + i];
    if (!(key[i] > -INFINITY)) out |= 1u << i;   // (a bias of -inf or NaN masks, too)
  }
  if (p.top < p.n) {
    double score[kMaxExpertGroups];
    for (int g = 0; g < p.n; ++g) {
      double a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < NV; ++i) {
        const int e = e0 + i;
        if (e >= g * p.per && e < (g + 1) * p.per && (out >> i & 1u) == 0) top2_merge(a, b, key[i], -INFINITY);
      }
      for (int o = G / 2; o > 0; o >>= 1)
        top2_merge(a, b, __shfl_xor_sync(mask, a, o), __shfl_xor_sync(mask, b, o));
      score[g] = p.sum == 2 && b > -INFINITY ? a + b : a;
    }
    for (int g = 0; g < p.n; ++g) {
      int above = 0;
      for (int h = 0; h < p.n; ++h) above += score[h] > score[g] || (score[h] == score[g] && h < g);
      if (above < p.top) continue;
      for (int i = 0; i < NV; ++i)
        if (e0 + i >= g * p.per && e0 + i < (g + 1) * p.per) gone |= 1u << i;
    }
  }
  for (int r = 0; r < p.k; ++r) {
    // first the experts that are not masked, then those that are
    double v = -INFINITY;
    int e = 0x7fffffff, cls = 2;
    for (int i = 0; i < NV; ++i) {
      if ((gone >> i & 1u) != 0) continue;
      const int c = out >> i & 1u;
      if (c < cls || (c == 0 && cls == 0 && key[i] > v)) {
        cls = c;
        v = key[i];
        e = e0 + i;
      }
    }
    for (int o = G / 2; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(mask, v, o);
      const int oe = __shfl_xor_sync(mask, e, o), oc = __shfl_xor_sync(mask, cls, o);
      const bool tie = oc == cls && (oc != 0 || ov == v);
      if (oc < cls || (oc == 0 && cls == 0 && ov > v) || (tie && oe < e)) {
        v = ov;
        e = oe;
        cls = oc;
      }
    }
    if (e >= e0 && e < e0 + NV) gone |= 1u << (e - e0);
    if (li == 0) who[r] = e;
  }
}

// ---- selection -----------------------------------------------------------------------------------

constexpr int kMaxCand = 32;       // candidates of a token

// A token's share of shared memory.
template <int G, int NV>
struct Token {
  // its keys, -inf for masked experts: a lane's next to each other, lanes four words further apart than that, so that
  // vectors of eight lanes fall on all banks
  static constexpr int kPad = NV >= 4 ? 4 : 0;
  alignas(16) float keys[G * (NV + kPad)];
  alignas(16) float cand[kMaxCand];   // candidates' keys, -inf past the last
  int e[kMaxCand];                    // and experts
  float top[kMaxCand];                // by rank
  int who[kMaxCand];
  union {
    double wide[kMaxExpertGroups];    // in 64 bits: candidates' keys, or scores
    float scores[2][kMaxExpertGroups];   // of groups that do not fall on lanes, and what they may be off
  };
  __device__ __forceinline__ float& key(int e) { return keys[e + e / NV * kPad]; }
};

// Whether two keys, the larger one first, may stand the other way round.  (Infinities do not.)
__device__ __forceinline__ bool near_by(float hi, float lo, float by) {
  return hi < INFINITY && hi - lo <= by * fmaxf(1.f, fabsf(hi));
}

// The score of a group with the largest keys a >= b, halved where it is the sum of both (b: 0 if there is no second), so that
// finite keys give a finite one; and what it may be off: as much as the keys are, which their sum need not show (1000 and
// -1000 add up to about nothing).  Logits are taken as they are.
template <bool kKeys>
__device__ __forceinline__ float2 score_of(const SelParams& p, float a, float b, float tol) {
  if (!kKeys) return make_float2(a, 0.f);
  b = p.sum == 1 ? a : (b > -INFINITY ? b : 0.f);
  return make_float2(fmaf(0.5f, a, 0.5f * b), tol * fmaxf(0.5f, fmaxf(fabsf(0.5f * a), fabsf(0.5f * b))));
}

// Whether all of a token's experts that are not masked have one logit and one bias (a token of zeros, a router that has
// learned nothing): all its keys are one number then, whatever its bits, and so are sums of as many of them.  Where a
// group's score is of one key and another's of two (`uneven`, in any lane), their order hangs on the key's sign, which its
// 32 bits tell only of a key beyond its error.
template <int G, int NV>
__device__ __noinline__ bool flat(const SelParams& p, int64_t row, Token<G, NV>& token, int lane, int e0, bool uneven, float tol) {
  const uint32_t mine = group_mask<G>(lane);
  // (first their keys in 32 bits, which are at hand: nearly always these differ)
  float lo = INFINITY, hi = -INFINITY, blo = INFINITY, bhi = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float v = token.key(e0 + i);
    hi = fmaxf(hi, v);
    if (v > -INFINITY) lo = fminf(lo, v);
  }
  __syncwarp(mine);
  const float key = group_fmax<G>(hi, mine);
  if (-group_fmax<G>(-lo, mine) != key) return false;
  if ((__ballot_sync(mine, uneven) & mine) != 0 && !(fabsf(key) > tol)) return false;
  lo = INFINITY;
  hi = -INFINITY;
  for (int i = 0; i < NV && e0 + i < p.E; ++i) {
    if (!(token.key(e0 + i) > -INFINITY)) continue;
    const float x = logit(p, row + e0 + i), b = p.bias != nullptr ? p.bias[e0 + i] : 0.f;
    lo = fminf(lo, x);
    hi = fmaxf(hi, x);
    blo = fminf(blo, b);
    bhi = fmaxf(bhi, b);
  }
  __syncwarp(mine);
  return -group_fmax<G>(-lo, mine) == group_fmax<G>(hi, mine) && -group_fmax<G>(-blo, mine) == group_fmax<G>(bhi, mine);
}

// How many groups come before this lane's, by scores in 64 bits of the keys that may be among a group's largest.
// `least`: the smallest key that the group's score counts (-inf: it is of the other key alone); `above`: the answer of the
// scores in 32 bits.
template <int G, int NV>
__device__ __noinline__ int groups_above64(const SelParams& p, int64_t row, Token<G, NV>& token, int lane, int e0, float m,
                                           float least, float tol, int above) {
  bool live = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) live |= token.key(e0 + i) > -INFINITY;
  if (flat<G, NV>(p, row, token, lane, e0, live && least == -INFINITY, tol)) return above;
  const uint32_t mine = group_mask<G>(lane);
  const int lanes = p.per / NV, g = e0 / p.per;
  const double total = softmax64<G, NV>(p, row, e0, m, mine);
  const float from = least - 2.f * tol * fmaxf(1.f, fabsf(least));
  double a = -INFINITY, b = -INFINITY;
  uint32_t need = 0;   // (collected first: the lanes' few then go side by side)
  for (int i = 0; i < NV && e0 + i < p.E; ++i) {
    const float v = token.key(e0 + i);
    if (v > -INFINITY && (least == -INFINITY || v >= from || v == INFINITY)) need |= 1u << i;
  }
  for (; need != 0; need &= need - 1) top2_merge(a, b, key64(p, row, e0 + __ffs(need) - 1, m, total), -INFINITY);
  __syncwarp(mine);
  for (int o = lanes / 2; o > 0; o >>= 1) top2_merge(a, b, __shfl_xor_sync(mine, a, o), __shfl_xor_sync(mine, b, o));
  const double s = p.sum == 2 && b > -INFINITY ? a + b : a;
  above = 0;
  for (int h = 0; h < p.n; ++h) {
    const double o = __shfl_sync(mine, s, h * lanes, G);
    above += h < g ? o >= s : o > s;
  }
  return above;
}

// The same for groups that do not fall on lanes, a group a lane: the groups that go, a bit each, those of this lane's.
template <int G, int NV>
__device__ __noinline__ uint64_t groups_dropped64(const SelParams& p, int64_t row, Token<G, NV>& token, int lane, int e0, float m,
                                                  float tol, bool uneven, uint64_t drop) {
  if (flat<G, NV>(p, row, token, lane, e0, uneven, tol)) return drop;
  const uint32_t mine = group_mask<G>(lane);
  const int li = lane & (G - 1);
  const double total = softmax64<G, NV>(p, row, e0, m, mine);
  __syncwarp(mine);   // (the scores in 32 bits have been read)
  for (int g = li; g < p.n; g += G) {
    float top = -INFINITY, least = -INFINITY;
    for (int e = g * p.per; e < (g + 1) * p.per; ++e) {
      const float v = token.key(e);
      least = fmaxf(least, fminf(top, v));
      top = fmaxf(top, v);
    }
    if (p.sum == 1) least = top;
    const float from = least - 2.f * tol * fmaxf(1.f, fabsf(least));
    double a = -INFINITY, b = -INFINITY;
    for (int e = g * p.per; e < (g + 1) * p.per; ++e) {
      const float v = token.key(e);
      if (v > -INFINITY && (least == -INFINITY || v >= from || v == INFINITY))
        top2_merge(a, b, key64(p, row, e, m, total), -INFINITY);
    }
    token.wide[g] = p.sum == 2 && b > -INFINITY ? a + b : a;
  }
  __syncwarp(mine);
  drop = 0;
  for (int g = li; g < p.n; g += G) {
    const double s = token.wide[g];
    int above = 0;
    for (int h = 0; h < p.n; ++h) above += h < g ? token.wide[h] >= s : token.wide[h] > s;
    if (above >= p.top) drop |= (uint64_t)1 << g;
  }
  return drop;
}

// One key twice by the same logit and bias is no doubt, but a tie.
__device__ __forceinline__ bool same_key(const SelParams& p, int64_t row, int e, int f) {
  return logit(p, row + e) == logit(p, row + f) && (p.bias == nullptr || p.bias[e] == p.bias[f]);
}

// The slots' experts by k rounds of a maximum over the lanes (a whole warp).  Returns whether two keys that follow each
// other are too near.
template <int G, int NV, bool kKeys>
__device__ __noinline__ bool select_rounds(const SelParams& p, int64_t row, Token<G, NV>& token, int lane, uint32_t allowed,
                                           float tol) {
  const int li = lane & (G - 1), e0 = li * NV;
  const uint32_t mine = group_mask<G>(lane);
  uint32_t u[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float v = token.key(e0 + i);
    u[i] = (allowed >> i & 1u) == 0 ? kTaken : (v > -INFINITY ? order_of(v) : kMasked);
  }
  uint32_t before = kTaken;   // the key and the expert of the slot before
  int expert = 0;
  bool doubt = false;
  for (int r = 0; r < p.k + (int)kKeys; ++r) {   // (one more than the slots, for the border)
    uint32_t best = u[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = max(best, u[i]);
    const uint32_t v = group_max<G>(best, 0xffffffffu);
    const int owner = __ffs(__ballot_sync(0xffffffffu, best == v) & mine) - 1;
    int il = 0;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i)
      if (u[i] == v) il = i;
    const int e = __shfl_sync(0xffffffffu, e0 + il, owner);
    if (kKeys && r > 0 && v > kMasked && near_by(value_of(before), value_of(v), tol)) {
      if (r < p.k) {
        doubt |= !same_key(p, row, expert, e);
      } else {   // the border: of all keys that follow
        uint32_t close = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) close |= u[i] > kMasked && near_by(value_of(before), value_of(u[i]), tol) ? 1u << i : 0u;
        bool other = false;
        for (; close != 0; close &= close - 1) other |= !same_key(p, row, expert, e0 + __ffs(close) - 1);
        __syncwarp(mine);
        doubt |= (__ballot_sync(mine, other) & mine) != 0;
      }
    }
    before = v;
    expert = e;
    if (r == p.k) break;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane == owner && i == il) u[i] = kTaken;
    if (lane == owner) token.who[r] = e;
  }
  return doubt;
}

// The order of a token's candidates by keys in 64 bits: whoever may be among the k is one.
template <int G, int NV>
__device__ __noinline__ void rank64(const SelParams& p, int64_t row, Token<G, NV>& token, int lane, int e0, float m,
                                    int count) {
  constexpr int kSlots = 32 / G;
  const int li = lane & (G - 1);
  const uint32_t mine = group_mask<G>(lane);
  const double total = softmax64<G, NV>(p, row, e0, m, mine);
  for (int c = li; c < count; c += G) token.wide[c] = key64(p, row, token.e[c], m, total);
  __syncwarp(mine);
  int rank[kSlots];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int own = q * G + li;
    rank[q] = kMaxCand;
    if (own >= count) continue;
    rank[q] = 0;
    const double v = token.wide[own];
    for (int c = 0; c < count; ++c) rank[q] += c < own ? token.wide[c] >= v : token.wide[c] > v;
  }
#pragma unroll
  for (int q = 0; q < kSlots; ++q)
    if (rank[q] < p.k) token.who[rank[q]] = token.e[q * G + li];
}

// Descending over the token's lanes.
template <int G>
__device__ __forceinline__ float sort_lanes(float v, int li) {
#pragma unroll
  for (int size = 2; size <= G; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      v = ((li & o) == 0) == ((li & size) == 0) ? fmaxf(v, w) : fminf(v, w);
    }
  return v;
}

// The largest G of two values a lane, descending over the lanes.
template <int G>
__device__ __forceinline__ float sort_pairs(float a, float b, int li) {
  a = sort_lanes<G>(a, li);
  b = sort_lanes<G>(b, li);
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, b, G - 1));   // (rises, then falls)
#pragma unroll
  for (int o = G / 2; o > 0; o /= 2) {
    const float w = __shfl_xor_sync(0xffffffffu, a, o);
    a = (li & o) == 0 ? fmaxf(a, w) : fminf(a, w);
  }
  return a;
}

// kKeys: keys are scores (with a bias, or summed), else logits.
template <int G, int NV, bool kKeys>
__global__ void __launch_bounds__(32 * kWarps, NV <= 16 ? 8 : 4) select_kernel(const __grid_constant__ SelParams p) {
  constexpr int kTok = 32 / G;       // tokens of a warp
  constexpr int kSlots = 32 / G;     // slots of a lane, and candidates
  constexpr uint32_t kAll = NV == 32 ? 0xffffffffu : (1u << (NV & 31)) - 1u;
  __shared__ Token<G, NV> shared[kWarps][kTok];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane & (G - 1), e0 = li * NV;
  constexpr uint32_t mask = 0xffffffffu;       // (all tokens of a warp take the same way)
  const uint32_t mine = group_mask<G>(lane);
  const int64_t at = ((int64_t)blockIdx.x * kWarps + warp) * kTok + lane / G;
  const int64_t t = min(at, p.T - 1);   // (lanes past the last token do its work again and store nothing)
  const int64_t row = t * p.E;
  Token<G, NV>& token = shared[warp][lane / G];
  after_previous_kernel();

  float key[NV];   // the logits, then the keys: -inf for masked experts
  load_row<NV>(p, row, e0, key);
  const bool softmax_all = !p.sigmoid && (kKeys || !p.renorm);
  float m = -FLT_MAX, z = 0.f, rz = 0.f;
  bool broken = false;   // a NaN or +inf: the selection goes by the rest, or as if it were the largest number
  if (softmax_all) {
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, key[i]);
    m = fminf(group_fmax<G>(m, mask), FLT_MAX);
#pragma unroll
    for (int i = 0; i < NV; ++i) z += exp_fast(key[i] - m);
    z = group_sum<G>(z, mask);
    broken = !(z <= FLT_MAX);
    if (__any_sync(mask, broken)) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) z += masked(key[i]) ? 0.f : exp_fast(fminf(key[i], FLT_MAX) - m);
      z = group_sum<G>(z, mask);
    }
    rz = z == 0.f ? 0.f : __fdiv_rn(1.f, z);
  }
  uint32_t allowed = e0 >= p.E ? 0u : (p.E - e0 >= NV ? kAll : (1u << (p.E - e0)) - 1u);
  if (kKeys) {
    float bias[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = 0.f;
    if (p.bias != nullptr) load_bias<NV>(p.bias, e0, p.E, bias);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float x = key[i];
      const float k = bias[i] + (p.sigmoid ? rcp_fast(1.f + exp_fast(-x)) : exp_fast(fminf(x, FLT_MAX) - m) * rz);
      key[i] = masked(x) || masked(k) ? -INFINITY : k;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (masked(key[i])) key[i] = -INFINITY;   // (NaN)
  }

  bool doubt = false;   // the same in all lanes of a token
  const float tol = p.sigmoid ? 0x1p-19f : 0x1p-18f;
  if (NV % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NV; i += 4)
      *reinterpret_cast<float4*>(&token.key(e0) + i) = make_float4(key[i], key[i + 1 < NV ? i + 1 : 0], key[i + 2 < NV ? i + 2 : 0],
                                                                   key[i + 3 < NV ? i + 3 : 0]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) token.key(e0 + i) = key[i];
  }
  if (p.top < p.n) {
    // scores of the groups: of masked experts nothing is added, and a group of none else comes last
    const int lanes = p.per / NV;   // of a group
    if (p.per % NV == 0 && (lanes & (lanes - 1)) == 0) {
      float a = -INFINITY, b = -INFINITY;   // the largest two keys of the lane, then of the group
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        b = fmaxf(b, fminf(a, key[i]));
        a = fmaxf(a, key[i]);
      }
      for (int o = lanes / 2; o > 0; o >>= 1) {
        const float oa = __shfl_xor_sync(mask, a, o), ob = __shfl_xor_sync(mask, b, o);
        b = fmaxf(fmaxf(b, ob), fminf(a, oa));
        a = fmaxf(a, oa);
      }
      const float2 score = score_of<kKeys>(p, a, b, tol);
      const float s = score.x;
      const int g = e0 / p.per;   // (of a lane past the last expert: no group's)
      int above = 0;
      for (int h = 0; h < p.n; ++h) {
        const float o = __shfl_sync(mask, s, h * lanes, G);
        above += h < g ? o >= s : o > s;
      }
      if (kKeys) {
        const uint32_t last = __ballot_sync(mask, e0 < p.E && above == p.top - 1) & mine;
        const uint32_t next = __ballot_sync(mask, e0 < p.E && above == p.top) & mine;
        const float sl = __shfl_sync(mask, s, __ffs(last) - 1), sn = __shfl_sync(mask, s, __ffs(next) - 1);
        // no group may cross the border if none reaches the middle between the two at it.  (Where one of these is infinite,
        // so are all on its side of the border, which no rounding moves; other infinite scores reach nowhere or NaN.)
        const float cut = 0.5f * sl + 0.5f * sn, off = score.y;
        const bool reach = e0 < p.E && (above < p.top ? s - off <= cut : s + off >= cut);
        if ((__ballot_sync(mask, reach) & mine) != 0 && sl < INFINITY && sn > -INFINITY)
          above = groups_above64<G, NV>(p, row, token, lane, e0, m, p.sum == 2 ? b : a, tol, above);
        __syncwarp();
      }
      if (above >= p.top) {
        allowed = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = -INFINITY;
      }
    } else {
      // groups that do not fall on lanes: through shared memory, a group a lane
      __syncwarp();
      bool uneven = false;   // a score of one key among those of two
      for (int g = li; g < p.n; g += G) {
        float a = -INFINITY, b = -INFINITY;
        for (int e = g * p.per; e < (g + 1) * p.per; ++e) {
          const float v = token.key(e);
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
        uneven |= p.sum == 2 && a > b && b == -INFINITY;
        const float2 score = score_of<kKeys>(p, a, b, tol);
        token.scores[0][g] = score.x;
        token.scores[1][g] = score.y;
      }
      __syncwarp();
      // how low those kept may reach, and how high those dropped (infinite ones as above)
      float lo = INFINITY, hi = -INFINITY;
      uint64_t drop = 0;
      for (int g = li; g < p.n; g += G) {
        const float s = token.scores[0][g], off = token.scores[1][g];
        int above = 0;
        for (int h = 0; h < p.n; ++h) above += h < g ? token.scores[0][h] >= s : token.scores[0][h] > s;
        if (above < p.top) {
          lo = fminf(lo, s - off);
        } else {
          hi = fmaxf(hi, s + off);
          drop |= (uint64_t)1 << g;
        }
      }
      if (kKeys) {
        lo = -group_fmax<G>(-lo, mask);
        hi = group_fmax<G>(hi, mask);
        if (lo <= hi && lo < INFINITY && hi > -INFINITY)
          drop = groups_dropped64<G, NV>(p, row, token, lane, e0, m, tol, uneven, drop);
        __syncwarp();
      }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) drop |= __shfl_xor_sync(mask, drop, o);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int g = min((e0 + i) / p.per, p.n - 1);
        if ((drop >> g & 1u) != 0) {
          allowed &= ~(1u << i);
          key[i] = -INFINITY;   // (masked ones of the groups that stay: only the rounds below choose them)
        }
      }
    }
  }

  // The bound: the k + 1st of the largest keys of half lanes, less what keys may be off
  bool rounds = p.k >= G;
  int count = 0;   // candidates of the token
  if (!rounds) {
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < NV; ++i) best[2 * i / NV] = fmaxf(best[2 * i / NV], key[i]);
    const float sorted = NV > 1 ? sort_pairs<G>(best[0], best[1], li) : sort_lanes<G>(best[0], li);
    float bound = __shfl_sync(mask, sorted, p.k, G);
    rounds = !(fabsf(bound) < INFINITY);
    // (not past the lowest number: masked experts, groups that go and lanes past the last expert have -inf and are none)
    if (kKeys) bound = fmaxf(bound - 2.f * tol * fmaxf(1.f, fabsf(bound)), -FLT_MAX);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) bits |= key[i] >= bound ? 1u << i : 0u;
    int upto = __popc(bits);
    int to = -upto;
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      const int v = __shfl_up_sync(mask, upto, o, G);
      if (li >= o) upto += v;
    }
    to += upto;
    count = __shfl_sync(mask, upto, G - 1, G);
    rounds = __any_sync(mask, rounds || count > kMaxCand);
    if (!rounds) {
      for (; bits != 0; bits &= bits - 1) token.e[to++] = e0 + __ffs(bits) - 1;
      __syncwarp();
      // ranks: candidates lie in the order of the experts, so that among equal ones the earlier comes first
      float own_key[kSlots];
      int own_e[kSlots], rank[kSlots];
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        const bool in = q * G + li < count;
        own_e[q] = in ? token.e[q * G + li] : 0;
        own_key[q] = in ? token.key(own_e[q]) : -INFINITY;
        token.cand[q * G + li] = own_key[q];
        rank[q] = 0;
      }
      __syncwarp();
      const int most = G == 32 ? count : __reduce_max_sync(mask, count);
      for (int c = 0; c < most; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(token.cand + c);
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          if (q > 0 && most <= q * G) break;
          const int at = q * G + li - c;
          rank[q] += (at > 0 ? v.x >= own_key[q] : v.x > own_key[q]) + (at > 1 ? v.y >= own_key[q] : v.y > own_key[q]) +
                     (at > 2 ? v.z >= own_key[q] : v.z > own_key[q]) + (at > 3 ? v.w >= own_key[q] : v.w > own_key[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (q * G + li < count) {
          token.top[rank[q]] = own_key[q];
          token.who[rank[q]] = own_e[q];
        }
      __syncwarp();
      if (kKeys) {
        // from the first key to the first one, from the k-th on, that is far enough from the next: two that are near and not
        // the same may stand the other way round, if only by what lies between them
        uint32_t near = 0, unlike = 0;   // a bit a key, against the next (there are more than k)
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          const int j = q * G + li;
          const bool close = j + 1 < count && near_by(token.top[j], token.top[j + 1], tol);
          const bool other = close && !same_key(p, row, token.who[j], token.who[j + 1]);
          near |= (__ballot_sync(mask, close) & mine) >> (lane - li) << (q * G & 31);
          unlike |= (__ballot_sync(mask, other) & mine) >> (lane - li) << (q * G & 31);
        }
        const int last = __ffs(~(near >> (p.k - 1))) + p.k - 2;   // (the last candidate's bit is 0)
        doubt = (unlike & ((2u << last) - 1u)) != 0;
      }
    }
  }
  if (rounds) {
    doubt = select_rounds<G, NV, kKeys>(p, row, token, lane, allowed, tol);
    if (kKeys) {   // its candidates are all experts that are left, if these are not too many
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) bits |= key[i] > -INFINITY ? 1u << i : 0u;
      int upto = __popc(bits);
      int to = -upto;
#pragma unroll
      for (int o = 1; o < G; o <<= 1) {
        const int v = __shfl_up_sync(mask, upto, o, G);
        if (li >= o) upto += v;
      }
      to += upto;
      count = __shfl_sync(mask, upto, G - 1, G);
      if (doubt && count <= kMaxCand)
        for (; bits != 0; bits &= bits - 1) token.e[to++] = e0 + __ffs(bits) - 1;
      __syncwarp();
    }
  }
  if (kKeys && doubt) {
    if (count > kMaxCand) select64<G, NV>(p, t, lane, token.who);
    else rank64<G, NV>(p, row, token, lane, e0, m, count);
  }
  __syncwarp();
  int sidx[kSlots];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) sidx[q] = q * G + li < p.k ? token.who[q * G + li] : 0;

  // weights, a slot a lane
  float xs[kSlots], M = -INFINITY;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const bool slot = q * G + li < p.k;
    xs[q] = slot ? logit(p, row + sidx[q]) : -INFINITY;
    M = fmaxf(M, xs[q]);
  }
  if (broken) rz = __int_as_float(0x7fffffff);
  float s[kSlots], sum = 0.f;
  if (p.renorm) M = group_fmax<G>(M, mask);
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    s[q] = 0.f;
    if (q * G >= p.k) continue;
    const bool slot = q * G + li < p.k;
    if (!p.renorm) s[q] = p.sigmoid ? sigmoid32(xs[q]) : expf(xs[q] - m) * rz;
    else if (M == -INFINITY) s[q] = xs[q] == -INFINITY ? 0.f : xs[q];   // (0 or NaN)
    else s[q] = p.sigmoid ? sigmoid_over(xs[q], fminf(M, 0.f)) : expf(xs[q] - M);
    if (!slot) s[q] = 0.f;
    sum += s[q];
  }
  if (p.renorm) {
    sum = group_sum<G>(sum, mask);
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
      if (q * G < p.k) s[q] = sum == 0.f ? 0.f : __fdiv_rn(s[q], sum);
  }
  if (at >= p.T) return;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int j = q * G + li;
    if (j >= p.k) continue;
    p.idx[t * p.k + j] = sidx[q];
    p.w[t * p.k + j] = s[q] * p.scale;
  }
}

// ---- gradient ------------------------------------------------------------------------------------

// d_j, a slot a lane:
//   renormalised      d_j = w_j (c_j - sum_m c_m h_m), sigmoid: times 1 - s_j
//   not renormalised  d_j = scale c_j s_j (1 - s_j); softmax: d_j = scale p_j (c_j - sum_m c_m p_m), and
//                     -scale p_e sum_m c_m p_m for the experts of no slot
// The rows are first written as of tokens without slots, in whole vectors, and then at the slots' experts, by the same
// warp: no lane looks through its experts for every slot (46 us at 65536 tokens of 256 experts).  Only a softmax that is not
// renormalised reads a whole row, and has lanes enough for it; else the slots alone say how many lanes a token
// has (16 for 8 slots: 22 us).  An expert in several slots gets the sum of their terms, in slot order, from
// the first of them.
template <int G, int NV, bool kDense>
__global__ void __launch_bounds__(32 * kWarps, NV <= 16 ? 12 : 6) select_bwd_kernel(const __grid_constant__ SelParams p) {
  constexpr int kTok = 32 / G, kSlots = kDense ? 32 / G : 1;   // (sparse: k is at most G)
  constexpr uint32_t mask = 0xffffffffu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane & (G - 1), e0 = li * NV;
  const int64_t at = ((int64_t)blockIdx.x * kWarps + warp) * kTok + lane / G;
  const int64_t t = min(at, p.T - 1);
  const int64_t row = t * p.E;
  after_previous_kernel();

  int e[kSlots];
  float c[kSlots], xs[kSlots];
  float M = -INFINITY;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int j = q * G + li;
    e[q] = -1;
    c[q] = 0.f;
    if (j < p.k) {
      e[q] = p.idx[t * p.k + j];
      c[q] = p.dw[t * p.k + j];
    }
    if (e[q] < 0 || e[q] >= p.E) e[q] = -1;   // (no expert: a slot without weight)
  }
  float v[NV], m = -FLT_MAX, rz = 0.f;
  if constexpr (kDense) {
    load_row<NV>(p, row, e0, v);
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, v[i]);
    m = group_fmax<G>(m, mask);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = __expf(v[i] - m);
      z += v[i];
    }
    z = group_sum<G>(z, mask);
    rz = z == 0.f ? 0.f : __fdiv_rn(1.f, z);
  } else {   // zeros, of all the warp's tokens, which lie on end
    const int64_t first = at - lane / G;
    if (first < p.T) fill_zero(p, first * p.E, (int)min((int64_t)kTok, p.T - first) * p.E, lane);
  }
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    xs[q] = e[q] >= 0 ? logit(p, row + e[q]) : -INFINITY;
    if (xs[q] == -INFINITY) c[q] = 0.f;   // (whatever the gradient of a weight that is nothing)
    M = fmaxf(M, xs[q]);
  }
  if (p.renorm) M = group_fmax<G>(M, mask);
  float h[kSlots], sum = 0.f, dot = 0.f;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    h[q] = 0.f;
    if (q * G >= p.k) continue;
    if (kDense) h[q] = __expf(xs[q] - m) * rz;
    else if (!p.renorm) h[q] = sigmoid32(xs[q]);
    else if (M == -INFINITY) h[q] = 0.f;
    else h[q] = p.sigmoid ? sigmoid_over(xs[q], fminf(M, 0.f)) : expf(xs[q] - M);
    if (e[q] < 0) h[q] = 0.f;
    sum += h[q];
  }
  if (p.renorm) {
    sum = group_sum<G>(sum, mask);
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
      if (q * G < p.k) h[q] = sum == 0.f ? 0.f : __fdiv_rn(h[q], sum);
  }
#pragma unroll
  for (int q = 0; q < kSlots; ++q) dot += c[q] * h[q];
  if (p.renorm || kDense) dot = group_sum<G>(dot, mask);
  float d[kSlots];
  bool first[kSlots];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    first[q] = e[q] >= 0;
    d[q] = 0.f;
    if (q * G >= p.k) continue;
    d[q] = h[q] == 0.f ? 0.f : p.scale * h[q] * (p.renorm ? c[q] - dot : c[q]);
    if (!kDense && p.sigmoid) d[q] *= sigmoid32(-xs[q]);   // (of a slot without an expert 1)
  }
  // whether an expert comes twice among a token's slots
  bool twice = false;
#pragma unroll
  for (int q = 0; q < kSlots; ++q)
#pragma unroll
    for (int r = 0; r <= q; ++r) {
      if (q * G >= p.k) break;
      for (int o = r == q ? 1 : 0; o < G; ++o) {
        const int other = __shfl_xor_sync(mask, e[r], o);
        twice |= other == e[q] && other >= 0;
      }
    }
  if (__any_sync(mask, twice)) {
    float total[kSlots] = {};
#pragma unroll
    for (int r = 0; r < kSlots; ++r)
      for (int rr = 0; rr < G; ++rr) {
        if (r * G + rr >= p.k) break;
        const int ej = __shfl_sync(mask, e[r], rr, G);
        const float dj = __shfl_sync(mask, d[r], rr, G);
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
          if (ej == e[q]) {
            total[q] += dj;
            if (r * G + rr < q * G + li) first[q] = false;
          }
      }
#pragma unroll
    for (int q = 0; q < kSlots; ++q) d[q] = total[q];
  }
  if constexpr (kDense) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] *= -rz * (p.scale * dot);
    if (at < p.T) store_row<NV>(p, row, e0, v);
  }
  __syncwarp();
  if (at >= p.T) return;
#pragma unroll
  for (int q = 0; q < kSlots; ++q)
    if (first[q]) put(p, row + e[q], kDense ? d[q] - h[q] * (p.scale * dot) : d[q]);
}

// ---- host side -----------------------------------------------------------------------------------

SelParams params_of(const Select& c) {
  SelParams p{};
  p.T = c.T;
  p.E = c.E;
  p.k = c.k;
  p.n = c.n;
  p.per = c.E / c.n;
  p.top = c.top;
  p.sum = c.sum;
  p.sigmoid = c.sigmoid;
  p.renorm = c.renorm;
  p.scale = c.scale;
  p.dtype = c.dtype;
  return p;
}

// A functor's call<G, NV>() for the number of experts, and lanes enough for more than `k` candidates' bounds.
template <class F>
cudaError_t by_experts(int E, int k, F f) {
  if (k < 8) {
    if (E <= 8) return f.template call<8, 1>();
    if (E <= 16) return f.template call<8, 2>();
    if (E <= 32) return f.template call<8, 4>();
  }
  if (k < 16) {
    if (E <= 16) return f.template call<16, 1>();
    if (E <= 32) return f.template call<16, 2>();
    if (E <= 64) return f.template call<16, 4>();
    if (E <= 128) return f.template call<16, 8>();
    if (E <= 256) return f.template call<16, 16>();
  }
  if (E <= 32) return f.template call<32, 1>();
  if (E <= 64) return f.template call<32, 2>();
  if (E <= 128) return f.template call<32, 4>();
  if (E <= 256) return f.template call<32, 8>();
  if (E <= 512) return f.template call<32, 16>();
  return f.template call<32, 32>();
}

int64_t blocks_of(int64_t T, int per_warp) { return (T + kWarps * per_warp - 1) / (kWarps * per_warp); }

struct Forward {
  const SelParams& p;
  cudaStream_t s;
  template <int G, int NV>
  cudaError_t call() const {
    const bool keys = p.bias != nullptr || (p.top < p.n && p.sum == 2);
    const int64_t blocks = blocks_of(p.T, 32 / G);
    return keys ? launch_after(select_kernel<G, NV, true>, blocks, 32 * kWarps, 0, 1, s, p)
                : launch_after(select_kernel<G, NV, false>, blocks, 32 * kWarps, 0, 1, s, p);
  }
};

struct Backward {
  const SelParams& p;
  cudaStream_t s;
  template <int G, int NV>
  cudaError_t call() const {
    if (!p.sigmoid && !p.renorm) return launch<G, NV, true>();
    return p.k <= 8 ? launch<8, 1, false>() : p.k <= 16 ? launch<16, 1, false>() : launch<32, 1, false>();
  }
  template <int G, int NV, bool kDense>
  cudaError_t launch() const {
    return launch_after(select_bwd_kernel<G, NV, kDense>, blocks_of(p.T, 32 / G), 32 * kWarps, 0, 1, s, p);
  }
};

cudaError_t forward(const Select& c, const void* logits, const float* bias, int32_t* idx, float* w,
                          cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  SelParams p = params_of(c);
  p.logits = logits;
  p.bias = bias;
  p.idx = idx;
  p.w = w;
  prof_mark(kKSelect, s, true);
  const cudaError_t e = by_experts(c.E, c.k, Forward{p, s});
  prof_mark(kKSelect, s, false);
  return e;
}

cudaError_t backward(const Select& c, const void* logits, const int32_t* idx, const float* dw, void* dl,
                              cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  SelParams p = params_of(c);
  p.logits = logits;
  p.idx = const_cast<int32_t*>(idx);
  p.dw = dw;
  p.dl = dl;
  prof_mark(kKSelectBwd, s, true);
  const cudaError_t e = by_experts(c.E, c.k, Backward{p, s});
  prof_mark(kKSelectBwd, s, false);
  return e;
}

}  // namespace

}  // namespace moe
