// Router of a mixture of experts: scores, choice and weights of each token.
//
//   s_i = softmax(x)_i or sigmoid(x_i);  c_i = s_i + bias_i
//   with groups: the topk_group groups whose `group_top` highest c sum
//   highest keep their experts; the top_k experts of highest c are chosen,
//   equal ones by the lower index; weight = scale * s_i (/ sum of the chosen).
//
// One warp per token, E / 32 neighbouring values per lane in registers: the
// row is read once and every reduction is a warp's.  A lane sorts the
// order-preserving integer images of its c, whose lowest five bits give way to
// the place (so a compare-exchange is one maximum and one minimum); a choice
// then is a maximum over the lanes' first keys (redux), and the lowest lane
// that has it gives up its first key.  Instructions bound the kernel, not the
// bytes (T * E logits): 1122 a token and 28.3 us for 16384 tokens of 256 experts
// in 8 groups, 6.2 us for 8192 of 128 without groups, 4.8 us for 16 (2000 a
// token and 62 us when the lanes searched their values in every round).
//
// The choice is exact: where two neighbours of the order up to place k + 1 (or
// a group taken and one left out) lie nearer than the dropped bits and the fp32
// evaluation's error bound, the warp decides the row again in pairs of fp32, and
// where that does not settle it either, in fp64.  Equal inputs are no such case:
// their order is by the index; but where the first one left out has the inputs of
// the last choice, all that are left out are held against it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "gemm_common.cuh"
#include "internal.h"
#include "moe.h"
#include "ptx.cuh"

namespace mx {

namespace {

struct RouteArgs {
  const void* x;
  const float* bias;
  int64_t ld;
  float* weights;
  int32_t* ids;
  int T, E, k, sigmoid, groups, keep, top, renorm, bf16, vec, bias_vec;
  float scale;
};

constexpr uint32_t kAll = 0xFFFFFFFFu;

// Order-preserving images of floating numbers: larger number, larger key, -0
// as +0, never 0 (the key of what has been taken).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// The score of logit x, given the row's largest logit and the sum of the
// exponentials relative to it (softmax).
__device__ __forceinline__ float score_of(bool sigmoid, float x, float m, float sum) {
  if (sigmoid) return 1.f / (1.f + expf(-x));
  return sum > 0.f ? (x == m ? 1.f : expf(x - m)) / sum : 0.f;
}

// ---- Rows that fp32 cannot decide are decided again in more bits: in pairs
// of fp32 (high + low part, together to 2^-40), and the very few that these
// leave open in fp64.  (A 64-bit operation of this GPU takes some hundred
// cycles: in fp64 alone one such row took 17 us, as long as all the others.)
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair quick_sum(float a, float b) {   // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  return quick_sum(p, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.h, b.h, -p))));
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair reciprocal(Pair a) {            // one Newton step from fp32's
  const float q = __frcp_rn(a.h);
  const float r = __fmaf_rn(-a.l, q, __fmaf_rn(-a.h, q, 1.f));
  return quick_sum(q, __fmul_rn(q, r));
}
__device__ __forceinline__ double mul(double a, double b) { return a * b; }
__device__ __forceinline__ double add(double a, double b) { return a + b; }
__device__ __forceinline__ double reciprocal(double a) { return 1.0 / a; }

// e^(x.h + x.l) for -80 <= x <= 80, to 2^-41: x = n ln 2 + r, |r| <= 0.35, with
// ln 2 in three parts of which the first has 14 bits (its products with n are
// exact); the Taylor sum of e^r to r^12 / 12!, whose terms from r^6 on need
// one fp32 only.
__device__ __forceinline__ Pair exp_pair(Pair x) {
  constexpr float kLn2a = 0x1.62e0p-1f, kLn2b = 0x1.0bfbe8p-15f, kLn2c = 0x1.cf79acp-40f;
  const float n = rintf(__fmul_rn(x.h, 1.44269504f));
  const float a = __fmaf_rn(-n, kLn2a, x.h);
  const float p = __fmul_rn(n, kLn2b), e = __fmaf_rn(n, kLn2b, -p);
  Pair r = two_sum(a, -p);
  r = quick_sum(r.h, __fadd_rn(__fmaf_rn(-n, kLn2c, __fsub_rn(r.l, e)), x.l));
  float t = 0x1.1eed8ep-29f;                                     // 1 / 12!
  t = __fmaf_rn(t, r.h, 0x1.ae6456p-26f);
  t = __fmaf_rn(t, r.h, 0x1.27e4fcp-22f);
  t = __fmaf_rn(t, r.h, 0x1.71de3ap-19f);
  t = __fmaf_rn(t, r.h, 0x1.a01a02p-16f);
  t = __fmaf_rn(t, r.h, 0x1.a01a02p-13f);
  t = __fmaf_rn(t, r.h, 0x1.6c16c2p-10f);                        // 1 / 6!
  Pair s = {t, 0.f};
  s = add({0x1.111112p-7f, -0x1.dddddep-32f}, mul(s, r));        // 1 / 5!
  s = add({0x1.555556p-5f, -0x1.555556p-30f}, mul(s, r));
  s = add({0x1.555556p-3f, -0x1.555556p-28f}, mul(s, r));
  s = add({0.5f, 0.f}, mul(s, r));
  s = add({1.f, 0.f}, mul(s, r));
  s = add({1.f, 0.f}, mul(s, r));
  const float scale = __int_as_float((127 + static_cast<int>(n)) << 23);
  return {__fmul_rn(s.h, scale), __fmul_rn(s.l, scale)};
}

// e^(x - m), 0 below e^-80 in pairs, and the sigmoid of x, as it is at -80 and
// 80 beyond these in pairs (2^-115: far below what pairs tell apart near 1; the
// sums of two such scores and the same bias are equal there, so near).
__device__ __noinline__ void exp_of_difference(float x, float m, Pair& y) {
  y = {x == m ? 1.f : 0.f, 0.f};
  if (x == m || x == -INFINITY) return;
  const Pair d = two_sum(x, -m);
  if (d.h >= -80.f) y = exp_pair(d);
}
__device__ __noinline__ void exp_of_difference(float x, float m, double& y) {
  y = x == m ? 1.0 : x == -INFINITY ? 0.0 : exp(static_cast<double>(x) - static_cast<double>(m));
}
__device__ __noinline__ void sigmoid_of(float x, Pair& y) {
  y = reciprocal(add({1.f, 0.f}, exp_pair({fminf(fmaxf(-x, -80.f), 80.f), 0.f})));
}
__device__ __noinline__ void sigmoid_of(float x, double& y) { y = 1.0 / (1.0 + exp(-static_cast<double>(x))); }

// s + b of a score and a bias; infinities of b stay.
__device__ __forceinline__ Pair plus_bias(Pair s, float b) {
  return isinf(b) ? Pair{b, 0.f} : add(s, Pair{b, 0.f});
}
__device__ __forceinline__ double plus_bias(double s, float b) { return s + static_cast<double>(b); }

// Order-preserving 64-bit images (-0 as +0), never 0; that of -inf is the lowest.
__device__ __forceinline__ uint64_t key_of(Pair v) {
  return (static_cast<uint64_t>(key_of(v.h)) << 32) | key_of(v.l);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  if (b == 1ull << 63) b = 0;
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ void from_key(uint64_t k, Pair& v) {
  v = {from_key(static_cast<uint32_t>(k >> 32)), from_key(static_cast<uint32_t>(k))};
}
__device__ __forceinline__ void from_key(uint64_t k, double& v) {
  v = __longlong_as_double(static_cast<long long>((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}
__device__ __forceinline__ Pair shuffled(Pair v, int o) {
  return {__shfl_xor_sync(kAll, v.h, o), __shfl_xor_sync(kAll, v.l, o)};
}
__device__ __forceinline__ double shuffled(double v, int o) { return __shfl_xor_sync(kAll, v, o); }
__device__ __forceinline__ float rounded(Pair v) { return v.h; }
__device__ __forceinline__ float rounded(double v) { return static_cast<float>(v); }
// Whether pairs leave open which of a >= b is higher, scores being good to
// `error`; never so in fp64.
__device__ __forceinline__ bool open(Pair a, Pair b, float error) {
  return (a.h - b.h) + (a.l - b.l) <= error + 0x1p-44f * (fabsf(a.h) + fabsf(b.h));
}
__device__ __forceinline__ bool open(double, double, float) { return false; }
// The key of a value that is `by` more than key k's (an infinite one stays).
__device__ __forceinline__ uint64_t moved(uint64_t k, float by) {
  Pair v;
  from_key(k, v);
  return key_of(isfinite(v.h) ? add(v, Pair{by, 0.f}) : Pair{v.h, 0.f});
}

__device__ __forceinline__ float logit_at(const RouteArgs& a, int t, int i) {
  const int64_t at = static_cast<int64_t>(t) * a.ld + i;
  return a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.x)[at]) : static_cast<const float*>(a.x)[at];
}

// Whether the groups of the mask have the same best logits (a.top of them),
// where these alone decide (one bias for all their experts, or none): then they
// are equal in any arithmetic, and their order is by the index.
__device__ __noinline__ bool equal_groups(const RouteArgs& a, int t, int lane, uint32_t groups) {
  const int size = a.E / a.groups;
  uint32_t best0 = 0, next0 = 0, high = 0, low = 0;   // of the first group; of all biases and of their inverted keys
  bool same = true;
#pragma unroll 1
  for (uint32_t m = groups; m != 0; m &= m - 1) {
    const int g = __ffs(m) - 1;
    uint32_t best = 0, next = 0;
    auto meet = [&](uint32_t b, uint32_t n) {
      next = max(max(next, n), min(best, b));
      best = max(best, b);
    };
#pragma unroll 1
    for (int i = g * size + lane; i < (g + 1) * size; i += 32) {
      const float x = logit_at(a, t, i), b = a.bias != nullptr ? __ldg(a.bias + i) : 0.f;
      if (!(x > -INFINITY && b > -INFINITY)) continue;
      meet(key_of(x), 0u);
      high = max(high, key_of(b));
      low = max(low, ~key_of(b));
    }
    __syncwarp();
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) meet(__shfl_xor_sync(kAll, best, o), __shfl_xor_sync(kAll, next, o));
    if (m == groups) {
      best0 = best;
      next0 = next;
    }
    same = same && best == best0 && (a.top == 1 || next == next0);
  }
  return same && warp_max(high) == ~warp_max(low);
}

// Decides row t in numbers F (Pair or double).  Lane l holds elements l * V ..
// l * V + V - 1 of the row, so the lowest lane and place of equal values is the
// lowest index.  At the end lane r < k holds the r-th choice: its index (-1:
// none), its logit and its score.  Returns whether a comparison that mattered
// stayed open.
template <int V, typename F>
__device__ __forceinline__ bool decide_in(const RouteArgs& a, int t, int lane, int& idx, float& xsel, float& ssel) {
  const bool biased = a.bias != nullptr, sigmoid = a.sigmoid != 0;
  constexpr uint64_t none = 0;                     // the key of what is switched off
  float x[V];
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float v = lane * V + j < a.E ? logit_at(a, t, lane * V + j) : -INFINITY;
    x[j] = v == v ? v : -INFINITY;
    m = fmaxf(m, x[j]);
  }
  m = from_key(warp_max(key_of(m)));
  // what is compared; sums of logits would not order as sums of scores do
  const bool by_score = a.groups > 1 && !biased && a.top == 2;
  F s[V];
  float unit = 1.f;                                // softmax: 1 / the sum
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (sigmoid)
      sigmoid_of(x[j], s[j]);
    else
      exp_of_difference(x[j], m, s[j]);
  }
  if (!sigmoid && m > -INFINITY) {
    F sum = s[0];
#pragma unroll
    for (int j = 1; j < V; ++j) sum = add(sum, s[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = add(sum, shuffled(sum, o));
    const F r = reciprocal(sum);
    unit = rounded(r);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = mul(s[j], r);
  }
  uint64_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float b = biased && lane * V + j < a.E ? __ldg(a.bias + lane * V + j) : 0.f;
    const bool on = x[j] > -INFINITY && b > -INFINITY;   // (a NaN bias switches off too)
    key[j] = !on ? none : biased ? key_of(plus_bias(s[j], b)) : static_cast<uint64_t>(key_of(x[j])) << 32;
  }
  const float error = 0x1p-39f * unit;
  bool near = false;
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const int span = size / V;                     // lanes of a group, where groups are whole lanes
    const bool whole = span * V == size && (span & (span - 1)) == 0 && span > 0;
    uint64_t best = none, next = none;
    auto meet = [&](uint64_t b, uint64_t n) {
      next = max(max(next, n), min(best, b));
      best = max(best, b);
    };
    auto compared = [&](int j) { return by_score && key[j] != none ? key_of(s[j]) : key[j]; };
    float slack = 0.f;                             // how far the group's value can be off
    auto value = [&]() {                           // the key of the group's value
      if (best == none) return best;
      F v1, v2;
      from_key(best, v1);
      slack = error + 0x1p-44f * fabsf(rounded(v1));
      if (a.top == 1 || next == none) return best;
      from_key(next, v2);
      slack += error + 0x1p-44f * fabsf(rounded(v2));   // (the sum may be far smaller than either)
      return key_of(isinf(rounded(v1)) || isinf(rounded(v2)) ? v1 : add(v1, v2));
    };
    uint64_t gkey = none;
    int group = lane;                              // the group whose value this lane holds
    if (whole) {
#pragma unroll
      for (int j = 0; j < V; ++j) meet(compared(j), none);
      for (int o = 1; o < span; o <<= 1) meet(__shfl_xor_sync(kAll, best, o), __shfl_xor_sync(kAll, next, o));
      gkey = value();
      group = lane / span;
    } else {
#pragma unroll 1
      for (int g = 0; g < a.groups; ++g) {
        best = next = none;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if ((lane * V + j) / size == g) meet(compared(j), none);
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) meet(__shfl_xor_sync(kAll, best, o), __shfl_xor_sync(kAll, next, o));
        if (lane == g) gkey = value();
      }
    }
    if (group >= a.groups) gkey = none;            // (lanes past the last group)
    const uint64_t mine = gkey;
    uint32_t kept = 0;
#pragma unroll 1
    for (int r = 0; r < a.keep; ++r) {
      const uint64_t top = warp_max(gkey);
      if (top == none) break;
      const int g = __shfl_sync(kAll, group, __ffs(__ballot_sync(kAll, gkey == top)) - 1);
      kept |= 1u << g;
      if (group == g) gkey = none;
    }
    if (std::is_same_v<F, Pair> && (biased || by_score)) {
      // the lowest that a group taken can be, the highest that one left out can be
      const bool taken = mine != none && ((kept >> (group & 31)) & 1u), left = mine != none && !taken;
      const uint64_t low = taken ? moved(mine, -slack) : ~0ull, high = left ? moved(mine, slack) : 0ull;
      const uint64_t lowest = ~warp_max(~low), highest = warp_max(high);
      if (highest >= lowest) {
        const bool in = (taken && low <= highest) || (left && high >= lowest);
        near = !equal_groups(a, t, lane, __reduce_or_sync(kAll, in ? 1u << (group & 31) : 0u));
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = (lane * V + j) / size;
      if (g >= a.groups || !((kept >> g) & 1u)) key[j] = none;
    }
  }
  // k rounds of the maximum over the warp and the lowest lane that has it
  idx = -1;
  xsel = 0.f;
  ssel = 0.f;
  uint64_t mine = none;                            // lane r: the key of choice r
#pragma unroll 1
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = key[0];
    int at = 0;
    float bs = rounded(s[0]);
#pragma unroll
    for (int j = 1; j < V; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
        bs = rounded(s[j]);
      }
    const uint64_t top = warp_max(best);
    if (top == none) break;
    const int who = __ffs(__ballot_sync(kAll, best == top)) - 1;
    const int i = __shfl_sync(kAll, lane * V + at, who);
    const float sv = __shfl_sync(kAll, bs, who);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane == who && j == at) key[j] = none;
    if (lane == r) {
      mine = top;
      idx = i;
      ssel = sv;
    }
  }
  if (idx >= 0) xsel = logit_at(a, t, idx);
  if (biased) {
    // neighbours among the chosen; the last of them against all that are left out
    // (the highest of these may be equal to it, with the same inputs, and hide
    // others that are near)
    const float bsel = idx >= 0 ? __ldg(a.bias + idx) : 0.f;
    const uint64_t key2 = __shfl_down_sync(kAll, mine, 1), last = __shfl_sync(kAll, mine, a.k - 1);
    const float x2 = __shfl_down_sync(kAll, xsel, 1), b2 = __shfl_down_sync(kAll, bsel, 1);
    const float xlast = __shfl_sync(kAll, xsel, a.k - 1), blast = __shfl_sync(kAll, bsel, a.k - 1);
    auto close = [&](uint64_t k1, uint64_t k2) {
      F v1, v2;
      from_key(k1, v1);
      from_key(k2, v2);
      return open(v1, v2, error);
    };
    if (lane < a.k - 1 && key2 != none) near = near || (close(mine, key2) && !(xsel == x2 && bsel == b2));
    if (last != none) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (key[j] != none && close(last, key[j]))
          near = near || !(xlast == x[j] && blast == __ldg(a.bias + lane * V + j));
    }
  }
  return __any_sync(kAll, near);
}

// The weight of this lane's choice.  Renormalised weights use scores relative
// to the largest chosen one, which do not vanish where all scores are small.
__device__ __forceinline__ float weight_of(const RouteArgs& a, int idx, float xsel, float ssel) {
  const bool on = idx >= 0;
  if (!a.renorm) return on ? a.scale * ssel : 0.f;
  const float m = from_key(warp_max(key_of(on ? xsel : -INFINITY)));
  float e = 0.f;
  if (on) {
    if (a.sigmoid) {
      const float c = fminf(m, 0.f);
      e = 1.f / (expf(c) + expf(c - xsel));
    } else {
      e = xsel == m ? 1.f : expf(xsel - m);
    }
  }
  const float total = warp_sum(e);
  return on ? a.scale * e / total : 0.f;
}

// A row that fp32 cannot decide, and its weights.
template <int V, typename F>
__device__ __noinline__ bool decide_again(const RouteArgs& a, int t, int lane, int& idx, float& w) {
  float xsel, ssel;
  const bool near = decide_in<V, F>(a, t, lane, idx, xsel, ssel);
  w = weight_of(a, idx, xsel, ssel);
  return near;
}

// This lane's V biases (zeros past E).
template <int V>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int lane, float (&b)[V]) {
  const float* p = a.bias + lane * V;
  if (V % 4 == 0 && a.bias_vec && lane * V + V <= a.E) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + j));
      b[j] = v.x;
      b[j + 1] = v.y;
      b[j + 2] = v.z;
      b[j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = lane * V + j < a.E ? __ldg(p + j) : 0.f;
  }
}

// key_of(v) with the place j of V in its lowest bits, the lower place higher;
// 0 for what is switched off.
constexpr int place_bits(int V) {
  int n = 0;
  while ((1 << n) < V) ++n;
  return n;
}
constexpr uint32_t place_mask(int V) { return (1u << place_bits(V)) - 1u; }
template <int V>
__device__ __forceinline__ uint32_t placed_key(float v, int j) {
  constexpr uint32_t kPlace = place_mask(V);
  return v > -INFINITY ? (key_of(v) & ~kPlace) | (kPlace - j) : 0u;   // (a NaN is switched off too)
}

// Descending order of a lane's V keys: Batcher's odd-even merge sort.
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q >= V) continue;
          if ((i + j) / (2 * p) != (i + j + q) / (2 * p)) continue;
          const uint32_t hi = max(k[i + j], k[i + j + q]), lo = min(k[i + j], k[i + j + q]);
          k[i + j] = hi;
          k[i + j + q] = lo;
        }
}

// Decides row t in fp32, as decide_in does.  Returns whether a comparison that
// mattered was too near for fp32.
template <int V>
__device__ __forceinline__ bool decide(const RouteArgs& a, int t, const float (&x)[V], int lane, int& idx, float& xsel,
                                       float& ssel) {
  constexpr uint32_t kPlace = place_mask(V);       // bits of a key that hold the place
  constexpr float kDropped = (kPlace + 1) * 0x1p-23f;   // what they can be of a value
  const bool biased = a.bias != nullptr, sigmoid = a.sigmoid != 0;
  const bool by_score = a.groups > 1 && !biased && a.top == 2;
  float m = -INFINITY, sum = 0.f;
  uint32_t key[V];
  if (!sigmoid && (biased || by_score || !a.renorm)) {
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, x[j]);
    m = from_key(warp_max(key_of(m)));
    if (m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < V; ++j) sum += x[j] == m ? 1.f : __expf(x[j] - m);
    }
    sum = warp_sum(sum);
  }
  // What fast scores are off by, in units of 2^-23.  The exponential of -v is good to
  // 2 + 1.7 v of it, its argument's rounding counted in.  Sigmoid: s (1 - s) times
  // that, below 1, the division's 2 and the sum's rounding: below 4.  Softmax, each
  // score: 2 of the largest possible one, `unit`, by the exponential and half of one by the
  // product: below 3.  What all scores have in common, of each: by their sum the mean
  // of its terms' errors by their weight (with n terms beside the largest at most that
  // of n equal ones: 4.5 for n = 31, 1 more for twice as many) and half of V + 4 (its
  // additions), by the division 2.  That moves the comparison of two near c by their
  // scores' difference only, which is that of their biases.  (16384 tokens with a
  // bias, of 256 / 64 experts: 21.5 / 11.8 us; 23.7 / 13.0 with the whole of `unit`
  // in its place, 20.9 / 11.2 without, which is wrong.)
  const float unit = sigmoid ? 1.f : sum > 0.f ? __fdividef(1.f, sum) : 0.f;
  const float common = sigmoid || !biased ? 0.f : (8.5f + place_bits(V) + 0.5f * V) * 0x1p-23f;
  const float error = (sigmoid ? 4.f : 3.f) * 0x1p-23f * unit;
  auto fast_score = [&](float v) {
    return sigmoid ? __fdividef(1.f, 1.f + __expf(-v)) : (v == m ? 1.f : __expf(v - m)) * unit;
  };
  if (biased) {
    float b[V];
    load_bias<V>(a, lane, b);
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = x[j] > -INFINITY ? placed_key<V>(fast_score(x[j]) + b[j], j) : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = placed_key<V>(x[j], j);
  }
  sort_down<V>(key);
  bool near = false;

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const int span = size / V;                     // lanes of a group, where groups are whole lanes
    const bool whole = span * V == size && (span & (span - 1)) == 0 && span > 0;
    // a group's value that is a logit of 16 bits has lost nothing to the place
    // (8192 tokens of 256 without bias: 9.9 us; 18.8 when equal ones were decided again)
    const bool exact = a.bf16 && !biased && a.top == 1;
    uint32_t gkey = 0;
    float gerr = 0.f;
    int group = lane;                              // the group whose value this lane holds
    // Of the values that stand for a key: the dropped bits and the scores' errors.
    auto value_of = [&](uint32_t k, float& err) {
      if (k == 0) return -INFINITY;
      const float c = from_key(k & ~kPlace);
      const float dropped = kDropped * fabsf(c);
      if (!by_score) {
        err += biased ? dropped + error + common * unit : dropped;
        return c;
      }
      // (of large logits the dropped bits are not small beside 1)
      const float v = fast_score(c);
      err += error + (dropped < 0.5f ? 2.f * dropped * v : fast_score(c + dropped) - v);
      return v;
    };
    auto set_group = [&](uint32_t best, uint32_t next) {
      float e = 0.f;
      const float v1 = value_of(best, e), v2 = a.top == 2 ? value_of(next, e) : -INFINITY;
      gkey = best != 0 ? key_of(v2 > -INFINITY ? v1 + v2 : v1) : 0u;
      gerr = exact ? 0.f : e + 0x1p-22f * fabsf(v1);
    };
    if (whole) {
      uint32_t best = key[0], next = V > 1 ? key[V > 1 ? 1 : 0] : 0u;
      for (int o = 1; o < span; o <<= 1) {
        const uint32_t b = __shfl_xor_sync(kAll, best, o), n = __shfl_xor_sync(kAll, next, o);
        next = max(max(next, n), min(best, b));
        best = max(best, b);
      }
      set_group(best, next);
      group = lane / span;
    } else {
      for (int g = 0; g < a.groups; ++g) {
        uint32_t best = 0, next = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int i = lane * V + static_cast<int>(kPlace - (key[j] & kPlace));
          if (key[j] != 0 && i >= g * size && i < (g + 1) * size) {
            next = max(next, min(best, key[j]));
            best = max(best, key[j]);
          }
        }
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t b = __shfl_xor_sync(kAll, best, o), n = __shfl_xor_sync(kAll, next, o);
          next = max(max(next, n), min(best, b));
          best = max(best, b);
        }
        if (lane == g) set_group(best, next);
      }
    }
    if (group >= a.groups) gkey = 0;               // (lanes past the last group)
    const uint32_t mine = gkey;
    uint32_t kept = 0;
    for (int r = 0; r < a.keep; ++r) {
      const uint32_t top = warp_max(gkey);
      if (top == 0) break;
      const int g = __shfl_sync(kAll, group, __ffs(__ballot_sync(kAll, gkey == top)) - 1);
      kept |= 1u << g;
      if (group == g) gkey = 0;
    }
    // the lowest that a group taken can be, the highest that one left out can be:
    // errors differ, and the sum of the best two may be far smaller than they
    const bool taken = (kept >> (group & 31)) & 1u;
    const float v = from_key(mine);
    const bool finite = fabsf(v) < INFINITY;
    const uint32_t low = mine != 0 && taken ? key_of(finite ? v - gerr : v) : kAll;
    const uint32_t high = mine != 0 && !taken ? key_of(finite ? v + gerr : v) : 0u;
    const uint32_t lowest = __reduce_min_sync(kAll, low), highest = warp_max(high);
    near = highest > lowest || (highest == lowest && !exact);
    if (whole) {
      if (!((kept >> (group & 31)) & 1u) || group >= a.groups) key[0] = 0;   // what follows a first key of 0 is not met
    } else {
      bool cut = false;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int g = (lane * V + static_cast<int>(kPlace - (key[j] & kPlace))) / size;
        if (key[j] != 0 && !((kept >> (g & 31)) & 1u)) {
          key[j] = 0;
          cut = true;
        }
      }
      if (__any_sync(kAll, cut)) sort_down<V>(key);
    }
  }

  near = __any_sync(kAll, near);
  // k rounds, and one more to see how near the first one left out is
  uint32_t mine = 0, after = 0;                    // lane r: what stands for choice r; every lane: for the one left out
  int iafter = -1;
  idx = -1;
  for (int r = 0; r <= a.k; ++r) {
    const uint32_t first = key[0] & ~kPlace;        // (a place counts within its lane only)
    const uint32_t top = warp_max(first);
    if (top == 0) break;
    const int who = __ffs(__ballot_sync(kAll, first == top)) - 1;
    const int i = __shfl_sync(kAll, lane * V + static_cast<int>(kPlace - (key[0] & kPlace)), who);
    if (r == a.k) {
      after = top;
      iafter = i;
      break;
    }
    if (lane == r) {
      mine = top;
      idx = i;
    }
    if (lane == who) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1];
      key[V - 1] = 0;
    }
  }
  xsel = idx >= 0 ? logit_at(a, t, idx) : 0.f;
  uint32_t key2 = __shfl_down_sync(kAll, mine, 1);
  int i2 = __shfl_down_sync(kAll, idx, 1);
  float x2 = __shfl_down_sync(kAll, xsel, 1);
  if (lane == a.k - 1) {
    key2 = after;
    i2 = iafter;
    if (i2 >= 0) x2 = logit_at(a, t, i2);
  }
  bool close = false, alike = false;               // alike: near, but of the same inputs
  auto tolerance = [&](float c) { return kDropped * fabsf(c) + error; };
  if (lane < a.k && idx >= 0 && i2 >= 0) {
    if (biased) {
      const float c1 = from_key(mine), c2 = from_key(key2);
      const float b1 = __ldg(a.bias + idx), b2 = __ldg(a.bias + i2);
      close = c1 - c2 <= tolerance(c1) + tolerance(c2) + common * fabsf(b1 - b2);
      alike = close && xsel == x2 && b1 == b2;
    } else {
      close = mine == key2;
      alike = close && xsel == x2;
    }
    close = close && !alike;
  }
  near = near || __any_sync(kAll, close);
  // Where the first one left out has the inputs of the last choice, one that is
  // near may stand behind it: all that are left are looked at.  (Keys of 16-bit
  // logits are exact.)
  if (!near && !(a.bf16 && !biased) && __shfl_sync(kAll, alike, a.k - 1)) {
    const uint32_t klast = __shfl_sync(kAll, mine, a.k - 1);
    const float xlast = __shfl_sync(kAll, xsel, a.k - 1), c1 = from_key(klast);
    const float blast = biased ? __ldg(a.bias + __shfl_sync(kAll, idx, a.k - 1)) : 0.f;
#pragma unroll 1
    for (int left = V; left > 0 && key[0] != 0; --left) {
      const uint32_t k2 = key[0] & ~kPlace;
      const int i = lane * V + static_cast<int>(kPlace - (key[0] & kPlace));
      const float c2 = from_key(k2), b2 = biased ? __ldg(a.bias + i) : 0.f;
      if (biased ? c1 - c2 <= tolerance(c1) + tolerance(c2) + common * fabsf(blast - b2) : k2 == klast)
        near = near || logit_at(a, t, i) != xlast || b2 != blast;
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1];
      key[V - 1] = 0;
    }
  }
  ssel = idx >= 0 && !a.renorm ? score_of(sigmoid, xsel, m, sum) : 0.f;
  return __any_sync(kAll, near);
}

// This lane's V logits of token t, a NaN as -inf (it is never chosen).
template <int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int t, int lane, float (&x)[V]) {
  const int64_t at = static_cast<int64_t>(t) * a.ld + lane * V;
  constexpr int kVec = V % 4 == 0 ? 4 : V % 2 == 0 ? 2 : 1;
  if (a.vec && lane * V + V <= a.E) {              // V logits at once, 4 at most
#pragma unroll
    for (int j = 0; j < V; j += kVec) {
      if (a.bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(a.x) + at + j;
        uint32_t w[2] = {0, 0};
        if constexpr (kVec == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[0] = v.x;
          w[1] = v.y;
        } else if constexpr (kVec == 2) {
          w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          w[0] = *p;
        }
#pragma unroll
        for (int q = 0; q < kVec; ++q)
          x[j + q] = __uint_as_float((q & 1) ? (w[q >> 1] & 0xFFFF0000u) : (w[q >> 1] << 16));
      } else {
        const float* p = static_cast<const float*>(a.x) + at + j;
        if constexpr (kVec == 4) {
          const float4 v = *reinterpret_cast<const float4*>(p);
          x[j] = v.x;
          x[j + 1] = v.y;
          x[j + 2] = v.z;
          x[j + 3] = v.w;
        } else if constexpr (kVec == 2) {
          const float2 v = *reinterpret_cast<const float2*>(p);
          x[j] = v.x;
          x[j + 1] = v.y;
        } else {
          x[j] = *p;
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = -INFINITY;
      if (lane * V + j < a.E)
        x[j] = a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.x)[at + j])
                      : static_cast<const float*>(a.x)[at + j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = x[j] == x[j] ? x[j] : -INFINITY;
}

// (Blocks an SM for few logits a lane: what the usual path needs, so that the rows
// that are decided again do not take them registers: 16384 x 64 12.2 us at 8.)
template <int V>
__global__ void __launch_bounds__(128, V == 1 ? 12 : V == 2 ? 10 : V == 3 ? 9 : V <= 8 ? 8 : V <= 16 ? 5 : 2)
    moe_route_kernel(const __grid_constant__ RouteArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  if (t >= a.T) return;   // warp-uniform; the kernel has no block barrier
  float x[V];
  load_row<V>(a, t, lane, x);
  int idx;
  float xsel, ssel, w;
  if (decide<V>(a, t, x, lane, idx, xsel, ssel)) {
    if (decide_again<V, Pair>(a, t, lane, idx, w)) decide_again<V, double>(a, t, lane, idx, w);
  } else {
    w = weight_of(a, idx, xsel, ssel);
  }
  if (lane < a.k) {
    const int64_t o = static_cast<int64_t>(t) * a.k + lane;
    a.ids[o] = idx;
    a.weights[o] = w;
  }
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteProblem& p, cudaStream_t s) {
  const RouteArgs a{p.logits, p.bias, p.ld, p.weights, p.ids, p.T, p.E, p.top_k, p.sigmoid, p.n_group, p.topk_group,
                    p.group_top, p.renormalize, p.bf16,
                    (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 && p.ld % 8 == 0,
                    (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0, p.scale};
  const int grid = static_cast<int>(ceil_div(p.T, 4));
  // Logits a lane: as few as hold the row, so that the groups of the usual numbers
  // of experts are whole lanes (8192 tokens, 8 groups of 160: four lanes of five
  // each, 14.3 us, 33.6 with eight a lane; of 384: 27 with twelve, 66 with
  // sixteen), or the next power of two where only that makes them so.
  const int size = p.E / p.n_group;
  auto whole = [&](int v) { return size % v == 0 && ((size / v) & (size / v - 1)) == 0; };
  int pow2 = 1;
  while (32 * pow2 < p.E) pow2 *= 2;
  int v = 1;
  for (int n : {2, 3, 4, 5, 6, 8, 12, 16, 32})
    if (32 * v < p.E) v = n;
  if (p.n_group > 1 && !whole(v) && whole(pow2)) v = pow2;
  switch (v) {
    case 1: return launch_pdl(moe_route_kernel<1>, grid, 128, 0, s, a);
    case 2: return launch_pdl(moe_route_kernel<2>, grid, 128, 0, s, a);
    case 3: return launch_pdl(moe_route_kernel<3>, grid, 128, 0, s, a);
    case 4: return launch_pdl(moe_route_kernel<4>, grid, 128, 0, s, a);
    case 5: return launch_pdl(moe_route_kernel<5>, grid, 128, 0, s, a);
    case 6: return launch_pdl(moe_route_kernel<6>, grid, 128, 0, s, a);
    case 8: return launch_pdl(moe_route_kernel<8>, grid, 128, 0, s, a);
    case 12: return launch_pdl(moe_route_kernel<12>, grid, 128, 0, s, a);
    case 16: return launch_pdl(moe_route_kernel<16>, grid, 128, 0, s, a);
    default: return launch_pdl(moe_route_kernel<32>, grid, 128, 0, s, a);
  }
}

}  // namespace mx
