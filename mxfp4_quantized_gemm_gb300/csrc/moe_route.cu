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
// bytes (T * E logits): 2000 a token and 62 us for 16384 tokens of 256 experts
// in 8 groups when the lanes searched their values in every round.
//
// The choice is exact: where two neighbours of the order up to place k + 1 (or
// the last group taken and the first left out) lie nearer than the dropped
// bits and the fp32 evaluation's error bound, the warp decides the row again
// in 64 bits.  Equal inputs are no such case: their order is by the index.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

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
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ double from_key(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & ~(1ull << 63)) : ~k));
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
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// The score of logit x, given the row's largest logit and 1 / the sum of the
// exponentials relative to it (softmax).
template <typename F>
__device__ __forceinline__ F score_of(bool sigmoid, float x, float m, F sum) {
  if (sigmoid) return F(1) / (F(1) + exp_of(-static_cast<F>(x)));
  if (x == -INFINITY || !(sum > F(0))) return F(0);
  return (x == m ? F(1) : exp_of(static_cast<F>(x) - static_cast<F>(m))) / sum;
}

// Keeps the higher two of (best, next) and (b, n).
template <typename F>
__device__ __forceinline__ void higher_two(F& best, F& next, F b, F n) {
  const F low = best < b ? best : b;
  best = best < b ? b : best;
  next = next < n ? n : next;
  next = next < low ? low : next;
}

// The value of a group whose highest two compared values are best and next.
template <typename F>
__device__ __forceinline__ F group_value(int top, F best, F next) {
  return top == 2 && next != -static_cast<F>(INFINITY) ? best + next : best;
}

// Decides one row in 64 bits.  Lane l holds elements l * V .. l * V + V - 1 of
// the row, so the lowest lane and place of equal values is the lowest index.
// At the end lane r < k holds the r-th choice: its index (-1: none), its logit
// and its score.
template <int V>
__device__ __forceinline__ void decide_exactly(const RouteArgs& a, const float (&x)[V], int lane, int& idx, float& xsel,
                                               double& ssel) {
  using F = double;
  using K = uint64_t;
  const F ninf = -static_cast<F>(INFINITY);
  const bool biased = a.bias != nullptr, sigmoid = a.sigmoid != 0;
  float m = -INFINITY;
  F sum = 0;
  if (!sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, x[j]);
    m = from_key(warp_max(key_of(m)));
    if (m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (x[j] != -INFINITY) sum += x[j] == m ? F(1) : exp_of(static_cast<F>(x[j]) - static_cast<F>(m));
    }
    sum = warp_sum(sum);
  }
  // what is compared; sums of logits would not order as sums of scores do
  const bool by_score = a.groups > 1 && !biased && a.top == 2;
  K key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = lane * V + j;
    F c = static_cast<F>(x[j]);
    if (biased && i < a.E) c = score_of<F>(sigmoid, x[j], m, sum) + static_cast<F>(__ldg(a.bias + i));
    key[j] = key_of(x[j] == -INFINITY || !(c == c) ? ninf : c);
  }
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const int span = size / V;                     // lanes of a group, where groups are whole lanes
    const bool whole = span * V == size && (span & (span - 1)) == 0 && span > 0;
    K gkey = key_of(ninf);
    int group = lane;                              // the group whose value this lane holds
    if (whole) {
      F best = ninf, next = ninf;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        F v = from_key(key[j]);
        if (by_score && v != ninf) v = score_of<F>(sigmoid, x[j], m, sum);
        higher_two(best, next, v, ninf);
      }
      for (int o = 1; o < span; o <<= 1) {
        const F b = __shfl_xor_sync(kAll, best, o), n = __shfl_xor_sync(kAll, next, o);
        higher_two(best, next, b, n);
      }
      gkey = key_of(group_value(a.top, best, next));
      group = lane / span;
    } else {
      for (int g = 0; g < a.groups; ++g) {
        F best = ninf, next = ninf;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int i = lane * V + j;
          if (i >= g * size && i < (g + 1) * size) {
            F v = from_key(key[j]);
            if (by_score && v != ninf) v = score_of<F>(sigmoid, x[j], m, sum);
            higher_two(best, next, v, ninf);
          }
        }
        for (int o = 1; o < 32; o <<= 1) {
          const F b = __shfl_xor_sync(kAll, best, o), n = __shfl_xor_sync(kAll, next, o);
          higher_two(best, next, b, n);
        }
        if (lane == g) gkey = key_of(group_value(a.top, best, next));
      }
    }
    if (group >= a.groups) gkey = 0;               // (lanes past the last group)
    uint32_t kept = 0;
    for (int r = 0; r < a.keep; ++r) {
      const K top = warp_max(gkey);
      const int g = __shfl_sync(kAll, group, __ffs(__ballot_sync(kAll, gkey == top)) - 1);
      kept |= 1u << g;
      if (group == g) gkey = 0;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = whole ? group : (lane * V + j) / size;
      if (g >= a.groups || !((kept >> g) & 1u)) key[j] = key_of(ninf);
    }
  }

  // k rounds of the maximum over the warp and the lowest lane that has it
  idx = -1;
  xsel = 0.f;
  const K none = key_of(ninf);
  for (int r = 0; r < a.k; ++r) {
    K best = key[0];
    int at = 0;
    float bx = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
        bx = x[j];
      }
    const K top = warp_max(best);
    if (top <= none) break;
    const int who = __ffs(__ballot_sync(kAll, best == top)) - 1;
    const int i = __shfl_sync(kAll, lane * V + at, who);
    const float xv = __shfl_sync(kAll, bx, who);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane == who && j == at) key[j] = 0;
    if (lane == r) {
      idx = i;
      xsel = xv;
    }
  }
  ssel = idx >= 0 ? score_of<F>(sigmoid, xsel, m, sum) : F(0);
}

// The weight of this lane's choice.  Renormalised weights use scores relative
// to the largest chosen one, which do not vanish where all scores are small.
template <typename F>
__device__ __forceinline__ float weight_of(const RouteArgs& a, int idx, float xsel, F ssel) {
  const bool on = idx >= 0;
  if (!a.renorm) return on ? static_cast<float>(static_cast<F>(a.scale) * ssel) : 0.f;
  const float m = from_key(warp_max(key_of(on ? xsel : -INFINITY)));
  F e = 0;
  if (on) {
    if (a.sigmoid) {
      const F c = m < 0.f ? static_cast<F>(m) : F(0);
      e = F(1) / (exp_of(c) + exp_of(c - static_cast<F>(xsel)));
    } else {
      e = xsel == m ? F(1) : exp_of(static_cast<F>(xsel) - static_cast<F>(m));
    }
  }
  const F total = warp_sum(e);
  return on ? static_cast<float>(static_cast<F>(a.scale) * e / total) : 0.f;
}

template <int V>
__device__ __noinline__ void decide_in_64_bits(const RouteArgs& a, const float (&x)[V], int lane, int& idx, float& w) {
  float xsel;
  double ssel;
  decide_exactly<V>(a, x, lane, idx, xsel, ssel);
  w = weight_of<double>(a, idx, xsel, ssel);
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

// key_of(v) with the place j in its lowest five bits, the lower place higher;
// 0 for what is switched off.
constexpr uint32_t kPlace = 31u;
__device__ __forceinline__ uint32_t placed_key(float v, int j) {
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

__device__ __forceinline__ float logit_at(const RouteArgs& a, int t, int i) {
  const int64_t at = static_cast<int64_t>(t) * a.ld + i;
  return a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.x)[at]) : static_cast<const float*>(a.x)[at];
}

// Decides row t in fp32, as decide_exactly does.  Returns whether a comparison
// that mattered was too near for fp32.
template <int V>
__device__ __forceinline__ bool decide(const RouteArgs& a, int t, const float (&x)[V], int lane, int& idx, float& xsel,
                                       float& ssel) {
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
  // Fast scores err by less than 2^-20 of the largest possible one, `unit`:
  // the exponential of -v errs by (2 + 1.2 v) 2^-23 e^-v < 2^-21.
  const float unit = sigmoid ? 1.f : sum > 0.f ? __fdividef(1.f, sum) : 0.f;
  auto fast_score = [&](float v) {
    return sigmoid ? __fdividef(1.f, 1.f + __expf(-v)) : (v == m ? 1.f : __expf(v - m)) * unit;
  };
  if (biased) {
    float b[V];
    load_bias<V>(a, lane, b);
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = x[j] > -INFINITY ? placed_key(fast_score(x[j]) + b[j], j) : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = placed_key(x[j], j);
  }
  sort_down<V>(key);
  bool near = false;

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const int span = size / V;                     // lanes of a group, where groups are whole lanes
    const bool whole = span * V == size && (span & (span - 1)) == 0 && span > 0;
    uint32_t gkey = 0;
    float gerr = 0.f;
    int group = lane;                              // the group whose value this lane holds
    // Of the values that stand for a key: the dropped bits (2^-18) and the scores' errors.
    auto value_of = [&](uint32_t k, float& err) {
      if (k == 0) return -INFINITY;
      const float c = from_key(k & ~kPlace);
      const float v = by_score ? fast_score(c) : c;
      err += biased ? 0x1p-18f * fabsf(c) + 0x1p-20f * unit
                    : by_score ? 0x1p-20f * unit + 0x1p-17f * fabsf(c) * v : 0x1p-18f * fabsf(c);
      return v;
    };
    auto set_group = [&](uint32_t best, uint32_t next) {
      float e = 0.f;
      const float v1 = value_of(best, e), v2 = a.top == 2 ? value_of(next, e) : -INFINITY;
      gkey = best != 0 ? key_of(group_value(a.top, v1, v2)) : 0u;
      gerr = e + 0x1p-22f * fabsf(v1);
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
    uint32_t kept = 0;
    float last = -INFINITY, last_err = 0.f;
    for (int r = 0; r <= a.keep; ++r) {
      const uint32_t top = warp_max(gkey);
      if (top == 0) break;
      const int who = __ffs(__ballot_sync(kAll, gkey == top)) - 1;
      const int g = __shfl_sync(kAll, group, who);
      const float v = from_key(top), err = __shfl_sync(kAll, gerr, who);
      if (r < a.keep) {
        kept |= 1u << g;
        last = v;
        last_err = err;
        if (group == g) gkey = 0;
      } else if (last - v <= last_err + err) {
        near = true;
      }
    }
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
  if (lane < a.k && idx >= 0 && i2 >= 0) {
    if (biased) {
      const float c1 = from_key(mine), c2 = from_key(key2);
      const bool same = xsel == x2 && __ldg(a.bias + idx) == __ldg(a.bias + i2);
      near = near || (c1 - c2 <= 0x1p-18f * (fabsf(c1) + fabsf(c2)) + 0x1p-19f * unit && !same);
    } else {
      near = near || (mine == key2 && xsel != x2);
    }
  }
  ssel = idx >= 0 && !a.renorm ? score_of<float>(sigmoid, xsel, m, sum) : 0.f;
  return __any_sync(kAll, near);
}

// This lane's V logits of token t, a NaN as -inf (it is never chosen).
template <int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int t, int lane, float (&x)[V]) {
  const int64_t at = static_cast<int64_t>(t) * a.ld + lane * V;
  constexpr int kVec = V < 4 ? V : 4;
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
        x[j] = a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.x)[at + j]) : static_cast<const float*>(a.x)[at + j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = x[j] == x[j] ? x[j] : -INFINITY;
}

template <int V>
__global__ void __launch_bounds__(128, V <= 8 ? 8 : V <= 16 ? 5 : 2) moe_route_kernel(const __grid_constant__ RouteArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  if (t >= a.T) return;   // warp-uniform; the kernel has no block barrier
  float x[V];
  load_row<V>(a, t, lane, x);
  int idx;
  float xsel, ssel, w;
  if (decide<V>(a, t, x, lane, idx, xsel, ssel))
    decide_in_64_bits<V>(a, x, lane, idx, w);
  else
    w = weight_of<float>(a, idx, xsel, ssel);
  if (lane < a.k) {
    const int64_t o = static_cast<int64_t>(t) * a.k + lane;
    a.ids[o] = idx;
    a.weights[o] = w;
  }
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteProblem& p, const DeviceInfo& dev, cudaStream_t s) {
  (void)dev;
  const RouteArgs a{p.logits, p.bias, p.ld, p.weights, p.ids, p.T, p.E, p.top_k, p.sigmoid, p.n_group, p.topk_group,
                    p.group_top, p.renormalize, p.bf16,
                    (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 && p.ld % 8 == 0, (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0, p.scale};
  const int grid = static_cast<int>(ceil_div(p.T, 4));
  if (p.E <= 32) return launch_pdl(moe_route_kernel<1>, grid, 128, 0, s, a);
  if (p.E <= 64) return launch_pdl(moe_route_kernel<2>, grid, 128, 0, s, a);
  if (p.E <= 128) return launch_pdl(moe_route_kernel<4>, grid, 128, 0, s, a);
  if (p.E <= 256) return launch_pdl(moe_route_kernel<8>, grid, 128, 0, s, a);
  if (p.E <= 512) return launch_pdl(moe_route_kernel<16>, grid, 128, 0, s, a);
  return launch_pdl(moe_route_kernel<32>, grid, 128, 0, s, a);
}

}  // namespace mx
