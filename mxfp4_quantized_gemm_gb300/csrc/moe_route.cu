// Router of a mixture of experts: scores, choice and weights of each token.
//
//   s_i = softmax(x)_i or sigmoid(x_i);  c_i = s_i + bias_i
//   with groups: the topk_group groups whose `group_top` highest c sum
//   highest keep their experts; the top_k experts of highest c are chosen,
//   equal ones by the lower index; weight = scale * s_i (/ sum of the chosen).
//
// One warp per token, E / 32 neighbouring values per lane in registers: the
// row is read once and every reduction is a warp's.  A choice takes k rounds
// of a 32-bit integer maximum over the warp (redux) on the order-preserving
// image of c; the lowest lane that has it has the lowest index.  Instructions
// bound the kernel, not the bytes (T * E logits).
//
// The choice is exact: without a bias the logits themselves are compared (the
// scores rise with them).  With a bias the compared sums are rounded, so
// where two neighbours of the order up to place k + 1 (or the last group
// taken and the first left out) lie nearer than the fp32 evaluation's error
// bound, the warp decides the row again in 64 bits.
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
  int T, E, k, sigmoid, groups, keep, top, renorm, bf16, vec;
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

template <typename F> struct Keys;
template <> struct Keys<float> { using T = uint32_t; };
template <> struct Keys<double> { using T = uint64_t; };

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
__device__ __forceinline__ F group_value(int top, F best, F next, F& mag) {
  const F ninf = -static_cast<F>(INFINITY);
  F v = best;
  mag = best < 0 ? -best : best;
  if (top == 2 && next != ninf) {
    v += next;
    mag += next < 0 ? -next : next;
  }
  return v;
}

// Decides one row.  Lane l holds elements l * V .. l * V + V - 1 of the row,
// so the lowest lane and place of equal values is the lowest index.  At the
// end lane r < k holds the r-th choice: its index (-1: none), its logit and its
// score.  Returns whether a comparison that mattered was nearer than the fp32
// evaluation's error.
template <typename F, int V>
__device__ __forceinline__ bool decide(const RouteArgs& a, const float (&x)[V], int lane, int& idx, float& xsel, F& ssel) {
  using K = typename Keys<F>::T;
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
  // Error bound of a compared value: scores err by the exponential's
  // roundings (softmax: the exponent's too, up to |x - m| 2^-24, and the
  // sum's) and the sum c by its own.
  const F rel = sigmoid ? F(0x1p-20) : F(0x1p-16);
  bool near = false;

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const int span = size / V;                     // lanes of a group, where groups are whole lanes
    const bool whole = span * V == size && (span & (span - 1)) == 0 && span > 0;
    K gkey = key_of(ninf);
    F gerr = 0;
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
      F mag;
      gkey = key_of(group_value(a.top, best, next, mag));
      gerr = mag;
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
        F mag;
        const F v = group_value(a.top, best, next, mag);
        if (lane == g) {
          gkey = key_of(v);
          gerr = mag;
        }
      }
    }
    if (group >= a.groups) gkey = 0;               // (lanes past the last group)
    gerr = (gerr + F(2)) * (biased || by_score ? rel : F(0));
    uint32_t kept = 0;
    F last = ninf, last_err = 0;
    for (int r = 0; r <= a.keep; ++r) {
      if (r == a.groups) break;
      const K top = warp_max(gkey);
      const int who = __ffs(__ballot_sync(kAll, gkey == top)) - 1;
      const int g = __shfl_sync(kAll, group, who);
      const F v = from_key(top);
      const F err = __shfl_sync(kAll, gerr, who);
      if (r < a.keep) {
        kept |= 1u << g;
        last = v;
        last_err = err;
        if (group == g) gkey = 0;
      } else if (v != ninf && last - v <= last_err + err) {
        near = biased || by_score;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = whole ? group : (lane * V + j) / size;
      if (g >= a.groups || !((kept >> g) & 1u)) key[j] = key_of(ninf);
    }
  }

  // k rounds of the maximum over the warp and the lowest lane that has it,
  // one more to see how near the first one left out is
  idx = -1;
  xsel = 0.f;
  F csel = ninf, cnext = ninf;
  float xnext = 0.f;
  int inext = 0;
  const K none = key_of(ninf);
  const int rounds = biased ? a.k + 1 : a.k;
  for (int r = 0; r < rounds; ++r) {
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
    if (r == a.k) {
      cnext = from_key(top);
      xnext = xv;
      inext = i;
    } else if (lane == r) {
      idx = i;
      xsel = xv;
      csel = from_key(top);
    }
  }
  ssel = idx >= 0 ? score_of<F>(sigmoid, xsel, m, sum) : F(0);
  if (biased) {
    // lane r against the choice after it (the first one left out after the last)
    F c2 = __shfl_down_sync(kAll, csel, 1);
    float x2 = __shfl_down_sync(kAll, xsel, 1);
    int i2 = __shfl_down_sync(kAll, idx, 1);
    if (lane == a.k - 1) {
      c2 = cnext;
      x2 = xnext;
      i2 = cnext == ninf ? -1 : inext;
    }
    if (lane < a.k && idx >= 0 && i2 >= 0) {
      const F a1 = csel < 0 ? -csel : csel, a2 = c2 < 0 ? -c2 : c2;
      const F s2 = score_of<F>(sigmoid, x2, m, sum);
      const bool same = xsel == x2 && __ldg(a.bias + idx) == __ldg(a.bias + i2);
      near = near || (csel - c2 <= rel * (ssel + s2) + F(0x1p-22) * (a1 + a2) && !same);
    }
    near = __any_sync(kAll, near);
  }
  return __any_sync(kAll, near);
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
  decide<double, V>(a, x, lane, idx, xsel, ssel);
  w = weight_of<double>(a, idx, xsel, ssel);
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
__global__ void __launch_bounds__(128) moe_route_kernel(const __grid_constant__ RouteArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  if (t >= a.T) return;   // warp-uniform; the kernel has no block barrier
  float x[V];
  load_row<V>(a, t, lane, x);
  int idx;
  float xsel, ssel, w;
  if (decide<float, V>(a, x, lane, idx, xsel, ssel))
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
                    (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 && p.ld % 8 == 0, p.scale};
  const int grid = static_cast<int>(ceil_div(p.T, 4));
  if (p.E <= 32) return launch_pdl(moe_route_kernel<1>, grid, 128, 0, s, a);
  if (p.E <= 64) return launch_pdl(moe_route_kernel<2>, grid, 128, 0, s, a);
  if (p.E <= 128) return launch_pdl(moe_route_kernel<4>, grid, 128, 0, s, a);
  if (p.E <= 256) return launch_pdl(moe_route_kernel<8>, grid, 128, 0, s, a);
  if (p.E <= 512) return launch_pdl(moe_route_kernel<16>, grid, 128, 0, s, a);
  return launch_pdl(moe_route_kernel<32>, grid, 128, 0, s, a);
}

}  // namespace mx
