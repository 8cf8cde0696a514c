// Router of a mixture of experts: scores, choice and weights of each token.
//
//   s_i = softmax(x)_i or sigmoid(x_i);  c_i = s_i + bias_i
//   with groups: the topk_group groups whose `group_top` highest c sum
//   highest keep their experts; the top_k experts of highest c are chosen,
//   equal ones by the lower index; weight = scale * s_i (/ sum of the chosen).
//
// One warp per token, its E / 32 values per lane in registers: the row is
// read once and every reduction is a warp's.  A choice takes k rounds of a
// 32-bit integer maximum over the warp (redux) on the order-preserving image
// of c and one minimum of the indexes that have it, about 60 cycles a round,
// which bounds the kernel: the bytes (T * E logits) are few.
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
  int T, E, k, sigmoid, groups, keep, top, renorm, bf16;
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

// Decides one row.  Lane l holds elements l, l + 32, ... of the row; at the
// end lane r < k holds the r-th choice: its index (-1: none), its logit and
// its score, and every lane the sum of the chosen scores relative to the
// largest, `total`, with `part` this lane's term of it.  Returns whether a
// comparison that mattered was nearer than the fp32 evaluation's error.
template <typename F, int V>
__device__ __forceinline__ bool decide(const RouteArgs& a, const float (&x)[V], int lane, int& idx, float& xsel, F& ssel) {
  using K = typename Keys<F>::T;
  const F ninf = -static_cast<F>(INFINITY);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) m = fmaxf(m, x[j]);
  m = from_key(warp_max(key_of(m)));
  // scores
  F s[V];
  F sum = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (a.sigmoid) {
      s[j] = F(1) / (F(1) + exp_of(-static_cast<F>(x[j])));
    } else {
      s[j] = x[j] == -INFINITY ? F(0) : (x[j] == m ? F(1) : exp_of(static_cast<F>(x[j]) - static_cast<F>(m)));
      sum += s[j];
    }
  }
  if (!a.sigmoid) {
    sum = warp_sum(sum);
    const F r = sum > F(0) ? F(1) / sum : F(0);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = sizeof(F) == 8 ? (sum > F(0) ? s[j] / sum : F(0)) : s[j] * r;
  }
  // what is compared
  const bool biased = a.bias != nullptr;
  K key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * 32 + lane;
    F c = static_cast<F>(x[j]);
    if (biased && i < a.E) c = s[j] + static_cast<F>(__ldg(a.bias + i));
    key[j] = key_of(x[j] == -INFINITY || !(c == c) ? ninf : c);
  }
  // Error bound of a compared value: scores err by the exponential's
  // roundings (softmax: the exponent's too, up to |x - m| 2^-24, and the
  // sum's) and the sum c by its own.
  const F rel = a.sigmoid ? F(0x1p-20) : F(0x1p-16);
  bool near = false;

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const bool by_score = !biased && a.top == 2;   // sums of logits would not order as sums of scores do
    K gkey = 0;                                    // lane g: group g's sum
    F gerr = 0;
    for (int g = 0; g < a.groups; ++g) {
      F best = ninf, next = ninf;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = j * 32 + lane;
        if (i >= g * size && i < (g + 1) * size) {
          const F c = from_key(key[j]);
          const F v = by_score && c != ninf ? s[j] : c;
          if (v > best) {
            next = best;
            best = v;
          } else if (v > next) {
            next = v;
          }
        }
      }
      const K k1 = warp_max(key_of(best));
      const F b1 = from_key(k1);
      F total = b1;
      F mag = b1 < 0 ? -b1 : b1;
      if (a.top == 2) {
        // the second highest: the owner of the highest offers its next
        const uint32_t own = __ballot_sync(kAll, key_of(best) == k1);
        const F b2 = from_key(warp_max(key_of(lane == __ffs(own) - 1 ? next : best)));
        if (b2 != ninf) {
          total += b2;
          mag += b2 < 0 ? -b2 : b2;
        }
      }
      if (lane == g) {
        gkey = key_of(total);
        gerr = (mag + F(2)) * (biased || by_score ? rel : F(0));
      }
    }
    uint32_t kept = 0;
    F last = ninf, last_err = 0;
    for (int r = 0; r <= a.keep; ++r) {
      if (r == a.groups) break;
      const K top = warp_max(gkey);
      const int who = __ffs(__ballot_sync(kAll, gkey == top)) - 1;
      const F v = from_key(top);
      const F err = __shfl_sync(kAll, gerr, who);
      if (r < a.keep) {
        kept |= 1u << who;
        last = v;
        last_err = err;
        if (lane == who) gkey = 0;
      } else if (v != ninf && last - v <= last_err + err) {
        near = near || (biased || by_score);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = j * 32 + lane;
      if (i < a.E && !((kept >> (i / size)) & 1u)) key[j] = key_of(ninf);
    }
  }

  // k rounds of the maximum and the lowest index that has it, one more to
  // see how near the first one left out is
  idx = -1;
  xsel = 0.f;
  ssel = 0;
  F csel = ninf, bsel = 0;
  const K none = key_of(ninf);
  const int rounds = biased ? a.k + 1 : a.k;
  for (int r = 0; r < rounds; ++r) {
    K best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const K top = warp_max(best);
    if (top <= none) break;
    const uint32_t i = __reduce_min_sync(kAll, best == top ? static_cast<uint32_t>(at * 32 + lane) : kAll);
    const int who = i & 31, jw = i >> 5;
    float xv = 0.f;
    F sv = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j == jw) {
        xv = x[j];
        sv = s[j];
        if (lane == who) key[j] = 0;
      }
    xv = __shfl_sync(kAll, xv, who);
    sv = __shfl_sync(kAll, sv, who);
    const bool mine = r < 32 ? lane == r : false;
    if (biased) {
      // against the one before it, which every lane can see by its own round
      const F cv = from_key(top);
      const F bv = static_cast<F>(__ldg(a.bias + i));
      const F pc = __shfl_sync(kAll, csel, (r + 31) & 31), ps = __shfl_sync(kAll, ssel, (r + 31) & 31);
      const float px = __shfl_sync(kAll, xsel, (r + 31) & 31);
      const F pb = __shfl_sync(kAll, bsel, (r + 31) & 31);
      if (r > 0) {
        const F mag = (cv < 0 ? -cv : cv) > (pc < 0 ? -pc : pc) ? (cv < 0 ? -cv : cv) : (pc < 0 ? -pc : pc);
        near = near || (pc - cv <= rel * (sv + ps) + F(0x1p-22) * mag && !(px == xv && pb == bv));
      }
      if (mine) {
        csel = cv;
        bsel = bv;
      }
    }
    if (mine && r < a.k) {
      idx = static_cast<int>(i);
      xsel = xv;
      ssel = sv;
    }
  }
  return near;
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

template <int V>
__global__ void __launch_bounds__(128) moe_route_kernel(const __grid_constant__ RouteArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  if (t >= a.T) return;   // warp-uniform; the kernel has no block barrier
  float x[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * 32 + lane;
    const int64_t at = static_cast<int64_t>(t) * a.ld + i;
    float v = -INFINITY;
    if (i < a.E)
      v = a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.x)[at]) : static_cast<const float*>(a.x)[at];
    x[j] = v == v ? v : -INFINITY;   // a NaN is never chosen
  }
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
                    p.group_top, p.renormalize, p.bf16, p.scale};
  const int grid = static_cast<int>(ceil_div(p.T, 4));
  if (p.E <= 32) return launch_pdl(moe_route_kernel<1>, grid, 128, 0, s, a);
  if (p.E <= 64) return launch_pdl(moe_route_kernel<2>, grid, 128, 0, s, a);
  if (p.E <= 128) return launch_pdl(moe_route_kernel<4>, grid, 128, 0, s, a);
  if (p.E <= 256) return launch_pdl(moe_route_kernel<8>, grid, 128, 0, s, a);
  if (p.E <= 512) return launch_pdl(moe_route_kernel<16>, grid, 128, 0, s, a);
  return launch_pdl(moe_route_kernel<32>, grid, 128, 0, s, a);
}

}  // namespace mx
