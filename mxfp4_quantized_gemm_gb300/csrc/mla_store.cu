// mxfp4_mla_store: what enters the latent cache, in one pass over the new
// tokens.  For token t with position p and cache slot c:
//   y      = lat / sqrt(mean(lat^2) + eps) * gamma       (lat = kv[t][0..L))
//   rot(x) : (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin) of the 32
//            pairs (2i, 2i + 1) or (i, i + 32), angle i of position p
//   cache[c] = bf16(y) | bf16(rot(kv[t][L..L+R)))
//   q_out[t][h] = bf16(rot(q[t][h]))                     for every head
// All arithmetic in fp32 (the squares' sum included), one rounding per value.
//
// Bound by HBM for many tokens (it reads and writes each value once) and by
// the launch and two dependent loads (position, then its table row) for few.
// One block per token: warp 0 holds the latent row in registers, and every
// thread of the other warps rotates 16 values of a head, the unit in which
// both pairings are closed (two 16-byte vectors holding pairs 8u..8u+7): its
// sixteen table values are loaded once and serve all the heads it visits.  Two
// heads are in flight per thread, asked for before the position is known, and
// eight blocks fit an SM: a token takes about 2.5 us from launch to store, so
// it is the tokens in flight that carry the bandwidth (one head a thread and
// three blocks per SM: 50 us at 8192 tokens x 64 heads; now 26.7 us, 5.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mla.h"
#include "mla_common.cuh"

namespace mx {

static __device__ uint32_t g_mla_store_error;

struct StoreArgs {
  const uint16_t* kv;
  const uint16_t* gamma;
  const uint16_t* q;
  uint16_t* q_out;
  const float* cos_sin;
  const int64_t* positions;
  const int64_t* slots;
  uint16_t* cache;
  int64_t ldkv, q_tok, q_head, o_tok, o_head, page_stride;
  int page_size, num_pages, max_pos;
  int H, L;
  float eps;
  bool interleaved;
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Unit u (0..3) of a 64-element row: vectors 2u, 2u + 1 interleaved, u and
// u + 4 otherwise; c, s: cos and sin of pairs 8u..8u+7.  Word by word, so that
// few values are unpacked at a time.
__device__ __forceinline__ void rotate_unit(uint4& va, uint4& vb, const float (&c)[8], const float (&s)[8],
                                            bool interleaved) {
  uint32_t a[4] = {va.x, va.y, va.z, va.w}, b[4] = {vb.x, vb.y, vb.z, vb.w};
  if (interleaved) {
    // a word is a pair
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = lo16(a[i]), a1 = hi16(a[i]), b0 = lo16(b[i]), b1 = hi16(b[i]);
      a[i] = pack_bf16x2(a0 * c[i] - a1 * s[i], a1 * c[i] + a0 * s[i]);
      b[i] = pack_bf16x2(b0 * c[4 + i] - b1 * s[4 + i], b1 * c[4 + i] + b0 * s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = lo16(a[i]), a1 = hi16(a[i]), b0 = lo16(b[i]), b1 = hi16(b[i]);
      a[i] = pack_bf16x2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
      b[i] = pack_bf16x2(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
    }
  }
  va = make_uint4(a[0], a[1], a[2], a[3]);
  vb = make_uint4(b[0], b[1], b[2], b[3]);
}

__device__ __forceinline__ void load_angles(const float* row, int u, float (&c)[8], float (&s)[8]) {
  const float4* cp = reinterpret_cast<const float4*>(row + 8 * u);
  const float4* sp = reinterpret_cast<const float4*>(row + kMlaRope / 2 + 8 * u);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 cv = __ldg(cp + i), sv = __ldg(sp + i);
    c[4 * i] = cv.x;
    c[4 * i + 1] = cv.y;
    c[4 * i + 2] = cv.z;
    c[4 * i + 3] = cv.w;
    s[4 * i] = sv.x;
    s[4 * i + 1] = sv.y;
    s[4 * i + 2] = sv.z;
    s[4 * i + 3] = sv.w;
  }
}

constexpr int kStoreThreads = 160;            // warp 0: the cache row; four warps: the queries

__global__ void __launch_bounds__(kStoreThreads, 8) mla_store_kernel(const StoreArgs a) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int step = a.interleaved ? 1 : 4;              // distance of a unit's two vectors
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    // ---- the cache row
    const int64_t pos = __ldg(a.positions + t), slot = __ldg(a.slots + t);
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    const bool slot_ok = slot >= 0 && slot < static_cast<int64_t>(a.num_pages) * a.page_size;
    if (lane == 0 && (!pos_ok || (slot >= 0 && !slot_ok))) atomicOr(&g_mla_store_error, kErrIndex);
    if (!pos_ok || !slot_ok) return;
    const uint16_t* x = a.kv + t * a.ldkv;
    uint16_t* row = a.cache + (slot / a.page_size) * a.page_stride +
                    (slot % a.page_size) * static_cast<int64_t>(a.L + kMlaRope);
    const int nv = a.L >> 3;                           // 16-byte vectors of the latent, at most 64
    uint4 xv[2], gv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = lane + 32 * i;
      xv[i] = v < nv ? __ldg(reinterpret_cast<const uint4*>(x) + v) : make_uint4(0, 0, 0, 0);
      gv[i] = v < nv ? __ldg(reinterpret_cast<const uint4*>(a.gamma) + v) : make_uint4(0, 0, 0, 0);
    }
    if (lane < 4) {
      // the shared key, while the sum is on its way
      float c[8], s[8];
      load_angles(a.cos_sin + pos * kMlaRope, lane, c, s);
      const int v0 = nv + (a.interleaved ? 2 * lane : lane);
      uint4 va = __ldg(reinterpret_cast<const uint4*>(x) + v0), vb = __ldg(reinterpret_cast<const uint4*>(x) + v0 + step);
      rotate_unit(va, vb, c, s, a.interleaved);
      reinterpret_cast<uint4*>(row)[v0] = va;
      reinterpret_cast<uint4*>(row)[v0 + step] = vb;
    }
    __syncwarp();
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[8];
      unpack8(xv[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float inv = 1.0f / sqrtf(ss / static_cast<float>(a.L) + a.eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = lane + 32 * i;
      if (v < nv) {
        float f[8], g[8];
        unpack8(xv[i], f);
        unpack8(gv[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * inv * g[e];
        reinterpret_cast<uint4*>(row)[v] = pack8(f);
      }
    }
    return;
  }
  // ---- the queries
  const int first = threadIdx.x - 32, stride = (blockDim.x - 32) >> 2;
  const int u = first & 3;
  int h = first >> 2;
  if (h >= a.H) return;
  const int v0 = a.interleaved ? 2 * u : u;
  const uint16_t* src = a.q + t * a.q_tok + h * a.q_head;
  uint16_t* dst = a.q_out + t * a.o_tok + h * a.o_head;
  auto load = [&](const uint16_t* p, uint4 (&v)[2]) {
    v[0] = reinterpret_cast<const uint4*>(p)[v0];
    v[1] = reinterpret_cast<const uint4*>(p)[v0 + step];
  };
  uint4 x[2], y[2];
  load(src, x);
  if (h + stride < a.H) load(src + stride * a.q_head, y);
  const int64_t pos = __ldg(a.positions + t);
  if (pos < 0 || pos >= a.max_pos) return;
  float c[8], s[8];
  load_angles(a.cos_sin + pos * kMlaRope, u, c, s);
  while (true) {
    rotate_unit(x[0], x[1], c, s, a.interleaved);
    reinterpret_cast<uint4*>(dst)[v0] = x[0];
    reinterpret_cast<uint4*>(dst)[v0 + step] = x[1];
    h += stride;
    if (h >= a.H) return;
    src += stride * a.q_head;
    dst += stride * a.o_head;
    x[0] = y[0];
    x[1] = y[1];
    if (h + stride < a.H) load(src + stride * a.q_head, y);
  }
}

cudaError_t launch_mla_store(const MlaStoreProblem& p, const DeviceInfo&, cudaStream_t s) {
  StoreArgs a{};
  a.kv = static_cast<const uint16_t*>(p.kv);
  a.gamma = static_cast<const uint16_t*>(p.gamma);
  a.q = static_cast<const uint16_t*>(p.q.p);
  a.q_out = static_cast<uint16_t*>(const_cast<void*>(p.q_out.p));
  a.cos_sin = p.cos_sin;
  a.positions = p.positions;
  a.slots = p.slots;
  a.cache = static_cast<uint16_t*>(p.cache.p);
  a.ldkv = p.ldkv;
  a.q_tok = p.q.tok;
  a.q_head = p.q.head;
  a.o_tok = p.q_out.tok;
  a.o_head = p.q_out.head;
  a.page_stride = p.cache.page_stride;
  a.page_size = p.cache.page_size;
  a.num_pages = p.cache.num_pages;
  a.max_pos = p.max_pos;
  a.H = p.H;
  a.L = p.L;
  a.eps = p.eps;
  a.interleaved = p.interleaved;
  const int64_t units = static_cast<int64_t>(p.H) * 4;                       // 16-value units of a token's queries
  const int64_t warps = ceil_div(units, 32);
  const int threads = warps < kStoreThreads / 32 - 1 ? 32 + static_cast<int>(warps) * 32 : kStoreThreads;
  return mla_launch(mla_store_kernel, dim3(static_cast<unsigned>(p.T)), threads, 0, s, a);
}

uint32_t mla_store_read_clear_error() { return read_clear_word(g_mla_store_error); }

}  // namespace mx
