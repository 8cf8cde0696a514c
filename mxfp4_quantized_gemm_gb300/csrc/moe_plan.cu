// What surrounds the experts' products: the pairs (token, slot) sorted by
// expert, the tokens quantized to their sorted rows, and the weighted sum of
// each token's results.
//
// The sort is counted, not compared: one block per expert counts all experts
// (every block the same histogram), so it knows its expert's first row tile
// without a word from another block, then places its own pairs in their
// order.  No atomic decides an order, so the same ids give the same plan.
// The ids are read E times from L2, a few microseconds for 65536 pairs.
//
// The gather reads each token once (bytes: 2 T K), quantizes it per 1x32
// (the rule of quant_math.cuh) and writes its codes and scales to the sorted
// row of each of its pairs, in the blocked form that one bulk copy per stage
// brings to the products: 17/32 bytes per value and pair.
//
// The sum reads each pair's bf16 result once and adds in fp32 in the order of
// the slots.  The results are rounded to bf16 on their way (half a step,
// 2^-8 of each term at most): kept in fp32 they would double the kernel's
// bytes, which are the second largest of a prompt's call after the products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_common.cuh"
#include "internal.h"
#include "layout.cuh"
#include "moe.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace mx {

static __device__ uint32_t g_moe_plan_error;

// ------------------------------------------------------------------- plan
namespace {

constexpr size_t kPlanHeader = 256;
// Histograms that a block keeps side by side: lanes that meet the same expert
// would otherwise add one after another (65536 pairs over 64 experts: 15 us).
constexpr int kHists = 8;
constexpr int kAhead = 8;   // loads of ids in flight per lane

struct PlanArgs {
  const int32_t* ids;
  int P, E;
  MoePlan plan;
};

// Ids p .. p + 3 (-1 past p1; p1 is P or a multiple of 128).
__device__ __forceinline__ int4 load_ids(const int32_t* ids, int p, int p1, bool vec) {
  if (vec && p + 3 < p1) return *reinterpret_cast<const int4*>(ids + p);
  return make_int4(p < p1 ? ids[p] : -1, p + 1 < p1 ? ids[p + 1] : -1, p + 2 < p1 ? ids[p + 2] : -1,
                   p + 3 < p1 ? ids[p + 3] : -1);
}

__global__ void __launch_bounds__(1024) moe_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int hists[];   // [E][kHists], then [E]: see below
  int* hist = hists + a.E * kHists;
  __shared__ int wsum[32], wtile[32], wall[32];
  const int tid = threadIdx.x, n_thr = blockDim.x, lane = tid & 31, warp = tid >> 5, n_warps = n_thr >> 5;
  const int e = blockIdx.x;
  for (int i = tid; i < a.E * kHists; i += n_thr) hists[i] = 0;
  griddep_launch_dependents();
  griddep_wait();
  __syncthreads();
  // The pairs are dealt to the warps in stretches of whole 128s, four
  // neighbours to a lane, so that a warp meets them in order in both passes.
  const int per = (a.P + n_warps * 128 - 1) / (n_warps * 128) * 128;   // pairs per warp
  const int p0 = warp * per < a.P ? warp * per : a.P, p1 = p0 + per < a.P ? p0 + per : a.P;
  const bool vec = (reinterpret_cast<uintptr_t>(a.ids) & 15) == 0;
  bool bad = false;
  int mine = 0;   // this expert's pairs among this lane's
  auto count = [&](int4 v) {
    const int id[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (static_cast<uint32_t>(id[j]) < static_cast<uint32_t>(a.E))
        atomicAdd(&hists[id[j] * kHists + (lane & (kHists - 1))], 1);
      else
        bad = bad || id[j] >= a.E;
      mine += id[j] == e;
    }
  };
  int at = p0;
  for (; vec && at + 128 * kAhead <= p1; at += 128 * kAhead) {
    int4 v[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) v[q] = *reinterpret_cast<const int4*>(a.ids + at + 128 * q + 4 * lane);
#pragma unroll
    for (int q = 0; q < kAhead; ++q) count(v[q]);
  }
  for (; at < p1; at += 128) count(load_ids(a.ids, at + 4 * lane, p1, vec));
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  __syncthreads();
  // row tiles before this expert's, and in all
  int before = 0, all = 0;
  for (int i = tid; i < a.E; i += n_thr) {
    int sum = 0;
#pragma unroll
    for (int q = 0; q < kHists; ++q) sum += hists[i * kHists + ((q + i) & (kHists - 1))];
    hist[i] = sum;
    const int n = (sum + kRowTile - 1) / kRowTile;
    all += n;
    if (i < e) before += n;
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  all = __reduce_add_sync(0xFFFFFFFFu, all);
  if (lane == 0) {
    wsum[warp] = mine;
    wtile[warp] = before;
    wall[warp] = all;
  }
  __syncthreads();
  int first = 0, tile0 = 0, tiles = 0;
  for (int w = 0; w < n_warps; ++w) {
    if (w < warp) first += wsum[w];
    tile0 += wtile[w];
    tiles += wall[w];
  }
  const int n = hist[e];
  if (e == 0) {
    for (int i = tid; i < 2 * kMoeTickets; i += n_thr) a.plan.tickets[i] = 0;
    if (tid == 0) a.plan.hdr[0] = tiles;
    if (bad) atomicOr(&g_moe_plan_error, kErrIndex);
  }
  for (int i = tid; i < (n + kRowTile - 1) / kRowTile; i += n_thr) {
    const int live = n - i * kRowTile < kRowTile ? n - i * kRowTile : kRowTile;
    a.plan.tile[tile0 + i] = e | (live << 16);
  }
  if (n == 0 && e != 0) return;
  auto place = [&](int p, int4 v) {   // by whole warps
    const int id[4] = {v.x, v.y, v.z, v.w};
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = __ballot_sync(0xFFFFFFFFu, id[j] == e);
    if (e != 0 && (m[0] | m[1] | m[2] | m[3]) == 0) return;
    const uint32_t lower = (1u << lane) - 1u;
    int r = tile0 * kRowTile + first + __popc(m[0] & lower) + __popc(m[1] & lower) + __popc(m[2] & lower) +
            __popc(m[3] & lower);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (id[j] == e) {
        a.plan.row_pair[r] = p + j;
        a.plan.pos[p + j] = r;
        ++r;
      } else if (e == 0 && p + j < p1 && static_cast<uint32_t>(id[j]) >= static_cast<uint32_t>(a.E)) {
        a.plan.pos[p + j] = -1;
      }
    }
    first += __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
  };
  for (at = p0; vec && at + 128 * kAhead <= p1; at += 128 * kAhead) {
    int4 v[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) v[q] = *reinterpret_cast<const int4*>(a.ids + at + 128 * q + 4 * lane);
#pragma unroll
    for (int q = 0; q < kAhead; ++q) place(at + 128 * q + 4 * lane, v[q]);
  }
  for (; at < p1; at += 128) place(at + 4 * lane, load_ids(a.ids, at + 4 * lane, p1, vec));
}

// ----------------------------------------------------------------- gather
struct GatherArgs {
  const uint16_t* x;
  int64_t ldx;
  int T, k, K, KT, R;
  int vec_ok;
  MoePlan plan;
  uint8_t* blocks;
  uint16_t* zero;
  int64_t ldz;
  int N;
};

// A warp owns k-tile gw % KT of the tokens gw / KT, + R, ...; lane l holds
// elements 8l..8l+7 of the k-tile, four lanes one 32-element block.
__global__ void __launch_bounds__(256, 4) moe_gather_kernel(const __grid_constant__ GatherArgs a) {
  const int lane = threadIdx.x & 31;
  const int gw = static_cast<int>((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
  // The products behind this kernel read the plan before they wait for it,
  // so they are let go only once the plan is complete.
  griddep_wait();
  griddep_launch_dependents();
  if (gw >= a.KT * a.R) return;   // warp-uniform; the kernel has no block barrier
  const int kt = gw % a.KT, r0 = gw / a.KT;
  const int e0 = kt * 256 + lane * 8;
  const int nb = (a.K + 31) >> 5;
  for (int t = r0; t < a.T; t += 2 * a.R) {
    uint4 v[2];
    int pos[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tt = t + j * a.R;
      v[j] = make_uint4(0, 0, 0, 0);
      pos[j] = -1;
      if (tt >= a.T) continue;
      // load8_words' rows are indexed by int leading dimensions; the row's
      // start is formed in 64 bits here
      v[j] = load8_words(a.x + static_cast<int64_t>(tt) * a.ldx, 0, 1, a.K, 0, e0, a.vec_ok != 0);
      if (lane < a.k) pos[j] = __ldcg(a.plan.pos + static_cast<int64_t>(tt) * a.k + lane);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tt = t + j * a.R;
      if (tt >= a.T) break;     // warp-uniform
      uint32_t sbyte;
      const uint32_t packed = quantize8_words(v[j], sbyte);
      const int b = lane >> 2;  // block of the k-tile; its group of four has one word of scales
      uint32_t word = (kt * 8 + b < nb ? sbyte : 0x7Fu) << (8 * (b & 3));
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
      for (int s = 0; s < a.k; ++s) {
        const int r = __shfl_sync(0xFFFFFFFFu, pos[j], s);
        if (r < 0) {
          if (a.zero != nullptr) {   // its result row, each k-tile's warp a share of it
            uint16_t* z = a.zero + (static_cast<int64_t>(tt) * a.k + s) * a.ldz;
            for (int n = kt * 32 + lane; n < a.N; n += a.KT * 32) z[n] = 0;
          }
          continue;
        }
        const int i = r & 127;
        uint8_t* blk = a.blocks + (static_cast<size_t>(r >> 7) * a.KT + kt) * kMoeBlockBytes;
        *reinterpret_cast<uint32_t*>(blk + (i << 7) + ((((lane >> 2) ^ (i & 7))) << 4) + ((lane & 3) << 2)) = packed;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(blk + kTileBytes + ((lane >> 4) << 9) + ((i & 31) << 4) + ((i >> 5) << 2)) = word;
      }
    }
  }
}

// ---------------------------------------------------------------- combine
struct CombineArgs {
  const uint16_t* parts;    // [P][ldp], ldp a multiple of 8
  int64_t ldp;
  const float* weights;
  const int32_t* pos;
  const uint16_t* residual;
  int64_t ldr;
  uint16_t* out;
  int64_t ldo;
  int k, N;
  int vec_ok;               // residual and out allow 16-byte accesses
};

// One thread per token and 8 columns, kUnroll results in flight.
__global__ void __launch_bounds__(128) moe_combine_kernel(const __grid_constant__ CombineArgs a) {
  constexpr int kUnroll = 4;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int n = (blockIdx.y * 128 + threadIdx.x) * 8;
  if (n >= a.N) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < a.k; s0 += kUnroll) {
    uint4 v[kUnroll];
    float w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t p = t * a.k + s0 + u;
      const bool on = s0 + u < a.k && __ldcg(a.pos + p) >= 0;
      w[u] = on ? a.weights[p] : 0.f;
      v[u] = on ? __ldcg(reinterpret_cast<const uint4*>(a.parts + p * a.ldp + n)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t q[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w[u], __uint_as_float(q[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w[u], __uint_as_float(q[i] & 0xFFFF0000u), acc[2 * i + 1]);
      }
    }
  }
  uint16_t* o = a.out + t * a.ldo + n;
  const uint16_t* res = a.residual != nullptr ? a.residual + t * a.ldr + n : nullptr;
  if (a.vec_ok != 0 && n + 8 <= a.N) {
    if (res != nullptr) {
      const uint4 r = *reinterpret_cast<const uint4*>(res);
      const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += __uint_as_float(q[i] << 16);
        acc[2 * i + 1] += __uint_as_float(q[i] & 0xFFFF0000u);
      }
    }
    *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                              pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < a.N) {
        const float v = acc[i] + (res != nullptr ? bf16_bits_to_float(res[i]) : 0.f);
        o[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
      }
  }
}

}  // namespace

size_t moe_plan_bytes(int64_t P, int E) {
  const int64_t rt = moe_max_tiles(P, E);
  const size_t ints = static_cast<size_t>(ceil_div(rt, 4) * 4) + static_cast<size_t>(rt) * kRowTile + static_cast<size_t>(P) + 2 * kMoeTickets;
  return kPlanHeader + 4 * ints + 64;
}

MoePlan moe_plan_at(void* base, int64_t P, int E) {
  const int64_t rt = moe_max_tiles(P, E);
  MoePlan p;
  p.hdr = static_cast<int32_t*>(base);
  p.tile = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(base) + kPlanHeader);
  p.row_pair = p.tile + ceil_div(rt, 4) * 4;       // 16-byte aligned
  p.pos = p.row_pair + rt * kRowTile;
  p.tickets = p.pos + P;
  p.max_tiles = static_cast<int>(rt);
  return p;
}

cudaError_t launch_moe_plan(const int32_t* ids, int P, int E, const MoePlan& plan, const DeviceInfo& dev,
                            cudaStream_t s) {
  (void)dev;
  const PlanArgs a{ids, P, E, plan};
  return launch_pdl(moe_plan_kernel, E, P <= 1024 ? 256 : 1024, E * (kHists + 1) * 4, s, a);
}

cudaError_t launch_moe_gather(const void* x, int64_t ldx, int T, int top_k, int K, const MoePlan& plan,
                              uint8_t* blocks, void* zero, int64_t ldz, int N, const DeviceInfo& dev, cudaStream_t s) {
  GatherArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.T = T;
  a.k = top_k;
  a.K = K;
  a.KT = static_cast<int>(padded_k(K) / kKTile);
  a.vec_ok = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (ldx % 8) == 0;
  a.plan = plan;
  a.blocks = blocks;
  a.zero = static_cast<uint16_t*>(zero);
  a.ldz = ldz;
  a.N = N;
  int64_t r = static_cast<int64_t>(dev.sm_count) * (T <= kDecodeMaxM ? 1 : 8) * 8 / a.KT;
  if (r > T) r = T;
  if (r < 1) r = 1;
  a.R = static_cast<int>(r);
  return launch_pdl(moe_gather_kernel, static_cast<int>((static_cast<int64_t>(a.KT) * r + 7) / 8), 256, 0, s, a);
}

cudaError_t launch_moe_combine(const void* parts, int64_t ldp, const float* weights, const MoePlan& plan,
                               const void* residual, int64_t ldr, void* out, int64_t ldo, int T, int top_k, int N,
                               const DeviceInfo& dev, cudaStream_t s) {
  (void)dev;
  CombineArgs a{};
  a.parts = static_cast<const uint16_t*>(parts);
  a.ldp = ldp;
  a.weights = weights;
  a.pos = plan.pos;
  a.residual = static_cast<const uint16_t*>(residual);
  a.ldr = ldr;
  a.out = static_cast<uint16_t*>(out);
  a.ldo = ldo;
  a.k = top_k;
  a.N = N;
  a.vec_ok = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && ldo % 8 == 0 &&
             (residual == nullptr || ((reinterpret_cast<uintptr_t>(residual) & 15) == 0 && ldr % 8 == 0));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(T), static_cast<unsigned>(ceil_div(N, 1024)), 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_combine_kernel, a);
}

uint32_t moe_plan_read_clear_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_moe_plan_error, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_moe_plan_error, &zero, sizeof(zero));
  return v;
}

}  // namespace mx
