// What surrounds the experts' products: the pairs (token, slot) sorted by
// expert, the tokens quantized to their sorted rows, and the weighted sum of
// each token's results.
//
// The sort is counted, not compared: one block per expert counts all experts
// (every block the same histogram), so it knows its expert's first row tile
// without a word from another block, then places its own pairs in their
// order.  No atomic decides an order, so the same ids give the same plan.
// The ids are read E times from L2: 65536 pairs of 64 experts take 19 us (3%
// of their call), 8192 of 64 6.3.
//
// The gather reads each token once (bytes: 2 T K), quantizes it per 1x32
// (the rule of quant_math.cuh) and writes its codes and scales to the sorted
// row of each of its pairs, in the blocked form that one bulk copy per stage
// brings to the products: 17/32 bytes per value and pair.  8192 x 8 pairs of
// 5120 values take 54 us, 178 MB of them written (46 us at the rate of writes
// alone).
//
// The sum reads each pair's bf16 result once and adds in fp32 in the order of
// the slots.  The results are rounded to bf16 on their way (half a step,
// 2^-8 of each term at most): kept in fp32 they would double the kernel's
// bytes, which are its time: 8192 x 8 results of 5120 take 124 us alone (6.7
// TB/s), 148 behind the product whose last results leave L2 meanwhile.
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

// This lane's 8 values of k-tile kt of token t, and the block's quantization of
// them written to the sorted rows of the token's pairs (lane j holds pair j's,
// -1 without an expert: its row of `zero`, if any, is zeroed, each k-tile's
// warp a share of it).
__device__ __forceinline__ uint4 load_unit(const GatherArgs& a, int t, int kt, int lane) {
  // load8_words indexes rows by an int leading dimension: the row's start is
  // formed in 64 bits here
  return load8_words(a.x + static_cast<int64_t>(t) * a.ldx, 0, 1, a.K, 0, kt * 256 + lane * 8, a.vec_ok != 0);
}
__device__ __forceinline__ void store_unit(const GatherArgs& a, int t, int kt, int lane, uint4 v, int pos) {
  uint32_t sbyte;
  const uint32_t packed = quantize8_words(v, sbyte);
  const int b = lane >> 2;  // block of the k-tile; its group of four has one word of scales
  uint32_t word = (kt * 8 + b < ((a.K + 31) >> 5) ? sbyte : 0x7Fu) << (8 * (b & 3));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
  // All of the block's codes for each of its four lanes: lane l writes block
  // l / 4 of one pair in four, so that a store covers the k-tile of four rows.
  uint4 codes;
  codes.x = __shfl_sync(0xFFFFFFFFu, packed, lane & ~3);
  codes.y = __shfl_sync(0xFFFFFFFFu, packed, (lane & ~3) + 1);
  codes.z = __shfl_sync(0xFFFFFFFFu, packed, (lane & ~3) + 2);
  codes.w = __shfl_sync(0xFFFFFFFFu, packed, (lane & ~3) + 3);
  // Lane j, for pair j: the row's place in 16-byte pieces (a multiple of 8: the
  // lowest bits hold the row's rotation), and its row of scales in the block.
  constexpr uint32_t kNowhere = 0xFFFFFFFFu;
  const int i = pos & 127;
  const uint32_t block = static_cast<uint32_t>(pos >> 7) * a.KT + kt;
  const uint32_t place = pos < 0 ? kNowhere : block * (kMoeBlockBytes / 16) + 8 * i + (i & 7);
  const int scale = kTileBytes - 128 * i + ((i & 31) << 4) + ((i >> 5) << 2);   // bytes from the row's codes
  for (int s = lane & 3; s < a.k + (lane & 3); s += 4) {   // (whole warps loop; lanes >= k hold no place)
    const uint32_t at = __shfl_sync(0xFFFFFFFFu, place, s);
    const int sc = __shfl_sync(0xFFFFFFFFu, scale, s);
    if (at == kNowhere) continue;
    uint8_t* row = a.blocks + static_cast<size_t>(at & ~7u) * 16;
    *reinterpret_cast<uint4*>(row + ((b ^ (at & 7)) << 4)) = codes;
    if ((b & 3) == 0) *reinterpret_cast<uint32_t*>(row + sc + ((b >> 2) << 9)) = word;
  }
  if (a.zero == nullptr) return;
  for (uint32_t none = __ballot_sync(0xFFFFFFFFu, lane < a.k && pos < 0); none != 0; none &= none - 1) {
    uint16_t* z = a.zero + (static_cast<int64_t>(t) * a.k + __ffs(none) - 1) * a.ldz;
    for (int n = kt * 32 + lane; n < a.N; n += a.KT * 32) z[n] = 0;
  }
}

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
  const int kt = gw % a.KT;
  for (int t = gw / a.KT; t < a.T; t += 2 * a.R) {
    uint4 v[2];
    int pos[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tt = t + j * a.R;
      v[j] = make_uint4(0, 0, 0, 0);
      pos[j] = -1;
      if (tt >= a.T) continue;
      v[j] = load_unit(a, tt, kt, lane);
      if (lane < a.k) pos[j] = __ldcg(a.plan.pos + static_cast<int64_t>(tt) * a.k + lane);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (t + j * a.R < a.T) store_unit(a, t + j * a.R, kt, lane, v[j], pos[j]);   // (uniform)
  }
}

// Both in one kernel for few pairs, whose calls last no longer than some
// launches: every block counts all ids for itself, every warp finds the places
// of its tokens' pairs, and block 0 writes what else the plan holds.  The first
// product finds its tiles from the ids meanwhile, as long as an expert's pairs
// fill two row tiles at most (us, one kernel against two: 37 x 4 pairs 22.1 /
// 22.7, one token of 8 29.2 / 31.4, 16 of 8 109.9 / 114.3).
constexpr int kFewPairs = kMoeFewPairs;
struct FewArgs {
  GatherArgs g;
  const int32_t* ids;
  int P, E;
};

__global__ void __launch_bounds__(256, 4) moe_few_kernel(const __grid_constant__ FewArgs f) {
  __shared__ __align__(16) int ids[kFewPairs];
  __shared__ int first[kMoeMaxExperts], sums[8];
  const GatherArgs& a = f.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gw = blockIdx.x * 8 + warp;
  for (int e = tid; e < kMoeMaxExperts; e += 256) first[e] = 0;
  // The product behind this kernel reads the ids before it waits for it, so it
  // is let go only once they are there.
  griddep_wait();
  griddep_launch_dependents();
  const bool mine = gw < a.KT * a.R;
  const int kt = gw % a.KT, t0 = gw / a.KT;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (mine && t0 < a.T) v = load_unit(a, t0, kt, lane);   // under way while the ids are counted
  __syncthreads();
  bool bad = false;
  int id[kFewPairs / 256];
#pragma unroll
  for (int q = 0; q < kFewPairs / 256; ++q) id[q] = tid + 256 * q < f.P ? f.ids[tid + 256 * q] : -1;
#pragma unroll
  for (int q = 0; q < kFewPairs / 256; ++q) {
    ids[tid + 256 * q] = id[q];
    if (static_cast<uint32_t>(id[q]) < static_cast<uint32_t>(f.E))
      atomicAdd(&first[id[q]], 1);
    else
      bad = bad || id[q] >= f.E;
  }
  __syncthreads();
  // counts to first rows: row tiles before each expert's, four experts a thread
  int n[4], tiles = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    n[q] = first[4 * tid + q];
    tiles += (n[q] + kRowTile - 1) / kRowTile;
  }
  int upto = tiles;   // inclusive sum over the threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += w;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sums[w];
  int at = upto - tiles;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    first[4 * tid + q] = at * kRowTile;
    for (int i = 0; i < n[q]; i += kRowTile, ++at)
      if (blockIdx.x == 0) a.plan.tile[at] = (4 * tid + q) | ((n[q] - i < kRowTile ? n[q] - i : kRowTile) << 16);
  }
  if (blockIdx.x == 0) {
    for (int i = tid; i < 2 * kMoeTickets; i += 256) a.plan.tickets[i] = 0;
    if (tid == 255) a.plan.hdr[0] = upto;
    if (bad) atomicOr(&g_moe_plan_error, kErrIndex);
  }
  __syncthreads();
  if (!mine) return;
  int slots = 1;   // a.k, up to a power of two
  while (slots < a.k) slots *= 2;
  for (int t = t0; t < a.T; t += a.R) {
    if (t != t0) v = load_unit(a, t, kt, lane);
    // lane j: the row of pair j of the token, after the pairs before it of its
    // expert.  `share` lanes count for each pair, every one a part of the ids
    // (none past the token's pairs: they would read on behind the last id).
    const int p0 = t * a.k;
    const int e = lane < a.k ? ids[p0 + lane] : -1;
    const bool on = static_cast<uint32_t>(e) < static_cast<uint32_t>(f.E);
    const int share = 32 / slots, pair = lane / share;
    const int other = __shfl_sync(0xFFFFFFFFu, e, pair), before = pair < a.k ? p0 + pair : 0;
    int n_before = 0;
    for (int c = 4 * (lane % share); c < before; c += 4 * share) {
      const int4 w = *reinterpret_cast<const int4*>(ids + c);
      n_before += (w.x == other) + (w.y == other && c + 1 < before) + (w.z == other && c + 2 < before) +
                  (w.w == other && c + 3 < before);
    }
    for (int o = 1; o < share; o <<= 1) n_before += __shfl_xor_sync(0xFFFFFFFFu, n_before, o);
    n_before = __shfl_sync(0xFFFFFFFFu, n_before, (lane * share) & 31);
    const int pos = on ? first[e] + n_before : -1;
    if (kt == 0 && lane < a.k) {
      a.plan.pos[p0 + lane] = pos;
      if (on) a.plan.row_pair[pos] = p0 + lane;
    }
    store_unit(a, t, kt, lane, v, pos);
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
  int k, N, chunks;         // chunks: blocks of a token
  int vec_ok;               // residual and out allow 16-byte accesses
};

// One thread per token and 8 columns, kUnroll results in flight; the blocks of a
// token follow one another, as its results do in memory.  A result is asked for
// beside the word that says whether there is one, and the residual before both
// (each behind the other, the sum over 8192 x 8 pairs took 170 us).
template <int kUnroll>
__global__ void __launch_bounds__(256) moe_combine_kernel(const __grid_constant__ CombineArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x / a.chunks;
  const int n = ((blockIdx.x - static_cast<int>(t) * a.chunks) * 256 + threadIdx.x) * 8;
  if (n >= a.N) return;
  uint16_t* o = a.out + t * a.ldo + n;
  const bool whole = a.vec_ok != 0 && n + 8 <= a.N;
  uint4 res = make_uint4(0, 0, 0, 0);
  if (a.residual != nullptr) {
    const uint16_t* r = a.residual + t * a.ldr + n;
    if (whole) {
      res = *reinterpret_cast<const uint4*>(r);
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < a.N) w[i >> 1] |= static_cast<uint32_t>(r[i]) << (16 * (i & 1));
      res = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  auto add = [&](uint4 v, float w) {
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = fmaf(w, __uint_as_float(q[i] << 16), acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, __uint_as_float(q[i] & 0xFFFF0000u), acc[2 * i + 1]);
    }
  };
  const int64_t p0 = t * a.k;
  for (int s0 = 0; s0 < a.k; s0 += kUnroll) {
    uint4 v[kUnroll];
    float w[kUnroll];
    int pos[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      // past the last slot the first one's again, unused (a test would hold the
      // loads apart: 157 us instead of 148)
      const int64_t p = p0 + (s0 + u < a.k ? s0 + u : 0);
      v[u] = __ldcg(reinterpret_cast<const uint4*>(a.parts + p * a.ldp + n));
      pos[u] = __ldcg(a.pos + p);
      w[u] = a.weights[p];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool on = s0 + u < a.k && pos[u] >= 0;   // (what an empty slot has in memory may be anything)
      add(make_uint4(on ? v[u].x : 0u, on ? v[u].y : 0u, on ? v[u].z : 0u, on ? v[u].w : 0u), on ? w[u] : 0.f);
    }
  }
  if (a.residual != nullptr) add(res, 1.f);
  const uint4 r = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                             pack_bf16x2(acc[6], acc[7]));
  if (whole) {
    *reinterpret_cast<uint4*>(o) = r;
  } else {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < a.N) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

}  // namespace

size_t moe_plan_bytes(int64_t P, int E) {
  const int64_t rt = moe_max_tiles(P, E);
  const size_t ints = static_cast<size_t>(ceil_div(rt, 4) * 4 + rt * kRowTile + P + 2 * kMoeTickets);
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

cudaError_t launch_moe_plan_gather(const int32_t* ids, int E, const void* x, int64_t ldx, int T, int top_k, int K,
                                   const MoePlan& plan, uint8_t* blocks, void* zero, int64_t ldz, int N,
                                   const DeviceInfo& dev, cudaStream_t s) {
  const int P = T * top_k;
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
  // eight warps a block, five blocks an SM (all that its registers let it hold);
  // one for few tokens, whose warps have one unit each all the same
  int64_t r = static_cast<int64_t>(dev.sm_count) * (T <= kDecodeMaxM ? 1 : 5) * 8 / a.KT;
  if (r > T) r = T;
  if (r < 1) r = 1;
  a.R = static_cast<int>(r);
  const int grid = static_cast<int>((static_cast<int64_t>(a.KT) * r + 7) / 8);
  if (P <= kFewPairs) return launch_pdl(moe_few_kernel, grid, 256, 0, s, FewArgs{a, ids, P, E});
  const PlanArgs p{ids, P, E, plan};
  // few pairs give a large block's barriers more to do than its lanes (us, 256
  // threads against 1024: 512 pairs 3.8 / 5.3, 900 3.7 / 4.9, 3000 5.1 / 4.8)
  const cudaError_t e = launch_pdl(moe_plan_kernel, E, P <= 2048 ? 256 : 1024, E * (kHists + 1) * 4, s, p);
  return e != cudaSuccess ? e : launch_pdl(moe_gather_kernel, grid, 256, 0, s, a);
}

cudaError_t launch_moe_combine(const void* parts, int64_t ldp, const float* weights, const MoePlan& plan,
                               const void* residual, int64_t ldr, void* out, int64_t ldo, int T, int top_k, int N,
                               cudaStream_t s) {
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
  a.chunks = static_cast<int>(ceil_div(N, 2048));
  // slots at once: of four, three and two (all of one) the most that divide the
  // slots with the fewest left over
  int unroll = top_k < 4 ? top_k : 4;
  for (int u = unroll - 1; u >= 2; --u)
    if (ceil_div(top_k, u) * u < ceil_div(top_k, unroll) * unroll) unroll = u;
  const int grid = T * a.chunks;
  switch (unroll) {
    case 1: return launch_pdl(moe_combine_kernel<1>, grid, 256, 0, s, a);
    case 2: return launch_pdl(moe_combine_kernel<2>, grid, 256, 0, s, a);
    case 3: return launch_pdl(moe_combine_kernel<3>, grid, 256, 0, s, a);
    default: return launch_pdl(moe_combine_kernel<4>, grid, 256, 0, s, a);
  }
}

uint32_t moe_plan_read_clear_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_moe_plan_error, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_moe_plan_error, &zero, sizeof(zero));
  return v;
}

}  // namespace mx
