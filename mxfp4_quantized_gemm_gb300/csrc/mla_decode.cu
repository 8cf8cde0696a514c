// mxfp4_mla_decode: absorbed latent attention of the newest tokens of each
// sequence over the paged latent cache.  With c_j the cache row of position
// j (latent L | rotated key R) and row r = (token i of q_len, head h),
//   s[r][j] = scale * (q_lat[r] . c_j[0..L) + q_rope[r] . c_j[L..L+R))
//   out[r]  = sum_j softmax_j(s[r])[j] c_j[0..L),   j < len - q_len + 1 + i.
// All heads read one latent row per position, so a step reads (L + R) values
// a position however many heads there are; at 64 heads that is 121 flop per
// byte, well below the card's 288, and HBM is the bound.
//
// A block takes up to 64 query rows of one sequence (a row group) and walks
// the positions in tiles of 128.  The accumulator of 64 rows x 512 latent
// values must stay in TMEM, whose 512 columns a 128-row fp32 accumulator of
// that width would fill by itself, so both products are formed transposed:
//   S^T [128 positions][rows] = C Q^T        (lanes = positions)
//   O^T [128 latent values][rows] += C^T P^T (L / 128 blocks, 64 columns each)
// which leaves room for two score tiles.  C feeds both products as the A
// operand, once with the latent values along K and once along M.  The tile
// (147 KB at L = 512) and the queries (74 KB) do not fit in shared memory
// twice, so the latent part streams through a ring of 128 x 128 pieces twice:
// from HBM for S^T, and from L2 shortly after for O^T.
//
// Roles: warp 0 copies (every lane one box of a page), warp 1 issues the
// score products, warp 2 the output products (two issuers, so that one's
// waits on barriers overlap the other's MMAs), warps 4..7 hold the softmax:
// thread = position, so a weight row P^T goes out as one 128-byte row.  The
// running maximum of a query row is shared by the 128 threads; it is raised
// only when some score passes it by 2^8 (first tile aside), which one barrier
// with an OR decides, and each thread keeps the sums of its own positions
// until the end of the sequence.
//
// Work split: the tiles of all row groups, in order, are cut evenly over the
// grid; a block takes its stretch wherever sequences begin and end, so a
// single long sequence spreads over all SMs.  A row group cut between blocks
// leaves unnormalized parts (fp32, with maximum and sum) that
// mla_combine_kernel joins.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>

#include "mla.h"
#include "mla_common.cuh"

namespace mx {

static __device__ uint32_t g_mla_decode_error;

constexpr int kDecThreads = 256;
constexpr int kTileTok = 128;                       // positions per tile
constexpr int kChunkBytes = kTileTok * 128;         // 128 positions x 64 values
constexpr int kDecStageBytes = 2 * kChunkBytes;     // 128 positions x 128 values
constexpr int kDecMaxStages = 5;
constexpr int kDecSmem = 227 * 1024;
constexpr int kDecScol = 256;                       // first TMEM column of the score tiles
constexpr int kMaxCtas = 256;

struct DecodeArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  __nv_bfloat16* out;
  float* lse;
  float* parts;
  int64_t table_stride, o_tok, o_head;
  int S, q_len, H, L;
  int page_size, num_pages, box_rows;
  int64_t capacity;       // positions a page-table row can hold
  int HB, TB, TPT;        // heads and tokens per box, tokens per row group
  int head_blocks, RT;    // row groups per token block, per sequence
  int stages;
  float c;                // scale * log2(e)
};

// Positions of sequence s (a bad length is cut to what the table holds).
__device__ __forceinline__ int seq_len(const DecodeArgs& a, int s) {
  const int n = __ldg(a.seq_lens + s);
  return n < 0 ? 0 : (n > a.capacity ? static_cast<int>(a.capacity) : n);
}
// Work units of one row group: its tiles, or one for an empty sequence
// (whose rows still have to be written).
__device__ __forceinline__ int group_units(int len) { return len == 0 ? 1 : (len + kTileTok - 1) / kTileTok; }

// A stretch of one row group's tiles.
struct Segment {
  int s, rt, len, t0, t1, nt;
};
// A block's stretch of the unit order (sequence, row group, tile).
struct Walk {
  int64_t left;       // units still to hand out
  int s, rt, off;
  __device__ __forceinline__ bool next(const DecodeArgs& a, Segment& g) {
    if (left <= 0) return false;
    g.s = s;
    g.rt = rt;
    g.len = seq_len(a, s);
    g.nt = group_units(g.len);
    g.t0 = off;
    const int64_t room = g.nt - off;
    const int take = static_cast<int>(left < room ? left : room);
    g.t1 = off + take;
    left -= take;
    off += take;
    if (off == g.nt) {
      off = 0;
      if (++rt == a.RT) {
        rt = 0;
        ++s;
      }
    }
    return true;
  }
  // the next stretch with positions in it
  __device__ __forceinline__ bool next_real(const DecodeArgs& a, Segment& g) {
    while (next(a, g))
      if (g.len > 0) return true;
    return false;
  }
};

// Units before sequence `upto` and of all sequences, by every thread of the
// block; `red` holds 2 x 32 values.
__device__ __forceinline__ void unit_sums(const DecodeArgs& a, int upto, int64_t* red, int64_t& before,
                                          int64_t& total) {
  int64_t b = 0, t = 0;
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const int64_t u = static_cast<int64_t>(group_units(seq_len(a, s))) * a.RT;
    t += u;
    if (s < upto) b += u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  }
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = b;
    red[32 + (threadIdx.x >> 5)] = t;
  }
  __syncthreads();
  before = total = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    before += red[w];
    total += red[32 + w];
  }
}

// Floats of one part: rows x L accumulators, then the rows' maxima and sums.
__host__ __device__ __forceinline__ int64_t part_floats(int rows, int L) {
  return static_cast<int64_t>(rows) * (L + 2);
}

// Row j of a row group: its token and head; false for rows that pad the group.
__device__ __forceinline__ bool group_row(const DecodeArgs& a, int rt, int j, int& tok, int& head) {
  const int ti = j / a.HB;
  tok = (rt / a.head_blocks) * a.TPT + ti;
  head = (rt % a.head_blocks) * a.HB + (j - ti * a.HB);
  return ti < a.TB && tok < a.q_len && head < a.H;
}

template <int NB>
__global__ void __launch_bounds__(kDecThreads, 1)
    mla_decode_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rmap,
                      const __grid_constant__ CUtensorMap cmap, const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nk = a.L >> 7;                                  // 128-value pieces of the latent
  uint8_t* psm = smem;                                      // P^T: 128 positions x 128 bytes
  uint8_t* rope = psm + kChunkBytes;                        // two rotated-key tiles
  uint8_t* ring = rope + 2 * kChunkBytes;
  uint8_t* qsm = ring + a.stages * kDecStageBytes;          // 2 nk + 1 chunks of NB rows x 64 values
  constexpr int kQChunk = NB * 128;

  __shared__ __align__(8) uint64_t full[2][kDecMaxStages], empty[kDecMaxStages];
  __shared__ __align__(8) uint64_t rope_full[2], s_full[2], p_full[2];
  __shared__ __align__(8) uint64_t q_full, pv_done, o_empty, drain[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int64_t red64[64];
  __shared__ Walk walk0;
  __shared__ __align__(16) float mref[NB], fac[NB], colmax[4][NB];
  __shared__ __align__(16) int lim[NB];
  __shared__ int64_t row_off[NB];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool abort = false;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[0][s], 1);
      mbar_init(&full[1][s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&rope_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&drain[i], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&pv_done, 1);
    mbar_init(&o_empty, 128);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  griddep_wait();
  // only now: the kernel behind reads seq_lens before its own wait
  if (threadIdx.x == 0) griddep_launch_dependents();

  // ---- this block's stretch of the units
  {
    int64_t none, total;
    unit_sums(a, 0, red64, none, total);
    // (at most one block per unit: blocks past that have no stretch)
    const int64_t n = min(static_cast<int64_t>(gridDim.x), total);
    const int64_t ub = blockIdx.x < n ? total * blockIdx.x / n : total;
    const int64_t ue = blockIdx.x < n ? total * (blockIdx.x + 1) / n : total;
    // the sequence that unit `ub` falls into: chunks of sequences per thread
    const int per = (a.S + kDecThreads - 1) / kDecThreads;
    const int s0 = threadIdx.x * per, s1 = min(a.S, s0 + per);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += static_cast<int64_t>(group_units(seq_len(a, s))) * a.RT;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) red64[warp] = incl;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < warp; ++w) base += red64[w];
    int64_t at = base + incl - mine;
    if (ub >= at && ub < at + mine) {
      int s = s0;
      for (; s < s1; ++s) {
        const int64_t u = static_cast<int64_t>(group_units(seq_len(a, s))) * a.RT;
        if (ub < at + u) break;
        at += u;
      }
      const int g = group_units(seq_len(a, s));
      walk0.left = ue - ub;
      walk0.s = s;
      walk0.rt = static_cast<int>((ub - at) / g);
      walk0.off = static_cast<int>((ub - at) % g);
    }
    if (threadIdx.x == 0 && ub >= ue) walk0.left = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  Walk walk = walk0;

  if (warp == 0) {
    // ---- copies.  Lane = (box of a tile, 64-value half of a piece).  A ring
    // slot has two full barriers, for pieces of the score and of the output
    // product: their issuers each see only their own pieces, and a barrier
    // whose phases one issuer skipped could be taken for complete a turn early.
    const int boxes = kTileTok / a.box_rows;
    const int box = lane >> 1, half = lane & 1;
    int slot = 0;
    uint32_t ph = 0;
    uint32_t fills[2] = {0, 0}, turn[2] = {0, 0};   // per slot: filled at all; parity of the next fill
    int i = 0, seg_no = 0;
    bool have_prev = false;
    int prev_page = 0, prev_row = 0, prev_boxes = 0;
    int rope_issued = 0;
    auto piece = [&](int use, int k, int page, int row, int nb) {
      if (!warp_wait(&empty[slot], ph ^ 1u, abort)) return;
      uint64_t* bar = &full[use][slot];
      if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(nb * a.box_rows * 256));
      __syncwarp();
      if (box < nb)
        tma_box_3d(ring + slot * kDecStageBytes + half * kChunkBytes + box * a.box_rows * 128, &cmap,
                   k * 128 + half * 64, row, page, bar);
      fills[use] |= 1u << slot;
      turn[use] ^= 1u << slot;
      if (++slot == a.stages) {
        slot = 0;
        ph ^= 1u;
      }
    };
    Segment g;
    while (!abort && walk.next_real(a, g)) {
      // the queries: their chunk buffer is free once the last score product of
      // the stretch before has read it
      if (seg_no > 0 && !warp_wait(&s_full[(i - 1) & 1], static_cast<uint32_t>((i - 1) >> 1) & 1u, abort)) break;
      const int h0 = (g.rt % a.head_blocks) * a.HB;
      const int tk0 = g.s * a.q_len + (g.rt / a.head_blocks) * a.TPT;
      if (lane == 0) mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>((2 * nk + 1) * a.HB * a.TB * 128));
      __syncwarp();
      if (lane < 2 * nk) tma_box_3d(qsm + lane * kQChunk, &qmap, lane * 64, h0, tk0, &q_full);
      if (lane == 31) tma_box_3d(qsm + 2 * nk * kQChunk, &rmap, 0, h0, tk0, &q_full);
      ++seg_no;
      for (int t = g.t0; t < g.t1; ++t, ++i) {
        const int tok0 = t * kTileTok;
        const int valid = min(kTileTok, g.len - tok0);
        const int nb = (valid + a.box_rows - 1) / a.box_rows;
        int page = 0, row = 0;
        if (box < nb && box < boxes) {
          const int tok = tok0 + box * a.box_rows;
          const int col = tok / a.page_size;
          row = tok - col * a.page_size;
          page = __ldg(a.page_table + g.s * a.table_stride + col);
          if (page < 0 || page >= a.num_pages) {
            atomicOr(&g_mla_decode_error, kErrIndex);
            page = a.num_pages;              // outside the map: the box is filled with zeros
          }
        }
        for (int k = 0; k < nk && !abort; ++k) piece(0, k, page, row, nb);
        if (abort) break;
        // the rotated keys; the buffer is free once tile i - 2's scores are formed
        if (i >= 2 && !warp_wait(&s_full[i & 1], static_cast<uint32_t>((i >> 1) + 1) & 1u, abort)) break;
        if (lane == 0) mbar_arrive_expect_tx(&rope_full[i & 1], static_cast<uint32_t>(nb * a.box_rows * 128));
        __syncwarp();
        if (half == 0 && box < nb)
          tma_box_3d(rope + (i & 1) * kChunkBytes + box * a.box_rows * 128, &cmap, a.L, row, page, &rope_full[i & 1]);
        ++rope_issued;
        if (have_prev)
          for (int k = 0; k < nk && !abort; ++k) piece(1, k, prev_page, prev_row, prev_boxes);
        if (abort) break;
        have_prev = true;
        prev_page = page;
        prev_row = row;
        prev_boxes = nb;
      }
    }
    if (have_prev)
      for (int k = 0; k < nk && !abort; ++k) piece(1, k, prev_page, prev_row, prev_boxes);
    if (abort) {
      // give the copies in flight a bounded time to land
      for (int s = 0; s < 2 * a.stages; ++s) {
        const int u = s & 1, at = s >> 1;
        bool late = false;
        if ((fills[u] >> at) & 1u) mbar_wait(&full[u][at], ((turn[u] >> at) & 1u) ^ 1u, late);
      }
      for (int b = 0; b < 2 && b < rope_issued; ++b) {
        bool late = false;
        const int last = rope_issued - 1 - ((rope_issued - 1 - b) & 1);
        mbar_wait(&rope_full[b], static_cast<uint32_t>(last >> 1) & 1u, late);
      }
      bool late = false;
      if (seg_no > 0) mbar_wait(&q_full, static_cast<uint32_t>(seg_no - 1) & 1u, late);
    }
  } else if (warp == 1) {
    // ---- score products S^T = C Q^T
    constexpr uint32_t idesc = idesc_bf16(128, NB);
    int slot = 0;
    uint32_t turn = 0;                       // parity of each slot's next fill for this issuer
    int i = 0, seg_no = 0;
    Segment g;
    auto skip = [&](int n) {
      slot += n;
      while (slot >= a.stages) slot -= a.stages;
    };
    const uint32_t ring_a = smem_u32(ring), q_a = smem_u32(qsm), rope_a = smem_u32(rope);
    while (!abort && walk.next_real(a, g)) {
      if (!warp_wait(&q_full, static_cast<uint32_t>(seg_no) & 1u, abort)) break;
      ++seg_no;
      for (int t = g.t0; t < g.t1; ++t, ++i) {
        const uint32_t d = tmem + kDecScol + static_cast<uint32_t>(i & 1) * 64u;
        // tile i - 2's scores have been read once its weights are out
        if (i >= 2 && !warp_wait(&p_full[i & 1], static_cast<uint32_t>((i >> 1) + 1) & 1u, abort)) break;
        for (int k = 0; k < nk; ++k) {
          if (!warp_wait(&full[0][slot], (turn >> slot) & 1u, abort)) break;
          turn ^= 1u << slot;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = ring_a + static_cast<uint32_t>(slot) * kDecStageBytes;
#pragma unroll
            for (int m = 0; m < 8; ++m)
              mma_bf16(d, sdesc_sw128(sa + (m >> 2) * kChunkBytes + (m & 3) * 32),
                       sdesc_sw128(q_a + (2 * k + (m >> 2)) * kQChunk + (m & 3) * 32), idesc, (k | m) != 0);
            mma_commit(&empty[slot]);
          }
          __syncwarp();
          skip(1);
        }
        if (abort || !warp_wait(&rope_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, abort)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sa = rope_a + static_cast<uint32_t>(i & 1) * kChunkBytes;
#pragma unroll
          for (int m = 0; m < 4; ++m)
            mma_bf16(d, sdesc_sw128(sa + m * 32), sdesc_sw128(q_a + 2 * nk * kQChunk + m * 32), idesc, 1u);
          mma_commit(&s_full[i & 1]);
        }
        __syncwarp();
        if (i > 0) skip(nk);                 // tile i - 1's pieces for the output product
      }
    }
    drain_mmas(&drain[0], abort);
  } else if (warp == 2) {
    // ---- output products O^T += C^T P^T
    constexpr uint32_t idesc = idesc_bf16(128, NB) | kIdescAMn | kIdescBMn;
    int slot = 0;
    uint32_t turn = 0;                       // parity of each slot's next fill for this issuer
    int i = 0, seg_no = 0;
    auto skip = [&](int n) {
      slot += n;
      while (slot >= a.stages) slot -= a.stages;
    };
    const uint32_t ring_a = smem_u32(ring), p_a = smem_u32(psm);
    Segment g, ahead;
    bool more = walk.next_real(a, ahead);
    skip(nk);                                // tile 0's pieces for the scores
    while (!abort && more) {
      g = ahead;
      more = walk.next_real(a, ahead);
      // the accumulator: the stretch before has been read out
      if (seg_no > 0 && !warp_wait(&o_empty, static_cast<uint32_t>(seg_no - 1) & 1u, abort)) break;
      ++seg_no;
      for (int t = g.t0; t < g.t1; ++t, ++i) {
        if (more || t + 1 < g.t1) skip(nk);  // tile i + 1's pieces for the scores
        const int valid = min(kTileTok, g.len - t * kTileTok);
        const int ks = (valid + 15) >> 4;    // 16-position steps that hold anything
        if (!warp_wait(&p_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, abort)) break;
        for (int k = 0; k < nk; ++k) {
          if (!warp_wait(&full[1][slot], (turn >> slot) & 1u, abort)) break;
          turn ^= 1u << slot;
          if ((valid & 15) != 0) {
            // rows of the last step past the sequence may hold anything
            // (0 x NaN): their weights are 0 and they are made 0 too
            uint8_t* st = ring + slot * kDecStageBytes;
            zero_rows(st, valid, ks * 16, lane);
            zero_rows(st + kChunkBytes, valid, ks * 16, lane);
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = sdesc_mn_sw128(ring_a + static_cast<uint32_t>(slot) * kDecStageBytes, kChunkBytes);
            const uint64_t bd = sdesc_mn_sw128(p_a, kChunkBytes);
            for (int m = 0; m < ks; ++m)
              mma_bf16(tmem + static_cast<uint32_t>(k) * 64u, ad + static_cast<uint64_t>(m) * 128u,
                       bd + static_cast<uint64_t>(m) * 128u, idesc, t != g.t0 || m != 0);
            mma_commit(&empty[slot]);
          }
          __syncwarp();
          skip(1);
        }
        if (abort) break;
        if (elect_one()) mma_commit(&pv_done);
        __syncwarp();
      }
    }
    drain_mmas(&drain[1], abort);
  } else if (warp >= 4) {
    // ---- softmax and output.  These threads meet at named barriers, so they
    // walk every tile even after a wait has given up.
    const int w = warp & 3, tid = threadIdx.x - 128;
    const uint32_t tl = tmem + (static_cast<uint32_t>(w * 32) << 16);
    float l[NB];
    int i = 0;
    Segment g;
    while (walk.next(a, g)) {
      // the rows of this group
      if (tid < NB) {
        int tok, head;
        const bool on = group_row(a, g.rt, tid, tok, head);
        const int n = g.len - a.q_len + 1 + tok;
        lim[tid] = on && n > 0 ? min(n, g.len) : 0;
        row_off[tid] = on ? (static_cast<int64_t>(g.s) * a.q_len + tok) * a.o_tok + head * a.o_head : -1;
      }
      named_sync(1, 128);
      const bool whole = g.t0 == 0 && g.t1 == g.nt;
      if (g.len > 0) {
#pragma unroll
        for (int j = 0; j < NB; ++j) l[j] = 0.f;
        for (int t = g.t0; t < g.t1; ++t, ++i) {
          const int pos = t * kTileTok + tid;
          // every row sees the whole tile: lim of the first token is the least
          const bool inside = (t + 1) * kTileTok <= g.len - a.q_len + 1;
          uint32_t r[NB];
          mbar_wait(&s_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, abort);
          __syncwarp();
          tc_fence_after();
          tmem_ld_cols<NB>(tl + kDecScol + static_cast<uint32_t>(i & 1) * 64u, r);
          tmem_wait_ld_of(r);
          if (!inside) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
              r[j] = pos < lim[j] ? __float_as_uint(__uint_as_float(r[j]) * a.c) : 0xFF800000u;
          } else {
#pragma unroll
            for (int j = 0; j < NB; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * a.c);
          }
          const bool first = t == g.t0;
          bool raise = first;
          if (!first) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < NB; j += 4) {
              const float4 m = *reinterpret_cast<const float4*>(&mref[j]);
              mx = fmaxf(mx, fmaxf(fmaxf(__uint_as_float(r[j]) - m.x, __uint_as_float(r[j + 1]) - m.y),
                                   fmaxf(__uint_as_float(r[j + 2]) - m.z, __uint_as_float(r[j + 3]) - m.w)));
            }
            raise = named_sync_or(1, 128, mx > kMaxSlack);
          }
          if (raise) {
            float keep0 = -INFINITY, keep1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              float v = __uint_as_float(r[j]);
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
              if (lane == (j & 31)) {
                if (j < 32) keep0 = v;
                else keep1 = v;
              }
            }
            if (lane < NB) colmax[w][lane] = keep0;
            if (NB > 32) colmax[w][32 + lane] = keep1;
            named_sync(1, 128);
            if (tid < NB) {
              float m = fmaxf(fmaxf(colmax[0][tid], colmax[1][tid]), fmaxf(colmax[2][tid], colmax[3][tid]));
              if (!first) m = fmaxf(m, mref[tid]);
              if (m == -INFINITY) m = 0.f;           // a row that sees nothing here sees nothing later
              fac[tid] = first ? 0.f : exp2_fast(mref[tid] - m);
              mref[tid] = m;
            }
            named_sync(1, 128);
            if (!first) {
              mbar_wait(&pv_done, static_cast<uint32_t>(i - 1) & 1u, abort);
              __syncwarp();
              tc_fence_after();
              for (int k = 0; k < nk; ++k) {
#pragma unroll
                for (int j = 0; j < NB; j += 16) {
                  uint32_t o[16];
                  tmem_ld16(tl + k * 64 + j, o);
                  tmem_wait_ld_of(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fac[j + e]);
                  tmem_st16(tl + k * 64 + j, o);
                }
              }
              tmem_wait_st();
#pragma unroll
              for (int j = 0; j < NB; ++j) l[j] *= fac[j];
            }
          }
          // weights, their sums, and the tile P^T (fp32 sums of the unrounded
          // weights; the weights themselves are rounded to bf16 for the MMA)
#pragma unroll
          for (int j = 0; j < NB; j += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&mref[j]);
            const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = exp2_fast(__uint_as_float(r[j + e]) - mm[e]);
              l[j + e] += p;
              r[j + e] = __float_as_uint(p);
            }
          }
          if (i > 0) {
            mbar_wait(&pv_done, static_cast<uint32_t>(i - 1) & 1u, abort);
            __syncwarp();
          }
          uint8_t* prow = psm + tid * 128;
#pragma unroll
          for (int ch = 0; ch < NB / 8; ++ch) {
            const uint32_t* v = &r[8 * ch];
            *reinterpret_cast<uint4*>(prow + ((ch ^ (tid & 7)) << 4)) =
                make_uint4(pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                           pack_bf16x2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                           pack_bf16x2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                           pack_bf16x2(__uint_as_float(v[6]), __uint_as_float(v[7])));
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&p_full[i & 1]);
        }
        // sums over the 128 positions of each thread's share: halves of the
        // columns change hands until a lane holds its own
        {
          int n = NB / 2, o = 16;
#pragma unroll
          for (; n >= 1 && o >= 1; n >>= 1, o >>= 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int j = 0; j < NB / 2; ++j) {
              if (j < n) {
                const float give = up ? l[j] : l[j + n], have = up ? l[j + n] : l[j];
                l[j] = have + __shfl_xor_sync(0xFFFFFFFFu, give, o);
              }
            }
          }
#pragma unroll
          for (; o >= 1; o >>= 1) l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], o);
        }
        if (NB == 64) {
          colmax[w][2 * lane] = l[0];
          colmax[w][2 * lane + 1] = l[1];
        } else if (NB == 32) {
          colmax[w][lane] = l[0];
        } else if ((lane & 1) == 0) {
          colmax[w][lane >> 1] = l[0];
        }
        named_sync(1, 128);
        float* part = a.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (g.t0 == 0 ? 1 : 0)) * part_floats(NB, a.L);
        if (tid < NB) {
          const float sum = (colmax[0][tid] + colmax[1][tid]) + (colmax[2][tid] + colmax[3][tid]);
          if (whole) {
            fac[tid] = sum == 0.f ? 0.f : 1.0f / sum;
            if (a.lse != nullptr && row_off[tid] >= 0) {
              int tok, head;
              group_row(a, g.rt, tid, tok, head);
              a.lse[(static_cast<int64_t>(g.s) * a.q_len + tok) * a.H + head] =
                  sum == 0.f ? -INFINITY : (mref[tid] + log2_fast(sum)) * kLn2;
            }
          } else if (row_off[tid] >= 0) {
            part[static_cast<int64_t>(NB) * a.L + tid] = sum == 0.f ? -INFINITY : mref[tid];
            part[static_cast<int64_t>(NB) * a.L + NB + tid] = sum;
          }
        }
        named_sync(1, 128);
        mbar_wait(&pv_done, static_cast<uint32_t>(i - 1) & 1u, abort);
        __syncwarp();
        tc_fence_after();
        for (int k = 0; k < nk; ++k) {
          uint32_t o[NB];
          tmem_ld_cols<NB>(tl + k * 64, o);
          tmem_wait_ld_of(o);
          if (k == nk - 1) {
            tc_fence_before();
            mbar_arrive(&o_empty);
          }
          const int d = k * 128 + w * 32 + lane;
          if (whole) {
            // two rows per pass: lane pairs swap a value so that each lane
            // stores two neighbouring ones
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
              const float f0 = fac[j], f1 = fac[j + 1];
              const float x0 = f0 == 0.f ? 0.f : __uint_as_float(o[j]) * f0;
              const float x1 = f1 == 0.f ? 0.f : __uint_as_float(o[j + 1]) * f1;
              const bool odd = (lane & 1) != 0;
              const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? x0 : x1, 1);
              const int64_t off = row_off[j + (odd ? 1 : 0)];
              if (off >= 0)
                *reinterpret_cast<uint32_t*>(a.out + off + (d & ~1)) = odd ? pack_bf16x2(got, x1) : pack_bf16x2(x0, got);
            }
          } else {
#pragma unroll
            for (int j = 0; j < NB; ++j)
              if (row_off[j] >= 0) part[static_cast<int64_t>(j) * a.L + d] = __uint_as_float(o[j]);
          }
        }
      } else {
        // an empty sequence: its rows are zero, their log-sum -inf
        for (int j = 0; j < NB; ++j) {
          if (row_off[j] < 0) continue;
          for (int d = tid * 8; d < a.L; d += 128 * 8)
            *reinterpret_cast<uint4*>(a.out + row_off[j] + d) = make_uint4(0, 0, 0, 0);
          if (a.lse != nullptr && tid == 0) {
            int tok, head;
            group_row(a, g.rt, j, tok, head);
            a.lse[(static_cast<int64_t>(g.s) * a.q_len + tok) * a.H + head] = -INFINITY;
          }
        }
      }
      named_sync(1, 128);                    // the row tables are rewritten next
    }
  }
  if (abort) atomicOr(&g_mla_decode_error, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ joining
// out[r] = sum_p 2^(m_p - M) O_p[r] / sum_p 2^(m_p - M) l_p over the parts p
// of a row group that was cut between blocks, in block order (the result
// does not depend on timing).  One block per group and `rows` rows; four
// groups of 128 threads (four values each, L <= 512) share out the parts.
constexpr int kCombThreads = 512;

__global__ void __launch_bounds__(kCombThreads) mla_combine_kernel(const DecodeArgs a, int grid, int NB, int rows) {
  __shared__ int64_t red64[64];
  __shared__ float wsum[4][kMlaMaxLatent];
  __shared__ float lsum[4];
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int group = blockIdx.x, s = group / a.RT, rt = group % a.RT;
  int64_t before, total;
  unit_sums(a, s, red64, before, total);     // seq_lens: complete before the kernel ahead let this one start
  const int units = group_units(seq_len(a, s));
  const int64_t u0 = before + static_cast<int64_t>(rt) * units, u1 = u0 + units;
  // owner(u): the block c whose stretch [c total / n, (c + 1) total / n) holds u
  const int64_t n = min(static_cast<int64_t>(grid), total);
  const int c0 = static_cast<int>(((u0 + 1) * n - 1) / total), c1 = static_cast<int>((u1 * n - 1) / total);
  griddep_wait();                            // (every block: the grid must not end before the one ahead)
  if (c0 == c1) return;                      // not cut: written by its block
  const int64_t pf = part_floats(NB, a.L);
  const int tg = threadIdx.x >> 7, x = threadIdx.x & 127;
  auto part = [&](int c) { return a.parts + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * pf; };
  for (int j = blockIdx.y * rows; j < min(NB, static_cast<int>(blockIdx.y + 1) * rows); ++j) {
    int tok, head;
    if (!group_row(a, rt, j, tok, head)) continue;
    const int64_t mo = static_cast<int64_t>(NB) * a.L + j;
    float M = -INFINITY;
    for (int c = c0; c <= c1; ++c) M = fmaxf(M, part(c)[mo]);
    const float ref = M == -INFINITY ? 0.f : M;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll 4
    for (int c = c0 + tg; c <= c1; c += 4) {
      const float* p = part(c);
      const float lp = p[mo + NB];
      const float wgt = exp2_fast(p[mo] - ref);
      const float4 v = 4 * x < a.L ? *reinterpret_cast<const float4*>(p + static_cast<int64_t>(j) * a.L + 4 * x)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
      if (lp != 0.f) {                       // a part whose positions this row does not see
        l += wgt * lp;
        acc[0] += wgt * v.x;
        acc[1] += wgt * v.y;
        acc[2] += wgt * v.z;
        acc[3] += wgt * v.w;
      }
    }
    if (x == 0) lsum[tg] = l;
#pragma unroll
    for (int e = 0; e < 4; ++e) wsum[tg][4 * x + e] = acc[e];
    __syncthreads();
    const float lt = (lsum[0] + lsum[1]) + (lsum[2] + lsum[3]);
    if (tg == 0 && 4 * x < a.L) {
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = (wsum[0][4 * x + e] + wsum[1][4 * x + e]) + (wsum[2][4 * x + e] + wsum[3][4 * x + e]);
        o[e] = lt == 0.f ? 0.f : v / lt;
      }
      __nv_bfloat16* dst = a.out + (static_cast<int64_t>(s) * a.q_len + tok) * a.o_tok + head * a.o_head + 4 * x;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      if (x == 0 && a.lse != nullptr)
        a.lse[(static_cast<int64_t>(s) * a.q_len + tok) * a.H + head] =
            lt == 0.f ? -INFINITY : (M + log2_fast(lt)) * kLn2;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host
struct RowSplit {
  int HB, TPT, TB, head_blocks, RT, NB;
};
// Query rows of a sequence in groups of at most 64: a token's heads in blocks
// of up to 64, and as many tokens as fit where there are fewer heads.
static RowSplit split_rows(int q_len, int H) {
  RowSplit r{};
  r.HB = H < 64 ? H : 64;
  r.TPT = 64 / r.HB;
  r.TB = r.TPT < q_len ? r.TPT : q_len;
  r.head_blocks = static_cast<int>(ceil_div(H, r.HB));
  r.RT = r.head_blocks * static_cast<int>(ceil_div(q_len, r.TPT));
  const int rows = r.HB * r.TB;
  r.NB = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
  return r;
}

static int decode_grid(int S, const RowSplit& r, int64_t capacity, int sm_count) {
  const int64_t most = static_cast<int64_t>(S) * r.RT * ceil_div(capacity > 0 ? capacity : 1, kTileTok);
  const int lim = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  return static_cast<int>(most < lim ? most : lim);
}

size_t mla_decode_workspace(int S, int q_len, int H, int L, int64_t max_len, int sm_count) {
  if (max_len <= kTileTok) return 0;         // one tile a sequence: nothing is cut
  const RowSplit r = split_rows(q_len, H);
  return static_cast<size_t>(decode_grid(S, r, max_len, sm_count)) * 2 * part_floats(r.NB, L) * sizeof(float);
}

bool mla_decode_fits(int S, int q_len, int H) {
  const int64_t tokens = static_cast<int64_t>(S) * q_len;
  return tokens * ceil_div(H, 64) < 0x7FFFFFFF;
}

static std::atomic<bool> g_decode_attr[3][64];

template <int NB>
static cudaError_t launch_decode_nb(const CUtensorMap (&maps)[3], DecodeArgs a, int grid, const DeviceInfo& dev,
                                    cudaStream_t s) {
  constexpr int kIdx = NB == 64 ? 2 : (NB == 32 ? 1 : 0);
  auto kern = mla_decode_kernel<NB>;
  if (!g_decode_attr[kIdx][dev.device].load(std::memory_order_acquire)) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kDecSmem - static_cast<int>(fa.sharedSizeBytes));
    if (e != cudaSuccess) return e;
    g_decode_attr[kIdx][dev.device].store(true, std::memory_order_release);
  }
  // ring stages that fit beside the queries, the weights and two rotated-key tiles
  const int fixed = 3 * kChunkBytes + (a.L / 64 + 1) * NB * 128 + 1024;
  int st = (kDecSmem - 4096 - fixed) / kDecStageBytes;
  if (st > kDecMaxStages) st = kDecMaxStages;
  a.stages = st;
  return mla_launch(kern, dim3(static_cast<unsigned>(grid)), kDecThreads, fixed + st * kDecStageBytes, s, maps[0],
                    maps[1], maps[2], a);
}

cudaError_t launch_mla_decode(const MlaDecodeProblem& p, const DeviceInfo& dev, cudaStream_t s) {
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
  cudaError_t e = mla_bind_context();
  if (e != cudaSuccess) return e;
  const RowSplit r = split_rows(p.q_len, p.H);
  DecodeArgs a{};
  a.page_table = p.page_table;
  a.seq_lens = p.seq_lens;
  a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(p.out.p));
  a.lse = p.lse;
  a.parts = static_cast<float*>(p.workspace);
  a.table_stride = p.table_stride;
  a.o_tok = p.out.tok;
  a.o_head = p.out.head;
  a.S = p.S;
  a.q_len = p.q_len;
  a.H = p.H;
  a.L = p.L;
  a.page_size = p.cache.page_size;
  a.num_pages = p.cache.num_pages;
  a.box_rows = kTileTok;                     // the largest power of two that pages divide into
  while (p.cache.page_size % a.box_rows != 0) a.box_rows >>= 1;
  a.capacity = static_cast<int64_t>(p.max_pages) * p.cache.page_size;
  if (a.capacity > 0x7FFFFF00) a.capacity = 0x7FFFFF00;
  a.HB = r.HB;
  a.TB = r.TB;
  a.TPT = r.TPT;
  a.head_blocks = r.head_blocks;
  a.RT = r.RT;
  a.c = p.scale * kLog2e;

  CUtensorMap maps[3];
  const int64_t T = static_cast<int64_t>(p.S) * p.q_len;
  const int64_t row = p.L + kMlaRope;
  if ((e = mla_tensor_map(&maps[0], p.q_lat.p, p.L, p.H, T, p.q_lat.head, p.q_lat.tok, 64, r.HB, r.TB)) != cudaSuccess)
    return e;
  if ((e = mla_tensor_map(&maps[1], p.q_rope.p, kMlaRope, p.H, T, p.q_rope.head, p.q_rope.tok, 64, r.HB, r.TB)) !=
      cudaSuccess)
    return e;
  if ((e = mla_tensor_map(&maps[2], p.cache.p, row, p.cache.page_size, p.cache.num_pages, row, p.cache.page_stride, 64,
                          a.box_rows, 1)) != cudaSuccess)
    return e;
  const int grid = decode_grid(p.S, r, a.capacity, dev.sm_count);
  e = r.NB == 16 ? launch_decode_nb<16>(maps, a, grid, dev, s)
                 : (r.NB == 32 ? launch_decode_nb<32>(maps, a, grid, dev, s)
                               : launch_decode_nb<64>(maps, a, grid, dev, s));
  if (e != cudaSuccess || a.capacity <= kTileTok) return e;
  // rows per joining block: enough blocks for a few per SM
  const int64_t groups = static_cast<int64_t>(p.S) * r.RT;
  int rows = static_cast<int>(groups * r.NB / (4 * dev.sm_count));
  rows = rows < 1 ? 1 : (rows > 16 ? 16 : rows);
  return mla_launch(mla_combine_kernel, dim3(static_cast<unsigned>(groups), static_cast<unsigned>(ceil_div(r.NB, rows))),
                    kCombThreads, 0, s, a, grid, r.NB, rows);
}

uint32_t mla_decode_read_clear_error() { return read_clear_word(g_mla_decode_error); }

}  // namespace mx
