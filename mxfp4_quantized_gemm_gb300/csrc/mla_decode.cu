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
// the positions in tiles of 64, each read once: two tiles (74 KB each at
// L = 512) and the queries (74 KB) fill shared memory.  The accumulator of
// 64 rows x 512 latent values must stay in TMEM, whose 512 columns a 128-row
// fp32 accumulator of that width would fill by itself, so the output product
// is formed transposed:
//   S   [64 rows][64 positions]      = Q C^T
//   O^T [128 latent values][rows]   += C^T P^T   (L / 128 blocks of 64 columns)
// which takes 256 columns and leaves room for two score tiles.  C is the B
// operand of the first product (latent values along K) and the A operand of
// the second (along M).
//
// Roles: warp 0 copies, warp 1 issues the score products, warp 2 the output
// products; warps 4..7 and 8..11 hold the softmax of a half of the tile's
// positions each; warps 12..15 write a finished accumulator out while the
// softmax is at the next stretch (131 KB of fp32 for a part: done by the softmax
// warps it stood for 17000 cycles between two stretches, four tiles' worth).  A
// row's running maximum is raised only when a score passes it by 2^8 (first
// tile aside), which one barrier with an OR decides.
//
// Where a tile's time goes (64 sequences of 4096, cycles of 4100 a tile): its
// place is free again about 8000 cycles after it was asked for, two at a time:
// 3200 to 3700 until it lands from HBM, 1600 of score products, 1000 of softmax,
// 1300 of output products.  Shared memory alone needs 2500 (operands and copies
// at 128 bytes a cycle), and so it is how long a place is held, with two of them,
// that sets the pace.  A third tile does not fit beside 64 rows of queries; beside
// 16 or 32 rows 2.8 or 2.5 tiles would, of which two whole ones are used.
// A copying warp spends about 430 cycles on each wait, arrival and copy, and
// each copy more costs it 16 by one thread and about 100 by lanes in turns.  Where
// a page holds whole tiles a group of chunks is one copy, and a tile comes in
// groups of 128 latent values, the last with the rotated key: each is multiplied
// as it lands and given back as the output product is done with it (16 x 4096
// 25.0 us, in two groups 25.5).  Smaller pages take a copy for each box of rows
// and chunk, by lanes that hold a box's page each, in two groups (32 x 3001 in
// pages of 16: 27.8 us; in four groups 30.4, by one thread 34.3).
//
// Work split: the tiles of all row groups, in order, are cut evenly over the
// grid; a block takes its stretch wherever sequences begin and end, so a
// single long sequence spreads over all SMs.  A row group cut between blocks
// leaves unnormalized parts (fp32, with maximum and sum) that
// mla_combine_kernel joins.
//
// Measured (rates by the bytes of the cache read once): 64 ragged sequences of up
// to 8192, 64 rows: 80.3 us, 4.3 TB/s; one of 131072: 42.8 us, 3.5 TB/s; 16 of up to
// 4096: 24.6 us.  From the end of the call ahead, in us (time stamps of calls in
// a graph, median block; where a block ends, the last one in brackets):
//                   first copy landed   last weights   block's end    joined, last
//   16 x 4096              3.4              11.0       14.2 (16.3)       22.5
//   1 x 131072             4.4              29.8       33.0 (34.7)       41.8
//   64 x 8192              3.7              63.6       66.7 (74.4)       82.1
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>

#include "mla.h"
#include "mla_common.cuh"

namespace mx {

static __device__ uint32_t g_mla_decode_error;

constexpr int kDecThreads = 512;
constexpr int kTileTok = 64;                        // positions per tile
constexpr int kChunkBytes = kTileTok * 128;         // 64 positions x 64 values
constexpr int kDecMaxBufs = 4;
constexpr int kDecSmem = 227 * 1024;
constexpr int kDecStatic = 2048;                    // most of it that the static part takes
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
  int bufs;               // tiles in shared memory
  int over;               // units that going over to another row group counts as
  int q_box, wide;        // chunks of the queries per copy; whether a copy takes all of a tile's group
  float c;                // |scale| * log2(e)
  bool flip;              // scale < 0: the scores change sign first
};

// Positions of sequence s (a bad length is cut to what the table holds).
__device__ __forceinline__ int cut_len(const DecodeArgs& a, int n) {
  return n < 0 ? 0 : (n > a.capacity ? static_cast<int>(a.capacity) : n);
}
__device__ __forceinline__ int seq_len(const DecodeArgs& a, int s) { return cut_len(a, __ldg(a.seq_lens + s)); }
// Work units of one row group: `over` for going over to it (queries to fetch, a
// part or the rows before it to write out), then its tiles; or one for an empty
// sequence (whose rows still have to be written).
__device__ __forceinline__ int group_units(int over, int len) {
  return len == 0 ? 1 : over + (len + kTileTok - 1) / kTileTok;
}
// Going over counts as three tiles where the blocks have 24 units and more of it
// counted as one, else as one: see decode_over.
__device__ __forceinline__ bool long_stretches(const DecodeArgs& a, int64_t units, int grid) {
  return a.over > 0 && units * a.RT >= 24 * static_cast<int64_t>(grid);
}
constexpr int kLongOver = 3;

// total / n and the like, in 32 bits where they fit (a 64-bit division takes
// several times as long, and this is on the way to the first load).
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The units 0 .. total - 1 cut over n blocks, the first total % n of which
// take one more.
struct Cut {
  int64_t q, r;
  __device__ __forceinline__ Cut(int64_t total, int grid, int& n) {
    n = total < grid ? static_cast<int>(total) : grid;
    q = div64(total, n);
    r = total - q * n;
  }
  __device__ __forceinline__ int64_t begin(int c) const { return c * q + (c < r ? c : r); }
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t big = (q + 1) * r;
    return static_cast<int>(u < big ? div64(u, q + 1) : r + div64(u - big, q));
  }
};

// A stretch of one row group's tiles.
struct Segment {
  int s, rt, len, t0, t1, nt;
};
// A block's stretch of the unit order (sequence, row group, going over, tiles).
struct Walk {
  int64_t left;       // units still to hand out
  int s, rt, off;
  int over;           // units of going over to a row group
  int own[2];         // up to 64 sequences: the lengths of the lane's
  static constexpr int kOwn = 64;
  // (from L2: it may be read before the kernels ahead are done, and again then)
  __device__ __forceinline__ void read_own(const DecodeArgs& a) {
    const int lane = threadIdx.x & 31, s0 = a.S <= 32 ? lane : 2 * lane, s1 = a.S <= 32 ? a.S : s0 + 1;
    const int n0 = s0 < a.S ? ld_relaxed(a.seq_lens + s0) : 0, n1 = s1 < a.S ? ld_relaxed(a.seq_lens + s1) : 0;
    own[0] = cut_len(a, n0);
    own[1] = cut_len(a, n1);
  }
  // (the whole warp)
  __device__ __forceinline__ int len_of(const DecodeArgs& a, int seq) const {
    if (a.S <= 32) return __shfl_sync(0xFFFFFFFFu, own[0], seq);
    if (a.S <= kOwn) return __shfl_sync(0xFFFFFFFFu, (seq & 1) ? own[1] : own[0], seq >> 1);
    return seq_len(a, seq);
  }
  // The block's stretch, found by each warp for itself (one round of loads,
  // no barrier).
  __device__ __forceinline__ void start(const DecodeArgs& a) {
    const int lane = threadIdx.x & 31;
    const int per = (a.S + 31) >> 5, s0 = min(a.S, lane * per), s1 = min(a.S, s0 + per);
    int64_t mine, incl;
    over = a.over;
#pragma unroll 1
    for (;;) {                               // (once, or twice in long stretches)
      mine = 0;
      if (a.S <= kOwn) {
        if (s0 < s1) mine = group_units(over, own[0]);
        if (s0 + 1 < s1) mine += group_units(over, own[1]);
      } else {
#pragma unroll 4
        for (int i = s0; i < s1; ++i) mine += group_units(over, seq_len(a, i));
      }
      incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      if (over == kLongOver || !long_stretches(a, __shfl_sync(0xFFFFFFFFu, incl, 31), static_cast<int>(gridDim.x))) break;
      over = kLongOver;
    }
    int n;
    const Cut cut(__shfl_sync(0xFFFFFFFFu, incl, 31) * a.RT, static_cast<int>(gridDim.x), n);
    left = 0;
    s = rt = off = 0;
    const int b = static_cast<int>(blockIdx.x);
    if (b >= n) return;
    const int64_t ub = cut.begin(b);
    left = cut.begin(b + 1) - ub;
    int64_t at = (incl - mine) * a.RT;
    const bool here = ub >= at && ub < incl * a.RT;
    if (here) {
      for (s = s0; s < s1; ++s) {
        const int g = group_units(over, a.S <= kOwn ? (s == s0 ? own[0] : own[1]) : seq_len(a, s));
        const int64_t u = static_cast<int64_t>(g) * a.RT;
        if (ub < at + u) {
          rt = static_cast<int>(div64(ub - at, g));
          off = static_cast<int>(ub - at - static_cast<int64_t>(rt) * g);
          break;
        }
        at += u;
      }
    }
    const int from = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
    s = __shfl_sync(0xFFFFFFFFu, s, from);
    rt = __shfl_sync(0xFFFFFFFFu, rt, from);
    off = __shfl_sync(0xFFFFFFFFu, off, from);
  }
  __device__ __forceinline__ bool next(const DecodeArgs& a, Segment& g) {
    while (left > 0) {
      g.s = s;
      g.rt = rt;
      g.len = len_of(a, s);
      const int units = group_units(over, g.len), from = off;
      g.nt = g.len == 0 ? 0 : units - over;
      const int64_t room = units - off;
      const int take = static_cast<int>(left < room ? left : room);
      left -= take;
      off += take;
      g.t0 = max(0, from - over);
      g.t1 = min(g.nt, max(0, off - over));
      if (off == units) {
        off = 0;
        if (++rt == a.RT) {
          rt = 0;
          ++s;
        }
        // nothing but going over to the next group: left to the block behind
        if (left > 0 && left <= over && len_of(a, s) > 0) left = 0;
      }
      if (g.len == 0 || g.t0 < g.t1) return true;
    }
    return false;
  }
  // the next stretch with positions in it
  __device__ __forceinline__ bool next_real(const DecodeArgs& a, Segment& g) {
    while (next(a, g))
      if (g.len > 0) return true;
    return false;
  }
};

// Floats of one part: rows x L accumulators, then the rows' maxima and sums.
__host__ __device__ __forceinline__ int64_t part_floats(int rows, int L) {
  return static_cast<int64_t>(rows) * (L + 2);
}

// The part that block c leaves of the group it begins, or goes on with.
__device__ __forceinline__ float* part_of(const DecodeArgs& a, int rows, int c, bool begins) {
  return a.parts + (static_cast<int64_t>(c) * 2 + (begins ? 1 : 0)) * part_floats(rows, a.L);
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
                      const __grid_constant__ CUtensorMap cmap0, const __grid_constant__ CUtensorMap cmap1,
                      const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nk = a.L >> 7;                                  // 128-value blocks of the latent
  const int chunks = 2 * nk + 1;                            // 64-value chunks of a cache row
  const int tile_bytes = chunks * kChunkBytes;
  // groups of a tile's chunks: the last three chunks, and in front of them two
  // to a group, or one group of all
  const int groups = a.wide || nk == 1 ? nk : 2;
  // the 64-row score MMA reads 64 rows of a query chunk whatever NB is: the
  // queries lie in front, so that what it reads past them is inside the buffer
  uint8_t* qsm = smem;                                      // chunks of NB rows x 64 values
  uint8_t* psm = qsm + chunks * NB * 128;                   // P: NB rows x 64 positions
  uint8_t* ring = psm + NB * 128;
  constexpr int kQChunk = NB * 128;

  __shared__ __align__(8) uint64_t full[4][kDecMaxBufs], empty[4][kDecMaxBufs];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], q_full, q_empty, pv_done, o_empty, drain[2];
  // of a stretch, by its number's parity: the softmax may be a whole stretch
  // ahead of the warps that write out, but not two
  __shared__ __align__(8) uint64_t o_full[2], fin_full[2];
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float fac[64];
  __shared__ float xch[2][64];
  // 1 / sum of a finished stretch's rows, for the warps that write it out.  They
  // give the accumulator back before they are done with the sums, so that those
  // of two further stretches may come in beside them: three in use at most.
  __shared__ __align__(16) float fin[3][NB];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool abort = false;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDecMaxBufs; ++s)
      for (int x = 0; x < 4; ++x) {
        mbar_init(&full[x][s], 1);
        mbar_init(&empty[x][s], 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 256);
      mbar_init(&drain[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&fin_full[i], 256);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&pv_done, 1);
    mbar_init(&o_empty, 128);
    fence_mbar_init();
  }
  if (warp == 0 && lane < 4)
    prefetch_tensor_map(lane == 0 ? &qmap : (lane == 1 ? &rmap : (lane == 2 ? &cmap0 : &cmap1)));
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // The lengths are most often what they were a while ago: up to 64 are read
  // and the stretch found while the kernels ahead still run, and read again
  // when they are done.  (All of it behind the wait, with its code still to be
  // fetched, put the first copy 6000 to 9000 cycles behind it.)
  Walk walk;
  walk.left = 0;
  if (a.S <= Walk::kOwn) {
    walk.read_own(a);
    walk.start(a);
  }
  // after the wait: whether the stretch was not as found, and now is
  auto settle = [&]() {
    if (a.S <= Walk::kOwn) {
      const int was0 = walk.own[0], was1 = walk.own[1];
      walk.read_own(a);
      if (!__any_sync(0xFFFFFFFFu, walk.own[0] != was0 || walk.own[1] != was1)) return false;
    }
    walk.start(a);
    return true;
  };
  if (warp != 0) {
    griddep_wait();
    settle();
  }

  if (warp == 0) {
    // ---- copies.  Lane = (box of the tile's positions, chunk), in turns.
    const int boxes = kTileTok / a.box_rows;
    const int box = lane & (boxes - 1);      // the lane's box, in every group
    Ring r(a.bufs);
    int seg_no = 0, fills = 0;
    Segment g{};
    // The page and row of the lane's box of tile t, and the boxes that hold
    // anything; asked for a tile ahead.
    int page = 0, row = 0, nb = 0;
    const int32_t* entry = a.page_table;
    auto find = [&](int t) {
      const int tok0 = t * kTileTok;
      nb = (min(kTileTok, g.len - tok0) + a.box_rows - 1) / a.box_rows;
      if (box < nb) {
        const int tok = tok0 + box * a.box_rows;
        const int col = tok / a.page_size;
        row = tok - col * a.page_size;
        entry = a.page_table + g.s * a.table_stride + col;
      }
    };
    bool sure = false;                       // the kernels ahead are done
    while (!abort) {
      const bool more = walk.next_real(a, g);
      if (more) find(g.t0);
      if (!sure) {
        griddep_wait();
        sure = true;
        // only now: the kernel behind reads seq_lens before its own wait
        if (lane == 0) griddep_launch_dependents();
        if (more && box < nb) page = __ldg(entry);
        if (settle()) continue;
      } else if (more && box < nb) {
        page = __ldg(entry);
      }
      if (!more) break;
      // the queries: their buffer is free once the last score product of the
      // stretch before has read it (a barrier of its own: a parity says nothing
      // about one that may be two phases behind, as s_full is to this warp)
      if (seg_no > 0 && !warp_wait(&q_empty, static_cast<uint32_t>(seg_no - 1) & 1u, abort)) break;
      const int h0 = (g.rt % a.head_blocks) * a.HB;
      const int tk0 = g.s * a.q_len + (g.rt / a.head_blocks) * a.TPT;
      if (lane == 0) mbar_arrive_expect_tx(&q_full, static_cast<uint32_t>(chunks * a.HB * a.TB * 128));
      __syncwarp();
      if (elect_one()) {
        for (int c = 0; c < 2 * nk; c += a.q_box) tma_box_4d(qsm + c * kQChunk, &qmap, 0, h0, tk0, c, &q_full);
        tma_box_4d(qsm + 2 * nk * kQChunk, &rmap, 0, h0, tk0, 0, &q_full);
      }
      __syncwarp();
      ++seg_no;
      for (int t = g.t0; t < g.t1; ++t) {
        const int cur_nb = nb, cur_row = row;
        int cur_page = page;
        if (box < cur_nb && (cur_page < 0 || cur_page >= a.num_pages)) {
          atomicOr(&g_mla_decode_error, kErrIndex);
          cur_page = a.num_pages;            // outside the map: the box is filled with zeros
        }
        if (t + 1 < g.t1) {
          find(t + 1);
          if (box < nb) page = __ldg(entry);
        }
        uint8_t* buf = ring + r.slot * tile_bytes;
        for (int x = 0, c0 = 0; x < groups; ++x) {
          const int c1 = x + 1 == groups ? chunks : (groups == nk ? 2 * x + 2 : 2 * nk - 2);
          if (!warp_wait(&empty[x][r.slot], r.turn ^ 1u, abort)) break;
          const uint32_t bytes = static_cast<uint32_t>((c1 - c0) * cur_nb * a.box_rows * 128);
          if (a.wide) {
            // (a tile is one box's rows: every lane has the same page and row)
            if (elect_one()) {
              mbar_arrive_expect_tx(&full[x][r.slot], bytes);
              tma_box_4d(buf + c0 * kChunkBytes, x + 1 < groups ? &cmap0 : &cmap1, 0, cur_row, cur_page, c0,
                         &full[x][r.slot]);
            }
          } else {
            if (lane == 0) mbar_arrive_expect_tx(&full[x][r.slot], bytes);
            __syncwarp();
            if (box < cur_nb)
              for (int c = c0 + lane / boxes; c < c1; c += 32 / boxes)
                tma_box_4d(buf + c * kChunkBytes + box * a.box_rows * 128, &cmap0, 0, cur_row, cur_page, c,
                           &full[x][r.slot]);
          }
          __syncwarp();
          c0 = c1;
          ++fills;
        }
        if (abort) break;
        r.step();
      }
    }
    if (abort) {
      // give the copies in flight a bounded time to land
      for (int x = 0; x < groups; ++x) drain_copies(full[x], (fills + groups - 1 - x) / groups, a.bufs);
      bool late = false;
      if (seg_no > 0) mbar_wait(&q_full, static_cast<uint32_t>(seg_no - 1) & 1u, late);
    }
  } else if (warp == 1) {
    // ---- score products S = Q C^T
    constexpr uint32_t idesc = idesc_bf16(64, kTileTok);
    const uint32_t ring_a = smem_u32(ring), q_a = smem_u32(qsm);
    Ring r(a.bufs);
    int i = 0, seg_no = 0;
    Segment g{};
    while (!abort && walk.next_real(a, g)) {
      if (!warp_wait(&q_full, static_cast<uint32_t>(seg_no) & 1u, abort)) break;
      ++seg_no;
      for (int t = g.t0; t < g.t1; ++t, ++i) {
        const uint32_t d = tmem + kDecScol + static_cast<uint32_t>(i & 1) * 64u;
        // tile i - 2's scores have been read once its weights are out
        if (i >= 2 && !warp_wait(&p_full[i & 1], static_cast<uint32_t>((i >> 1) + 1) & 1u, abort)) break;
        const uint32_t sb = ring_a + static_cast<uint32_t>(r.slot * tile_bytes);
        for (int x = 0, c0 = 0; x < groups; ++x) {
          const int c1 = x + 1 == groups ? chunks : (groups == nk ? 2 * x + 2 : 2 * nk - 2);
          if (!warp_wait(&full[x][r.slot], r.turn, abort)) break;
          tc_fence_after();
          if (elect_one()) {
            uint64_t ad = sdesc_sw128(q_a + static_cast<uint32_t>(c0 * kQChunk));
            uint64_t bd = sdesc_sw128(sb + static_cast<uint32_t>(c0 * kChunkBytes));
            for (int c = c0; c < c1; ++c, ad += kQChunk >> 4, bd += kChunkBytes >> 4) {
#pragma unroll
              for (int m = 0; m < 4; ++m) mma_bf16(d, ad + 2 * m, bd + 2 * m, idesc, (c | m) != 0);
            }
            if (x + 1 == groups) {
              mma_commit(&s_full[i & 1]);
              if (t + 1 == g.t1) mma_commit(&q_empty);
            }
          }
          __syncwarp();
          c0 = c1;
        }
        if (abort) break;
        r.step();
      }
    }
    drain_mmas(&drain[0], abort);
  } else if (warp == 2) {
    // ---- output products O^T += C^T P^T
    constexpr uint32_t idesc = idesc_bf16(128, NB) | kIdescAMn;
    const uint32_t ring_a = smem_u32(ring);
    const uint64_t pd = sdesc_sw128(smem_u32(psm));
    Ring r(a.bufs);
    int i = 0, seg_no = 0;
    Segment g{};
    while (!abort && walk.next_real(a, g)) {
      // the accumulator: the stretch before has been read out
      if (seg_no > 0 && !warp_wait(&o_empty, static_cast<uint32_t>(seg_no - 1) & 1u, abort)) break;
      ++seg_no;
      for (int t = g.t0; t < g.t1; ++t, ++i) {
        const int valid = min(kTileTok, g.len - t * kTileTok);
        const int ks = (valid + 15) >> 4;    // 16-position steps that hold anything
        // (the weights come from scores of this very tile: it has landed)
        if (!warp_wait(&p_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, abort)) break;
        if ((valid & 15) != 0) {
          // rows of the last step past the sequence may hold anything
          // (0 x NaN): their weights are 0 and they are made 0 too
          for (int c = 0; c < 2 * nk; ++c)
            zero_rows(ring + r.slot * tile_bytes + c * kChunkBytes, valid, ks * 16, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (elect_one()) {
          uint64_t ad = sdesc_mn_sw128(ring_a + static_cast<uint32_t>(r.slot * tile_bytes), kChunkBytes);
          for (int k = 0; k < nk; ++k, ad += (2 * kChunkBytes) >> 4) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (m < ks)
                mma_bf16(tmem + static_cast<uint32_t>(k) * 64u, ad + m * 128, pd + m * 2, idesc, t != g.t0 || m != 0);
            if (groups == nk || k + 2 >= nk) mma_commit(&empty[k + groups - nk][r.slot]);
          }
          mma_commit(&pv_done);
          if (t + 1 == g.t1) mma_commit(&o_full[(seg_no - 1) & 1]);
        }
        __syncwarp();
        r.step();
      }
    }
    drain_mmas(&drain[1], abort);
  } else if (warp >= 4) {
   const Walk walk0 = walk;
   if (warp < 12) {
    // ---- softmax.  These threads meet at named barriers, so they walk every
    // tile even after a wait has given up.  A 64-row MMA leaves row 16 w + x in
    // lane 32 w + x (x < 16); read 16 lanes at a time, a thread has two rows, of
    // which the four threads of a quad hold eight columns each.  (A row to a
    // thread left half the lanes idle: 1200 cycles a tile.)
    const int w = warp & 3, half = (warp - 4) >> 2, tid = threadIdx.x - 128;
    const int quad = lane & 3, row[2] = {16 * w + (lane >> 2), 16 * w + (lane >> 2) + 8};
    const bool mine = 16 * w < NB;           // (NB is 16, 32 or 64)
    const uint32_t tl = tmem + (static_cast<uint32_t>(w * 32) << 16);
    const int kb0 = half == 0 ? 0 : (nk + 1) >> 1, kb1 = half == 0 ? (nk + 1) >> 1 : nk;   // this half's latent blocks
    int i = 0, seg_no = 0;
    Segment g{};
    while (walk.next(a, g)) {
      int tok[2], head[2], see[2];
      bool on[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        on[e] = group_row(a, g.rt, row[e], tok[e], head[e]) && mine;
        see[e] = on[e] ? max(0, min(g.len, g.len - a.q_len + 1 + tok[e])) : 0;
      }
      const bool whole = g.t0 == 0 && g.t1 == g.nt;
      if (g.len > 0) {
        float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};    // l: of the thread's own columns
        for (int t = g.t0; t < g.t1; ++t, ++i) {
          const bool first = t == g.t0;
          uint32_t x[16];
          mbar_wait(&s_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, abort);
          __syncwarp();
          tc_fence_after();
          tmem_ld_16x32(tl + kDecScol + static_cast<uint32_t>((i & 1) * 64 + half * 32), x);
          tmem_wait_ld_of(x);
          if (a.flip) {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] ^= 0x80000000u;
          }
          const int j0 = t * kTileTok + half * 32;
          if (j0 + 32 > min(see[0], see[1])) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (j0 + (j >> 2) * 8 + quad * 2 + (j & 1) >= see[(j >> 1) & 1]) x[j] = 0xFF800000u;
          }
          float mx[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a0 = fmaxf(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
            const float a1 = fmaxf(__uint_as_float(x[4 + 2 * e]), __uint_as_float(x[5 + 2 * e]));
            mx[e] = fmaxf(max3(a0, __uint_as_float(x[8 + 2 * e]), __uint_as_float(x[9 + 2 * e])),
                          max3(a1, __uint_as_float(x[12 + 2 * e]), __uint_as_float(x[13 + 2 * e])));
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], o));
#pragma unroll
          for (int e = 0; e < 2; ++e) mx[e] *= a.c;
          if (first || named_sync_or(1, 256, mine && fmaxf(mx[0] - m[0], mx[1] - m[1]) > kMaxSlack)) {
            if (mine && quad == 0) {
              xch[half][row[0]] = mx[0];
              xch[half][row[1]] = mx[1];
            }
            named_sync(1, 256);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float mn = fmaxf(mx[e], xch[half ^ 1][row[e]]);
                if (!first) mn = fmaxf(mn, m[e]);
                if (mn == -INFINITY) mn = 0.f;         // a row that sees nothing here sees nothing later
                const float f = exp2_fast(m[e] - mn);
                if (half == 0 && quad == 0) fac[row[e]] = f;
                l[e] = first ? 0.f : l[e] * f;         // (f may be infinite at first: m is no maximum yet)
                m[e] = mn;
              }
            }
            named_sync(1, 256);
            if (!first) {
              mbar_wait(&pv_done, static_cast<uint32_t>(i - 1) & 1u, abort);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int k = kb0; k < kb1; ++k) {
#pragma unroll 1
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
            }
          }
          // weights (rounded to bf16 for the MMA) and their fp32 sum (unrounded)
          uint32_t p[8];                     // [columns 8 j ..][row]
          const uint64_t c2 = pair2f(a.c, a.c);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int e = j & 1;
            float x0, x1;
            split2(fma2(pair2(x[2 * j], x[2 * j + 1]), c2, pair2f(-m[e], -m[e])), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            sum[e] = add2(sum[e], pair2f(x0, x1));
            p[j] = pack_bf16x2(x0, x1);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float s0, s1;
            split2(sum[e], s0, s1);
            l[e] += s0 + s1;
          }
          if (i > 0) {
            // the product before has read its weights
            mbar_wait(&pv_done, static_cast<uint32_t>(i - 1) & 1u, abort);
            __syncwarp();
          }
          if (mine) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int r = row[j & 1];
              *reinterpret_cast<uint32_t*>(psm + r * 128 + (((half * 4 + (j >> 1)) ^ (r & 7)) << 4) + quad * 4) = p[j];
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&p_full[i & 1]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
          l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
        }
        // the halves' sums meet in fac: the next stretch writes xch before any
        // barrier, but fac only behind one
        named_sync(1, 256);                  // fac is free
        if (half == 1 && mine && quad == 0) {
          fac[row[0]] = l[0];
          fac[row[1]] = l[1];
        }
        named_sync(1, 256);
        if (half == 0 && mine && quad == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = row[e];
            const float sum = l[e] + fac[r];
            fin[seg_no % 3][r] = sum == 0.f ? 0.f : 1.0f / sum;
            if (whole) {
              if (a.lse != nullptr && on[e])
                a.lse[(static_cast<int64_t>(g.s) * a.q_len + tok[e]) * a.H + head[e]] =
                    sum == 0.f ? -INFINITY : (m[e] + log2_fast(sum)) * kLn2;
            } else if (on[e]) {
              float* part = part_of(a, NB, blockIdx.x, g.t0 == 0) + static_cast<int64_t>(NB) * a.L;
              part[r] = sum == 0.f ? -INFINITY : m[e];
              part[NB + r] = sum;
            }
          }
        }
        mbar_arrive(&fin_full[seg_no & 1]);
        ++seg_no;
      } else {
        // an empty sequence: its rows are zero, their log-sum -inf
        for (int j = 0; j < NB; ++j) {
          int tj, hj;
          if (!group_row(a, g.rt, j, tj, hj)) continue;
          __nv_bfloat16* dst = a.out + (static_cast<int64_t>(g.s) * a.q_len + tj) * a.o_tok + hj * a.o_head;
          for (int d = tid * 8; d < a.L; d += 256 * 8) *reinterpret_cast<uint4*>(dst + d) = make_uint4(0, 0, 0, 0);
        }
        if (half == 0 && quad == 0 && a.lse != nullptr) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (on[e]) a.lse[(static_cast<int64_t>(g.s) * a.q_len + tok[e]) * a.H + head[e]] = -INFINITY;
        }
      }
    }
   }
    // ---- finished accumulators: latent value 128 k + 32 w + lane of all rows.
    // Warps 12..15 write out all but the block's last, which the softmax warps
    // have nothing else to do beside: there each four take every third block k.
    const int w = warp & 3, four = (warp >> 2) - 1;     // 0, 1: softmax, 2: warps 12..15
    const uint32_t tl = tmem + (static_cast<uint32_t>(w * 32) << 16);
    constexpr int kCols = NB < 32 ? NB : 32;
    const bool odd = (lane & 1) != 0;
    int seg_no = 0;
    Segment g{};
    walk = walk0;
    for (; walk.next_real(a, g); ++seg_no) {
      const bool last = walk.left <= 0;
      if (warp < 12 && !last) continue;
      mbar_wait(&fin_full[seg_no & 1], static_cast<uint32_t>(seg_no >> 1) & 1u, abort);
      mbar_wait(&o_full[seg_no & 1], static_cast<uint32_t>(seg_no >> 1) & 1u, abort);
      const float* inv = fin[seg_no % 3];
      __syncwarp();
      tc_fence_after();
      const bool whole = g.t0 == 0 && g.t1 == g.nt;
      float* part = whole ? nullptr : part_of(a, NB, blockIdx.x, g.t0 == 0);
      const int tok0 = (g.rt / a.head_blocks) * a.TPT, h0 = (g.rt % a.head_blocks) * a.HB;
      __nv_bfloat16* out0 = a.out + (static_cast<int64_t>(g.s) * a.q_len + tok0) * a.o_tok + h0 * a.o_head;
#pragma unroll 1
      for (int k = last ? four : 0; k < nk; k += last ? 3 : 1) {
        const int d = k * 128 + w * 32 + lane;
        // the next row's place in the group and in the output
        int hi = 0, ti = 0;
        __nv_bfloat16* dst = out0 + (d & ~1);
#pragma unroll 1
        for (int j0 = 0; j0 < NB; j0 += kCols) {
          uint32_t o[kCols];
          tmem_ld_cols<kCols>(tl + k * 64 + j0, o);
          tmem_wait_ld_of(o);
          if (!last && k + 1 == nk && j0 + kCols == NB) {
            tc_fence_before();
            mbar_arrive(&o_empty);
          }
          if (whole) {
            // two rows per pass: lane pairs swap a value so that each lane
            // stores two neighbouring ones, of the even or of the odd row
#pragma unroll
            for (int j = 0; j < kCols; j += 2) {
              const float f0 = inv[j0 + j], f1 = inv[j0 + j + 1];
              const float x0 = f0 == 0.f ? 0.f : __uint_as_float(o[j]) * f0;
              const float x1 = f1 == 0.f ? 0.f : __uint_as_float(o[j + 1]) * f1;
              const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? x0 : x1, 1);
              const uint32_t v = odd ? pack_bf16x2(got, x1) : pack_bf16x2(x0, got);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const bool on = ti < a.TB && tok0 + ti < a.q_len && h0 + hi < a.H;
                st_global_if(dst, v, on && odd == (x == 1));
                dst += a.o_head;
                if (++hi == a.HB) {
                  hi = 0;
                  ++ti;
                  dst += a.o_tok - a.HB * a.o_head;
                }
              }
            }
          } else {
            float* dst = part + static_cast<int64_t>(j0) * a.L + d;
            const int n = a.HB * a.TB - j0;  // rows that pad the group are not read again
#pragma unroll
            for (int j = 0; j < kCols; ++j, dst += a.L)
              if (j < n) *dst = __uint_as_float(o[j]);
          }
        }
      }
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
// of a row group that was cut between blocks (the order of the sums depends
// on the shape alone).  A unit of work is V x 128 latent values of a row
// (lane = V times four values): `warps` warps share its parts out and meet in
// shared memory; a block of 8 warps takes 8 / warps units.  Bound by latency
// (the lengths, then the parts, from L2), so a call should fit the card at
// once: whole rows to a warp where there are many, and eight loads in flight.
// The 20 MB of parts of 152 blocks take 2 to 5 us; four rows of a value to a
// store and a lane (512 contiguous bytes) took as long.
constexpr int kCombWarps = 8;

template <int V>
__global__ void __launch_bounds__(kCombWarps * 32, 3) mla_combine_kernel(const DecodeArgs a, int grid, int NB, int warps) {
  __shared__ int64_t sums[2][kCombWarps];
  __shared__ __align__(16) float4 acc_s[kCombWarps][V][32];
  __shared__ float2 ml_s[kCombWarps];
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int group = blockIdx.x, s = group / a.RT, rt = group % a.RT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // units before this sequence and of all (seq_lens: complete before the
  // kernel ahead let this one start)
  int64_t before = 0, total = 0;
  int over = a.over;
#pragma unroll 1
  for (;;) {                                 // (as the blocks ahead: once or twice)
    before = total = 0;
    for (int i = threadIdx.x; i < a.S; i += kCombWarps * 32) {
      const int64_t u = group_units(over, seq_len(a, i));
      total += u;
      if (i < s) before += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
      total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
    if (lane == 0) {
      sums[0][warp] = before;
      sums[1][warp] = total;
    }
    __syncthreads();
    before = total = 0;
    for (int w = 0; w < kCombWarps; ++w) {
      before += sums[0][w];
      total += sums[1][w];
    }
    if (over == kLongOver || !long_stretches(a, total, grid)) break;
    over = kLongOver;
    __syncthreads();                         // the sums have been read
  }
  const int units = group_units(over, seq_len(a, s));
  const int64_t u0 = before * a.RT + static_cast<int64_t>(rt) * units;
  int n;
  const Cut cut(total * a.RT, grid, n);
  const int c0 = cut.owner(u0 + min(units - 1, over)), c1 = cut.owner(u0 + units - 1);   // of the first and the last tile
  griddep_wait();                            // (every block: the grid must not end before the one ahead)
  if (c0 == c1) return;                      // not cut: written by its block
  const int nk = a.L / (128 * V), per = kCombWarps / warps;   // units a block takes at a time
  const int team = warp / warps, member = warp % warps;
  const int unit = blockIdx.y * per + team;
  const int j = unit / nk, k = unit % nk;    // row and its V x 128 values
  int tok = 0, head = 0;
  const bool on = j < NB && group_row(a, rt, j, tok, head);
  float M = -INFINITY, l = 0.f;
  float4 v[V];
#pragma unroll
  for (int x = 0; x < V; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
    const int64_t pf = part_floats(NB, a.L);
    // the part of block c: the one it begins the group with, or goes on with
    const float* base = a.parts + static_cast<int64_t>(j) * a.L + k * V * 128 + lane * 4;
    const float* stat = a.parts + static_cast<int64_t>(NB) * a.L + j;
    constexpr int kBatch = V >= 4 ? 2 : (V == 2 ? 4 : 8);
    for (int c = c0 + member; c <= c1; c += kBatch * warps) {
      float4 o[kBatch][V];
      float m[kBatch], ls[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int ci = c + i * warps;
        const int64_t at = (static_cast<int64_t>(ci) * 2 + (ci == c0 ? 1 : 0)) * pf;
        const bool in = ci <= c1;
        m[i] = in ? stat[at] : -INFINITY;
        ls[i] = in ? stat[at + NB] : 0.f;
#pragma unroll
        for (int x = 0; x < V; ++x)
          o[i][x] = in ? *reinterpret_cast<const float4*>(base + at + x * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float Mn = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) Mn = fmaxf(Mn, m[i]);
      const float ref = Mn == -INFINITY ? 0.f : Mn, f = exp2_fast(M - ref);
      l *= f;
#pragma unroll
      for (int x = 0; x < V; ++x) v[x] = make_float4(v[x].x * f, v[x].y * f, v[x].z * f, v[x].w * f);
      M = Mn;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (ls[i] == 0.f) continue;          // no part, or one whose positions this row does not see
        const float wgt = exp2_fast(m[i] - ref);
        l += wgt * ls[i];
#pragma unroll
        for (int x = 0; x < V; ++x) {
          v[x].x += wgt * o[i][x].x;
          v[x].y += wgt * o[i][x].y;
          v[x].z += wgt * o[i][x].z;
          v[x].w += wgt * o[i][x].w;
        }
      }
    }
  }
  if (warps > 1) {
#pragma unroll
    for (int x = 0; x < V; ++x) acc_s[warp][x][lane] = v[x];
    if (lane == 0) ml_s[warp] = make_float2(M, l);
    __syncthreads();
    if (member != 0) return;
    float Mt = M;
    for (int w = 1; w < warps; ++w) Mt = fmaxf(Mt, ml_s[warp + w].x);
    const float ref = Mt == -INFINITY ? 0.f : Mt, f = exp2_fast(M - ref);
    l *= f;
#pragma unroll
    for (int x = 0; x < V; ++x) v[x] = make_float4(v[x].x * f, v[x].y * f, v[x].z * f, v[x].w * f);
    for (int w = 1; w < warps; ++w) {
      const float2 ml = ml_s[warp + w];
      if (ml.y == 0.f) continue;
      const float wgt = exp2_fast(ml.x - ref);
      l += wgt * ml.y;
#pragma unroll
      for (int x = 0; x < V; ++x) {
        const float4 o = acc_s[warp + w][x][lane];
        v[x].x += wgt * o.x;
        v[x].y += wgt * o.y;
        v[x].z += wgt * o.z;
        v[x].w += wgt * o.w;
      }
    }
    M = Mt;
  }
  if (!on) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int64_t at = static_cast<int64_t>(s) * a.q_len + tok;
  __nv_bfloat16* dst = a.out + at * a.o_tok + head * a.o_head + k * V * 128 + lane * 4;
#pragma unroll
  for (int x = 0; x < V; ++x)
    *reinterpret_cast<uint2*>(dst + x * 128) =
        l == 0.f ? make_uint2(0u, 0u)
                 : make_uint2(pack_bf16x2(v[x].x * inv, v[x].y * inv), pack_bf16x2(v[x].z * inv, v[x].w * inv));
  if (k == 0 && lane == 0 && a.lse != nullptr) a.lse[at * a.H + head] = l == 0.f ? -INFINITY : (M + log2_fast(l)) * kLn2;
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

// Going over to another row group is counted as a tile where 64 rows have to be
// written out for it, and as three where the blocks have 24 units and more, so
// that many go over in the middle of their work.  Counted as 0, 1, 3 (ragged
// lengths): 10 tiles a block 35.2, 33.6, 34.9 us; 15 48.7, 47.0, 47.4; 28 86.2, 84.7,
// 79.4.  For groups of fewer rows it is nothing (32 rows, 65 sequences of up to
// 426: 16.7, 18.2, 19.2).
static int decode_over(int NB) { return NB == 64 ? 1 : 0; }

// Blocks of a call, and what going over counts as (nothing where each tile has a
// block of its own).
static int decode_grid(int S, const RowSplit& r, int64_t capacity, int sm_count, int* over) {
  const int64_t most = static_cast<int64_t>(S) * r.RT * ceil_div(capacity > 0 ? capacity : 1, kTileTok);
  const int lim = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  *over = most > lim ? decode_over(r.NB) : 0;
  return static_cast<int>(most < lim ? most : lim);
}

size_t mla_decode_workspace(int S, int q_len, int H, int L, int64_t max_len, int sm_count) {
  if (max_len <= kTileTok) return 0;         // one tile a sequence: nothing is cut
  const RowSplit r = split_rows(q_len, H);
  int over;
  return static_cast<size_t>(decode_grid(S, r, max_len, sm_count, &over)) * 2 * part_floats(r.NB, L) * sizeof(float);
}

bool mla_decode_fits(int S, int q_len, int H) {
  const int64_t tokens = static_cast<int64_t>(S) * q_len;
  return tokens * ceil_div(H, 64) < 0x7FFFFFFF;
}

static std::atomic<bool> g_decode_attr[3][64];

template <int NB>
static cudaError_t launch_decode_nb(const CUtensorMap (&maps)[4], DecodeArgs a, int grid, const DeviceInfo& dev,
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
  // tiles that fit beside the queries and the weights
  const int chunks = a.L / 64 + 1;
  const int fixed = (chunks + 1) * NB * 128 + 1024, tile = chunks * kChunkBytes;
  a.bufs = (kDecSmem - kDecStatic - fixed) / tile;
  if (a.bufs > kDecMaxBufs) a.bufs = kDecMaxBufs;
  return mla_launch(kern, dim3(static_cast<unsigned>(grid)), kDecThreads, fixed + a.bufs * tile, s, maps[0],
                    maps[1], maps[2], maps[3], a);
}

cudaError_t launch_mla_decode(const MlaDecodeProblem& p, const DeviceInfo& dev, cudaStream_t s) {
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
  cudaError_t e = bind_device_context();
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
  a.flip = p.scale < 0.f;
  a.c = positive_scale(a.flip ? -p.scale : p.scale);

  // Chunks to a copy: all of the queries, or of a tile's group, where their rows
  // lie as the products want them (a full group of rows, pages of whole tiles).
  // A copy of one chunk takes as long to issue as one of all of them.
  const int values = 2 * (p.L / 128);
  a.q_box = r.HB * r.TB == r.NB ? values : 1;
  a.wide = a.box_rows == kTileTok ? 1 : 0;
  CUtensorMap maps[4];
  const int64_t T = static_cast<int64_t>(p.S) * p.q_len;
  const int64_t row = p.L + kMlaRope;
  if ((e = mla_tensor_map_chunks(&maps[0], p.q_lat.p, p.L, p.H, T, p.q_lat.head, p.q_lat.tok, a.q_box, r.HB, r.TB)) !=
      cudaSuccess)
    return e;
  if ((e = mla_tensor_map_chunks(&maps[1], p.q_rope.p, kMlaRope, p.H, T, p.q_rope.head, p.q_rope.tok, 1, r.HB, r.TB)) !=
      cudaSuccess)
    return e;
  for (int x = 0; x < 2; ++x) {
    const int box = !a.wide ? 1 : (x == 0 ? 2 : 3);
    if ((e = mla_tensor_map_chunks(&maps[2 + x], p.cache.p, row, p.cache.page_size, p.cache.num_pages, row,
                                   p.cache.page_stride, box, a.box_rows, 1)) != cudaSuccess)
      return e;
  }
  const int grid = decode_grid(p.S, r, a.capacity, dev.sm_count, &a.over);
  e = r.NB == 16 ? launch_decode_nb<16>(maps, a, grid, dev, s)
                 : (r.NB == 32 ? launch_decode_nb<32>(maps, a, grid, dev, s)
                               : launch_decode_nb<64>(maps, a, grid, dev, s));
  if (e != cudaSuccess || a.capacity <= kTileTok) return e;
  // a whole row to a warp where there are rows for a few warps per SM; warps
  // that share a row's parts out: for the parts of a group that the grid cuts
  // on average, four to a warp
  const int64_t groups = static_cast<int64_t>(p.S) * r.RT;
  const int nk = p.L / 128;
  const int V = groups * r.NB <= dev.sm_count || nk == 3 ? 1 : nk;
  int warps = 1;
  while (warps < kCombWarps && static_cast<int64_t>(warps) * 4 * groups < grid + groups) warps *= 2;
  // ... but no second round of blocks (three fit an SM), which costs more than
  // a round of loads
  const int units = r.HB * r.TB * (nk / V);
  while (warps > 1 && groups * ceil_div(static_cast<int64_t>(units) * warps, kCombWarps) > 3 * dev.sm_count) warps /= 2;
  const int per = kCombWarps / warps;
  auto join = V == 4 ? mla_combine_kernel<4> : (V == 2 ? mla_combine_kernel<2> : mla_combine_kernel<1>);
  return mla_launch(join, dim3(static_cast<unsigned>(groups), static_cast<unsigned>(ceil_div(units, per))),
                    kCombWarps * 32, 0, s, a, grid, r.NB, warps);
}

uint32_t mla_decode_read_clear_error() { return read_clear_word(g_mla_decode_error); }

}  // namespace mx
