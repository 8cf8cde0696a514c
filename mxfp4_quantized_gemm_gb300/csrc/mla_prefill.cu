// mxfp4_mla_prefill: expanded latent attention of ragged prompts.  Per head
//   s[i][j] = scale * (q_nope_i . k_nope_j + q_rope_i . k_rope_j)
//   out_i   = sum_j softmax_j(s_i)[j] v_j
// with k_rope shared by all heads, j < k_len, and for causal calls
// j <= i + k_len - q_len (the newest query sees every key).
//
// Bound by the tensor cores: 2 (dn + R + dv) flop a (query, key, head).  A
// block takes 128 queries of one head and walks the keys in tiles of 128 with
// tcgen05 MMAs: S = Q K^T into one of two TMEM score tiles (128 columns each),
// then O += P V with the weights P as the A operand straight from TMEM (bf16,
// written over the score tile they come from), O (128 x dv <= 256 columns)
// staying in TMEM for the whole walk.  The two halves of q and k come through
// tensor maps of their own, so that nothing is concatenated in memory, and
// the value tile is read in place from the expanding projection's output
// [token][head][dn + dv] (its rows are the MMA's K: N-contiguous operand).
//
// Long prompts run in pairs of blocks (kPair: a 2-CTA cluster, cta_group::2
// MMAs of 256 queries).  One block alone is held by shared memory: at dn + R =
// dv = 256 a tile's MMAs take 2144 cycles, while its operands (1536 cycles at
// 128 bytes a cycle) and the copies that bring them (1024) share the same
// memory, and its MMAs ran at 124 (scores) and 175 cycles (output) instead of
// 71 and 126.  In a pair each block holds and reads half of the keys (rows) and
// half of the values (columns), and its copies halve too.
//
// Roles: warp 0 copies keys and warp 3 values, each through a ring of 32 KB
// slots of its own; warp 1 issues every product (in rank 0 of a pair, whose
// barriers count the copies of both blocks; warp 2 of rank 1 clears the rest of
// value tiles that end a sequence, and only then lets rank 0 have them); warps 4..7 and 8..11 hold the softmax, thread = (query, half of the tile's
// keys).  Each query's running maximum is raised only when a score passes it
// by 2^8, decided per 32 queries by a barrier with an OR over the two warps
// that hold them.
//
// Order of the products: S(0), S(1), O(0), S(2), O(1), ...  The next scores go
// first, so that their softmax runs beside the product of the tile before,
// and S(t + 2) may overwrite the weights of tile t as soon as O(t), issued
// before it by the same thread, has read them.
//
// Slot size: an issuing warp spends about 50 cycles an MMA and 155 a slot
// (wait, commit); a copying warp spends 430 cycles a slot (wait, arrival,
// copy) and 16 for each further copy.  With one or two slots a tile both stay
// below the MMAs' time; with four (16 KB) they did not.
//
// The grid is one block (or pair) per SM (pair of SMs) that walks query tiles:
// the next tile's copies and first scores run while the softmax warps write the
// last one out.  (A block per tile spent 14000 cycles on each, the time of six
// key tiles, before its first and after its last product.)  How they are dealt
// out: QueryTiles.
//
// Measured (dn + R = dv = 256, 64 heads; from card to card): 8192 tokens 1310 to
// 1335 us, 1.65 to 1.68 PFLOP/s, the rate that the power limit leaves a long run
// of matrix products; six ragged prompts of 156 to 781 tokens on up to 1000
// others 147 to 153 us: of a query tile's 10 us, 7 key tiles at 1.16 us, then 1.7
// until the last product is done and 1.7 to write it out, during which the next
// tile's scores are formed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>

#include "mla.h"
#include "mla_common.cuh"

namespace mx {

static __device__ uint32_t g_mla_prefill_error;

constexpr int kPreThreads = 384;
constexpr int kPreTile = 128;                 // queries of a block, and keys per tile
constexpr int kPreChunk = 16384;              // 128 rows x 64 values
constexpr int kSlotBytes = 2 * kPreChunk;
constexpr int kPreMaxSlots = 4;               // slots of a ring
constexpr int kPreSmem = 227 * 1024;
constexpr int kPreStatic = 2048;              // most of it that the static part takes
constexpr int kPreScol = 256;                 // first TMEM column of the score tiles

// A slot holds, of a block alone, 128 values of 128 keys or all values of 64
// keys (two value slots a tile); of a block of a pair, all values of its 64
// keys or its half of the values of 128 keys.
template <bool kPair>
struct PreShape {
  static constexpr int kKeyRows = kPair ? 64 : 128;     // keys in a key slot
  static constexpr int kKeyChunks = kPair ? 4 : 2;      // 64-value chunks in a key slot
  static constexpr int kKeyChunkBytes = kKeyRows * 128;
  static constexpr int kValRows = kPair ? 128 : 64;     // keys in a value slot
  static constexpr int kValBlockBytes = kValRows * 128; // 64 values of them
  static constexpr int kQueries = kPair ? 256 : 128;
  static constexpr int kBlocks = kPair ? 2 : 1;
};

struct PrefillArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  __nv_bfloat16* out;
  float* lse;
  int64_t o_tok, o_head;
  int S, H, Tq, Tk, dn, dv;
  int nq;               // 64-value chunks of q and k (the last is the rotated one)
  int dvn;              // dv rounded up to the MMA's N
  int kslots, vslots;   // ring slots of the keys and of the values
  float c;              // |scale| * log2(e)
  bool flip;            // scale < 0: the scores change sign first
  bool causal;
};

// Query rows and keys of sequence s, kept inside the tensors.
struct Extent {
  int q0, qn, k0, kn;
};
// (Offsets out of range are cut here, and reported by check_offsets.)
__device__ __forceinline__ int clamp_to(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }
__device__ __forceinline__ Extent extent(const PrefillArgs& a, int s) {
  Extent e;
  e.q0 = clamp_to(__ldg(a.cu_q + s), a.Tq);
  e.qn = max(0, clamp_to(__ldg(a.cu_q + s + 1), a.Tq) - e.q0);
  e.k0 = clamp_to(__ldg(a.cu_k + s), a.Tk);
  e.kn = max(0, clamp_to(__ldg(a.cu_k + s + 1), a.Tk) - e.k0);
  return e;
}

// By one warp of the grid: both offsets ascending inside the tensors, and the
// queries' from 0 to the last row (the rows that they leave out are not written).
__device__ __forceinline__ void check_offsets(const PrefillArgs& a, int lane) {
  bool bad = false;
  for (int s = lane; s <= a.S; s += 32) {
    const int q = __ldg(a.cu_q + s), k = __ldg(a.cu_k + s);
    bad |= s == 0 ? q != 0 || k < 0 : q < __ldg(a.cu_q + s - 1) || k < __ldg(a.cu_k + s - 1);
    bad |= s == a.S && (q != a.Tq || k > a.Tk);
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(&g_mla_prefill_error, kErrIndex);
}

// A query tile of a block or pair, and what its keys amount to.
struct QueryTile {
  Extent ex;
  int h;
  int qi0;     // this block's first query, within its sequence
  int rows;    // this block's queries (0 in rank 1 of a pair whose sequence ends in rank 0)
  int see0;    // keys visible to this block's first query ...
  int see1;    // ... and to the last of the block or pair
  int tiles;   // key tiles
};

// The query tiles of a block or pair.  A sequence whose queries are no whole
// number of tiles has the short one in front, where causal queries see the
// fewest keys.
//
// Up to 32 sequences (a lane each) and 64 rounds: the tiles are numbered by
// their keys, the most first, head by head within a number, and dealt out to
// and fro; that leaves the blocks' loads 1..5% apart where dealing them out in
// sequence order left 5..20%.  A block takes what it was dealt in the order of
// the heads, so that all blocks are at about the same heads at a time and find
// their keys and values in L2.  Its list is made by all its warps together.
// Otherwise: in sequence order, last tile first, head by head, found by each
// warp for itself (more rounds even out by themselves).
struct ListedTile {
  uint32_t tile, seq_head;                 // seq_head: the sequence in the upper 5 bits
};
constexpr int kPreListed = 64;

template <bool kPair>
struct QueryTiles {
  static constexpr int kQ = PreShape<kPair>::kQueries;
  Extent own;                              // up to 32 sequences: the lane's
  int s0, s1, first, incl, total, round, rank;
  int listed;                              // tiles of the list, or -1
  const ListedTile* list;
  // of the lane's sequence: the first of its tiles with `keys` key tiles or more
  __device__ __forceinline__ int with_keys(const PrefillArgs& a, int keys) const {
    const int n = incl - first;
    if (keys <= 0) return 0;
    const int64_t need = static_cast<int64_t>(keys - 1) * kPreTile + 1;
    if (own.kn < need) return n;
    if (!a.causal) return 0;
    // tile t ends before query (t + 1) kQ - short, which sees `back` keys more
    const int64_t end = need - (own.kn - own.qn) + (n * static_cast<int64_t>(kQ) - own.qn);
    const int64_t t = ((end + kQ - 1) >> (kPair ? 8 : 7)) - 1;
    return t < 0 ? 0 : (t > n ? n : static_cast<int>(t));
  }
  // what a round deals to this block or pair
  __device__ __forceinline__ int64_t dealt(int r) const {
    const int n = static_cast<int>(gridDim.x) / PreShape<kPair>::kBlocks;
    const int c = static_cast<int>(blockIdx.x) / PreShape<kPair>::kBlocks;
    return static_cast<int64_t>(r) * n + ((r & 1) ? n - 1 - c : c);
  }
  // (all threads of the block)
  __device__ __forceinline__ QueryTiles(const PrefillArgs& a, int rank_, ListedTile* room) : round(0), rank(rank_), list(room) {
    const int lane = threadIdx.x & 31, per = (a.S + 31) >> 5;
    s0 = min(a.S, lane * per);
    s1 = min(a.S, s0 + per);
    int mine = 0;
    own = lane < a.S ? extent(a, lane) : Extent{0, 0, 0, 0};
    if (a.S <= 32) {
      mine = (own.qn + kQ - 1) / kQ;
    } else {
#pragma unroll 4
      for (int s = s0; s < s1; ++s) mine += (extent(a, s).qn + kQ - 1) / kQ;
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    first = incl - mine;
    total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    const int64_t n = gridDim.x / PreShape<kPair>::kBlocks, all = static_cast<int64_t>(total) * a.H;
    listed = -1;
    if (a.S > 32 || all > kPreListed * n) return;
    const int rounds = (static_cast<int>(all) + static_cast<int>(n) - 1) / static_cast<int>(n);
    listed = rounds - (rounds > 0 && dealt(rounds - 1) >= all ? 1 : 0);
    const int most = static_cast<int>(
        __reduce_max_sync(0xFFFFFFFFu, (static_cast<uint32_t>(own.kn) + kPreTile - 1) / kPreTile));
    auto head = [&](int r) { return r < listed ? static_cast<int>(dealt(r)) % a.H : 0x7FFFFFFF; };
    const int h0 = head(lane), h1 = head(lane + 32);
    for (int r = threadIdx.x >> 5; r < listed; r += kPreThreads / 32) {
      const int at = static_cast<int>(dealt(r)), number = at / a.H, h = at - number * a.H;
      const int place = __popc(__ballot_sync(0xFFFFFFFFu, h0 < h || (h0 == h && lane < r))) +
                        __popc(__ballot_sync(0xFFFFFFFFu, h1 < h || (h1 == h && lane + 32 < r)));
      // its key tiles: the most that more than `number` tiles have
      int lo = 0, hi = most;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__reduce_add_sync(0xFFFFFFFFu, mine - with_keys(a, mid)) > number)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int from_tile = with_keys(a, lo), to_tile = with_keys(a, lo + 1);
      const int skip = number - __reduce_add_sync(0xFFFFFFFFu, mine - to_tile);
      int upto = to_tile - from_tile;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
      }
      if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, upto > skip)) - 1)
        room[place] = ListedTile{static_cast<uint32_t>(to_tile - (upto - skip)),
                                 static_cast<uint32_t>(lane) << 27 | static_cast<uint32_t>(h)};
    }
    __syncthreads();
  }
  __device__ __forceinline__ bool next(const PrefillArgs& a, QueryTile& x) {
    int tile;
    if (listed >= 0) {
      if (round >= listed) return false;
      const ListedTile at = list[round++];
      const int from = static_cast<int>(at.seq_head >> 27);
      tile = static_cast<int>(at.tile);
      x.h = static_cast<int>(at.seq_head & 0x07FFFFFFu);
      x.ex.q0 = __shfl_sync(0xFFFFFFFFu, own.q0, from);
      x.ex.qn = __shfl_sync(0xFFFFFFFFu, own.qn, from);
      x.ex.k0 = __shfl_sync(0xFFFFFFFFu, own.k0, from);
      x.ex.kn = __shfl_sync(0xFFFFFFFFu, own.kn, from);
    } else {
      const int64_t all = static_cast<int64_t>(total) * a.H, at = dealt(round);
      if (at >= all) return false;                    // (the rounds that follow lie past the end too)
      ++round;
      // (a 64-bit division takes several times a 32-bit one)
      x.h = all <= 0x7FFFFFFF ? static_cast<int>(at) / total : static_cast<int>(at / total);
      const int want = total - 1 - static_cast<int>(at - static_cast<int64_t>(x.h) * total);
      // the lane whose share holds it
      const bool here = want >= first && want < incl;
      int seq = 0;
      tile = want - first;
      if (here)
        for (seq = s0; seq < s1; ++seq) {
          const int m = (extent(a, seq).qn + kQ - 1) / kQ;
          if (tile < m) break;
          tile -= m;
        }
      const int from = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
      tile = __shfl_sync(0xFFFFFFFFu, tile, from);
      x.ex = extent(a, __shfl_sync(0xFFFFFFFFu, seq, from));
    }
    const int end = x.ex.qn - ((x.ex.qn + kQ - 1) / kQ - 1 - tile) * kQ;   // one past its last query
    x.qi0 = max(0, end - kQ) + rank * kPreTile;
    x.rows = clamp_to(end - x.qi0, kPreTile);
    const int back = x.ex.kn - x.ex.qn;
    x.see0 = a.causal ? clamp_to(x.qi0 + 1 + back, x.ex.kn) : x.ex.kn;
    x.see1 = a.causal ? clamp_to(end + back, x.ex.kn) : x.ex.kn;
    x.tiles = (x.see1 + kPreTile - 1) / kPreTile;
    return true;
  }
  // the next tile that sees any key
  __device__ __forceinline__ bool next_real(const PrefillArgs& a, QueryTile& x) {
    while (next(a, x))
      if (x.tiles > 0) return true;
    return false;
  }
};

// Keys of a value slot that no query of the tile sees may hold anything (0 x
// NaN): their weights are 0 and they are made 0 too, by one warp.  `valid`: the
// slot's keys that count.
template <int kRows>
__device__ __forceinline__ void clear_values(uint8_t* slot, int nv, int valid, int lane) {
  if (valid >= kRows) return;
  for (int k = 0; k < nv; ++k) zero_rows(slot + k * kRows * 128, valid, kRows, lane);
  fence_proxy_async_smem();
  __syncwarp();
}

template <bool kPair>
__global__ void __launch_bounds__(kPreThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap qn_map, const __grid_constant__ CUtensorMap qr_map,
                       const __grid_constant__ CUtensorMap kn_map, const __grid_constant__ CUtensorMap kr_map,
                       const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap o_map,
                       const PrefillArgs a) {
  using Shape = PreShape<kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qsm = smem;                                // nq chunks of 128 queries x 64 values
  uint8_t* kring = qsm + a.nq * kPreChunk;
  uint8_t* vring = kring + a.kslots * kSlotBytes;
  uint8_t* osm = vring + a.vslots * kSlotBytes;       // two 64-value blocks of 128 queries, on their way out

  __shared__ __align__(8) uint64_t kfull[kPreMaxSlots], kempty[kPreMaxSlots], vfull[kPreMaxSlots], vempty[kPreMaxSlots];
  __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ float xch[2][kPreTile];
  __shared__ ListedTile list[kPreListed];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  bool abort = false;
  if (threadIdx.x == 0) {
    // rank 0's full barriers also count rank 1: its copies (one arrival, and
    // their bytes), and its weights (one arrival per softmax thread)
    const uint32_t both = kPair && leader ? 2 : 1;
    for (int s = 0; s < kPreMaxSlots; ++s) {
      mbar_init(&kfull[s], both);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], both);
      mbar_init(&vempty[s], 1);
    }
    mbar_init(&q_full, both);
    mbar_init(&q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kPair ? 512 : 256);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane < 5)
    prefetch_tensor_map(lane == 0 ? &qn_map : (lane == 1 ? &qr_map : (lane == 2 ? &kn_map : (lane == 3 ? &kr_map : &v_map))));
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync_all();                      // both blocks' barriers and TMEM exist
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  QueryTiles<kPair> walk(a, static_cast<int>(rank), list);
  QueryTile x;
  // Copies of a pair are counted on rank 0's barriers, where the products that
  // read both blocks' shared memory are issued.  (Barriers of rank 1's own with
  // warps that pass their phases on would hand the copies over by threads that
  // neither wrote nor read them, a hop later.)
  auto expect = [&](uint64_t* bar, int bytes) {
    if (kPair)
      mbar_arrive_expect_tx_cluster(mapa_shared(smem_u32(bar), 0), static_cast<uint32_t>(bytes));
    else
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(bytes));
  };
  auto copy = [&](void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    if (kPair)
      tma_box_3d_pair(dst, map, c0, c1, c2, mapa_shared(smem_u32(bar), 0));
    else
      tma_box_3d(dst, map, c0, c1, c2, bar);
  };

  if (warp == 0) {
    // ---- queries and keys
    Ring r(a.kslots);
    int fills = 0, no = 0;
    while (!abort && walk.next_real(a, x)) {
      // the queries' place is free once the last scores of the tile before are
      // formed.  (A barrier of its own, with one phase a query tile: a parity
      // says nothing about a barrier that may be two phases behind, as s_full
      // is to a warp that does not wait for each of its phases.)
      if (no > 0 && !warp_wait_of<kPair>(&q_empty, static_cast<uint32_t>(no - 1) & 1u, abort)) break;
      if (elect_one()) {
        expect(&q_full, a.nq * kPreChunk);
        for (int k = 0; k + 1 < a.nq; ++k)
          copy(qsm + k * kPreChunk, &qn_map, k * 64, x.h, x.ex.q0 + x.qi0, &q_full);
        copy(qsm + (a.nq - 1) * kPreChunk, &qr_map, 0, x.h, x.ex.q0 + x.qi0, &q_full);
      }
      __syncwarp();
      ++no;
      for (int t = 0; t < x.tiles && !abort; ++t) {
        const int tok = x.ex.k0 + t * kPreTile + static_cast<int>(rank) * Shape::kKeyRows;
        for (int k = 0; k < a.nq; k += Shape::kKeyChunks) {
          if (!warp_wait_of<kPair>(&kempty[r.slot], r.turn ^ 1u, abort)) break;
          if (elect_one()) {
            const int n = min(Shape::kKeyChunks, a.nq - k);     // chunks of this slot
            uint8_t* dst = kring + r.slot * kSlotBytes;
            expect(&kfull[r.slot], n * Shape::kKeyChunkBytes);
            for (int y = 0; y < n; ++y) {
              if (k + y + 1 < a.nq)
                copy(dst + y * Shape::kKeyChunkBytes, &kn_map, (k + y) * 64, x.h, tok, &kfull[r.slot]);
              else
                copy(dst + y * Shape::kKeyChunkBytes, &kr_map, 0, 0, tok, &kfull[r.slot]);
            }
          }
          __syncwarp();
          r.step();
          ++fills;
        }
      }
    }
    // the products' last arrivals here, which in a pair come from rank 0 and
    // must not find a block that has ended
    wait_emptied<kPair>(kempty, fills, r.n, abort);
    if (no > 0) warp_wait_of<kPair>(&q_empty, static_cast<uint32_t>(no - 1) & 1u, abort);
    if (abort && leader) {
      // give the copies in flight a bounded time to land (rank 0's barriers may
      // wait for rank 1 as well: bounded all the same; rank 1's copies, which
      // are counted there, are older than the wait that gave up here, as all
      // of a warp's are)
      drain_copies(kfull, fills, r.n);
      bool late = false;
      if (no > 0) mbar_wait(&q_full, static_cast<uint32_t>(no - 1) & 1u, late);
    }
  } else if (warp == 3) {
    // ---- values
    const int half = kPair ? a.dvn >> 1 : a.dvn;      // this block's columns
    const int v0 = static_cast<int>(rank) * half, nv = (half + 63) >> 6;
    Ring r(a.vslots);
    int fills = 0;
    while (!abort && walk.next_real(a, x)) {
      for (int t = 0; t < x.tiles && !abort; ++t) {
        for (int tok = t * kPreTile; tok < min((t + 1) * kPreTile, x.see1); tok += Shape::kValRows) {
          if (!warp_wait_of<kPair>(&vempty[r.slot], r.turn ^ 1u, abort)) break;
          if (elect_one()) {
            const int bytes = nv * Shape::kValBlockBytes;
            uint8_t* dst = vring + r.slot * kSlotBytes;
            if (kPair && !leader && tok + kPreTile > x.see1) {
              // (to be cleared first: counted here, and passed on by warp 2)
              mbar_arrive_expect_tx(&vfull[r.slot], static_cast<uint32_t>(bytes));
              for (int k = 0; k < nv; ++k)
                tma_box_3d(dst + k * Shape::kValBlockBytes, &v_map, v0 + k * 64, x.h, x.ex.k0 + tok, &vfull[r.slot]);
            } else {
              expect(&vfull[r.slot], bytes);
              for (int k = 0; k < nv; ++k)
                copy(dst + k * Shape::kValBlockBytes, &v_map, v0 + k * 64, x.h, x.ex.k0 + tok, &vfull[r.slot]);
            }
          }
          __syncwarp();
          r.step();
          ++fills;
        }
      }
    }
    wait_emptied<kPair>(vempty, fills, r.n, abort);
    if (abort && leader) drain_copies(vfull, fills, r.n);
  } else if (warp == 1 && leader) {
    // ---- the products
    constexpr uint32_t idesc_s = idesc_bf16(Shape::kQueries, 128);
    const uint32_t idesc_o = idesc_bf16(Shape::kQueries, a.dvn) | kIdescBMn;
    const uint32_t q_a = smem_u32(qsm), k_a = smem_u32(kring), v_a = smem_u32(vring);
    const int nv = ((kPair ? a.dvn >> 1 : a.dvn) + 63) >> 6;
    Ring rk(a.kslots), rv(a.vslots);
    // O += P(u) V(u) of tile number u: `valid` of its keys count; `first` of its query tile
    auto output = [&](int u, int valid, bool first) {
      const int ks = (valid + 15) >> 4;               // 16-key steps that hold anything
      const uint32_t p = tmem + kPreScol + static_cast<uint32_t>(u & 1) * 128u;
      if (!warp_wait_tmem_of<kPair>(&p_full[u & 1], static_cast<uint32_t>(u >> 1) & 1u, abort)) return;
      constexpr int kSteps = Shape::kValRows / 16;
      for (int j = 0; kSteps * j < ks; ++j) {
        if (!warp_wait_of<kPair>(&vfull[rv.slot], rv.turn, abort)) return;
        clear_values<Shape::kValRows>(vring + rv.slot * kSlotBytes, nv, valid - j * Shape::kValRows, lane);
        tc_fence_after();
        if (elect_one()) {
          const uint64_t bd = sdesc_mn_sw128(v_a + static_cast<uint32_t>(rv.slot) * kSlotBytes, Shape::kValBlockBytes);
#pragma unroll
          for (int m = 0; m < kSteps; ++m) {
            const int step = kSteps * j + m;          // the weights of keys 64.. start 64 columns on
            if (step < ks)
              mma_bf16_ts_of<kPair>(tmem, p + static_cast<uint32_t>((step >> 2) * 64 + (step & 3) * 8), bd + m * 128,
                                    idesc_o, !first || step != 0);
          }
          mma_commit_of<kPair>(&vempty[rv.slot]);
          if (kSteps * (j + 1) >= ks) mma_commit_of<kPair>(&pv_done[u & 1]);
        }
        __syncwarp();
        rv.step();
      }
    };
    int i = 0, no = 0;
    bool more = walk.next_real(a, x);
    while (!abort && more) {
      if (!warp_wait_of<kPair>(&q_full, static_cast<uint32_t>(no) & 1u, abort)) break;
      ++no;
      for (int t = 0; t < x.tiles && !abort; ++t, ++i) {
        // S(i) = Q K^T; its score tile is free: the weights over it were
        // waited for and their product issued one turn ago
        const uint32_t d = tmem + kPreScol + static_cast<uint32_t>(i & 1) * 128u;
        for (int k = 0; k < a.nq; k += Shape::kKeyChunks) {
          if (!warp_wait_of<kPair>(&kfull[rk.slot], rk.turn, abort)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = q_a + static_cast<uint32_t>(k) * kPreChunk;
            const uint32_t sb = k_a + static_cast<uint32_t>(rk.slot) * kSlotBytes;
#pragma unroll
            for (int y = 0; y < Shape::kKeyChunks; ++y) {
              if (k + y >= a.nq) break;
#pragma unroll
              for (int m = 0; m < 4; ++m)
                mma_bf16_of<kPair>(d, sdesc_sw128(sa + y * kPreChunk + m * 32),
                                   sdesc_sw128(sb + y * Shape::kKeyChunkBytes + m * 32), idesc_s, (k | y | m) != 0);
            }
            mma_commit_of<kPair>(&kempty[rk.slot]);
            if (k + Shape::kKeyChunks >= a.nq) {
              mma_commit_of<kPair>(&s_full[i & 1]);
              if (t + 1 == x.tiles) mma_commit_of<kPair>(&q_empty);
            }
          }
          __syncwarp();
          rk.step();
        }
        if (t > 0 && !abort) output(i - 1, kPreTile, t == 1);
      }
      const int last = x.see1 - (x.tiles - 1) * kPreTile;
      const bool only = x.tiles == 1;
      more = walk.next_real(a, x);                    // (beside the last softmax)
      if (!abort) output(i - 1, last, only);
    }
    drain_mmas<kPair>(&drained, abort);
  } else if (kPair && warp == 2 && !leader) {
    // ---- rank 1: value tiles that end a sequence.  (A slot's phases here are
    // its tiles of that kind: the next one is copied only when rank 0's product
    // has given this one back.)
    const int nv = ((a.dvn >> 1) + 63) >> 6;
    Ring r(a.vslots);
    uint32_t phases = 0;                              // bit: the parity of a slot's next phase
    while (!abort && walk.next_real(a, x)) {
      for (int t = 0; t < x.tiles; ++t, r.step()) {
        const int valid = x.see1 - t * kPreTile;
        if (valid >= kPreTile) continue;
        if (!warp_wait(&vfull[r.slot], (phases >> r.slot) & 1u, abort)) break;
        phases ^= 1u << r.slot;
        clear_values<Shape::kValRows>(vring + r.slot * kSlotBytes, nv, valid, lane);
        if (elect_one()) mbar_arrive_cluster_release(mapa_shared(smem_u32(&vfull[r.slot]), 0));
        __syncwarp();
      }
    }
  } else if (warp == 2 && blockIdx.x == 0) {
    check_offsets(a, lane);
  } else if (warp >= 4) {
    // ---- softmax.  Warps w and w + 4 hold the same 32 queries and meet at
    // named barriers, so they walk every tile even after a wait has given up.
    const int q4 = warp & 3, g = (warp - 4) >> 2;
    const int row = q4 * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    const int dvp = (a.dv + 31) & ~31;                // accumulator columns, in halves of 16
    int i = 0;
    QueryTile then;
    for (bool more = walk.next(a, x); more; x = then) {
      const int back = x.ex.kn - x.ex.qn;
      const int see = row < x.rows ? (a.causal ? clamp_to(x.qi0 + row + 1 + back, x.ex.kn) : x.ex.kn) : 0;
      float m = 0.f, l = 0.f;
      for (int t = 0; t < x.tiles; ++t, ++i) {
        const uint32_t sb = tl + kPreScol + static_cast<uint32_t>((i & 1) * 128 + g * 64);
        uint32_t r[64];
        mbar_wait_tmem_of<kPair>(&s_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, abort);
        // O(i - 2) was done before S(i), but its arrival here is another message:
        // waited for, so that no phase of the barrier is skipped
        if (i >= 2) mbar_wait_tmem_of<kPair>(&pv_done[i & 1], static_cast<uint32_t>((i - 2) >> 1) & 1u, abort);
        __syncwarp();
        tc_fence_after();
        tmem_ld_cols<64>(sb, r);
        tmem_wait_ld_of(r);
        const int j0 = t * kPreTile + g * 64;
        if (a.flip) {
#pragma unroll
          for (int j = 0; j < 64; ++j) r[j] ^= 0x80000000u;
        }
        if ((t + 1) * kPreTile > x.see0) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (j0 + j >= see) r[j] = 0xFF800000u;
        }
        // four chains, so that the maximum is not a run of 64 dependent steps
        float m4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(__uint_as_float(r[e]), __uint_as_float(r[4 + e]));
#pragma unroll
        for (int j = 8; j < 64; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], __uint_as_float(r[j + e]), __uint_as_float(r[j + 4 + e]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.c;
        if (t == 0 || named_sync_or(1 + q4, 64, mx - m > kMaxSlack)) {
          xch[g][row] = mx;
          named_sync(1 + q4, 64);
          float mn = fmaxf(mx, xch[g ^ 1][row]);
          if (t > 0) mn = fmaxf(mn, m);
          if (mn == -INFINITY) mn = 0.f;              // a query that sees no key of the first tile sees none
          if (t > 0) {
            const float f = exp2_fast(m - mn);
            l *= f;
            mbar_wait_tmem_of<kPair>(&pv_done[(i - 1) & 1], static_cast<uint32_t>((i - 1) >> 1) & 1u, abort);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = g * (dvp >> 1); c < (g + 1) * (dvp >> 1); c += 16) {
              uint32_t o[16];
              tmem_ld16(tl + c, o);
              tmem_wait_ld_of(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tl + c, o);
            }
            tmem_wait_st();
          }
          m = mn;
          named_sync(1 + q4, 64);                     // xch is free again
        }
        // weights (rounded to bf16 for the MMA) and their fp32 sum (unrounded)
        uint32_t p[32];
        const uint64_t c2 = pair2f(a.c, a.c), m2 = pair2f(-m, -m);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float x0, x1;
          split2(fma2(pair2(r[2 * j], r[2 * j + 1]), c2, m2), x0, x1);
          x0 = exp2_fast(x0);
          x1 = exp2_fast(x1);
          sum[j & 1] = add2(sum[j & 1], pair2f(x0, x1));
          p[j] = pack_bf16x2(x0, x1);
        }
        float s0, s1;
        split2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        tmem_st_cols<32>(sb, p);
        tmem_wait_st();
        tc_fence_before();
        if (kPair && !leader) {
          // Weights in TMEM, handed on as PTX has tcgen05 operations handed from
          // thread to thread: completed and fenced by each thread, which then
          // arrives; a relaxed wait and a fence on the other side.  (Ordinary
          // memory is not part of it.  A release here, with an acquire there,
          // makes 8192 tokens x 64 heads 1777 us in place of 1325, and a local
          // barrier with one thread that passes it on with a release 1512.)
          mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&p_full[i & 1]), 0));
        } else {
          mbar_arrive(&p_full[i & 1]);
        }
      }
      // ---- output
      xch[g][row] = l;
      named_sync(1 + q4, 64);
      l = xch[0][row] + xch[1][row];
      named_sync(1 + q4, 64);                         // xch is free again
      more = walk.next(a, then);                      // (beside the last output product)
      if (x.tiles > 0) {
        mbar_wait_tmem_of<kPair>(&pv_done[(i - 1) & 1], static_cast<uint32_t>((i - 1) >> 1) & 1u, abort);
        __syncwarp();
        tc_fence_after();
      }
      const float f = l == 0.f ? 0.f : 1.0f / l;
      const int64_t tok = static_cast<int64_t>(x.ex.q0) + x.qi0 + row;
      __nv_bfloat16* dst = a.out + tok * a.o_tok + x.h * a.o_head;
      // A full tile goes out through shared memory by tensor stores, 64 values
      // of 128 queries each (four warps at a time, through a buffer of their
      // own); rows of a tile that ends a sequence are stored one by one, so that
      // the next sequence's stay untouched.  (Row by row throughout, 16 of each
      // 128-byte line at a time: 7500 cycles a tile.)
      const bool full_tile = x.rows == kPreTile;
      uint8_t* stage = osm + g * kPreChunk;
      // four warps each take every second 64-value block
#pragma unroll 1
      for (int b = g; b * 64 < a.dv; b += 2) {
#pragma unroll 1
        for (int c = b * 64; c < min(b * 64 + 64, dvp); c += 32) {
          uint32_t o[32];
          if (x.tiles > 0) {
            tmem_ld_cols<32>(tl + c, o);
            tmem_wait_ld_of(o);
          }
          uint4 w[4];
          uint32_t* wv = reinterpret_cast<uint32_t*>(w);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            wv[e] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
          if (full_tile) {
            if ((c & 63) == 0) {
              if (row == 0) tma_store_wait_read();
              named_sync(5 + g, 128);                 // the buffer has been read
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<uint4*>(stage + row * 128 + (((((c & 63) >> 3) + y) ^ (row & 7)) << 4)) = w[y];
          } else if (row < x.rows) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (c + y * 8 < a.dv) *reinterpret_cast<uint4*>(dst + c + y * 8) = w[y];   // dv is a multiple of 8
          }
        }
        if (full_tile) {
          fence_proxy_async_smem();
          named_sync(5 + g, 128);
          if (row == 0) tma_store_3d(&o_map, stage, b * 64, x.h, x.ex.q0 + x.qi0);
          __syncwarp();
        }
      }
      if (g == 0 && row < x.rows && a.lse != nullptr)
        a.lse[tok * a.H + x.h] = l == 0.f ? -INFINITY : (m + log2_fast(l)) * kLn2;
    }
    if (row == 0) tma_store_wait_read();
    __syncwarp();
  }
  if (abort) atomicOr(&g_mla_prefill_error, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync_all();                      // no MMA or arrival of either block is under way
  tc_fence_after();
  if (warp == 1) {
    if (kPair)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host
static std::atomic<int> g_prefill_grid[2][64];   // blocks that fit the device at once

template <bool kPair>
static cudaError_t launch_prefill(const MlaPrefillProblem& p, PrefillArgs a, const DeviceInfo& dev, cudaStream_t s) {
  using Shape = PreShape<kPair>;
  auto kern = mla_prefill_kernel<kPair>;
  cudaError_t e;
  const int most = kPreSmem - kPreStatic;
  int fit = g_prefill_grid[kPair ? 1 : 0][dev.device].load(std::memory_order_acquire);
  if (fit == 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPreSmem - static_cast<int>(fa.sharedSizeBytes));
    if (e != cudaSuccess) return e;
    fit = dev.sm_count;
    if (kPair) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count) & ~1u);
      cfg.blockDim = dim3(kPreThreads);
      cfg.dynamicSmemBytes = static_cast<size_t>(most);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return e;
      if (clusters < 1) return cudaErrorInvalidConfiguration;
      fit = 2 * clusters;
    }
    g_prefill_grid[kPair ? 1 : 0][dev.device].store(fit, std::memory_order_release);
  }
  // N of the output product: a multiple of 16, of 32 over a pair
  a.dvn = kPair ? (p.dv + 31) & ~31 : (p.dv + 15) & ~15;
  const int fixed = a.nq * kPreChunk + 2 * kPreChunk + 1024;
  const int slots = (most - fixed) / kSlotBytes;      // 4 or 5
  a.vslots = slots / 2;
  a.kslots = slots - a.vslots;
  CUtensorMap m[6];
  if ((e = mla_tensor_map(&m[0], p.q_nope.p, p.dn, p.H, p.Tq, p.q_nope.head, p.q_nope.tok, 64, 1, kPreTile)) !=
          cudaSuccess ||
      (e = mla_tensor_map(&m[1], p.q_rope.p, kMlaRope, p.H, p.Tq, p.q_rope.head, p.q_rope.tok, 64, 1, kPreTile)) !=
          cudaSuccess ||
      (e = mla_tensor_map(&m[2], p.k_nope.p, p.dn, p.H, p.Tk, p.k_nope.head, p.k_nope.tok, 64, 1, Shape::kKeyRows)) !=
          cudaSuccess ||
      (e = mla_tensor_map(&m[3], p.k_rope.p, kMlaRope, 1, p.Tk, kMlaRope, p.k_rope.tok, 64, 1, Shape::kKeyRows)) !=
          cudaSuccess ||
      (e = mla_tensor_map(&m[4], p.v.p, p.dv, p.H, p.Tk, p.v.head, p.v.tok, 64, 1, Shape::kValRows)) != cudaSuccess ||
      (e = mla_tensor_map(&m[5], p.out.p, p.dv, p.H, p.Tq, p.out.head, p.out.tok, 64, 1, kPreTile)) != cudaSuccess)
    return e;
  // no more blocks than tiles (at most one partly filled tile per sequence)
  const int64_t blocks = (static_cast<int64_t>(p.Tq) / Shape::kQueries + p.S) * p.H * Shape::kBlocks;
  const unsigned grid = static_cast<unsigned>(blocks < fit ? blocks : fit);
  return mla_launch_clusters(kern, dim3(grid), Shape::kBlocks, kPreThreads, fixed + slots * kSlotBytes, s, m[0], m[1],
                             m[2], m[3], m[4], m[5], a);
}

cudaError_t launch_mla_prefill(const MlaPrefillProblem& p, const DeviceInfo& dev, cudaStream_t s) {
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
  const cudaError_t e = bind_device_context();
  if (e != cudaSuccess) return e;
  PrefillArgs a{};
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(p.out.p));
  a.lse = p.lse;
  a.o_tok = p.out.tok;
  a.o_head = p.out.head;
  a.S = p.S;
  a.H = p.H;
  a.Tq = p.Tq;
  a.Tk = p.Tk;
  a.dn = p.dn;
  a.dv = p.dv;
  a.nq = static_cast<int>(ceil_div(p.dn, 64)) + 1;
  a.flip = p.scale < 0.f;
  a.c = positive_scale(a.flip ? -p.scale : p.scale);
  a.causal = p.causal;
  // a pair where the average prompt fills more than one block of it
  return p.Tq > static_cast<int64_t>(p.S) * kPreTile ? launch_prefill<true>(p, a, dev, s)
                                                     : launch_prefill<false>(p, a, dev, s);
}

uint32_t mla_prefill_read_clear_error() { return read_clear_word(g_mla_prefill_error); }

}  // namespace mx
