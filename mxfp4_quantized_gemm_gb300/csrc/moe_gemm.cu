// Grouped W4A4 MXFP4 products of a mixture of experts on the sm_103a
// block-scaled tensor cores.
//
//   y[r][n] = sum_k deq(A)[r][k] * deq(W[expert(r)])[n][k] + bias[expert(r)][n]
//
// for the rows r that the plan sorted by expert (row tiles of 128, each of
// one expert), as
//   rows:   out[pair(r)][n] = bf16_RNE(y), or
//   gated:  columns are pairs (gate, up); h = act(gate, up) in fp32 is
//           quantized per 1x32 (one rounding) into the blocked activations of
//           the second product.
//
// Few tokens: the weights of the experts they reach are nearly all the bytes
// and HBM is the bound (64 x 8 of 128 experts, a network of 5120 x 1024: 151 us,
// 0.87 of the measured rate over the whole call).  Many: the tensor pipe's four
// MMAs and scale copies per 256-wide k-step, 381 ns alone, 393 here (8192 x 8 of
// 64, gated: 228 us); the rows of the same call are bound by HBM's writes (671 MB
// in 185 us; nothing but writes goes at 3.85 TB/s).
// One kernel serves both, one CTA per SM: the ring, the
// tile (128 activation rows x 256 weight rows) and the roles are those of
// gemm.cu, and only the live rows of a row tile are loaded and stored.
//
// The number of tiles is known on the device only, so every CTA derives its
// share from the plan (struct Walk): whole rounds of units of a few tiles of
// one row tile, then single tiles, and what is left whole, in halves or cut
// along (tile, k-step).  A cut tile's parts go to memory in fp32; the CTA whose part arrives
// last (a counter per tile) adds them in CTA order, so the sum does not
// depend on who is last, and no CTA ever waits for another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "gemm_common.cuh"
#include "internal.h"
#include "layout.cuh"
#include "moe.h"
#include "ptx.cuh"

namespace mx {

static __device__ uint32_t g_moe_gemm_error;

namespace {

using C = Cfg<128>;
constexpr int kUnit = 4;                           // tiles of one row tile that a CTA takes in turn
constexpr int kPartFloats = 128 * kTileN;          // one part of a cut tile
constexpr int kMinSteps = 2;                       // k-steps a CTA takes at least where tiles are cut
constexpr int kCutSteps = 12, kCutRows = 10;       // what cutting costs, in k-steps: 12 and one for 10 rows (see Walk)
// Rows up to which a tile is finished row by row (16 alike; 48: 300 x 3 of 20 24.1
// us in place of 23.7, 1024 x 8 of 64 149.5 in place of 148.1).
constexpr int kFewRows = 32;
// Warp 0 brings the weights, warp 2 the activations, warp 1 issues the MMAs,
// warp 3 finds the segments for all of them; warps 4..11 are the epilogue.  The
// epilogue holds 128 columns of a row in registers: it takes over what the
// first warpgroup gives up (56 + 2 x 224 = 3 x 168 registers, the launch's).
// With 168 it spilled a kilobyte a thread.
constexpr int kMoeThreads = 384;
constexpr int kFirstEpiWarp = 4;
constexpr int kFewBatch = 16;                      // rows of a tile of few rows that are handed out at once
// Staging of bf16 rows that allow no wide access: per epilogue warp 8 rows of
// 128 columns, a pitch apart whose 16-byte pieces meet different banks.
constexpr int kStagePitch = 256 + 16;
constexpr int kStageWarp = 8 * kStagePitch;
static_assert(8 * kStageWarp >= kFewBatch * kTileN * 4, "the rows handed out share the staging area");
constexpr int kSegs = 8;                           // segments found ahead
constexpr int kSegBytes = 32;
constexpr int kSegReaders = 3 + 8;                 // both producers, the MMA issuer and the epilogue warps
// Of few pairs: their ids, the number of row tiles, each one's expert.
constexpr int kFewWords = kMoeFewPairs + 2 + kMoeFewPairs + 2;
constexpr int kMoeSmem = C::kSmem + 8 * kStageWarp + kSegs * kSegBytes + kFewWords * 2;
static_assert(kMoeFewPairs <= 2 * kRowTile, "few pairs of an expert fill two row tiles at most");
static_assert(kMoeMaxExperts * 4 <= 8 * kStageWarp, "the counts of few pairs stand in the staging area");
static_assert(kMoeSmem <= kMaxSmem, "ring and staging exceed shared memory");

struct MoeArgs {
  const uint8_t* a_blocks;
  const uint8_t* w_packed;
  size_t w_stride;                                 // bytes of one expert's packed weights
  const uint16_t* bias;
  int bias_vec;                                    // rows of bias allow 16-byte loads
  int N, KT, n_tiles, unit;
  uint16_t* out;
  int64_t ldo;
  int out_n;                                       // columns of out that may be written (N, or padding too)
  int out_vec;                                     // rows of out allow 16-byte accesses
  uint8_t* h_blocks;
  int KT2;
  float a1, a3, limit, shift;                      // of the activation (see gated)
  const int32_t* hdr;
  const int32_t* tile;
  int max_tiles;
  const int32_t* row_pair;
  int32_t* tickets;
  float* parts;
  const int32_t* ids;                              // of few pairs (else null): see FewPlan
  int P, E;
};

struct __align__(16) Segment {
  int rt, nt;    // row tile, column tile; rt < 0: no more segments
  int k0, len;   // first k-step, k-steps
  int half;      // 0, 1: that half of the column tile; -1: all of it
  int left;      // index among the cut tiles, or -1
  int info;      // the row tile's expert | live rows << 16
};
static_assert(sizeof(Segment) == 32, "two 16-byte words");

// A CTA's share of the tiles, segment by segment.
//  1. whole rounds of units: `unit` neighbouring tiles of one row tile, whose
//     activations (and their scales in TMEM) serve them all (8192 x 8 of 64:
//     products 229 + 185 us by four, 229 + 188 by two, 231 + 193 by one, 231 + 189
//     by eight);
//  2. whole rounds of single tiles;
//  3. the fewer than G tiles left: each on a CTA of its own, or as halves on
//     two, or cut evenly along (tile, k-step) over all CTAs together with one
//     of the rounds before, whichever takes the fewest k-steps, with the cost
//     of the cut's sums: what every row of a tile leaves in memory is written
//     and read once per part.  A tile is cut for at most four CTAs: the sum reads
//     every part (ten parts of 128 rows took 30 us).  16 rows of K = 14336 by
//     512 to 2048 columns take 24 us, uncut 34; 500 rows by 2048 uncut 42, cut 46;
//     2048 rows of K = 28672 by 2048 columns uncut 110, cut 124.
struct Walk {
  int units_per_row, unit_end, units, u, i;   // units: this CTA's next, tile of it
  int t_end, t;                               // single tiles: this CTA's next
  int h_end, h;                               // halves (two per tile from t_end)
  int its, parts_ctas, it, it1;               // cut tiles from t_end

  __device__ __forceinline__ void init(const MoeArgs& g, int row_tiles) {
    const int G = gridDim.x, c = blockIdx.x;
    units_per_row = (g.n_tiles + g.unit - 1) / g.unit;
    units = row_tiles * units_per_row;
    const int rounds = units / G;
    const int tiles = row_tiles * g.n_tiles;
    h = h_end = its = it = it1 = 0;
    parts_ctas = 1;
    u = c;
    i = 0;
    t = t_end = tiles;
    unit_end = rounds * G;
    if (unit_end >= units) return;
    const int t0 = (unit_end / units_per_row) * g.n_tiles + (unit_end % units_per_row) * g.unit;
    const int singles = (tiles - t0) / G;
    t = t0 + c;
    t_end = t0 + singles * G;
    const int rest = tiles - t_end;
    if (rest == 0) return;
    const int whole = 2 * rest > G ? g.KT : (g.KT + 1) / 2;
    const int rows = g.P / row_tiles, cost = kCutSteps + (rows < kRowTile ? rows : kRowTile) / kCutRows;
    const int even = static_cast<int>(static_cast<long long>(rest) * g.KT / G), quarter = (g.KT + 3) / 4;
    if ((singles > 0 ? even : (even > quarter ? even : quarter)) + cost < whole) {
      if (singles > 0) t_end -= G;
      const int cut = tiles - t_end;
      its = cut * g.KT;
      parts_ctas = its / kMinSteps < G ? its / kMinSteps : G;
      if (parts_ctas > 4 * cut) parts_ctas = 4 * cut;
      if (c < parts_ctas) {
        it = sk_begin(c, its, parts_ctas);
        it1 = sk_begin(c + 1, its, parts_ctas);
      }
    } else if (2 * rest > G) {
      t_end = tiles;
    } else {
      h = c;
      h_end = 2 * rest;
    }
  }

  __device__ __forceinline__ void place(const MoeArgs& g, int tile, Segment& s) {
    s.rt = tile / g.n_tiles;
    s.nt = tile - s.rt * g.n_tiles;
    s.half = -1;
    s.k0 = 0;
    s.len = g.KT;
    s.left = -1;
  }

  __device__ __forceinline__ bool next(const MoeArgs& g, Segment& s) {
    if (u < unit_end && u < units) {
      const int rt = u / units_per_row, n0 = (u - rt * units_per_row) * g.unit;
      place(g, rt * g.n_tiles + n0 + i, s);
      if (++i == g.unit || s.nt + 1 == g.n_tiles) {
        i = 0;
        u += gridDim.x;
      }
      return true;
    }
    if (t < t_end) {
      place(g, t, s);
      t += gridDim.x;
      return true;
    }
    if (h < h_end) {
      place(g, t_end + (h >> 1), s);
      s.half = h & 1;
      h += gridDim.x;
      return true;
    }
    if (it >= it1) return false;
    const int left = it / g.KT;
    place(g, t_end + left, s);
    s.left = left;
    s.k0 = it - left * g.KT;
    s.len = g.KT - s.k0 < it1 - it ? g.KT - s.k0 : it1 - it;
    it += s.len;
    return true;
  }
};

// The plan of few pairs, found from the ids by one warp: the kernel that writes
// the plan for the others is still at work then, and this one can request its
// weights beside it (the first product's start waits for it otherwise).
struct FewPlan {
  // The ids, the number of row tiles and their experts to `w`; counts: room for
  // E words.
  static __device__ __forceinline__ void init(const MoeArgs& g, int lane, int* counts, uint16_t* w) {
    int id[kMoeFewPairs / 32];
#pragma unroll
    for (int q = 0; q < kMoeFewPairs / 32; ++q) id[q] = lane + 32 * q < g.P ? __ldcg(g.ids + lane + 32 * q) : -1;
    for (int e = lane; e < g.E; e += 32) counts[e] = 0;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kMoeFewPairs / 32; ++q) {
      const bool on = static_cast<uint32_t>(id[q]) < static_cast<uint32_t>(g.E);
      if (on) atomicAdd(&counts[id[q]], 1);
      w[lane + 32 * q] = on ? static_cast<uint16_t>(id[q]) : static_cast<uint16_t>(0xFFFF);
    }
    __syncwarp();
    const int per = (g.E + 31) / 32, e0 = lane * per, e1 = e0 + per < g.E ? e0 + per : g.E;
    int n = 0;
    for (int e = e0; e < e1; ++e) n += (counts[e] + kRowTile - 1) / kRowTile;
    int upto = n;   // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) w[kMoeFewPairs] = static_cast<uint16_t>(upto);
    uint16_t* tile = w + kMoeFewPairs + 1 + upto - n;
    for (int e = e0; e < e1; ++e)
      for (int i = counts[e]; i > 0; i -= kRowTile) *tile++ = static_cast<uint16_t>(e);
  }
  static __device__ __forceinline__ int row_tiles(const uint16_t* w) { return w[kMoeFewPairs]; }
  // The word of row tile rt, as the plan's.
  static __device__ __forceinline__ int tile(const uint16_t* w, int rt, int lane) {
    const uint16_t* experts = w + kMoeFewPairs + 1;
    const int e = experts[rt];
    // the expert's rows, without its first tile's if this is its second
    int rows = rt > 0 && experts[rt - 1] == e ? -kRowTile : 0;
#pragma unroll 1
    for (int q = 0; q < kMoeFewPairs; q += 32) rows += __popc(__ballot_sync(0xFFFFFFFFu, w[q + lane] == e));
    return e | ((rows < kRowTile ? rows : kRowTile) << 16);
  }
};

__device__ __forceinline__ int loaded_rows(int live) { return (live + 15) & ~15; }

// One lane of the converged warp, chosen by the hardware: what it issues keeps
// its descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Place of the part of cut tile `left` that CTA c leaves (each CTA's range cuts
// at most two tiles).
__device__ __forceinline__ int part_slot(const Walk& w, int KT, int left, int c) {
  return 2 * c + (sk_begin(c, w.its, w.parts_ctas) / KT == left ? 0 : 1);
}

// Where 8 columns (group c8 of 32) of a row stand in a part: 1 KiB per row,
// the groups rotated by the row, so that a warp's lanes hit different L2
// slices both when they hold the same group of 32 rows (the writer: with
// rows at the same place the stores took ten times as long) and when they
// hold the groups of one row (the reader, 1 KiB side by side).
__device__ __forceinline__ int part_at(int row, int c8) { return row * kTileN + ((c8 ^ row) & 31) * 8; }
// 32 bytes at once, cached in L2 only.
__device__ __forceinline__ void stg_32B(void* p, const uint32_t* r) {
  asm volatile("st.global.cg.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void ldg_32B(const float* p, float (&v)[8]) {
  asm volatile("ld.global.cg.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}

// E8M0 byte of a block whose largest magnitude has fp32 bits `am`, by the rule
// of quant_math.cuh, and the multiplier 2^(127 - byte) of its values.
__device__ __forceinline__ uint32_t scale_byte_f32(uint32_t am, float& inv) {
  const uint32_t ef = am >> 23;
  const uint32_t sbyte = ef == 0xFF ? 0xFFu : (ef > 2 ? ef - 2 : 0u);
  inv = __uint_as_float((254u - (ef == 0xFF ? 0u : sbyte)) << 23);
  return sbyte;
}
// Codes of 4 scaled values, 2 bytes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1_codes4_f32(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "mov.b32 %0, {b0, b1, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// One 1x32 block of fp32 values held by one thread: its 16 code bytes and,
// the return value, its scale byte, by the rule of quant_math.cuh applied to
// the fp32 values (no step through bf16).
__device__ __forceinline__ uint32_t quantize32_f32(const float (&v)[32], uint4& codes) {
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  float inv;
  const uint32_t sbyte = scale_byte_f32(am, inv);
  const bool nonfinite = sbyte == 0xFFu;
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[8 * q] * inv), "f"(v[8 * q + 1] * inv), "f"(v[8 * q + 2] * inv), "f"(v[8 * q + 3] * inv),
          "f"(v[8 * q + 4] * inv), "f"(v[8 * q + 5] * inv), "f"(v[8 * q + 6] * inv), "f"(v[8 * q + 7] * inv));
    w[q] = nonfinite ? 0u : d;
  }
  codes = make_uint4(w[0], w[1], w[2], w[3]);
  return sbyte;
}

// All three activations are g / (1 + 2^(g (a1 + a3 g^2))) (u + shift) with g and
// u clamped: SiLU and the clamped form with a1 = -alpha log2 e, the tanh form
// of GELU since (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)).  (As three branches,
// unrolled over a row, the code outgrew the instruction cache: 16000 cycles a
// tile instead of 2500.)  The clamps keep a NaN.  a3 meets the gate before the
// gate's square, which is infinite for gates beyond 2^64: 0 times that would be a
// NaN in the forms without a cubic term.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float gated(const MoeArgs& g, float gate, float up) {
  gate = min_nan(gate, g.limit);
  up = max_nan(min_nan(up, g.limit), -g.limit);
  const float z = gate * fmaf(g.a3 * gate, gate, g.a1);
  return __fdividef(gate, 1.f + exp2_approx(z)) * (up + g.shift);
}

// 128 columns of one row (acc), from column n0 of its expert: stored as bf16,
// or gated and quantized.  `pair`: the row's pair, -1 past the live rows;
// `bias`: of columns n0 + 4 lane .. n0 + 4 lane + 3.  All 32 lanes call this
// together.
template <bool kGated>
__device__ __forceinline__ void finish(const MoeArgs& g, const Segment& s, uint2 bias, int pair, int rl, int h,
                                       int lane, uint8_t* stage, uint32_t (&acc)[128]) {
  if (s.half >= 0) {
    if (h != 0) return;                            // half a tile is in the first 128 columns
    h = s.half;
  }
  const int n0 = s.nt * kTileN + h * 128;
  if (g.bias != nullptr) {                         // (no + 0 without one: -0 stays)
#pragma unroll
    for (int c = 0; c < 128; c += 2) {
      const uint32_t w = __shfl_sync(0xFFFFFFFFu, (c & 2) ? bias.y : bias.x, c >> 2);
      acc[c] = __float_as_uint(__uint_as_float(acc[c]) + __uint_as_float(w << 16));
      acc[c + 1] = __float_as_uint(__uint_as_float(acc[c + 1]) + __uint_as_float(w & 0xFFFF0000u));
    }
  }
  if constexpr (!kGated) {
    if (g.out_vec != 0 && n0 + 128 <= g.out_n) {
      // Four lanes exchange their rows' 16-column pieces until each holds the
      // same piece of all four rows: then they write 128 neighbouring bytes of a
      // row, whole cache lines.  (64 bytes at a time through shared memory, the
      // second product of 8192 tokens took 252 us; 32 bytes per row 290.)
      const int q = lane & 3;
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 64) {
        uint32_t w[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[j][i] = pack_bf16x2(__uint_as_float(acc[c0 + 16 * j + 2 * i]),
                                  __uint_as_float(acc[c0 + 16 * j + 2 * i + 1]));
#pragma unroll
        for (int bit = 1; bit < 4; bit <<= 1) {
          const bool up = (q & bit) != 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j & bit) continue;                 // pieces j and j | bit change places across the lanes
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? w[j][i] : w[j | bit][i], bit);
              if (up)
                w[j][i] = got;
              else
                w[j | bit][i] = got;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = __shfl_sync(0xFFFFFFFFu, pair, (lane & ~3) + j);
          if (p < 0) continue;
          uint16_t* dst = g.out + static_cast<int64_t>(p) * g.ldo + n0 + c0 + 16 * q;
          if (g.out_vec > 1) {
            stg_32B(dst, w[j]);
          } else {
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
            *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[j][4], w[j][5], w[j][6], w[j][7]);
          }
        }
      }
      return;
    }
    // Rows that allow no wide access or end inside the tile: 8 rows at a time
    // through the warp's staging area, then a row at a time in aligned words of
    // two columns, which straddle the staged ones where the row starts at an odd
    // column: 24.4 us for 1500 x 2 tokens of 1001 columns, of 1024 six less (whole
    // lines).  Column by column it took 30, by 16 bytes a lane, put together from
    // two pieces at a place that depends on the row, 25.5.
    const int count = g.N - n0 < 128 ? g.N - n0 : 128;
    for (int b = 0; b < 4; ++b) {
      if ((lane >> 3) == b) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(stage + (lane & 7) * kStagePitch + c * 16) = make_uint4(
              pack_bf16x2(__uint_as_float(acc[8 * c]), __uint_as_float(acc[8 * c + 1])),
              pack_bf16x2(__uint_as_float(acc[8 * c + 2]), __uint_as_float(acc[8 * c + 3])),
              pack_bf16x2(__uint_as_float(acc[8 * c + 4]), __uint_as_float(acc[8 * c + 5])),
              pack_bf16x2(__uint_as_float(acc[8 * c + 6]), __uint_as_float(acc[8 * c + 7])));
      }
      __syncwarp();
#pragma unroll 4
      for (int r = 0; r < 8; ++r) {
        const int p = __shfl_sync(0xFFFFFFFFu, pair, 8 * b + r);
        uint16_t* dst = g.out + static_cast<int64_t>(p < 0 ? 0 : p) * g.ldo + n0;
        const int end = p < 0 ? 0 : count;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(stage + r * kStagePitch);
        const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 1) & 1;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = lane + 32 * u, c = 2 * i + odd;
          const uint32_t v = __funnelshift_r(row[i], row[i + 1], 16 * odd);   // (past the row's end: unused)
          if (c + 1 < end)
            *reinterpret_cast<uint32_t*>(dst + c) = v;
          else if (c < end)
            dst[c] = static_cast<uint16_t>(v);
        }
        if (odd != 0 && lane == 0 && end > 0) dst[0] = static_cast<uint16_t>(row[0]);
      }
      __syncwarp();
    }
  } else {
    const int kt2 = s.nt >> 1, grp = s.nt & 1;
    uint8_t* blk = g.h_blocks + (static_cast<size_t>(s.rt) * g.KT2 + kt2) * kMoeBlockBytes;
    uint32_t scales = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float v[32];
      // columns past N (a partial last tile) are zeros: their weights are
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = gated(g, __uint_as_float(acc[64 * b + 2 * j]), __uint_as_float(acc[64 * b + 2 * j + 1]));
      uint4 codes;
      const uint32_t sb = n0 + 64 * b < g.N ? quantize32_f32(v, codes) : 0x7Fu;
      if (n0 + 64 * b >= g.N) codes = make_uint4(0, 0, 0, 0);
      scales |= sb << (8 * b);
      const int chunk = grp * 4 + h * 2 + b;
      if (pair >= 0) *reinterpret_cast<uint4*>(blk + (rl << 7) + ((chunk ^ (rl & 7)) << 4)) = codes;
    }
    if (pair < 0) return;
    uint8_t* sc = blk + kTileBytes + ((rl & 31) << 4) + ((rl >> 5) << 2) + 2 * h;
    *reinterpret_cast<uint16_t*>(sc + (grp << 9)) = static_cast<uint16_t>(scales);
    // the last k-tile's second half has no columns: its weights are zero
    // codes, and a scale of 1 keeps the product zero whatever is there
    if (grp == 0 && s.nt + 1 == g.n_tiles) *reinterpret_cast<uint16_t*>(sc + kAtomBytes) = 0x7F7F;
  }
}

// One row of a tile, 8 columns per lane (group c8 of the tile's 32, where `on`):
// + bias, stored as bf16 by neighbouring lanes, or gated and quantized, 8
// lanes per 1x32 block.  All 32 lanes call this together.
template <bool kGated>
__device__ __forceinline__ void finish_row(const MoeArgs& g, const Segment& s, int row, int pair, int c8, bool on,
                                           const uint32_t (&b)[4], float (&v)[8]) {
  const int n0 = s.nt * kTileN + 8 * c8;
  if (g.bias != nullptr) {                         // (no + 0 without one: -0 stays)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __uint_as_float((i & 1) ? (b[i >> 1] & 0xFFFF0000u) : (b[i >> 1] << 16));
  }
  if constexpr (!kGated) {
    if (!on || n0 >= g.N) return;
    uint16_t* dst = g.out + static_cast<int64_t>(pair) * g.ldo + n0;
    if (g.out_vec != 0 && n0 + 8 <= g.out_n) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n0 + i < g.N) dst[i] = static_cast<uint16_t>(pack_bf16x2(v[i], 0.f));
    }
  } else {
    float h[4];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = n0 + 2 * i < g.N ? gated(g, v[2 * i], v[2 * i + 1]) : 0.f;
      am = max(am, __float_as_uint(h[i]) & 0x7FFFFFFFu);
    }
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 4));
    if (!on) return;
    float inv;
    const uint32_t sbyte = scale_byte_f32(am, inv);
    const uint32_t codes = sbyte == 0xFFu ? 0u : e2m1_codes4_f32(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
    const int grp = s.nt & 1, chunk = grp * 4 + (c8 >> 3);
    uint8_t* blk = g.h_blocks + (static_cast<size_t>(s.rt) * g.KT2 + (s.nt >> 1)) * kMoeBlockBytes;
    *reinterpret_cast<uint16_t*>(blk + (row << 7) + ((chunk ^ (row & 7)) << 4) + 2 * (c8 & 7)) =
        static_cast<uint16_t>(codes);
    uint8_t* sc = blk + kTileBytes + ((row & 31) << 4) + ((row >> 5) << 2);
    // (a block past the last column is zeros: scale 1, as padding has)
    if ((c8 & 7) == 0) sc[(grp << 9) + (c8 >> 3)] = n0 < g.N ? static_cast<uint8_t>(sbyte) : static_cast<uint8_t>(0x7F);
    if (c8 == 0 && grp == 0 && s.nt + 1 == g.n_tiles) *reinterpret_cast<uint32_t*>(sc + kAtomBytes) = 0x7F7F7F7Fu;
  }
}

// n neighbouring bias values of an expert from column n0 (zeros past N or
// without a bias) as words of two, by wide loads where rows allow them.
template <int kN>
__device__ __forceinline__ void load_bias(const MoeArgs& g, int expert, int n0, uint32_t (&w)[kN / 2]) {
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) w[i] = 0;
  if (g.bias == nullptr || n0 >= g.N) return;
  const uint16_t* p = g.bias + static_cast<size_t>(expert) * g.N + n0;
  if (g.bias_vec != 0 && n0 + kN <= g.N) {
    if constexpr (kN == 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x;
      w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (n0 + i < g.N) w[i >> 1] |= static_cast<uint32_t>(__ldg(p + i)) << (16 * (i & 1));
  }
}

// The sum of a cut tile's parts in CTA order, by all epilogue warps: a warp
// takes a row, a lane 8 columns of it (32 bytes of each part: a whole sector),
// so that the loads of several rows and parts are in flight together.
template <bool kGated>
__device__ __forceinline__ void finish_cut(const MoeArgs& g, const Walk& walk, const Segment& s, int expert, int rows,
                                           int c_lo, int c_hi, int warp, int lane) {
  uint32_t b[4];
  load_bias<8>(g, expert, s.nt * kTileN + 8 * lane, b);
  constexpr int kRows = 2, kAhead = 2;
  const int count = c_hi - c_lo + 1;
  // lane l: where the part of contributor l stands
  const int place0 = lane < count ? part_slot(walk, g.KT, s.left, c_lo + lane) : 0;
  for (int row0 = warp; row0 < rows; row0 += 8 * kRows) {
    float acc[kRows][8];
    int pair[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[q][i] = 0.f;
      pair[q] = !kGated && row0 + 8 * q < rows ? __ldcg(g.row_pair + s.rt * kRowTile + row0 + 8 * q) : 0;
    }
    for (int c = 0; c < count; c += kAhead) {
      float v[kAhead][kRows][8];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        int slot = __shfl_sync(0xFFFFFFFFu, place0, (c + a) & 31);
        if (c + a >= 32 && c + a < count) slot = part_slot(walk, g.KT, s.left, c_lo + c + a);
        const float* p = g.parts + static_cast<size_t>(slot) * kPartFloats;
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
          const int row = row0 + 8 * q;
          if (c + a < count && row < rows) {
            ldg_32B(p + part_at(row, lane), v[a][q]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[a][q][i] = 0.f;
          }
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
#pragma unroll
        for (int q = 0; q < kRows; ++q)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[q][i] += v[a][q][i];
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q)
      if (row0 + 8 * q < rows) finish_row<kGated>(g, s, row0 + 8 * q, pair[q], lane, true, b, acc[q]);   // (uniform)
  }
}

// The scale copies and MMAs of a k-step, from the stage's descriptors.  What the
// issuing warp does between them holds the tensor pipe up, so the stage's two
// descriptors are formed once and the others are sums with constants: no
// address in shared memory carries into the fields above it.  (8192 tokens' first
// product: 278 us with every descriptor and barrier address formed on its own and
// two k-steps' scales copied together against it, 236 so, a k-step at a time, and
// 228 without tests between the instructions.)
struct StageDescs {
  uint32_t tile, scales;   // low words at the stage's start; the high words are constants
  __device__ __forceinline__ explicit StageDescs(uint32_t stage)
      : tile(static_cast<uint32_t>(sdesc_sw128(stage))), scales(static_cast<uint32_t>(sdesc_scales(stage))) {}
};
__device__ __forceinline__ uint64_t tile_desc(uint32_t low) {
  return (sdesc_sw128(0) & 0xFFFFFFFF00000000ull) | low;
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t low) {
  return (sdesc_scales(0) & 0xFFFFFFFF00000000ull) | low;
}
constexpr int kStageSa = (C::kW + C::kA) >> 4;   // activation scales, in 16-byte pieces from the stage's start
// Half a weight block (128 rows: a code tile, then its two scale atoms).
constexpr int kHalfScales = 2 * kTileBytes;
__device__ __forceinline__ void copy_scales(const StageDescs& d, uint32_t sfb, uint32_t sfa, bool copy_a, bool half) {
  if (copy_a) {
    tmem_cp_scales(sfa, scale_desc(d.scales + kStageSa));
    tmem_cp_scales(sfa + 4, scale_desc(d.scales + kStageSa + (kAtomBytes >> 4)));
  }
  constexpr int kSw = (2 * kTileBytes) >> 4, kAtom = kAtomBytes >> 4;
  static_assert(kHalfScales == 2 * kTileBytes && kAtomBytes == 512, "both forms start alike");
  if (half) {   // atom a: k's half a
    tmem_cp_scales(sfb, scale_desc(d.scales + kSw));
    tmem_cp_scales(sfb + 8, scale_desc(d.scales + kSw + kAtom));
  } else {      // atom 2 q + a: rows 128 q.., k's half a
    tmem_cp_scales(sfb, scale_desc(d.scales + kSw));
    tmem_cp_scales(sfb + 4, scale_desc(d.scales + kSw + 2 * kAtom));
    tmem_cp_scales(sfb + 8, scale_desc(d.scales + kSw + kAtom));
    tmem_cp_scales(sfb + 12, scale_desc(d.scales + kSw + 3 * kAtom));
  }
}
__device__ __forceinline__ void commit_at(uint32_t bar) {   // mma_commit of a barrier's shared address
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <int kN>
__device__ __forceinline__ void issue_mmas(uint32_t tmem, const StageDescs& d, uint32_t sfb, uint32_t sfa,
                                           uint32_t accumulate) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    mma_mxf4(tmem, tile_desc(d.tile + (C::kW >> 4) + 2 * q), tile_desc(d.tile + 2 * q),
             idesc_mxf4(128, kN, (q & 1) * 2, (q & 1) * 2), sfa + 4 * (q >> 1), sfb + 8 * (q >> 1),
             (accumulate != 0 || q != 0) ? 1u : 0u);
}

template <bool kGated>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_gemm_kernel(const __grid_constant__ MoeArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* seg_full = acc_empty + 1;
  uint64_t* seg_empty = seg_full + kSegs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seg_empty + kSegs);
  volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* no_more = last_flag + 1;   // set by warp 3 behind its last record
  uint8_t* staging = smem + C::kRing + 512;
  uint8_t* segs = staging + 8 * kStageWarp;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool abort = false;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 2);   // both producers, and their bytes
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kEpiThreads / 32);
    *no_more = 0;
    for (int q = 0; q < kSegs; ++q) {
      mbar_init(&seg_full[q], 1);
      mbar_init(&seg_empty[q], kSegReaders);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 3 && g.ids != nullptr)
    FewPlan::init(g, lane, reinterpret_cast<int*>(staging), reinterpret_cast<uint16_t*>(segs + kSegs * kSegBytes));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The next record of the ring of segments, for one reader; false at the end.
  Segment s;
  int sslot = 0;
  uint32_t sphase = 0;
  auto read_segment = [&]() -> bool {
    const int4* p = reinterpret_cast<const int4*>(segs + sslot * kSegBytes);
    const int4 lo = p[0], hi = p[1];
    s.rt = lo.x;
    s.nt = lo.y;
    s.k0 = lo.z;
    s.len = lo.w;
    s.half = hi.x;
    s.left = hi.y;
    s.info = hi.z;
    return s.rt >= 0;
  };
  auto next_segment = [&]() -> bool { return mbar_wait(&seg_full[sslot], sphase, abort) && read_segment(); };
  // For the epilogue, whose warps share hardware barriers, which have no limit: they
  // all go through every record that was handed out, also where a wait for an
  // accumulator ran out, and leave together.  This wait ends because warp 3's do.
  auto next_of_all = [&]() -> bool {
    const uint32_t bar = smem_u32(&seg_full[sslot]);
    while (!mbar_try_wait(bar, sphase)) {
      if (*no_more == 0) continue;
      __threadfence_block();
      if (mbar_test_wait(bar, sphase)) break;
      abort = true;
      return false;
    }
    return read_segment();
  };
  auto done_segment = [&]() {
    mbar_arrive(&seg_empty[sslot]);
    if (++sslot == kSegs) {
      sslot = 0;
      sphase ^= 1;
    }
  };

  if (warp < kFirstEpiWarp) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
   if (warp == 0 || warp == 2) {
    if (lane == 0) {
      // ---- producers: warp 0 brings the weight block of each k-step (one bulk
      // copy), warp 2 the live activation rows' codes and scales.  The weights
      // do not wait for the kernel before this one.
      const bool weights = warp == 0;
      if (!weights) griddep_wait();
      int i = 0, st = 0;
      uint32_t phase = 1;
      while (next_segment()) {
        const int info = s.info, len = s.len, half = s.half;
        const uint8_t* base;
        uint32_t bytes, pitch;
        if (weights) {
          base = g.w_packed + static_cast<size_t>(info & 0xFFFF) * g.w_stride +
                 static_cast<size_t>(s.nt) * g.KT * kWeightBlockBytes;
          bytes = half < 0 ? C::kW : C::kW / 2;
          pitch = kWeightBlockBytes;
        } else {
          base = g.a_blocks + static_cast<size_t>(s.rt) * g.KT * kMoeBlockBytes;
          bytes = loaded_rows(info >> 16) * 128 + C::kSA;
          pitch = kMoeBlockBytes;
        }
        const uint8_t* src = base + static_cast<size_t>(s.k0) * pitch;
        done_segment();
        for (int j = 0; j < len; ++j, src += pitch) {
          if (!mbar_wait(&empty[st], phase, abort)) break;
          uint8_t* dst = smem + st * C::kStageBytes;
          mbar_arrive_expect_tx(&full[st], bytes);
          if (weights) {
            if (half < 0) {
              bulk_g2s(dst, src, kWeightBlockBytes, &full[st]);
            } else {
              bulk_g2s(dst, src + half * kTileBytes, kTileBytes, &full[st]);
              bulk_g2s(dst + kHalfScales, src + 2 * kTileBytes + half * 2 * kAtomBytes, 2 * kAtomBytes, &full[st]);
            }
          } else if (bytes == C::kALoad + C::kSA) {
            bulk_g2s(dst + C::kW, src, C::kALoad + C::kSA, &full[st]);
          } else {
            bulk_g2s(dst + C::kW, src, bytes - C::kSA, &full[st]);
            bulk_g2s(dst + C::kW + C::kA, src + kTileBytes, C::kSA, &full[st]);
          }
          ++i;
          if (++st == C::kStages) {
            st = 0;
            phase ^= 1;
          }
        }
      }
      if (abort) {   // the copies in flight land before the block may end
        bool late = false;
        for (int q = i < C::kStages ? 0 : i - C::kStages; q < i; ++q)
          mbar_wait(&full[q % C::kStages], (q / C::kStages) & 1, late);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer: one accumulator, one segment at a time; the activation
    // scales of a row tile stay in TMEM across its column tiles where they fit
    // (K <= 6144), as in gemm.cu.  The whole warp walks the stages and one
    // elected lane issues (in a branch of lane 0 alone a k-step's four MMAs and
    // four to six copies took 1050 cycles to issue).
    constexpr uint32_t kSfaRes = C::kSfBase + C::kStages * 16u;
    const bool resident = kSfaRes + 8u * static_cast<uint32_t>(g.KT) <= C::kTmemCols;
    const uint32_t ring = smem_u32(smem);
    const uint32_t full_at = smem_u32(full), empty_at = smem_u32(empty), full_acc_at = smem_u32(acc_full);
    // columns of the scales of k-step k in stage st
    const uint32_t sfa0 = tmem + (resident ? kSfaRes : C::kSfBase), sfa_k = resident ? 8 : 0;
    const uint32_t sfb0 = tmem + C::kSfBase + (resident ? 0 : C::kSfbOff), sfb_st = resident ? 16 : C::kSfSlot;
    const uint32_t sfa_st = resident ? 0 : C::kSfSlot;
    int cur_rt = -1;
    uint32_t have = 0;
    int st = 0;
    uint32_t phase = 0;
    bool issued = false;
    for (int seg = 0; __all_sync(0xFFFFFFFFu, next_segment()); ++seg) {   // (a wait may end for one lane alone)
      const int len = s.len, half = s.half;
      int k = s.k0;
      if (s.rt != cur_rt) {
        cur_rt = s.rt;
        have = 0;
      }
      __syncwarp();
      if (elect_one()) mbar_arrive(&seg_empty[sslot]);
      if (++sslot == kSegs) {
        sslot = 0;
        sphase ^= 1;
      }
      // Whole tiles whose activations' scales are all there, or all to be copied, go
      // without a test between the instructions of a k-step (8192 tokens' first
      // product 239 -> 228 us); halves and mixed ones with.
      const uint32_t all = resident ? ((1u << len) - 1u) << k : 0u;
      const int form = half >= 0 ? 0 : resident && (have & all) == all ? 1 : (have & all) == 0 ? 2 : 0;
      for (int j = 0; j < len; ++j, ++k) {
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(full_at + 8 * st, phase))) {
          mbar_wait(&full[st], phase, abort);
          abort = __any_sync(0xFFFFFFFFu, abort);
          if (abort) break;
        }
        tc_fence_after();
        const StageDescs d(ring + st * C::kStageBytes);
        const uint32_t sfa = sfa0 + sfa_k * k + sfa_st * st, sfb = sfb0 + sfb_st * st;
        auto copies = [&]() { copy_scales(d, sfb, sfa, ((have >> (k & 31)) & 1u) == 0, half >= 0); };
        auto mmas = [&]() {
          if (half < 0)
            issue_mmas<kTileN>(tmem, d, sfb, sfa, j != 0 ? 1u : 0u);
          else
            issue_mmas<128>(tmem, d, sfb, sfa, j != 0 ? 1u : 0u);
        };
        auto commits = [&]() {
          commit_at(empty_at + 8 * st);
          if (j + 1 == len) commit_at(full_acc_at);
        };
        if (j == 0) {   // the first scales while the accumulator is read out
          if (elect_one()) copies();
          __syncwarp();
          mbar_wait(acc_empty, (seg & 1) ^ 1, abort);
          abort = __any_sync(0xFFFFFFFFu, abort);
          if (abort) break;
          tc_fence_after();
          if (elect_one()) {
            mmas();
            commits();
          }
        } else if (form == 1) {
          if (elect_one()) {
            copy_scales(d, sfb, sfa, false, false);
            issue_mmas<kTileN>(tmem, d, sfb, sfa, 1u);
            commits();
          }
        } else if (form == 2) {
          if (elect_one()) {
            copy_scales(d, sfb, sfa, true, false);
            issue_mmas<kTileN>(tmem, d, sfb, sfa, 1u);
            commits();
          }
        } else if (elect_one()) {
          copies();
          mmas();
          commits();
        }
        __syncwarp();
        issued = true;
        if (++st == C::kStages) {
          st = 0;
          phase ^= 1;
        }
      }
      have |= all;
      if (abort) break;
    }
    __syncwarp();
    if (abort && issued) {   // the MMAs in flight end before TMEM is given back
      bool late = false;
      const int last = st == 0 ? C::kStages - 1 : st - 1;
      mbar_wait(&empty[last], st == 0 ? phase ^ 1 : phase, late);
    }
   } else {
    // ---- warp 3: the segments of this CTA, ahead of the other roles.  The plan
    // is complete when this kernel starts (the kernel before it lets it start
    // only after its own wait for the plan); that of few pairs it finds itself.
    // A segment's tile word is loaded while the one before it is handed out.
    const bool few_pairs = g.ids != nullptr;
    const uint16_t* found = reinterpret_cast<const uint16_t*>(segs + kSegs * kSegBytes);
    int tiles32 = 0;                              // loaded beside their number, for the first segments
    if (!few_pairs && lane < g.max_tiles) tiles32 = __ldcg(g.tile + lane);
    Walk walk;
    walk.init(g, few_pairs ? FewPlan::row_tiles(found) : __ldcg(g.hdr));
    int rt = -1;
    int info = 0;
    bool more = true;
    while (more && !abort) {
      more = walk.next(g, s);
      if (!more) s.rt = -1;
      if (more && s.rt != rt) {
        rt = s.rt;
        info = few_pairs ? FewPlan::tile(found, rt, lane)
               : rt < 32 ? __shfl_sync(0xFFFFFFFFu, tiles32, rt & 31)
                         : __ldcg(g.tile + rt);
      }
      mbar_wait(&seg_empty[sslot], sphase ^ 1, abort);
      abort = __any_sync(0xFFFFFFFFu, abort);
      if (abort) break;
      uint8_t* rec = segs + sslot * kSegBytes;
      if (lane == 0) {
        reinterpret_cast<int4*>(rec)[0] = make_int4(s.rt, s.nt, s.k0, s.len);
        reinterpret_cast<int4*>(rec)[1] = make_int4(s.half, s.left, info, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_full[sslot]);
      if (++sslot == kSegs) {
        sslot = 0;
        sphase ^= 1;
      }
    }
    __threadfence_block();
    if (lane == 0) *no_more = 1;
   }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---- epilogue: warp w drains accumulator rows 32 (w % 4).., columns 128 h..
    griddep_wait();
    griddep_launch_dependents();
    const int q = warp & 3;
    const int h = (warp - kFirstEpiWarp) >> 2;
    const int rl = q * 32 + lane;
    uint8_t* stage = staging + (warp - kFirstEpiWarp) * kStageWarp;
    const int ew = warp - kFirstEpiWarp;
    bool staged = false;                          // a warp's staging area may still be read by its warp
    // how the cut tiles are dealt out, for their sums
    Walk walk;
    walk.init(g, __ldcg(g.hdr));
    int pair_rt = -1, pair_of_row = -1;           // the row tile whose pairs this lane has: of row rl, or of row lane
    bool pair_few = false;                        // where the tile has few rows
    for (int seg = 0; __all_sync(0xFFFFFFFFu, next_of_all()); ++seg) {
      const int rows = s.info >> 16, expert = s.info & 0xFFFF;
      const bool whole = s.len == g.KT, few = whole && rows <= kFewRows;
      const int first_c8 = s.half > 0 ? 16 : 0;
      if (!kGated && (s.rt != pair_rt || few != pair_few)) {
        pair_rt = s.rt;
        pair_few = few;
        const int row = few ? lane : rl;
        pair_of_row = row < rows ? __ldcg(g.row_pair + static_cast<int64_t>(s.rt) * kRowTile + row) : -1;
      }
      const int pair = kGated ? (rl < rows ? 0 : -1) : pair_of_row;
      uint32_t b[4] = {0, 0, 0, 0}, b4[2] = {0, 0};
      if (few)
        load_bias<8>(g, expert, s.nt * kTileN + 8 * ((lane + first_c8) & 31), b);
      else
        load_bias<4>(g, expert, s.nt * kTileN + (s.half < 0 ? h : s.half) * 128 + 4 * lane, b4);
      // this warp has read the record
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[sslot]);
      if (++sslot == kSegs) {
        sslot = 0;
        sphase ^= 1;
      }
      mbar_wait(acc_full, seg & 1, abort);
      const bool ok = !__any_sync(0xFFFFFFFFu, abort);
      tc_fence_after();
      uint32_t r[128];
      if (q * 32 < rows) {
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 16)
          tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + h * 128 + c0,
                    *reinterpret_cast<uint32_t(*)[16]>(&r[c0]));
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);      // accumulator free for the next segment
      const bool live = rl < rows;
      if (!ok) {
#pragma unroll
        for (int c = 0; c < 128; ++c) r[c] = 0u;
      }
      if (few) {
        // Few rows: the lanes that hold them hand their columns out through
        // shared memory, 16 rows at a time, a row to a warp.
        float* sums = reinterpret_cast<float*>(staging);
        if (staged) epi_barrier();
        staged = false;
        for (int row0 = 0; row0 < rows; row0 += 16) {
          if (q == 0 && live && (lane >> 4) == (row0 >> 4) && (s.half < 0 || h == 0)) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              uint32_t* p = reinterpret_cast<uint32_t*>(sums + part_at(lane - row0, h * 16 + c));
              *reinterpret_cast<uint4*>(p) = make_uint4(r[8 * c], r[8 * c + 1], r[8 * c + 2], r[8 * c + 3]);
              *reinterpret_cast<uint4*>(p + 4) = make_uint4(r[8 * c + 4], r[8 * c + 5], r[8 * c + 6], r[8 * c + 7]);
            }
          }
          epi_barrier();
          for (int row = row0 + ew; row < rows && row < row0 + 16; row += 8) {
            const float4* p = reinterpret_cast<const float4*>(sums + part_at(row - row0, lane));
            const float4 lo = p[0], hi = p[1];
            float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            finish_row<kGated>(g, s, row, kGated ? 0 : __shfl_sync(0xFFFFFFFFu, pair, row), (lane + first_c8) & 31,
                               s.half < 0 || lane < 16, b, v);
          }
          epi_barrier();
        }
        continue;
      }
      if (whole) {
        if (q * 32 < rows) finish<kGated>(g, s, make_uint2(b4[0], b4[1]), pair, rl, h, lane, stage, r);
        staged = true;
        continue;
      }
      // A cut tile: this CTA's part to its slot; the last of the tile's CTAs
      // adds the parts.
      if (live) {
        float* p = g.parts + static_cast<size_t>(part_slot(walk, g.KT, s.left, blockIdx.x)) * kPartFloats;
#pragma unroll
        for (int c = 0; c < 16; ++c) stg_32B(p + part_at(rl, h * 16 + c), &r[8 * c]);
      }
      const int c_lo = sk_owner(s.left * g.KT, walk.its, walk.parts_ctas);
      const int c_hi = sk_owner(s.left * g.KT + g.KT - 1, walk.its, walk.parts_ctas);
      epi_barrier();
      if (threadIdx.x == kFirstEpiWarp * 32) {
        __threadfence();                          // the barrier's writes before the count
        const int before = atomicAdd(g.tickets + s.left, 1);
        __threadfence();                          // the count before the others' parts
        *last_flag = before == c_hi - c_lo;
      }
      epi_barrier();
      if (*last_flag != 0) finish_cut<kGated>(g, walk, s, expert, rows, c_lo, c_hi, ew, lane);
      epi_barrier();                              // the flag may be written again
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (abort) atomicOr(&g_moe_gemm_error, kErrTimeout);
}

std::atomic<bool> g_attr_set[64][2];

template <bool kGated>
cudaError_t launch(const MoeArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
  if (!g_attr_set[dev.device][kGated].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(moe_gemm_kernel<kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeSmem);
    if (e != cudaSuccess) return e;
    g_attr_set[dev.device][kGated].store(true, std::memory_order_release);
  }
  return launch_pdl(moe_gemm_kernel<kGated>, dev.sm_count, kMoeThreads, kMoeSmem, s, a);
}

}  // namespace

size_t moe_gemm_parts_bytes(int sm_count) { return static_cast<size_t>(2) * sm_count * kPartFloats * sizeof(float); }

cudaError_t launch_moe_gemm(const MoeGemmProblem& p, const MoePlan& plan, const DeviceInfo& dev, cudaStream_t s) {
  MoeArgs a{};
  a.a_blocks = p.a_blocks;
  a.w_packed = p.w_packed;
  a.w_stride = static_cast<size_t>(weight_packed_bytes(p.N, p.K));
  a.bias = static_cast<const uint16_t*>(p.bias);
  a.bias_vec = (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0 && p.N % 8 == 0;
  a.N = p.N;
  a.KT = static_cast<int>(padded_k(p.K) / kKTile);
  a.n_tiles = static_cast<int>(ceil_div(p.N, kTileN));
  a.unit = a.n_tiles < kUnit ? a.n_tiles : kUnit;
  a.out = static_cast<uint16_t*>(p.out);
  a.ldo = p.ldo;
  a.out_n = p.out_n;
  a.out_vec = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0 && p.ldo % 16 == 0  ? 2
              : (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % 8 == 0 ? 1
                                                                                 : 0;
  a.h_blocks = p.h_blocks;
  a.KT2 = static_cast<int>(padded_k(p.N / 2) / kKTile);
  constexpr float kLog2e = 1.4426950408889634f;
  a.limit = p.act == MoeAct::kSwigluClamp ? p.limit : __builtin_huge_valf();
  a.shift = p.act == MoeAct::kSwigluClamp ? 1.f : 0.f;
  const float by = p.act == MoeAct::kSwigluClamp ? p.alpha : p.act == MoeAct::kGeluTanh ? 1.5957691216057308f : 1.f;
  a.a1 = fmaxf(-FLT_MAX, fminf(-kLog2e * by, FLT_MAX));   // (times a gate of 0 it is 0)
  a.a3 = p.act == MoeAct::kGeluTanh ? 0.044715f * a.a1 : 0.f;
  a.hdr = plan.hdr;
  a.tile = plan.tile;
  a.max_tiles = plan.max_tiles;
  a.row_pair = plan.row_pair;
  a.tickets = plan.tickets + p.which * kMoeTickets;
  a.parts = p.parts;
  a.ids = p.ids;
  a.P = p.P;
  a.E = p.E;
  return p.h_blocks != nullptr ? launch<true>(a, dev, s) : launch<false>(a, dev, s);
}

uint32_t moe_gemm_read_clear_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_moe_gemm_error, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_moe_gemm_error, &zero, sizeof(zero));
  return v;
}

}  // namespace mx
