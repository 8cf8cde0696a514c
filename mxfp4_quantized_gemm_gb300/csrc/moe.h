// Mixture of experts in MXFP4: host-side declarations of moe_route.cu,
// moe_plan.cu and moe_gemm.cu (entry points in capi.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace mx {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxGroups = 32;
// Bytes of one blocked activation block (128 rows of one k-tile: codes, then
// two scale atoms), as blocked_bytes() counts them.
constexpr int kMoeBlockBytes = kTileBytes + 2 * kAtomBytes;

struct MoeRouteProblem {
  const void* logits;      // [T][ld], bf16 or fp32
  bool bf16;
  int64_t ld;
  const float* bias;       // [E] or null
  int T, E, top_k;
  bool sigmoid;
  int n_group, topk_group, group_top;
  bool renormalize;
  float scale;
  float* weights;          // [T][top_k]
  int32_t* ids;            // [T][top_k]
};
cudaError_t launch_moe_route(const MoeRouteProblem& p, cudaStream_t s);

// The routed pairs (token t, slot j), pair t * top_k + j, sorted by expert:
// every expert's rows fill row tiles of 128, in the order of the pairs.
struct MoePlan {
  int32_t* hdr;            // [0]: row tiles in use
  int32_t* tile;           // [max_tiles]: expert | live rows << 16
  int32_t* row_pair;       // [max_tiles * 128]: pair of a sorted row (live rows only)
  int32_t* pos;            // [P]: sorted row of a pair, -1 where it has no expert
  int32_t* tickets;        // [2][kMoeTickets]: parts that have arrived, per cut tile of either product
  int max_tiles;
};
constexpr int kMoeTickets = 1024;   // cut tiles: fewer than two a CTA
// Row tiles that P pairs over E experts fill at most.
inline int64_t moe_max_tiles(int64_t P, int E) { return P / kRowTile + (P < E ? P : E); }
size_t moe_plan_bytes(int64_t P, int E);
MoePlan moe_plan_at(void* base, int64_t P, int E);

// The plan, and Q(x[t]) to the sorted rows of the token's pairs in blocked form;
// rows of `zero` (bf16 [P][ldz], N values, or null) whose pair has no expert are
// zeroed.
cudaError_t launch_moe_plan_gather(const int32_t* ids, int E, const void* x, int64_t ldx, int T, int top_k, int K,
                                   const MoePlan& plan, uint8_t* blocks, void* zero, int64_t ldz, int N,
                                   const DeviceInfo& dev, cudaStream_t s);
// Pairs up to which one kernel does both; the first product then starts beside
// it and finds the plan from the ids itself.
constexpr int kMoeFewPairs = 256;
// out[t] = bf16(residual[t] + sum_j weights[t][j] * parts[t * top_k + j]).
cudaError_t launch_moe_combine(const void* parts, int64_t ldp, const float* weights, const MoePlan& plan,
                               const void* residual, int64_t ldr, void* out, int64_t ldo, int T, int top_k, int N,
                               cudaStream_t s);
uint32_t moe_plan_read_clear_error();

enum class MoeAct : int { kSilu = 0, kGeluTanh = 1, kSwigluClamp = 2 };
struct MoeGemmProblem {
  const uint8_t* a_blocks;  // blocked activations of the sorted rows
  const uint8_t* w_packed;  // E packed matrices of N rows
  const void* bias;         // bf16 [E][N] or null
  int E, N, K;
  // rows: bf16 results of sorted row r to out[row_pair[r]], or
  // gated (h_blocks set): act of the column pairs (gate, up), quantized, as
  // the blocked activations of N / 2 columns.
  void* out;
  int64_t ldo;
  int out_n;                // columns of out that may be written: N, or more where the row is padded
  uint8_t* h_blocks;
  MoeAct act;
  float alpha, limit;
  int which;                // ticket set
  const int32_t* ids;       // of at most kMoeFewPairs pairs where the kernel ahead makes the plan, else null
  int P;
  float* parts;             // moe_gemm_parts_bytes()
};
size_t moe_gemm_parts_bytes(int sm_count);
cudaError_t launch_moe_gemm(const MoeGemmProblem& p, const MoePlan& plan, const DeviceInfo& dev, cudaStream_t s);
uint32_t moe_gemm_read_clear_error();

}  // namespace mx
