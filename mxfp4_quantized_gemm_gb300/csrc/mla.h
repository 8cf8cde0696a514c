// Latent attention (MLA) over a paged latent cache: host-side declarations of
// mla_store.cu, mla_decode.cu and mla_prefill.cu (entry points in capi.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace mx {

constexpr int kMlaRope = 64;          // rotated elements of a cache row
constexpr int kMlaMaxLatent = 512;    // largest latent width

// A strided bf16 tensor [token][head][element], strides in elements.
struct MlaTensor {
  const void* p;
  int64_t tok, head;
};
// The paged cache: row = latent L | rotated key R, rows of a page contiguous.
struct MlaCache {
  void* p;
  int64_t page_stride;   // elements
  int page_size, num_pages;
};

struct MlaStoreProblem {
  const void* kv;        // bf16 [T][ldkv]: latent L | key R
  int64_t ldkv;
  const void* gamma;     // bf16 [L]
  float eps;
  MlaTensor q, q_out;    // [T][H][R]
  int H;
  const float* cos_sin;  // [max_pos][R]: cos | sin
  int max_pos;
  const int64_t* positions;
  const int64_t* slots;
  MlaCache cache;
  int T, L;
  bool interleaved;
};
cudaError_t launch_mla_store(const MlaStoreProblem& p, const DeviceInfo& dev, cudaStream_t s);
uint32_t mla_store_read_clear_error();

struct MlaDecodeProblem {
  MlaTensor q_lat, q_rope, out;
  MlaCache cache;
  const int32_t* page_table;
  int64_t table_stride;
  int max_pages;
  const int32_t* seq_lens;
  float* lse;            // [S * q_len][H] or null
  int S, q_len, H, L;
  float scale;
  void* workspace;
};
// Scratch of the parts of split sequences for this grid limit; 0 where no
// sequence can be split.
size_t mla_decode_workspace(int S, int q_len, int H, int L, int64_t max_len, int sm_count);
// Whether the row groups fit the grids (their number below 2^31).
bool mla_decode_fits(int S, int q_len, int H);
cudaError_t launch_mla_decode(const MlaDecodeProblem& p, const DeviceInfo& dev, cudaStream_t s);
uint32_t mla_decode_read_clear_error();

struct MlaPrefillProblem {
  MlaTensor q_nope, q_rope, k_nope, k_rope, v, out;   // k_rope: one head
  const int32_t* cu_q;
  const int32_t* cu_k;
  float* lse;            // [Tq][H] or null
  int S, Tq, Tk, H, dn, dv;
  float scale;
  bool causal;
};
cudaError_t launch_mla_prefill(const MlaPrefillProblem& p, const DeviceInfo& dev, cudaStream_t s);
uint32_t mla_prefill_read_clear_error();

}  // namespace mx
