// Device and launch helpers shared by the latent-attention kernels.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mla.h"
#include "ptx.cuh"
#include "tensor_map.h"

namespace mx {

// One lane of the (converged) warp, chosen by the hardware.  MMAs issued
// under this predicate keep their descriptors in uniform registers: a group
// of four 128 x 64 x 16 MMAs with its wait and commit issues in 180 ns, and
// in 241 ns when the loop runs in a branch taken by lane 0 alone.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A bounded mbarrier wait by a whole converged warp, whose lanes go on (or
// give up) together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, bool& abort) {
  mbar_wait(bar, parity, abort);
  abort = __any_sync(0xFFFFFFFFu, abort);
  return !abort;
}
// The same for a barrier on which, in a pair of CTAs, the peer's copies,
// threads or MMAs arrive as well: acquiring at the scope of both.
template <bool kPair>
__device__ __forceinline__ bool warp_wait_of(uint64_t* bar, uint32_t parity, bool& abort) {
  if (kPair)
    mbar_wait_cluster(bar, parity, abort);
  else
    mbar_wait(bar, parity, abort);
  abort = __any_sync(0xFFFFFFFFu, abort);
  return !abort;
}

// The bounded wait of a thread that goes on with TMEM alone, which its
// tcgen05.fence::after_thread_sync orders behind the wait: in a pair relaxed at
// cluster scope, the form that PTX gives for tcgen05 operations handed from
// thread to thread.  (An acquire at that scope would order ordinary memory too,
// and takes 2000 cycles where the thread has stores under way.)
__device__ __forceinline__ bool mbar_try_wait_relaxed_cluster(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool kPair>
__device__ __forceinline__ bool mbar_wait_tmem_of(uint64_t* bar, uint32_t parity, bool& abort) {
  if (!kPair) return mbar_wait(bar, parity, abort);
  if (abort) return false;
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_relaxed_cluster(a, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_relaxed_cluster(a, parity)) {
    if (clock64() - t0 > kWaitCycles) {
      abort = true;
      return false;
    }
  }
  return true;
}
template <bool kPair>
__device__ __forceinline__ bool warp_wait_tmem_of(uint64_t* bar, uint32_t parity, bool& abort) {
  mbar_wait_tmem_of<kPair>(bar, parity, abort);
  abort = __any_sync(0xFFFFFFFFu, abort);
  return !abort;
}

// One arrival on a barrier of another CTA (address from mapa_shared), ordering
// this thread's own operations before it.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// One arrival there that also announces bytes of this thread's copies to come
// (relaxed: the copies' own completion orders what they write).
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr),
               "r"(bytes)
               : "memory");
}

// bf16 MMAs of one CTA, or of a CTA pair (cta_group::2, issued by rank 0): A
// from shared memory, or from TMEM (_ts).
template <bool kPair>
__device__ __forceinline__ void mma_bf16_of(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_bf16(d, adesc, bdesc, idesc, acc);
}
template <bool kPair>
__device__ __forceinline__ void mma_bf16_ts_of(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t acc) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  else
    mma_bf16_ts(d, a_tmem, bdesc, idesc, acc);
}
// Arrive (in both CTAs of a pair) when the issuing thread's MMAs so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit_of(uint64_t* bar) {
  if (kPair)
    mma_commit_pair(bar);
  else
    mma_commit(bar);
}

// A place in a ring of n slots with a full and an empty barrier each: the slot
// and the parity of the current turn round the ring.  One warp fills it and
// one warp empties it (a warp that skipped another's phases could take a
// barrier for complete a turn early).
struct Ring {
  int n;
  int slot = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ explicit Ring(int slots) : n(slots) {}
  __device__ __forceinline__ void step() {
    if (++slot == n) {
      slot = 0;
      turn ^= 1u;
    }
  }
};
// For the filling warp, at its end: the last `n` of its `fills` fills have been
// emptied (a wait for the phase of each slot that no further fill waits for).
template <bool kPair>
__device__ __forceinline__ void wait_emptied(uint64_t* empty, int fills, int n, bool& abort) {
  for (int f = fills > n ? fills - n : 0; f < fills; ++f)
    if (!warp_wait_of<kPair>(&empty[f % n], static_cast<uint32_t>(f / n) & 1u, abort)) return;
}
// For the filling warp, after a wait that gave up: a bounded wait for the
// copies of the `fills` fills so far that may be in flight (the last of each
// of the n slots).
__device__ __forceinline__ void drain_copies(uint64_t* full, int fills, int n) {
  for (int f = fills > n ? fills - n : 0; f < fills; ++f) {
    bool late = false;
    mbar_wait(&full[f % n], static_cast<uint32_t>(f / n) & 1u, late);
  }
}

// After a wait that gave up, by a whole warp that issued MMAs: a bounded wait
// for those in flight, before their TMEM is freed.
template <bool kPair = false>
__device__ __forceinline__ void drain_mmas(uint64_t* bar, bool abort) {
  if (!abort) return;
  if (elect_one()) mma_commit_of<kPair>(bar);
  __syncwarp();
  bool late = false;
  mbar_wait(bar, 0, late);
  __syncwarp();
}

__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// One box of a 3-D tensor map -> shared memory, completion counted on `bar`.
__device__ __forceinline__ void tma_box_3d(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// The same, completion counted on a barrier of either CTA of a pair (address
// from mapa_shared).
__device__ __forceinline__ void tma_box_3d_pair(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2,
                                                uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar)
      : "memory");
}

// One box of a 4-D tensor map.
__device__ __forceinline__ void tma_box_4d(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// A word that another kernel may be writing: read from L2, and never kept in L1.
__device__ __forceinline__ int ld_relaxed(const int* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One box, shared memory -> a 3-D tensor map; and the wait, by the same thread,
// until its boxes have been read from shared memory (which may then be used
// again, or given up: the writes complete with the grid).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(smem_src))
      : "memory");
}
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Descriptor of an operand whose M or N elements are contiguous (64 of them
// per 128-byte row, rows along K), with the 128-byte swizzle: 8-row atoms
// every 1024 bytes along K, the next 64 elements of M or N `block` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t block) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(block >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
// Instruction-descriptor bits: the operand's M (A) or N (B) elements contiguous.
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;

// tmem_wait_ld that the loaded registers depend on, so that nothing that
// reads them moves ahead of it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// N consecutive columns (a multiple of 16) of the calling warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_ld16(taddr + i, *reinterpret_cast<uint32_t(*)[16]>(&r[i]));
}
// 16 lanes x 32 columns, over the whole warp: thread t holds, of columns 8 j +
// 2 (t % 4) and the next, lane t / 4 in r[4 j], r[4 j + 1] and lane t / 4 + 8 in
// r[4 j + 2], r[4 j + 3].
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_st16(taddr + i, *reinterpret_cast<const uint32_t(*)[16]>(&r[i]));
}

// Pairs of fp32 values in one 64-bit register: an FMA or an addition of both
// is one instruction.
__device__ __forceinline__ uint64_t pair2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ uint64_t pair2f(float lo, float hi) {
  return pair2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ void split2(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^x (two units in the last place of fp32; -inf gives 0).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// log2(x); log2(0) = -inf.
__device__ __forceinline__ float log2_fast(float x) { return __log2f(x); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A row's running maximum is raised only when a score passes it by more than
// this many powers of two: until then exp2(s - max) stays below 2^8, which
// neither fp32 sums nor the bf16 weights (whose relative rounding does not
// depend on their size) lose anything to.
constexpr float kMaxSlack = 8.0f;

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier over `threads` threads that also ORs their predicate.
__device__ __forceinline__ bool named_sync_or(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}

// A predicated 4-byte store (no branch in a run of them).
__device__ __forceinline__ void st_global_if(void* p, uint32_t v, bool on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.u32 q, %2, 0;\n\t"
      "@q st.global.b32 [%0], %1;\n\t}" ::"l"(p),
      "r"(v), "r"(static_cast<uint32_t>(on))
      : "memory");
}

// Zeroes 16-byte chunks of rows [row0, row1) of a 128-byte-row tile, by one
// warp (whole rows: the swizzle permutes chunks within a row).
__device__ __forceinline__ void zero_rows(uint8_t* tile, int row0, int row1, int lane) {
  for (int i = row0 * 8 + lane; i < row1 * 8; i += 32) reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ host
// The factor from scores to powers of two.  Hidden scores are -inf and stay
// so under any positive factor; 0 x -inf would not, so a scale of zero becomes
// the least normal number, which leaves all finite scores equal just the same.
inline float positive_scale(float scale) {
  const float c = scale * kLog2e;
  return c < 1.17549435e-38f ? 1.17549435e-38f : c;
}

// Tensor map of a bf16 tensor of `n` dimensions (innermost first) with strides
// (elements) of all but the innermost, read in boxes with the 128-byte swizzle
// and zero fill outside.
template <int n>
cudaError_t mla_tensor_map_nd(CUtensorMap* map, const void* p, const int64_t (&d)[n], const int64_t (&stride)[n - 1],
                              const int (&b)[n]) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  cuuint64_t dims[n], strides[n - 1];
  cuuint32_t box[n], estr[n];
  for (int i = 0; i < n; ++i) {
    dims[i] = static_cast<cuuint64_t>(d[i]);
    box[i] = static_cast<cuuint32_t>(b[i]);
    estr[i] = 1;
  }
  for (int i = 0; i + 1 < n; ++i) strides[i] = static_cast<cuuint64_t>(stride[i]) * 2;
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n, const_cast<void*>(p), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// [d2][d1][d0]
inline cudaError_t mla_tensor_map(CUtensorMap* map, const void* p, int64_t d0, int64_t d1, int64_t d2, int64_t s1,
                                  int64_t s2, int b0, int b1, int b2) {
  return mla_tensor_map_nd<3>(map, p, {d0, d1, d2}, {s1, s2}, {b0, b1, b2});
}
// The same tensor as 64-value chunks of d0 (a multiple of 64), `chunks` of them
// to a box, which lie one behind the other: [chunk][b2][b1][64].
inline cudaError_t mla_tensor_map_chunks(CUtensorMap* map, const void* p, int64_t d0, int64_t d1, int64_t d2, int64_t s1,
                                         int64_t s2, int chunks, int b1, int b2) {
  return mla_tensor_map_nd<4>(map, p, {64, d1, d2, d0 / 64}, {s1, s2, 64}, {64, b1, b2, chunks});
}

// Launch as a programmatic dependent of the kernel ahead on the stream, in
// clusters of `cluster` blocks.
template <typename... Params, typename... Args>
cudaError_t mla_launch_clusters(void (*kern)(Params...), dim3 grid, int cluster, int threads, int smem, cudaStream_t s,
                                Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}
template <typename... Params, typename... Args>
cudaError_t mla_launch(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, Args&&... args) {
  return mla_launch_clusters(kern, grid, 1, threads, smem, s, static_cast<Args&&>(args)...);
}

// Reads and clears a translation unit's device error word.
template <typename Word>
uint32_t read_clear_word(Word& word) {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, word, sizeof(v)) != cudaSuccess) return 0;
  if (v != 0) cudaMemcpyToSymbol(word, &zero, sizeof(zero));
  return v;
}

}  // namespace mx
