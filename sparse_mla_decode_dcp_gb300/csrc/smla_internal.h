// Internal launcher interface shared by the C-ABI layer and the kernel
// translation units.  Not installed; the public surface is include/smla.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace smla {

struct IndexArgs {
  const int32_t* req_id;
  const int32_t* block_table;
  int64_t bt_row_stride;
  int32_t bt_width;
  int32_t num_reqs;
  const int32_t* topk;
  int32_t T, K, D, rank, block_size;
  int32_t interleave;  // I: runs of I consecutive positions per rank
  int32_t* local_slots;
  int32_t* valid_count;  // may be null
};

constexpr int kMaxMerge = 16;

// Division of a non-negative 32-bit int (< 2^31) by a divisor fixed for the
// whole launch, as a multiply-high, an add and a shift (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994):
// with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (umulhi(n, m) + n) >> s.
struct FastDiv {
  uint32_t d, mul, shift;
};

inline FastDiv make_fastdiv(uint32_t d) {
  FastDiv f;
  f.d = d;
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  f.shift = s;
  f.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
  return f;
}

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t fastdiv(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}
#endif

struct DecodeArgs {
  const uint16_t* q;  // bf16 [T, H, 576]
  const uint8_t* kv;  // [num_slots, 656]
  int64_t num_slots;
  const int32_t* slots;  // [T, K]
  int32_t T, H, K;
  float sm_scale;
  uint16_t* out;  // bf16 [T, H, 512]
  float* lse;     // [T, H]
  void* workspace;
  size_t workspace_bytes;
  // filled by the launcher from the workspace (split-K partials)
  int32_t splits;
  int32_t split_entries;  // raw entries of every split of a row but the last
  uint16_t* ws_o;    // [T, splits, H, 512] fp16: each split's O / l (its own softmax average)
  float* ws_ml;      // [T, splits, 2 halves, 2, H]: log2-domain max, then sum
  int32_t* ws_tick;  // [kTickRows, 2] arrival counters, left at zero by every call
  int32_t combine_in_kernel;  // 1: the last split to arrive merges the row; 0: a second kernel
  int32_t single_split;       // set by the caller: no split-K whatever T (needs K <= 2048)
  // Fused DCP step only (D > 0): global top-k ids are converted per shard in
  // the kernel prologue and all shards' keys share one softmax.
  int32_t D, block_size, num_reqs, interleave;
  FastDiv div_I, div_D, div_bs;  // set by the fused and dense launchers
  // Dense decode only: row t belongs to request t / S, whose context length
  // is ctx_lens[t / S]; raw entries are positions (dense_rank < 0, all D
  // pools) or dense_rank's local positions; max_ctx bounds the positions.
  const int32_t* ctx_lens;
  int32_t S, dense_rank, max_ctx;
  int32_t window, sinks;  // windowed decode only
  // q [T*H, 576] bf16 for TMA, set by the launcher: boxes of 64 dims x 128
  // head rows (128-byte swizzle) and 32 dims x 128 head rows (64-byte swizzle)
  CUtensorMap q_lat, q_rope;
  const int32_t* req_id;
  const int32_t* topk;
  const uint8_t* pools[kMaxMerge];
  int64_t pool_slots[kMaxMerge];
  const int32_t* bts[kMaxMerge];
  int64_t bt_stride[kMaxMerge];
  int32_t bt_width[kMaxMerge];
};

struct TopkArgs {
  const float* scores;      // [T, row_stride]: select: by local position; merge: candidates
  const int32_t* cand_ids;  // merge only: [T, row_stride] global ids, -1 = none
  const int32_t* n_cand;    // select: [T] candidates per row; merge: see `chunk`
  int64_t row_stride;
  int32_t L, M, T, K, kp;   // kp: the sort's size, a power of two >= K (set by the launcher)
  int32_t D, rank, interleave;
  FastDiv div_I;            // set by the launcher
  int32_t* out_ids;         // [T, K]
  float* out_scores;        // [T, K] or null
  // Chunked selection (set by the launcher; 0 = one CTA per row).  Select:
  // CTA (i, c) takes positions [c chunk, (c + 1) chunk) of row i and writes
  // their K best, unsorted and -1 padded, to chunk_ids / chunk_scores
  // [T, gridDim.y, K].  Merge of those: row i's entries are its first
  // ceil(n_cand[i] / chunk) slabs of K (n_cand clipped to [0, L]).
  int32_t chunk;
  int32_t* chunk_ids;
  float* chunk_scores;
};

struct MapsArgs {
  const int32_t* ctx_lens;     // [B] cached positions, the new tokens included
  const int32_t* q_lens;       // [B] new tokens
  int32_t B, T, D, rank, block_size, interleave;
  FastDiv div_I, div_D, div_bs, div_ID;  // set by the launcher
  const int32_t* free_blocks;  // [num_free]
  int32_t num_free;
  int32_t* block_table;        // [B, bt_row_stride]
  int64_t bt_row_stride;
  int32_t bt_width;
  int32_t* row_start;          // [B + 1] or null
  int32_t* req_id;             // [T] or null
  int32_t* positions;          // [T] or null
  int32_t* slots;              // [T]
  int32_t* local_lens;         // [B] or null
  int32_t* blocks_taken;       // [1] or null
};

struct CacheWriteArgs {
  const uint16_t* kv;          // bf16 [T, 576], rows kv_row_stride apart
  int64_t kv_row_stride;
  int32_t T;
  const uint16_t* gamma;       // bf16 [512], or null: no norm
  float eps;
  const int32_t* positions;    // [T] (with cos_sin)
  const float* cos_sin;        // [num_positions, 64]: 32 cosines, 32 sines; null: no rotation
  int32_t num_positions;
  int32_t rope_pairs;          // 1: pairs (2i, 2i + 1); 0: pairs (i, i + 32)
  const int32_t* slots;        // [T], -1 = not this cache's
  uint8_t* kv_cache;
  int64_t num_slots;
};

struct CacheGatherArgs {
  const uint8_t* kv_cache;
  int64_t num_slots;
  const int32_t* slots;        // [N], -1 = a row of zeros
  int32_t N;
  void* out;                   // bf16 or fp32 [N, 576], rows out_row_stride apart
  int64_t out_row_stride;
};

struct MergeArgs {
  const uint16_t* outs[kMaxMerge];
  const float* lses[kMaxMerge];
  int32_t D, T, H;
  uint16_t* out;
  float* lse;
};

#ifdef __CUDACC__
// Programmatic dependent launch.  A kernel launched by launch_overlapped may
// be scheduled once every CTA of the kernel before it on the stream has
// signalled (griddep_launch_dependents) or exited, so that its launch
// overlaps that kernel's end; griddep_wait then holds it until that kernel
// has completed and its writes are visible.  Every such kernel waits before
// it touches global memory, and reads it by plain loads, never through the
// read-only path (__ldg, ld.global.nc): that is for memory nobody writes while
// the kernel runs, and this one runs from before the other's end.
__device__ __forceinline__ void griddep_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                              cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

cudaError_t launch_filter_convert(const IndexArgs& a, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_fused(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_dense(const DecodeArgs& a, cudaStream_t s);
// over 416-byte fp4 rows
cudaError_t launch_decode_fp4(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_fused_fp4(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_window(const DecodeArgs& a, bool fp4, cudaStream_t s);
// The split-K workspace begins with two arrival counters for each of up to
// this many rows; calls with more rows merge their splits in a second kernel.
constexpr int32_t kTickRows = 16384;
constexpr size_t kTickBytes = size_t(kTickRows) * 2 * sizeof(int32_t);
// Library-owned split-K scratch (no allocation by anyone at call time).
constexpr size_t kNoAllocScratchBytes = (size_t(32) << 20) + kTickBytes + 256;
// compacted entries one decode cluster handles (the key list in its shared
// memory): a decode without split-K needs K at most this
constexpr int32_t kDecodeMaxList = 2048;
cudaError_t launch_decode_noalloc(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_merge(const MergeArgs& a, cudaStream_t s);
// workspace: null, or topk_workspace_bytes(T, L, K) bytes (16-byte aligned)
// that long rows' chunked selection uses
cudaError_t launch_topk_select(const TopkArgs& a, void* workspace, cudaStream_t s);
size_t topk_workspace_bytes(int32_t T, int32_t L, int32_t K);
cudaError_t launch_topk_merge(const TopkArgs& a, cudaStream_t s);
size_t decode_workspace_bytes(int32_t T, int32_t H, int32_t K);
size_t fp4_decode_workspace_bytes(int32_t T, int32_t H, int32_t K);
size_t window_decode_workspace_bytes(int32_t T, int32_t H, int32_t K);

cudaError_t launch_step_maps(const MapsArgs& a, cudaStream_t s);
cudaError_t maps_error_word(uint32_t* flags, bool clear);
cudaError_t launch_cache_write(const CacheWriteArgs& a, bool fp4, cudaStream_t s);
cudaError_t launch_cache_gather(const CacheGatherArgs& a, bool fp4, bool fp32, cudaStream_t s);
cudaError_t cache_error_word(uint32_t* flags, bool clear);

// The fused step from and to host memory (smla_host.cu): the caller's host
// buffers and the device staging buffers their copies fill (the decode's q
// and topk point at the same staging memory).
struct HostBuffers {
  const void* q;        // host bf16 [T, H, 576]
  const int32_t* topk;  // host [T, K]
  void* out;            // host bf16 [T, H, 512]
  float* lse;           // host [T, H]
  uint16_t* q_dev;      // device staging [T, H, 576]
  int32_t* topk_dev;    // device staging [T, K]
};
cudaError_t launch_fused_host(const DecodeArgs& a, const HostBuffers& h, int groups,
                              cudaStream_t s);

// Each kernel translation unit owns one device error word.
cudaError_t index_error_word(uint32_t* flags, bool clear);
cudaError_t decode_error_word(uint32_t* flags, bool clear);
cudaError_t decode_fp4_error_word(uint32_t* flags, bool clear);
cudaError_t decode_window_error_word(uint32_t* flags, bool clear);

}  // namespace smla
