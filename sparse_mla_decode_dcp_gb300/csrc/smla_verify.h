// Internal launcher interface of the verification step's operators (drafted
// trees) and of the 8-bit products.  Not installed; the public surface is
// include/smla.h.
#pragma once

#include "smla_internal.h"

namespace smla {

// Nodes of one request's tree; the walk and the masks hold a node's index in
// 8 bits and in up to four 64-bit words.
constexpr int kMaxTreeNodes = 256;

struct TreeMapsArgs {
  const int32_t* parents;      // [T]
  const int32_t* row_start;    // [B + 1]
  const int32_t* prefix_lens;  // [B] (with positions)
  int32_t B, T, max_nodes;
  uint64_t* masks;             // [T, ceil(max_nodes / 64)]
  int32_t* positions;          // [T] or null
};

struct TreeAcceptArgs {
  const int32_t* parents;      // [T]
  const int32_t* tokens;       // [T]
  const int32_t* targets;      // [T]
  const int32_t* row_start;    // [B + 1]
  int32_t B, T;
  int32_t* accepted;           // [B]
  int32_t* rows;               // [T]
  int32_t* next_tokens;        // [B]
};

struct CacheMoveArgs {
  uint8_t* kv_cache;
  int64_t num_slots;
  const int32_t* rows;         // [N], -1 = nothing
  int32_t N;
  const int32_t* src_slots;    // [T]
  int32_t T;
  const int32_t* dst_slots;    // [N], -1 = another cache's
};

struct TreeDecodeArgs {
  const uint16_t* q;           // bf16 [T, H, 576]
  int32_t T, B, H;
  float sm_scale;
  const int32_t* row_start;    // [B + 1]
  const int32_t* prefix_lens;  // [B]
  int32_t max_prefix;
  const uint64_t* masks;       // [T, mask_words]
  int32_t max_nodes, mask_words;
  const int32_t* positions;    // [T] (with a window)
  int32_t window, sinks;       // window 0: none
  int32_t D, rank, block_size, interleave;  // rank -1: all pools
  FastDiv div_ID, div_bs;      // set by the launcher
  const uint8_t* pools[kMaxMerge];
  int64_t pool_slots[kMaxMerge];
  const int32_t* bts[kMaxMerge];
  int64_t bt_stride[kMaxMerge];
  int32_t bt_width[kMaxMerge];
  const int32_t* draft_slots[kMaxMerge];  // [T] each
  uint16_t* out;               // bf16 [T, H, 512]
  float* lse;                  // [T, H]
  void* workspace;
  // set by the launcher
  int32_t split;               // a tile of rows may be cut into key ranges
  int32_t min_units;           // key tiles a pair takes at least
  void* ws_desc;               // per pair: the cut tile it begins
  float* ws_ml;                // [2 pairs, 128, 2]
  uint16_t* ws_o;              // fp16 [2 pairs, 128, 512]
};

// A batch of matrices: entry (g, row, col) is at g * batch + row * rows + col
// * cols, in elements.
struct Strides {
  int64_t batch, rows, cols;
};

struct QuantiseArgs {
  const uint16_t* x;  // bf16, columns contiguous
  Strides xs;
  int32_t G, M, K;
  uint8_t* codes;     // columns contiguous
  Strides cs;
  float* scales;      // [G, M, ceil(K / 128)]
  Strides ss;
};

struct MatmulArgs {
  CUtensorMap a_map, b_map;  // set by the launcher
  const uint8_t* a;          // [G, M, K], columns contiguous
  Strides as;
  const float* a_scales;     // [G, M, ceil(K / 128)]
  Strides ass;
  const uint8_t* b;          // [G, N, K], columns contiguous
  Strides bs;
  const float* b_scales;     // [G, ceil(N / 128), ceil(K / 128)]
  Strides bss;
  int32_t G, M, N, K;
  void* out;                 // [G, M, N], columns contiguous
  Strides os;
  int32_t out_fp32;
  // set by the launcher
  int32_t m_tiles, n_tiles, k_blocks, splits, stages, vec;
  uint32_t tiles;            // of all batches
};

// max_keys: of a request
cudaError_t launch_tree_decode(const TreeDecodeArgs& a, int64_t max_keys, bool fp4, cudaStream_t s);
// what the call needs, and what it and any of fewer rows, requests or keys need
size_t tree_decode_workspace_bytes(int32_t T, int32_t B, int32_t H, int64_t max_keys);
size_t tree_decode_most_workspace_bytes(int32_t T, int32_t B, int32_t H, int64_t max_keys);
cudaError_t tree_decode_error_word(uint32_t* flags, bool clear);

cudaError_t launch_fp8_quantise(const QuantiseArgs& a, cudaStream_t s);
cudaError_t launch_fp8_matmul(const MatmulArgs& a, cudaStream_t s);
cudaError_t matmul_error_word(uint32_t* flags, bool clear);

cudaError_t launch_tree_maps(const TreeMapsArgs& a, cudaStream_t s);
cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t s);
cudaError_t launch_cache_move(const CacheMoveArgs& a, bool fp4, cudaStream_t s);
cudaError_t tree_error_word(uint32_t* flags, bool clear);

}  // namespace smla
