// A drafted tree's bookkeeping: who sees whom (masks and rotary positions from
// the parents), which nodes the model agrees with (the greedy walk), and the
// accepted nodes' cache rows going from their drafts' slots to their own.
//
// All three move a few bytes a node and are bound by launch and memory
// latency, so each does its work in as few dependent steps as it can.  64 trees
// of 16 nodes: 3.0 us for the maps of a call among others (4,096 of up to 64
// nodes: 3.9); walk, move and a gather of 512 rows 7.9 us.
#include "../../include/smla.h"
#include "smla_verify.h"

namespace smla {
namespace {

__device__ unsigned int g_tree_error;

constexpr int kMapThreads = 256;

// The rows of request b, or an empty span (and an error bit) when they do not
// lie in [0, T) or are more than `most`.
__device__ __forceinline__ int32_t tree_span(const int32_t* row_start, int32_t b, int32_t T,
                                             int32_t most, int32_t& n, unsigned& err) {
  const int32_t first = row_start[b];
  const int64_t rows = int64_t(row_start[b + 1]) - first;
  const bool ok = first >= 0 && rows >= 0 && rows <= most && first + rows <= T;
  if (!ok) err |= SMLA_DEVERR_TREE;
  n = ok ? int32_t(rows) : 0;
  return first;
}

// Masks and positions.  A node's ancestors are gathered by doubling: after
// round r a node knows its nearest 2^r ancestors' bits, how many steps up they
// reach and the ancestor at their end, so that a chain of n nodes takes log2 n
// rounds through shared memory instead of n dependent ones.  One thread a
// node; a request's threads lie in one CTA (`group` of them, a power of two).
template <int W>
__global__ void __launch_bounds__(kMapThreads) tree_maps_kernel(const TreeMapsArgs a, int group) {
  __shared__ uint64_t s_mask[W][kMapThreads];
  __shared__ int16_t s_up[kMapThreads], s_steps[kMapThreads];
  const int tid = threadIdx.x;
  const int j = tid & (group - 1);
  const int base = tid - j;
  const int64_t req = int64_t(blockIdx.x) * (kMapThreads / group) + tid / group;
  griddep_launch_dependents();
  griddep_wait();
  unsigned err = 0;
  int32_t n = 0, first = 0;
  if (req < a.B) first = tree_span(a.row_start, int32_t(req), a.T, a.max_nodes, n, err);
  if (j != 0) err = 0;  // told once
  int up = -1;
  if (j < n) {
    up = a.parents[first + j];
    if (up < -1 || up >= j) {
      err |= SMLA_DEVERR_TREE;
      up = -1;
    }
  }
  uint64_t mask[W];
#pragma unroll
  for (int w = 0; w < W; ++w) mask[w] = (j >> 6) == w ? 1ull << (j & 63) : 0;
  int steps = up >= 0;
  while (__syncthreads_or(up >= 0)) {
#pragma unroll
    for (int w = 0; w < W; ++w) s_mask[w][tid] = mask[w];
    s_up[tid] = int16_t(up);
    s_steps[tid] = int16_t(steps);
    __syncthreads();
    if (up >= 0) {
      const int p = base + up;
#pragma unroll
      for (int w = 0; w < W; ++w) mask[w] |= s_mask[w][p];
      steps += s_steps[p];
      up = s_up[p];
    }
  }
  if (j < n) {
    const int64_t t = first + j;
#pragma unroll
    for (int w = 0; w < W; ++w) a.masks[t * W + w] = mask[w];
    if (a.positions) a.positions[t] = a.prefix_lens[req] + steps;
  }
  // rows behind the last tree
  const int64_t threads = int64_t(gridDim.x) * kMapThreads;
  for (int64_t t = max(a.row_start[a.B], 0) + int64_t(blockIdx.x) * kMapThreads + tid; t < a.T; t += threads) {
#pragma unroll
    for (int w = 0; w < W; ++w) a.masks[t * W + w] = 0;
    if (a.positions) a.positions[t] = 0;
  }
  if (err) atomicOr(&g_tree_error, err);
}

// One warp walks one tree: from node 0, the accepted one, to the lowest child
// whose token is the model's, and so on.  `visit(i, row)` is called by every
// lane for the i-th accepted row; returns their number and the last one's
// target.  Every node's way on is found at once (a lane looks at the nodes lane,
// lane + 32, ... as children), so that a step of the walk is one load from shared
// memory: `next` [kMaxTreeNodes] is the warp's, 0 where a node has no way on.
// 64 chains of 64 nodes, four of five tokens right: 21.2 us when each step looked
// for its child by ballots, 8.6 so.
template <class Visit>
__device__ __forceinline__ int walk(const TreeAcceptArgs& a, int32_t first, int32_t n, int lane, uint8_t* next,
                                    int32_t& target, Visit visit) {
  constexpr int kPer = kMaxTreeNodes / 32;
  target = -1;
  if (n == 0) return 0;
  int32_t parent[kPer], token[kPer], goal[kPer];
  __syncwarp();  // the last walk's reads
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int j = 32 * k + lane;
    parent[k] = j < n ? a.parents[first + j] : -1;
    if (parent[k] >= j) parent[k] = -1;  // not a node before
    token[k] = j < n ? a.tokens[first + j] : 0;
    if (32 * k < n) next[j] = 0;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) goal[k] = parent[k] >= 0 ? a.targets[first + parent[k]] : 0;
#pragma unroll
  for (int k = kPer - 1; k >= 0; --k) {  // the lowest child's is the last to be written
    if (32 * k >= n) continue;
    const bool fits = parent[k] >= 0 && token[k] == goal[k];
    const unsigned same = __match_any_sync(0xffffffffu, fits ? parent[k] : -1 - lane);
    __syncwarp();
    if (fits && lane == __ffs(same) - 1) next[parent[k]] = uint8_t(32 * k + lane);
  }
  __syncwarp();
  int cur = 0, count = 0;
  while (true) {
    visit(count, first + cur);
    ++count;
    const int to = next[cur];
    if (to == 0) break;
    cur = to;
  }
  target = a.targets[first + cur];
  return count;
}

// Up to kOneCta requests: one CTA, a warp each, whose paths stay in shared memory
// while the counts before them are summed.  1, 16 and 32 requests of 16 nodes:
// 2.1, 2.8 and 3.5 us, by the two launches below 3.8, 4.7 and 4.8; 64 (two a
// warp) 5.8 and 5.0.
constexpr int kOneCta = 32;

__global__ void __launch_bounds__(32 * kOneCta) tree_accept_small_kernel(const TreeAcceptArgs a) {
  __shared__ uint8_t path[kOneCta][kMaxTreeNodes], next[kOneCta][kMaxTreeNodes];
  __shared__ int count[kOneCta];
  const int b = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  unsigned err = 0;
  int32_t first = 0, accepted = 0;
  if (b < a.B) {
    int32_t n, target;
    first = tree_span(a.row_start, b, a.T, kMaxTreeNodes, n, err);
    accepted = walk(a, first, n, lane, next[b], target,
                    [&](int at, int32_t row) { path[b][at] = uint8_t(row - first); });
    if (lane == 0) {
      a.accepted[b] = accepted;
      a.next_tokens[b] = target;
    }
  }
  if (lane == 0) count[b] = accepted;
  __syncthreads();
  // every warp sums all counts
  int upto = count[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31);
  const int at = __shfl_sync(0xffffffffu, upto, b) - accepted;
  // (spans that overlap may hold more than T accepted rows)
  for (int k = lane; k < accepted && at + k < a.T; k += 32) a.rows[at + k] = first + path[b][k];
  for (int t = total + int(threadIdx.x); t < a.T; t += 32 * kOneCta) a.rows[t] = -1;
  if (err && lane == 0) atomicOr(&g_tree_error, err);
}

// More: one launch counts, the next walks again with its CTA's place summed
// from the counts (a walk costs less than a round trip of its path).
constexpr int kWalkWarps = 8;

__global__ void __launch_bounds__(32 * kWalkWarps) tree_count_kernel(const TreeAcceptArgs a) {
  __shared__ uint8_t next[kWalkWarps][kMaxTreeNodes];
  const int lane = threadIdx.x & 31;
  const int b = int(blockIdx.x) * kWalkWarps + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  if (b >= a.B) return;
  unsigned err = 0;
  int32_t n, target;
  const int32_t first = tree_span(a.row_start, b, a.T, kMaxTreeNodes, n, err);
  const int c = walk(a, first, n, lane, next[threadIdx.x >> 5], target, [](int, int32_t) {});
  if (lane == 0) {
    a.accepted[b] = c;
    a.next_tokens[b] = target;
    if (err) atomicOr(&g_tree_error, err);
  }
}

__global__ void __launch_bounds__(32 * kWalkWarps) tree_rows_kernel(const TreeAcceptArgs a) {
  __shared__ int s_before[kWalkWarps], s_total[kWalkWarps];
  __shared__ uint8_t next[kWalkWarps][kMaxTreeNodes];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b0 = int(blockIdx.x) * kWalkWarps;
  griddep_launch_dependents();
  griddep_wait();
  int before = 0, total = 0;
  for (int b = threadIdx.x; b < a.B; b += 32 * kWalkWarps) {
    const int c = a.accepted[b];
    total += c;
    before += b < b0 ? c : 0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kWalkWarps; ++w) {
    before += s_before[w];
    total += s_total[w];
  }
  const int b = b0 + warp;
  if (b < a.B) {
    const int o = b0 + lane;
    before += __reduce_add_sync(0xffffffffu, lane < warp ? a.accepted[o] : 0);
    unsigned err = 0;
    int32_t n, target;
    const int32_t first = tree_span(a.row_start, b, a.T, kMaxTreeNodes, n, err);
    walk(a, first, n, lane, next[warp], target, [&](int at, int32_t row) {
      if (lane == 0 && before + at < a.T) a.rows[before + at] = row;  // (spans may overlap)
    });
  }
  for (int64_t t = total + int64_t(blockIdx.x) * 32 * kWalkWarps + threadIdx.x; t < a.T;
       t += int64_t(gridDim.x) * 32 * kWalkWarps)
    a.rows[t] = -1;
}

// A warp moves eight entries: it asks for all their rows' bytes, 16 a lane,
// before it stores any.
constexpr int kMoveWarps = 4;
constexpr int kMoveRows = 8;

template <int kRowBytes>
__global__ void __launch_bounds__(32 * kMoveWarps) cache_move_kernel(const CacheMoveArgs a) {
  constexpr int kPieces = kRowBytes / 16;
  constexpr int kRounds = (kPieces + 31) / 32;
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (int64_t(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5)) * kMoveRows;
  griddep_launch_dependents();
  griddep_wait();
  unsigned err = 0;
  int32_t src = -1, dst = -1;
  if (lane < kMoveRows && i0 + lane < a.N) {
    const int32_t row = a.rows[i0 + lane];
    dst = row == -1 ? -1 : a.dst_slots[i0 + lane];
    if (dst >= 0) {
      src = row >= 0 && row < a.T ? a.src_slots[row] : -1;
      if (src < 0 || src >= a.num_slots || dst >= a.num_slots) {  // a row would be lost
        err = SMLA_DEVERR_SLOT_RANGE;
        src = dst = -1;
      }
    }
  }
  uint4 v[kMoveRows][kRounds];
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) {
    const int32_t s = __shfl_sync(0xffffffffu, src, r);
    const int32_t d = __shfl_sync(0xffffffffu, dst, r);
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
      if (d >= 0 && 32 * k + lane < kPieces)
        v[r][k] = reinterpret_cast<const uint4*>(a.kv_cache + int64_t(s) * kRowBytes)[32 * k + lane];
  }
#pragma unroll
  for (int r = 0; r < kMoveRows; ++r) {
    const int32_t d = __shfl_sync(0xffffffffu, dst, r);
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
      if (d >= 0 && 32 * k + lane < kPieces)
        reinterpret_cast<uint4*>(a.kv_cache + int64_t(d) * kRowBytes)[32 * k + lane] = v[r][k];
  }
  if (err) atomicOr(&g_tree_error, err);
}

}  // namespace

cudaError_t launch_tree_maps(const TreeMapsArgs& a, cudaStream_t s) {
  int group = 32;
  while (group < a.max_nodes) group *= 2;
  const int64_t per = kMapThreads / group;
  const unsigned grid = a.B > 0 ? unsigned((a.B + per - 1) / per) : 1;  // padding rows alone, too
  switch ((a.max_nodes + 63) / 64) {
    case 1: return launch_overlapped(tree_maps_kernel<1>, grid, kMapThreads, 0, s, a, group);
    case 2: return launch_overlapped(tree_maps_kernel<2>, grid, kMapThreads, 0, s, a, group);
    case 3: return launch_overlapped(tree_maps_kernel<3>, grid, kMapThreads, 0, s, a, group);
    default: return launch_overlapped(tree_maps_kernel<4>, grid, kMapThreads, 0, s, a, group);
  }
}

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t s) {
  if (a.B <= kOneCta) return launch_overlapped(tree_accept_small_kernel, 1, 32 * kOneCta, 0, s, a);
  const unsigned grid = unsigned((a.B + kWalkWarps - 1) / kWalkWarps);
  const cudaError_t e = launch_overlapped(tree_count_kernel, grid, 32 * kWalkWarps, 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_overlapped(tree_rows_kernel, grid, 32 * kWalkWarps, 0, s, a);
}

cudaError_t launch_cache_move(const CacheMoveArgs& a, bool fp4, cudaStream_t s) {
  const int64_t per = kMoveWarps * kMoveRows;
  const unsigned grid = unsigned((int64_t(a.N) + per - 1) / per);
  return fp4 ? launch_overlapped(cache_move_kernel<SMLA_FP4_ROW_BYTES>, grid, 32 * kMoveWarps, 0, s, a)
             : launch_overlapped(cache_move_kernel<SMLA_ROW_BYTES>, grid, 32 * kMoveWarps, 0, s, a);
}

cudaError_t tree_error_word(uint32_t* flags, bool clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_error, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags |= v;
  if (clear) {
    v = 0;
    e = cudaMemcpyToSymbol(g_tree_error, &v, sizeof(v));
  }
  return e;
}

}  // namespace smla
