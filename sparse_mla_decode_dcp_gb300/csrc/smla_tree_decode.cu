// Attention of drafted trees over the packed latent cache (8- or 4-bit rows).
//
// Row (t, h) of request b attends the request's prefix (this rank's share of
// its positions, or all pools') and those nodes of its tree that its mask
// names and some pool holds:
//   s_k = sm_scale <q, k>,  lse = ln sum exp s_k,  out = sum exp(s_k - lse) latent_k
// A row with no key is written as (0, -inf).
//
// One CTA a row: four warps take keys in turn, one score a warp at a time,
// and keep their own running maximum, sum and output, which meet at the end.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "../../include/smla.h"
#include "smla_verify.h"

namespace smla {
namespace {

__device__ unsigned int g_tree_decode_error;

// Of the first n positions, how many pool d holds.
__device__ __forceinline__ int32_t pool_rows(const TreeDecodeArgs& a, int32_t n, int32_t d) {
  const int32_t full = int32_t(fastdiv(uint32_t(n), a.div_ID));
  const int64_t rest = int64_t(n) - int64_t(full) * a.div_ID.d - int64_t(d) * a.interleave;
  return full * a.interleave + int32_t(min(max(rest, int64_t(0)), int64_t(a.interleave)));
}

// A request's keys in their order: the prefix positions of pool 0, of pool 1
// and so on (or of one rank), then the tree's nodes.
struct Keys {
  int32_t first, nodes;        // the request's rows
  int32_t before[kMaxMerge + 1];  // prefix keys before pool d
  int32_t total;               // prefix keys and nodes
};

__device__ __forceinline__ int32_t prefix_keys(const Keys& k) { return k.total - k.nodes; }

// Address of key i's cache row, or null (and an error bit, where it is one)
// for a node no pool holds and an entry that is out of range.
__device__ __forceinline__ const uint8_t* key_row(const TreeDecodeArgs& a, const Keys& keys, int32_t req,
                                                  int32_t i, int row_bytes, unsigned& err) {
  int d = max(a.rank, 0);
  int64_t slot;
  if (i < prefix_keys(keys)) {
    if (a.rank < 0)
      while (i >= keys.before[d + 1]) ++d;
    const int32_t lp = i - keys.before[d];
    const int32_t col = int32_t(fastdiv(uint32_t(lp), a.div_bs));
    const int32_t blk = col < a.bt_width[d] ? a.bts[d][req * a.bt_stride[d] + col] : -1;
    if (blk < 0) {
      err |= SMLA_DEVERR_BLOCK_TABLE;
      return nullptr;
    }
    slot = int64_t(blk) * a.block_size + (lp - col * a.block_size);
  } else {
    const int32_t row = keys.first + (i - prefix_keys(keys));
    slot = a.draft_slots[d][row];
    if (a.rank < 0)
      while (slot < 0 && d + 1 < a.D) slot = a.draft_slots[++d][row];
    if (slot < 0) return nullptr;
  }
  if (slot >= a.pool_slots[d]) {
    err |= SMLA_DEVERR_SLOT_RANGE;
    return nullptr;
  }
  return a.pools[d] + slot * row_bytes;
}

// Fills `keys` for request b; false (and an error bit) for rows that lie
// outside T or are too many.  A prefix out of range leaves no keys.
__device__ bool request_keys(const TreeDecodeArgs& a, int32_t b, Keys& keys, unsigned& err) {
  const int32_t first = a.row_start[b];
  const int64_t n = int64_t(a.row_start[b + 1]) - first;
  if (first < 0 || n < 0 || n > a.max_nodes || first + n > a.T) {
    err |= SMLA_DEVERR_TREE;
    return false;
  }
  const int32_t prefix = a.prefix_lens[b];
  const bool ok = prefix >= 0 && prefix <= a.max_prefix;
  if (!ok) err |= SMLA_DEVERR_CONTEXT;
  keys.first = first;
  keys.nodes = ok ? int32_t(n) : 0;
  int32_t sum = 0;
  for (int d = 0; d < a.D; ++d) {
    keys.before[d] = a.rank < 0 ? sum : 0;
    if (ok && (a.rank < 0 || a.rank == d)) sum += pool_rows(a, prefix, d);
  }
  keys.before[a.D] = sum;
  keys.total = sum + keys.nodes;
  return true;
}

template <bool kFp4>
__device__ __forceinline__ float key_value(const uint8_t* row, int c) {
  constexpr int kRope = kFp4 ? 288 : 528;
  if (c >= SMLA_V_DIM)
    return __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(row + kRope)[c - SMLA_V_DIM]) << 16);
  if constexpr (kFp4) {
    const float s = float(*reinterpret_cast<const __nv_fp8_e4m3*>(row + 256 + c / 16));
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(row[c / 2]), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    return s * (c & 1 ? f.y : f.x);
  } else {
    return reinterpret_cast<const float*>(row + SMLA_V_DIM)[c / 128] *
           float(*reinterpret_cast<const __nv_fp8_e4m3*>(row + c));
  }
}

constexpr int kWarps = 4;

template <bool kFp4>
__global__ void __launch_bounds__(32 * kWarps) tree_decode_kernel(const __grid_constant__ TreeDecodeArgs a) {
  constexpr int kRowBytes = kFp4 ? SMLA_FP4_ROW_BYTES : SMLA_ROW_BYTES;
  __shared__ Keys keys;
  __shared__ int s_req;
  __shared__ float s_out[kWarps][SMLA_V_DIM], s_m[kWarps], s_l[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t t = int32_t(blockIdx.x) / a.H, h = int32_t(blockIdx.x) % a.H;
  griddep_launch_dependents();
  griddep_wait();
  unsigned err = 0;
  if (tid == 0) {
    int lo = 0, hi = a.B;  // the last request that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.row_start[mid] <= t) lo = mid;
      else hi = mid;
    }
    const bool ok = t >= a.row_start[lo] && t < a.row_start[lo + 1] && request_keys(a, lo, keys, err);
    s_req = ok ? lo : -1;
  }
  __syncthreads();
  if (err) atomicOr(&g_tree_decode_error, err);
  if (s_req < 0) return;
  err = 0;
  const uint16_t* q = a.q + (int64_t(t) * a.H + h) * SMLA_QK_DIM;
  float qv[SMLA_QK_DIM / 32], o[SMLA_V_DIM / 32] = {};
#pragma unroll
  for (int k = 0; k < SMLA_QK_DIM / 32; ++k) qv[k] = __uint_as_float(uint32_t(q[32 * k + lane]) << 16);
  float m = -INFINITY, l = 0.f;
  for (int32_t i = warp; i < keys.total; i += kWarps) {
    const int32_t j = i - prefix_keys(keys);
    if (j >= 0 && !((a.masks[int64_t(t) * a.mask_words + (j >> 6)] >> (j & 63)) & 1)) continue;
    const uint8_t* row = key_row(a, keys, s_req, i, kRowBytes, err);
    if (row == nullptr) continue;
    float k[SMLA_QK_DIM / 32], s = 0.f;
#pragma unroll
    for (int c = 0; c < SMLA_QK_DIM / 32; ++c) {
      k[c] = key_value<kFp4>(row, 32 * c + lane);
      s = fmaf(qv[c], k[c], s);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.sm_scale;
    const float top = fmaxf(m, s);
    const float keep = expf(m - top), p = expf(s - top);
    l = l * keep + p;
    m = top;
#pragma unroll
    for (int c = 0; c < SMLA_V_DIM / 32; ++c) o[c] = fmaf(p, k[c], o[c] * keep);
  }
  if (err) atomicOr(&g_tree_decode_error, err);
#pragma unroll
  for (int c = 0; c < SMLA_V_DIM / 32; ++c) s_out[warp][32 * c + lane] = o[c];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, w[kWarps];
  for (int x = 0; x < kWarps; ++x) top = fmaxf(top, s_m[x]);
  for (int x = 0; x < kWarps; ++x) {
    w[x] = s_m[x] == -INFINITY ? (s_l[x] == s_l[x] ? 0.f : 1.f) : expf(s_m[x] - top);
    sum += s_l[x] * w[x];
  }
  for (int c = tid; c < SMLA_V_DIM; c += 32 * kWarps) {
    float v = 0.f;
    for (int x = 0; x < kWarps; ++x) v += w[x] * s_out[x][c];
    reinterpret_cast<__nv_bfloat16*>(a.out)[(int64_t(t) * a.H + h) * SMLA_V_DIM + c] =
        __float2bfloat16_rn(sum == 0.f ? 0.f : v / sum);
  }
  if (tid == 0) a.lse[int64_t(t) * a.H + h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

size_t tree_decode_workspace_bytes(int32_t, int32_t, int32_t, int64_t) { return 0; }

cudaError_t launch_tree_decode(const TreeDecodeArgs& args, bool fp4, cudaStream_t s) {
  TreeDecodeArgs a = args;
  // a round past 2^31 positions never completes
  const uint64_t round = uint64_t(a.interleave) * uint32_t(a.D);
  a.div_ID = make_fastdiv(uint32_t(round > (1ull << 31) ? (1ull << 31) : round));
  a.div_bs = make_fastdiv(uint32_t(a.block_size));
  const unsigned grid = unsigned(a.T) * unsigned(a.H);
  return fp4 ? launch_overlapped(tree_decode_kernel<true>, grid, 32 * kWarps, 0, s, a)
             : launch_overlapped(tree_decode_kernel<false>, grid, 32 * kWarps, 0, s, a);
}

cudaError_t tree_decode_error_word(uint32_t* flags, bool clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_decode_error, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags |= v;
  if (clear) {
    v = 0;
    e = cudaMemcpyToSymbol(g_tree_decode_error, &v, sizeof(v));
  }
  return e;
}

}  // namespace smla
