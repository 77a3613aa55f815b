// Step maps: a decode or prefill step's request ids, positions and cache
// slots, and the block-table entries its new tokens need, from the requests'
// lengths.
//
// Request b has c = ctx[b] cached positions, q[b] of them new.  Of the first
// n positions rank r holds rows(n) = (n div ID) I + clamp(n mod ID - r I, 0,
// I) (ID = I D), which fill nb(n) = ceil(rows(n) / block_size) blocks.  So
// the request takes need = nb(c) - nb(c - q) blocks from the free list, at
// the exclusive sum of the needs before it, and its rows start at the
// exclusive sum of the q before it.
//
// One launch.  Every CTA computes both sums for all requests itself (two
// lengths each, one block scan) and keeps them in shared memory, so that no
// CTA waits for another; then its rows each find their request by a binary
// search of the row starts.  A new block's first local position belongs to a
// new token (the old tokens' blocks cover every older position), so the row
// of that token writes the block-table entry, and a row in a new block reads
// its block id from the free list, never an entry another row may be
// writing.  A row costs 12 bytes out and at most 4 in.  Measured on a GB300: 1
// request 1.7 us, 64 decode rows 1.9, 512 2.7; 509 requests with 66,170 rows
// 3.8 us.  Up to there a launch's own latency and, past 256 requests, one more
// scan bound it; 8,192 requests take 32 scans and 19 us, little beside the
// attention of as many requests.
#include <atomic>

#include "../../include/smla.h"
#include "smla_internal.h"

namespace smla {
namespace {

__device__ unsigned int g_maps_error;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct ReqSpan {
  int32_t row_start;   // first row
  int32_t first_free;  // first free-list entry
  int32_t old_len;     // cached positions before the step
  int32_t old_blocks;  // blocks they fill on this rank
};

__device__ __forceinline__ int32_t rank_rows(const MapsArgs& a, int32_t n) {
  const int32_t full = int32_t(fastdiv(uint32_t(n), a.div_ID));
  const int64_t rem = int64_t(n) - int64_t(full) * a.div_ID.d;
  const int64_t mine = rem - int64_t(a.rank) * a.interleave;
  return full * a.interleave + int32_t(min(max(mine, int64_t(0)), int64_t(a.interleave)));
}

__device__ __forceinline__ int32_t blocks_of(const MapsArgs& a, int32_t rows) {
  const int32_t full = int32_t(fastdiv(uint32_t(rows), a.div_bs));
  return full + (rows > full * a.block_size ? 1 : 0);
}

__global__ void __launch_bounds__(kThreads) step_maps_kernel(const MapsArgs a) {
  extern __shared__ ReqSpan span[];  // [B]
  __shared__ int64_t warp_q[kWarps], warp_need[kWarps];
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const bool first_cta = blockIdx.x == 0;
  griddep_launch_dependents();
  griddep_wait();
  unsigned err = 0;

  // 1) both exclusive sums, requests in chunks of one per thread; 64-bit, so
  //    that lengths that do not fit T are recognised.  A chunk's lengths are
  //    loaded while the chunk before it is summed.
  int64_t q_base = 0, need_base = 0;
  int32_t c_next = 0, q_next = 0;
  auto fetch = [&](int b) {
    c_next = b < a.B ? a.ctx_lens[b] : 0;
    q_next = b < a.B ? a.q_lens[b] : 0;
  };
  fetch(tid);
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int32_t c = c_next, q = q_next;
    if (b0 + kThreads < a.B) fetch(b + kThreads);
    if (b < a.B) {
      if (c < 0 || q < 0 || q > c) {
        err |= SMLA_DEVERR_CONTEXT;
        c = max(c, 0);
        q = 0;
      }
    }
    const int32_t rows = rank_rows(a, c);
    const int32_t old_blocks = blocks_of(a, rank_rows(a, c - q));
    const int32_t need = blocks_of(a, rows) - old_blocks;
    int64_t iq = q, in = need;  // inclusive warp scans
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t yq = __shfl_up_sync(0xffffffffu, iq, off);
      const int64_t yn = __shfl_up_sync(0xffffffffu, in, off);
      if (lane >= off) {
        iq += yq;
        in += yn;
      }
    }
    __syncthreads();  // the previous chunk's sums are read
    if (lane == 31) {
      warp_q[warp] = iq;
      warp_need[warp] = in;
    }
    __syncthreads();
    int64_t pq = q_base, pn = need_base;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        pq += warp_q[w];
        pn += warp_need[w];
      }
      q_base += warp_q[w];
      need_base += warp_need[w];
    }
    if (b < a.B) {
      const int32_t start = int32_t(min(pq + iq - q, int64_t(INT32_MAX)));
      span[b].row_start = start;
      span[b].first_free = int32_t(min(pn + in - need, int64_t(INT32_MAX)));
      span[b].old_len = c - q;
      span[b].old_blocks = old_blocks;
      if (first_cta) {
        if (a.row_start) a.row_start[b] = start;
        if (a.local_lens) a.local_lens[b] = rows;
      }
    }
  }
  if (q_base > a.T) err |= SMLA_DEVERR_CONTEXT;
  if (first_cta && tid == 0) {
    if (a.row_start) a.row_start[a.B] = int32_t(min(q_base, int64_t(INT32_MAX)));
    if (a.blocks_taken) *a.blocks_taken = int32_t(min(need_base, int64_t(INT32_MAX)));
  }
  __syncthreads();

  // 2) this CTA's rows
  const int32_t total = int32_t(min(q_base, int64_t(a.T)));
  for (int64_t row = int64_t(blockIdx.x) * kThreads + tid; row < a.T;
       row += int64_t(gridDim.x) * kThreads) {
    const int32_t t = int32_t(row);
    int32_t req = 0, pos = 0, slot = -1;
    if (t < total) {
      int lo = 0, hi = a.B;  // the last request that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (span[mid].row_start <= t)
          lo = mid;
        else
          hi = mid;
      }
      const ReqSpan sp = span[lo];
      req = lo;
      pos = sp.old_len + (t - sp.row_start);
      const uint32_t g = fastdiv(uint32_t(pos), a.div_I);
      const uint32_t round = fastdiv(g, a.div_D);
      if (int32_t(g - round * uint32_t(a.D)) == a.rank) {
        const int32_t lp = int32_t(round) * a.interleave + (pos - int32_t(g) * a.interleave);
        const int32_t col = int32_t(fastdiv(uint32_t(lp), a.div_bs));
        const int32_t at = lp - col * a.block_size;
        int32_t blk = -1;
        int32_t* entry = a.block_table + int64_t(lo) * a.bt_row_stride + col;
        if (col >= a.bt_width) {
          err |= SMLA_DEVERR_BLOCK_TABLE;
        } else if (col >= sp.old_blocks) {
          const int64_t f = int64_t(sp.first_free) + (col - sp.old_blocks);
          if (f < a.num_free)
            blk = a.free_blocks[f];
          else
            err |= SMLA_DEVERR_FREE_BLOCKS;
          if (at == 0) *entry = blk;
          if (f < a.num_free && blk < 0) err |= SMLA_DEVERR_BLOCK_TABLE;
        } else {
          blk = *entry;
          if (blk < 0) err |= SMLA_DEVERR_BLOCK_TABLE;
        }
        if (blk >= 0) {
          const int64_t s64 = int64_t(blk) * a.block_size + at;
          if (s64 > INT32_MAX)
            err |= SMLA_DEVERR_BLOCK_TABLE;
          else
            slot = int32_t(s64);
        }
      }
    }
    if (a.req_id) a.req_id[t] = req;
    if (a.positions) a.positions[t] = pos;
    a.slots[t] = slot;
  }
  if (err) atomicOr(&g_maps_error, err);
}

}  // namespace

// The kernel's shared-memory limit, once per device and for the largest batch:
// a limit set for each launch's own batch would be lowered by another host
// thread between the setting and the launch.
static cudaError_t allow_all_spans() {
  constexpr int kDevices = 64;
  constexpr int kBytes = SMLA_MAX_STEP_REQS * int(sizeof(ReqSpan));
  static_assert(kBytes <= 227 * 1024 - 4096, "spans fit shared memory");
  static std::atomic<bool> done[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < kDevices;
  if (tracked && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(step_maps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e == cudaSuccess && tracked) done[dev].store(true, std::memory_order_release);
  return e;
}

cudaError_t launch_step_maps(const MapsArgs& args, cudaStream_t s) {
  MapsArgs a = args;
  a.div_I = make_fastdiv(uint32_t(a.interleave));
  a.div_D = make_fastdiv(uint32_t(a.D));
  a.div_bs = make_fastdiv(uint32_t(a.block_size));
  // a round past 2^31 positions never completes
  const uint64_t round = uint64_t(a.interleave) * uint32_t(a.D);
  a.div_ID = make_fastdiv(uint32_t(round > (1ull << 31) ? (1ull << 31) : round));
  const size_t smem = size_t(a.B) * sizeof(ReqSpan);
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_all_spans();
    if (e != cudaSuccess) return e;
  }
  const int64_t need = (int64_t(a.T) + kThreads - 1) / kThreads;
  const unsigned grid = unsigned(need < 1 ? 1 : need > 152 ? 152 : need);
  return launch_overlapped(step_maps_kernel, grid, kThreads, smem, s, a);
}

cudaError_t maps_error_word(uint32_t* flags, bool clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_maps_error, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags |= v;
  if (clear) {
    v = 0;
    e = cudaMemcpyToSymbol(g_maps_error, &v, sizeof(v));
  }
  return e;
}

}  // namespace smla
