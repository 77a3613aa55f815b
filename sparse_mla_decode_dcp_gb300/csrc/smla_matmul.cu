// 8-bit matrix product with a scale for each block of 128: for each batch
// entry,
//   out[m, n] = sum_g sa[m, g] sb[n / 128, g] sum_{k in group g} a[m, k] b[n, k]
// with e4m3 codes a (rows of activations, one scale for 128 columns) and b
// (weights, one scale for 128 x 128), groups of 128 k.
//
// The tensor cores sum one group at a time: a scale is any fp32 number, so the
// group's sums come back from tensor memory and are added, times their scale,
// to fp32 sums in registers while the next group's MMAs run (two accumulators
// in turn).  TMA brings a group's codes as 128-byte rows in the MMA's
// swizzle, several groups ahead.
//
// One operand's rows are the MMA's 128 lanes, the other's its columns.  Many
// activation rows lie along the lanes (kSwap false, tiles of 128 x 128, and with
// enough of them the pairs' of 256 x 160 to 256 x 256 below); up to 64 of them
// along the columns, where a tile of 16, 32 or 64 wastes little, and the
// weights' rows along the lanes: such a call is bound by the weights' bytes.  A weight tile of
// 128 rows has one scale a group either way.
//
// With few tiles the groups are split over the CTAs of a cluster, whose sums
// meet through distributed shared memory in the order of their groups.
//
// Warps: 0 loads (one lane), 1 issues the MMAs (one lane), 2 holds tensor
// memory, 4 and up read the sums.  Every wait is bounded; one that gives up
// sets SMLA_DEVERR_TIMEOUT and the CTA unwinds.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "../../include/smla.h"
#include "smla_pair.cuh"
#include "smla_verify.h"

namespace smla {
namespace {

using namespace sm100;

__device__ unsigned int g_matmul_error;

constexpr int kGroup = 128;        // k of a scale, bytes of a tile's row
constexpr int kLaneRows = 128;
constexpr int kScaleChunk = 16;    // groups whose scales are fetched together
constexpr int kMaxStages = 8;
constexpr int kMaxSplits = 8;

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages], sum_full[2], sum_empty[2], end;
  uint32_t tbase;
  int abort;
};

template <bool kSwap, int kCols>
struct Shape {
  static constexpr int kSumWarps = kSwap ? 4 : 8;
  static constexpr int kThreads = 32 * (4 + kSumWarps);
  static constexpr int kPerThread = kCols * 4 / kSumWarps;  // sums of a thread
  static constexpr int kStageBytes = (kLaneRows + kCols) * kGroup;
  static constexpr int kScaled = kSwap ? kCols : kLaneRows;  // activation rows of a tile
  static constexpr int kScaleBytes = 2 * kScaleChunk * kScaled * 4;
  static constexpr int kPitch = kSwap ? kLaneRows : kCols + 4;  // of the exchanged sums
  static constexpr int kExchange = (kSwap ? kCols : kLaneRows) * kPitch * 4;
  static constexpr uint32_t kTmemCols = 2 * kCols < 32 ? 32 : 2 * kCols;
};

template <int kCount>
__device__ __forceinline__ void load_sums(uint32_t addr, uint32_t* r) {
  if constexpr (kCount == 32) tmem_ld32(addr, r);
  else tmem_ld16(addr, r);
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t bf16x2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kN consecutive results of row m from column n (a multiple of kN) on.  A
// single one is stored by itself; more as wide as a.vec says the rows are
// aligned (2: to 32 bytes, 1: to 16), one by one at the end of a row.
template <int kN>
__device__ __forceinline__ void store_row(const MatmulArgs& a, int64_t g, int32_t m, int32_t n,
                                          const float* v) {
  static_assert(kN == 1 || kN == 4 || kN % 16 == 0, "whole vectors");
  const int64_t at = g * a.os.batch + int64_t(m) * a.os.rows + n;
  float* of = static_cast<float*>(a.out) + at;
  __nv_bfloat16* oh = static_cast<__nv_bfloat16*>(a.out) + at;
  if constexpr (kN >= 4) {
    if (a.vec && n + kN <= a.N) {
      if (a.out_fp32) {
#pragma unroll
        for (int j = 0; j < kN; j += 4)
          *reinterpret_cast<float4*>(of + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        return;
      }
      if constexpr (kN >= 16) {
        if (a.vec == 2) {  // whole sectors
#pragma unroll
          for (int j = 0; j < kN; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = bf16x2(v[j + 2 * i], v[j + 2 * i + 1]);
            stg256(oh + j, w);
          }
          return;
        }
      }
#pragma unroll
      for (int j = 0; j < kN; j += 4)
        *reinterpret_cast<uint2*>(oh + j) = make_uint2(bf16x2(v[j], v[j + 1]), bf16x2(v[j + 2], v[j + 3]));
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    if (n + j >= a.N) continue;
    if (a.out_fp32) of[j] = v[j];
    else oh[j] = __float2bfloat16_rn(v[j]);
  }
}

// Results of consecutive rows, `stride` apart.  Instructions bound it: with an
// address and the output's type looked at for each result a tile of 64 rows
// took 2.4 us more (128 heads' 64 x 512 x 128 11.8 us instead of 5.7, 64 rows
// through 24576 x 1536 13.4 instead of 10.7).
template <int kN, class T>
__device__ __forceinline__ void store_column(T* o, int64_t stride, int32_t rows, const float* v) {
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    if (j < rows) *o = T(v[j]);
    o += stride;
  }
}

template <bool kSwap, int kCols>
__global__ void __launch_bounds__(Shape<kSwap, kCols>::kThreads, kSwap ? 2 : 1)
    fp8_matmul_kernel(const __grid_constant__ MatmulArgs a) {
  using S = Shape<kSwap, kCols>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Ctl ctl;
  __shared__ __align__(16) float scales[2][kScaleChunk][S::kScaled];
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  volatile int* abort = &ctl.abort;

  // this CTA's tiles and its share of their groups; split tiles are one a CTA
  const uint32_t split = blockIdx.x % uint32_t(a.splits);
  const uint32_t tile0 = blockIdx.x / uint32_t(a.splits), step = gridDim.x / uint32_t(a.splits);
  const int kb0 = int(int64_t(a.k_blocks) * split / a.splits);
  const int kbs = int(int64_t(a.k_blocks) * (split + 1) / a.splits) - kb0;
  struct Place {
    int32_t g, n_tile, m0;
  };
  auto place = [&](uint32_t tile) {
    const uint32_t per_batch = uint32_t(a.m_tiles) * uint32_t(a.n_tiles);
    const uint32_t g = tile / per_batch, in_batch = tile - g * per_batch;
    const uint32_t n_tile = in_batch / uint32_t(a.m_tiles);
    return Place{int32_t(g), int32_t(n_tile),
                 int32_t(in_batch - n_tile * uint32_t(a.m_tiles)) * (kSwap ? kCols : kLaneRows)};
  };

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&a.a_map);
    prefetch_tensormap(&a.b_map);
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.sum_full[i], 1);
      mbar_init(&ctl.sum_empty[i], S::kSumWarps);
    }
    mbar_init(&ctl.end, 1);
    ctl.abort = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 2) {
    tmem_alloc(&ctl.tbase, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = ctl.tbase;
  griddep_launch_dependents();
  griddep_wait();

  float acc[S::kPerThread];
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t sm0 = smem_u32(sm);
      int s = 0;
      uint32_t lap = 0;  // of the stages
      bool ok = true;
      for (uint32_t tile = tile0; ok && tile < a.tiles; tile += step) {
        const Place p = place(tile);
        const int32_t l_row = kSwap ? p.n_tile * 128 : p.m0, c_row = kSwap ? p.m0 : p.n_tile * 128;
        for (int i = 0; i < kbs; ++i) {
          if (lap > 0 && !wait_bounded(&ctl.empty[s], (lap - 1) & 1, abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT)) {
            ok = false;
            break;
          }
          const uint32_t at = sm0 + s * S::kStageBytes;
          mbar_arrive_expect_tx(&ctl.full[s], S::kStageBytes);
          const int32_t x = (kb0 + i) * kGroup;
          tma_load_3d(at, kSwap ? &a.b_map : &a.a_map, x, l_row, p.g, &ctl.full[s]);
          tma_load_3d(at + kLaneRows * kGroup, kSwap ? &a.a_map : &a.b_map, x, c_row, p.g, &ctl.full[s]);
          if (++s == a.stages) {
            s = 0;
            ++lap;
          }
        }
      }
      // the CTA leaves when its loads have landed, whatever became of the rest
      int no_abort = 0;
      for (int j = 0; j < a.stages; ++j) {
        const uint32_t used = lap + (j < s);  // loads of stage j
        if (used > 0)
          wait_bounded(&ctl.full[j], (used - 1) & 1, &no_abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_f16_f32(128, kCols, false, false);
    const bool leader = elect_one();
    uint32_t issued = 0;
    int s = 0;
    uint32_t lap = 0;
    bool ok = true;
    for (uint32_t tile = tile0; ok && tile < a.tiles; tile += step) {
      for (int i = 0; i < kbs; ++i) {
        const int b = issued & 1;
        bool go = wait_bounded(&ctl.full[s], lap & 1, abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
        if (go && issued >= 2)
          go = wait_bounded(&ctl.sum_empty[b], ((issued >> 1) - 1) & 1, abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
        ok = __all_sync(0xffffffffu, go);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t at = smem_u32(sm) + s * S::kStageBytes;
          const uint64_t ad = sdesc_sw128(at, 16, 1024);
          const uint64_t bd = sdesc_sw128(at + kLaneRows * kGroup, 16, 1024);
#pragma unroll
          for (int k = 0; k < kGroup / 32; ++k)
            mma_ss_f8(tb + b * kCols, ad + 2 * k, bd + 2 * k, idesc, k > 0);
          mma_commit(&ctl.empty[s]);
          mma_commit(&ctl.sum_full[b]);
        }
        __syncwarp();
        ++issued;
        if (++s == a.stages) {
          s = 0;
          ++lap;
        }
      }
    }
    // every MMA has completed before tensor memory is given back
    if (issued > 0) {
      if (leader) mma_commit(&ctl.end);
      __syncwarp();
      int no_abort = 0;
      wait_bounded(&ctl.end, 0, &no_abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
    }
  } else if (warp >= 4) {
    const int t = tid - 128;
    const int quad = warp & 3;
    const int half = (warp - 4) >> 2;  // which columns, with eight warps
    const int row = 32 * quad + lane;
    uint64_t sum[S::kPerThread / 2];
    // A chunk's scales sa sb are fetched into registers while the chunk before
    // it (of the tile before, at a tile's begin) is summed.
    constexpr int kSumThreads = 32 * S::kSumWarps;
    constexpr int kFetch = (kScaleChunk * S::kScaled + kSumThreads - 1) / kSumThreads;
    float next[kFetch];
    auto fetch = [&](const Place& p, int i0) {
#pragma unroll
      for (int f = 0; f < kFetch; ++f) {
        const int e = t + kSumThreads * f;
        const int k = i0 + e / S::kScaled;
        const int m = p.m0 + e % S::kScaled;
        next[f] = 0.f;
        if (e < kScaleChunk * S::kScaled && k < kbs && m < a.M)
          next[f] = a.a_scales[p.g * a.ass.batch + m * a.ass.rows + (kb0 + k) * a.ass.cols] *
                    a.b_scales[p.g * a.bss.batch + p.n_tile * a.bss.rows + (kb0 + k) * a.bss.cols];
      }
    };
    if (tile0 < a.tiles) fetch(place(tile0), 0);
    uint32_t done = 0, chunks = 0;  // groups, and chunks of scales, so far
    for (uint32_t tile = tile0; tile < a.tiles; tile += step) {
      const Place p = place(tile);
#pragma unroll
      for (int j = 0; j < S::kPerThread / 2; ++j) sum[j] = 0;
      for (int i = 0; i < kbs; ++i, ++done) {
        if (i % kScaleChunk == 0) {
          // the buffer's last readers are two chunks back, before the barrier of
          // the chunk between
          float* buffer = &scales[chunks & 1][0][0];
#pragma unroll
          for (int f = 0; f < kFetch; ++f) {
            const int e = t + kSumThreads * f;
            if (e < kScaleChunk * S::kScaled) buffer[e] = next[f];
          }
          named_bar_sync(1, kSumThreads);
          ++chunks;
          if (i + kScaleChunk < kbs) fetch(p, i + kScaleChunk);
          else if (tile + step < a.tiles) fetch(place(tile + step), 0);
        }
        const int b = done & 1;
        ok = __all_sync(0xffffffffu, wait_bounded(&ctl.sum_full[b], (done >> 1) & 1, abort, &g_matmul_error,
                                                  SMLA_DEVERR_TIMEOUT));
        // a warp that gives up goes on to the barriers with what it has
        if (ok) {
          tc_fence_after();
          const uint32_t at = tmem_addr(tb, 32 * quad, b * kCols + half * S::kPerThread);
          const float* sc = scales[(chunks - 1) & 1][i % kScaleChunk];
          constexpr int kStep = S::kPerThread < 32 ? S::kPerThread : 32;
#pragma unroll
          for (int c = 0; c < S::kPerThread; c += kStep) {
            uint32_t r[kStep];
            load_sums<kStep>(at + c, r);
            tmem_ld_wait();
            if (c + kStep == S::kPerThread) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ctl.sum_empty[b]);
            }
#pragma unroll
            for (int j = 0; j < kStep / 2; ++j) {
              uint64_t s2;
              if constexpr (kSwap) {
                const float2 f = *reinterpret_cast<const float2*>(sc + c + 2 * j);
                s2 = pack2(f.x, f.y);
              } else {
                s2 = pack2(sc[row], sc[row]);
              }
              sum[c / 2 + j] = fma2(pack2(r[2 * j], r[2 * j + 1]), s2, sum[c / 2 + j]);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < S::kPerThread / 2; ++j) {
        const float2 f = unpack2(sum[j]);
        acc[2 * j] = f.x;
        acc[2 * j + 1] = f.y;
      }
      if (a.splits == 1) {
        if constexpr (kSwap) {
          // a warp stores 32 columns of a row at a time
          const int32_t n = p.n_tile * 128 + row;
          if (n < a.N) {
            const int64_t at = p.g * a.os.batch + p.m0 * a.os.rows + n;
            const int32_t rows = min(a.M - p.m0, kCols);
            if (a.out_fp32) store_column<kCols>(static_cast<float*>(a.out) + at, a.os.rows, rows, acc);
            else store_column<kCols>(static_cast<__nv_bfloat16*>(a.out) + at, a.os.rows, rows, acc);
          }
        } else if (p.m0 + row < a.M) {
          store_row<S::kPerThread>(a, p.g, p.m0 + row, p.n_tile * 128 + half * S::kPerThread, acc);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tb, S::kTmemCols);
  if (a.splits == 1) return;
  const Place p = place(tile0);

  // the cluster's sums, through the operand stages (every load of theirs has
  // been consumed)
  const uint32_t mine = smem_u32(sm);
  if (warp >= 4) {
    const int row = 32 * (warp & 3) + lane;
    const int half = (warp - 4) >> 2;
    float* x = reinterpret_cast<float*>(sm);
    if constexpr (kSwap) {
#pragma unroll
      for (int j = 0; j < kCols; ++j) x[j * S::kPitch + row] = acc[j];
    } else {
#pragma unroll
      for (int j = 0; j < S::kPerThread; j += 4)
        *reinterpret_cast<float4*>(x + row * S::kPitch + half * S::kPerThread + j) =
            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    }
  }
  cluster_sync();
  // four columns of the output a thread, this CTA's share of the tile
  constexpr int kRowsOut = kSwap ? kCols : kLaneRows;   // output rows of the tile
  constexpr int kQuads = (kSwap ? kLaneRows : kCols) / 4;
  for (int e = int(split) * S::kThreads + tid; e < kRowsOut * kQuads; e += a.splits * S::kThreads) {
    const int i = e / kQuads;
    const int c = 4 * (e % kQuads);
    float v[4] = {};
    for (int s = 0; s < a.splits; ++s) {
      const float4 p = ld_cluster_f4(map_to_cta(mine + uint32_t(i * S::kPitch + c) * 4, uint32_t(s)));
      v[0] += p.x;
      v[1] += p.y;
      v[2] += p.z;
      v[3] += p.w;
    }
    if (p.m0 + i < a.M && p.n_tile * 128 + c < a.N) store_row<4>(a, p.g, p.m0 + i, p.n_tile * 128 + c, v);
  }
  cluster_sync();  // nobody's sums go while they are read
}

// Many rows: a CTA pair (cta_group::2) makes 256 x kCols results a tile, each
// CTA 128 of the activation rows, in kCols columns of its tensor memory; each
// holds half of both operands (the pair's MMAs read the other's half of the
// weights), so a byte of shared memory serves twice the products of a 128 x 128
// tile.  Of two accumulators one's group is summed into registers (eight warps,
// half of the columns a thread) while the next group's MMAs fill the other.
// Pairs take tiles in turn, rows first.
//
// What bounds it is the way from L2: with 160, 192, 224 and 256 columns a group
// takes 364, 388, 423 and 434 ns, 11.1 to 11.5 TB/s of operands over all SMs,
// while the MMAs need less (56% of the tensor cores' time with 224).  4001 rows
// through 4096 x 16384: 217 us, 2.5 PFLOP/s.  16 columns are read from tensor
// memory at a time: 32 (and with 256 columns a few spilled registers) took 267 us
// with 256 columns instead of 222 and 227 with 224; a third and fourth
// accumulator (160, 128 columns) nothing less.
struct PairCtl {
  uint64_t full[kMaxStages], peer_full[kMaxStages], empty[kMaxStages], sum_full[2], sum_empty[2], end;
  uint32_t tbase;
  int abort;
};
constexpr int kPairThreads = 384;
constexpr int kPairStages = 6;
// of a CTA: 128 activation rows, half of the tile's columns
template <int kCols> constexpr int kPairStageBytes = (128 + kCols / 2) * kGroup;
template <int kCols> constexpr int kPairSmem = kPairStages * kPairStageBytes<kCols> + 1024;
constexpr int kPairChunk = 8;  // groups whose scales are fetched together
// registers a thread: launched with 168, then shared out by groups of four warps
constexpr int kPairSumRegs = 224, kPairOtherRegs = 56;
static_assert(8 * kPairSumRegs + 4 * kPairOtherRegs <= 12 * 168, "no more than the launch has");

template <int kCols>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    fp8_matmul_pair_kernel(const __grid_constant__ MatmulArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PairCtl ctl;
  // a thread's sums: half of the tile's columns, 16 read at a time; those have
  // one weight scale, the tile's columns up to three
  constexpr int kHalf = kCols / 2, kReads = kHalf / 16, kScales = 4;
  static_assert(kCols % 32 == 0 && kCols <= 256, "halves are whole reads, and a read lies in one block of 128");
  __shared__ float sa[2][kPairChunk][128], sb[2][kPairChunk][kScales];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = int(cluster_ctarank());
  volatile int* abort = &ctl.abort;
  const int kbs = a.k_blocks;
  const uint32_t tile0 = blockIdx.x >> 1, step = gridDim.x >> 1;
  struct Place {
    int32_t g, n0, m0;  // the tile's first column, this CTA's first row
  };
  auto place = [&](uint32_t tile) {
    const uint32_t per_batch = uint32_t(a.m_tiles) * uint32_t(a.n_tiles);
    const uint32_t g = tile / per_batch, in_batch = tile - g * per_batch;
    const uint32_t n_tile = in_batch / uint32_t(a.m_tiles);
    return Place{int32_t(g), int32_t(n_tile) * kCols, int32_t(in_batch - n_tile * uint32_t(a.m_tiles)) * 256 + 128 * C};
  };
  if (tid == 0) {
    prefetch_tensormap(&a.a_map);
    prefetch_tensormap(&a.b_map);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.peer_full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.sum_full[i], 1);
      mbar_init(&ctl.sum_empty[i], 16);  // both CTAs' summing warps
    }
    mbar_init(&ctl.end, 1);
    ctl.abort = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 2) {
    tmem_alloc_pair(&ctl.tbase, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tb = ctl.tbase;
  griddep_launch_dependents();
  griddep_wait();

  if (warp < 4) {
    regs_decrease<kPairOtherRegs>();
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t sm0 = smem_u32(sm);
        int s = 0;
        uint32_t lap = 0;
        bool ok = true;
        for (uint32_t tile = tile0; ok && tile < a.tiles; tile += step) {
          const Place p = place(tile);
          for (int i = 0; i < kbs; ++i) {
            if (lap > 0 &&
                !wait_bounded(&ctl.empty[s], (lap - 1) & 1, abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT)) {
              ok = false;
              break;
            }
            const uint32_t at = sm0 + s * kPairStageBytes<kCols>;
            mbar_arrive_expect_tx(&ctl.full[s], kPairStageBytes<kCols>);
            tma_load_3d(at, &a.a_map, i * kGroup, p.m0, p.g, &ctl.full[s]);
            tma_load_3d(at + 128 * kGroup, &a.b_map, i * kGroup, p.n0 + kHalf * C, p.g, &ctl.full[s]);
            if (++s == kPairStages) {
              s = 0;
              ++lap;
            }
          }
        }
        // the CTA leaves when its loads have landed, whatever became of the rest
        int no_abort = 0;
        for (int j = 0; j < kPairStages; ++j) {
          const uint32_t used = lap + (j < s);
          if (used > 0)
            wait_bounded(&ctl.full[j], (used - 1) & 1, &no_abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      constexpr uint32_t idesc = idesc_f16_f32(256, kCols, false, false);
      const bool leader = elect_one();
      uint32_t issued = 0;
      int s = 0;
      uint32_t lap = 0;
      bool ok = true;
      for (uint32_t tile = tile0; ok && tile < a.tiles; tile += step) {
        for (int i = 0; i < kbs; ++i) {
          ok = wait_bounded(&ctl.full[s], lap & 1, abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
          if (C == 1) {  // tells the first CTA that this one's half has landed
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // (written by TMA, whose completion this warp has waited for)
            if (leader) mbar_arrive_at(map_to_cta(smem_u32(&ctl.peer_full[s]), 0));
            __syncwarp();
          } else {
            const int b = issued & 1;
            ok = ok && wait_bounded(&ctl.peer_full[s], lap & 1, abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT) &&
                 (issued < 2 || wait_bounded(&ctl.sum_empty[b], ((issued >> 1) - 1) & 1, abort, &g_matmul_error,
                                             SMLA_DEVERR_TIMEOUT));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              const uint32_t at = smem_u32(sm) + s * kPairStageBytes<kCols>;
              const uint64_t ad = sdesc_sw128(at, 16, 1024);
              const uint64_t bd = sdesc_sw128(at + 128 * kGroup, 16, 1024);
#pragma unroll
              for (int k = 0; k < kGroup / 32; ++k)
                mma_ss_f8_pair(tb + 256 * b, ad + 2 * k, bd + 2 * k, idesc, k > 0);
              mma_commit_pair(&ctl.empty[s]);
              mma_commit_pair(&ctl.sum_full[b]);
            }
            __syncwarp();
          }
          ++issued;
          if (++s == kPairStages) {
            s = 0;
            ++lap;
          }
        }
      }
      // every MMA has completed before tensor memory is given back
      if (C == 0 && leader) mma_commit_pair(&ctl.end);
      __syncwarp();
      int no_abort = 0;
      wait_bounded(&ctl.end, 0, &no_abort, &g_matmul_error, SMLA_DEVERR_TIMEOUT);
    }
  } else {
    regs_increase<kPairSumRegs>();
    const int t = tid - 128, quad = warp & 3, half = (warp - 4) >> 2;
    const int row = 32 * quad + lane;
    const uint32_t sum_empty = map_to_cta(smem_u32(&ctl.sum_empty[0]), 0);
    uint64_t sum[kHalf / 2];
    float next[kPairChunk / 2], next_b = 0.f;
    auto fetch = [&](const Place& p, int i0) {
      const int m = p.m0 + (t & 127);
#pragma unroll
      for (int f = 0; f < kPairChunk / 2; ++f) {
        const int k = i0 + 2 * f + (t >> 7);
        next[f] = k < kbs && m < a.M ? a.a_scales[p.g * a.ass.batch + m * a.ass.rows + k * a.ass.cols] : 0.f;
      }
      const int k = i0 + t / kScales, n = p.n0 / 128 + t % kScales;
      if (t < kScales * kPairChunk)
        next_b = k < kbs && n * 128 < a.N ? a.b_scales[p.g * a.bss.batch + n * a.bss.rows + k * a.bss.cols] : 0.f;
    };
    if (tile0 < a.tiles) fetch(place(tile0), 0);
    uint32_t done = 0, chunks = 0;
    bool ok = true;
    for (uint32_t tile = tile0; tile < a.tiles; tile += step) {
      const Place p = place(tile);
#pragma unroll
      for (int j = 0; j < kHalf / 2; ++j) sum[j] = 0;
      // the scales of this half's first reads, and of those from `cut` on
      const int first = p.n0 % 128 + kHalf * half, block = first / 128;
      const int cut = kCols == 256 ? kReads : (128 - first % 128) / 16;
      for (int i = 0; i < kbs; ++i, ++done) {
        if (i % kPairChunk == 0) {
          // the buffer's last readers are two chunks back, before the barrier of
          // the chunk between
#pragma unroll
          for (int f = 0; f < kPairChunk / 2; ++f) sa[chunks & 1][2 * f + (t >> 7)][t & 127] = next[f];
          if (t < kScales * kPairChunk) sb[chunks & 1][t / kScales][t % kScales] = next_b;
          named_bar_sync(1, 256);
          ++chunks;
          if (i + kPairChunk < kbs) fetch(p, i + kPairChunk);
          else if (tile + step < a.tiles) fetch(place(tile + step), 0);
        }
        const int b = done & 1;
        ok = __all_sync(0xffffffffu, wait_bounded(&ctl.sum_full[b], (done >> 1) & 1, abort, &g_matmul_error,
                                                  SMLA_DEVERR_TIMEOUT));
        // a warp that gives up goes on to the barriers with what it has
        if (ok) {
          tc_fence_after();
          const float f = sa[(chunks - 1) & 1][i % kPairChunk][row];
          const float* fb = &sb[(chunks - 1) & 1][i % kPairChunk][block];
          const float f0 = f * fb[0], f1 = kCols == 256 ? f0 : f * fb[1];
          const uint64_t s0 = pack2(f0, f0), s1 = pack2(f1, f1);
          const uint32_t at = tmem_addr(tb, 32 * quad, 256 * b + kHalf * half);
          uint32_t r[2][16];
          tmem_ld16(at, r[0]);
#pragma unroll
          for (int c = 0; c < kReads; ++c) {
            tmem_ld_wait();
            if (c + 1 < kReads) tmem_ld16(at + 16 * (c + 1), r[(c + 1) & 1]);
            if (c + 1 == kReads) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_at(sum_empty + 8 * b);  // read: wait::ld, fence
            }
            const uint64_t s2 = c < cut ? s0 : s1;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sum[8 * c + j] = fma2(pack2(r[c & 1][2 * j], r[c & 1][2 * j + 1]), s2, sum[8 * c + j]);
          }
        }
      }
      if (p.m0 + row < a.M) {
#pragma unroll
        for (int c = 0; c < kHalf / 16; ++c) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = unpack2(sum[8 * c + j]);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
          }
          store_row<16>(a, p.g, p.m0 + row, p.n0 + kHalf * half + 16 * c, v);
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // neither CTA reaches into the other any more
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tb, 512);
  __syncwarp();
  cluster_sync();
}

// cuTensorMapEncodeTiled, looked up once through the runtime.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* fn) {
  static std::mutex m;
  static EncodeFn cached = nullptr;
  std::lock_guard<std::mutex> lock(m);
  if (cached == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorNotSupported;
    cached = reinterpret_cast<EncodeFn>(p);
  }
  *fn = cached;
  return cudaSuccess;
}

// Boxes of 128 columns x `box_rows` rows of a batch of code matrices, in the
// 128-byte swizzle; columns and rows past the end read as zeros.
cudaError_t encode_codes(CUtensorMap* map, const uint8_t* p, const Strides& st, int32_t G, int32_t rows,
                         int32_t K, uint32_t box_rows) {
  EncodeFn enc = nullptr;
  const cudaError_t e = encode_fn(&enc);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {cuuint64_t(K), cuuint64_t(rows), cuuint64_t(G)};
  const cuuint64_t strides[2] = {cuuint64_t(st.rows), cuuint64_t(G > 1 ? st.batch : st.rows)};
  const cuuint32_t box[3] = {kGroup, box_rows, 1}, ones[3] = {1, 1, 1};
  if (enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p), dims, strides, box, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

constexpr int kSms = 152;
// Clusters of CTAs, one an SM, that are resident together (as
// cudaOccupancyMaxActiveClusters tells): one more waits for a whole tile of
// another's (100 x 2048 x 2048, 16 tiles: 13.7 us by clusters of eight, of
// which 15 fit, 7.2 by four; 1 x 2112 x 7168, 17 tiles: 10.8 and 7.1).
constexpr int clusters_that_fit(int ctas) { return ctas == 2 ? 76 : ctas == 4 ? 36 : 15; }
// Groups from which a tile's are split (64 x 4096 x 512, 4 groups: 5.6 us by
// clusters of two, 4.2 by one CTA; x 1024, 8 groups: 6.0 and 6.2; 1 x 2048 x 1024
// 3.8 and 4.2).
constexpr int kLeastSplit = 8;

template <bool kSwap, int kCols>
cudaError_t launch(MatmulArgs& a, cudaStream_t s) {
  using S = Shape<kSwap, kCols>;
  constexpr int kMaxSmem = kMaxStages * S::kStageBytes < 180 * 1024 ? kMaxStages * S::kStageBytes : 180 * 1024;
  static_assert(S::kExchange <= kMaxSmem, "the exchanged sums fit");
  // shared-memory limit, once per device
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < 64;
  if (!tracked || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fp8_matmul_kernel<kSwap, kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxSmem + 1024);
    if (e != cudaSuccess) return e;
    if (tracked) done[dev].store(true, std::memory_order_release);
  }
  a.m_tiles = int32_t((int64_t(a.M) + (kSwap ? kCols : kLaneRows) - 1) / (kSwap ? kCols : kLaneRows));
  const int64_t tiles = int64_t(a.G) * a.m_tiles * a.n_tiles;
  a.tiles = uint32_t(tiles);
  // Two CTAs an SM along the columns: one's loads run while the other starts or
  // ends, and each of its groups' way through the tensor core and back (64 x 7168
  // x 7168 in 112 CTAs of 28 groups 18.2 us, in 224 of 14 13.7; 64 x 18432 x 7168
  // 40.5 and 30.8).  Clusters that fit without have all of the shared memory (64 x
  // 4096 x 7168, 32 of four: 11.4 us with 7 stages, 12.6 with 3).
  constexpr int kPerSm = kSwap ? 2 : 1;
  // few tiles: 1 x 576 x 2048 takes 6.4 us by a CTA a tile, 4.0 by clusters; 64 x
  // 576 x 7168 28.6 and 7.7, 128 x 512 x 16384 60.2 and 13.2
  a.splits = 1;
  while (a.splits < kMaxSplits && tiles <= kPerSm * clusters_that_fit(2 * a.splits) && a.k_blocks >= kLeastSplit &&
         a.k_blocks >= 4 * a.splits)
    a.splits *= 2;
  const int per_split = (a.k_blocks + a.splits - 1) / a.splits;
  const bool shared = kSwap && (a.splits == 1 || tiles > clusters_that_fit(a.splits));
  const int most = (shared ? kMaxSmem / 2 : kMaxSmem) / S::kStageBytes;
  const int64_t total = tiles > kSms * 2 ? (tiles + 2 * kSms - 1) / (2 * kSms) * per_split : per_split;
  a.stages = int(total < most ? total : most);
  const int64_t ctas = kSwap && a.splits == 1 && tiles > 2 * kSms ? 2 * kSms : tiles * a.splits;
  size_t smem = size_t(a.stages) * S::kStageBytes;
  if (a.splits > 1 && smem < size_t(S::kExchange)) smem = S::kExchange;
  // As many CTAs on an SM as tensor memory holds and no more: one that waited
  // for another's would hold up its cluster, which may hold up that one.
  constexpr size_t kResident = 512 / S::kTmemCols;
  constexpr size_t kStatic = S::kScaleBytes + sizeof(Ctl);
  const size_t least = size_t(228 * 1024) / (kResident + 1) + 1;
  if (smem + 1024 + kStatic < least) smem = least - 1024 - kStatic;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = smem + 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(a.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fp8_matmul_kernel<kSwap, kCols>, a);
}

template <int kCols>
cudaError_t launch_pairs(MatmulArgs& a, cudaStream_t s) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < 64;
  if (!tracked || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fp8_matmul_pair_kernel<kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPairSmem<kCols>);
    if (e != cudaSuccess) return e;
    if (tracked) done[dev].store(true, std::memory_order_release);
  }
  a.m_tiles = int32_t((int64_t(a.M) + 255) / 256);
  a.n_tiles = int32_t((int64_t(a.N) + kCols - 1) / kCols);
  a.tiles = uint32_t(int64_t(a.G) * a.m_tiles * a.n_tiles);
  a.splits = 1;
  const unsigned pairs = a.tiles < kSms / 2 ? a.tiles : kSms / 2;
  return launch_overlapped(fp8_matmul_pair_kernel<kCols>, 2 * pairs, kPairThreads, kPairSmem<kCols>, s, a);
}

// The pairs' tile width, 0 for a call whose tiles of 128 x 128 are so few that
// clusters share a tile's groups (300 x 2048 x 2048, 48 tiles: 9.5 us so, 9.9 by
// pairs; 130 x 4096 x 7168, 64: 18.8, 23.6; 512 x 2560 x 2048, 80: 10.3, 9.8;
// 1024 x 2048 x 7168, 128: 28.9, 24.2; 512 x 6144 x 7168, 192: 56.8, 25.2).
// Else the one whose rounds of 76 tiles bring the least bytes, 128 + cols / 2
// rows a CTA.  4001 x 4096 x
// 16384 takes 222 us with 256 columns, 217 with 224, 248 with 192 and 280 with
// 160; 4096 x 7168 x 2048 57.5, 62.4, 66.1 and 75.0; 300 x 7168 x 16384 57.6,
// 56.2, 53.1 and 95.3; 2000 x 3000 x 1024 21.1, 19.9, 18.2 and 17.3.
int pair_width(const MatmulArgs& a) {
  if (int64_t(a.G) * ((int64_t(a.M) + 127) / 128) * a.n_tiles <= kSms / 2) return 0;
  int best = 0;
  int64_t least = INT64_MAX;
  for (const int cols : {256, 224, 192, 160}) {
    const int64_t tiles = int64_t(a.G) * ((int64_t(a.M) + 255) / 256) * ((int64_t(a.N) + cols - 1) / cols);
    const int64_t time = (tiles + kSms / 2 - 1) / (kSms / 2) * (256 + cols);
    if (time < least) {
      least = time;
      best = cols;
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_fp8_matmul(const MatmulArgs& args, cudaStream_t s) {
  MatmulArgs a = args;
  a.k_blocks = int32_t((int64_t(a.K) + kGroup - 1) / kGroup);
  a.n_tiles = int32_t((int64_t(a.N) + 127) / 128);
  // 16 rows through 24576 x 1536 take 6.4 us with tiles of 16 columns, 11.6 with
  // 64 and 16.3 along the lanes; 32 rows 7.1, 9.6 and 15.6; 64 rows 10.0 and 16.5
  const int cols = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  cudaError_t e = encode_codes(&a.a_map, a.a, a.as, a.G, a.M, a.K, uint32_t(cols));
  const int width = a.M > 128 ? pair_width(a) : 0;
  if (e == cudaSuccess) e = encode_codes(&a.b_map, a.b, a.bs, a.G, a.N, a.K, width ? width / 2 : 128);
  if (e != cudaSuccess) return e;
  const uint64_t bytes = a.out_fp32 ? 4 : 2;
  const uint64_t ends = reinterpret_cast<uintptr_t>(a.out) | (uint64_t(a.os.rows) * bytes) |
                        (a.G > 1 ? uint64_t(a.os.batch) * bytes : 0);
  a.vec = ends % 32 == 0 ? 2 : ends % 16 == 0 ? 1 : 0;
  switch (cols) {
    case 16: return launch<true, 16>(a, s);
    case 32: return launch<true, 32>(a, s);
    case 64: return launch<true, 64>(a, s);
    default: break;
  }
  switch (width) {
    case 160: return launch_pairs<160>(a, s);
    case 192: return launch_pairs<192>(a, s);
    case 224: return launch_pairs<224>(a, s);
    case 256: return launch_pairs<256>(a, s);
    default: return launch<false, 128>(a, s);
  }
}

cudaError_t matmul_error_word(uint32_t* flags, bool clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_matmul_error, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags |= v;
  if (clear) {
    v = 0;
    e = cudaMemcpyToSymbol(g_matmul_error, &v, sizeof(v));
  }
  return e;
}

}  // namespace smla
