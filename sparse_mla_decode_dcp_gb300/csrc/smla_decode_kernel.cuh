// Sparse, dense and windowed MLA decode over the packed latent cache (8- or
// 4-bit rows) on tcgen05 tensor cores.
//
// What it computes ("FlashMLA sparse fp8 path + DCP + MTP", implementation
// breakdown steps 1 and 3; "[eldritch] attention: support DCP in SM120
// FlashInfer sparse MLA", Why): for query row t and head h, over the valid
// local slots j of row t,
//     s_j = sm_scale * <q[t,h,0:576], (latent_j || rope_j)>
//     lse = ln sum_j exp(s_j),   out = sum_j exp(s_j - lse) * latent_j
// with latent_j = e4m3(code) * scale[dim / 128] (fp8 rows) or e2m1(code) *
// e4m3 scale[dim / 16] (fp4 rows).  A row with no valid slot is written as
// the merge identity (out = 0, lse = -inf).
//
// Design (GB300, one cluster of two CTAs per query row):
//   * Heads are the MMA M dimension (M = 128, heads padded with zero rows),
//     so the 576-wide latent keys are shared by all heads (MQA-style).
//   * The fp32 accumulator O[128 x 512] alone fills a whole SM's tensor
//     memory, so CTA c of the pair owns value dims [256c, 256c + 256).  The
//     QK^T contraction is split by key dimension the same way: CTA c
//     contracts latent dims [256c, 256c + 256) (its value half) and rope dims
//     [32c, 32c + 32), 288 key dims each, so every cache byte is fetched by
//     one CTA.  The fp32 partial scores are exchanged through distributed
//     shared memory each tile: each CTA finishes half of the tile's keys and
//     sends the other its P of them, so no FLOP and no exponential is
//     computed twice.
//   * Q (this CTA's key-dim half) and P live in tensor memory as the A
//     operand; K/V tiles are the B operand in shared memory (128-byte
//     swizzle): one buffer serves as K (K-major) for QK^T and as V
//     (MN-major) for PV.
//   * Keys are dequantised to fp16 with a single rounding: the e4m3 code is
//     exact in fp16 and the fp32 scale is split into fp16 hi + lo parts, so
//     code*hi + code*lo is rounded once by a fused multiply-add.  fp16 keeps
//     3 more mantissa bits than bf16, which keeps score errors well inside
//     the LSE tolerance even for rows with a single valid slot.  An fp4
//     row's code x scale has at most 6 significant bits and lies in [2^-10,
//     2688] (or is 0), so its keys are exact in fp16.
//   * Valid slots are compacted in order in the prologue (-1 never costs a
//     load or an MMA).  Loader threads hold a tile's fp8 rows in registers
//     while the tile before it is read out of a raw stage in shared memory;
//     fp4 rows are converted from registers, loaded a tile ahead.  Four operand
//     tiles are in flight.
//   * The partial score tiles travel as asynchronous remote stores counted on
//     the receiving CTA's mbarrier (st.async + expect_tx).
//   * Softmax in the log2 domain with a lazily moved reference maximum: the
//     O accumulator in TMEM is rescaled only when the row maximum grows by
//     more than 2^8.
//
// Warp roles: 4 (fp8 rows) or 8 (fp4) warps of softmax and epilogue (TMEM
// lanes 0-127, one or two threads a head row), 4 that dequantise, one that
// allocates TMEM and issues every MMA (one elected lane: QK^T of a tile, then
// PV of the tile two before it, once the softmax has stored that tile's P)
// and 3 that load cache rows (fp8) or, two of them, convert rope values (fp4).
// Every wait is bounded; a wait that runs out sets SMLA_DEVERR_TIMEOUT and
// the CTA unwinds.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <atomic>
#include <mutex>

#include "../../include/smla.h"
#include "smla_internal.h"
#include "smla_sm100.cuh"

namespace smla {
namespace {

using namespace sm100;

__device__ unsigned int g_decode_error;

// What a row's raw entries are: local slots of one pool (per-shard decode),
// global top-k positions over D pools (fused DCP step), the positions of the
// row's whole causal context (dense decode), or of its first positions and
// the window that ends at it (windowed decode).
enum : int { kModeSlots = 0, kModeTopk = 1, kModeDense = 2, kModeWindow = 3 };
constexpr bool generated(int mode) { return mode == kModeDense || mode == kModeWindow; }

constexpr int kTileN = 64;        // keys per tile (MMA N of QK^T, K of PV)
constexpr int kStages = 4;        // fp16 operand tiles in flight
constexpr int kRawStages = 1;     // raw cache-row tiles in shared memory (one more in registers)
constexpr int kLoaders = 96;
constexpr int kMaxList = kDecodeMaxList;  // compacted slots one cluster handles
// a windowed row's entries need no compaction: what shared memory holds
constexpr int kWindowList = 2096;

// tensor-memory columns (512 allocated)
constexpr uint32_t kOCol = 0;     // O half: 256 fp32 columns
constexpr uint32_t kSCol = 256;   // S tile: 64 fp32 columns
constexpr uint32_t kPCol = 320;   // P tile: 64 fp16 = 32 columns
constexpr uint32_t kQCol = 352;   // Q part: 288 fp16 = 144 columns
constexpr uint32_t kRefCol = 496; // references of a row's two threads, 2 buffers
constexpr uint32_t kTmemCols = 512;

// N consecutive columns of a warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t addr, uint32_t* r) {
  if constexpr (N == 32) tmem_ld32(addr, r);
  else tmem_ld16(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t addr, const uint32_t* r) {
  if constexpr (N == 16) tmem_st16(addr, r);
  else tmem_st8(addr, r);
}

// shared-memory layout (offsets from a 1024-byte aligned base)
constexpr int kKBlockBytes = kTileN * 128;          // 64 keys x 64 fp16, 128-byte swizzle
constexpr int kRopeBlock = 4 * kKBlockBytes;        // 64 keys x 32 fp16, 64-byte swizzle
constexpr int kOpTileBytes = kRopeBlock + kTileN * 64;  // 256 latent + 32 rope dims
constexpr int kRawTileBytes = kTileN * 336;  // one tile of staged fp8 rows
// Per tile and direction the pair exchanges the fp32 partial scores of half
// the tile's keys (XA) and then the fp16 P of the other half plus each row's
// reference maximum and partial sum (XB).
constexpr int kXABytes = 128 * (kTileN / 2) * 4;
constexpr int kXBPBytes = 128 * (kTileN / 2) * 2;
constexpr int kXBBytes = kXBPBytes + 128 * 8;
constexpr int kXBytes = kXABytes + kXBBytes;         // one buffer set
constexpr int kOffOp = 0;
constexpr int kOffRaw = kOffOp + kStages * kOpTileBytes;
// fp4 rows have no raw stage: the list of their addresses takes its place
constexpr int kOffRows = kOffRaw;
static_assert(kWindowList * 8 <= kRawStages * kRawTileBytes && kMaxList <= kWindowList, "row addresses fit");
constexpr int kOffX = kOffRaw + kRawStages * kRawTileBytes;
constexpr int kOffList = kOffX + 2 * kXBytes;  // two buffer sets
constexpr int kBtStageMax = 2 * kXBytes / 4;    // staged block-table entries (fused prologue)
constexpr int kOffListShard = kOffList + kWindowList * 4;  // fused step: shard of each key
constexpr int kOffCtl = kOffListShard + kWindowList;
constexpr int kCtlBytes = 784;
constexpr int kSmemBytes = kOffCtl + kCtlBytes + 1024;  // + control block + alignment slack

// Per shard: its staged block-table row's offset in the staging area, the
// row's meaningful columns and the pool's slot count (one 16-byte read).
struct __align__(16) ShardMeta {
  int32_t bt_off, bt_width;
  int64_t pool_slots;
};

struct Ctl {
  uint64_t q_tma, q_ready, full[kStages], freed[kStages], raw_full[kRawStages], raw_empty[kRawStages],
      s_full, s_free, pv_done, p_full, xa[2], xb[2], sums, end;
  uint32_t tbase;
  int n_list;
  int abort;
  int is_last;
  int warp_cnt[8];  // the compacting warps' valid counts
  // fused step: per shard, its pool and this row's request row of its table
  const uint8_t* pool[kMaxMerge];
  const int32_t* bt_row[kMaxMerge];
  ShardMeta meta[kMaxMerge];
  int bt_staged;              // the rows fit the staging area
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Wait sites, recorded in bits 8.. of the device error word when a wait
// gives up (diagnostic).
enum WaitSite : uint32_t {
  kWsSFull = 0, kWsExchange, kWsPvDone, kWsPvLast, kWsFreed, kWsQReady, kWsFull, kWsSFree,
  kWsPFull, kWsDrain, kWsRaw, kWsRawEmpty, kWsExchangeP
};

// Every wait is bounded in time (kWaitNs of the global timer); a wait that
// gives up records TIMEOUT plus its site and raises the CTA's abort flag so
// the other roles stop waiting too.
constexpr uint64_t kWaitNs = 2000000000ull;

template <bool kCluster>
__device__ __forceinline__ bool probe_phase(uint64_t* bar, uint32_t parity) {
  return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}

template <bool kCluster>
__device__ __forceinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            uint32_t site) {
  const uint64_t t0 = globaltimer_ns();
  uint32_t it = 0;
  while (!probe_phase<kCluster>(bar, parity)) {
    if (*abort) return false;
    if ((++it & 63u) == 0 && globaltimer_ns() - t0 > kWaitNs) {
      atomicOr(&g_decode_error, SMLA_DEVERR_TIMEOUT | (1u << (8 + site)));
      *abort = 1;
      return false;
    }
  }
  return true;
}

#ifdef SMLA_WAITS_OUT_OF_LINE
// The waiting itself as one function, where the including file asks for it:
// the code of sixteen warps in five roles is smaller by its copies.  Measured
// both ways: 4-bit decodes 2-3% sooner (four pools 52.2 -> 51.2 us, one rank
// 29.8 -> 29.0), windows 0.4-1.6%; but dense decode 635 -> 647 us, the 8-bit
// fused step (inputs in L2) 61.7 -> 61.8, so those keep the copies.
template <bool kCluster>
__noinline__ __device__ bool wait_longer_called(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                uint32_t site) {
  return wait_longer<kCluster>(bar, parity, abort, site);
}
#endif

template <bool kCluster>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           uint32_t site) {
  if (probe_phase<kCluster>(bar, parity)) return true;
#ifdef SMLA_WAITS_OUT_OF_LINE
  return wait_longer_called<kCluster>(bar, parity, abort, site);
#else
  return wait_longer<kCluster>(bar, parity, abort, site);
#endif
}

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint32_t site) {
  return wait_phase<false>(bar, parity, abort, site);
}

__device__ __forceinline__ bool wait_bar_cluster(uint64_t* bar, uint32_t parity,
                                                 volatile int* abort, uint32_t site) {
  return wait_phase<true>(bar, parity, abort, site);
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Nonzero when a bf16 of the pair in `w` would not fit fp16 (|x| >= 65536:
// bf16 has no value between 65280 and 65536, and fp16's largest is 65504;
// inf and NaN included): each 15-bit magnitude plus 0x3880 reaches bit 15
// exactly when it is >= 0x4780, with no carry between the halves.
__device__ __forceinline__ uint32_t bf16x2_over_fp16(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + 0x38803880u) & 0x80008000u;
}

__device__ __forceinline__ uint32_t bf16x8_over_fp16(const uint4& v) {
  return bf16x2_over_fp16(v.x) | bf16x2_over_fp16(v.y) | bf16x2_over_fp16(v.z) |
         bf16x2_over_fp16(v.w);
}

// A latent group scale the fp16 keys cannot carry: its dequantised values
// (up to 448 x scale) overflow fp16, or a nonzero scale so small that
// 2^8 x scale is an fp16 subnormal (the keys lose precision); NaN included.
__device__ __forceinline__ bool scale_out_of_range(float s) {
  return !(s <= 65504.f / 448.f) || (s != 0.f && s < 0x1p-22f);
}

// 8 bf16 -> 8 fp16 (exact in fp16's normal range)
__device__ __forceinline__ uint4 bf16x8_to_f16x8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = h2_bits(
        __floats2half2_rn(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Two e4m3 codes (bytes `sel` picks) -> fp16x2 holding code * 2^-8, exactly,
// on the integer pipe: the sign moves to fp16's sign bit and the 7 exponent /
// mantissa bits drop in one position lower (4-bit exponent under fp16's
// 5-bit field, bias 7 vs 15), which makes normal and subnormal codes alike
// land on code * 2^-8.  (e4m3 NaN codes, which no quantiser emits, are not
// special-cased.)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_scaled_down(uint32_t w, uint32_t sel) {
  const uint32_t y = __byte_perm(w, 0u, sel);  // code a in bits 15:8, code b in 31:24
  return (y & 0x80008000u) | ((y & 0x7F007F00u) >> 1);
}

// 8 e4m3 codes -> 8 fp16 values code * scale with one rounding: hi + lo is
// the fp32 scale * 2^8 split into two fp16 parts, and fma(c, hi, c * lo)
// rounds once.
__device__ __forceinline__ uint4 e4m3x8_scaled(uint2 codes, __half2 hi, __half2 lo) {
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t bits = e4m3x2_to_f16x2_scaled_down(w[k], p == 0 ? 0x1404u : 0x3424u);
      const __half2 c = *reinterpret_cast<const __half2*>(&bits);
      o[2 * k + p] = h2_bits(__hfma2(c, hi, __hmul2(c, lo)));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 2^x; results below 2^-126 flush to zero (a softmax weight that small is
// zero in the fp16 P tile anyway)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The two CTAs of a pair split the work by key dimension, symmetrically:
// CTA c gathers and contracts latent dims [256c, 256c + 256) (the value dims
// of its O half) and rope dims [32c, 32c + 32), 288 key dims each, laid out
// in its operand tile as dims 0..255 (latent) and 256..287 (rope).  Every
// cache byte is fetched by one CTA (the 16 bytes of scales by both).  All of
// it is runtime data of the CTA's rank, so the two CTAs share one
// instruction stream (half the code, for the instruction cache).
constexpr int kQkDims = 288;
constexpr int kKSteps = kQkDims / 16;  // MMA K = 16

// Softmax warps with a head row to work on: a warp whose 32 rows are all
// padding computes, exchanges and stores nothing (its rows of S, P and O hold
// arbitrary values that no other row sees).
__device__ __forceinline__ int softmax_warps(int H) { return (H + 31) >> 5; }

struct HalfRt {
  int c;  // CTA rank in the pair
};

__device__ __forceinline__ HalfRt half_of(uint32_t c) {
  HalfRt r;
  r.c = int(c);
  return r;
}

// A cache row's format.
struct Fp8Rows {
  static constexpr bool kFp4 = false;
  static constexpr int kRowThreads = 1;
  static constexpr int kRowBytes = SMLA_ROW_BYTES;
  // CTA c stages the bytes of its half of a row, at kRawStride per row, in
  // kPieces pieces of 16 bytes.
  // pieces 0..15: codes [256c, 256c + 256) -> raw [0, 256); piece 16: the
  // four fp32 scales [512, 528) -> raw [256, 272); pieces 17..20: rope bf16
  // [528 + 64c, 592 + 64c) -> raw [272, 336)
  static constexpr int kPieces = 21;
  static constexpr int kRawStride = 336;
  static constexpr int kRawScales = 256;
  static constexpr int kRawRope = 272;
  static constexpr int kCodes = 8;  // 16-byte code pieces of one converter thread (its 128 dims)
  static __device__ __forceinline__ int piece_src(int c, int j) {
    return j < 16 ? 256 * c + 16 * j : j == 16 ? 512 : 528 + 64 * c + 16 * (j - 17);
  }
};

// CTA c's half of a 4-bit row: codes [128c, 128c + 128), sixteen e4m3 scales
// [256 + 16c, 272 + 16c), rope bf16 [288 + 64c, 352 + 64c).
struct Fp4Rows {
  static constexpr bool kFp4 = true;
  static constexpr int kRowThreads = 2;
  static constexpr int kRowBytes = SMLA_FP4_ROW_BYTES;
};

// The warps of a CTA: 4 or 8 softmax warps (kRowThreads threads a head row,
// each finishing kCols of a tile's key columns), 4 converter warps, the MMA
// warp, 3 warps that load fp8 rows or, two of them, convert fp4 rows' rope
// values.  Two threads a row shorten the softmax's chain, which
// bounds the fp4 kernels (sparse step of 4 pools, 64 rows of 2048 entries,
// H = 128: 58.2 -> 54.3 us; 2 rows of 64 9.5 -> 8.4), but leave the loaders 128
// instead of 168 registers, and fp8's rows, half again as long, then arrive
// late (fused step, inputs in L2, 62.8 -> 66.9 us, dense decode 649 -> 690): one
// thread there.
template <class F>
struct Roles {
  static constexpr int kSoftmaxWarps = 4 * F::kRowThreads;
  static constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
  static constexpr int kConvWarp0 = kSoftmaxWarps;
  static constexpr int kMmaWarp = kConvWarp0 + 4;
  static constexpr int kLoaderWarp0 = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kLoaderWarp0 + 3);
  static constexpr int kCols = kTileN / 2 / F::kRowThreads;
};

// fp8 rows: converter thread (key, part) of CTA c converts its key's code
// pieces [8 part, 8 part + 8) (tile dims 128 part .. 128 part + 127: scale
// group 2c + part) and rope pieces 2 part, 2 part + 1 (tile dims 256 + 16 part
// .. 256 + 16 part + 15).
constexpr int kRopePerPart = 2;

// Cache row of entry `idx` of the compacted list (fp8 rows).
template <int kMode>
__device__ __forceinline__ const uint8_t* row_ptr(const DecodeArgs& a, const Ctl* ctl,
                                                  const int* list, const uint8_t* shard,
                                                  int idx) {
  const uint8_t* pool = kMode != kModeSlots ? ctl->pool[shard[idx]] : a.kv;
  return pool + int64_t(list[idx]) * Fp8Rows::kRowBytes;
}

__device__ __forceinline__ void split_scale(float s, __half2& hi, __half2& lo) {
  const float x = 256.f * s;  // the integer code decode leaves a factor 2^-8 out
  const __half h = __float2half_rn(x);
  hi = __half2half2(h);
  lo = __half2half2(__float2half_rn(x - __half2float(h)));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
               :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Operand tile address of 8 consecutive dims from tile dim `ldim` of `key`:
// dims 0..255 in four 128-byte-swizzled K-blocks, dims 256..287 (rope) in
// one 64-byte-swizzled block.
__device__ __forceinline__ uint32_t op_addr(uint32_t op, int key, int ldim) {
  return ldim < 256 ? op + (ldim >> 6) * kKBlockBytes + sw128_offset(key, (ldim & 63) >> 3)
                    : op + kRopeBlock + sw64_offset(key, (ldim - 256) >> 3);
}

// 8 e2m1 codes (one 32-bit word, dim i in nibble i) times their group's scale,
// exact in fp16: at most 6 significant bits, 2^-10 to 2688.  The conversion
// instruction keeps a tile's dims in their order; shifts and masks would leave
// them in another, for no clear gain (2 rows of 64 entries 6.8 against 6.5 us, 64
// rows of 2048 52.8 against 53.6).
__device__ __forceinline__ uint4 e2m1x8_scaled(uint32_t w, __half2 scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h =
        __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t((w >> (8 * i)) & 0xffu), __NV_E2M1);
    o[i] = h2_bits(__hmul2(__half2(h), scale));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One converter thread's staged pieces of its key: its code pieces, 2 rope
// pieces and the scale of its codes' group.
struct ConvRegs {
  uint4 cur[Fp8Rows::kCodes + kRopePerPart];
  float scale;
};

// Read this thread's staged pieces of its key (`row` = the key's staged row;
// zeros for a key past the row's valid count).  Lanes read rows kRawStride
// apart, an odd number of 16-byte units: 8 consecutive keys hit 8 different
// bank groups.
__device__ __forceinline__ void read_row(uint32_t row, bool live, int c, int part, ConvRegs& r) {
  using F = Fp8Rows;
  const uint32_t code0 = row + 16 * F::kCodes * part;
  const uint32_t rope0 = row + F::kRawRope + 32 * part;
#pragma unroll
  for (int k = 0; k < F::kCodes; ++k)
    r.cur[k] = live ? lds128(code0 + 16 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int q = 0; q < kRopePerPart; ++q)
    r.cur[F::kCodes + q] = live ? lds128(rope0 + 16 * q) : make_uint4(0, 0, 0, 0);
  // the one scale group of this thread's codes
  r.scale = live ? ld_shared_f32(row + F::kRawScales + 4 * (2 * c + part)) : 0.f;
}

// Convert the read pieces into the swizzled fp16 operand tile at `op` (the
// same code path for both CTA ranks and parts).
// Returns true when the key's scale or rope values do not fit the fp16 keys.
__device__ __forceinline__ bool convert_row(const ConvRegs& r, uint32_t op, int key, int part) {
  using F = Fp8Rows;
  __half2 hi, lo;
  split_scale(r.scale, hi, lo);
#pragma unroll
  for (int k = 0; k < F::kCodes; ++k) {
    const int ldim = 128 * part + 16 * k;
    sts128(op_addr(op, key, ldim), e4m3x8_scaled(make_uint2(r.cur[k].x, r.cur[k].y), hi, lo));
    sts128(op_addr(op, key, ldim + 8), e4m3x8_scaled(make_uint2(r.cur[k].z, r.cur[k].w), hi, lo));
  }
  uint32_t over = 0;
#pragma unroll
  for (int q = 0; q < kRopePerPart; ++q) {
    over |= bf16x8_over_fp16(r.cur[F::kCodes + q]);
    sts128(op_addr(op, key, 256 + 16 * part + 8 * q), bf16x8_to_f16x8(r.cur[F::kCodes + q]));
  }
  return over != 0 || scale_out_of_range(r.scale);
}

// The loader warps' loop (fp8 rows).  Loader ld owns pieces ld + 96k of every
// tile (64 rows x 21 pieces = 14 x 96), so consecutive lanes read consecutive
// 16 bytes of a row (whole sectors, few transactions).  A tile's pieces are
// loaded into registers while the raw stage holds the tile before it, and
// stored once the converter warps have read that tile out of the stage.
// Load-issue stalls (the memory system's request slots) fall on these warps,
// not on the converters.
static_assert(kTileN * Fp8Rows::kRawStride <= (1 << 15) && Fp8Rows::kRowBytes <= (1 << 10) &&
                  kTileN <= (1 << 7),
              "packed piece offsets fit their fields");

// Each piece's place is the same in every tile: its row r in the tile, its
// source offset in the cache row and its destination offset in the raw
// stage, packed once as r << 25 | src << 15 | dst (dst < 2^15, src < 2^10).
// A loader forms its pieces' places before the set-up barrier, while other
// warps' first loads are on the way.
struct Pieces {
  static constexpr int kPer = kTileN * Fp8Rows::kPieces / kLoaders;
  static_assert(kPer * kLoaders == kTileN * Fp8Rows::kPieces, "a tile's pieces fill the rounds");
  uint32_t pk[kPer];
  __device__ __forceinline__ void place(int c, int ld) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int p = ld + kLoaders * k;
      const int r = int((uint32_t(p) * 3121u) >> 16);  // p / 21, exact for p < 64 * 21
      const int j = p - r * Fp8Rows::kPieces;
      pk[k] = uint32_t(r) << 25 | uint32_t(Fp8Rows::piece_src(c, j)) << 15 |
              uint32_t(r * Fp8Rows::kRawStride + 16 * j);
    }
  }
};

template <int kMode>
__device__ void loader_loop(const DecodeArgs& a, Ctl* ctl, uint8_t* sm, int n, int ntiles,
                            const Pieces& pieces, volatile int* abort) {
  const int* list = reinterpret_cast<const int*>(sm + kOffList);
  const uint8_t* list_shard = sm + kOffListShard;
  const uint32_t raw0 = smem_u32(sm + kOffRaw);
  constexpr int kPiecesPerLoader = Pieces::kPer;
  const uint32_t (&pk)[kPiecesPerLoader] = pieces.pk;
  uint4 buf[kPiecesPerLoader];
  auto load = [&](int tile) {
    const int base = tile * kTileN;
    const uint32_t rows = uint32_t(min(kTileN, n - base));
#pragma unroll
    for (int k = 0; k < kPiecesPerLoader; ++k) {
      const uint32_t r = pk[k] >> 25;
      if (r < rows) {
        const uint8_t* row = row_ptr<kMode>(a, ctl, list, list_shard, base + int(r));
        buf[k] = ldg_stream(row + ((pk[k] >> 15) & 1023u));
      }
    }
  };
  auto store = [&](int tile, uint32_t stage) {
    const uint32_t rows = uint32_t(min(kTileN, n - tile * kTileN));
#pragma unroll
    for (int k = 0; k < kPiecesPerLoader; ++k)
      if ((pk[k] >> 25) < rows) sts128(stage + (pk[k] & 0x7fffu), buf[k]);
  };
  if (ntiles > 0) load(0);
#pragma unroll 1
  for (int t = 0; t < ntiles; ++t) {
    const int st = t % kRawStages;
    if (t >= kRawStages &&
        !wait_bar(&ctl->raw_empty[st], ((t - kRawStages) / kRawStages) & 1, abort, kWsRawEmpty))
      break;
    store(t, raw0 + st * kRawTileBytes);
    mbar_arrive(&ctl->raw_full[st]);
    if (t + 1 < ntiles) load(t + 1);
  }
}

// The converter threads' tile loop (fp8 rows): each staged tile is converted into the
// fp16 operand stage once the MMAs of the tile two back have released it,
// then handed back to the loaders (one arrival per warp).
__device__ void convert_loop(Ctl* ctl, uint8_t* sm, int n, int ntiles, int key, int c, int part,
                             int lane, volatile int* abort) {
  const uint32_t raw0 = smem_u32(sm + kOffRaw);
  const uint32_t op0 = smem_u32(sm + kOffOp);
  bool out_of_range = false;
#pragma unroll 1
  for (int i = 0; i < ntiles; ++i) {
    const int st = i % kRawStages;
    if (!wait_bar(&ctl->raw_full[st], (i / kRawStages) & 1, abort, kWsRaw)) break;
    ConvRegs r;
    read_row(raw0 + st * kRawTileBytes + key * Fp8Rows::kRawStride, key < n - i * kTileN, c, part, r);
    // the raw stage goes back to the loaders as soon as the warp has read it
    // (the warp barrier orders the lanes' reads before lane 0's release), so
    // they refill it while this tile is converted
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->raw_empty[st]);
    // q was staged in the operand stages
    if (i == 0 && !wait_bar(&ctl->q_ready, 0, abort, kWsQReady)) break;
    if (i >= kStages &&
        !wait_bar(&ctl->freed[i % kStages], ((i - kStages) / kStages) & 1, abort, kWsFreed))
      break;
    out_of_range |= convert_row(r, op0 + (i % kStages) * kOpTileBytes, key, part) &&
                    key < n - i * kTileN;
    fence_async_shared();
    mbar_arrive(&ctl->full[i % kStages]);
  }
  if (out_of_range) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
}

// fp4 rows go straight from global memory into registers and from there into
// the operand stages: a half row is 13 pieces of 16 bytes, few enough for the
// converters to hold a tile of them ahead, and the trip through a raw stage
// (208 of some 1100 wavefronts of shared memory a tile) is saved.  The converter warps take
// the codes, warp w keys [16 w, 16 w + 16) of a tile: eight lanes read the 128
// bytes of a key's codes (lane j piece j: dims 32 j .. of the CTA's half, two
// scale groups), so that a load instruction reads whole lines.  Two more warps
// take the rope values, four lanes a key.  Against loader warps and a raw
// stage: 2 rows of 64 entries 7.6 -> 6.5 us, one pool's 32 rows of 2048 (two
// splits) 32.0 -> 29.9, four pools' 64 rows 55.1 -> 53.6, windows of 1088
// entries 66.2 -> 63.0.  The list holds the rows' addresses (formed from slot
// and shard at each load: four pools 60.8 us), and each tile's are read a tile
// early.
constexpr int kRopeThreads = 64;

struct Fp4Regs {
  uint4 code[4];
  uint32_t scale[4];
};

__device__ void convert_codes(Ctl* ctl, uint8_t* sm, int n, int ntiles, int c, int d,
                              volatile int* abort) {
  const uint8_t* const* rows = reinterpret_cast<const uint8_t* const*>(sm + kOffRows);
  const uint32_t op0 = smem_u32(sm + kOffOp);
  const int lane = d & 31;
  const int j = lane & 7;
  const int key0 = (d >> 5) * 16 + (lane >> 3);  // this lane's keys: key0 + 4 i
  const uint8_t* row[4];
  auto place = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = tile * kTileN + key0 + 4 * i;
      row[i] = idx < n ? rows[idx] : nullptr;
    }
  };
  auto load = [&](int tile, Fp4Regs& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.code[i] = row[i] ? ldg_stream(row[i] + 128 * c + 16 * j) : make_uint4(0, 0, 0, 0);
      r.scale[i] = row[i] ? reinterpret_cast<const uint16_t*>(row[i] + 256 + 16 * c)[j] : 0;
    }
    place(tile + 1);
  };
  // Lane j stores its four 16-byte chunks from chunk j / 2 on, so that a key's
  // eight lanes (two to each of four K-blocks) hit eight bank groups at a time.
  const int rot = j >> 1;
  Fp4Regs cur, next;
  place(0);
  if (ntiles > 0) load(0, cur);
  bool nan = false;
#pragma unroll 1
  for (int i = 0; i < ntiles; ++i) {
    if (i + 1 < ntiles) load(i + 1, next);
    // q was staged in the operand stages
    if (i == 0 && !wait_bar(&ctl->q_ready, 0, abort, kWsQReady)) break;
    if (i >= kStages &&
        !wait_bar(&ctl->freed[i % kStages], ((i - kStages) / kStages) & 1, abort, kWsFreed))
      break;
    const uint32_t blk = op0 + (i % kStages) * kOpTileBytes + (j >> 1) * kKBlockBytes;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 ss =
          __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(cur.scale[k]), __NV_E4M3));
      const uint32_t sb = h2_bits(ss);
      nan |= (sb & 0x7fffu) > 0x7c00u || (sb & 0x7fff0000u) > 0x7c000000u;
      const __half2 s0 = __low2half2(ss), s1 = __high2half2(ss);
      uint4 v = cur.code[k];
      if (rot & 1) v = make_uint4(v.y, v.z, v.w, v.x);
      if (rot & 2) v = make_uint4(v.z, v.w, v.x, v.y);
      const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int chunk = (m + rot) & 3;
        sts128(blk + sw128_offset(key0 + 4 * k, 4 * (j & 1) + chunk),
               e2m1x8_scaled(word[m], chunk < 2 ? s0 : s1));
      }
    }
    fence_async_shared();
    mbar_arrive(&ctl->full[i % kStages]);
    cur = next;
  }
  if (nan) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
}

__device__ void convert_rope(Ctl* ctl, uint8_t* sm, int n, int ntiles, int c, int d,
                             volatile int* abort) {
  const uint8_t* const* rows = reinterpret_cast<const uint8_t* const*>(sm + kOffRows);
  const uint32_t op0 = smem_u32(sm + kOffOp) + kRopeBlock;
  uint4 cur[4], next[4];
  auto load = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = tile * kTileN + 16 * i + (d >> 2);
      next[i] = idx < n ? ldg_stream(rows[idx] + 288 + 64 * c + 16 * (d & 3)) : make_uint4(0, 0, 0, 0);
    }
  };
  if (ntiles > 0) load(0);
  uint32_t over = 0;
#pragma unroll 1
  for (int i = 0; i < ntiles; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) cur[k] = next[k];
    if (i + 1 < ntiles) load(i + 1);
    if (i == 0 && !wait_bar(&ctl->q_ready, 0, abort, kWsQReady)) break;
    if (i >= kStages &&
        !wait_bar(&ctl->freed[i % kStages], ((i - kStages) / kStages) & 1, abort, kWsFreed))
      break;
    const uint32_t op = op0 + (i % kStages) * kOpTileBytes;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      over |= bf16x8_over_fp16(cur[k]);
      sts128(op + sw64_offset(16 * k + (d >> 2), d & 3), bf16x8_to_f16x8(cur[k]));
    }
    fence_async_shared();
    mbar_arrive(&ctl->full[i % kStages]);
  }
  if (over) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
}

// The softmax warps' epilogue: each thread of a head row stores its share of
// the columns of the CTA's O half (thread g of two: [128 g, 128 g + 128)), O / l as bf16 into the output or, with
// split-K, as this split's partial in fp16 (its own softmax average, so
// within the range of the fp16 value rows; 2^-11 relative), whose log2-domain
// reference maximum and sum (-inf and 0 when it holds no partial) go beside
// it.  With the in-kernel combine the split then counts itself in: the CTA
// whose split arrives last for its row and value half learns so in
// `ctl->is_last` and combines the row once all its warps are free (see
// combine_splits).  A split whose CTA gave up on a wait (`ok` false,
// SMLA_DEVERR_TIMEOUT set) still arrives, contributing nothing, so the
// counter always completes and the workspace stays valid for the next call.
template <class F>
__device__ __forceinline__ void row_epilogue(const DecodeArgs& a, Ctl* ctl, int C, int64_t t,
                                             int split, int ntiles, float m_ref, float l,
                                             uint32_t tb, int quad, int g, int h, bool live_warp,
                                             bool ok) {
  constexpr int kShare = 256 / F::kRowThreads;
  const bool live = h < a.H;
  const bool partial = a.splits > 1;
  const bool has = ok && ntiles > 0 && live_warp;
  if (partial) {
    float* ml = a.ws_ml + ((t * a.splits + split) * 2 + C) * 2 * a.H;
    if (live && g == 0) {
      ml[h] = has ? m_ref : -INFINITY;
      ml[a.H + h] = has ? l : 0.f;
    }
  } else if (ok && live && C == 0 && g == 0) {
    a.lse[t * a.H + h] = (ntiles == 0) ? -INFINITY : (m_ref + log2f(l)) * kLn2;
  }
  const int64_t row = (partial ? t * a.splits + split : t) * a.H + (live ? h : 0);
  uint4* dst = reinterpret_cast<uint4*>((partial ? a.ws_o : a.out) + row * SMLA_V_DIM + C * 256 + g * kShare);
  if (has) {
    // tcgen05.ld is warp-collective: every lane loads, only live heads store
    const float inv = partial && !(l > 0.f) ? 0.f : 1.f / l;
    // 32-byte stores fill whole sectors (`out` itself may be 16-byte aligned)
    const bool whole = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
    for (int cc = 0; cc < kShare / 32; ++cc) {
      uint32_t r[32], o[16];
      tmem_ld32(tmem_addr(tb, 32 * quad, kOCol + kShare * g + 32 * cc), r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float x0 = __uint_as_float(r[2 * j]) * inv;
        const float x1 = __uint_as_float(r[2 * j + 1]) * inv;
        if (partial) {
          o[j] = h2_bits(__floats2half2_rn(x0, x1));
        } else {
          const __nv_bfloat162 v = __floats2bfloat162_rn(x0, x1);
          o[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
      if (live && whole) {
        stg256(dst + cc * 4, o);
        stg256(dst + cc * 4 + 2, o + 8);
      } else if (live) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[cc * 4 + k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
  } else if (!partial && ok && ntiles == 0 && live) {
#pragma unroll 1
    for (int k = 0; k < kShare / 8; ++k) dst[k] = make_uint4(0, 0, 0, 0);
  }
  if (!partial) return;
  if (!a.combine_in_kernel) {  // split_combine_kernel merges after this grid
    if (h == 0 && g == 0) ctl->is_last = 0;
    return;
  }
  __threadfence();
  named_bar_sync(2, Roles<F>::kSoftmaxThreads);
  if (h == 0 && g == 0) ctl->is_last = (atomicAdd(a.ws_tick + t * 2 + C, 1) == a.splits - 1);
}

// Split-K combine of one row's value half, run by all threads of the CTA
// whose split arrived last, after the roles have finished (TMEM released,
// the peer no longer writing into this CTA's shared memory).  With m_s and
// l_s the splits' log2-domain maxima and sums, M = max m_s over the splits
// that hold a partial, L = sum l_s 2^(m_s - M), out = sum 2^(m_s - M) O_s / L
// and LSE = (M + log2 L) ln 2: the same split merge as across shards, here
// over the key ranges of one shard.
//
// A split holds a partial for every head or for none (a split with a valid
// key has l >= 1 for each head: its largest key contributes 2^0), so the
// non-empty splits are listed once, from head 0's sums.  Each thread owns
// fixed float4 columns of the output (a warp covers 512 contiguous bytes of
// one head row) and accumulates them over the listed splits with independent
// loads, 11 or 8 columns per pass, two passes; the per-(split, head) weights sit
// in the operand stages, per head M and 1 / L beside the exchange buffers.
// Splits are taken kCombChunk at a time.  The sums run in split order, as
// the per-head M and L do.
constexpr int kCombChunk = (kStages * kOpTileBytes) / (128 * 4);  // splits whose weights fit
static_assert(kCombChunk * 4 + 1024 + 16 <= 2 * kXBytes, "split list and head stats fit");

template <class F>
__device__ void combine_splits(const DecodeArgs& a, uint8_t* sm, int C, int64_t t) {
  constexpr int kThreads = Roles<F>::kThreads;
  constexpr int kCombItems = (4096 + kThreads - 1) / kThreads;  // float4 columns per pass
  static_assert(2 * kCombItems * kThreads >= 128 * (SMLA_V_DIM / 2) / 4, "two passes cover a value half");
  const int S = a.splits;
  const int H = a.H;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  float* s_m = reinterpret_cast<float*>(sm + kOffX);  // per head: M
  float* s_inv = s_m + 128;                           // per head: 1 / L (0 when empty)
  int* s_n = reinterpret_cast<int*>(s_m + 256);       // listed splits in this chunk
  int* s_list = s_n + 4;                              // the non-empty splits of the chunk
  float* s_w = reinterpret_cast<float*>(sm + kOffOp); // [listed split][head] weights
  const float* ml_row = a.ws_ml + (t * S * 2 + C) * 2 * H;  // split sp at + sp * 4H
  __threadfence();
  if (tid < H) {
    const float* ms = ml_row + tid;
    float M = -INFINITY;
    int sp = 0;
    for (; sp + 8 <= S; sp += 8) {
      float m8[8], l8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m8[k] = __ldcg(ms + int64_t(sp + k) * 4 * H);
        l8[k] = __ldcg(ms + int64_t(sp + k) * 4 * H + H);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (l8[k] != 0.f && (m8[k] > M || m8[k] != m8[k])) M = m8[k];  // NaN propagates
    }
    for (; sp < S; ++sp) {
      const float m1 = __ldcg(ms + int64_t(sp) * 4 * H), l1 = __ldcg(ms + int64_t(sp) * 4 * H + H);
      if (l1 != 0.f && (m1 > M || m1 != m1)) M = m1;
    }
    float L = 0.f;
    if (M != -INFINITY) {
      sp = 0;
      for (; sp + 8 <= S; sp += 8) {
        float m8[8], l8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m8[k] = __ldcg(ms + int64_t(sp + k) * 4 * H);
          l8[k] = __ldcg(ms + int64_t(sp + k) * 4 * H + H);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (l8[k] != 0.f) L += l8[k] * ex2(m8[k] - M);
      }
      for (; sp < S; ++sp) {
        const float l1 = __ldcg(ms + int64_t(sp) * 4 * H + H);
        if (l1 != 0.f) L += l1 * ex2(__ldcg(ms + int64_t(sp) * 4 * H) - M);
      }
    }
    s_m[tid] = M;
    s_inv[tid] = (M == -INFINITY) ? 0.f : 1.f / L;
    if (C == 0) a.lse[t * H + tid] = (M == -INFINITY) ? -INFINITY : (M + log2f(L)) * kLn2;
  }
  const int n_items = H * (SMLA_V_DIM / 2) / 4;  // float4 columns of the value half
  const int n_chunks = (S + kCombChunk - 1) / kCombChunk;
  const uint16_t* o_row = a.ws_o + t * S * H * SMLA_V_DIM + C * 256;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const int it0 = pass * kCombItems * kThreads + tid;
    if (pass * kCombItems * kThreads >= n_items) break;  // uniform
    int32_t off[kCombItems];  // float offset of the column in a split's O rows (head = off / 512)
#pragma unroll
    for (int k = 0; k < kCombItems; ++k) {
      const int it = it0 + k * kThreads;
      const int itc = it < n_items ? it : 0;
      off[k] = (itc >> 6) * SMLA_V_DIM + (itc & 63) * 4;
    }
    float4 acc[kCombItems];
#pragma unroll
    for (int k = 0; k < kCombItems; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int ch = 0; ch < n_chunks; ++ch) {
      const int sp0 = ch * kCombChunk;
      if (pass == 0 || n_chunks > 1) {
        __syncthreads();  // head stats written; the previous chunk's list and weights consumed
        if (warp == 0) {
          // non-empty splits of the chunk, in split order
          const int sp_end = min(S, sp0 + kCombChunk);
          int cnt = 0;
          for (int sb = sp0; sb < sp_end; sb += 32) {
            const int sp = sb + lane;
            const bool ne = sp < sp_end && __ldcg(ml_row + int64_t(sp) * 4 * H + H) != 0.f;
            const unsigned m = __ballot_sync(0xffffffffu, ne);
            if (ne) s_list[cnt + __popc(m & ((1u << lane) - 1u))] = sp;
            cnt += __popc(m);
          }
          if (lane == 0) *s_n = cnt;
        }
        __syncthreads();
        const int n = *s_n;
        for (int idx = tid; idx < n * H; idx += kThreads) {
          const int j = idx / H;
          const int hh = idx - j * H;
          const float* p = ml_row + int64_t(s_list[j]) * 4 * H + hh;
          const float m1 = __ldcg(p), l1 = __ldcg(p + H);
          s_w[idx] = (l1 != 0.f) ? l1 * ex2(m1 - s_m[hh]) * s_inv[hh] : 0.f;
        }
        __syncthreads();
      }
      const int n = *s_n;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const uint16_t* src = o_row + int64_t(s_list[j]) * H * SMLA_V_DIM;
        const float* wj = s_w + j * H;
#pragma unroll
        for (int k = 0; k < kCombItems; ++k) {
          const uint2 raw = __ldcg(reinterpret_cast<const uint2*>(src + off[k]));
          const float2 v0 = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
          const float2 v1 = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
          const float w = wj[off[k] >> 9];
          acc[k].x = fmaf(w, v0.x, acc[k].x);
          acc[k].y = fmaf(w, v0.y, acc[k].y);
          acc[k].z = fmaf(w, v1.x, acc[k].z);
          acc[k].w = fmaf(w, v1.y, acc[k].w);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kCombItems; ++k) {
      const int it = it0 + k * kThreads;
      if (it < n_items) {
        __nv_bfloat162 lo = __floats2bfloat162_rn(acc[k].x, acc[k].y);
        __nv_bfloat162 hi = __floats2bfloat162_rn(acc[k].z, acc[k].w);
        uint2 o;
        o.x = *reinterpret_cast<uint32_t*>(&lo);
        o.y = *reinterpret_cast<uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(a.out + (t * H + (it >> 6)) * SMLA_V_DIM + C * 256 + (it & 63) * 4) = o;
      }
    }
  }
  if (tid == 0) a.ws_tick[t * 2 + C] = 0;
}

// Store 8 q loads (64 dims) as fp16 pairs into 32 (or 16) TMEM columns.
__device__ __forceinline__ void q_store_group(const uint4* raw, uint32_t addr, bool full) {
  uint32_t qr[32];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint4 v = bf16x8_to_f16x8(raw[k]);
    qr[4 * k + 0] = v.x;
    qr[4 * k + 1] = v.y;
    qr[4 * k + 2] = v.z;
    qr[4 * k + 3] = v.w;
  }
  if (full)
    tmem_st32(addr, qr);
  else
    tmem_st16(addr, qr);  // trailing 32 dims
}

// q staging in the prologue, in the operand stages (idle until the tile
// loop): four 16 KB boxes of 64 latent dims x 128 head rows (128-byte
// swizzle) and one 8 KB box of 32 rope dims x 128 head rows (64-byte
// swizzle).
constexpr int kQLatBox = 128 * 128;
constexpr int kQBytes = 4 * kQLatBox + 128 * 64;
static_assert(kQBytes <= kStages * kOpTileBytes, "q staging fits the operand stages");

// Issue the TMA loads of this CTA's 288 q dims of token t (latent dims
// [256c, 256c + 256), rope dims [32c, 32c + 32)) for 128 head rows.
__device__ __forceinline__ void issue_q_tma(const DecodeArgs& a, int64_t t, int c, uint32_t dst,
                                            uint64_t* bar) {
  mbar_arrive_expect_tx(bar, kQBytes);
  const int32_t y = int32_t(t * a.H);
#pragma unroll
  for (int k = 0; k < 4; ++k) tma_load_2d(dst + k * kQLatBox, &a.q_lat, 256 * c + 64 * k, y, bar);
  tma_load_2d(dst + 4 * kQLatBox, &a.q_rope, 512 + 32 * c, y, bar);
}

// Convert head row h of the staged q into tensor memory as fp16 pairs (the
// A operand of QK^T), 64 dims per group of 32 columns; reads follow the
// boxes' swizzles, so 8 consecutive rows hit 8 different bank groups.
// (thread g of two takes groups 3 g ..).
// Returns true when a q value of the row does not fit fp16 (the operand
// precision of QK^T).
template <class F>
__device__ bool q_to_tmem(uint32_t tb, int quad, int g, int h, bool live, uint32_t src) {
  const uint32_t base = tmem_addr(tb, 32 * quad, kQCol);
  uint32_t over = 0;
#pragma unroll 1
  for (int grp = 3 * g; grp < (g || F::kRowThreads == 1 ? 5 : 3); ++grp) {
    uint4 raw[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      uint32_t addr;
      if (grp < 4)
        addr = src + grp * kQLatBox + sw128_offset(h, v);
      else
        addr = src + 4 * kQLatBox + sw64_offset(h, v & 3);
      raw[v] = (live && (grp < 4 || v < 4)) ? lds128(addr) : make_uint4(0, 0, 0, 0);
      over |= bf16x8_over_fp16(raw[v]);
    }
    q_store_group(raw, base + 32 * grp, grp < 4);
  }
  tmem_st_wait();
  return over != 0;
}

// MMA issue, fully unrolled: computing each descriptor in a loop about
// doubles the time an issue takes, which for the N = 64 QK^T steps is slower
// than the tensor core runs them (44 clocks each).  A descriptor's start address field is the byte address / 16, so
// stepping through a stage adds a constant to the stage's base descriptor
// (shared-memory addresses stay below 256 KB: no carry leaves the field).
__device__ __forceinline__ void issue_qk(uint32_t tb, uint32_t op) {
  constexpr uint32_t idesc = idesc_f16_f32(128, kTileN, false, false);
  const uint64_t lat = sdesc_sw128(op, 16, 1024);
  const uint64_t rope = sdesc_sw64(op + kRopeBlock, 16, 512);
#pragma unroll
  for (int k = 0; k < kKSteps; ++k) {
    // 16 dims = 32 bytes of a row; a 128-byte swizzled K-block holds 64 dims
    const uint64_t bd = k < 16 ? lat + uint64_t((k >> 2) * (kKBlockBytes >> 4) + (k & 3) * 2)
                               : rope + uint64_t((k - 16) * 2);
    mma_ts(tb + kSCol, tb + kQCol + 8 * k, bd, idesc, k > 0);
  }
}

// PV of one tile: P (TMEM) x V, V = the operand stage read MN-major, 16 keys
// = 2048 bytes per step.
__device__ __forceinline__ void issue_pv(uint32_t tb, uint32_t op, bool accumulate) {
  constexpr uint32_t idesc = idesc_f16_f32(128, 256, false, true);
  const uint64_t v = sdesc_sw128(op, kKBlockBytes, 1024);
#pragma unroll
  for (int k = 0; k < kTileN / 16; ++k)
    mma_ts(tb + kOCol, tb + kPCol + 8 * k, v + uint64_t(k * (2048 >> 4)), idesc, accumulate || k > 0);
}

template <int kMode, class F>
__device__ void run_cta(const DecodeArgs& a, uint8_t* sm, Ctl* ctl, const HalfRt& hr, int64_t t,
                        int split, uint32_t peer, const Pieces& pieces) {
  const int C = hr.c;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  volatile int* abort = &ctl->abort;
  const int n = ctl->n_list;
  const int ntiles = (n + kTileN - 1) / kTileN;
  using R = Roles<F>;
  const uint32_t tb = ctl->tbase;

  if (warp < R::kSoftmaxWarps) {
    // ------------------------------------------------ softmax + epilogue
    cluster_wait();  // the peer's barriers are initialised
    constexpr int G = F::kRowThreads;
    constexpr int kCols = R::kCols;
    const int h = tid & 127;      // head row == TMEM lane
    const int quad = warp & 3;    // the warp's 32 lanes of TMEM
    const int g = G == 1 ? 0 : warp >> 2;  // which of the row's threads
    const bool live_warp = quad < softmax_warps(a.H);
    const uint32_t xa_bytes = softmax_warps(a.H) * (kXABytes / 4);
    const uint32_t xb_bytes = softmax_warps(a.H) * (kXBBytes / 4);
    const uint32_t lanes = tmem_addr(tb, 32 * quad, 0);
    const float scale_log2 = a.sm_scale * kLog2e;
    float m_ref = -INFINITY;  // log2-domain reference maximum
    float l = 0.f;            // the sum (two threads a row: this one's columns' share)
    // Key-column split of the softmax: CTA c finishes the scores of keys
    // [32c, 32c + 32) of each tile (its own partial plus the peer's, XA),
    // each of the row's G threads kCols of them, computes their P against a
    // reference maximum, and sends that P and the reference (XB, to the row's
    // thread g of the peer); P of all 64 keys then sits in both CTAs.  With
    // one thread a row the partial sum goes along and both CTAs add it up;
    // with two, each leaves its reference in tensor memory for the other, and
    // the sums meet once, after the last tile.  All of a row's threads move
    // the shared reference R to the same largest of theirs, so O, l and P
    // stay consistent.
    // Buffers alternate by tile parity: the peer writes tile i into buffer
    // set i % 2 only after it has received this CTA's tile-i partial scores,
    // which this CTA sent after it had read tile i - 2 out of that set.
    const int own0 = 32 * C + kCols * g, peer0 = 32 * (1 - C) + kCols * g;  // key columns
    const uint32_t x_l = smem_u32(sm + kOffX);
    const uint32_t peer_x = map_to_cta(x_l, peer);
    const uint32_t peer_xa0 = map_to_cta(smem_u32(&ctl->xa[0]), peer);
    const uint32_t peer_xa1 = map_to_cta(smem_u32(&ctl->xa[1]), peer);
    const uint32_t peer_xb0 = map_to_cta(smem_u32(&ctl->xb[0]), peer);
    const uint32_t peer_xb1 = map_to_cta(smem_u32(&ctl->xb[1]), peer);
    if (tid == 0 && ntiles > 0) {
      for (int b = 0; b < 2 && b < ntiles; ++b) {
        mbar_arrive_expect_tx(&ctl->xa[b], xa_bytes);
        mbar_arrive_expect_tx(&ctl->xb[b], xb_bytes);
      }
      if (G == 2) mbar_arrive_expect_tx(&ctl->sums, softmax_warps(a.H) * 512);
    }
    // The loop is software-pipelined across tiles: while the P of tile i is
    // in flight between the CTAs, the scores of tile i + 1 are read and the
    // peer's half of them sent, so the two exchanges of consecutive tiles
    // overlap.
    float sown[kCols];  // this thread's partial scores of its own columns, next tile
    // Read tile t's partial scores (QK^T of tile t done), release S for the
    // next QK^T, send the peer's columns, keep the own.
    auto start_tile = [&](int t) -> bool {
      if (!__all_sync(0xffffffffu, wait_bar(&ctl->s_full, t & 1, abort, kWsSFull))) return false;
      tc_fence_after();
      uint32_t r[kCols], o[kCols];
      tmem_ldn<kCols>(lanes + kSCol + peer0, r);
      tmem_ldn<kCols>(lanes + kSCol + own0, o);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&ctl->s_free);
      const int b = t & 1;
      const uint32_t xa_p = peer_x + b * kXBytes;
#pragma unroll
      for (int j4 = 0; j4 < kCols / 4; ++j4)
        st_async_v4(xa_p + ((kCols / 4 * g + j4) * 128 + h) * 16, __uint_as_float(r[4 * j4]),
                    __uint_as_float(r[4 * j4 + 1]), __uint_as_float(r[4 * j4 + 2]),
                    __uint_as_float(r[4 * j4 + 3]), b ? peer_xa1 : peer_xa0);
#pragma unroll
      for (int j = 0; j < kCols; ++j) sown[j] = __uint_as_float(o[j]);
      return true;
    };
    // A warp whose wait gave up leaves the loop (at give_up below); the
    // others' waits give up too, since every wait is an mbarrier wait that
    // sees the CTA's abort flag.  The softmax warps enter the loop on one
    // reduced decision and meet again only at the epilogue's barrier.
    bool ok = ntiles == 0 || !live_warp || start_tile(0);
    ok = !named_bar_or(5, R::kSoftmaxThreads, !ok);
    int i = 0;
    for (; i < ntiles && ok && live_warp; ++i) {
      const int b = i & 1;
      const uint32_t xa_l = x_l + b * kXBytes;     // this CTA's buffer set b
      const uint32_t xa_p = peer_x + b * kXBytes;  // the peer's
      // 1) full scores of this thread's columns of tile i
      ok = __all_sync(0xffffffffu, wait_bar_cluster(&ctl->xa[b], (i >> 1) & 1, abort, kWsExchange));
      if (!ok) goto give_up;
      float f[kCols];
#pragma unroll
      for (int j4 = 0; j4 < kCols / 4; ++j4) {
        const float4 v = ld_shared_f4(xa_l + ((kCols / 4 * g + j4) * 128 + h) * 16);
        f[4 * j4] = sown[4 * j4] + v.x;
        f[4 * j4 + 1] = sown[4 * j4 + 1] + v.y;
        f[4 * j4 + 2] = sown[4 * j4 + 2] + v.z;
        f[4 * j4 + 3] = sown[4 * j4 + 3] + v.w;
      }
      if (tid == 0 && i + 2 < ntiles) mbar_arrive_expect_tx(&ctl->xa[b], xa_bytes);
      const int valid = min(kTileN, n - i * kTileN) - own0;  // valid columns of this thread's
      if (valid < kCols) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) f[j] = (j < valid) ? f[j] : -INFINITY;
      }
      float mq[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mq[k] = f[k];
#pragma unroll
      for (int j = 8; j < kCols; ++j) mq[j & 7] = fmaxf(mq[j & 7], f[j]);
      const float mx = scale_log2 * fmaxf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])),
                                          fmaxf(fmaxf(mq[4], mq[5]), fmaxf(mq[6], mq[7])));
      // 2) P of this thread's columns against its reference (R, or its own
      //    maximum when that exceeds R by more than 2^8)
      const float my_ref = (mx > m_ref + 8.f) ? mx : m_ref;
      uint32_t pk[kCols / 2];
      float l_part = 0.f;
      // P against reference `ref` (fp16 pairs, one rounding) and its sum;
      // nothing valid yet: zeros
      auto own_p = [&](float ref) {
        l_part = 0.f;
        if (ref == -INFINITY) {
#pragma unroll
          for (int j = 0; j < kCols / 2; ++j) pk[j] = 0u;
          return;
        }
        float sums[4] = {0.f, 0.f, 0.f, 0.f};
        const float neg_m = -ref;
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          const float p0 = ex2(fmaf(f[2 * j], scale_log2, neg_m));
          const float p1 = ex2(fmaf(f[2 * j + 1], scale_log2, neg_m));
          sums[j & 3] += p0 + p1;
          pk[j] = h2_bits(__floats2half2_rn(p0, p1));
        }
        l_part = (sums[0] + sums[1]) + (sums[2] + sums[3]);
      };
      own_p(my_ref);
      // 3) P and reference go to the peer: with the partial sum, or, with two
      //    threads a row, the reference also to the other (whose wait on XB
      //    counts this thread's arrival)
      const uint32_t xb_p = xa_p + kXABytes;
      const uint32_t xbb = b ? peer_xb1 : peer_xb0;
#pragma unroll
      for (int q = 0; q < kCols / 8; ++q)
        st_async_v4(xb_p + ((kCols / 8 * g + q) * 128 + h) * 16, __uint_as_float(pk[4 * q]),
                    __uint_as_float(pk[4 * q + 1]), __uint_as_float(pk[4 * q + 2]),
                    __uint_as_float(pk[4 * q + 3]), xbb);
      if constexpr (G == 1) {
        st_async_v2(xb_p + kXBPBytes + h * 8, my_ref, l_part, xbb);
      } else {
        st_async_f32(xb_p + kXBPBytes + (g * 128 + h) * 4, my_ref, xbb);
        tmem_st1(lanes + kRefCol + 2 * b + g, __float_as_uint(my_ref));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ctl->xb[b]);
      }
      // 4) while that is in flight: tile i + 1's scores (its QK^T could start
      //    once S(i) was read)
      if (i + 1 < ntiles && !start_tile(i + 1)) goto give_up;
      // 5) the peer's P of tile i and the row's references
      ok = __all_sync(0xffffffffu, wait_bar_cluster(&ctl->xb[b], (i >> 1) & 1, abort, kWsExchangeP));
      if (!ok) goto give_up;
      const uint32_t xb_l = xa_l + kXABytes;
      uint32_t pp[kCols / 2];
#pragma unroll
      for (int q = 0; q < kCols / 8; ++q) {
        const uint4 v = lds128(xb_l + ((kCols / 8 * g + q) * 128 + h) * 16);
        pp[4 * q] = v.x;
        pp[4 * q + 1] = v.y;
        pp[4 * q + 2] = v.z;
        pp[4 * q + 3] = v.w;
      }
      // 6) the shared reference moves to the largest of the row's (identically
      //    in all its threads); what was computed against a smaller one is
      //    redone
      float peer_ref, l_peer = 0.f, r_new;
      if constexpr (G == 1) {
        const float2 peer_rl = ld_shared_f2(xb_l + kXBPBytes + h * 8);
        peer_ref = peer_rl.x;
        l_peer = peer_rl.y;
        r_new = fmaxf(my_ref, peer_ref);
      } else {
        uint32_t other;
        tc_fence_after();
        tmem_ld1(lanes + kRefCol + 2 * b + (1 - g), other);
        peer_ref = ld_shared_f32(xb_l + kXBPBytes + (g * 128 + h) * 4);
        const float peer_other = ld_shared_f32(xb_l + kXBPBytes + ((1 - g) * 128 + h) * 4);
        tmem_ld_wait();
        r_new = fmaxf(fmaxf(my_ref, __uint_as_float(other)), fmaxf(peer_ref, peer_other));
      }
      if (tid == 0 && i + 2 < ntiles) mbar_arrive_expect_tx(&ctl->xb[b], xb_bytes);
      float alpha = 1.f;  // O and l
      bool rescale = false;
      if (r_new != m_ref) {
        alpha = ex2(m_ref - r_new);  // 0 while nothing was valid yet
        rescale = (i > 0);
      }
      // own P against a smaller reference: recomputed from the fp32 scores
      // (one rounding); the peer's: scaled in fp32 and rounded once more
      if (my_ref != r_new) own_p(r_new);
      if (peer_ref != r_new) {
        const float fp = (peer_ref == -INFINITY) ? 0.f : ex2(peer_ref - r_new);
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&pp[j]));
          pp[j] = h2_bits(__floats2half2_rn(v.x * fp, v.y * fp));
        }
        l_peer *= fp;
      }
      m_ref = r_new;
      // one thread a row: the same sum on both CTAs, keys 0..31 first
      l = l * alpha + (G == 2 ? l_part : C ? l_peer + l_part : l_part + l_peer);
      if (i > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(&ctl->pv_done, (i - 1) & 1, abort, kWsPvDone));
        if (!ok) goto give_up;
        tc_fence_after();
      }
      // P(i) replaces P(i-1), which PV(i-1) has finished reading: two keys a
      // column
      tmem_stn<kCols / 2>(lanes + kPCol + own0 / 2, pk);
      tmem_stn<kCols / 2>(lanes + kPCol + peer0 / 2, pp);
      if (i > 0) {
        // tcgen05.ld/st are warp-collective: the warp rescales together when
        // any of its rows needs it, each lane by its own factor (1 if none),
        // a row's threads each their share of O's columns
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int cc = 8 / G * g; cc < 8 / G * (g + 1); ++cc) {
            uint32_t r[32];
            tmem_ld32(lanes + kOCol + 32 * cc, r);
            tmem_ld_wait();
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) r[jj] = __float_as_uint(__uint_as_float(r[jj]) * alpha);
            tmem_st32(lanes + kOCol + 32 * cc, r);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
      // this thread's share of P(i) is in TMEM: once all have arrived the MMA
      // warp issues PV(i); its completion releases the operand stage and lets
      // the next P overwrite this one
      mbar_arrive(&ctl->p_full);
    }
    if (false) {
    give_up:
      // this warp's wait gave up (the CTA's abort flag is up, so every
      // other wait of the CTA gives up too)
      ok = false;
    }
    // epilogue
    if (ok && ntiles > 0 && live_warp) {
      if constexpr (G == 2) {
        // the row's four shares of the sum meet in its own slot of the first
        // exchange buffer (every reader of that slot has sent its P, or
        // arrived, after reading it) and are added in one order
        const uint32_t slot = h * 16 + (2 * C + g) * 4;
        st_async_f32(map_to_cta(x_l, uint32_t(C)) + slot, l,
                     map_to_cta(smem_u32(&ctl->sums), uint32_t(C)));
        st_async_f32(peer_x + slot, l, map_to_cta(smem_u32(&ctl->sums), peer));
        ok = __all_sync(0xffffffffu, wait_bar_cluster(&ctl->sums, 0, abort, kWsExchange));
        const float4 v = ld_shared_f4(x_l + h * 16);
        l = (v.x + v.y) + (v.z + v.w);
      }
      ok = __all_sync(0xffffffffu,
                      ok && wait_bar(&ctl->pv_done, (ntiles - 1) & 1, abort, kWsPvLast));
      tc_fence_after();
    }
    // one decision for all softmax warps (the epilogue below uses a named
    // barrier of theirs)
    ok = !named_bar_or(4, R::kSoftmaxThreads, !ok);
    // this CTA sends nothing more: the peer may leave once it has arrived too
    // (each waits for that at its very end, behind the stores below)
    __syncwarp();
    cluster_arrive_relaxed();
    row_epilogue<F>(a, ctl, C, t, split, ntiles, m_ref, l, tb, quad, g, h, live_warp, ok);
  } else if (warp < R::kMmaWarp) {
    // ------------------------------------------------ dequantise
    // Converter d owns key d % 64 of every tile and half d / 64 of its
    // pieces, so each warp stores 32 consecutive rows of one chunk column
    // (conflict-free under the 128-byte swizzle).
    const int d = tid - 32 * R::kConvWarp0;
    if constexpr (F::kFp4)
      convert_codes(ctl, sm, n, ntiles, C, d, abort);
    else
      convert_loop(ctl, sm, n, ntiles, d & (kTileN - 1), C, d >> 6, lane, abort);
  } else if (warp >= R::kLoaderWarp0) {
    // ------------------------------------------------ stage cache rows, or rope
    if constexpr (!F::kFp4) {
      loader_loop<kMode>(a, ctl, sm, n, ntiles, pieces, abort);
    } else if (tid < 32 * R::kLoaderWarp0 + kRopeThreads) {
      convert_rope(ctl, sm, n, ntiles, C, tid - 32 * R::kLoaderWarp0, abort);
    }
  } else {
    // ------------------------------------------------ MMA issue
    // QK(i) needs its operand stage converted and S(i - 1) read by the
    // softmax, PV(i) the softmax's P(i); the warp sleeps on each barrier
    // until the hardware wakes it at the phase change.  Issuing PV here
    // rather than from a softmax thread keeps the MMA issue and a per-tile
    // barrier of the softmax warps off the softmax's chain.
    // The whole warp runs the loop on values that are the same in every lane
    // and one elected lane issues: descriptors then stay in uniform registers,
    // and the 18 instructions of QK^T take ~400 clocks to issue (1200 when one
    // lane ran the loop alone; dense decode 673 -> 645 us, windows of 4,112
    // entries 153 -> 136).
    const uint32_t op0 = __shfl_sync(0xffffffffu, smem_u32(sm + kOffOp), 0);
    const uint32_t tbu = __shfl_sync(0xffffffffu, tb, 0);
    const int nt = __shfl_sync(0xffffffffu, ntiles, 0);
    const bool leader = elect_one();
    bool ok = wait_bar(&ctl->q_ready, 0, abort, kWsQReady);
    const int steps = __all_sync(0xffffffffu, ok) ? nt + 2 : 0;
    // QK(j), then PV(j - 2): the softmax stores P(j - 2) after it has read
    // S(j - 1), which frees S for QK(j)
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      if (j < nt) {
        ok = wait_bar(&ctl->full[j % kStages], (j / kStages) & 1, abort, kWsFull) &&
             (j == 0 || wait_bar(&ctl->s_free, (j - 1) & 1, abort, kWsSFree));
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (leader) {
          issue_qk(tbu, op0 + (j % kStages) * kOpTileBytes);
          mma_commit(&ctl->s_full);
        }
        __syncwarp();
      }
      const int i = j - 2;
      if (i >= 0) {
        ok = wait_bar(&ctl->p_full, i & 1, abort, kWsPFull);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (leader) {
          issue_pv(tbu, op0 + (i % kStages) * kOpTileBytes, i > 0);
          mma_commit(&ctl->pv_done);
          mma_commit(&ctl->freed[i % kStages]);
        }
        __syncwarp();
      }
    }
    // drain: every MMA issued above has completed before TMEM is released
    // (waited on even after an abort, with its own bound).  A CTA whose row
    // has no valid slot issued no MMA and has nothing to drain.
    if (ntiles > 0) {
      if (leader) mma_commit(&ctl->end);
      __syncwarp();
      int no_abort = 0;
      wait_bar(&ctl->end, 0, &no_abort, kWsDrain);
    }
  }
}

// The raw entries [0, limit) of a generated row (positions, or local
// positions of one rank): entry v is position v, or v + skip from entry
// `first` on (a window behind a gap).
struct RowRange {
  int32_t limit = 0, first = 0, skip = 0;
};

// Resolve raw entry v to (slot, shard).  Per-shard launch: the entry
// already is a local slot.  Fused DCP step and merged dense decode: the
// entry is a global position v; with interleave size I, runs of I positions
// go to the shards in turn, so v is owned by shard (v div I) mod D at local
// position (v div (I D)) I + v mod I (I = 1: shard v mod D, position
// v div D).  Dense decode of one rank: the entry is that rank's local
// position itself.  The local position then goes through that shard's
// block-table row for this request (staged in shared memory at `bt` when it
// fits, else read from global memory).  `range` bounds the valid entries of
// a generated row and places them.  Returns false for -1 / foreign / invalid
// entries, recording input errors in `err`.
template <int kMode>
__device__ __forceinline__ int32_t place_entry(int32_t v, const RowRange& range) {
  return kMode == kModeWindow && v >= range.first ? v + range.skip : v;
}

template <int kMode>
__device__ __forceinline__ bool resolve_entry(const DecodeArgs& a, const Ctl* ctl, const int32_t* bt,
                                              bool staged, bool req_ok, const RowRange& range,
                                              int32_t v, int32_t& slot, int& shard,
                                              unsigned& err) {
  if (kMode == kModeSlots) {
    if (v >= a.num_slots) {
      err |= SMLA_DEVERR_SLOT_RANGE;
      return false;
    }
    slot = v;
    shard = 0;
    return v >= 0;
  }
  // Pools: every entry takes the same straight-line path (no branch per
  // check), so the entries of a thread overlap their shared-memory reads.
  const bool live = v >= 0 && req_ok && !(generated(kMode) && v >= range.limit);
  const int32_t vv = place_entry<kMode>(live ? v : 0, range);
  int d;
  int32_t lp;
  if (generated(kMode) && a.dense_rank >= 0) {
    d = a.dense_rank;
    lp = vv;
  } else {
    const uint32_t g = fastdiv(uint32_t(vv), a.div_I);  // run of I positions
    const uint32_t round = fastdiv(g, a.div_D);         // round of D runs
    d = int(g - round * uint32_t(a.D));
    lp = int32_t(round) * a.interleave + (vv - int32_t(g) * a.interleave);
  }
  const ShardMeta m = ctl->meta[d];
  const int32_t col = int32_t(fastdiv(uint32_t(lp), a.div_bs));
  const bool in_table = col < m.bt_width;
  const int32_t colc = in_table ? col : 0;  // every table has a column 0
  const int32_t blk = staged ? bt[m.bt_off + colc] : ctl->bt_row[d][colc];
  const int64_t s64 = int64_t(blk) * a.block_size + (lp - col * a.block_size);
  const bool in_pool = s64 < m.pool_slots;
  err |= (live && (!in_table || blk < 0)) ? unsigned(SMLA_DEVERR_BLOCK_TABLE) : 0u;
  err |= (live && in_table && blk >= 0 && !in_pool) ? unsigned(SMLA_DEVERR_SLOT_RANGE) : 0u;
  slot = int32_t(s64);
  shard = d;
  return live && in_table && blk >= 0 && in_pool;
}

// How many of the first n positions rank `dense_rank` holds: whole rounds of
// I*D positions give I each, then the partial round.
__device__ __forceinline__ int32_t rank_rows(const DecodeArgs& a, int32_t n) {
  // a round that does not fit 32 bits never completes
  const int64_t ID = int64_t(a.interleave) * a.D;
  const int32_t full = ID > n ? 0 : n / int32_t(ID);
  const int64_t mine = int64_t(n) - full * ID - int64_t(a.dense_rank) * a.interleave;
  return full * a.interleave + int32_t(min(max(mine, int64_t(0)), int64_t(a.interleave)));
}

// Dense and windowed decode: the request of row t and the range of its raw
// entries.  Dense: its positions 0..p (p its own), or that many positions'
// share of one rank in the per-rank form.  Windowed: the first min(sinks, w0)
// positions and [w0, p], w0 = max(p + 1 - window, 0), or one rank's share of
// both.  False for every row of a request (and an error bit) when the
// request's context is shorter than its query tokens or runs past max_ctx.
template <int kMode>
__device__ __forceinline__ bool dense_row(const DecodeArgs& a, int64_t t, int32_t& req,
                                          RowRange& range, unsigned& err) {
  req = int32_t(t / a.S);
  const int32_t ctx = a.ctx_lens[req];
  if (ctx < a.S || ctx > a.max_ctx) {  // the request's query tokens are part of its context
    err |= SMLA_DEVERR_CONTEXT;
    range.limit = 0;
    return false;
  }
  const int32_t n = ctx - a.S + int32_t(t - int64_t(req) * a.S) + 1;  // positions 0..n-1
  if (kMode == kModeDense) {
    range.limit = a.dense_rank < 0 ? n : rank_rows(a, n);
  } else {
    const int32_t w0 = max(n - a.window, 0);
    const int32_t s1 = min(a.sinks, w0);
    const bool merged = a.dense_rank < 0;
    const int32_t cw = merged ? w0 : rank_rows(a, w0);
    range.first = merged ? s1 : rank_rows(a, s1);
    range.skip = cw - range.first;
    range.limit = (merged ? n : rank_rows(a, n)) - range.skip;
  }
  return true;
}

// A generated row's split with no position of it (a short context under a
// long max_ctx) skips the set-up and publishes what the full path would: the
// row's (0, -inf) half without split-K, else an empty partial (-inf, 0)
// that counts in like any other split.  Both CTAs of the pair take this path
// together (the test depends only on the row and the split); it touches no
// tensor memory and no peer shared memory.
template <class F>
__device__ void publish_empty_split(const DecodeArgs& a, uint8_t* sm, Ctl* ctl, int64_t t, int split,
                                    int C) {
  constexpr int kThreads = Roles<F>::kThreads;
  const int tid = threadIdx.x;
  if (a.splits == 1) {
    for (int idx = tid; idx < a.H * 32; idx += kThreads) {  // 32 x 16 bytes per head half
      uint4* dst = reinterpret_cast<uint4*>(a.out + (t * a.H + (idx >> 5)) * SMLA_V_DIM + C * 256);
      dst[idx & 31] = make_uint4(0, 0, 0, 0);
    }
    if (C == 0)
      for (int h = tid; h < a.H; h += kThreads) a.lse[t * a.H + h] = -INFINITY;
    return;
  }
  float* ml = a.ws_ml + ((t * a.splits + split) * 2 + C) * 2 * a.H;
  for (int h = tid; h < a.H; h += kThreads) {
    ml[h] = -INFINITY;
    ml[a.H + h] = 0.f;
  }
  if (!a.combine_in_kernel) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) ctl->is_last = (atomicAdd(a.ws_tick + t * 2 + C, 1) == a.splits - 1);
  __syncthreads();
  if (ctl->is_last) combine_splits<F>(a, sm, C, t);
}

// Decodes of the serving step are launched behind the step's short kernels.
template <int kMode, class F>
constexpr bool overlapped() { return F::kFp4 || kMode == kModeWindow; }

template <int kMode, class F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Roles<F>::kThreads, 1)
    sparse_mla_decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int kSoftmaxWarps = Roles<F>::kSoftmaxWarps;
  constexpr int kMmaWarp = Roles<F>::kMmaWarp;
  constexpr int kLoaderWarp0 = Roles<F>::kLoaderWarp0;
  constexpr int kRowThreads = F::kRowThreads;
  constexpr bool kPools = kMode != kModeSlots;  // entries resolve through D pools
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(sm + kOffCtl);
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t c = cluster_ctarank();
  const uint32_t peer = c ^ 1u;
  const uint32_t item = blockIdx.x >> 1;
  // serving-step decodes: every row's first split, then every row's second ...
  const uint32_t inner = overlapped<kMode, F>() ? a.T : a.splits;
  uint32_t outer = overlapped<kMode, F>() ? 0 : item;
  if (a.splits > 1) outer = item / inner;
  const int64_t t = overlapped<kMode, F>() ? item - outer * inner : outer;
  const int split = int(overlapped<kMode, F>() ? outer : item - outer * inner);
  const int e_begin = split * a.split_entries;
  const int e_end = int(min(uint32_t(a.K), uint32_t(e_begin) + uint32_t(a.split_entries)));

  const HalfRt hr = half_of(c);
  // a separate split combine (if any) may be scheduled on SMs this grid
  // leaves idle
  griddep_launch_dependents();
  // a generated row's split without a position: published, nothing to do
  auto empty_split = [&]() -> bool {
    int32_t r;
    RowRange range;
    unsigned e2 = 0;
    const bool row_ok = dense_row<kMode>(a, t, r, range, e2);
    if (row_ok && min(e_end, range.limit) > e_begin) return false;
    if (tid == 0 && e2) atomicOr(&g_decode_error, e2);
    publish_empty_split<F>(a, sm, ctl, t, split, hr.c);
    return true;
  };
  if (kMode == kModeDense && empty_split()) return;
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tbase, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&ctl->q_tma, 1);
    mbar_init(&ctl->q_ready, 32 * kSoftmaxWarps);
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&ctl->full[st], F::kFp4 ? 128 + kRopeThreads : 128);
      mbar_init(&ctl->freed[st], 1);
    }
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->s_free, 32 * kRowThreads * softmax_warps(a.H));  // one arrival per softmax thread
    mbar_init(&ctl->pv_done, 1);
    mbar_init(&ctl->p_full, 32 * kRowThreads * softmax_warps(a.H));
    for (int st = 0; st < kRawStages; ++st) {
      mbar_init(&ctl->raw_full[st], kLoaders);  // one arrival per loader
      mbar_init(&ctl->raw_empty[st], 4);        // one arrival per converter warp
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->xa[b], 1);  // one expect_tx arrival per phase
      // with two threads a row, also one arrival per reference left in tensor memory
      mbar_init(&ctl->xb[b], 1 + (kRowThreads == 2 ? 64 * softmax_warps(a.H) : 0));
    }
    mbar_init(&ctl->sums, 1);
    mbar_init(&ctl->end, 1);
    ctl->abort = 0;
    fence_mbar_init_cluster();
  }
  if (overlapped<kMode, F>()) {
    griddep_wait();  // set-up so far overlaps the end of the kernel before
    if (kMode == kModeWindow && empty_split()) {
      tc_fence_before();
      __syncthreads();  // tensor memory's address has been written
      tc_fence_after();
      if (warp == kMmaWarp) tmem_dealloc(ctl->tbase, kTmemCols);
      return;
    }
  }
  // q lands in the (still idle) operand stages while the CTA sets up
  if (tid == 0) issue_q_tma(a, t, hr.c, smem_u32(sm + kOffOp), &ctl->q_tma);
  Pieces pieces;
  if (!F::kFp4 && warp >= kLoaderWarp0) pieces.place(hr.c, tid - 32 * kLoaderWarp0);
  // The compacting warps' raw entries (kPer each of the row's split, see the
  // compaction below) are loaded before the set-up barrier, so that their
  // memory round trip overlaps the request id's.
  constexpr int kListThreads = Roles<F>::kThreads - 32 * kSoftmaxWarps;  // every warp but the softmax warps
  constexpr int kPer =
      ((kMode == kModeWindow ? kWindowList : kMaxList) + kListThreads - 1) / kListThreads;
  int32_t vs[kPer];
  if (!generated(kMode) && warp >= kSoftmaxWarps) {
    const int j0 = e_begin + (tid - 32 * kSoftmaxWarps) * kPer;
    const int32_t* src = (kMode == kModeTopk ? a.topk : a.slots) + t * a.K;
    if (j0 + kPer <= e_end && (reinterpret_cast<uintptr_t>(src + j0) & 15u) == 0) {
#pragma unroll
      for (int q4 = 0; q4 < kPer / 4; ++q4) {
        const int4 w = reinterpret_cast<const int4*>(src + j0)[q4];
        vs[4 * q4] = w.x;
        vs[4 * q4 + 1] = w.y;
        vs[4 * q4 + 2] = w.z;
        vs[4 * q4 + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) vs[k] = (j0 + k < e_end) ? src[j0 + k] : -1;
    }
  }
  if (kPools && tid < a.D) {
    // per-shard pointers of this row's request, read once
    const int32_t r = generated(kMode) ? int32_t(t / a.S) : a.req_id[t];
    const bool ok = r >= 0 && r < a.num_reqs;
    ctl->pool[tid] = a.pools[tid];
    ctl->bt_row[tid] = a.bts[tid] + (ok ? int64_t(r) * a.bt_stride[tid] : 0);
  }
  if (kPools && tid == 0) {
    // the request's block-table rows of all shards, staged in the exchange
    // buffers (idle until the tile loop) when they fit
    int off = 0;
    for (int d = 0; d < a.D; ++d) {
      ctl->meta[d].bt_off = off;
      ctl->meta[d].bt_width = a.bt_width[d];
      ctl->meta[d].pool_slots = a.pool_slots[d];
      off += a.bt_width[d];
    }
    // a window's entries span few blocks: each reads its table entry itself
    ctl->bt_staged = kMode != kModeWindow && off <= kBtStageMax;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp < kSoftmaxWarps) {
    // Q half -> TMEM, overlapping the compaction below
    // the whole q tile landed (issued by thread 0 before the set-up barrier)
    bool qok = wait_bar(&ctl->q_tma, 0, &ctl->abort, kWsQReady);
    const int quad = warp & 3, h = tid & 127;
    if (quad < softmax_warps(a.H) &&
        q_to_tmem<F>(ctl->tbase, quad, kRowThreads == 1 ? 0 : warp >> 2, h, qok && h < a.H, smem_u32(sm + kOffOp)))
      atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
    tc_fence_before();
    mbar_arrive(&ctl->q_ready);
    named_bar_sync(6, Roles<F>::kThreads);  // the list's length is known
  } else {
    // Ordered compaction of the split's valid entries by the 256 threads of
    // the other warps (idle until the tile loop): thread d owns the kPer
    // contiguous entries from e_begin + kPer d on, resolves them with all loads
    // in flight at once, and a block scan gives each thread its output
    // offset.  Both CTAs of the pair build the same list, so their tiles hold
    // the same keys.
    const int d = tid - 32 * kSoftmaxWarps;
    int* list = reinterpret_cast<int*>(sm + kOffList);
    uint8_t* list_shard = sm + kOffListShard;
    const uint8_t** rows = reinterpret_cast<const uint8_t**>(sm + kOffRows);
    unsigned err = 0;
    bool req_ok = true;
    RowRange range;
    if (kMode == kModeTopk) {
      const int32_t r = a.req_id[t];
      req_ok = r >= 0 && r < a.num_reqs;
      if (!req_ok && d == 0) err |= SMLA_DEVERR_REQ_ID;
    } else if (generated(kMode)) {
      int32_t r;
      unsigned e2 = 0;
      req_ok = dense_row<kMode>(a, t, r, range, e2);
      if (d == 0) err |= e2;
    }
    // A window's entries are valid unless an input is not: the threads take
    // them in turn, each entry at its own place in the list.  One that is not
    // valid sends the CTA through the compaction below.
    bool listed = false;
    if (kMode == kModeWindow) {
      const int cnt = req_ok ? min(e_end, range.limit) - e_begin : 0;
      bool all = true;
#pragma unroll 2
      for (int j = d; j < cnt; j += kListThreads) {
        int32_t slot = -1;
        int sh = 0;
        unsigned e1 = 0;
        all = resolve_entry<kMode>(a, ctl, nullptr, false, req_ok, range, e_begin + j, slot, sh, e1) &&
              all;
        if constexpr (F::kFp4) {
          rows[j] = ctl->pool[sh] + int64_t(slot) * F::kRowBytes;
        } else {
          list[j] = slot;
          list_shard[j] = uint8_t(sh);
        }
      }
      listed = !named_bar_or(3, kListThreads, !all);
      if (listed && d == 0) ctl->n_list = max(cnt, 0);
    }
    if (!listed) {
      // 1) this thread's kPer raw entries (loaded before the set-up barrier,
      //    by 16-byte loads when the row allows; a generated row's entries are
      //    just their indices), and, with D pools, the request's block-table
      //    rows copied into shared memory by all the compacting threads
      const int j0 = e_begin + d * kPer;
      if (generated(kMode)) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) vs[k] = j0 + k;
      }
      int32_t* bt = reinterpret_cast<int32_t*>(sm + kOffX);
      const bool staged = kPools && ctl->bt_staged;
      if (staged) {
        const uint32_t bt0 = smem_u32(bt);
#pragma unroll 1
        for (int sd = 0; sd < a.D; ++sd) {
#pragma unroll 1
          for (int col = d; col < ctl->meta[sd].bt_width; col += kListThreads)
            cp_async_4(bt0 + 4u * uint32_t(ctl->meta[sd].bt_off + col), ctl->bt_row[sd] + col);
        }
        cp_async_commit();
        cp_async_wait<0>();
        named_bar_sync(3, kListThreads);  // every thread's copies are visible
      }
      // 2) resolve them from registers and shared memory
      int shards[kPer];
      unsigned keep = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int32_t v = vs[k];
        vs[k] = -1;
        shards[k] = 0;
        const bool ok = resolve_entry<kMode>(a, ctl, bt, staged, req_ok, range,
                                             j0 + k < e_end ? v : -1, vs[k], shards[k], err);
        keep |= unsigned(ok) << k;
      }
      const int cnt = __popc(keep);
      int incl = cnt;  // inclusive warp scan
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      if (lane == 31) ctl->warp_cnt[warp - kSoftmaxWarps] = incl;
      named_bar_sync(3, kListThreads);
      int wbase = 0, total = 0;
#pragma unroll
      for (int w = 0; w < kListThreads / 32; ++w) {
        const int x = ctl->warp_cnt[w];
        wbase += (w < warp - kSoftmaxWarps) ? x : 0;
        total += x;
      }
      int pos = wbase + incl - cnt;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (keep & (1u << k)) {
          if constexpr (F::kFp4) {
            rows[pos] = (kPools ? ctl->pool[shards[k]] : a.kv) + int64_t(vs[k]) * F::kRowBytes;
          } else {
            list[pos] = vs[k];
            list_shard[pos] = uint8_t(shards[k]);
          }
          ++pos;
        }
      }
      if (d == 0) ctl->n_list = total;
    }
    if (err) atomicOr(&g_decode_error, err);
    // the list is complete: its readers start on the first rows while q is
    // still on its way into tensor memory
    named_bar_arrive(6, Roles<F>::kThreads);
    named_bar_sync(3, kListThreads);
  }
  // The peer's barriers are initialised, and its staged block tables read,
  // before any remote store: only the softmax warps, which send them, wait
  // for that before their loop.
  __syncwarp();
  cluster_arrive();

  run_cta<kMode, F>(a, sm, ctl, hr, t, split, peer, pieces);

  if (warp >= kSoftmaxWarps) {
    __syncwarp();
    cluster_wait();
    cluster_arrive_relaxed();
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // the peer no longer writes into this CTA's shared memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(ctl->tbase, kTmemCols);
  }
  if (a.splits > 1 && ctl->is_last) combine_splits<F>(a, sm, hr.c, t);
}

// Split-K combine of one row's value half for eight heads, one warp per
// head, launched after the decode grid with programmatic stream
// serialisation.  With m_s and l_s the splits' log2-domain maxima and sums,
// M = max m_s over the splits that hold a partial (l_s != 0), L = sum l_s
// 2^(m_s - M), out = sum_s 2^(m_s - M) O_s / L, LSE = (M + log2 L) ln 2: the
// merge of "partial attention results" by their LSE, here over the key ranges
// of one row.  A row whose splits all hold nothing comes out as the merge
// identity (0, -inf).  Lanes own float4 columns lane and lane + 32 of the
// head's value half (two 512-byte coalesced reads per split) and take the
// splits in ascending order, eight at a time, each load independent.
constexpr int kCombHeads = 8;

__device__ __forceinline__ float max_nan(float x, float y) {
  return (x != x || y != y) ? __int_as_float(0x7fc00000) : fmaxf(x, y);
}

__global__ void __launch_bounds__(kCombHeads * 32)
    split_combine_kernel(const uint16_t* __restrict__ ws_o, const float* __restrict__ ws_ml,
                         uint16_t* __restrict__ out, float* __restrict__ lse, int32_t H, int32_t S) {
  griddep_wait();  // the decode grid's partials are complete and visible
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = (H + kCombHeads - 1) / kCombHeads;
  const int64_t t = blockIdx.x / (2 * G);
  const int r = int(blockIdx.x - t * 2 * G);
  const int C = r / G;
  const int h = (r - C * G) * kCombHeads + warp;
  if (h >= H) return;
  const int64_t ml_stride = 4 * int64_t(H);  // floats from one split's stats to the next
  const float* ml = ws_ml + (t * S * 2 + C) * 2 * int64_t(H) + h;  // split sp: m at sp * 4H, l at + H
  float M = -INFINITY;
  for (int sp = lane; sp < S; sp += 32) {
    const float m1 = __ldcg(ml + sp * ml_stride), l1 = __ldcg(ml + sp * ml_stride + H);
    if (l1 != 0.f) M = max_nan(M, m1);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f;
  if (M != -INFINITY) {
    for (int sp = lane; sp < S; sp += 32) {
      const float m1 = __ldcg(ml + sp * ml_stride), l1 = __ldcg(ml + sp * ml_stride + H);
      if (l1 != 0.f) L += l1 * ex2(m1 - M);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  }
  const float inv = (M == -INFINITY) ? 0.f : 1.f / L;
  const uint2* o_row =
      reinterpret_cast<const uint2*>(ws_o + (t * S * H + h) * SMLA_V_DIM + C * 256) + lane;
  const int64_t o_stride = int64_t(H) * SMLA_V_DIM / 4;  // 4-value groups from one split's row to the next
  float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
  for (int base = 0; base < S; base += 32) {
    const int sp = base + lane;
    float m1 = 0.f, l1 = 0.f;
    if (sp < S) {
      m1 = __ldcg(ml + sp * ml_stride);
      l1 = __ldcg(ml + sp * ml_stride + H);
    }
    const bool held = l1 != 0.f;  // this split wrote its partial
    const float w_lane = held ? l1 * ex2(m1 - M) * inv : 0.f;
    unsigned mask = __ballot_sync(0xffffffffu, held);
    while (mask) {
      int idx[8];
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        idx[k] = mask ? __ffs(mask) - 1 : -1;
        w[k] = __shfl_sync(0xffffffffu, w_lane, idx[k] < 0 ? 0 : idx[k]);
        mask &= mask - 1u;
      }
      float4 v0[8], v1[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint2* src = o_row + (base + (idx[k] < 0 ? idx[0] : idx[k])) * o_stride;
        const uint2 r0 = __ldcg(src), r1 = __ldcg(src + 32);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r0.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&r0.y));
        const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&r1.x));
        const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&r1.y));
        v0[k] = make_float4(a.x, a.y, b.x, b.y);
        v1[k] = make_float4(c.x, c.y, d.x, d.y);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (idx[k] >= 0) {
          a0.x = fmaf(w[k], v0[k].x, a0.x);
          a0.y = fmaf(w[k], v0[k].y, a0.y);
          a0.z = fmaf(w[k], v0[k].z, a0.z);
          a0.w = fmaf(w[k], v0[k].w, a0.w);
          a1.x = fmaf(w[k], v1[k].x, a1.x);
          a1.y = fmaf(w[k], v1[k].y, a1.y);
          a1.z = fmaf(w[k], v1[k].z, a1.z);
          a1.w = fmaf(w[k], v1[k].w, a1.w);
        }
      }
    }
  }
  auto pack = [](float4 v) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y);
    __nv_bfloat162 hi = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  };
  uint2* dst = reinterpret_cast<uint2*>(out + (t * H + h) * SMLA_V_DIM + C * 256) + lane;
  dst[0] = pack(a0);
  dst[32] = pack(a1);
  if (C == 0 && lane == 0) lse[t * H + h] = (M == -INFINITY) ? -INFINITY : (M + log2f(L)) * kLn2;
}

// Which combine merges a row's splits.  The in-kernel one overlaps the CTAs
// still running, but one CTA reads every split's partial with a bounded
// number of loads in flight (two rounds of loads per split); the separate
// kernel spreads the reads over (row, half, 8 heads) CTAs for a fixed cost
// (its launch and the wait for this grid to drain).  So the separate kernel
// is taken when the decode grid fits in one wave on the GPU's SMs, whose
// other SMs then sit idle, and there are at least four splits per row.
bool combine_in_kernel(int64_t decode_ctas, int splits, int sms) {
  return decode_ctas > sms || splits < 4;
}

// Split-K policy, a function of the shape alone: enough clusters to cover the
// GB300's 76 SM pairs when there are few query rows, at least 256 top-k
// entries per split, and at most kMaxList entries per split.
constexpr int kClusterSlots = 76;

int decode_splits(int32_t T, int32_t K) {
  const int64_t k = K;  // K may be close to 2^31
  int64_t s = (T > 0) ? kClusterSlots / T : 1;
  s = min(s, (k + 255) / 256);
  s = max(s, (k + kMaxList - 1) / kMaxList);
  return int(max(s, int64_t(1)));
}

// The serving step's decodes take the splits that end first by a model of a
// launch, in 1/100 us, like decode_splits a function of the shape alone, with
// at most `list` entries per split.
//
// Within one wave of pairs, fitted to fp4 decodes of 1-64 rows of 128-2048
// entries (H = 128): 950 for a pair's set-up and epilogue, 145 a tile of 64
// keys, 7 a pair at work on the GPU, and 420 + 12 a split for the kernel that
// merges splits; the counts it picks are within 4% of the best and 0.1% on
// average.  Measured against at least 256 entries a split: 1 row of 512
// entries 8 splits 12.2 us (2: 15.1), 1 of 2048 16 splits 14.3 (8: 15.5), 16 of
// 512 4 splits 15.3 (2: 17.0).
//
// Past one wave a pair takes 810 (with splits 1100) and 135 a tile, and the
// places the last wave of large splits leaves free take one small split a row,
// counted as a tenth longer: 80 rows of 2048 entries 99.6 -> 90 us, 100 rows
// 100.5 -> 94, 8-bit windows of 4,112 entries, 64 rows, 125.5 -> 121.6 (131
// with a row's splits one after the other).  110 and 160 rows stay whole (100.7
// us, 101.4 at best; 150.2, 155.4).
struct SplitPlan {
  int splits, entries;  // of a row, and of every split but the last
};

SplitPlan plan_splits(int32_t T, int32_t K, int list) {
  const int lo = max((K + list - 1) / list, 1);
  auto equal = [&](int s) { return SplitPlan{s, max((K + s - 1) / s, 1)}; };
  if (T <= 0) return equal(lo);
  if (int64_t(T) * lo <= kClusterSlots) {
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int s = 1; int64_t(T) * s <= kClusterSlots && (s - 1) * kTileN < K; ++s) {
      const int tiles = ((K + s - 1) / s + kTileN - 1) / kTileN;
      const int64_t cost = 950 + 145 * int64_t(tiles) + 7 * T * s + (s > 1 ? 420 + 12 * s : 0);
      if (cost < best_cost) {
        best_cost = cost;
        best = s;
      }
    }
    return equal(max(best, lo));
  }
  // More than a wave: the splits of equal size, or larger ones first and a
  // small one of each row in the places the last wave leaves free.
  const int n = (K + kTileN - 1) / kTileN;
  auto pair = [](int tiles, bool split) { return (split ? 1100 : 810) + 135 * int64_t(tiles); };
  SplitPlan best = equal(lo);
  int64_t best_cost = (int64_t(T) * lo + kClusterSlots - 1) / kClusterSlots *
                      pair((best.entries + kTileN - 1) / kTileN, lo > 1);
  for (int p = min(list / kTileN, n - 1); p > n / (lo + 1); --p) {
    const int s = (n + p - 1) / p;
    const int64_t large = pair(p, true), small = pair(n - (s - 1) * p, true) * 11 / 10;
    const int64_t count = int64_t(T) * (s - 1);
    const int64_t waves = count / kClusterSlots;     // full ones
    const int64_t over = count - waves * kClusterSlots;
    const int64_t room = kClusterSlots - over;       // places for small splits beside the last large ones
    const int64_t beside = room * (large / small);
    const int64_t end = (waves + (over > 0)) * large;
    const int64_t left = max(T - beside, int64_t(0));
    const int64_t cost =
        (lo == 1 ? 500 : 0) +  // rows that were whole are merged
        max(end, min(waves * large + (T + room - 1) / room * small,
                     (waves + 1) * large + (left + kClusterSlots - 1) / kClusterSlots * small));
    if (cost < best_cost) {
      best_cost = cost;
      best = {s, p * kTileN};
    }
  }
  return best;
}

// The arrival counters come first, in a region of one size whatever the shape:
// a workspace serves calls of any shapes in turn, and no call's partials may
// lie where another's counters do.  The last 256 bytes are not written, so
// that a workspace of a call's own size ends in zeros, as it always has.
struct WsLayout {
  size_t o_off, ml_off, total;
};

WsLayout ws_layout(int32_t T, int32_t H, int32_t S) {
  WsLayout w{0, 0, 0};
  if (S == 1 || T <= 0) return w;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  w.o_off = kTickBytes;
  w.ml_off = w.o_off + up(size_t(T) * S * H * SMLA_V_DIM * sizeof(uint16_t));
  w.total = w.ml_off + up(size_t(T) * S * 2 * 2 * H * sizeof(float)) + 256;
  return w;
}


// cuTensorMapEncodeTiled, looked up once through the runtime (no link-time
// dependency on the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_tiled_fn(EncodeTiledFn* fn) {
  static std::mutex m;
  static EncodeTiledFn cached = nullptr;
  std::lock_guard<std::mutex> lock(m);
  if (cached == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorNotSupported;
    cached = reinterpret_cast<EncodeTiledFn>(p);
  }
  *fn = cached;
  return cudaSuccess;
}

// Tensor maps over q viewed as [T*H rows, 576] bf16: boxes of 64 dims x 128
// rows with 128-byte swizzle, and 32 dims x 128 rows with 64-byte swizzle.
// Rows past T*H read as zeros.
cudaError_t encode_q_maps(DecodeArgs& a) {
  EncodeTiledFn enc = nullptr;
  cudaError_t e = encode_tiled_fn(&enc);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[2] = {SMLA_QK_DIM, cuuint64_t(a.T) * cuuint64_t(a.H)};
  const cuuint64_t strides[1] = {SMLA_QK_DIM * sizeof(uint16_t)};
  const cuuint32_t box_lat[2] = {64, 128}, box_rope[2] = {32, 128}, ones[2] = {1, 1};
  void* q = const_cast<uint16_t*>(a.q);
  if (enc(&a.q_lat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q, dims, strides, box_lat, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      enc(&a.q_rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q, dims, strides, box_rope, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

// The kernels' shared-memory size attribute, set once per device and kernel,
// safe when several host threads make their first launch at once.
constexpr int kMaxDevices = 64;

template <int kMode, class F>
cudaError_t ensure_smem_attribute(int dev) {
  static std::atomic<bool> done[kMaxDevices];
  static std::mutex m;
  const bool tracked = dev >= 0 && dev < kMaxDevices;
  if (tracked && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  std::lock_guard<std::mutex> lock(m);
  if (tracked && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(sparse_mla_decode_kernel<kMode, F>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess && tracked) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int kMode, class F = Fp8Rows>
cudaError_t launch_impl(const DecodeArgs& args, cudaStream_t s) {
  DecodeArgs a = args;
  {
    const cudaError_t e = encode_q_maps(a);
    if (e != cudaSuccess) return e;
  }
  if (overlapped<kMode, F>()) {
    const SplitPlan plan = plan_splits(a.T, a.K, kMode == kModeWindow ? kWindowList : kMaxList);
    a.splits = plan.splits;
    a.split_entries = plan.entries;
  } else {
    a.splits = a.single_split ? 1 : decode_splits(a.T, a.K);
    a.split_entries = int32_t((int64_t(a.K) + a.splits - 1) / a.splits);
  }
  const WsLayout w = ws_layout(a.T, a.H, a.splits);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  a.ws_o = w.total ? reinterpret_cast<uint16_t*>(ws + w.o_off) : nullptr;
  a.ws_ml = w.total ? reinterpret_cast<float*>(ws + w.ml_off) : nullptr;
  a.ws_tick = w.total ? reinterpret_cast<int32_t*>(ws) : nullptr;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = ensure_smem_attribute<kMode, F>(dev);
  if (e != cudaSuccess) return e;
  const int64_t ctas = 2 * int64_t(a.T) * a.splits;
  int sms = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // The serving step's decodes merge in a second kernel unless the last CTAs
  // can merge behind others' work (more than a wave), or two splits fill most
  // of the GPU, which the second kernel would wait for (rows of 2048 entries,
  // second kernel against last CTA: 25 rows in 3 splits 29.7 us, 31.4; 19 in 4
  // 23.7, 27.6; 20 in 2 35.2, 35.9; 34 in 2 37.7, 36.4; 80 in 2 102.0, 94.2).
  const bool last_merges = ctas > sms || (a.splits == 2 && 4 * ctas >= 3 * sms);
  a.combine_in_kernel = a.T <= kTickRows &&  // rows that have counters
                        (overlapped<kMode, F>() ? last_merges : combine_in_kernel(ctas, a.splits, sms));
  if (overlapped<kMode, F>()) {
    e = launch_overlapped(sparse_mla_decode_kernel<kMode, F>, unsigned(ctas), Roles<F>::kThreads, kSmemBytes, s, a);
  } else {
    sparse_mla_decode_kernel<kMode, F><<<dim3(unsigned(ctas)), dim3(Roles<F>::kThreads), kSmemBytes, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || a.splits == 1 || a.T == 0 || a.combine_in_kernel) return e;
  // the separate split combine, scheduled while the decode grid drains
  const unsigned combine = unsigned(int64_t(a.T) * 2 * ((a.H + kCombHeads - 1) / kCombHeads));
  return launch_overlapped(split_combine_kernel, combine, kCombHeads * 32, 0, s,
                           static_cast<const uint16_t*>(a.ws_o), static_cast<const float*>(a.ws_ml),
                           a.out, a.lse, a.H, a.splits);
}

// Multiply-shift constants of the divisions by I, D and the block size.
void set_divisors(DecodeArgs& a) {
  a.div_I = make_fastdiv(uint32_t(a.interleave));
  a.div_D = make_fastdiv(uint32_t(a.D));
  a.div_bs = make_fastdiv(uint32_t(a.block_size));
}

// This translation unit's error word, ORed into *flags.
cudaError_t read_error_word(uint32_t* flags, bool clear) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_decode_error, sizeof(v));
  if (e != cudaSuccess) return e;
  *flags |= v;
  if (clear) {
    v = 0;
    e = cudaMemcpyToSymbol(g_decode_error, &v, sizeof(v));
  }
  return e;
}

}  // namespace

}  // namespace smla
