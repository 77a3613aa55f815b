// C ABI of the library: host-side argument checks, then one launch per call
// (the host-buffer form of the fused step: its copies and a launch per row
// group).  Every check runs before anything touches the GPU, so a rejected
// call has no side effect and needs no device.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/smla.h"
#include "smla_internal.h"
#include "smla_verify.h"

namespace {

inline bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

// A call's status.  A failed call also clears the error that the runtime keeps
// for the thread: the next call's launch asks for it and would report this one.
inline smla_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return SMLA_OK;
  cudaGetLastError();
  return SMLA_ERR_CUDA;
}

}  // namespace

static_assert(SMLA_NOALLOC_SCRATCH_BYTES == smla::kNoAllocScratchBytes,
              "header and library agree on the scratch size");

extern "C" {

const char* smla_status_string(smla_status status) {
  switch (status) {
    case SMLA_OK: return "SMLA_OK";
    case SMLA_ERR_INVALID_ARG: return "SMLA_ERR_INVALID_ARG";
    case SMLA_ERR_UNSUPPORTED: return "SMLA_ERR_UNSUPPORTED";
    case SMLA_ERR_WORKSPACE: return "SMLA_ERR_WORKSPACE";
    case SMLA_ERR_CUDA: return "SMLA_ERR_CUDA";
    default: return "SMLA_UNKNOWN_STATUS";
  }
}

smla_status smla_get_device_error(uint32_t* flags, int clear) {
  if (flags == nullptr) return SMLA_ERR_INVALID_ARG;
  *flags = 0;
  cudaError_t e = smla::index_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::decode_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::decode_fp4_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::decode_window_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::maps_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::cache_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::tree_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::matmul_error_word(flags, clear != 0);
  if (e == cudaSuccess) e = smla::tree_decode_error_word(flags, clear != 0);
  return from_cuda(e);
}

smla_status smla_dcp_filter_convert_index(
    const int32_t* req_id_per_token, const int32_t* block_table,
    int64_t bt_row_stride, int32_t bt_width, int32_t num_reqs,
    const int32_t* topk_global, int32_t T, int32_t K, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, int32_t* local_slots, int32_t* valid_count,
    void* stream) {
  if (T < 0 || K < 1 || D < 1 || rank < 0 || rank >= D || block_size < 1 ||
      interleave < 1 || num_reqs < 1 || bt_width < 1 || bt_row_stride < bt_width)
    return SMLA_ERR_INVALID_ARG;
  if (T == 0) return SMLA_OK;
  if (!req_id_per_token || !block_table || !topk_global || !local_slots)
    return SMLA_ERR_INVALID_ARG;
  if (misaligned(req_id_per_token, 4) || misaligned(block_table, 4) ||
      misaligned(topk_global, 4) || misaligned(local_slots, 4) ||
      (valid_count && misaligned(valid_count, 4)))
    return SMLA_ERR_INVALID_ARG;
  smla::IndexArgs a;
  a.req_id = req_id_per_token;
  a.block_table = block_table;
  a.bt_row_stride = bt_row_stride;
  a.bt_width = bt_width;
  a.num_reqs = num_reqs;
  a.topk = topk_global;
  a.T = T;
  a.K = K;
  a.D = D;
  a.rank = rank;
  a.block_size = block_size;
  a.interleave = interleave;
  a.local_slots = local_slots;
  a.valid_count = valid_count;
  return from_cuda(smla::launch_filter_convert(a, static_cast<cudaStream_t>(stream)));
}

size_t smla_decode_workspace_size(int32_t T, int32_t H, int32_t K) {
  if (T < 0 || H < 1 || H > SMLA_MAX_HEADS || K < 1) return 0;
  return smla::decode_workspace_bytes(T, H, K);
}

// Checks of the per-rank sparse decode's arguments, whatever the rows' format;
// fills `a` with everything but the workspace.
static smla_status slots_args(const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
                              const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
                              float sm_scale, uint16_t* out, float* lse, smla::DecodeArgs& a) {
  if (T < 0 || K < 1 || H < 1 || num_slots < 0 || !std::isfinite(sm_scale) ||
      !(sm_scale > 0.f))
    return SMLA_ERR_INVALID_ARG;
  if (H > SMLA_MAX_HEADS) return SMLA_ERR_UNSUPPORTED;
  if (T == 0) return SMLA_OK;
  if (!q || !kv_cache || !local_slots || !out || !lse) return SMLA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(kv_cache, 16) || misaligned(out, 16) ||
      misaligned(local_slots, 4) || misaligned(lse, 4))
    return SMLA_ERR_INVALID_ARG;
  a = smla::DecodeArgs{};
  a.q = q;
  a.kv = kv_cache;
  a.num_slots = num_slots;
  a.slots = local_slots;
  a.T = T;
  a.H = H;
  a.K = K;
  a.sm_scale = sm_scale;
  a.out = out;
  a.lse = lse;
  return SMLA_OK;
}

// Takes the caller's workspace of at least `need` bytes.
static smla_status take_workspace(void* workspace, size_t workspace_bytes, size_t need,
                                  smla::DecodeArgs& a) {
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || misaligned(workspace, 256)))
    return SMLA_ERR_WORKSPACE;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return SMLA_OK;
}

smla_status smla_sparse_mla_decode(
    const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
    const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
    float sm_scale, uint16_t* out, float* lse, void* workspace,
    size_t workspace_bytes, void* stream) {
  smla::DecodeArgs a;
  smla_status st =
      slots_args(q, kv_cache, num_slots, local_slots, T, H, K, sm_scale, out, lse, a);
  if (st != SMLA_OK || T == 0) return st;
  st = take_workspace(workspace, workspace_bytes, smla::decode_workspace_bytes(T, H, K), a);
  if (st != SMLA_OK) return st;
  return from_cuda(smla::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

// Entries of a row the serving step's decodes take (their split arithmetic is
// 32-bit).
constexpr int32_t kMaxEntries = 1 << 30;

size_t smla_fp4_decode_workspace_size(int32_t T, int32_t H, int32_t K) {
  if (T < 0 || H < 1 || H > SMLA_MAX_HEADS || K < 1 || K > kMaxEntries) return 0;
  return smla::fp4_decode_workspace_bytes(T, H, K);
}

smla_status smla_sparse_mla_decode_fp4(
    const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
    const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
    float sm_scale, uint16_t* out, float* lse, void* workspace,
    size_t workspace_bytes, void* stream) {
  smla::DecodeArgs a;
  smla_status st =
      slots_args(q, kv_cache, num_slots, local_slots, T, H, K, sm_scale, out, lse, a);
  if (st != SMLA_OK || T == 0) return st;
  if (K > kMaxEntries) return SMLA_ERR_UNSUPPORTED;
  st = take_workspace(workspace, workspace_bytes, smla_fp4_decode_workspace_size(T, H, K), a);
  if (st != SMLA_OK) return st;
  return from_cuda(smla::launch_decode_fp4(a, static_cast<cudaStream_t>(stream)));
}

smla_status smla_sparse_mla_decode_noalloc(
    const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
    const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
    float sm_scale, uint16_t* out, float* lse, void* stream) {
  smla::DecodeArgs a;
  const smla_status st =
      slots_args(q, kv_cache, num_slots, local_slots, T, H, K, sm_scale, out, lse, a);
  if (st != SMLA_OK || T == 0) return st;
  if (smla::decode_workspace_bytes(T, H, K) > SMLA_NOALLOC_SCRATCH_BYTES)
    return SMLA_ERR_WORKSPACE;
  return from_cuda(smla::launch_decode_noalloc(a, static_cast<cudaStream_t>(stream)));
}

// Checks of the fused step's arguments shared by its device and host forms;
// fills `a` with everything but the staging of q and the top-k ids.
static smla_status fused_args(
    const void* q, int32_t T, int32_t H, int32_t K, float sm_scale,
    const int32_t* req_id_per_token, const void* topk_global, int32_t num_reqs, int32_t D,
    int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, const void* out, const void* lse,
    smla::DecodeArgs& a) {
  if (T < 0 || K < 1 || H < 1 || D < 1 || block_size < 1 || interleave < 1 || num_reqs < 1 ||
      !std::isfinite(sm_scale) || !(sm_scale > 0.f))
    return SMLA_ERR_INVALID_ARG;
  if (H > SMLA_MAX_HEADS || D > SMLA_MAX_DCP) return SMLA_ERR_UNSUPPORTED;
  if (T == 0) return SMLA_OK;
  if (!q || !req_id_per_token || !topk_global || !out || !lse || !kv_caches ||
      !num_slots || !block_tables || !bt_row_strides || !bt_widths)
    return SMLA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) ||
      misaligned(req_id_per_token, 4) || misaligned(topk_global, 4))
    return SMLA_ERR_INVALID_ARG;
  a = smla::DecodeArgs{};
  for (int d = 0; d < D; ++d) {
    if (!kv_caches[d] || misaligned(kv_caches[d], 16) || num_slots[d] < 0 ||
        !block_tables[d] || misaligned(block_tables[d], 4) || bt_widths[d] < 1 ||
        bt_row_strides[d] < bt_widths[d])
      return SMLA_ERR_INVALID_ARG;
    a.pools[d] = kv_caches[d];
    a.pool_slots[d] = num_slots[d];
    a.bts[d] = block_tables[d];
    a.bt_stride[d] = bt_row_strides[d];
    a.bt_width[d] = bt_widths[d];
  }
  a.T = T;
  a.H = H;
  a.K = K;
  a.sm_scale = sm_scale;
  a.D = D;
  a.block_size = block_size;
  a.interleave = interleave;
  a.num_reqs = num_reqs;
  a.req_id = req_id_per_token;
  return SMLA_OK;
}

smla_status smla_dcp_sparse_mla_decode_fused(
    const uint16_t* q, int32_t T, int32_t H, int32_t K, float sm_scale,
    const int32_t* req_id_per_token, const int32_t* topk_global, int32_t num_reqs,
    int32_t D, int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  smla::DecodeArgs a;
  smla_status st =
      fused_args(q, T, H, K, sm_scale, req_id_per_token, topk_global, num_reqs, D, block_size,
                 interleave, kv_caches, num_slots, block_tables, bt_row_strides, bt_widths, out,
                 lse, a);
  if (st != SMLA_OK || T == 0) return st;
  st = take_workspace(workspace, workspace_bytes, smla::decode_workspace_bytes(T, H, K), a);
  if (st != SMLA_OK) return st;
  a.q = q;
  a.topk = topk_global;
  a.out = out;
  a.lse = lse;
  return from_cuda(smla::launch_decode_fused(a, static_cast<cudaStream_t>(stream)));
}

smla_status smla_dcp_sparse_mla_decode_fused_fp4(
    const uint16_t* q, int32_t T, int32_t H, int32_t K, float sm_scale,
    const int32_t* req_id_per_token, const int32_t* topk_global, int32_t num_reqs,
    int32_t D, int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  smla::DecodeArgs a;
  smla_status st =
      fused_args(q, T, H, K, sm_scale, req_id_per_token, topk_global, num_reqs, D, block_size,
                 interleave, kv_caches, num_slots, block_tables, bt_row_strides, bt_widths, out,
                 lse, a);
  if (st != SMLA_OK || T == 0) return st;
  if (K > kMaxEntries) return SMLA_ERR_UNSUPPORTED;
  st = take_workspace(workspace, workspace_bytes, smla_fp4_decode_workspace_size(T, H, K), a);
  if (st != SMLA_OK) return st;
  a.q = q;
  a.topk = topk_global;
  a.out = out;
  a.lse = lse;
  return from_cuda(smla::launch_decode_fused_fp4(a, static_cast<cudaStream_t>(stream)));
}

smla_status smla_dcp_sparse_mla_decode_fused_host(
    const uint16_t* q_host, const int32_t* topk_host, uint16_t* out_host, float* lse_host,
    uint16_t* q_dev, int32_t* topk_dev, uint16_t* out_dev, float* lse_dev,
    int32_t T, int32_t H, int32_t K, float sm_scale, const int32_t* req_id_per_token,
    int32_t num_reqs, int32_t D, int32_t block_size, int32_t interleave,
    const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides,
    const int32_t* bt_widths, void* workspace, size_t workspace_bytes, int32_t chunks,
    void* stream) {
  smla::DecodeArgs a;
  smla_status st =
      fused_args(q_dev, T, H, K, sm_scale, req_id_per_token, topk_dev, num_reqs, D, block_size,
                 interleave, kv_caches, num_slots, block_tables, bt_row_strides, bt_widths,
                 out_dev, lse_dev, a);
  if (st != SMLA_OK) return st;
  if (chunks < 1 || chunks > SMLA_MAX_HOST_CHUNKS) return SMLA_ERR_INVALID_ARG;
  if (T == 0) return SMLA_OK;
  if (!q_host || !topk_host || !out_host || !lse_host) return SMLA_ERR_INVALID_ARG;
  const int groups = chunks < T ? chunks : T;
  if (groups > 1 && K > smla::kDecodeMaxList) return SMLA_ERR_UNSUPPORTED;
  if (groups == 1) {
    const size_t need = smla::decode_workspace_bytes(T, H, K);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                     misaligned(workspace, 256)))
      return SMLA_ERR_WORKSPACE;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
  }
  a.q = q_dev;
  a.topk = topk_dev;
  a.out = out_dev;
  a.lse = lse_dev;
  smla::HostBuffers h{q_host, topk_host, out_host, lse_host, q_dev, topk_dev};
  return from_cuda(smla::launch_fused_host(a, h, groups, static_cast<cudaStream_t>(stream)));
}

// Raw entries per row of the dense decode: positions 0..max_ctx-1, or the
// largest count of them one rank holds.
static int32_t dense_entries(int32_t max_ctx, int32_t D, int32_t interleave, int32_t rank) {
  if (rank < 0) return max_ctx;
  const int64_t id = int64_t(interleave) * D;
  const int64_t held = ((int64_t(max_ctx) + id - 1) / id) * interleave;
  return int32_t(held < INT32_MAX ? held : INT32_MAX);
}

size_t smla_dense_decode_workspace_size(int32_t T, int32_t H, int32_t max_ctx, int32_t D,
                                        int32_t interleave, int32_t rank) {
  if (T < 0 || H < 1 || H > SMLA_MAX_HEADS || max_ctx < 1 || D < 1 || interleave < 1 ||
      rank < -1 || rank >= D)
    return 0;
  return smla::decode_workspace_bytes(T, H, dense_entries(max_ctx, D, interleave, rank));
}

// Checks of the dense and windowed decode's arguments; fills `a` with
// everything but K and the workspace.
static smla_status generated_args(
    const uint16_t* q, int32_t B, int32_t S, int32_t H, float sm_scale, const int32_t* ctx_lens,
    int32_t max_ctx, int32_t D, int32_t rank, int32_t block_size, int32_t interleave,
    const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides, const int32_t* bt_widths,
    uint16_t* out, float* lse, smla::DecodeArgs& a) {
  if (B < 0 || S < 1 || H < 1 || max_ctx < 1 || D < 1 || rank < -1 || rank >= D ||
      block_size < 1 || interleave < 1 || !std::isfinite(sm_scale) || !(sm_scale > 0.f))
    return SMLA_ERR_INVALID_ARG;
  if (H > SMLA_MAX_HEADS || D > SMLA_MAX_DCP) return SMLA_ERR_UNSUPPORTED;
  if (int64_t(B) * S > INT32_MAX) return SMLA_ERR_INVALID_ARG;
  if (B == 0) return SMLA_OK;
  if (!q || !ctx_lens || !out || !lse || !kv_caches || !num_slots || !block_tables ||
      !bt_row_strides || !bt_widths)
    return SMLA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(ctx_lens, 4))
    return SMLA_ERR_INVALID_ARG;
  a = smla::DecodeArgs{};
  for (int d = 0; d < D; ++d) {
    const bool used = rank < 0 || d == rank;
    if (used && (!kv_caches[d] || misaligned(kv_caches[d], 16) || num_slots[d] < 0 ||
                 !block_tables[d] || misaligned(block_tables[d], 4) || bt_widths[d] < 1 ||
                 bt_row_strides[d] < bt_widths[d]))
      return SMLA_ERR_INVALID_ARG;
    a.pools[d] = used ? kv_caches[d] : nullptr;
    a.pool_slots[d] = used ? num_slots[d] : 0;
    a.bts[d] = used ? block_tables[d] : nullptr;
    a.bt_stride[d] = used ? bt_row_strides[d] : 0;
    a.bt_width[d] = used ? bt_widths[d] : 0;
  }
  a.q = q;
  a.T = B * S;
  a.H = H;
  a.sm_scale = sm_scale;
  a.out = out;
  a.lse = lse;
  a.D = D;
  a.block_size = block_size;
  a.interleave = interleave;
  a.num_reqs = B;
  a.ctx_lens = ctx_lens;
  a.S = S;
  a.dense_rank = rank;
  a.max_ctx = max_ctx;
  return SMLA_OK;
}

smla_status smla_dcp_dense_mla_decode(
    const uint16_t* q, int32_t B, int32_t S, int32_t H, float sm_scale,
    const int32_t* ctx_lens, int32_t max_ctx, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  smla::DecodeArgs a;
  smla_status st = generated_args(q, B, S, H, sm_scale, ctx_lens, max_ctx, D, rank, block_size,
                                  interleave, kv_caches, num_slots, block_tables, bt_row_strides,
                                  bt_widths, out, lse, a);
  if (st != SMLA_OK || B == 0) return st;
  a.K = dense_entries(max_ctx, D, interleave, rank);
  st = take_workspace(workspace, workspace_bytes, smla::decode_workspace_bytes(a.T, H, a.K), a);
  if (st != SMLA_OK) return st;
  return from_cuda(smla::launch_decode_dense(a, static_cast<cudaStream_t>(stream)));
}

// The most positions of a run of n that the row's raw entries cover: all of
// them, or what one rank holds of a run that begins with its share.
static int64_t held_at_most(int32_t n, int32_t D, int32_t interleave, int32_t rank) {
  if (rank < 0) return n;
  const int64_t round = int64_t(interleave) * D;
  const int64_t rest = n % round;
  return n / round * interleave + (rest < interleave ? rest : interleave);
}

// Raw entries per row of the windowed decode: the sinks and the window, and
// never more than the context.
static int32_t window_entries(int32_t max_ctx, int32_t window, int32_t sinks, int32_t D,
                              int32_t interleave, int32_t rank) {
  const int64_t all = held_at_most(max_ctx, D, interleave, rank);
  const int64_t kept =
      held_at_most(window < max_ctx ? window : max_ctx, D, interleave, rank) +
      held_at_most(sinks < max_ctx ? sinks : max_ctx, D, interleave, rank);
  return int32_t(kept < all ? kept : all);
}

// The windowed decode's positions and rounds of I*D positions are 32-bit.
static bool window_unsupported(int32_t max_ctx, int32_t D, int32_t interleave) {
  return max_ctx > kMaxEntries || int64_t(interleave) * D > INT32_MAX;
}

size_t smla_window_decode_workspace_size(int32_t T, int32_t H, int32_t max_ctx, int32_t window,
                                         int32_t sinks, int32_t D, int32_t interleave,
                                         int32_t rank) {
  if (T < 0 || H < 1 || H > SMLA_MAX_HEADS || max_ctx < 1 || window < 1 || sinks < 0 || D < 1 ||
      interleave < 1 || rank < -1 || rank >= D || window_unsupported(max_ctx, D, interleave))
    return 0;
  return smla::window_decode_workspace_bytes(
      T, H, window_entries(max_ctx, window, sinks, D, interleave, rank));
}

smla_status smla_dcp_window_mla_decode(
    const uint16_t* q, int32_t B, int32_t S, int32_t H, float sm_scale,
    const int32_t* ctx_lens, int32_t max_ctx, int32_t window, int32_t sinks, int32_t D,
    int32_t rank, int32_t block_size, int32_t interleave, int32_t format,
    const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides, const int32_t* bt_widths,
    uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 1 || sinks < 0 || (format != SMLA_CACHE_FP8 && format != SMLA_CACHE_FP4))
    return SMLA_ERR_INVALID_ARG;
  smla::DecodeArgs a;
  smla_status st = generated_args(q, B, S, H, sm_scale, ctx_lens, max_ctx, D, rank, block_size,
                                  interleave, kv_caches, num_slots, block_tables, bt_row_strides,
                                  bt_widths, out, lse, a);
  if (st != SMLA_OK || B == 0) return st;
  if (window_unsupported(max_ctx, D, interleave)) return SMLA_ERR_UNSUPPORTED;
  a.window = window;
  a.sinks = sinks;
  a.K = window_entries(max_ctx, window, sinks, D, interleave, rank);
  st = take_workspace(workspace, workspace_bytes, smla::window_decode_workspace_bytes(a.T, H, a.K), a);
  if (st != SMLA_OK) return st;
  return from_cuda(smla::launch_decode_window(a, format == SMLA_CACHE_FP4,
                                              static_cast<cudaStream_t>(stream)));
}

smla_status smla_dcp_step_maps(
    const int32_t* ctx_lens, const int32_t* q_lens, int32_t B, int32_t T, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, const int32_t* free_blocks, int32_t num_free,
    int32_t* block_table, int64_t bt_row_stride, int32_t bt_width, int32_t* row_start,
    int32_t* req_id, int32_t* positions, int32_t* slots, int32_t* local_lens,
    int32_t* blocks_taken, void* stream) {
  if (B < 0 || T < 0 || D < 1 || rank < 0 || rank >= D || block_size < 1 || interleave < 1 ||
      num_free < 0 || bt_width < 1 || bt_row_stride < bt_width)
    return SMLA_ERR_INVALID_ARG;
  if (B > SMLA_MAX_STEP_REQS) return SMLA_ERR_UNSUPPORTED;
  if (B == 0 && T == 0) return SMLA_OK;
  if ((B > 0 && (!ctx_lens || !q_lens || !block_table)) || (T > 0 && !slots) ||
      (num_free > 0 && !free_blocks))
    return SMLA_ERR_INVALID_ARG;
  for (const int32_t* p : {ctx_lens, q_lens, free_blocks, static_cast<const int32_t*>(block_table),
                           static_cast<const int32_t*>(row_start),
                           static_cast<const int32_t*>(req_id),
                           static_cast<const int32_t*>(positions),
                           static_cast<const int32_t*>(slots),
                           static_cast<const int32_t*>(local_lens),
                           static_cast<const int32_t*>(blocks_taken)})
    if (misaligned(p, 4)) return SMLA_ERR_INVALID_ARG;
  smla::MapsArgs a{};
  a.ctx_lens = ctx_lens;
  a.q_lens = q_lens;
  a.B = B;
  a.T = T;
  a.D = D;
  a.rank = rank;
  a.block_size = block_size;
  a.interleave = interleave;
  a.free_blocks = free_blocks;
  a.num_free = num_free;
  a.block_table = block_table;
  a.bt_row_stride = bt_row_stride;
  a.bt_width = bt_width;
  a.row_start = row_start;
  a.req_id = req_id;
  a.positions = positions;
  a.slots = slots;
  a.local_lens = local_lens;
  a.blocks_taken = blocks_taken;
  return from_cuda(smla::launch_step_maps(a, static_cast<cudaStream_t>(stream)));
}

smla_status smla_mla_cache_write(
    const uint16_t* kv, int64_t kv_row_stride, int32_t T, const uint16_t* gamma, float eps,
    const int32_t* positions, const float* cos_sin, int32_t num_positions, int32_t rope_pairs,
    const int32_t* slots, int32_t format, uint8_t* kv_cache, int64_t num_slots, void* stream) {
  if (T < 0 || num_slots < 0 || (format != SMLA_CACHE_FP8 && format != SMLA_CACHE_FP4) ||
      kv_row_stride < SMLA_QK_DIM || kv_row_stride % 8 != 0 ||
      (gamma && !(std::isfinite(eps) && eps > 0.f)) || (cos_sin && num_positions < 1))
    return SMLA_ERR_INVALID_ARG;
  if (T == 0) return SMLA_OK;
  if (!kv || !slots || !kv_cache || (cos_sin && !positions)) return SMLA_ERR_INVALID_ARG;
  if (misaligned(kv, 16) || misaligned(gamma, 16) || misaligned(kv_cache, 16) ||
      misaligned(slots, 4) || misaligned(positions, 4) || misaligned(cos_sin, 4))
    return SMLA_ERR_INVALID_ARG;
  smla::CacheWriteArgs a{};
  a.kv = kv;
  a.kv_row_stride = kv_row_stride;
  a.T = T;
  a.gamma = gamma;
  a.eps = eps;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.num_positions = num_positions;
  a.rope_pairs = rope_pairs != 0;
  a.slots = slots;
  a.kv_cache = kv_cache;
  a.num_slots = num_slots;
  return from_cuda(smla::launch_cache_write(a, format == SMLA_CACHE_FP4,
                                            static_cast<cudaStream_t>(stream)));
}

smla_status smla_mla_cache_gather(const uint8_t* kv_cache, int64_t num_slots, int32_t format,
                                  const int32_t* slots, int32_t N, void* out,
                                  int64_t out_row_stride, int32_t out_fp32, void* stream) {
  if (N < 0 || num_slots < 0 || (format != SMLA_CACHE_FP8 && format != SMLA_CACHE_FP4) ||
      out_row_stride < SMLA_QK_DIM || out_row_stride % (out_fp32 ? 4 : 8) != 0)
    return SMLA_ERR_INVALID_ARG;
  if (N == 0) return SMLA_OK;
  if (!kv_cache || !slots || !out) return SMLA_ERR_INVALID_ARG;
  if (misaligned(kv_cache, 16) || misaligned(slots, 4) || misaligned(out, 16))
    return SMLA_ERR_INVALID_ARG;
  smla::CacheGatherArgs a{};
  a.kv_cache = kv_cache;
  a.num_slots = num_slots;
  a.slots = slots;
  a.N = N;
  a.out = out;
  a.out_row_stride = out_row_stride;
  return from_cuda(smla::launch_cache_gather(a, format == SMLA_CACHE_FP4, out_fp32 != 0,
                                             static_cast<cudaStream_t>(stream)));
}

static_assert(SMLA_MAX_TREE_NODES == smla::kMaxTreeNodes, "header and kernels agree on a tree's size");

smla_status smla_tree_maps(const int32_t* parents, const int32_t* row_start,
                           const int32_t* prefix_lens, int32_t B, int32_t T, int32_t max_nodes,
                           uint64_t* masks, int32_t* positions, void* stream) {
  if (B < 0 || T < 0 || max_nodes < 1) return SMLA_ERR_INVALID_ARG;
  if (max_nodes > SMLA_MAX_TREE_NODES) return SMLA_ERR_UNSUPPORTED;
  if (T == 0) return SMLA_OK;
  if (!parents || !row_start || !masks || (positions && B > 0 && !prefix_lens)) return SMLA_ERR_INVALID_ARG;
  if (misaligned(parents, 4) || misaligned(row_start, 4) || misaligned(prefix_lens, 4) ||
      misaligned(masks, 8) || misaligned(positions, 4))
    return SMLA_ERR_INVALID_ARG;
  const smla::TreeMapsArgs a = {parents, row_start, prefix_lens, B, T, max_nodes, masks, positions};
  return from_cuda(smla::launch_tree_maps(a, static_cast<cudaStream_t>(stream)));
}

// The most keys of a request: its prefix, or one rank's share of it, and its
// tree's nodes.
static int64_t tree_keys(int32_t max_prefix, int32_t max_nodes, int32_t D, int32_t interleave, int32_t rank) {
  return held_at_most(max_prefix, D, interleave, rank) + max_nodes;
}

static bool tree_unsupported(int32_t H, int32_t max_prefix, int32_t max_nodes, int32_t D) {
  return H > SMLA_MAX_HEADS || D > SMLA_MAX_DCP || max_prefix > kMaxEntries ||
         max_nodes > SMLA_MAX_TREE_NODES;
}

size_t smla_tree_decode_workspace_size(int32_t T, int32_t H, int32_t B, int32_t max_prefix,
                                       int32_t max_nodes, int32_t D, int32_t interleave, int32_t rank) {
  if (T < 0 || H < 1 || B < 0 || max_prefix < 0 || max_nodes < 1 || D < 1 || interleave < 1 || rank < -1 ||
      rank >= D || tree_unsupported(H, max_prefix, max_nodes, D))
    return 0;
  return smla::tree_decode_most_workspace_bytes(T, B, H, tree_keys(max_prefix, max_nodes, D, interleave, rank));
}

// Both forms; window 0: the whole prefix.
static smla_status tree_decode(
    const uint16_t* q, int32_t T, int32_t H, float sm_scale, const int32_t* row_start,
    const int32_t* prefix_lens, const int32_t* positions, int32_t B, int32_t max_prefix, const uint64_t* masks,
    int32_t max_nodes, int32_t window, int32_t sinks, const int32_t* const* draft_slots, int32_t D, int32_t rank, int32_t block_size, int32_t interleave,
    int32_t format, const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides, const int32_t* bt_widths,
    uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || H < 1 || B < 0 || max_prefix < 0 || max_nodes < 1 || D < 1 || rank < -1 || rank >= D ||
      block_size < 1 || interleave < 1 || (format != SMLA_CACHE_FP8 && format != SMLA_CACHE_FP4) ||
      !std::isfinite(sm_scale) || !(sm_scale > 0.f))
    return SMLA_ERR_INVALID_ARG;
  if (tree_unsupported(H, max_prefix, max_nodes, D) || int64_t(T) * H > INT32_MAX)
    return SMLA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return SMLA_OK;
  if (!q || !row_start || !prefix_lens || !masks || !draft_slots || !kv_caches || !num_slots ||
      !block_tables || !bt_row_strides || !bt_widths || !out || !lse)
    return SMLA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(row_start, 4) ||
      misaligned(prefix_lens, 4) || misaligned(masks, 8) ||
      (window > 0 && (!positions || misaligned(positions, 4))))
    return SMLA_ERR_INVALID_ARG;
  smla::TreeDecodeArgs a{};
  for (int d = 0; d < D; ++d) {
    if (rank >= 0 && d != rank) continue;
    if (!kv_caches[d] || misaligned(kv_caches[d], 16) || num_slots[d] < 0 || !block_tables[d] ||
        misaligned(block_tables[d], 4) || bt_widths[d] < 1 || bt_row_strides[d] < bt_widths[d] ||
        !draft_slots[d] || misaligned(draft_slots[d], 4))
      return SMLA_ERR_INVALID_ARG;
    a.pools[d] = kv_caches[d];
    a.pool_slots[d] = num_slots[d];
    a.bts[d] = block_tables[d];
    a.bt_stride[d] = bt_row_strides[d];
    a.bt_width[d] = bt_widths[d];
    a.draft_slots[d] = draft_slots[d];
  }
  // a window that no node's position reaches past shuts out nothing
  if (int64_t(window) >= int64_t(max_prefix) + max_nodes) window = 0;
  const int64_t keys = window > 0 ? int64_t(window_entries(max_prefix, window, sinks, D, interleave, rank)) + max_nodes
                                  : tree_keys(max_prefix, max_nodes, D, interleave, rank);
  const size_t need = smla::tree_decode_workspace_bytes(T, B, H, keys);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || misaligned(workspace, 256)))
    return SMLA_ERR_WORKSPACE;
  a.q = q;
  a.T = T;
  a.B = B;
  a.H = H;
  a.sm_scale = sm_scale;
  a.row_start = row_start;
  a.prefix_lens = prefix_lens;
  a.max_prefix = max_prefix;
  a.masks = masks;
  a.max_nodes = max_nodes;
  a.mask_words = (max_nodes + 63) / 64;
  a.positions = positions;
  a.window = window;
  a.sinks = sinks;
  a.D = D;
  a.rank = rank;
  a.block_size = block_size;
  a.interleave = interleave;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return from_cuda(smla::launch_tree_decode(a, keys, format == SMLA_CACHE_FP4, static_cast<cudaStream_t>(stream)));
}

smla_status smla_dcp_tree_mla_decode(
    const uint16_t* q, int32_t T, int32_t H, float sm_scale, const int32_t* row_start,
    const int32_t* prefix_lens, int32_t B, int32_t max_prefix, const uint64_t* masks, int32_t max_nodes,
    const int32_t* const* draft_slots, int32_t D, int32_t rank, int32_t block_size, int32_t interleave,
    int32_t format, const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides, const int32_t* bt_widths,
    uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return tree_decode(q, T, H, sm_scale, row_start, prefix_lens, nullptr, B, max_prefix, masks, max_nodes, 0, 0,
                     draft_slots, D, rank, block_size, interleave, format, kv_caches, num_slots, block_tables,
                     bt_row_strides, bt_widths, out, lse, workspace, workspace_bytes, stream);
}

smla_status smla_dcp_tree_window_mla_decode(
    const uint16_t* q, int32_t T, int32_t H, float sm_scale, const int32_t* row_start,
    const int32_t* prefix_lens, const int32_t* positions, int32_t B, int32_t max_prefix, const uint64_t* masks,
    int32_t max_nodes, int32_t window, int32_t sinks, const int32_t* const* draft_slots, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, int32_t format, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables, const int64_t* bt_row_strides,
    const int32_t* bt_widths, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 1 || sinks < 0) return SMLA_ERR_INVALID_ARG;
  return tree_decode(q, T, H, sm_scale, row_start, prefix_lens, positions, B, max_prefix, masks, max_nodes, window,
                     sinks, draft_slots, D, rank, block_size, interleave, format, kv_caches, num_slots, block_tables,
                     bt_row_strides, bt_widths, out, lse, workspace, workspace_bytes, stream);
}

smla_status smla_tree_accept(const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                             const int32_t* row_start, int32_t B, int32_t T, int32_t* accepted,
                             int32_t* rows, int32_t* next_tokens, void* stream) {
  if (B < 0 || T < 0) return SMLA_ERR_INVALID_ARG;
  if (B > SMLA_MAX_STEP_REQS) return SMLA_ERR_UNSUPPORTED;
  if (B == 0 && T == 0) return SMLA_OK;
  if ((T > 0 && (!parents || !tokens || !targets || !rows)) || !row_start ||
      (B > 0 && (!accepted || !next_tokens)))
    return SMLA_ERR_INVALID_ARG;
  if (misaligned(parents, 4) || misaligned(tokens, 4) || misaligned(targets, 4) ||
      misaligned(row_start, 4) || misaligned(accepted, 4) || misaligned(rows, 4) ||
      misaligned(next_tokens, 4))
    return SMLA_ERR_INVALID_ARG;
  const smla::TreeAcceptArgs a = {parents, tokens, targets, row_start, B, T, accepted, rows, next_tokens};
  return from_cuda(smla::launch_tree_accept(a, static_cast<cudaStream_t>(stream)));
}

smla_status smla_mla_cache_move(int32_t format, uint8_t* kv_cache, int64_t num_slots,
                                const int32_t* rows, int32_t N, const int32_t* src_slots, int32_t T,
                                const int32_t* dst_slots, void* stream) {
  if (N < 0 || T < 0 || num_slots < 0 || (format != SMLA_CACHE_FP8 && format != SMLA_CACHE_FP4))
    return SMLA_ERR_INVALID_ARG;
  if (N == 0) return SMLA_OK;
  if (!kv_cache || !rows || (T > 0 && !src_slots) || !dst_slots) return SMLA_ERR_INVALID_ARG;
  if (misaligned(kv_cache, 16) || misaligned(rows, 4) || misaligned(src_slots, 4) ||
      misaligned(dst_slots, 4))
    return SMLA_ERR_INVALID_ARG;
  const smla::CacheMoveArgs a = {kv_cache, num_slots, rows, N, src_slots, T, dst_slots};
  return from_cuda(smla::launch_cache_move(a, format == SMLA_CACHE_FP4, static_cast<cudaStream_t>(stream)));
}

// Whether an array's entries lie apart: with the dimensions in the order of
// their strides, each steps past all that the ones before it span.
struct Dim {
  int64_t count, stride;
};
static bool apart(Dim x, Dim y, Dim z) {
  Dim d[3] = {x, y, z};
  std::sort(d, d + 3, [](const Dim& p, const Dim& q) { return p.stride < q.stride; });
  int64_t span = 1;
  for (const Dim& e : d) {
    if (e.count <= 1) continue;
    if (e.stride < span) return false;
    const bool fits = e.count - 1 <= (INT64_MAX - span) / e.stride;
    span = fits ? (e.count - 1) * e.stride + span : INT64_MAX;
  }
  return true;
}

smla_status smla_fp8_quantise(const uint16_t* x, int64_t x_batch_stride, int64_t x_row_stride, int32_t G,
                              int32_t M, int32_t K, uint8_t* codes, int64_t codes_batch_stride,
                              int64_t codes_row_stride, float* scales, int64_t scales_batch_stride,
                              int64_t scales_row_stride, int64_t scales_col_stride, void* stream) {
  if (G < 0 || M < 0 || K < 1 || x_batch_stride < 0 || x_row_stride < 0 || codes_batch_stride < 0 ||
      codes_row_stride < 0 || scales_batch_stride < 0 || scales_row_stride < 0 || scales_col_stride < 0)
    return SMLA_ERR_INVALID_ARG;
  if (G == 0 || M == 0) return SMLA_OK;
  if (!x || !codes || !scales || misaligned(x, 2) || misaligned(scales, 4)) return SMLA_ERR_INVALID_ARG;
  if (!apart({K, 1}, {M, codes_row_stride}, {G, codes_batch_stride}) ||
      !apart({(int64_t(K) + 127) / 128, scales_col_stride}, {M, scales_row_stride}, {G, scales_batch_stride}))
    return SMLA_ERR_INVALID_ARG;
  const smla::QuantiseArgs a = {x, {x_batch_stride, x_row_stride, 1}, G, M, K,
                                codes, {codes_batch_stride, codes_row_stride, 1},
                                scales, {scales_batch_stride, scales_row_stride, scales_col_stride}};
  return from_cuda(smla::launch_fp8_quantise(a, static_cast<cudaStream_t>(stream)));
}

// Strides of a batch of code matrices that the tensor maps take.
static smla_status code_strides(const uint8_t* p, int64_t batch, int64_t row, int32_t G, int32_t K) {
  if (!p || misaligned(p, 16) || row < K || row % 16 != 0 || (G > 1 && (batch < 1 || batch % 16 != 0)))
    return SMLA_ERR_INVALID_ARG;
  constexpr int64_t kMost = int64_t(1) << 40;
  return row >= kMost || (G > 1 && batch >= kMost) ? SMLA_ERR_UNSUPPORTED : SMLA_OK;
}

smla_status smla_fp8_matmul(const uint8_t* a, int64_t a_batch_stride, int64_t a_row_stride,
                            const float* a_scales, int64_t a_scales_batch_stride,
                            int64_t a_scales_row_stride, int64_t a_scales_col_stride, const uint8_t* b,
                            int64_t b_batch_stride, int64_t b_row_stride, const float* b_scales,
                            int64_t b_scales_batch_stride, int64_t b_scales_row_stride,
                            int64_t b_scales_col_stride, int32_t G, int32_t M, int32_t N, int32_t K,
                            void* out, int64_t out_batch_stride, int64_t out_row_stride, int32_t out_fp32,
                            void* stream) {
  if (G < 0 || M < 0 || N < 0 || K < 1 || a_scales_batch_stride < 0 || a_scales_row_stride < 0 ||
      a_scales_col_stride < 0 || b_scales_batch_stride < 0 || b_scales_row_stride < 0 ||
      b_scales_col_stride < 0 || out_batch_stride < 0 || out_row_stride < 0)
    return SMLA_ERR_INVALID_ARG;
  if (G == 0 || M == 0 || N == 0) return SMLA_OK;
  smla_status st = code_strides(a, a_batch_stride, a_row_stride, G, K);
  if (st == SMLA_OK) st = code_strides(b, b_batch_stride, b_row_stride, G, K);
  if (st != SMLA_OK) return st;
  if (!a_scales || !b_scales || !out || misaligned(a_scales, 4) || misaligned(b_scales, 4) ||
      misaligned(out, out_fp32 ? 4 : 2) || (M > 1 && out_row_stride < 1) || (G > 1 && out_batch_stride < 1))
    return SMLA_ERR_INVALID_ARG;
  if (int64_t(G) * (int64_t(M) / 16 + 1) * (int64_t(N) / 128 + 1) > (int64_t(1) << 27))
    return SMLA_ERR_UNSUPPORTED;
  if (!apart({N, 1}, {M, out_row_stride}, {G, out_batch_stride})) return SMLA_ERR_INVALID_ARG;
  smla::MatmulArgs m{};
  m.a = a;
  m.as = {a_batch_stride, a_row_stride, 1};
  m.a_scales = a_scales;
  m.ass = {a_scales_batch_stride, a_scales_row_stride, a_scales_col_stride};
  m.b = b;
  m.bs = {b_batch_stride, b_row_stride, 1};
  m.b_scales = b_scales;
  m.bss = {b_scales_batch_stride, b_scales_row_stride, b_scales_col_stride};
  m.G = G;
  m.M = M;
  m.N = N;
  m.K = K;
  m.out = out;
  m.os = {out_batch_stride, out_row_stride, 1};
  m.out_fp32 = out_fp32 != 0;
  return from_cuda(smla::launch_fp8_matmul(m, static_cast<cudaStream_t>(stream)));
}

size_t smla_topk_select_workspace_size(int32_t T, int32_t L, int32_t K) {
  if (T < 0 || L < 0 || K < 1 || K > SMLA_MAX_TOPK) return 0;
  return smla::topk_workspace_bytes(T, L, K);
}

smla_status smla_topk_select(const float* scores, int64_t row_stride, int32_t L,
                             const int32_t* n_cand, int32_t T, int32_t K, int32_t D,
                             int32_t rank, int32_t interleave, int32_t* out_ids,
                             float* out_scores, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (T < 0 || L < 0 || row_stride < L || D < 1 || rank < 0 || rank >= D || interleave < 1)
    return SMLA_ERR_INVALID_ARG;
  if (K < 1 || K > SMLA_MAX_TOPK) return SMLA_ERR_UNSUPPORTED;
  if (T == 0) return SMLA_OK;
  if (!scores || !n_cand || !out_ids) return SMLA_ERR_INVALID_ARG;
  if (misaligned(scores, 4) || misaligned(n_cand, 4) || misaligned(out_ids, 4) ||
      (out_scores && misaligned(out_scores, 4)))
    return SMLA_ERR_INVALID_ARG;
  const size_t need = smla::topk_workspace_bytes(T, L, K);
  if (workspace != nullptr && (workspace_bytes < need || misaligned(workspace, 16)))
    return SMLA_ERR_WORKSPACE;
  smla::TopkArgs a{};
  a.scores = scores;
  a.n_cand = n_cand;
  a.row_stride = row_stride;
  a.L = L;
  a.T = T;
  a.K = K;
  a.D = D;
  a.rank = rank;
  a.interleave = interleave;
  a.out_ids = out_ids;
  a.out_scores = out_scores;
  return from_cuda(smla::launch_topk_select(a, need > 0 ? workspace : nullptr,
                                            static_cast<cudaStream_t>(stream)));
}

smla_status smla_dcp_topk_merge(const int32_t* cand_ids, const float* cand_scores,
                                int64_t row_stride, int32_t M, int32_t T, int32_t K,
                                int32_t* out_ids, float* out_scores, void* stream) {
  if (T < 0 || M < 0 || row_stride < M) return SMLA_ERR_INVALID_ARG;
  if (K < 1 || K > SMLA_MAX_TOPK) return SMLA_ERR_UNSUPPORTED;
  if (T == 0) return SMLA_OK;
  if (!cand_ids || !cand_scores || !out_ids) return SMLA_ERR_INVALID_ARG;
  if (misaligned(cand_ids, 4) || misaligned(cand_scores, 4) || misaligned(out_ids, 4) ||
      (out_scores && misaligned(out_scores, 4)))
    return SMLA_ERR_INVALID_ARG;
  smla::TopkArgs a{};
  a.scores = cand_scores;
  a.cand_ids = cand_ids;
  a.row_stride = row_stride;
  a.M = M;
  a.T = T;
  a.K = K;
  a.D = 1;
  a.interleave = 1;
  a.out_ids = out_ids;
  a.out_scores = out_scores;
  return from_cuda(smla::launch_topk_merge(a, static_cast<cudaStream_t>(stream)));
}

smla_status smla_dcp_lse_merge(const uint16_t* const* outs,
                               const float* const* lses, int32_t D, int32_t T,
                               int32_t H, uint16_t* out, float* lse,
                               void* stream) {
  if (D < 1 || T < 0 || H < 1) return SMLA_ERR_INVALID_ARG;
  if (D > SMLA_MAX_DCP) return SMLA_ERR_UNSUPPORTED;
  if (T == 0) return SMLA_OK;
  if (!outs || !lses || !out || !lse) return SMLA_ERR_INVALID_ARG;
  if (misaligned(out, 16) || misaligned(lse, 4)) return SMLA_ERR_INVALID_ARG;
  smla::MergeArgs a;
  for (int d = 0; d < D; ++d) {
    if (!outs[d] || !lses[d] || misaligned(outs[d], 16) || misaligned(lses[d], 4))
      return SMLA_ERR_INVALID_ARG;
    a.outs[d] = outs[d];
    a.lses[d] = lses[d];
  }
  for (int d = D; d < smla::kMaxMerge; ++d) {
    a.outs[d] = nullptr;
    a.lses[d] = nullptr;
  }
  a.D = D;
  a.T = T;
  a.H = H;
  a.out = out;
  a.lse = lse;
  return from_cuda(smla::launch_merge(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
