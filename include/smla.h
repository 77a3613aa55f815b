/*
 * smla.h -- C ABI of the GB300 sparse MLA decode library under
 * decode-context-parallel (DCP).
 *
 * The hot path has three steps, one call each:
 *
 *   1. smla_dcp_filter_convert_index  global top-k ids -> this rank's slots
 *   2. smla_sparse_mla_decode         attention over the packed fp8 cache,
 *                                     returning out and the softmax LSE
 *   3. smla_dcp_lse_merge             LSE-weighted merge of D partials
 *
 * and three more entry points run it differently:
 *
 *   smla_dcp_sparse_mla_decode_fused  steps 1-3 for D pools held by one GPU,
 *                                     in a single launch
 *   smla_dcp_sparse_mla_decode_fused_host
 *                                     the same from and to pinned host
 *                                     memory, copies overlapping the decode
 *   smla_sparse_mla_decode_noalloc    step 2 with library-owned split-K
 *                                     scratch (no workspace argument)
 *
 * and the dense form of the decode (every cached position of a request's
 * causal context instead of a top-k list):
 *
 *   smla_dcp_dense_mla_decode         per rank or merged over D pools
 *
 * and the step before the path, the global top-k of indexer scores:
 *
 *   smla_topk_select                  per row (per rank: as global ids)
 *   smla_dcp_topk_merge               top-k of the ranks' candidates
 *
 * and the rest of a serving step, over the 8-bit or a 4-bit cache:
 *
 *   smla_dcp_step_maps                request ids, positions, slots and new
 *                                     block-table entries from the requests'
 *                                     lengths
 *   smla_mla_cache_write              latent norm, rotary positions,
 *                                     quantisation and scatter into the cache
 *   smla_mla_cache_gather             cache rows back to bf16 or fp32
 *   smla_sparse_mla_decode_fp4, smla_dcp_sparse_mla_decode_fused_fp4
 *                                     step 2 and steps 1-3 over fp4 rows
 *   smla_dcp_window_mla_decode        the dense decode limited to a sliding
 *                                     window and a few first tokens (sinks)
 *
 * and the verification of drafted trees of tokens:
 *
 *   smla_tree_maps                    who sees whom, and rotary positions,
 *                                     from the nodes' parents
 *   smla_dcp_tree_mla_decode          attention of a tree's nodes over the
 *                                     cached prefix and each other
 *   smla_dcp_tree_window_mla_decode   the same limited to a sliding window
 *                                     and a few first tokens (sinks)
 *   smla_tree_accept                  the nodes the model agrees with
 *   smla_mla_cache_move               their cache rows, to their own slots
 *
 * and the projections around the attention, in 8 bits:
 *
 *   smla_fp8_quantise                 bf16 rows to e4m3, a scale for 128
 *   smla_fp8_matmul                   their product with e4m3 weights that
 *                                     have a scale for 128 x 128
 *
 * Sources (page title, then section):
 *   [P1] "[eldritch] attention: support DCP in SM120 FlashInfer sparse MLA"
 *   [P2] "[Bugfix][Attention] Stabilize sparse-MLA DCP for GLM PCP evals"
 *   [P3] "FlashMLA sparse fp8 path + DCP + MTP" (vLLM PR #46514 summary)
 *
 * Conventions shared by every call:
 *   - Pointers marked "device" point to memory of the current CUDA device;
 *     the caller allocates and owns all of it.  The library never allocates,
 *     frees or synchronises, and keeps no pointer after a call returns, with
 *     two exceptions: smla_sparse_mla_decode_noalloc's split-K scratch is a
 *     library-owned device array of SMLA_NOALLOC_SCRATCH_BYTES per GPU, whose
 *     device address the library looks up once per device and keeps, and
 *     smla_dcp_sparse_mla_decode_fused_host creates its streams and events
 *     once per device and keeps them.
 *   - Every call is asynchronous on `stream` (a cudaStream_t passed as void*,
 *     NULL = legacy default stream) and takes every scalar by value, so no
 *     call issues a host->device copy of its own or a host sync [P2 "DCP
 *     decode rank scalar"]; smla_dcp_sparse_mla_decode_fused_host copies
 *     only the caller's host buffers it is given, asynchronously.
 *   - Arguments are checked on the host before any launch; a failing check
 *     returns a status and launches nothing.  A failed launch returns
 *     SMLA_ERR_CUDA.  No C++ exception crosses this boundary.
 *   - T = 0 is a no-op that returns SMLA_OK.
 *   - Inputs the host cannot check (an id that runs past its block table, a
 *     slot past the pool) are caught in the kernels: the offending entry is
 *     treated as -1 and a bit is set in the device error word, readable with
 *     smla_get_device_error.  No kernel traps.
 *   - Index tensors are int32, row-major and contiguous.
 *   - The serving step's calls (the last lists above) launch with programmatic
 *     stream serialisation: their launch overlaps the end of the kernel before
 *     them on the stream, and they wait for its completion before they touch
 *     memory.
 */
#ifndef SMLA_H_
#define SMLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int smla_status;

enum {
  SMLA_OK = 0,
  SMLA_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned buffer   */
  SMLA_ERR_UNSUPPORTED = 2, /* valid but outside the supported envelope    */
  SMLA_ERR_WORKSPACE = 3,   /* workspace missing, too small or misaligned  */
  SMLA_ERR_CUDA = 4         /* a CUDA runtime call or launch failed        */
};

/* Bits of the device error word. */
enum {
  SMLA_DEVERR_BLOCK_TABLE = 1u, /* id past the block table / unallocated block */
  SMLA_DEVERR_REQ_ID = 2u,      /* req_id_per_token outside [0, num_reqs)      */
  SMLA_DEVERR_SLOT_RANGE = 4u,  /* local slot >= num_slots                     */
  SMLA_DEVERR_TIMEOUT = 8u,     /* a bounded wait inside a kernel gave up      */
  SMLA_DEVERR_CONTEXT = 16u,    /* a context shorter than its request's query
                                   tokens or past max_ctx; step maps: that, a
                                   negative length or more rows than T        */
  SMLA_DEVERR_RANGE = 32u,      /* a q or rope value, or a latent group scale,
                                   that the fp16 keys cannot carry (below)    */
  SMLA_DEVERR_FREE_BLOCKS = 64u, /* step maps: the free list is too short     */
  SMLA_DEVERR_POSITION = 128u,  /* cache write: a position outside the table  */
  SMLA_DEVERR_TREE = 1u << 30   /* a drafted tree whose rows lie outside T or
                                   are too many, or a parent that does not
                                   come before its node                       */
};
/* The decode kernels compute QK^T and PV on fp16 operands: q and the rope
 * values are converted from bf16 and each latent value is dequantised as
 * e4m3 code x scale, rounded once to fp16.  SMLA_DEVERR_RANGE is set when a
 * q or rope value of a row has |x| >= 65536 (inf / NaN included), when a
 * group scale exceeds 65504 / 448 (its dequantised values would overflow
 * fp16), or when a nonzero scale is below 2^-22 (its keys would be fp16
 * subnormals and lose precision).  The result is still written; the bit says
 * it may be outside the stated tolerances.  An fp4 row's latent values are
 * exact in the kernel's keys and its rope values within 2^-18; for those rows
 * the bit stands for the q and rope values and for a NaN scale.
 * The tree decodes take 8-bit rows' codes and rope values, and q, as
 * they are into QK^T, so that there the bit stands for a scale as above (of
 * the values) and for a q that is not finite; over 4-bit rows it is as above. */
/* With SMLA_DEVERR_TIMEOUT, bits 8..29 of the word tell which of the decode
 * kernel's internal waits gave up (a diagnostic bitmask, one bit per site). */

/* Largest gathered head count the decode kernel takes [P3 implementation
 * breakdown step 4: heads pad to the 64/128 kernel envelope]. */
#define SMLA_MAX_HEADS 128
/* Largest number of partials smla_dcp_lse_merge combines in one call. */
#define SMLA_MAX_DCP 16
/* Packed fp8_ds_mla row: 512 e4m3 codes | 4 fp32 scales | 64 bf16 rope. */
#define SMLA_ROW_BYTES 656
#define SMLA_QK_DIM 576
#define SMLA_V_DIM 512

/* Packed 4-bit row: 256 bytes of e2m1 codes (byte i holds dim 2i in its low
 * nibble, dim 2i + 1 in its high one) | 32 e4m3 scales, scale g for dims
 * 16g .. 16g + 15 | 64 bf16 rope.  Latent dim c = e2m1(code c) *
 * e4m3(scale[c div 16]); e2m1 is sign, 2 exponent and 1 mantissa bits: 0,
 * 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives. */
#define SMLA_FP4_ROW_BYTES 416
/* Row formats, where a call takes either. */
enum { SMLA_CACHE_FP8 = 0, SMLA_CACHE_FP4 = 1 };

/* Human-readable name of a status code (static string, never NULL). */
const char* smla_status_string(smla_status status);

/* Reads the device error word of the current device into *flags (a host
 * pointer) as an OR of SMLA_DEVERR_* bits; clears it when `clear` != 0.
 * This call synchronises with the device (it is a diagnostic, not part of
 * the hot path). */
smla_status smla_get_device_error(uint32_t* flags, int clear);

/*
 * Step 1 -- DCP filter + convert [P3 implementation breakdown step 2 and
 * the _forward_fp8_kv_mixed_batch snippet; P1 Summary].
 *
 * For row i (request r = req_id_per_token[i]) and entry j, with t =
 * topk_global[i*K + j] and interleave size I (runs of I consecutive
 * positions go to the ranks in turn; the pages name the size,
 * cp_kv_cache_interleave_size, and validate only I = 1 [P3 implementation
 * breakdown step 4]):
 *   t < 0 or (t div I) mod D != rank  -> local_slots[i*K + j] = -1
 *   otherwise lp = (t div (I*D))*I + t mod I (rank-local position; I = 1:
 *             t div D), local_slots[i*K + j] = block_table[r*bt_row_stride +
 *             lp div block_size] * block_size + lp mod block_size
 * The -1s stay in place (compact_valid_to_front = False).  With D = 1 and
 * rank = 0 this is the plain paged request-index -> slot conversion.
 * valid_count[i] (optional, may be NULL) receives the number of
 * non-negative outputs of row i.
 *
 *   req_id_per_token  device int32 [T]
 *   block_table       device int32 [num_reqs, bt_row_stride]; columns
 *                     [0, bt_width) are meaningful, -1 = unallocated
 *   topk_global       device int32 [T, K], global token positions, -1 padded
 *   local_slots       device int32 [T, K] output (may not alias inputs)
 *   valid_count       device int32 [T] output or NULL
 * Errors: INVALID_ARG for null pointers (T > 0), T < 0, K < 1, D < 1,
 * rank outside [0, D), block_size < 1, interleave < 1, num_reqs < 1,
 * bt_width < 1 or bt_row_stride < bt_width.  On the device an out-of-range
 * request id or a position past the block table (or in a -1 block) yields -1
 * and sets a device error bit.
 */
smla_status smla_dcp_filter_convert_index(
    const int32_t* req_id_per_token, const int32_t* block_table,
    int64_t bt_row_stride, int32_t bt_width, int32_t num_reqs,
    const int32_t* topk_global, int32_t T, int32_t K, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, int32_t* local_slots,
    int32_t* valid_count, void* stream);

/*
 * Bytes of caller-owned workspace smla_sparse_mla_decode needs for (T, H,
 * K); 0 means none.  The size follows from the shape alone, so a caller can
 * allocate the workspace once at start-up [P1 Implementation Notes:
 * per-device scratch allocated at initialisation; P2 "FlashInfer sparse-MLA
 * DCP workspace": size derived from tokens x gathered heads].  Few rows are
 * split over more key ranges than many, so a smaller batch may need more than
 * a larger one: a workspace for batches of several sizes has the largest of
 * their sizes.
 * Returns 0 for invalid shapes.
 */
size_t smla_decode_workspace_size(int32_t T, int32_t H, int32_t K);

/*
 * Step 2 -- sparse MLA decode with LSE return [P1 Why; P3 implementation
 * breakdown steps 1 and 3; the _forward_fp8_kv_mixed_batch snippet].
 *
 * For row i, head h, over the valid entries j of local_slots row i
 * (slot >= 0; every occurrence counts):
 *   k_j   = dequant(kv_cache row slot_j)              576 dims
 *           (latent dim c = e4m3(code c) * scale[c div 128], rope = bf16)
 *   s_j   = sm_scale * <q[i,h,:], k_j>
 *   lse   = log(sum_j exp(s_j))           natural log, sm_scale included
 *   out   = sum_j exp(s_j - lse) * latent_j           512 dims
 * A row with no valid entry is written as the merge identity out = 0,
 * lse = -inf [P3 executive summary 1, implementation breakdown step 3].
 *
 *   q           device bf16 [T, H, 576] (16-byte aligned); H is the
 *               gathered head count [P1 Implementation Notes]
 *   kv_cache    device uint8 [num_slots, 656] (16-byte aligned)
 *   local_slots device int32 [T, K], -1 = masked (scattered, any order)
 *   out         device bf16 [T, H, 512] output, contiguous, 16-byte aligned
 *   lse         device fp32 [T, H] output, row = token (spec decode rows
 *               b*S + s) [P3 implementation breakdown steps 1 and 5]
 *   workspace   device scratch of at least
 *               smla_decode_workspace_size(T, H, K) bytes, 256-byte aligned,
 *               zero-filled before its first use (every call, including one
 *               that sets SMLA_DEVERR_TIMEOUT, leaves its arrival counters
 *               zero again); may be NULL when that size is 0.  One
 *               workspace serves calls of any shapes in turn, of this and of
 *               every other decode that takes one, as long as nothing else
 *               writes to it in between.  Calls that run concurrently need
 *               distinct workspaces.
 * When the size is not 0 the rows are split over several key ranges
 * (split-K) and each range's partial (its normalised output in fp16, its
 * maximum and sum in fp32) goes through the workspace.  The
 * partials are merged by their LSE in the decode kernel (the last range of
 * a row to finish merges it) when the decode grid is larger than one wave
 * on the GPU or there are fewer than four ranges per row, up to 16,384 rows;
 * otherwise by a second kernel launched on `stream` with programmatic stream
 * serialisation.  Without split-K the call is a single kernel launch.
 * Errors: INVALID_ARG for null pointers, T < 0, K < 1, H < 1, num_slots < 0,
 * sm_scale not finite and positive, misaligned q/kv_cache/out; UNSUPPORTED
 * for H > SMLA_MAX_HEADS; WORKSPACE
 * when the workspace is too small, NULL or misaligned.  A slot >= num_slots
 * is treated as -1 and sets SMLA_DEVERR_SLOT_RANGE.
 */
smla_status smla_sparse_mla_decode(
    const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
    const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
    float sm_scale, uint16_t* out, float* lse, void* workspace,
    size_t workspace_bytes, void* stream);

/*
 * Step 2 without caller scratch.  The pages have no counterpart to this call:
 * it exists for callers that cannot allocate device memory -- code that runs
 * inside CUDA stream capture, where cudaMalloc is not allowed, or hosts that
 * forbid device allocation after start-up -- and so cannot provide the
 * workspace smla_sparse_mla_decode wants.
 *
 * Same arguments, semantics and errors as smla_sparse_mla_decode minus the
 * workspace: the split-K scratch is a library-owned array of
 * SMLA_NOALLOC_SCRATCH_BYTES in device memory, which every GPU that loads the
 * library holds until the process exits.  A shape whose scratch need
 * (smla_decode_workspace_size) exceeds that size returns SMLA_ERR_WORKSPACE
 * and launches nothing.  The call allocates nothing (no cudaMalloc, no
 * cudaFree, no allocating library routine); it clears the scratch's arrival
 * counters with cudaMemsetAsync on `stream` before each launch.
 *
 * The first call on a device looks up the array's device address there (with
 * that device current); make that first call before any stream capture.
 * Every call on a device shares the one array and it keeps the last call's
 * contents, so calls that overlap on the GPU (e.g. on two streams at once)
 * race and must be serialised by the caller.
 */
#define SMLA_NOALLOC_SCRATCH_BYTES (((size_t)32 << 20) + 131328)
smla_status smla_sparse_mla_decode_noalloc(
    const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
    const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
    float sm_scale, uint16_t* out, float* lse, void* stream);

/*
 * Steps 1-3 in one launch (fused DCP step for D shards held by one GPU; with
 * split-K, a second launch may merge the key ranges, as for
 * smla_sparse_mla_decode).
 *
 * Computes exactly what the three calls above compute for D shard pools --
 * filter + convert per shard, sparse MLA decode per shard, LSE merge -- in a
 * single kernel: the global-to-local conversion of "FlashMLA sparse fp8 path
 * + DCP + MTP" (implementation breakdown step 2) runs in the kernel's
 * prologue for every shard, the compacted keys of all shards share one online
 * softmax, and since the LSE merge of per-shard softmax partials equals the
 * softmax over the union of their keys ("[eldritch] attention: support DCP in
 * SM120 FlashInfer sparse MLA", Why: the merge reduces partial attention
 * results), the output is the merged (out, lse) directly.  A row whose ids
 * all map to nothing is written as (0, -inf).
 *
 *   q, T, H, K, sm_scale, out, lse   as in smla_sparse_mla_decode (out/lse
 *                                    receive the merged result)
 *   req_id_per_token, topk_global, num_reqs, D, block_size, interleave
 *                                    as in smla_dcp_filter_convert_index
 *   kv_caches      host array of D device pointers, pool d = uint8
 *                  [num_slots[d], 656], 16-byte aligned
 *   num_slots      host array of D pool sizes
 *   block_tables   host array of D device pointers, table d = int32
 *                  [num_reqs, bt_row_strides[d]], columns [0, bt_widths[d])
 *   workspace      >= smla_decode_workspace_size(T, H, K) bytes, same rules
 *                  as for smla_sparse_mla_decode
 * Errors: as the three calls above (INVALID_ARG for interleave < 1);
 * UNSUPPORTED for D > SMLA_MAX_DCP.
 * Device-side input errors (ids past a block table, bad request ids, slots
 * past a pool) drop the entry and set the device error word.
 */
smla_status smla_dcp_sparse_mla_decode_fused(
    const uint16_t* q, int32_t T, int32_t H, int32_t K, float sm_scale,
    const int32_t* req_id_per_token, const int32_t* topk_global, int32_t num_reqs,
    int32_t D, int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The fused DCP step for callers whose q, top-k ids and results live in
 * host memory (the pages have no counterpart: it is the same step,
 * smla_dcp_sparse_mla_decode_fused, with its host<->device copies).
 *
 * The rows are cut into `chunks` contiguous groups (1 <= chunks <=
 * SMLA_MAX_HOST_CHUNKS, at most T).  Group g's q rows and top-k ids are
 * copied into the device staging buffers, its decode is launched as soon as
 * they have landed, and its out and lse rows are copied back as soon as its
 * decode ends, so the copies of some groups overlap the decode of others.
 * With chunks > 1 each group's decode runs without split-K (every group
 * keeps its own SM pairs, side by side with the others), which needs
 * K <= 2048; with chunks == 1 the copies, the decode (the usual split-K
 * policy and workspace) and the copies back run one after the other.
 *
 *   q_host, topk_host       pinned host bf16 [T, H, 576], int32 [T, K]
 *   out_host, lse_host      pinned host bf16 [T, H, 512], fp32 [T, H] outputs
 *   q_dev, topk_dev,        device staging buffers of the same shapes (16-byte
 *   out_dev, lse_dev        aligned; 4 for lse_dev), owned by the caller;
 *                           they hold the step's device copies afterwards
 *   other arguments         as for smla_dcp_sparse_mla_decode_fused
 *                           (req_id_per_token, pools, block tables and
 *                           workspace in device memory)
 * Everything is ordered after the work already queued on `stream`, and work
 * queued on `stream` after the call waits for the whole step, including the
 * copies back: the host buffers hold the results once `stream` has reached
 * that point.  The groups run on library-owned streams and events (created
 * on a device's first call, kept until the process exits); the call is
 * serialised per device, so concurrent calls from several host threads
 * queue one after the other.  Made inside CUDA stream capture on `stream`
 * (after one call outside it on the device), the library's streams join the
 * capture through those events and the graph replays the whole step.
 * Errors: as smla_dcp_sparse_mla_decode_fused, plus INVALID_ARG for a null
 * or misaligned host or staging buffer or chunks outside [1,
 * SMLA_MAX_HOST_CHUNKS]; UNSUPPORTED for chunks > 1 with K > 2048.
 */
#define SMLA_MAX_HOST_CHUNKS 8
smla_status smla_dcp_sparse_mla_decode_fused_host(
    const uint16_t* q_host, const int32_t* topk_host, uint16_t* out_host, float* lse_host,
    uint16_t* q_dev, int32_t* topk_dev, uint16_t* out_dev, float* lse_dev,
    int32_t T, int32_t H, int32_t K, float sm_scale, const int32_t* req_id_per_token,
    int32_t num_reqs, int32_t D, int32_t block_size, int32_t interleave,
    const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides,
    const int32_t* bt_widths, void* workspace, size_t workspace_bytes, int32_t chunks,
    void* stream);

/*
 * Dense MLA decode with LSE return under DCP [P3 key snippets: the dense
 * FlashMLA decode path, whose LSE comes back as [batch, heads, seq_len] and
 * is flattened to [tokens, heads] for the DCP merge; implementation breakdown
 * step 5].
 *
 * Request b has S query tokens (S > 1: an MTP / speculative step); token s
 * sits at position p = ctx_lens[b] - S + s and attends every cached position
 * 0..p of its request (causal), with the attention of smla_sparse_mla_decode
 * over those positions' cache rows.  Position t lives on rank (t div I) mod
 * D at local position (t div (I*D))*I + t mod I, as in
 * smla_dcp_filter_convert_index.
 *   rank = -1       attend all D pools in one launch: out/lse are the merged
 *                   result (the LSE merge of the ranks' partials)
 *   rank in [0, D)  attend only rank's positions: out/lse are that rank's
 *                   partial, to be combined with smla_dcp_lse_merge
 * Rows come out in token order b*S + s: out [B*S, H, 512], lse [B*S, H] --
 * the pages' [batch, heads, seq_len] -> [tokens, heads] flattening.
 *
 *   q              device bf16 [B*S, H, 576]
 *   ctx_lens       device int32 [B], each in [S, max_ctx]
 *   max_ctx        host bound on every ctx_lens[b] (sizes the split-K)
 *   kv_caches, num_slots, block_tables, bt_row_strides, bt_widths
 *                  host arrays of D entries as in
 *                  smla_dcp_sparse_mla_decode_fused (block-table row b
 *                  belongs to request b); with rank >= 0 only entry [rank]
 *                  is read and the others may be NULL / 0
 *   workspace      >= smla_dense_decode_workspace_size(B*S, H, max_ctx, D,
 *                  interleave, rank) bytes, same rules as for
 *                  smla_sparse_mla_decode
 * Errors: INVALID_ARG for null pointers, B < 0, S < 1, H < 1, max_ctx < 1,
 * D < 1, rank outside [-1, D), block_size < 1, interleave < 1, a bad pool or
 * table entry that is read, misaligned q/out/lse; UNSUPPORTED for H >
 * SMLA_MAX_HEADS or D > SMLA_MAX_DCP; WORKSPACE as for smla_sparse_mla_decode.
 * On the device a request whose context is outside [S, max_ctx] comes out
 * as (0, -inf) in all its rows and sets SMLA_DEVERR_CONTEXT; a position past
 * a block table sets SMLA_DEVERR_BLOCK_TABLE.
 */
size_t smla_dense_decode_workspace_size(int32_t T, int32_t H, int32_t max_ctx, int32_t D,
                                        int32_t interleave, int32_t rank);
smla_status smla_dcp_dense_mla_decode(
    const uint16_t* q, int32_t B, int32_t S, int32_t H, float sm_scale,
    const int32_t* ctx_lens, int32_t max_ctx, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Global top-k selection of indexer scores: the step that produces the
 * path's global top-k ids ["[eldritch] ..." Summary: global sparse top-k
 * token ids; P3 related PRs: the DCP sparse indexer's global top-k merge].
 * The pages print no rule; the rule taken: keep the K largest scores, ranked
 * by score descending and then token id ascending, -1 padded when a row has
 * fewer than K candidates; NaN ranks below every number, -0 equals +0.
 *
 * smla_topk_select: row i's candidates are the local positions
 * j < n_cand[i] (clipped to [0, L]) of rank `rank`, with scores
 * scores[i*row_stride + j]; the ids written are their global positions:
 * local position j of rank r is global position (j div I)*I*D + r*I +
 * j mod I, the inverse of smla_dcp_filter_convert_index's rule (D = 1,
 * rank = 0: the plain top-k of positions 0..n-1).
 *   scores      device fp32 [T, row_stride]
 *   n_cand      device int32 [T]
 *   out_ids     device int32 [T, K] output
 *   out_scores  device fp32 [T, K] output (the kept scores) or NULL
 *   workspace   NULL, or device scratch of at least
 *               smla_topk_select_workspace_size(T, L, K) bytes, 16-byte
 *               aligned (no initial contents); calls that run concurrently
 *               need distinct workspaces.  With it, a call of at most 32
 *               rows whose L is at least 16 x max(16384, 8 x K rounded up
 *               to a power of two) cuts each row into min(8, SMs / T)
 *               chunks, one CTA each keeping the chunk's K best, and a
 *               second launch selects the row's K best among those; without
 *               it (or when the size is 0) each row is walked whole, by two
 *               CTAs (a cluster) when L >= 16384 and 2 T CTAs fit on the
 *               GPU at once, else by one.  The result is the same either
 *               way.
 *
 * smla_dcp_topk_merge: row i's candidates are the entries j < M with
 * cand_ids[i*row_stride + j] >= 0 (global ids, unique per row) and their
 * cand_scores; writes the top K of the union by the same rule -- with each
 * rank's smla_topk_select output concatenated, exactly the unsharded top-k.
 *
 * Errors: INVALID_ARG for null pointers (T > 0), T < 0, L < 0, M < 0,
 * row_stride < L (or < M), D < 1, rank outside [0, D), interleave < 1,
 * misaligned buffers; UNSUPPORTED for K outside [1, SMLA_MAX_TOPK];
 * WORKSPACE for a non-NULL workspace smaller than the size below or not
 * 16-byte aligned.
 *
 * smla_topk_select_workspace_size: bytes of the optional workspace for
 * (T, L, K), from the shape alone; 0 when no row can be long enough to be
 * cut, or for invalid shapes.
 */
#define SMLA_MAX_TOPK 16384
size_t smla_topk_select_workspace_size(int32_t T, int32_t L, int32_t K);
smla_status smla_topk_select(const float* scores, int64_t row_stride, int32_t L,
                             const int32_t* n_cand, int32_t T, int32_t K, int32_t D,
                             int32_t rank, int32_t interleave, int32_t* out_ids,
                             float* out_scores, void* workspace, size_t workspace_bytes,
                             void* stream);
smla_status smla_dcp_topk_merge(const int32_t* cand_ids, const float* cand_scores,
                                int64_t row_stride, int32_t M, int32_t T, int32_t K,
                                int32_t* out_ids, float* out_scores, void* stream);

/*
 * Step 3 -- LSE-weighted merge of D partials [P1 Why, Scope / Limitations
 * (the ag_rs flow); P3 executive summary 1 and implementation breakdown
 * step 3].  With M = max_d lse_d[t,h]:
 *   M = -inf  -> out = 0, lse = -inf
 *   otherwise lse = M + log(sum_d exp(lse_d - M)),
 *             out = sum_d exp(lse_d - lse) * out_d
 * On one GPU this stands in for the cross-rank LSE all-gather plus output
 * reduce-scatter.
 *
 *   outs  host array of D device pointers, each bf16 [T, H, 512], 16-byte
 *         aligned
 *   lses  host array of D device pointers, each fp32 [T, H]
 *   out   device bf16 [T, H, 512] output (may alias none of the inputs)
 *   lse   device fp32 [T, H] output
 * Errors: INVALID_ARG for null pointers, D < 1, T < 0, H < 1, misaligned
 * buffers; UNSUPPORTED for D > SMLA_MAX_DCP.
 */
smla_status smla_dcp_lse_merge(const uint16_t* const* outs,
                               const float* const* lses, int32_t D, int32_t T,
                               int32_t H, uint16_t* out, float* lse,
                               void* stream);

/*
 * Steps 1-3 over fp4 rows (SMLA_FP4_ROW_BYTES each).
 *
 * smla_sparse_mla_decode_fp4 is smla_sparse_mla_decode and
 * smla_dcp_sparse_mla_decode_fused_fp4 is smla_dcp_sparse_mla_decode_fused
 * with the pools' rows in the 4-bit format: same arguments, results, errors
 * and workspace rules (smla_fp4_decode_workspace_size gives the size; key
 * ranges are chosen by the shape, and merged in a second kernel when the grid
 * does not fill the GPU); UNSUPPORTED for K > 2^30.
 * smla_dcp_filter_convert_index and smla_dcp_lse_merge do not read cache
 * rows and serve either format.  The latent keys are exact in the kernel's
 * fp16 operands.
 */
size_t smla_fp4_decode_workspace_size(int32_t T, int32_t H, int32_t K);
smla_status smla_sparse_mla_decode_fp4(
    const uint16_t* q, const uint8_t* kv_cache, int64_t num_slots,
    const int32_t* local_slots, int32_t T, int32_t H, int32_t K,
    float sm_scale, uint16_t* out, float* lse, void* workspace,
    size_t workspace_bytes, void* stream);
smla_status smla_dcp_sparse_mla_decode_fused_fp4(
    const uint16_t* q, int32_t T, int32_t H, int32_t K, float sm_scale,
    const int32_t* req_id_per_token, const int32_t* topk_global, int32_t num_reqs,
    int32_t D, int32_t block_size, int32_t interleave, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables,
    const int64_t* bt_row_strides, const int32_t* bt_widths, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Windowed decode with sinks: smla_dcp_dense_mla_decode in which token s of
 * request b, at position p = ctx_lens[b] - S + s, attends the positions
 * t <= p with t < sinks or t > p - window (the last `window` positions, its
 * own among them, and the request's first `sinks`).  A window of at least
 * max_ctx is the dense decode.  Only those positions' block-table entries and
 * cache rows are read: blocks behind the window may have been given back.
 *
 *   window       >= 1
 *   sinks        >= 0
 *   format       SMLA_CACHE_FP8 or SMLA_CACHE_FP4: the rows of every pool
 *   workspace    >= smla_window_decode_workspace_size(B*S, H, max_ctx, window,
 *                sinks, D, interleave, rank) bytes, same rules as for
 *                smla_sparse_mla_decode
 *   the rest     as for smla_dcp_dense_mla_decode; a rank that holds none of
 *                a token's positions returns (0, -inf) for it
 * With SMLA_CACHE_FP8 the LSE carries the keys' rounding to fp16 (2^-11 a key
 * value, so a few 10^-6 of it over a thousand keys); 4-bit keys are exact.
 * Errors: as smla_dcp_dense_mla_decode, plus INVALID_ARG for window < 1,
 * sinks < 0 or another format, and UNSUPPORTED for max_ctx > 2^30 or
 * interleave * D > 2^31 - 1.
 */
size_t smla_window_decode_workspace_size(int32_t T, int32_t H, int32_t max_ctx, int32_t window,
                                         int32_t sinks, int32_t D, int32_t interleave,
                                         int32_t rank);
smla_status smla_dcp_window_mla_decode(
    const uint16_t* q, int32_t B, int32_t S, int32_t H, float sm_scale,
    const int32_t* ctx_lens, int32_t max_ctx, int32_t window, int32_t sinks, int32_t D,
    int32_t rank, int32_t block_size, int32_t interleave, int32_t format,
    const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides, const int32_t* bt_widths,
    uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Step maps of one rank, from the requests' lengths: what a prefill, decode
 * or mixed step needs to write its new tokens' cache rows and to run the
 * calls above.
 *
 * Request b has ctx_lens[b] cached positions, its q_lens[b] new tokens
 * included (0 <= q_lens[b] <= ctx_lens[b]).  Its rows are row_start[b] ..
 * row_start[b + 1] - 1, row_start the exclusive sum of q_lens; row i of
 * request b is position p = ctx_lens[b] - q_lens[b] + (i - row_start[b]).
 *   req_id[i] = b, positions[i] = p
 *   slots[i]  = this rank's cache slot of p (through block_table, as
 *               smla_dcp_filter_convert_index maps it), -1 where another
 *               rank holds p
 *   rows i >= row_start[B] up to T (padding of a captured step): req_id 0,
 *               position 0, slot -1
 *   local_lens[b] = how many of the request's positions this rank holds
 * The positions already cached fill the first ceil(count / block_size)
 * columns of the request's block_table row on this rank; the columns the new
 * tokens add are taken from free_blocks in request order, column order, and
 * written to block_table.  *blocks_taken = how many, over all requests: the
 * caller drops that many from the front of its free list.
 *
 *   ctx_lens, q_lens   device int32 [B]
 *   free_blocks        device int32 [num_free], distinct block ids (NULL when
 *                      num_free is 0)
 *   block_table        device int32 [B, bt_row_stride], read and written
 *   slots              device int32 [T] output; T is at least the sum of
 *                      q_lens
 *   row_start [B + 1], req_id [T], positions [T], local_lens [B],
 *   blocks_taken [1]   device int32 outputs, each may be NULL
 * No output may alias an input or another output.  A repeated call on the
 * same lengths and free list writes the same values.
 * Errors: INVALID_ARG for B < 0, T < 0, D < 1, rank outside [0, D),
 * block_size < 1, interleave < 1, num_free < 0, bt_width < 1 or
 * bt_row_stride < bt_width, a NULL array that is needed, misaligned arrays;
 * UNSUPPORTED for B > SMLA_MAX_STEP_REQS.  B = 0 and T = 0 is a no-op.  On
 * the device, lengths outside 0 <= q <= ctx count as no new tokens and set
 * SMLA_DEVERR_CONTEXT, as does a sum of q_lens past T (the rows that fit are
 * written); a free list that is too short leaves -1 in block_table and slots
 * and sets SMLA_DEVERR_FREE_BLOCKS; a column past bt_width, an unallocated or
 * negative block and a slot past 2^31 - 1 give slot -1 and set
 * SMLA_DEVERR_BLOCK_TABLE.
 */
#define SMLA_MAX_STEP_REQS 8192
smla_status smla_dcp_step_maps(
    const int32_t* ctx_lens, const int32_t* q_lens, int32_t B, int32_t T, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, const int32_t* free_blocks, int32_t num_free,
    int32_t* block_table, int64_t bt_row_stride, int32_t bt_width, int32_t* row_start,
    int32_t* req_id, int32_t* positions, int32_t* slots, int32_t* local_lens,
    int32_t* blocks_taken, void* stream);

/*
 * Cache write: a step's latent rows, normalised, rotated and quantised into
 * the packed cache at their slots.
 *
 * For row i with slots[i] >= 0, latent x = kv[i, 0:512] and rope part
 * z = kv[i, 512:576]:
 *   y = x * gamma / sqrt(mean(x^2) + eps)  (gamma NULL: y = x)
 *   fp8 row: scale[g] = fp32(max |y| / 448) over dims 128g .. 128g + 127,
 *            codes = e4m3(y / scale)
 *   fp4 row: scale[g] = e4m3(max |y| / 6) over dims 16g .. 16g + 15,
 *            codes = e2m1(y / scale)
 *            (nearest, ties to even, past the largest code to the largest)
 *   rope:    each pair (a, b) becomes (a c - b s, a s + b c), rounded to bf16,
 *            with c = cos_sin[positions[i], j], s = cos_sin[positions[i],
 *            32 + j] for pair j (cos_sin NULL: copied as it is); pair j is
 *            values (2j, 2j + 1) when rope_pairs != 0, else (j, j + 32)
 * Scales and codes are rounded once, from the quotients above computed to
 * about 45 bits (with a norm, where mean(x^2) + eps is at least 2^-100); a
 * group whose scale is 0 (fp8: or below 2^-126) has zero codes.  A group with
 * a value y that is not finite in fp32, and every group of a normalised row
 * with a latent that is not finite or a sum of squares past fp32, gets a NaN
 * scale.  Rows with slot -1 write nothing; the slots of one
 * call are distinct (a slot given twice ends with an undefined mix of its
 * rows).
 *
 *   kv          device bf16, row i at kv + i * kv_row_stride (elements; a
 *               multiple of 8, at least 576), 16-byte aligned
 *   gamma       device bf16 [512], 16-byte aligned, or NULL
 *   positions   device int32 [T] (may be NULL without cos_sin)
 *   cos_sin     device fp32 [num_positions, 64] or NULL
 *   slots       device int32 [T]
 *   format      SMLA_CACHE_FP8 or SMLA_CACHE_FP4
 *   kv_cache    device uint8 [num_slots, 656 or 416], 16-byte aligned
 * Errors: INVALID_ARG for T < 0, num_slots < 0, another format, a bad stride,
 * eps not finite and positive (with gamma), num_positions < 1 (with cos_sin),
 * NULL or misaligned arrays.  On the device a slot >= num_slots sets
 * SMLA_DEVERR_SLOT_RANGE and a position outside [0, num_positions) of a row
 * with a slot sets SMLA_DEVERR_POSITION; such a row writes nothing.
 */
smla_status smla_mla_cache_write(
    const uint16_t* kv, int64_t kv_row_stride, int32_t T, const uint16_t* gamma, float eps,
    const int32_t* positions, const float* cos_sin, int32_t num_positions, int32_t rope_pairs,
    const int32_t* slots, int32_t format, uint8_t* kv_cache, int64_t num_slots, void* stream);

/*
 * Cache gather: row slots[n] of the cache, dequantised, as row n of `out`
 * (512 latent values, then 64 rope values; bf16, rounded once, or fp32) --
 * the cached context of a prefill chunk, for instance.  Slot -1 gives a row
 * of zeros; so does a slot >= num_slots, which sets SMLA_DEVERR_SLOT_RANGE.
 *
 *   slots           device int32 [N], any order, repeats allowed
 *   out             device bf16 (out_fp32 = 0) or fp32 [N, 576], row n at
 *                   n * out_row_stride elements (at least 576; a multiple of
 *                   8, of 4 for fp32), 16-byte aligned
 *   the rest        as for smla_mla_cache_write
 */
smla_status smla_mla_cache_gather(const uint8_t* kv_cache, int64_t num_slots, int32_t format,
                                  const int32_t* slots, int32_t N, void* out,
                                  int64_t out_row_stride, int32_t out_fp32, void* stream);

/*
 * Drafted trees.  A verification step brings, for request b, the n_b nodes of
 * a tree of drafted tokens as its rows row_start[b] .. row_start[b + 1] - 1;
 * node j is row row_start[b] + j.  parents[row] is the index (in the tree) of
 * the node before it, less than its own, or -1 for a node that follows the
 * prefix (the request's cached positions) directly.  By custom node 0 is the
 * last token sampled and the only such node.  n_b is 0 .. max_nodes, at most
 * SMLA_MAX_TREE_NODES; rows from row_start[B] up to T are padding.
 *
 * smla_tree_maps writes, with W = ceil(max_nodes / 64):
 *   masks [T, W]    bit m mod 64 of word m div 64 is set when node m is the
 *                   row's own or one of its ancestors
 *   positions [T]   prefix_lens[b] + the node's depth (its number of
 *                   ancestors), the place of its token if it is accepted
 * and zeros in both for the padding rows.
 *
 *   parents         device int32 [T]
 *   row_start       device int32 [B + 1]
 *   prefix_lens     device int32 [B] (may be NULL without positions)
 *   masks           device uint64 [T, W] output, 8-byte aligned
 *   positions       device int32 [T] output or NULL
 * Errors: INVALID_ARG for B < 0, T < 0, max_nodes < 1, a NULL array that is
 * needed, misaligned arrays; UNSUPPORTED for max_nodes > SMLA_MAX_TREE_NODES.
 * T = 0 is a no-op.  On the device a parent that is below -1 or not before
 * its node counts as -1, a request whose rows are more than max_nodes or lie
 * outside [0, T) writes nothing; both set SMLA_DEVERR_TREE.
 */
#define SMLA_MAX_TREE_NODES 256
smla_status smla_tree_maps(const int32_t* parents, const int32_t* row_start,
                           const int32_t* prefix_lens, int32_t B, int32_t T, int32_t max_nodes,
                           uint64_t* masks, int32_t* positions, void* stream);

/*
 * Tree attention with LSE return: row row_start[b] + j (node j of request b),
 * each head, attends
 *   - the request's prefix, positions 0 .. prefix_lens[b] - 1, through its
 *     block-table rows: of all D pools (rank = -1: out and lse are the merged
 *     result) or of one rank (rank >= 0: its partial, for smla_dcp_lse_merge);
 *     position t lives on rank (t div I) mod D, as in
 *     smla_dcp_filter_convert_index
 *   - each node m of its tree whose bit is set in the row's mask (bit m mod 64
 *     of word m div 64, as smla_tree_maps writes them; any mask is taken) and
 *     which some pool holds: draft_slots[d][row of m] >= 0 is its cache slot
 *     in pool d, -1 where that pool does not hold it.  Merged, the lowest pool
 *     that holds it counts; with rank >= 0 only draft_slots[rank] is read.
 *     The slots may be a smla_dcp_step_maps call's (the drafts lie where their
 *     positions' blocks are) or rows outside every block (a scratch area, from
 *     which smla_mla_cache_move brings the accepted ones).
 * with the attention of smla_sparse_mla_decode over those cache rows.  Over
 * 8-bit rows the scores are sums of exact products (of q's latent values those
 * below 2^-10 of the largest of them are taken to within 2^-17 of it), scaled in
 * fp32, so lse is good to fp32 sums; values and probabilities round to fp16.
 * A row with nothing to attend is written as (0, -inf).  Rows of out and lse that
 * belong to no request (behind row_start[B], padding) are left as they were.
 *
 *   q              device bf16 [T, H, 576], 16-byte aligned
 *   row_start      device int32 [B + 1]
 *   prefix_lens    device int32 [B], each in [0, max_prefix]
 *   max_prefix     host bound on every prefix_lens[b], at least 0
 *   masks          device uint64 [T, ceil(max_nodes / 64)]
 *   max_nodes      host bound on every request's rows
 *   draft_slots    host array of D device pointers, int32 [T] each
 *   format         SMLA_CACHE_FP8 or SMLA_CACHE_FP4: the rows of every pool
 *   kv_caches, num_slots, block_tables, bt_row_strides, bt_widths
 *                  host arrays of D entries as in smla_dcp_dense_mla_decode;
 *                  with rank >= 0 only entry [rank] is read
 *   out            device bf16 [T, H, 512], 16-byte aligned
 *   lse            device fp32 [T, H]
 *   workspace      >= smla_tree_decode_workspace_size(T, H, B, max_prefix,
 *                  max_nodes, D, interleave, rank) bytes, 256-byte aligned;
 *                  needs no initial contents.  That size also serves every
 *                  call of fewer rows, heads, requests, prefix or nodes.  Calls
 *                  that run concurrently need distinct workspaces.
 * Errors: INVALID_ARG for T < 0, H < 1, B < 0, max_prefix < 0, max_nodes < 1,
 * D < 1, rank outside [-1, D), block_size < 1, interleave < 1, another format,
 * sm_scale not finite and positive, NULL or misaligned arrays, a bad pool or
 * table entry that is read; UNSUPPORTED for H > SMLA_MAX_HEADS, D >
 * SMLA_MAX_DCP, max_nodes > SMLA_MAX_TREE_NODES, max_prefix > 2^30 or T * H >
 * 2^31 - 1; WORKSPACE as for smla_sparse_mla_decode.  T = 0 and B = 0 are
 * no-ops.
 * On the device a request whose rows are more than max_nodes or lie outside
 * [0, T) writes nothing and sets SMLA_DEVERR_TREE; a prefix outside [0,
 * max_prefix] gives (0, -inf) in all the request's rows and sets
 * SMLA_DEVERR_CONTEXT; a position past a block table or in an unallocated
 * block, and a slot past its pool, are not attended and set
 * SMLA_DEVERR_BLOCK_TABLE and SMLA_DEVERR_SLOT_RANGE.
 */
size_t smla_tree_decode_workspace_size(int32_t T, int32_t H, int32_t B, int32_t max_prefix,
                                       int32_t max_nodes, int32_t D, int32_t interleave, int32_t rank);
smla_status smla_dcp_tree_mla_decode(
    const uint16_t* q, int32_t T, int32_t H, float sm_scale, const int32_t* row_start,
    const int32_t* prefix_lens, int32_t B, int32_t max_prefix, const uint64_t* masks, int32_t max_nodes,
    const int32_t* const* draft_slots, int32_t D, int32_t rank, int32_t block_size, int32_t interleave,
    int32_t format, const uint8_t* const* kv_caches, const int64_t* num_slots,
    const int32_t* const* block_tables, const int64_t* bt_row_strides, const int32_t* bt_widths,
    uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same with a window and sinks, for a model whose steps run through
 * smla_dcp_window_mla_decode: a node at position p = positions[its row] attends
 * of the keys above those at positions t with t < sinks or t > p - window,
 * where a prefix key's t is its place in the request and a drafted node's its
 * own position.  A chain of nodes attends what smla_dcp_window_mla_decode gives
 * the same tokens.  Only the block-table entries and cache rows of positions
 * that a node at the prefix's end attends are read: blocks behind that window
 * may have been given back.
 *
 *   positions    device int32 [T], as smla_tree_maps writes them: the prefix's
 *                length plus the node's depth (outside [prefix_lens[b],
 *                prefix_lens[b] + max_nodes) it counts as the nearest of these)
 *   window       >= 1 (from max_prefix + max_nodes on nothing is left out)
 *   sinks        >= 0
 *   the rest     as for smla_dcp_tree_mla_decode; its workspace size serves
 * Errors: as smla_dcp_tree_mla_decode, plus INVALID_ARG for window < 1, sinks <
 * 0 and NULL or misaligned positions.
 */
smla_status smla_dcp_tree_window_mla_decode(
    const uint16_t* q, int32_t T, int32_t H, float sm_scale, const int32_t* row_start,
    const int32_t* prefix_lens, const int32_t* positions, int32_t B, int32_t max_prefix, const uint64_t* masks,
    int32_t max_nodes, int32_t window, int32_t sinks, const int32_t* const* draft_slots, int32_t D, int32_t rank,
    int32_t block_size, int32_t interleave, int32_t format, const uint8_t* const* kv_caches,
    const int64_t* num_slots, const int32_t* const* block_tables, const int64_t* bt_row_strides,
    const int32_t* bt_widths, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * smla_tree_accept walks each tree greedily: node 0 is accepted, and from an
 * accepted node the walk goes on to its lowest child whose token is the
 * node's target (the token the model chose after it), until there is none.
 *   accepted[b]     the number of accepted nodes (0 for an empty tree)
 *   rows            the accepted nodes' rows, of request 0 from its node 0
 *                   on, then of request 1 and so on; -1 behind the last one
 *                   up to T.  With q_lens = accepted and ctx_lens = the
 *                   prefix + accepted, row i of smla_dcp_step_maps is the
 *                   place of the token in rows[i].
 *   next_tokens[b]  the last accepted node's target (-1 for an empty tree)
 *
 *   parents, tokens, targets   device int32 [T]
 *   row_start                  device int32 [B + 1]
 *   accepted [B], rows [T], next_tokens [B]   device int32 outputs
 * No output may alias an input or another output.
 * Errors: INVALID_ARG for B < 0, T < 0, a NULL array that is needed,
 * misaligned arrays; UNSUPPORTED for B > SMLA_MAX_STEP_REQS.  B = 0 and T = 0
 * is a no-op.  On the device a request of more than SMLA_MAX_TREE_NODES rows,
 * or with rows outside [0, T), counts as empty and sets SMLA_DEVERR_TREE.
 * Above 32 requests the call is two launches, the second with programmatic
 * stream serialisation behind the first.
 */
smla_status smla_tree_accept(const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                             const int32_t* row_start, int32_t B, int32_t T, int32_t* accepted,
                             int32_t* rows, int32_t* next_tokens, void* stream);

/*
 * Cache move: for i < N with rows[i] != -1 and dst_slots[i] >= 0, the cache
 * row in slot src_slots[rows[i]] is copied, byte for byte, to slot
 * dst_slots[i].  With smla_tree_accept's rows, the drafts' slots and
 * smla_dcp_step_maps' slots it brings the accepted tokens to their places.
 * A slot that is written is not read by the same call, nor written twice
 * (else it ends with an undefined mix).
 *
 *   kv_cache     device uint8 [num_slots, 656 or 416], 16-byte aligned
 *   rows         device int32 [N]
 *   src_slots    device int32 [T]
 *   dst_slots    device int32 [N]
 * Errors: INVALID_ARG for N < 0, T < 0, num_slots < 0, another format, NULL or
 * misaligned arrays.  N = 0 is a no-op.  On the device a row outside [0, T),
 * a negative source slot or a slot >= num_slots moves nothing and sets
 * SMLA_DEVERR_SLOT_RANGE.
 */
smla_status smla_mla_cache_move(int32_t format, uint8_t* kv_cache, int64_t num_slots,
                                const int32_t* rows, int32_t N, const int32_t* src_slots, int32_t T,
                                const int32_t* dst_slots, void* stream);

/*
 * Rows to 8 bits: for each of G batches' M rows and each group of 128 columns
 * (the last may be shorter),
 *   scales[g, m, j] = fp32(max |x| / 448) over columns 128 j .. 128 j + 127
 *   codes[g, m, k]  = e4m3(x[g, m, k] / scale), nearest, ties to even
 * each rounded once.  A group whose scale is 0 or below 2^-126 has zero codes;
 * a group with a value that is not finite has a NaN scale and zero codes.
 *
 *   x        device bf16; entry (g, m, k) at g * batch + m * row + k (strides
 *            in elements; 16-byte aligned rows load fastest)
 *   codes    device uint8 (e4m3) output, the same with its own strides
 *   scales   device fp32 output, entry (g, m, j) at g * batch + m * row +
 *            j * col
 * No output may alias x, the other output or its own entries: taken in the
 * order of their strides, each dimension of more than one entry steps past all
 * that the ones before it span.
 * Errors: INVALID_ARG for G < 0, M < 0, K < 1, a negative stride, outputs whose
 * own entries are not apart as above, NULL or misaligned arrays.  G = 0 or M =
 * 0 is a no-op.
 */
smla_status smla_fp8_quantise(const uint16_t* x, int64_t x_batch_stride, int64_t x_row_stride, int32_t G,
                              int32_t M, int32_t K, uint8_t* codes, int64_t codes_batch_stride,
                              int64_t codes_row_stride, float* scales, int64_t scales_batch_stride,
                              int64_t scales_row_stride, int64_t scales_col_stride, void* stream);

/*
 * 8-bit matrix product with block scales, for each of G batches (the heads of
 * an absorbed projection, for instance; G = 1: one product):
 *   out[g, m, n] = sum_j a_scales[g, m, j] b_scales[g, n div 128, j]
 *                  sum_{k = 128 j .. 128 j + 127} a[g, m, k] b[g, n, k]
 * A group's products are summed by the tensor cores in fp32, the groups in
 * fp32, and the result is rounded once.  M, N and K are any sizes.  A row's
 * result does not depend on the other rows' values, and a repeated call gives
 * the same bits.
 *
 *   a          device uint8 (e4m3), entry (g, m, k) at g * batch + m * row + k
 *   a_scales   device fp32, entry (g, m, j) at g * batch + m * row + j * col
 *              (with a col stride of M, as a [K / 128, M] matrix, they are
 *              fetched fastest)
 *   b          device uint8 (e4m3), entry (g, n, k) at g * batch + n * row + k
 *   b_scales   device fp32, entry (g, n div 128, j) by their strides
 *   out        device bf16 (out_fp32 = 0) or fp32, entry (g, m, n) at
 *              g * batch + m * row + n
 * a and b are 16-byte aligned, with row strides of at least K and row and
 * (G > 1) batch strides that are positive multiples of 16.  Strides of
 * scales may be 0 (a shared scale).  out may not alias an input, nor its own
 * entries each other (as smla_fp8_quantise's outputs).
 * Errors: INVALID_ARG for G < 0, M < 0, N < 0, K < 1, a bad stride, an out whose
 * own entries are not apart, NULL or misaligned arrays; UNSUPPORTED for strides of 2^40 bytes and more and for
 * more than 2^27 tiles of 16 x 128 results.  G, M or N = 0 is a no-op.
 */
smla_status smla_fp8_matmul(const uint8_t* a, int64_t a_batch_stride, int64_t a_row_stride,
                            const float* a_scales, int64_t a_scales_batch_stride,
                            int64_t a_scales_row_stride, int64_t a_scales_col_stride, const uint8_t* b,
                            int64_t b_batch_stride, int64_t b_row_stride, const float* b_scales,
                            int64_t b_scales_batch_stride, int64_t b_scales_row_stride,
                            int64_t b_scales_col_stride, int32_t G, int32_t M, int32_t N, int32_t K,
                            void* out, int64_t out_batch_stride, int64_t out_row_stride, int32_t out_fp32,
                            void* stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* SMLA_H_ */
