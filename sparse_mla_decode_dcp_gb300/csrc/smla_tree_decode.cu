// Attention of drafted trees over the packed latent cache (8- or 4-bit rows)
// on tcgen05 tensor cores.
//
// Row (t, h) of request b attends the request's prefix (this rank's share of
// its positions, or all pools') and those nodes of its tree that its mask
// names and some pool holds:
//   s_k = sm_scale <q, k>,  lse = ln sum exp s_k,  out = sum exp(s_k - lse) latent_k
// A row with no key is written as (0, -inf).  A windowed call's row, at position
// p, attends of these the keys at positions t < sinks and t > p - window.
//
// Design (a cluster of two CTAs works on 128 rows and 64 keys at a time):
//   * A request's rows, its nodes times the heads, share its keys, so they are
//     taken as one list and cut into tiles of 128 whatever the head count: 16
//     heads of 8 nodes fill a tile as 128 heads of one do.
//   * MMAs of the pair (cta_group::2, M = 128): each CTA holds 64 of the rows,
//     all 512 value columns of their accumulator (256 tensor-memory columns,
//     two halves of the columns in the two halves of the lanes) and 64 scores,
//     and every CTA's score and output is whole: no partial scores travel.
//     For QK^T each CTA supplies half of the tile's keys (32, all 576 dims),
//     for PV half of the value dims (256, of all 64 keys), so that only
//     signals, no data, go between the CTAs.
//   * fp8 rows: QK^T takes the cache's codes as they are, copied into the
//     MMA's layout asynchronously (cp.async).  The query's latent part is an
//     e4m3 sum hi + lo of each row's values times a power of two: bf16 has 8
//     significant bits, hi the first 4 and lo the rest, exactly down to 2^-10
//     of the row's largest latent and within 2^-17 of it below.  The four scale
//     groups and the rope part (bf16 as it is) have score accumulators of
//     their own, which meet, times the fp32 scales, in the softmax: the log
//     sum is as exact as fp32 sums are.  Values are codes times scales,
//     rounded once to fp16.
//   * fp4 rows: codes times scales are exact in fp16, for keys and values.
//   * A row's 64 scores lie in two lanes, 32 each, whose threads agree on the
//     maximum through shared memory.  Softmax by powers of two against a
//     reference that moves only when p would grow past 2^8.
//   * Masks are looked at in the tiles that hold nodes or missing rows; a
//     node's row that is not finite is kept out of the value tile (its score
//     spoils the rows that see it), so that masked places do not show.
//   * With a window the list of a request's keys leaves out the positions that
//     none of its nodes sees: a key has the last position that sees it, and only
//     tiles with keys that some node no longer sees compare.  The batch below with
//     a window of 4,096 and 4 sinks: 0.82 ms; with one that leaves out a node's
//     last few keys alone 2.34 (the look-up of a key's row and the code cost 13%).
//   * All requests' (row tile, key tile) units form one line that is cut into
//     equal ranges, one a pair, so that ragged batches fill the GPU.  A row
//     tile that a cut falls into leaves partial results (fp16, with their
//     maximum and sum), which a second kernel merges.
//
// A key tile takes 1.7 us of a pair (8-bit rows; 4-bit ones 1.9): a batch of 32
// requests of 16 nodes, 128 heads and 2,048 to 32,768 positions 2.07 ms, 780
// TFLOP/s.  Its MMAs alone take 0.75 us.  What bounds it is the shared-memory data
// pipe, nearly always busy (two thirds for the warps: value tiles, scales,
// copies; a third for the tensor cores' operands), and so the softmax, a chain of
// steps that each wait in it: fewer dependent steps helped (scales asked for with
// the scores, one wait a tile, exponentials while the maxima travel: 2.18 ms
// after 2.44), and so did less code (below), less traffic at the cost of longer
// chains did not (a quarter of the scale loads by tensor-memory fragments and
// shuffles: 2.65; rows gathered by TMA, 128 bytes a piece: 2.88).
//
// Warps: 0-7 softmax and output (two threads a lane of tensor memory), 8-15
// convert cache rows, 16 issues the MMAs (the first CTA's, for both; the
// second's tells it of its keys), 17 lists the pair's work, 18 looks up the
// keys' rows, 19 copies fp8 rows into the K tiles.  Every wait is bounded; one that
// gives up sets SMLA_DEVERR_TIMEOUT and the CTA unwinds.
#include "smla_decode_kernel.cuh"

#include "smla_pair.cuh"
#include "smla_verify.h"

namespace smla {
namespace {

constexpr int kPairRows = 128, kCtaRows = 64;
constexpr int kTileKeys = 64, kCtaKeys = 32;
constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kIssueWarp = kSoftWarps + kConvWarps;
constexpr int kTreeWarps = kIssueWarp + 4;
constexpr int kTreeThreads = 32 * kTreeWarps;
constexpr int kWarpKeys = kCtaKeys / kConvWarps;  // of each CTA, a converter warp's
constexpr int kItems = 8;   // work items listed ahead
constexpr int kPlaces = 4;  // tiles whose rows are looked up ahead
constexpr int kPairs = 76;

// Shared memory: operand tiles in blocks of 128 bytes a row, Q and P by this
// CTA's 64 rows, K by its 32 keys, V by 64 keys (64 dims a block).
constexpr int kQBlock = kCtaRows * 128, kKBlock = kCtaKeys * 128, kVBlock = kTileKeys * 128;
constexpr int kQSize = 9 * kQBlock, kVSize = 4 * kVBlock;
// fp8 rows: Q is hi (4 blocks of 128 codes), lo (4) and the rope part (64
// bf16), a K tile 4 blocks of codes and the rope block, three tiles ahead.
// fp4 rows: 8 blocks of 64 fp16 and the rope block, two tiles.
template <bool kFp4> struct Shared {
  static constexpr int kStages = kFp4 ? 2 : 3;
  static constexpr int kKSize = (kFp4 ? 9 : 5) * kKBlock;
  static constexpr int kOffV = kQSize + kStages * kKSize;
  static constexpr int kOffP = kOffV + 2 * kVSize;
  static constexpr int kPSize = kCtaRows * 128;
  // P tiles.  PV is issued behind QK^T of the next tile, so that with two a
  // tile's scores tell that PV of the tile two before has read its P
  static constexpr int kProbs = kFp4 ? 1 : 2;
  static constexpr int kOffCtl = kOffP + kProbs * kPSize;
};

// tensor memory: the output's 2 x 128 columns, a tile's scores (32 columns for
// each of up to five accumulators)
constexpr uint32_t kOutCol = 0, kScoreCol = 256;

// A request's keys in their order: the prefix positions of pool 0, of pool 1
// and so on (or of one rank), then the tree's nodes.
struct Keys {
  int32_t first, nodes;           // the request's rows (no nodes when its prefix is out of range)
  int32_t before[kMaxMerge + 1];  // prefix keys before pool d
  int32_t prefix, total;
  int32_t length;                 // the prefix's positions (more than its keys, with a window)
  // windowed calls: of pool d's rows its listed keys are the first sinks and, from
  // row sinks + gap on, those in the window; rows from edge on are seen by every node
  int32_t sinks[kMaxMerge], gap[kMaxMerge], edge[kMaxMerge];
};

// A row tile of a request over a range of its key tiles.
struct Item {
  int32_t req;
  int32_t rows;          // of the tile that exist; 0: the end of the list
  int32_t skip;          // rows of the request before the tile
  int32_t tile0, tiles;  // key tiles
  int32_t part;          // -1: all of the row tile's keys; else the partial result's place
  Keys keys;
};

struct TreeCtl {
  // s_read: fp8 rows, of the scores of groups 0 and 1 and of the rest (qk: [0], of
  // all); both, fp4 rows: of even and odd tiles' scores
  uint64_t qk[2], s_read[2], pv[2], k_free[3], k_full[3], k_read[3], k_peer[3], v_full[2], q_full, p_full[2],
      out_read, top[2], sum, item_full[kItems], item_empty[kItems], place_full[kPlaces], place_empty[kPlaces], end;
  uint32_t tbase;
  int abort;
  uint64_t valid[16];                     // per tile (mod 16): which of its keys exist
  // windowed calls, per tile: the last position that sees a key, counted from the
  // prefix's end (255: every node does), and the first of these.  (A tile's are
  // written when PV of the tile seven before is done.)
  alignas(16) uint8_t until[8][kTileKeys];
  int32_t soonest[16];
  const uint8_t* row[kPlaces][kTileKeys];  // the keys' cache rows
  float row_scale[2][kCtaRows];           // fp8 rows, per item (mod 2): 2^-up of a row's latents
  float tops[2][32 * kSoftWarps], sums[32 * kSoftWarps];
  Item items[kItems];
  int64_t warp_units[kTreeWarps], warp_later[kTreeWarps];
  int64_t start;                          // of the pair's range, within its first request
  int32_t start_req;
  // fp8 rows only, so last: per tile (mod 4), the keys' scales by group
  alignas(16) float scales[4][4][kTileKeys];
};
template <bool kFp4>
constexpr int tree_smem() {
  return Shared<kFp4>::kOffCtl + int(kFp4 ? offsetof(TreeCtl, scales) : sizeof(TreeCtl)) + 1024;
}
static_assert(tree_smem<false>() <= 227 * 1024 && tree_smem<true>() <= 227 * 1024, "shared memory per CTA");

struct SplitTile {
  int32_t row, rows;     // first row (of T * H) and how many
  int32_t parts, place;  // partial results: `place`, then the first of each pair behind
};

// Every wait is bounded: it gives up after so many looks, each of which
// suspends the thread for up to kSuspendNs (2.6 s in all), or when another wait
// of the CTA has; the first to do so leaves its site in ctl->abort, which the
// CTA reports at its end.  A few instructions a wait matter: the roles' code
// runs once a tile each, and from some 90 KB of it on warps wait for
// instructions (the batch of 32 requests above: 5.1 ms with waits that read the
// timer and every loop unrolled, 154 KB; 2.18 with 102 KB, 2.02 with 91, whose
// loops that run once a launch or an item are not unrolled).
//
// All but those of the list for a place and for the list's next item are for
// work on a few tiles.  Those are for a whole item (2 us a key tile: 2.6 s at 80
// M keys), so they look longer; when the items are not worked on, another wait
// gives up and ends them.
constexpr int kLooks = 1 << 17, kLooksForItem = 1 << 28;

__noinline__ __device__ bool look_again(uint64_t* bar, uint32_t parity, volatile int* abort, int site, int looks) {
#pragma unroll 1
  for (int n = looks; n > 0 && *abort == 0; --n)
    if (mbar_try_wait(bar, parity)) return true;
  if (*abort == 0) *abort = site + 1;
  return false;
}

__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, TreeCtl* ctl, int site,
                                          int looks = kLooks) {
  return mbar_try_wait(bar, parity) || look_again(bar, parity, &ctl->abort, site, looks);
}

// Of the first n positions, how many pool d holds.
__device__ __forceinline__ int32_t pool_rows(const TreeDecodeArgs& a, int32_t n, int32_t d) {
  const int32_t full = int32_t(fastdiv(uint32_t(n), a.div_ID));
  const int64_t rest = int64_t(n) - int64_t(full) * a.div_ID.d - int64_t(d) * a.interleave;
  return full * a.interleave + int32_t(min(max(rest, int64_t(0)), int64_t(a.interleave)));
}

// A windowed call lists, of a prefix's positions, the first sinks and those in
// the window of a node that follows the prefix directly: from here on.
__device__ __forceinline__ int32_t window_start(const TreeDecodeArgs& a, int32_t prefix) {
  return max(prefix - a.window + 1, min(a.sinks, prefix));
}

// Keys of a prefix that are listed of pool d.
template <bool kWindow>
__device__ __forceinline__ int32_t pool_keys(const TreeDecodeArgs& a, int32_t prefix, int32_t d) {
  const int32_t n = pool_rows(a, prefix, d);
  if (!kWindow) return n;
  return pool_rows(a, min(a.sinks, prefix), d) + n - pool_rows(a, window_start(a, prefix), d);
}

// The last position that sees a listed key at position t, counted from the
// prefix's end at `length` (nodes' positions are less than 256 past it).
__device__ __forceinline__ int32_t seen_until(const TreeDecodeArgs& a, int32_t t, int32_t length) {
  return t < a.sinks ? 255 : int32_t(min(int64_t(t) + a.window - 1 - length, int64_t(255)));
}

// A node's position counted from there: as given, where a tree of max_nodes
// nodes may have it.
__device__ __forceinline__ int32_t node_position(const TreeDecodeArgs& a, int32_t row, int32_t length) {
  return min(max(a.positions[row], length), length + a.max_nodes - 1) - length;
}

// What a request brings: its rows and keys.  No rows (and an error bit) when
// they lie outside T or are too many; no keys when its prefix is out of range.
struct Request {
  int32_t first, nodes, prefix, keys;  // prefix: as given, -1 when out of range
};

template <bool kWindow>
__device__ __forceinline__ Request load_request(const TreeDecodeArgs& a, int32_t b, unsigned& err) {
  Request r;
  r.first = a.row_start[b];
  const int64_t n = int64_t(a.row_start[b + 1]) - r.first;
  r.prefix = a.prefix_lens[b];
  const bool rows_ok = r.first >= 0 && n >= 0 && n <= a.max_nodes && r.first + n <= a.T;
  if (!rows_ok) err |= SMLA_DEVERR_TREE;
  r.nodes = rows_ok ? int32_t(n) : 0;
  r.keys = 0;
  if (r.prefix < 0 || r.prefix > a.max_prefix) {
    if (rows_ok && n > 0) err |= SMLA_DEVERR_CONTEXT;
    r.prefix = -1;
  } else {
    const int32_t listed = kWindow ? min(a.sinks, r.prefix) + r.prefix - window_start(a, r.prefix) : r.prefix;
    r.keys = (a.rank < 0 ? listed : pool_keys<kWindow>(a, r.prefix, a.rank)) + r.nodes;
  }
  return r;
}

__device__ __forceinline__ int32_t row_tiles(const TreeDecodeArgs& a, const Request& r) {
  return int32_t((int64_t(r.nodes) * a.H + kPairRows - 1) / kPairRows);
}
// A request without keys has one tile of none.
__device__ __forceinline__ int32_t key_tiles(const Request& r) {
  return max((r.keys + kTileKeys - 1) / kTileKeys, 1);
}
// Units of a row tile: its key tiles where it may be cut, else one.
__device__ __forceinline__ int32_t tile_units(const TreeDecodeArgs& a, const Request& r) {
  return a.split ? key_tiles(r) : 1;
}

// x / y of numbers that seldom need 64 bits.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return uint32_t(x) / uint32_t(y);
  return x / y;
}

// A key's place while its table entry is on the way.
struct Place {
  int32_t d, offset, entry;
  int32_t until;  // windowed calls
  bool prefix, live;
};

template <bool kWindow>
__device__ __forceinline__ Place find_key(const TreeDecodeArgs& a, const Keys& keys, int32_t req, int32_t i) {
  Place p;
  p.live = i < keys.total;
  p.prefix = i < keys.prefix;
  p.d = max(a.rank, 0);
  p.offset = 0;
  p.entry = -1;
  p.until = 255;
  if (p.prefix) {
    if (a.rank < 0)
      while (i >= keys.before[p.d + 1]) ++p.d;
    int32_t lp = i - keys.before[p.d];
    if (kWindow && lp >= keys.sinks[p.d]) {
      lp += keys.gap[p.d];
      if (lp < keys.edge[p.d]) {
        const int32_t round = int32_t(uint32_t(lp) / uint32_t(a.interleave));
        const int64_t t = (int64_t(round) * a.D + p.d) * a.interleave + (lp - round * a.interleave);
        p.until = seen_until(a, int32_t(t), keys.length);
      }
    }
    const int32_t col = int32_t(fastdiv(uint32_t(lp), a.div_bs));
    p.offset = lp - col * a.block_size;
    if (col < a.bt_width[p.d]) p.entry = a.bts[p.d][req * a.bt_stride[p.d] + col];
  } else if (p.live) {
    const int32_t row = keys.first + (i - keys.prefix);
    p.entry = a.draft_slots[p.d][row];
    if (a.rank < 0)
      while (p.entry < 0 && p.d + 1 < a.D) p.entry = a.draft_slots[++p.d][row];
    if (kWindow) p.until = seen_until(a, keys.length + node_position(a, row, keys.length), keys.length);
  }
  return p;
}

// Address of the key's cache row, or null (with an error bit, where it is
// one).
__device__ __forceinline__ const uint8_t* key_row(const TreeDecodeArgs& a, const Place& p, int row_bytes,
                                                  unsigned& err) {
  if (!p.live) return nullptr;
  if (p.entry < 0) {
    if (p.prefix) err |= SMLA_DEVERR_BLOCK_TABLE;
    return nullptr;
  }
  const int64_t slot = p.prefix ? int64_t(p.entry) * a.block_size + p.offset : p.entry;
  if (slot >= a.pool_slots[p.d]) {
    err |= SMLA_DEVERR_SLOT_RANGE;
    return nullptr;
  }
  return a.pools[p.d] + slot * row_bytes;
}

// fp16 values that are not finite, to zero.
__device__ __forceinline__ uint32_t only_finite(uint32_t w) {
  const __half2 v = *reinterpret_cast<const __half2*>(&w);
  return w & __heq2_mask(__hsub2(v, v), __half2half2(__ushort_as_half(0)));
}
__device__ __forceinline__ uint4 only_finite(uint4 v) {
  return make_uint4(only_finite(v.x), only_finite(v.y), only_finite(v.z), only_finite(v.w));
}

// A consumer's place in the pair's list of items.
struct Cursor {
  int item = -1, tile = 0, tiles = 0;
  bool end = false;
  __device__ __forceinline__ const Item& at(const TreeCtl* ctl) const { return ctl->items[item % kItems]; }
  // To the next item's first tile; false at the end of the list.
  __device__ __forceinline__ bool next_item(TreeCtl* ctl) {
    ++item;
    tile = 0;
    const bool ok = tree_wait(&ctl->item_full[item % kItems], (item / kItems) & 1, ctl, kWsRaw, kLooksForItem);
    end = !__all_sync(0xffffffffu, ok) || at(ctl).rows == 0;
    tiles = end ? 0 : at(ctl).tiles;
    return !end;
  }
  __device__ __forceinline__ void next_tile(TreeCtl* ctl) {
    if (!end && (item < 0 || ++tile == tiles)) next_item(ctl);
  }
};

// Hands an item's place back to the list (one arrival a warp).
__device__ __forceinline__ void leave_item(TreeCtl* ctl, int item, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&ctl->item_empty[item % kItems]);
}

// ---------------------------------------------------------------- work list
template <bool kWindow>
__device__ void list_work(const TreeDecodeArgs& a, TreeCtl* ctl, int C, int64_t units, int64_t per_pair,
                          int lane) {
  const int pair = int(blockIdx.x >> 1);
  const int64_t u_begin = per_pair * pair;
  const int64_t u_end = min(u_begin + per_pair, units);
  int64_t u = u_begin;
  int32_t req = ctl->start_req;
  int64_t in_req = ctl->start;  // units of `req` before u
  int item = 0;
  SplitTile begun = {0, 0, 0, 0};
  bool ok = true;
  while (ok && u < u_end && req < a.B) {
    unsigned ignored = 0;
    const Request r = load_request<kWindow>(a, req, ignored);
    const int32_t per_tile = tile_units(a, r);
    const int64_t all = int64_t(row_tiles(a, r)) * per_tile;
    // this lane's pool and the prefix keys up to it
    const int32_t held =
        r.prefix >= 0 && lane < a.D && (a.rank < 0 || lane == a.rank) ? pool_keys<kWindow>(a, r.prefix, lane) : 0;
    int32_t upto = held;
#pragma unroll 1
    for (int o = 1; o < kMaxMerge; o <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    int32_t tile = 0, k0 = 0;
    if (in_req != 0) {
      tile = int32_t(quotient(in_req, per_tile));
      k0 = int32_t(in_req - int64_t(tile) * per_tile);
    }
    for (; in_req < all && u < u_end; ++tile, k0 = 0) {
      const int32_t take = int32_t(min(int64_t(per_tile - k0), u_end - u));
      const bool whole = take == per_tile;
      const int slot = item % kItems;
      if (item >= kItems)
        ok = tree_wait(&ctl->item_empty[slot], (item / kItems - 1) & 1, ctl, kWsRawEmpty, kLooksForItem);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      Item& it = ctl->items[slot];
      if (lane < a.D) it.keys.before[lane] = a.rank < 0 ? upto - held : 0;
      if (lane == a.D - 1) it.keys.before[a.D] = upto;
      if (kWindow && lane < a.D && r.prefix >= 0) {
        const int32_t start = window_start(a, r.prefix);
        it.keys.sinks[lane] = pool_rows(a, min(a.sinks, r.prefix), lane);
        it.keys.gap[lane] = pool_rows(a, start, lane) - it.keys.sinks[lane];
        it.keys.edge[lane] = pool_rows(a, min(max(start, r.prefix - a.window + a.max_nodes), r.prefix), lane);
      }
      const int32_t skip = tile * kPairRows;
      const int32_t rows = min(kPairRows, r.nodes * a.H - skip);
      if (lane == 0) {
        it.keys.first = r.first;
        it.keys.nodes = r.prefix >= 0 ? r.nodes : 0;
        it.keys.total = r.keys;
        it.keys.prefix = r.keys - it.keys.nodes;
        it.keys.length = r.prefix;
        it.req = req;
        it.rows = rows;
        it.skip = skip;
        it.tile0 = a.split ? k0 : 0;
        it.tiles = a.split ? take : key_tiles(r);
        it.part = whole ? -1 : 2 * pair + (item > 0);
      }
      if (!whole && k0 == 0) {
        begun.row = r.first * a.H + skip;
        begun.rows = rows;
        begun.parts = int32_t(quotient(u + per_tile - 1, per_pair)) - pair + 1;
        begun.place = 2 * pair + (item > 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->item_full[slot]);
      ++item;
      u += take;
      in_req += take;
    }
    ++req;
    in_req = 0;
  }
  // the end of the list
  const int slot = item % kItems;
  if (ok && item >= kItems)
    ok = tree_wait(&ctl->item_empty[slot], (item / kItems - 1) & 1, ctl, kWsRawEmpty, kLooksForItem);
  if (__all_sync(0xffffffffu, ok) && lane == 0) {
    ctl->items[slot].rows = 0;
    mbar_arrive(&ctl->item_full[slot]);
  }
  if (a.split && C == 0 && lane == 0) static_cast<SplitTile*>(a.ws_desc)[pair] = begun;
}

// --------------------------------------------------------------- the keys' rows
// One warp, two keys a lane, and a tile ahead.  A missing key's row is read
// from somewhere else (a row of q is longer than a cache row): its score is
// masked, and what goes into the value tile is made finite.
template <bool kWindow>
__device__ void look_up_rows(const TreeDecodeArgs& a, TreeCtl* ctl, int row_bytes, int lane) {
  const uint8_t* elsewhere = reinterpret_cast<const uint8_t*>(a.q);
  unsigned err = 0;
  Cursor ahead;
  Place place[2];
#pragma unroll 1
  for (int t = -1;; ++t) {  // tile t is stored, t + 1 looked up
    const uint8_t* row[2];
    int32_t until[2];
    if (t >= 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        row[h] = key_row(a, place[h], row_bytes, err);
        until[h] = place[h].until;
      }
    }
    const int before = ahead.item;
    ahead.next_tile(ctl);
    if (before >= 0 && ahead.item != before) leave_item(ctl, before, lane);
    if (!ahead.end) {
      const Item& it = ahead.at(ctl);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        place[h] = find_key<kWindow>(a, it.keys, it.req, (it.tile0 + ahead.tile) * kTileKeys + 32 * h + lane);
    }
    if (t >= 0) {
      const int slot = t % kPlaces;
      if (t >= kPlaces &&
          !__all_sync(0xffffffffu, tree_wait(&ctl->place_empty[slot], (t / kPlaces - 1) & 1, ctl, kWsRawEmpty)))
        break;
      uint32_t have[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        have[h] = __ballot_sync(0xffffffffu, row[h] != nullptr);
        ctl->row[slot][32 * h + lane] = row[h] ? row[h] : elsewhere;
        if (kWindow) ctl->until[t & 7][32 * h + lane] = uint8_t(until[h]);
      }
      if (kWindow) {
        const int32_t soonest = __reduce_min_sync(0xffffffffu, min(until[0], until[1]));
        if (lane == 0) ctl->soonest[t & 15] = soonest;
      }
      if (lane == 0) ctl->valid[t & 15] = uint64_t(have[1]) << 32 | have[0];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->place_full[slot]);
    }
    if (ahead.end) break;
  }
  if (err) atomicOr(&g_decode_error, err);
}

// --------------------------------------------------------------- converters
// Whether any of a tile's keys may hold what a masked place must not show.
template <bool kWindow>
__device__ __forceinline__ bool must_mend(const TreeDecodeArgs& a, const TreeCtl* ctl, const Item& it, int tile,
                                          int g) {
  return (it.tile0 + tile + 1) * kTileKeys > it.keys.prefix || ctl->valid[g & 15] != ~0ull ||
         (kWindow && ctl->soonest[g & 15] < a.max_nodes - 1);
}

// A warp's eight rows of q on their way to the Q operand (a row's 1,152 bytes
// as nine pieces of 128, one in each block), rows past the tile's as zeros;
// each format then converts them in place.
__device__ __forceinline__ void stage_queries(const TreeDecodeArgs& a, const Item& it, uint32_t q0, int C, int w,
                                              int lane) {
  const int64_t row0 = int64_t(it.keys.first) * a.H + it.skip + kCtaRows * C;
  const int live = it.rows - kCtaRows * C;
#pragma unroll 6
  for (int k = 0; k < 8 * 72 / 32; ++k) {
    const int e = 32 * k + lane;
    const int r = 8 * w + e / 72, chunk = e % 72;  // 8 dims each
    const uint32_t at = q0 + (chunk >> 3) * kQBlock + sw128_offset(r, chunk & 7);
    if (r < live) cp_async_16(at, a.q + (row0 + r) * SMLA_QK_DIM + 8 * chunk);
    else sts128(at, make_uint4(0, 0, 0, 0));
  }
}

// 8-bit rows.  The copying warp brings this CTA's keys (codes, rope) into the
// K tiles, three tiles ahead, and both CTAs' scales.  A converter warp makes
// value rows of four keys of this CTA, whose codes come from the K tile, and
// of four of the peer's, whose half of the codes it loads a tile ahead.  16
// lanes take a key's half of the codes, 16 each; the eight chunks that a
// quarter of a warp stores together lie in eight bank groups.
struct Fp8Keys {
  static constexpr bool kFp4 = false;
  static constexpr int kRowBytes = SMLA_ROW_BYTES;
  using Sm = Shared<false>;

  // 16 codes times their scale, rounded once.  Scales from 2^-10 on split into
  // fp16 hi + lo as they are (lo is good to 2^-25, 2^-15 of the scale); any
  // scale, as 2^8 times itself against codes times 2^-8.
  static __device__ __forceinline__ void values(uint4 c, float scale, uint4* v) {
    const __half h = __float2half_rn(scale);
    const __half2 hi = __half2half2(h), lo = __half2half2(__float2half_rn(scale - __half2float(h)));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[k]), __NV_E4M3));
      const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[k] >> 16), __NV_E4M3));
      o[2 * k] = h2_bits(__hfma2(a, hi, __hmul2(a, lo)));
      o[2 * k + 1] = h2_bits(__hfma2(b, hi, __hmul2(b, lo)));
    }
    v[0] = make_uint4(o[0], o[1], o[2], o[3]);
    v[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  static __device__ __forceinline__ void any_values(uint4 c, float scale, bool mend, uint4* v) {
    __half2 hi, lo;
    split_scale(scale, hi, lo);
    v[0] = e4m3x8_scaled(make_uint2(c.x, c.y), hi, lo);
    v[1] = e4m3x8_scaled(make_uint2(c.z, c.w), hi, lo);
    if (mend) {
      v[0] = only_finite(v[0]);
      v[1] = only_finite(v[1]);
    }
  }

  // The copying warp.
  static __device__ void copy_rows(uint8_t* sm, TreeCtl* ctl, int C, int lane) {
    const uint32_t k0 = smem_u32(sm) + kQSize;
    const uint32_t to = (lane >> 3) * kKBlock;
    Cursor cur;
    for (int t = 0;; ++t) {
      const int before = cur.item;
      cur.next_tile(ctl);
      if (before >= 0 && cur.item != before) leave_item(ctl, before, lane);
      if (cur.end) break;
      const int slot = t % kPlaces, st = t % 3;
      // the K tile is free once QK^T and the converters of the tile three
      // before have read it
      const bool ready =
          tree_wait(&ctl->place_full[slot], (t / kPlaces) & 1, ctl, kWsRaw) &&
          (t < 3 || (tree_wait(&ctl->k_free[st], (t / 3 - 1) & 1, ctl, kWsFreed) &&
                     tree_wait(&ctl->k_read[st], (t / 3 - 1) & 1, ctl, kWsRawEmpty)));
      if (!__all_sync(0xffffffffu, ready)) break;
      const uint8_t* const* row = ctl->row[slot];
      const uint32_t k_tile = k0 + st * Sm::kKSize;
#pragma unroll 1
      for (int i0 = 0; i0 < kCtaKeys; i0 += 8) {
        const uint8_t* p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = row[kCtaKeys * C + i0 + i];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          cp_async_16(k_tile + to + sw128_offset(i0 + i, lane & 7), p[i] + 16 * lane);
      }
      const uint32_t table = smem_u32(&ctl->scales[t & 3][lane & 3][lane >> 2]);
#pragma unroll 1
      for (int i0 = 0; i0 < 8; i0 += 4) {
        const uint8_t *rope[4], *scale[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rope[i] = row[kCtaKeys * C + 4 * (i0 + i) + (lane >> 3)];
          scale[i] = row[8 * (i0 + i) + (lane >> 2)];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cp_async_16(k_tile + 4 * kKBlock + sw128_offset(4 * (i0 + i) + (lane >> 3), lane & 7),
                      rope[i] + 528 + 16 * (lane & 7));
          cp_async_4(table + 32 * (i0 + i), scale[i] + 512 + 4 * (lane & 3));
        }
      }
      cp_async_arrive(&ctl->k_full[st]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->place_empty[slot]);
    }
    cp_async_wait_all();
  }

  static __device__ __forceinline__ __nv_bfloat162 magnitudes(uint32_t w) {
    return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  }
  // The staged rows as the A operands of QK^T, eight a warp, two at a time.
  static __device__ __forceinline__ void convert_queries(uint32_t q0, float* row_scale, int w, int lane) {
    const uint32_t at = q0 + (lane >> 2) * kQBlock;  // dims 16 lane ..
    const uint32_t to = q0 + (lane >> 3) * kQBlock;
#pragma unroll 1
    for (int r0 = 8 * w; r0 < 8 * w + 8; r0 += 2) {
      uint4 v[2][2], rope[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[i][0] = lds128(at + sw128_offset(r0 + i, 2 * (lane & 3)));
        v[i][1] = lds128(at + sw128_offset(r0 + i, 2 * (lane & 3) + 1));
        rope[i] = lds128(q0 + 8 * kQBlock + sw128_offset(r0 + i, lane & 7));
      }
      uint32_t top[2], top_rope[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        auto most = [](uint4 x) {
          return __hmax2_nan(__hmax2_nan(magnitudes(x.x), magnitudes(x.y)), __hmax2_nan(magnitudes(x.z), magnitudes(x.w)));
        };
        auto larger = [](__nv_bfloat162 m) {  // its bits: a NaN's are above infinity's
          const uint32_t bits = *reinterpret_cast<const uint32_t*>(&m);
          return max(bits & 0xffffu, bits >> 16);
        };
        top[i] = larger(__hmax2_nan(most(v[i][0]), most(v[i][1])));
        top_rope[i] = larger(most(rope[i]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = __reduce_max_sync(0xffffffffu, top[i]);
        top_rope[i] = __reduce_max_sync(0xffffffffu, top_rope[i]);
      }
      __syncwarp();  // every lane has read the rows
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + i;
        const uint32_t x[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
        // the latents times 2^up have their largest value in [2^7, 2^8); the rope
        // part stays as it is (times 2^up it would overflow beside tiny latents)
        const int exponent = int(top[i] >> 7);
        const int up = top[i] == 0 ? 0 : max(min(134 - exponent, 120), -120);
        const float by = __uint_as_float(uint32_t(127 + up) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hi[k] = lo[k] = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // times 2^up as fp16: exact from 2^-17 on, within 2^-25 below
            const uint32_t w2 = x[2 * k + j];
            const __half2 f = __floats2half2_rn(__uint_as_float(w2 << 16) * by, __uint_as_float(w2 & 0xffff0000u) * by);
            const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
            const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3));
            hi[k] |= uint32_t(c) << (16 * j);
            lo[k] |= uint32_t(__nv_cvt_halfraw2_to_fp8x2(__hsub2(f, b), __NV_SATFINITE, __NV_E4M3)) << (16 * j);
          }
        }
        sts128(to + sw128_offset(r, lane & 7), make_uint4(hi[0], hi[1], hi[2], hi[3]));
        sts128(to + 4 * kQBlock + sw128_offset(r, lane & 7), make_uint4(lo[0], lo[1], lo[2], lo[3]));
        // a query that is not finite has no score that is
        if (lane == 0) {
          const bool finite = max(top[i], top_rope[i]) < 0x7f80u;
          row_scale[r] = __uint_as_float(finite ? uint32_t(127 - up) << 23 : 0x7fc00000u);
          if (!finite) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
        }
      }
    }
  }

  template <bool kWindow>
  static __device__ void run(const TreeDecodeArgs& a, uint8_t* sm, TreeCtl* ctl, int C, int w, int lane) {
    constexpr int kPer = kWarpKeys / 2;  // keys of a half warp
    const uint32_t base = smem_u32(sm);
    const uint32_t v_full = map_to_cta(smem_u32(&ctl->v_full[0]), 0), q_full = map_to_cta(smem_u32(&ctl->q_full), 0);
    const int first = kWarpKeys * w;
    const int own_keys = kCtaKeys * C + first, peer_keys = kCtaKeys * (1 - C) + first;
    const int j = lane & 15, key = lane >> 4;  // 16 codes from 16 j on; of keys key, key + 2, ...
    const int swap = (j >> 2) & 1, group = 2 * C + (j >> 3);
    const uint32_t from = base + kQSize + group * kKBlock;
    const uint32_t to = base + Sm::kOffV + (j >> 2) * kVBlock;
    bool bad = false, ok = true;
    uint4 peer[kPer];
    auto load_peer = [&](int t) {
      const int slot = t % kPlaces;
      if (!__all_sync(0xffffffffu, tree_wait(&ctl->place_full[slot], (t / kPlaces) & 1, ctl, kWsRaw))) return false;
      const uint8_t* p[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) p[i] = ctl->row[slot][peer_keys + 2 * i + key];
#pragma unroll
      for (int i = 0; i < kPer; ++i) peer[i] = ldg_stream(p[i] + 256 * C + 16 * j);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->place_empty[slot]);
      return true;
    };
    Cursor ahead, now;
    ahead.next_tile(ctl);
    if (!ahead.end) {
      stage_queries(a, ahead.at(ctl), base, C, w, lane);  // while the keys are looked up
      ok = load_peer(0);
    }
    int st = 0, lap = 0;  // the K tile and its uses
    for (int g = 0; ok; ++g) {
      // to the next tile; an item is handed back when it is left
      const int before = now.item;
      now.next_tile(ctl);
      if (before >= 0 && now.item != before) leave_item(ctl, before, lane);
      if (now.end) break;
      const Item& it = now.at(ctl);
      if (now.tile == 0) {  // the item's rows, in place of the last one's
        if (g > 0) {
          if (!__all_sync(0xffffffffu, tree_wait(&ctl->k_free[(g - 1) % 3], ((g - 1) / 3) & 1, ctl, kWsFreed))) break;
          stage_queries(a, it, base, C, w, lane);
        }
        cp_async_wait_all();
        __syncwarp();
        convert_queries(base, ctl->row_scale[now.item & 1], w, lane);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(q_full);  // written: every lane has fenced its part
      }
      {
        // V: free once PV of the tile two before is done
        ok = tree_wait(&ctl->k_full[st], lap & 1, ctl, kWsRaw) &&
             (g < 2 || tree_wait(&ctl->pv[g & 1], ((g >> 1) - 1) & 1, ctl, kWsPvDone));
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t k_tile = from + st * Sm::kKSize, v_tile = to + (g & 1) * kVSize;
        const float* scales = ctl->scales[g & 3][group];
        const bool mend = must_mend<kWindow>(a, ctl, it, now.tile, g);
        uint4 own[kPer];
        float s_own[kPer], s_peer[kPer];
        bool plain = !mend;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          own[i] = lds128(k_tile + sw128_offset(first + 2 * i + key, j & 7));
          s_own[i] = scales[own_keys + 2 * i + key];
          s_peer[i] = scales[peer_keys + 2 * i + key];
          plain &= s_own[i] >= 0x1p-10f && s_own[i] <= 65504.f / 448.f;
          plain &= s_peer[i] >= 0x1p-10f && s_peer[i] <= 65504.f / 448.f;  // (a NaN is neither)
        }
        // chunks in the order this lane stores them
        auto turned = [&](uint4 c) { return swap ? make_uint4(c.z, c.w, c.x, c.y) : c; };
        auto store = [&](int i, const uint4* x, const uint4* y) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t c = 2 * (j & 3) + (s ^ swap);
            sts128(v_tile + sw128_offset(own_keys + 2 * i + key, c), x[s]);
            sts128(v_tile + sw128_offset(peer_keys + 2 * i + key, c), y[s]);
          }
        };
        if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            uint4 x[2], y[2];
            values(turned(own[i]), s_own[i], x);
            values(turned(peer[i]), s_peer[i], y);
            store(i, x, y);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kPer; ++i) {
            uint4 c = own[0], d = peer[0];
            float s = s_own[0], s2 = s_peer[0];
#pragma unroll
            for (int k = 1; k < kPer; ++k) {
              if (i == k) {
                c = own[k];
                d = peer[k];
                s = s_own[k];
                s2 = s_peer[k];
              }
            }
            uint4 x[2], y[2];
            any_values(turned(c), s, mend, x);
            any_values(turned(d), s2, mend, y);
            bad |= scale_out_of_range(s) && ((ctl->valid[g & 15] >> (own_keys + 2 * i + key)) & 1);
            bad |= scale_out_of_range(s2) && ((ctl->valid[g & 15] >> (peer_keys + 2 * i + key)) & 1);
            store(i, x, y);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_at(v_full + 8 * (g & 1));  // written: every lane has fenced its part
          mbar_arrive(&ctl->k_read[st]);
        }
        ahead.next_tile(ctl);
        if (!ahead.end) ok = load_peer(g + 1);
      }
      if (++st == 3) {
        st = 0;
        ++lap;
      }
    }
    if (bad) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
  }
};

// 4-bit rows: K and V tiles from registers, loaded a tile ahead.  8 lanes take
// a key's half of the codes, 32 each.
struct Fp4Keys {
  static constexpr bool kFp4 = true;
  static constexpr int kRowBytes = SMLA_FP4_ROW_BYTES;
  using Sm = Shared<true>;

  static __device__ __forceinline__ void convert_queries(uint32_t q0, int w, int lane) {
    uint32_t over = 0;
#pragma unroll 2
    for (int k = 0; k < 8 * 72 / 32; ++k) {
      const int e = 32 * k + lane;
      const int r = 8 * w + e / 72, chunk = e % 72;
      const uint32_t at = q0 + (chunk >> 3) * kQBlock + sw128_offset(r, chunk & 7);
      const uint4 v = lds128(at);
      over |= bf16x8_over_fp16(v);
      sts128(at, bf16x8_to_f16x8(v));
    }
    if (over) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
  }

  struct Half {
    uint4 code;
    uint32_t scale;
    __device__ __forceinline__ void load(const uint8_t* row, int half, int lane) {
      code = ldg_stream(row + 128 * half + 16 * (lane & 7));
      scale = reinterpret_cast<const uint16_t*>(row + 256 + 16 * half)[lane & 7];
    }
    // the lane's four chunks, in the order it stores them
    __device__ __forceinline__ void values(uint4* v, int lane) const {
      const int rot = (lane >> 1) & 3;
      const __half2 s = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(scale), __NV_E4M3));
      const __half2 s0 = __low2half2(s), s1 = __high2half2(s);
      uint4 c = code;
      if (rot & 1) c = make_uint4(c.y, c.z, c.w, c.x);
      if (rot & 2) c = make_uint4(c.z, c.w, c.x, c.y);
      const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) v[m] = e2m1x8_scaled(word[m], ((m + rot) & 3) < 2 ? s0 : s1);
    }
    __device__ __forceinline__ bool nan() const { return (((scale & 0x7f7fu) + 0x0101u) & 0x8080u) != 0; }
  };

  template <bool kWindow>
  static __device__ void run(const TreeDecodeArgs& a, uint8_t* sm, TreeCtl* ctl, int C, int w, int lane) {
    constexpr int kPer = kWarpKeys / 4;  // keys of a quarter warp
    const uint32_t base = smem_u32(sm);
    const uint32_t k_full = map_to_cta(smem_u32(&ctl->k_full[0]), 0), v_full = map_to_cta(smem_u32(&ctl->v_full[0]), 0),
                   q_full = map_to_cta(smem_u32(&ctl->q_full), 0);
    const int first = kWarpKeys * w;
    const int own_keys = kCtaKeys * C + first, peer_keys = kCtaKeys * (1 - C) + first;
    const int j = lane & 7, key = lane >> 3, rot = (lane >> 1) & 3;
    uint32_t over = 0;
    bool bad = false, ok = true;
    Half own[kPer], other[kPer], peer[kPer];
    uint4 rope[kPer];
    auto load = [&](int t) {
      const int slot = t % kPlaces;
      if (!__all_sync(0xffffffffu, tree_wait(&ctl->place_full[slot], (t / kPlaces) & 1, ctl, kWsRaw))) return false;
      const uint8_t *p[kPer], *q[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        p[i] = ctl->row[slot][own_keys + 4 * i + key];
        q[i] = ctl->row[slot][peer_keys + 4 * i + key];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        own[i].load(p[i], C, lane);
        other[i].load(p[i], 1 - C, lane);
        rope[i] = ldg_stream(p[i] + 288 + 16 * j);
        peer[i].load(q[i], C, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->place_empty[slot]);
      return true;
    };
    Cursor ahead, now;
    ahead.next_tile(ctl);
    if (!ahead.end) {
      stage_queries(a, ahead.at(ctl), base, C, w, lane);  // while the keys are looked up
      ok = load(0);
    }
    for (int g = 0; ok; ++g) {
      const int before = now.item;
      now.next_tile(ctl);
      if (before >= 0 && now.item != before) leave_item(ctl, before, lane);
      if (now.end) break;
      const Item& it = now.at(ctl);
      const int st = g & 1;
      if (now.tile == 0) {  // the item's rows, in place of the last one's
        if (g > 0) {
          if (!__all_sync(0xffffffffu, tree_wait(&ctl->k_free[(g - 1) & 1], ((g - 1) >> 1) & 1, ctl, kWsFreed))) break;
          stage_queries(a, it, base, C, w, lane);
        }
        cp_async_wait_all();
        __syncwarp();
        convert_queries(base, w, lane);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(q_full);
      }
      const uint64_t valid = ctl->valid[g & 15];
      // K: free once QK^T of the tile two before is done
      if (g >= 2 && !__all_sync(0xffffffffu, tree_wait(&ctl->k_free[st], ((g >> 1) - 1) & 1, ctl, kWsFreed))) break;
      const uint32_t k_tile = base + kQSize + st * Sm::kKSize;
      const uint32_t k_block = k_tile + (j >> 1) * kKBlock;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = first + 4 * i + key;
        if ((valid >> (own_keys + 4 * i + key)) & 1) {
          bad |= own[i].nan() || other[i].nan();
          over |= bf16x8_over_fp16(rope[i]);
        }
        uint4 x[4], y[4];
        own[i].values(x, lane);
        other[i].values(y, lane);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t at = k_block + sw128_offset(row, 4 * (j & 1) + ((m + rot) & 3));
          sts128(at + 4 * C * kKBlock, x[m]);
          sts128(at + 4 * (1 - C) * kKBlock, y[m]);
        }
        sts128(k_tile + 8 * kKBlock + sw128_offset(row, j), bf16x8_to_f16x8(rope[i]));
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(k_full + 8 * st);  // (K, V and Q: as over 8-bit rows)
      // V: free once PV of the tile two before is done
      if (g >= 2 && !__all_sync(0xffffffffu, tree_wait(&ctl->pv[st], ((g >> 1) - 1) & 1, ctl, kWsPvDone))) break;
      const bool mend = must_mend<kWindow>(a, ctl, it, now.tile, g);
      const uint32_t v_block = base + Sm::kOffV + st * kVSize + (j >> 1) * kVBlock;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        uint4 x[4], y[4];
        own[i].values(x, lane);
        peer[i].values(y, lane);
        if (mend) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            x[m] = only_finite(x[m]);
            y[m] = only_finite(y[m]);
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int c = 4 * (j & 1) + ((m + rot) & 3);
          sts128(v_block + sw128_offset(own_keys + 4 * i + key, c), x[m]);
          sts128(v_block + sw128_offset(peer_keys + 4 * i + key, c), y[m]);
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(v_full + 8 * st);
      ahead.next_tile(ctl);
      if (!ahead.end) ok = load(g + 1);
    }
    if (bad || over) atomicOr(&g_decode_error, SMLA_DEVERR_RANGE);
  }
};

// ------------------------------------------------------------------- MMAs
// The first CTA's warp; the peer's keys have landed when its own says so.
template <class F>
__device__ void issue_mmas(uint8_t* sm, TreeCtl* ctl, uint32_t tb, int lane) {
  using Sm = Shared<F::kFp4>;
  constexpr int kSt = Sm::kStages;
  constexpr uint32_t qk_desc = idesc_f16_f32(128, kTileKeys, false, false);  // fp16, and e4m3 in its kind
  constexpr uint32_t rope_desc = idesc_bf16_f32(128, kTileKeys);
  constexpr uint32_t pv_desc = idesc_f16_f32(128, 256, false, true);
  const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
  const uint32_t tbu = __shfl_sync(0xffffffffu, tb, 0);
  const bool leader = elect_one();
  Cursor cur;
  int g = 0;  // tiles so far
  bool ok = true;
  while (ok && cur.next_item(ctl)) {
    const int n = cur.tiles;
    leave_item(ctl, cur.item, lane);
    for (int j = 0; j <= n; ++j) {
      if (j < n) {
        const int t = g + j, st = t % kSt;
        ok = tree_wait(&ctl->k_full[st], (t / kSt) & 1, ctl, kWsFull);
        if (!F::kFp4) ok = ok && tree_wait(&ctl->k_peer[st], (t / kSt) & 1, ctl, kWsFull);
        ok = ok && (j > 0 || tree_wait(&ctl->q_full, cur.item & 1, ctl, kWsQReady));
        const uint64_t ad = sdesc_sw128(base, 16, 1024);
        const uint64_t bd = sdesc_sw128(base + kQSize + st * Sm::kKSize, 16, 1024);
        if constexpr (F::kFp4) {
          ok = ok && (t < 2 || tree_wait(&ctl->s_read[t & 1], ((t >> 1) - 1) & 1, ctl, kWsSFree));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll 1
            for (int q = 0; q < 9; ++q)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss_f16_pair(tbu + kScoreCol + 32 * (t & 1), ad + uint64_t(q * (kQBlock >> 4) + 2 * k),
                                bd + uint64_t(q * (kKBlock >> 4) + 2 * k), qk_desc, q > 0 || k > 0);
            mma_commit_pair(&ctl->qk[t & 1]);
          }
        } else {
          // Groups of 128 codes, 32 an MMA, in two halves: the first is made
          // while the softmax reads the second of the tile before.
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            ok = __all_sync(0xffffffffu, ok && (t == 0 || tree_wait(&ctl->s_read[h], (t - 1) & 1, ctl, kWsSFree)));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              if (h == 0) fence_async_shared();  // the copies were generic writes
#pragma unroll 1
              for (int q = 2 * h; q < 2 * h + 2; ++q) {
                const uint64_t qd = ad + uint64_t(q * (kQBlock >> 4)), kd = bd + uint64_t(q * (kKBlock >> 4));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  mma_ss_f8_pair(tbu + kScoreCol + 32 * q, qd + 2 * k, kd + 2 * k, qk_desc, k > 0);
                  mma_ss_f8_pair(tbu + kScoreCol + 32 * q, qd + 4 * (kQBlock >> 4) + 2 * k, kd + 2 * k, qk_desc, 1);
                }
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (leader) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss_f16_pair(tbu + kScoreCol + 128, ad + uint64_t(8 * (kQBlock >> 4) + 2 * k),
                              bd + uint64_t(4 * (kKBlock >> 4) + 2 * k), rope_desc, k > 0);
            mma_commit_pair(&ctl->qk[0]);
          }
        }
        if (leader) mma_commit_pair(&ctl->k_free[st]);
        __syncwarp();
      }
      if (j > 0) {
        const int t = g + j - 1, pb = t % Sm::kProbs;
        ok = tree_wait(&ctl->v_full[t & 1], (t >> 1) & 1, ctl, kWsFull) &&
             tree_wait(&ctl->p_full[pb], (t / Sm::kProbs) & 1, ctl, kWsPFull) &&
             (j > 1 || cur.item == 0 || tree_wait(&ctl->out_read, (cur.item - 1) & 1, ctl, kWsSFree));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t ad = sdesc_sw128(base + Sm::kOffP + pb * Sm::kPSize, 16, 1024);
          const uint32_t v = base + Sm::kOffV + (t & 1) * kVSize;
#pragma unroll 1
          for (int k = 0; k < kTileKeys / 16; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mma_ss_f16_pair(tbu + kOutCol + 128 * i, ad + 2 * k,
                              sdesc_sw128(v + 2 * i * kVBlock, kVBlock, 1024) + uint64_t(k * (2048 >> 4)), pv_desc,
                              j > 1 || k > 0);
          mma_commit_pair(&ctl->pv[t & 1]);
        }
        __syncwarp();
      }
    }
    g += n;
  }
  // every MMA has completed before tensor memory is given back
  if (leader) mma_commit_pair(&ctl->end);
  __syncwarp();
}

// The second CTA's: tells the first's when its copies of a K tile have landed.
template <class F>
__device__ void tell_peer(TreeCtl* ctl, int lane) {
  const uint32_t k_peer = map_to_cta(smem_u32(&ctl->k_peer[0]), 0);
  Cursor cur;
  int t = 0;
  while (cur.next_item(ctl)) {
    const int n = cur.tiles;
    leave_item(ctl, cur.item, lane);
    for (int j = 0; !F::kFp4 && j < n; ++j, ++t) {
      if (!__all_sync(0xffffffffu, tree_wait(&ctl->k_full[t % 3], (t / 3) & 1, ctl, kWsFull))) return;
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(k_peer + 8 * (t % 3));  // copied: this warp has waited for it and fenced
    }
  }
}

// ------------------------------------------------------- softmax and output
// 32 bits of a row's mask from node j0 on; nodes before 0 are prefix keys,
// which every row sees.
__device__ __forceinline__ uint32_t seen_from(const uint64_t* mask, int words, int j0) {
  if (j0 <= -32) return 0xffffffffu;
  if (j0 < 0) return (uint32_t(mask[0]) << -j0) | ((1u << -j0) - 1u);
  const int w = j0 >> 6, s = j0 & 63;
  if (w >= words) return 0;
  uint64_t x = mask[w] >> s;
  if (s > 32 && w + 1 < words) x |= mask[w + 1] << (64 - s);
  return uint32_t(x);
}

// Windowed calls, of a tile with keys that not every node sees: which of 16 keys
// the item's row sees.
__noinline__ __device__ uint32_t in_window(const TreeDecodeArgs& a, const Item& it, int row, const uint8_t* until) {
  const int32_t position = node_position(a, it.keys.first + (it.skip + row) / a.H, it.keys.length);
  uint32_t seen = 0;
#pragma unroll 1
  for (int k = 0; k < 16; ++k) seen |= uint32_t(position <= until[k]) << k;
  return seen;
}

template <class F, bool kWindow>
__device__ void softmax_rows(const TreeDecodeArgs& a, uint8_t* sm, TreeCtl* ctl, uint32_t tb, int C, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  // the thread's row; which 32 keys and 256 value dims its lane holds, and
  // which half of those are the thread's
  const int r = tid & 63, half = (tid >> 6) & 1, part = tid >> 7;
  const uint32_t lanes = tmem_addr(tb, 32 * (warp & 3), 0);
  const uint32_t p_row = smem_u32(sm) + Shared<F::kFp4>::kOffP;
  const uint32_t s_read = map_to_cta(smem_u32(&ctl->s_read[0]), 0), p_full = map_to_cta(smem_u32(&ctl->p_full[0]), 0),
                 out_read = map_to_cta(smem_u32(&ctl->out_read), 0);
  Cursor cur;
  int g = 0;
  bool ok = true;
  while (ok && cur.next_item(ctl)) {
    const Item& it = cur.at(ctl);
    const int n = cur.tiles;
    const int row = kCtaRows * C + r;  // of the tile
    const bool live = row < it.rows;
    const int64_t out_row = int64_t(it.keys.first) * a.H + it.skip + row;
    const uint64_t* mask =
        a.masks + (live ? int64_t(it.keys.first) + (it.skip + row) / a.H : it.keys.first) * a.mask_words;
    // the reference is a score, not its product with c2: of scores so large that
    // the product rounds by more than fp16's range, the largest still has p = 1
    float m_ref = -INFINITY, l = 0.f;
    const float c2 = a.sm_scale * kLog2e;
    float latents = 1.f;  // fp8 rows: the row's scale
    const int prefix = it.keys.prefix;
    int first = it.tile0 * kTileKeys + kCtaKeys * half + 16 * part;  // key of s[0]
    for (int j = 0; j < n; ++j, ++g, first += kTileKeys) {
      const int b = g & 1;
      const uint32_t scores = lanes + kScoreCol + 16 * part;
      // the mask's words are on their way while the scores are computed
      const uint32_t seen = first + 16 > prefix ? seen_from(mask, a.mask_words, first - prefix) : 0xffffu;
      uint32_t s[16];
      if constexpr (F::kFp4) {
        ok = __all_sync(0xffffffffu, tree_wait(&ctl->qk[b], (g >> 1) & 1, ctl, kWsSFull));
        if (!ok) break;
        tc_fence_after();
        tmem_ld16(scores + 32 * b, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(s_read + 8 * b);  // read: wait::ld, fence
      } else {
        // sum = scores of groups 0, 1 by their scales, then of 2, 3 and the rope;
        // the scales are asked for while the scores are on their way
        uint64_t sum[8];
        uint32_t x[2][16];
        float4 f[2][4];
        auto scales = [&](int q) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4* sc = reinterpret_cast<const float4*>(&ctl->scales[g & 3][q + i][kCtaKeys * half + 16 * part]);
#pragma unroll
            for (int k = 0; k < 4; ++k) f[i][k] = sc[k];
          }
        };
        auto add = [&](int i, bool set) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sum[2 * k] = fma2(pack2(x[i][4 * k], x[i][4 * k + 1]), pack2(f[i][k].x, f[i][k].y), set ? 0 : sum[2 * k]);
            sum[2 * k + 1] =
                fma2(pack2(x[i][4 * k + 2], x[i][4 * k + 3]), pack2(f[i][k].z, f[i][k].w), set ? 0 : sum[2 * k + 1]);
          }
        };
        ok = __all_sync(0xffffffffu, tree_wait(&ctl->qk[0], g & 1, ctl, kWsSFull));
        if (!ok) break;
        if (j == 0) latents = ctl->row_scale[cur.item & 1][r];
        tc_fence_after();
        tmem_ld16(scores, x[0]);
        tmem_ld16(scores + 32, x[1]);
        scales(0);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(s_read);  // read: wait::ld, fence
        add(0, true);
        add(1, false);
        tmem_ld16(scores + 64, x[0]);
        tmem_ld16(scores + 96, x[1]);
        tmem_ld16(scores + 128, s);
        scales(2);
        tmem_ld_wait();
        tc_fence_before();
        add(0, false);
        add(1, false);
        __syncwarp();
        if (lane == 0) mbar_arrive_at(s_read + 8);  // the scales have been read, too
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = unpack2(sum[k]);
          s[2 * k] = __float_as_uint(fmaf(f.x, latents, __uint_as_float(s[2 * k])));
          s[2 * k + 1] = __float_as_uint(fmaf(f.y, latents, __uint_as_float(s[2 * k + 1])));
        }
      }
      uint32_t see = seen & uint32_t(ctl->valid[g & 15] >> (kCtaKeys * half + 16 * part)) & 0xffffu;
      if (kWindow && live && ctl->soonest[g & 15] < a.max_nodes - 1)
        see &= in_window(a, it, row, &ctl->until[g & 7][kCtaKeys * half + 16 * part]);
      if (see != 0xffffu) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (!((see >> k) & 1)) s[k] = 0xff800000u;
      }
      float top = __uint_as_float(s[0]);
#pragma unroll
      for (int k = 1; k < 16; ++k) top = fmaxf(top, __uint_as_float(s[k]));
      ctl->tops[b][tid] = top;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->top[b]);
      // p by the reference so far, while the maxima travel; once more by the new
      // one if a row's has moved
      float alpha = 1.f, sum;
      uint32_t p[8];
      bool any_moves = false;
#pragma unroll 1
      for (;;) {
        const float ref = m_ref == -INFINITY ? 0.f : m_ref;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 below = unpack2(mul2(add2(pack2(s[2 * k], s[2 * k + 1]), pack2(-ref, -ref)), pack2(c2, c2)));
          const float x = ex2(below.x), y = ex2(below.y);
          sum += x + y;
          p[k] = h2_bits(__floats2half2_rn(x, y));
        }
        if (any_moves) break;
        ok = __all_sync(0xffffffffu, tree_wait(&ctl->top[b], (g >> 1) & 1, ctl, kWsExchange));
        if (!ok) break;
        top = fmaxf(fmaxf(ctl->tops[b][r], ctl->tops[b][64 + r]), fmaxf(ctl->tops[b][128 + r], ctl->tops[b][192 + r]));
        const bool moves = (top - m_ref) * c2 > 8.f;
        any_moves = __any_sync(0xffffffffu, moves);
        if (!any_moves) break;
        if (moves) {
          alpha = ex2((m_ref - top) * c2);
          m_ref = top;
        }
      }
      if (!ok) break;
      l = l * alpha + sum;
      // the output moves once PV of the tile before has been added to it; so is
      // P's place free then, where there is one
      const bool any = j > 0 && any_moves;
      if (any || (F::kFp4 && j > 0))
        ok = __all_sync(0xffffffffu, tree_wait(&ctl->pv[b ^ 1], ((g - 1) >> 1) & 1, ctl, kWsPvDone));
      if (!ok) break;
      if (any) {
        tc_fence_after();
#pragma unroll 1
        for (int cc = 4 * part; cc < 4 * part + 4; ++cc) {
          uint32_t o[32];
          tmem_ld32(lanes + kOutCol + 32 * cc, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(lanes + kOutCol + 32 * cc, o);
        }
        tmem_st_wait();
      }
      const int pb = F::kFp4 ? 0 : b;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        sts128(p_row + pb * Shared<F::kFp4>::kPSize + sw128_offset(r, 4 * half + 2 * part + q),
               make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]));
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(p_full + 8 * pb);  // written: every lane has fenced its part
    }
    if (!ok) break;
    ctl->sums[tid] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->sum);
    ok = __all_sync(0xffffffffu, tree_wait(&ctl->sum, cur.item & 1, ctl, kWsExchange) &&
                                     tree_wait(&ctl->pv[(g - 1) & 1], ((g - 1) >> 1) & 1, ctl, kWsPvLast));
    if (!ok) break;
    tc_fence_after();
    l = (ctl->sums[r] + ctl->sums[64 + r]) + (ctl->sums[128 + r] + ctl->sums[192 + r]);
    const bool partial = it.part >= 0;
    const int64_t place = partial ? int64_t(it.part) * kPairRows + row : out_row;
    if (live && half == 0 && part == 0) {
      if (partial) {
        a.ws_ml[2 * place] = m_ref;
        a.ws_ml[2 * place + 1] = l;
      } else {
        a.lse[place] = l == 0.f ? -INFINITY : (m_ref * c2 + log2f(l)) * kLn2;
      }
    }
    uint16_t* dst = (partial ? a.ws_o : a.out) + place * SMLA_V_DIM + 256 * half;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const bool aligned = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
    for (int cc = 4 * part; cc < 4 * part + 4; ++cc) {
      uint32_t x[32], o[16];
      tmem_ld32(lanes + kOutCol + 32 * cc, x);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        // a row with no key has no output, whatever its tile's other rows hold
        const float y = l == 0.f ? 0.f : __uint_as_float(x[2 * k]) * inv;
        const float z = l == 0.f ? 0.f : __uint_as_float(x[2 * k + 1]) * inv;
        if (partial) {
          o[k] = h2_bits(__floats2half2_rn(y, z));
        } else {
          const __nv_bfloat162 v = __floats2bfloat162_rn(y, z);
          o[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
      if (live && aligned) {
        stg256(dst + 32 * cc, o);
        stg256(dst + 32 * cc + 16, o + 8);
      } else if (live) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<uint4*>(dst + 32 * cc)[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_at(out_read);  // read: wait::ld, fence
    leave_item(ctl, cur.item, lane);
  }
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <class F, bool kWindow>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTreeThreads, 1)
    tree_decode_kernel(const __grid_constant__ TreeDecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TreeCtl* ctl = reinterpret_cast<TreeCtl*>(sm + Shared<F::kFp4>::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = int(cluster_ctarank());
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->qk[i], 1);
      mbar_init(&ctl->pv[i], 1);
      mbar_init(&ctl->v_full[i], 2 * kConvWarps);  // both CTAs'
      mbar_init(&ctl->top[i], kSoftWarps);
      mbar_init(&ctl->s_read[i], 2 * kSoftWarps);
      mbar_init(&ctl->p_full[i], 2 * kSoftWarps);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ctl->k_free[i], 1);
      mbar_init(&ctl->k_full[i], F::kFp4 ? 2 * kConvWarps : 32);  // fp8: the copying warp's threads
      mbar_init(&ctl->k_read[i], kConvWarps);
      mbar_init(&ctl->k_peer[i], 1);
    }
    for (int i = 0; i < kPlaces; ++i) {
      mbar_init(&ctl->place_full[i], 1);
      mbar_init(&ctl->place_empty[i], kConvWarps + !F::kFp4);  // and the copying warp
    }
    mbar_init(&ctl->q_full, 2 * kConvWarps);
    mbar_init(&ctl->out_read, 2 * kSoftWarps);
    mbar_init(&ctl->sum, kSoftWarps);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ctl->item_full[i], 1);
      mbar_init(&ctl->item_empty[i], kSoftWarps + kConvWarps + 2 + !F::kFp4);  // all but the list's own
    }
    mbar_init(&ctl->end, 1);
    ctl->abort = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kIssueWarp) {
    tmem_alloc_pair(&ctl->tbase, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = ctl->tbase;
  cluster_arrive();
  griddep_launch_dependents();
  griddep_wait();

  // all requests' units, and where this pair's range begins: a request a
  // thread, and the later ones (of batches past the block's threads) in turn
  unsigned err = 0;
  int64_t v = 0, later = 0;
#pragma unroll 1
  for (int32_t b = tid; b < a.B; b += kTreeThreads) {
    const Request r = load_request<kWindow>(a, b, err);
    const int64_t n = int64_t(row_tiles(a, r)) * tile_units(a, r);
    if (b == tid) v = n;
    else later += n;
  }
  if (err && blockIdx.x == 0) atomicOr(&g_decode_error, err);
  int64_t upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (a.B > kTreeThreads) later = warp_sum(later);
  if (lane == 31) {
    ctl->warp_units[warp] = upto;
    ctl->warp_later[warp] = later;
  }
  __syncthreads();
  const int64_t of_warp = lane < kTreeWarps ? ctl->warp_units[lane] : 0;
  int64_t base = warp_sum(of_warp);  // of the block's first requests
  int64_t begin = warp_sum(lane < warp ? of_warp : 0) + upto - v;
  int64_t units = base;
  if (a.B > kTreeThreads) units += warp_sum(lane < kTreeWarps ? ctl->warp_later[lane] : 0);
  const int64_t pairs = gridDim.x >> 1;
  const int64_t per_pair = max(quotient(units + pairs - 1, pairs), int64_t(a.min_units));
  const int64_t u0 = per_pair * (blockIdx.x >> 1);
#pragma unroll 1
  for (int32_t b0 = 0;;) {
    if (begin <= u0 && u0 < begin + v) {
      ctl->start_req = b0 + tid;
      ctl->start = u0 - begin;
    }
    b0 += kTreeThreads;
    if (b0 >= a.B || base > u0) break;
    const int32_t b = b0 + tid;
    v = 0;
    if (b < a.B) {
      unsigned ignored = 0;
      const Request r = load_request<kWindow>(a, b, ignored);
      v = int64_t(row_tiles(a, r)) * tile_units(a, r);
    }
    upto = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    __syncthreads();  // the sums before have been read
    if (lane == 31) ctl->warp_units[warp] = upto;
    __syncthreads();
    begin = base + upto - v;
#pragma unroll 1
    for (int w = 0; w < kTreeWarps; ++w) {
      if (w < warp) begin += ctl->warp_units[w];
      base += ctl->warp_units[w];
    }
  }
  __syncthreads();
  cluster_wait();  // the peer's barriers are initialised

  if (warp < kSoftWarps) {
    softmax_rows<F, kWindow>(a, sm, ctl, tb, C, tid);
  } else if (warp < kIssueWarp) {
    F::template run<kWindow>(a, sm, ctl, C, warp - kSoftWarps, lane);
  } else {
    if (warp == kIssueWarp) {
      if (C == 0) issue_mmas<F>(sm, ctl, tb, lane);
      else tell_peer<F>(ctl, lane);
      // also after a wait that gave up: the pair's MMAs have completed
      for (int n = kLooks; n > 0 && !mbar_try_wait(&ctl->end, 0); --n) {
      }
    } else if (warp == kIssueWarp + 1) {
      list_work<kWindow>(a, ctl, C, units, per_pair, lane);
    } else if (warp == kIssueWarp + 2) {
      look_up_rows<kWindow>(a, ctl, F::kRowBytes, lane);
    } else if constexpr (!F::kFp4) {
      F::copy_rows(sm, ctl, C, lane);
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // neither CTA reaches into the other any more
  tc_fence_after();
  if (tid == 0 && ctl->abort) atomicOr(&g_decode_error, SMLA_DEVERR_TIMEOUT | (1u << (7 + ctl->abort)));
  if (warp == kIssueWarp) tmem_dealloc_pair(tb, 512);
  __syncwarp();
  cluster_sync();
}

// Merges the row tiles that were cut: with m and l the parts' references (scores)
// and sums, M = max m over the parts that hold a key, out = sum l 2^(c2 (m - M)) O
// / sum l 2^(c2 (m - M)).  One warp a row, 16 value dims a lane, parts in the order
// of their keys.
constexpr int kMergeWarps = 8;
constexpr int kMergeBlocks = kPairRows / kMergeWarps;

__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeDecodeArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = int(blockIdx.x) / kMergeBlocks;
  const int row = int(blockIdx.x) % kMergeBlocks * kMergeWarps + warp;
  griddep_launch_dependents();
  griddep_wait();
  const SplitTile t = static_cast<const SplitTile*>(a.ws_desc)[pair];
  if (row >= t.rows) return;
  auto place = [&](int i) { return int64_t(i == 0 ? t.place : 2 * (pair + i)) * kPairRows + row; };
  float top = -INFINITY;
  for (int i = lane; i < t.parts; i += 32) {
    const float m = a.ws_ml[2 * place(i)];
    if (a.ws_ml[2 * place(i) + 1] != 0.f) top = fmaxf(top, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float c2 = a.sm_scale * kLog2e;
  float sum = 0.f, acc[16] = {};
#pragma unroll 4
  for (int i = 0; i < t.parts; ++i) {
    const int64_t p = place(i);
    const float m = a.ws_ml[2 * p], l = a.ws_ml[2 * p + 1];
    const uint4* src = reinterpret_cast<const uint4*>(a.ws_o + p * SMLA_V_DIM + 16 * lane);
    const uint4 lo = src[0], hi = src[1];
    const float w = l == 0.f ? 0.f : l * exp2f((m - top) * c2);
    sum += w;
    const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[k]));
      acc[2 * k] = fmaf(w, f.x, acc[2 * k]);
      acc[2 * k + 1] = fmaf(w, f.y, acc[2 * k + 1]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    o[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint4* dst = reinterpret_cast<uint4*>(a.out + (int64_t(t.row) + row) * SMLA_V_DIM + 16 * lane);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (lane == 0) a.lse[int64_t(t.row) + row] = sum == 0.f ? -INFINITY : (top * c2 + log2f(sum)) * kLn2;
}

// How a call is laid out, from its shape alone: its pairs, and whether a row
// tile may be cut.
struct TreePlan {
  int pairs, min_units;
  bool split;
  size_t ml_off, o_off, bytes;
  size_t most_bytes;  // of this call and any with fewer rows, requests or keys
};

// Key tiles that a pair takes at least.  One request of 8 nodes and 16 heads
// over 300 / 2,000 / 4,000 positions, 8-bit rows: 18.1 / 24.3 / 46 us with 1
// (the merge then reads a part a tile), 18.7 / 23.3 / 26.4 with 2, 20.6 / 22.6 /
// 26.5 with 3.
constexpr int kMinUnits = 2;
// Row tiles of more key tiles than this are cut.  Where there are fewer than
// half as many row tiles as pairs: the request above over 300 / 500 positions
// 21.4 / 26.6 us whole, 18.7 / 20.1 cut.  Else the merge and the second loads of
// the queries cost more than an even share gives: 8 and 32 requests of 128
// heads over 300 positions 23.0 and 67.4 us whole, 25.1 and 75.5 cut; from 600
// on there is no difference.
constexpr int kWholeOfFew = 2, kWholeOfMany = 8;

TreePlan plan_tree(int32_t T, int32_t B, int32_t H, int64_t max_keys) {
  TreePlan p;
  const int64_t key_tiles = (max_keys + kTileKeys - 1) / kTileKeys;
  const int64_t row_tiles = int64_t(T) * H / kPairRows + (B < T ? B : T);
  p.split = key_tiles > (2 * row_tiles <= kPairs ? kWholeOfFew : kWholeOfMany);
  p.min_units = p.split ? kMinUnits : 1;
  auto pairs = [](int64_t units, int64_t least) {
    const int64_t need = (units + least - 1) / least;
    return int(need < 1 ? 1 : need < kPairs ? need : kPairs);
  };
  p.pairs = pairs(p.split ? row_tiles * key_tiles : row_tiles, p.min_units);
  p.ml_off = 4096;
  auto o_off = [&](int n) { return p.ml_off + size_t(2) * n * kPairRows * 2 * sizeof(float); };
  auto bytes = [&](int n) { return o_off(n) + size_t(2) * n * kPairRows * SMLA_V_DIM * sizeof(uint16_t); };
  p.o_off = o_off(p.pairs);
  p.bytes = p.split ? bytes(p.pairs) : 0;
  // fewer rows may be cut where these are not
  p.most_bytes = key_tiles > kWholeOfFew ? bytes(pairs(row_tiles * key_tiles, kMinUnits)) : 0;
  static_assert(kPairs * sizeof(SplitTile) <= 4096, "descriptors fit");
  return p;
}

}  // namespace

size_t tree_decode_workspace_bytes(int32_t T, int32_t B, int32_t H, int64_t max_keys) {
  return T > 0 && B > 0 ? plan_tree(T, B, H, max_keys).bytes : 0;
}

size_t tree_decode_most_workspace_bytes(int32_t T, int32_t B, int32_t H, int64_t max_keys) {
  return T > 0 && B > 0 ? plan_tree(T, B, H, max_keys).most_bytes : 0;
}

template <class F, bool kWindow>
static cudaError_t launch_tree(const TreeDecodeArgs& a, int pairs, cudaStream_t s) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < 64;
  if (!tracked || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(tree_decode_kernel<F, kWindow>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             tree_smem<F::kFp4>());
    if (e != cudaSuccess) return e;
    if (tracked) done[dev].store(true, std::memory_order_release);
  }
  return launch_overlapped(tree_decode_kernel<F, kWindow>, unsigned(2 * pairs), kTreeThreads, tree_smem<F::kFp4>(), s, a);
}

cudaError_t launch_tree_decode(const TreeDecodeArgs& args, int64_t max_keys, bool fp4, cudaStream_t s) {
  TreeDecodeArgs a = args;
  // a round past 2^31 positions never completes
  const uint64_t round = uint64_t(a.interleave) * uint32_t(a.D);
  a.div_ID = make_fastdiv(uint32_t(round > (1ull << 31) ? (1ull << 31) : round));
  a.div_bs = make_fastdiv(uint32_t(a.block_size));
  const TreePlan p = plan_tree(a.T, a.B, a.H, max_keys);
  a.split = p.split;
  a.min_units = p.min_units;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  a.ws_desc = ws;
  a.ws_ml = p.split ? reinterpret_cast<float*>(ws + p.ml_off) : nullptr;
  a.ws_o = p.split ? reinterpret_cast<uint16_t*>(ws + p.o_off) : nullptr;
  const bool window = a.window > 0;
  const cudaError_t e = fp4 ? (window ? launch_tree<Fp4Keys, true>(a, p.pairs, s) : launch_tree<Fp4Keys, false>(a, p.pairs, s))
                            : (window ? launch_tree<Fp8Keys, true>(a, p.pairs, s) : launch_tree<Fp8Keys, false>(a, p.pairs, s));
  if (e != cudaSuccess || !p.split) return e;
  return launch_overlapped(tree_merge_kernel, unsigned(p.pairs * kMergeBlocks), 32 * kMergeWarps, 0, s, a);
}

cudaError_t tree_decode_error_word(uint32_t* flags, bool clear) { return read_error_word(flags, clear); }

}  // namespace smla
