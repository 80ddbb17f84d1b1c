// Attention of a chunk of new tokens over a paged key/value cache, on tensor
// cores.
//
//     S = q K^T scale,  o = softmax(S) V  over the keys that each query sees,
//
// in one pass over the keys with a running maximum m and sum l (base 2).  The
// query heads that share a key head are rows of one tile: row r of a tile is
// token r / group, head r % group, so a page that is read serves all of them,
// and single tokens fill a tile as far as they can.
//
// A work item is (sequence, key head, unit of query tiles, range of key blocks).
// Two kernels, by what bounds them:
//
//   PAIR   chunks of more than one tile: tensor-bound.  An item is two 128-row
//          tiles that share every K/V block, softmax group t and issuer t for
//          tile t, as in the packed forward.
//   SPLIT  a sequence whose new rows fit one tile (single tokens, drafts):
//          bound by HBM.  The two groups take alternate key blocks of the one
//          tile.  With 32 rows or fewer (64) the tile holds them four times
//          (twice) over, 32 (64) rows apart: each warp of a group then takes
//          its own quarter (half) of a block's keys for the same rows, so the
//          exponentials of few rows are spread over all four schedulers
//          instead of one.  What the groups and warps have summed, up to
//          eight parts of a row, is joined in shared memory at the end.
//
// Roles of a CTA (384 threads, 1 per SM):
//   warps 0-7   softmax: warpgroup t's thread owns TMEM lane (row) threadIdx
//               % 128 of tile t; P = 2^(S scale log2e - m) goes back over S as
//               bf16 (the one rounding of the probabilities: the tensor cores
//               take P in V's type), O is rescaled when m grows by more than
//               2^8
//   warp 8      producer: all lanes fetch page numbers, each lane issues the
//               TMA box of its page.  PAIR takes items by cluster launch
//               control; SPLIT's are the CTA's equal share of all key blocks
//   warps 9,10  MMA issuers (S = Q K^T, O += P V) of group t
//   warp 11     brings the queries, and clears what a sequence's last V block
//               holds past its length (unwritten rows may be NaN, and 0 * NaN
//               is not 0)
// The lengths are read on the device, so a captured launch follows them.
#define ZL_TRY_WAIT_HINT_NS 10000
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "paged.h"

namespace zl {
namespace {

__device__ uint32_t g_paged_err;

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp0 = 9;
constexpr int kAuxWarp = 11;
constexpr int kReaders = 11;                   // 2 issuer threads, 8 softmax warps, the aux warp
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;
constexpr int kMinBlocks = 2;                  // SPLIT: key blocks of a CTA at least, one for each group
constexpr float kLn2 = 0.6931471805599453f;

// K/V blocks of 128 keys in shared memory.  PAIR holds two query tiles and
// needs depth only to cover the latency; SPLIT lives from bytes in flight.
// PAIR's issuers both pass every stage of one ring.  In SPLIT each issuer has
// half of the stages as a ring of its own: a wait on an mbarrier's parity is
// only right for a thread that sees every phase, and an issuer that skipped
// the other's blocks in a shared ring would take a phase two before the one
// it waits for (a block that lands late) for its own.
template <int HD, bool PAIR>
__host__ __device__ constexpr int stages() { return HD == 128 ? (PAIR ? 4 : 6) : (PAIR ? 8 : 12); }

// A work item as the producer hands it out.
struct Item {
  int id;             // PAIR: the item's number, SPLIT: its segment; -1: no item left
  int len;            // keys of the sequence
  int hk, s0, s1;     // SPLIT: key head and key blocks
  int slot;           // SPLIT: partial slot, or -1: the rows are final
};

template <int HD, bool PAIR>
struct Stages {
  static constexpr int kRing = PAIR ? stages<HD, PAIR>() : stages<HD, PAIR>() / 2;
  // Stage and parity of the u-th block half (K or V) of ring t.
  static __device__ __forceinline__ uint32_t stage(int t, uint32_t u) { return (PAIR ? 0u : t * kRing) + u % kRing; }
  static __device__ __forceinline__ uint32_t parity(uint32_t u) { return (u / kRing) & 1u; }
};

template <int HD, bool PAIR>
struct PagedSmem {
  static constexpr int kStages = stages<HD, PAIR>();
  uint8_t q[PAIR ? 2 : 1][kBlockM * HD * 2];   // HD/64 boxes of [128 rows][128 B], 128-byte swizzle
  uint8_t kv[kStages][kBlockN * HD * 2];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kStages], kv_empty[kStages], tail[kStages];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t turn[2], grp_sync[2], all_sync;
  ItemRing ring;
  Item item[2];                                // what the ring's slots hold
  uint32_t tmem_base;
  int abort_flag;
  union {
    float2 ml[2 * kBlockM];                    // SPLIT: m and l of every group's rows
    int64_t chunk_blocks[kMaxSegs / 32];       // SPLIT, at the start: weights of 32 segments each
  };
};

// Block ranges [b0, b1) of 128 keys.
struct Range {
  int b0, b1;
};

// Keys [lo, hi) that the query at position p of a sequence of `len` sees.
__device__ __forceinline__ void keys_of(const PagedAttnHead& a, int len, int p, int* lo, int* hi) {
  *hi = a.causal ? max(0, min(len, p + 1)) : len;
  *lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
}

// Blocks that queries [t0, t1) of the sequence see.
__device__ __forceinline__ Range blocks_of(const PagedAttnHead& a, int len, int q_len, int t0, int t1) {
  int lo, hi, x;
  keys_of(a, len, len - q_len + t0, &lo, &x);
  keys_of(a, len, len - q_len + t1 - 1, &x, &hi);
  if (hi <= lo) return {0, 0};
  return {lo / kBlockN, (hi + kBlockN - 1) / kBlockN};
}

// One work item, as every role sees it.
struct Work {
  int seq, q_row0, q_len, len;
  int hk;
  int tile0;        // first query tile
  int s0, s1;       // the item's key blocks
  bool final;       // its rows are final: they go to o and lse
  int64_t part;     // else: PAIR: the first partial row of the split, SPLIT: of the slot
  Range tile[2];    // each tile's blocks within [s0, s1)
  bool has[2];      // the tile exists
  bool idle;        // PAIR: a split without keys that is not the first
};

template <int N>
__device__ __forceinline__ int find_seg(const PagedAttnArgs<N>& a, int it) {
  int lo = 0, hi = a.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.segs[mid].item0 <= it) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ Range cut(Range r, int s0, int s1) {
  const int b0 = max(r.b0, s0), b1 = min(r.b1, s1);
  return b1 > b0 ? Range{b0, b1} : Range{s0, s0};
}

// The blocks that the splits of a PAIR unit (first tile `tile0`) divide: the
// union of its tiles'.
__device__ __forceinline__ Range pair_blocks(const PagedAttnHead& a, int len, int q_len, int tile0) {
  const int t0 = tile0 * a.tile_tokens;
  Range r = blocks_of(a, len, q_len, t0, min(q_len, t0 + a.tile_tokens));
  if (t0 + a.tile_tokens < q_len) {
    const Range s = blocks_of(a, len, q_len, t0 + a.tile_tokens, min(q_len, t0 + 2 * a.tile_tokens));
    if (r.b1 <= r.b0) return s;
    if (s.b1 > s.b0) r = {min(r.b0, s.b0), max(r.b1, s.b1)};
  }
  return r;
}

// Items of a segment: key head outermost, then the unit, last tokens first
// (under a causal mask they see the most), then the split.
template <int N>
__device__ __forceinline__ Work decode_pair(const PagedAttnArgs<N>& a, const Item& item) {
  const PagedSeg& s = a.segs[find_seg(a, item.id)];
  Work w;
  w.seq = s.seq;
  w.q_row0 = s.q_row0;
  w.q_len = s.q_len;
  w.len = item.len;
  const int tiles = (s.q_len + a.tile_tokens - 1) / a.tile_tokens;
  const int units = (tiles + 1) / 2;
  int x = item.id - s.item0;
  const int split = x % s.splits;
  x /= s.splits;
  const int u = units - 1 - x % units;
  w.hk = x / units;
  w.tile0 = 2 * u;
  const Range r = pair_blocks(a, item.len, s.q_len, w.tile0);
  w.s0 = min(r.b1, r.b0 + split * a.split_blocks);
  w.s1 = min(r.b1, w.s0 + a.split_blocks);
  w.final = r.b1 - r.b0 <= a.split_blocks;
  w.part = s.part0 + static_cast<int64_t>(split) * s.q_len;
  w.idle = w.s1 <= w.s0 && split > 0;
  w.has[0] = true;
  w.has[1] = w.tile0 + 1 < tiles;
  const int t0 = w.tile0 * a.tile_tokens;
  w.tile[0] = cut(blocks_of(a, w.len, s.q_len, t0, min(s.q_len, t0 + a.tile_tokens)), w.s0, w.s1);
  w.tile[1] = w.tile[0];
  if (w.has[1])
    w.tile[1] = cut(blocks_of(a, w.len, s.q_len, t0 + a.tile_tokens, min(s.q_len, t0 + 2 * a.tile_tokens)), w.s0, w.s1);
  return w;
}

template <int N>
__device__ __forceinline__ Work decode_split(const PagedAttnArgs<N>& a, const Item& item) {
  const PagedSeg& s = a.segs[item.id];
  Work w;
  w.seq = s.seq;
  w.q_row0 = s.q_row0;
  w.q_len = s.q_len;
  w.len = item.len;
  w.hk = item.hk;
  w.tile0 = 0;
  w.s0 = item.s0;
  w.s1 = item.s1;
  w.final = item.slot < 0;
  w.part = static_cast<int64_t>(item.slot) * a.slot_rows;
  w.idle = false;
  w.has[0] = true;
  w.has[1] = false;
  w.tile[0] = w.tile[1] = {item.s0, item.s1};
  return w;
}

template <bool PAIR, int N>
__device__ __forceinline__ Work decode(const PagedAttnArgs<N>& a, const Item& item) {
  if constexpr (PAIR) return decode_pair(a, item);
  else return decode_split(a, item);
}

// Copies of a SPLIT tile's rows: 4, 2 or 1, 128 / copies rows apart.
__device__ __forceinline__ int row_copies(int rows) { return rows <= 32 ? 4 : rows <= 64 ? 2 : 1; }

__device__ __forceinline__ void drain_delay(uint64_t ns) {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < ns) {
  }
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int32_t x, int32_t y,
                                             int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
      :: "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A ring reader's next item; false: none left, or a wait ran out.
template <typename SM>
__device__ __forceinline__ bool take(SM* sm, uint32_t n, uint32_t code, bool warp_wide, Item* item) {
  const uint32_t s = n & 1u;
  bool ok = mbar_wait(&sm->ring.full[s], (n >> 1) & 1u, &sm->abort_flag, &g_paged_err, code);
  if (warp_wide) ok = __all_sync(0xffffffffu, ok);
  if (!ok) return false;
  const volatile Item* i = &sm->item[s];
  item->id = i->id;
  item->len = i->len;
  item->hk = i->hk;
  item->s0 = i->s0;
  item->s1 = i->s1;
  item->slot = i->slot;
  if (warp_wide) __syncwarp();
  if (!warp_wide || (threadIdx.x & 31) == 0) mbar_arrive(&sm->ring.empty[s]);
  return item->id >= 0;
}

// ------------------------------------------------------------------ producer
// Hands out the n-th item once every reader has taken the slot's previous one.
template <typename SM>
__device__ __forceinline__ bool publish(SM* sm, uint32_t n, const Item& item) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t s = n & 1u;
    ok = mbar_wait(&sm->ring.empty[s], ((n >> 1) & 1u) ^ 1u, &sm->abort_flag, &g_paged_err, ERR_TIMEOUT_PRODUCER);
    if (ok) {
      sm->item[s] = item;
      mbar_arrive(&sm->ring.full[s]);
    }
  }
  return __shfl_sync(0xffffffffu, ok, 0);
}

// The length of a segment's sequence, within the call's bound.
template <int N>
__device__ __forceinline__ int length_of(const PagedAttnArgs<N>& a, int seg) {
  const int len = __ldg(a.kv_lens + a.segs[seg].seq);
  if (len >= 0 && len <= a.max_kv_len) return len;
  atomicOr(&g_paged_err, ERR_BAD_PAGE);
  return len < 0 ? 0 : a.max_kv_len;
}

// Brings an item's K/V blocks into the rings; `ask` requests the next PAIR
// item when the last block is next.  uses0 / uses1: the rings' counts.
template <int HD, bool PAIR, int N>
__device__ __forceinline__ bool load_blocks(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps,
                                            const Work& w, uint32_t& uses0, uint32_t& uses1, bool ask) {
  using Ring = Stages<HD, PAIR>;
  const int lane = threadIdx.x & 31;
  const int page = 1 << a.page_shift;
  const int box_rows = min(page, kBlockN);
  const int32_t* row = a.page_table + static_cast<int64_t>(w.seq) * a.table_cols;
  // page numbers of the item's blocks, 32 at a time, the next 32 on their way
  const int e0 = (w.s0 * kBlockN) >> a.page_shift;
  const int e1 = min((min(w.len, w.s1 * kBlockN) + page - 1) >> a.page_shift, a.table_cols);
  int chunk = 0;
  int cur = e0 + lane < e1 ? __ldg(row + e0 + lane) : 0;
  int nxt = e0 + 32 + lane < e1 ? __ldg(row + e0 + 32 + lane) : 0;
  for (int j = w.s0; j < w.s1; ++j) {
    if (ask && j == w.s1 - 1 && lane == 0) ring_ask(&sm->ring);
    const int rel = ((j * kBlockN) >> a.page_shift) - e0;
    if ((rel >> 5) != chunk) {
      ++chunk;
      cur = nxt;
      nxt = e0 + 32 * (chunk + 1) + lane < e1 ? __ldg(row + e0 + 32 * (chunk + 1) + lane) : 0;
    }
    const int valid = min(kBlockN, w.len - j * kBlockN);
    const int boxes = (valid + box_rows - 1) / box_rows;
    int pg = __shfl_sync(0xffffffffu, cur, ((rel & 31) + lane) & 31);
    if (lane < boxes && (pg < 0 || pg >= a.num_pages)) {
      atomicOr(&g_paged_err, ERR_BAD_PAGE);            // reads page 0 in its place
      pg = 0;
    }
    const int y = ((pg * a.num_kv_heads + w.hk) << a.page_shift) + ((j * kBlockN) & (page - 1));
    const int ring = PAIR ? 0 : (j - w.s0) & 1;
    uint32_t& uses = ring ? uses1 : uses0;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t st = Ring::stage(ring, uses);
      if (!__all_sync(0xffffffffu, mbar_wait(&sm->kv_empty[st], Ring::parity(uses) ^ 1u, &sm->abort_flag,
                                             &g_paged_err, ERR_TIMEOUT_PRODUCER)))
        return false;
      // a V block that the sequence ends in goes by way of the aux warp
      uint64_t* bar = kv == 1 && valid < kBlockN ? &sm->tail[st] : &sm->kv_full[st];
      if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * box_rows * HD * 2));
      __syncwarp();
      if (lane < boxes) {
        const CUtensorMap* map = kv ? &maps.v : &maps.k;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
          tma_load_2d(sm->kv[st] + c * kBlockN * 128 + lane * box_rows * 128, map, bar, c * 64, y);
      }
      ++uses;
    }
  }
  return true;
}

// PAIR: the CTA's own item first, then stolen ones, in launch order.
template <int HD, int N>
__device__ void produce_pair(PagedSmem<HD, true>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps) {
  const int lane = threadIdx.x & 31;
  uint32_t uses0 = 0, uses1 = 0, steal_ph = 0;
  Item item = {static_cast<int>(blockIdx.x), 0, 0, 0, 0, 0};
  for (uint32_t n = 0;; ++n) {
    if (item.id >= 0) item.len = length_of(a, find_seg(a, item.id));
    if (!publish(sm, n, item) || item.id < 0) return;
    const Work w = decode_pair(a, item);
    if (!load_blocks<HD, true, N>(sm, a, maps, w, uses0, uses1, true)) return;
    int next = -2;
    if (lane == 0) {
      if (w.s1 <= w.s0) ring_ask(&sm->ring);
      next = ring_answer(&sm->ring, steal_ph, a.n_items, &sm->abort_flag, &g_paged_err, ERR_TIMEOUT_PRODUCER);
    }
    next = __shfl_sync(0xffffffffu, next, 0);
    if (next == -2) return;
    item.id = next;
  }
}

// Key blocks that one key head of a SPLIT segment counts for (a sequence
// without keys still has rows to write).
template <int N>
__device__ __forceinline__ int weight_of(const PagedAttnArgs<N>& a, int seg, int len, int* b0) {
  const Range r = blocks_of(a, len, a.segs[seg].q_len, 0, a.segs[seg].q_len);
  *b0 = r.b0;
  return max(1, r.b1 - r.b0);
}

// SPLIT, all warps: the blocks of every 32 segments.
template <int HD, int N>
__device__ __forceinline__ void sum_chunks(PagedSmem<HD, false>* sm, const PagedAttnArgs<N>& a) {
  const int lane = threadIdx.x & 31;
  for (int chunk = threadIdx.x & ~31; chunk < a.n_segs; chunk += kThreads) {
    int b0, w = 0;
    if (chunk + lane < a.n_segs) w = weight_of(a, chunk + lane, length_of(a, chunk + lane), &b0);
    int64_t sum = static_cast<int64_t>(w) * a.num_kv_heads;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) sm->chunk_blocks[chunk / 32] = sum;
  }
}

// SPLIT: the blocks of all (sequence, key head) units stand in one line, which
// is cut into equal pieces, one per CTA: every SM has the same number of
// blocks whatever the lengths, and only units that a cut goes through are
// joined afterwards.  A CTA's piece of the unit that its range starts inside
// goes to slot 2c, of the unit that goes on behind its range to 2c + 1, and
// joins[c] tells the join what begins in slot 2c + 1.
template <int HD, int N>
__device__ void produce_split(PagedSmem<HD, false>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps) {
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  uint32_t uses0 = 0, uses1 = 0, n = 0;
  int64_t total = 0;
  for (int s = 0; s < a.n_segs; s += 32) total += sm->chunk_blocks[s / 32];
  const int64_t per = max(static_cast<int64_t>(kMinBlocks), (total + gridDim.x - 1) / gridDim.x);
  int64_t g = c * per;
  const int64_t end = min(total, g + per);
  PagedJoin join = {0, 0, 0, -1};
  // the segments that hold block g: 32 at a time
  int64_t base = 0;            // blocks before the chunk of segments
  int chunk = 0;
  while (g < end && base + sm->chunk_blocks[chunk / 32] <= g) {
    base += sm->chunk_blocks[chunk / 32];
    chunk += 32;
  }
  int len = 0, w_seg = 0, b0 = 0;
  int64_t incl = 0;
  for (; g < end; chunk += 32) {
    const int s = chunk + lane;
    len = 0;
    w_seg = 0;
    b0 = 0;
    if (s < a.n_segs) {
      len = length_of(a, s);
      w_seg = weight_of(a, s, len, &b0);
    }
    incl = static_cast<int64_t>(w_seg) * a.num_kv_heads;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    incl += base;
    base = __shfl_sync(0xffffffffu, incl, 31);
    // all units of this chunk that the range meets
    while (g < end && g < base) {
      const int k = __ffs(__ballot_sync(0xffffffffu, incl > g)) - 1;      // g's segment in the chunk
      const int weight = __shfl_sync(0xffffffffu, w_seg, k);
      const int64_t seg_end = __shfl_sync(0xffffffffu, incl, k);
      const int64_t off = g - (seg_end - static_cast<int64_t>(weight) * a.num_kv_heads);
      const int hk = static_cast<int>(off / weight);
      const int blk = static_cast<int>(off - static_cast<int64_t>(hk) * weight);
      const int cnt = static_cast<int>(min(static_cast<int64_t>(weight - blk), end - g));
      const int first = __shfl_sync(0xffffffffu, b0, k);
      Item item;
      item.id = chunk + k;
      item.len = __shfl_sync(0xffffffffu, len, k);
      item.hk = hk;
      const Range r = blocks_of(a, item.len, a.segs[item.id].q_len, 0, a.segs[item.id].q_len);
      item.s0 = r.b1 > r.b0 ? first + blk : 0;
      item.s1 = r.b1 > r.b0 ? first + blk + cnt : 0;
      item.slot = blk > 0 ? 2 * c : blk + cnt < weight ? 2 * c + 1 : -1;
      if (blk == 0 && cnt < weight)
        join = {a.segs[item.id].q_row0, a.segs[item.id].q_len, hk, static_cast<int>((g + weight - 1) / per)};
      if (!publish(sm, n++, item)) return;
      const Work w = decode_split(a, item);
      if (!load_blocks<HD, false, N>(sm, a, maps, w, uses0, uses1, false)) return;
      g += cnt;
    }
  }
  if (lane == 0) a.joins[c] = join;
  publish(sm, n, Item{-1, 0, 0, 0, 0, 0});
}

// ------------------------------------------------------------------ MMA issuer t
template <int HD, bool PAIR, int N>
__device__ void issue(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a, uint32_t tmem, int t) {
  using Ring = Stages<HD, PAIR>;
  constexpr uint32_t idesc_qk = idesc_bf16(kBlockM, kBlockN, false, false);
  constexpr uint32_t idesc_pv = idesc_bf16(kBlockM, HD, false, true);
  volatile int* abort_flag = &sm->abort_flag;
  const uint32_t code = ERR_TIMEOUT_MMA;
  const int qt = PAIR ? t : 0;
  const uint64_t q_desc = sdesc_sw128(smem_u32(sm->q[qt]), 16, 1024);
  const uint32_t tS = tmem + 256u * t;
  const uint32_t tO = tS + 128u;
  uint32_t kv_it = 0, q_it = 0, blk_it = 0;
  for (uint32_t n = 0;; ++n) {
    Item item;
    if (!take(sm, n, code, false, &item)) return;
    const Work w = decode<PAIR>(a, item);
    if (w.s1 <= w.s0) continue;
    const bool has = PAIR ? w.has[t] : true;
    if (has && !mbar_wait(&sm->q_full[qt], q_it & 1u, abort_flag, &g_paged_err, code)) return;
    bool first = true;
    // PAIR: both issuers pass every stage, and each uses the blocks that its
    // tile sees; SPLIT: issuer t's blocks alternate with the other's, in its
    // own ring
    const int last_mine = PAIR ? w.tile[t].b1 - 1 : w.s1 - 1 - ((w.s1 - 1 - w.s0 - t) & 1);
    for (int j = PAIR ? w.s0 : w.s0 + t; j < w.s1; j += PAIR ? 1 : 2) {
      const bool mine = has && (!PAIR || (j >= w.tile[t].b0 && j < w.tile[t].b1));
      uint32_t st = Ring::stage(t, kv_it);
      if (!mbar_wait(&sm->kv_full[st], Ring::parity(kv_it), abort_flag, &g_paged_err, code)) return;
      if (mine) {
        tc_fence_after();
        const uint64_t k_desc = sdesc_sw128(smem_u32(sm->kv[st]), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint64_t off16 = ((ks >> 2) * (kBlockM * 128) + (ks & 3) * 32) >> 4;
          umma_ss(tS, q_desc + off16, k_desc + off16, idesc_qk, ks > 0 ? 1u : 0u);
        }
        umma_commit(&sm->s_full[t]);
        if (j == last_mine) umma_commit(&sm->q_empty[qt]);
        umma_commit(&sm->kv_empty[st]);
      } else {
        mbar_arrive(&sm->kv_empty[st]);
      }
      ++kv_it;
      st = Ring::stage(t, kv_it);
      if (!mbar_wait(&sm->kv_full[st], Ring::parity(kv_it), abort_flag, &g_paged_err, code)) return;
      if (mine) {
        if (!mbar_wait(&sm->p_full[t], blk_it & 1u, abort_flag, &g_paged_err, code)) return;
        tc_fence_after();
        const uint64_t v_desc = sdesc_sw128(smem_u32(sm->kv[st]), kBlockN * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < kBlockN / 16; ++ks)
          umma_ts(tO, tS + ks * 8, v_desc + static_cast<uint64_t>(ks * (2048 >> 4)), idesc_pv,
                  (!first || ks > 0) ? 1u : 0u);
        first = false;
        ++blk_it;
        if (PAIR || j < w.s1 - 1) umma_commit(&sm->kv_empty[st]);   // SPLIT's epilogue joins parts in the last V stage
      } else {
        mbar_arrive(&sm->kv_empty[st]);
      }
      ++kv_it;
    }
    if (has) {
      // An issuer without a block in this item does not wait for the softmax
      // group's work on the one before: it must not complete o_full, or could
      // complete it a second time before the group has seen the first.
      if (first) umma_commit(&sm->q_empty[qt]);
      else umma_commit(&sm->o_full[t]);
      ++q_it;
    }
  }
}

// ------------------------------------------------------------------ aux warp
// Brings each item's queries once the previous item has released them (a warp
// of its own, so that the producer runs ahead with keys meanwhile), and clears
// the end of a sequence's last V block.
template <int HD, bool PAIR, int N>
__device__ void assist(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps) {
  using Ring = Stages<HD, PAIR>;
  const int lane = threadIdx.x & 31;
  const uint32_t code = ERR_TIMEOUT_OTHER;
  uint32_t base0 = 0, base1 = 0, phases = 0;     // uses of ring 0 and 1 by earlier items; parity of each tail barrier
  uint32_t q_it0 = 0, q_it1 = 0;
  for (uint32_t n = 0;; ++n) {
    Item item;
    if (!take(sm, n, code, true, &item)) return;
    const Work w = decode<PAIR>(a, item);
    if (w.s1 <= w.s0) continue;
    bool ok = true;
    if (lane == 0) {
#pragma unroll
      for (int t = 0; t < (PAIR ? 2 : 1); ++t) {
        if (!w.has[t]) continue;
        uint32_t& q_it = t ? q_it1 : q_it0;
        if (!mbar_wait(&sm->q_empty[t], (q_it & 1u) ^ 1u, &sm->abort_flag, &g_paged_err, code)) {
          ok = false;
          break;
        }
        ++q_it;
        const int copies = PAIR ? 1 : row_copies(w.q_len * a.group);
        const CUtensorMap* map = &maps.q[PAIR ? 0 : copies >> 1];
        const int rows = (kBlockM / copies) / a.group * a.group;
        mbar_arrive_expect_tx(&sm->q_full[t], static_cast<uint32_t>(copies * rows * HD * 2));
        for (int r = 0; r < copies; ++r)
#pragma unroll
          for (int c = 0; c < HD / 64; ++c)
            tma_load_3d(sm->q[t] + c * kBlockM * 128 + r * (kBlockM / copies) * 128, map, &sm->q_full[t], c * 64,
                        w.hk * a.group, w.q_row0 + (w.tile0 + t) * a.tile_tokens);
      }
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) return;
    const int jt = w.len / kBlockN, valid = w.len % kBlockN;
    if (valid > 0 && jt >= w.s0 && jt < w.s1) {
      const int ring = PAIR ? 0 : (jt - w.s0) & 1;
      const uint32_t blk = static_cast<uint32_t>(PAIR ? jt - w.s0 : (jt - w.s0) >> 1);
      const uint32_t st = Ring::stage(ring, (ring ? base1 : base0) + 2u * blk + 1u);
      if (!__all_sync(0xffffffffu, mbar_wait(&sm->tail[st], (phases >> st) & 1u, &sm->abort_flag, &g_paged_err, code)))
        return;
      phases ^= 1u << st;
      // rows [valid, 128) of every 64-column box: whole 128-byte rows
      for (int x = lane; x < (kBlockN - valid) * 8; x += 32)
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
          *reinterpret_cast<uint4*>(sm->kv[st] + c * kBlockN * 128 + valid * 128 + x * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->kv_full[st]);
    }
    const uint32_t blocks = static_cast<uint32_t>(w.s1 - w.s0);
    base0 += 2u * (PAIR ? blocks : (blocks + 1) / 2);
    base1 += 2u * (PAIR ? 0u : blocks / 2);
  }
}

// ------------------------------------------------------------------ softmax
// One arrival for a warp: what its lanes did before is ordered before it.
// SPLIT's short chain gains by it (the lanes of an arrival on one barrier go
// one after another); PAIR, whose groups take turns, is 2% faster with an
// arrival of every thread (prompt chunks 627 against 640 us).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A barrier among warps that each count as one; `uses` counts the calls.
__device__ __forceinline__ bool warps_sync(uint64_t* bar, uint32_t& uses, volatile int* abort_flag, uint32_t code) {
  warp_arrive(bar);
  const bool ok = mbar_wait(bar, uses & 1u, abort_flag, &g_paged_err, code);
  ++uses;
  return __all_sync(0xffffffffu, ok);
}

// P of 32 scores as 16 packed columns; adds their sum to acc.
__device__ __forceinline__ void exp_pack(const uint32_t (&s)[32], float sl2, float neg_m, uint64_t (&acc)[2],
                                         uint32_t (&p)[16]) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
  const uint64_t negm2 = f2_pack(neg_m, neg_m);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sl2x2, negm2);
    float x0, x1;
    f2_unpack(x, x0, x1);
    const float e0 = fast_exp2(x0);
    const float e1 = fast_exp2(x1);
    acc[i & 1] = f2_add(acc[i & 1], f2_pack(e0, e1));
    p[i] = pack_bf16x2(e0, e1);
  }
}

// Scores of columns [col0, col0 + 32) outside [lo, hi) become -inf.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int col0, int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (col0 + i < lo || col0 + i >= hi) s[i] = __float_as_uint(-INFINITY);
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    m0 = fmax3(m0, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    m1 = fmax3(m1, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
  }
  return fmaxf(m0, m1);
}

// The running maximum after a block whose own is m_blk; *alpha: the factor of
// what was summed before.  A row that has seen nothing keeps -inf.
__device__ __forceinline__ bool raise_max(float m_blk, float* m_run, float* alpha) {
  const float m_new = fmaxf(*m_run, m_blk);
  const bool need = m_new > *m_run + kRescaleThreshold;
  *alpha = 1.f;
  if (need) {
    *alpha = fast_exp2(*m_run - m_new);
    *m_run = m_new;
  }
  return need;
}

template <int HD>
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int c = 0; c < HD / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld();
    reg_fence(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st32(tO + c * 32, o);
  }
}

__device__ __forceinline__ float neg_or_zero(float m) { return m == -INFINITY ? 0.f : -m; }

// PAIR: group t runs tile t.
template <int HD, int N>
__device__ void softmax_pair(PagedSmem<HD, true>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = warp >> 2;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + 256u * t + lane_off;
  const uint32_t tO = tS + 128u;
  const float sl2 = a.scale_log2;
  volatile int* abort_flag = &sm->abort_flag;
  const uint32_t code = ERR_TIMEOUT_SOFTMAX;
  const int row_tok = row / a.group, row_head = row - row_tok * a.group;
  uint32_t blk_it = 0, q_it = 0, turn_it = 0, sync_uses = 0;
  if (t == 1) mbar_arrive(&sm->turn[0]);         // the first turn is group 0's
  for (uint32_t n = 0;; ++n) {
    Item item;
    if (!take(sm, n, code, true, &item)) break;
    const Work w = decode_pair(a, item);
    if (w.idle) continue;
    const bool has = w.has[t];
    const int tok0 = (w.tile0 + t) * a.tile_tokens;
    const int tokens = min(a.tile_tokens, w.q_len - tok0);
    const int tok = tok0 + row_tok;
    const bool row_ok = has && row_tok < tokens;
    float m_run = -INFINITY, l_run = 0.f;
    bool first = true;
    if (w.s1 > w.s0) {
      // this row's keys, and the keys that every row of the tile sees
      int lo, hi, lo_all, hi_all, x;
      const int p0 = w.len - w.q_len;
      keys_of(a, w.len, p0 + tok, &lo, &hi);
      keys_of(a, w.len, p0 + tok0, &x, &hi_all);
      keys_of(a, w.len, p0 + tok0 + max(0, tokens - 1), &lo_all, &x);
      bool ok = true;
      for (int j = w.s0; j < w.s1; ++j, ++turn_it) {
        const bool mine = has && j >= w.tile[t].b0 && j < w.tile[t].b1;
        if (!__all_sync(0xffffffffu,
                        (!mine || mbar_wait(&sm->s_full[t], blk_it & 1u, abort_flag, &g_paged_err, code)) &&
                            mbar_wait(&sm->turn[t], turn_it & 1u, abort_flag, &g_paged_err, code))) {
          ok = false;
          break;
        }
        if (!mine) {
          mbar_arrive(&sm->turn[t ^ 1]);
          continue;
        }
        tc_fence_after();
        uint32_t s[4][32];
        float m_raw;
        const int k0 = j * kBlockN;
        if (k0 >= lo_all && k0 + kBlockN <= hi_all) {
          float r[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) r[c] = tmem_ld32_max(tS + c * 32, s[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            reg_fence(s[c]);
            reg_fence_f(r[c]);
          }
          m_raw = fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
          tmem_wait_ld();
          m_raw = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            reg_fence(s[c]);
            mask32(s[c], k0 + c * 32, lo, hi);
            m_raw = fmaxf(m_raw, max32(s[c]));
          }
        }
        float alpha;
        const bool need = raise_max(m_raw * sl2, &m_run, &alpha);
        l_run *= alpha;
        const float neg_m = neg_or_zero(m_run);
        uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
          exp_pack(s[c], sl2, neg_m, acc, p);
          tmem_st16(tS + 16 * c, p);
        }
        mbar_arrive(&sm->turn[t ^ 1]);
        if (!first && __any_sync(0xffffffffu, need)) rescale_o<HD>(tO, alpha);
        first = false;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm->p_full[t]);
        ++blk_it;
        float ls0, ls1;
        f2_unpack(f2_add(acc[0], acc[1]), ls0, ls1);
        l_run += ls0 + ls1;
      }
      if (!ok) break;
      if (!first) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm->o_full[t], q_it & 1u, abort_flag, &g_paged_err, code))) break;
        ++q_it;
        tc_fence_after();
      }
    }
    if (!has) continue;
    // ---------------------------------------------------------- epilogue
    const bool seen = l_run > 0.f;
    const float inv_l = seen ? 1.f / l_run : 0.f;
    const float lse = seen ? (m_run + log2f(l_run)) * kLn2 : -INFINITY;
    const int h = w.hk * a.group + row_head;
    const bool loaded = w.s1 > w.s0;            // this item's Q went through q[t]
    const bool final_rows = w.final;
    // a full tile of final rows leaves by TMA through the tile's own Q
    // buffer; rows without keys would read O as it was: per thread
    const bool by_tma = final_rows && loaded && !first && tokens == a.tile_tokens;
    if (loaded && !by_tma && row == 0) mbar_arrive(&sm->q_empty[t]);
    if (by_tma) {
      const uint32_t r7 = static_cast<uint32_t>(row & 7);
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld();
        reg_fence(o);
        uint8_t* box_row = sm->q[t] + (c >> 1) * (kBlockM * 128) + row * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4 pk;
          uint32_t* v = &pk.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = seen ? __uint_as_float(o[8 * k + 2 * e]) * inv_l : 0.f;
            const float x1 = seen ? __uint_as_float(o[8 * k + 2 * e + 1]) * inv_l : 0.f;
            v[e] = pack_bf16x2(x0, x1);
          }
          const uint32_t ch = static_cast<uint32_t>((c & 1) * 4 + k);
          *reinterpret_cast<uint4*>(box_row + ((ch ^ r7) << 4)) = pk;
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&sm->grp_sync[t]);
      const uint32_t phase = sync_uses++;
      if (row == 0) {
        if (!mbar_wait(&sm->grp_sync[t], phase & 1u, abort_flag, &g_paged_err, code)) break;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
          tma_store_3d(&maps.o, sm->q[t] + c * (kBlockM * 128), c * 64, w.hk * a.group, w.q_row0 + tok0);
        bulk_commit_group();
        bulk_wait_group_read0();
        mbar_arrive(&sm->q_empty[t]);
      }
      if (row_ok) a.lse[static_cast<int64_t>(h) * a.lse_stride + w.q_row0 + tok] = lse;
    } else {
      const int64_t out = final_rows
          ? (static_cast<int64_t>(w.q_row0 + tok) * a.num_heads + h)
          : ((w.part + tok) * a.num_heads + h);
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        if (loaded && !first) {
          tmem_ld32(tO + c * 32, o);
          tmem_wait_ld();
          reg_fence(o);
        }
        __syncwarp();
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = seen ? __float_as_uint(__uint_as_float(o[i]) * inv_l) : 0u;
          if (final_rows) {
            uint4* d4 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + out * HD + c * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint4 pk;
              uint32_t* u = &pk.x;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = pack_bf16x2(__uint_as_float(o[8 * v + 2 * e]), __uint_as_float(o[8 * v + 2 * e + 1]));
              d4[v] = pk;
            }
          } else {
            uint4* d4 = reinterpret_cast<uint4*>(a.o_part + out * HD + c * 32);
#pragma unroll
            for (int v = 0; v < 8; ++v) d4[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
        }
        __syncwarp();
      }
      if (row_ok) {
        if (final_rows)
          a.lse[static_cast<int64_t>(h) * a.lse_stride + w.q_row0 + tok] = lse;
        else
          a.lse_part[out] = lse;
      }
    }
  }
  if (row == 0) bulk_wait_group0();              // the group's stores, before the CTA leaves
}

// SPLIT: group t takes every other block; with copies of the rows, a warp
// takes its own part of a block's columns.
template <int HD, int N>
__device__ void softmax_split(PagedSmem<HD, false>* sm, const PagedAttnArgs<N>& a, uint32_t tmem) {
  using Ring = Stages<HD, false>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = warp >> 2, quad = warp & 3;
  const int row = quad * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + 256u * t + lane_off;
  const uint32_t tO = tS + 128u;
  const float sl2 = a.scale_log2;
  volatile int* abort_flag = &sm->abort_flag;
  const uint32_t code = ERR_TIMEOUT_SOFTMAX;
  uint32_t blk_it = 0, q_it = 0, sync_uses = 0, base0 = 0, base1 = 0;
  for (uint32_t n = 0;; ++n) {
    Item item;
    if (!take(sm, n, code, true, &item)) return;
    const Work w = decode_split(a, item);
    const int rows = w.q_len * a.group;
    const int copies = row_copies(rows);
    const int span = kBlockM / copies;           // rows of a copy
    const int r = row & (span - 1);              // the row it stands for
    const int nch = 4 / copies;                  // 32-column pieces of a block that are this warp's,
    const int ch0 = (quad / nch) * nch;          // from this one on
    const bool warp_rows = (r & ~31) < rows;     // the warp has a row at all
    const int tok = r / a.group;
    int lo, hi, lo_all, hi_all, x;
    const int p0 = w.len - w.q_len;
    keys_of(a, w.len, p0 + tok, &lo, &hi);
    keys_of(a, w.len, p0, &x, &hi_all);
    keys_of(a, w.len, p0 + w.q_len - 1, &lo_all, &x);
    float m_run = -INFINITY, l_run = 0.f;
    bool first = true;
    for (int j = w.s0 + t; j < w.s1; j += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm->s_full[t], blk_it & 1u, abort_flag, &g_paged_err, code))) return;
      ++blk_it;
      if (warp_rows) {
        tc_fence_after();
        const int k0 = j * kBlockN;
        const bool whole = k0 >= lo_all && k0 + kBlockN <= hi_all;
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < nch) tmem_ld32(tS + (ch0 + c) * 32, s[c]);
        tmem_wait_ld();
        float m_raw = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < nch) {
            reg_fence(s[c]);
            if (!whole) mask32(s[c], k0 + (ch0 + c) * 32, lo, hi);
            m_raw = fmaxf(m_raw, max32(s[c]));
          }
        float alpha;
        const bool need = raise_max(m_raw * sl2, &m_run, &alpha);
        l_run *= alpha;
        const float neg_m = neg_or_zero(m_run);
        uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < nch) {
            uint32_t p[16];
            exp_pack(s[c], sl2, neg_m, acc, p);
            tmem_st16(tS + (ch0 + c) * 16, p);
          }
        if (nch < 4) {                           // the other warps' columns do not count for this copy
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < ch0 || c >= ch0 + nch) tmem_st16(tS + c * 16, z);
        }
        if (!first && __any_sync(0xffffffffu, need)) rescale_o<HD>(tO, alpha);
        first = false;
        tmem_wait_st();
        tc_fence_before();
        float ls0, ls1;
        f2_unpack(f2_add(acc[0], acc[1]), ls0, ls1);
        l_run += ls0 + ls1;
      }
      warp_arrive(&sm->p_full[t]);
    }
    const bool loaded = w.s1 > w.s0;
    if (!loaded) {                               // nothing is seen
      const int F8 = HD / 8;
      for (int y = threadIdx.x; y < rows * F8; y += 2 * kBlockM) {
        const int rr = y / F8, tk = rr / a.group, h = w.hk * a.group + rr - tk * a.group;
        const int64_t orow = static_cast<int64_t>(w.q_row0 + tk) * a.num_heads + h;
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + orow * HD)[y % F8] = make_uint4(0, 0, 0, 0);
        if (y % F8 == 0) a.lse[static_cast<int64_t>(h) * a.lse_stride + w.q_row0 + tk] = -INFINITY;
      }
      continue;
    }
    if (w.s1 - w.s0 > t) {                       // the group had a block
      if (!__all_sync(0xffffffffu, mbar_wait(&sm->o_full[t], q_it & 1u, abort_flag, &g_paged_err, code))) return;
      ++q_it;
      tc_fence_after();
    }
    // ---------------------------------------------------------- join the parts of each row
    // part i: group i / copies, copy i % copies
    sm->ml[t * kBlockM + row] = make_float2(m_run, l_run);
    if (!warps_sync(&sm->all_sync, sync_uses, abort_flag, code)) return;
    const int parts = 2 * copies;
    float m_all = -INFINITY;
    for (int i = 0; i < parts; ++i) m_all = fmaxf(m_all, sm->ml[i * span + r].x);
    float l_all = 0.f;
    for (int i = 0; i < parts; ++i) {
      const float2 v = sm->ml[i * span + r];
      if (v.x != -INFINITY) l_all += v.y * fast_exp2(v.x - m_all);
    }
    const float scale = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_all) / l_all;
    if (t == 0 && quad * 32 < span && r < rows) {   // the first copy's threads know the row's LSE
      const int h = w.hk * a.group + r - tok * a.group;
      const float lse = l_all > 0.f ? (m_all + log2f(l_all)) * kLn2 : -INFINITY;
      if (w.final)
        a.lse[static_cast<int64_t>(h) * a.lse_stride + w.q_row0 + tok] = lse;
      else
        a.lse_part[w.part + r] = lse;
    }
    // Through the item's last V stage, which its issuer leaves to this
    // epilogue: [part][row][width] floats, 16-byte pieces swizzled by the
    // row, in as few passes over the columns as the stage allows (one for
    // eight rows or fewer).
    const int blocks = w.s1 - w.s0;
    const int ring = (blocks - 1) & 1;
    const uint32_t st = Ring::stage(ring, (ring ? base1 : base0) + 2u * static_cast<uint32_t>((blocks - 1) >> 1) + 1u);
    base0 += 2u * static_cast<uint32_t>((blocks + 1) / 2);
    base1 += 2u * static_cast<uint32_t>(blocks / 2);
    float4* stage = reinterpret_cast<float4*>(sm->kv[st]);
    const int passes = copies * rows <= 32 ? 1 : copies * rows <= 64 ? 2 : 4;
    const int width = HD / passes;               // columns of a pass
    const int f4 = width / 4;                    // 16-byte pieces of a row, 4 at least
    const int swz_mask = min(7, f4 - 1);
    const int part = t * copies + row / span;
#pragma unroll 1
    for (int c = 0; c < passes; ++c) {
      if (warp_rows) {
        float4* dst = stage + (part * rows + r) * f4;
#pragma unroll 1
        for (int x = 0; x < width / 16; ++x) {
          uint32_t o[16];
          __syncwarp();
          tmem_ld16(tO + c * width + x * 16, o);
          tmem_wait_ld();
          reg_fence(o);
          if (r < rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
              if (scale != 0.f)                  // else O may never have been written
                v = make_float4(__uint_as_float(o[4 * i]) * scale, __uint_as_float(o[4 * i + 1]) * scale,
                                __uint_as_float(o[4 * i + 2]) * scale, __uint_as_float(o[4 * i + 3]) * scale);
              dst[(4 * x + i) ^ (r & swz_mask)] = v;
            }
          }
        }
      }
      if (!warps_sync(&sm->all_sync, sync_uses, abort_flag, code)) return;
      for (int y = threadIdx.x; y < rows * f4; y += 2 * kBlockM) {
        const int rr = y / f4, f = y - rr * f4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) {
          const float4 u = stage[(i * rows + rr) * f4 + (f ^ (rr & swz_mask))];
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        const int col = c * width + 4 * f;
        if (w.final) {
          const int tk = rr / a.group, h = w.hk * a.group + rr - tk * a.group;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) +
                                    (static_cast<int64_t>(w.q_row0 + tk) * a.num_heads + h) * HD + col) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        } else {
          *reinterpret_cast<float4*>(a.o_part + (w.part + rr) * HD + col) = v;
        }
      }
      fence_proxy_async_smem();                  // TMA may write the stage after this
      if (!warps_sync(&sm->all_sync, sync_uses, abort_flag, code)) return;
    }
    if (threadIdx.x == 0) mbar_arrive(&sm->kv_empty[st]);
  }
}

template <int HD, bool PAIR, int N>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedAttnArgs<N> args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  auto* sm = reinterpret_cast<PagedSmem<HD, PAIR>*>(smem_raw);
  if (!PAIR && threadIdx.x == 0) args.joins[blockIdx.x].last = -1;   // also when this CTA gives up a wait
  if ((smem_u32(smem_raw) & 1023u) != 0) {       // the declared alignment; the swizzle needs it
    if (threadIdx.x == 0) atomicOr(&g_paged_err, ERR_BAD_WORK);
    return;
  }
  constexpr int kStages = stages<HD, PAIR>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm->q_full[t], 1);
      mbar_init(&sm->q_empty[t], 2);             // PAIR: the last S and the epilogue; SPLIT: both issuers' last S
      mbar_init(&sm->s_full[t], 1);
      mbar_init(&sm->p_full[t], PAIR ? 128 : 4); // the group's threads, or its warps
      mbar_init(&sm->o_full[t], 1);
      mbar_init(&sm->turn[t], 128);
      mbar_init(&sm->grp_sync[t], 4);
    }
    mbar_init(&sm->all_sync, 8);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm->kv_full[s], 1);
      mbar_init(&sm->kv_empty[s], PAIR ? 2 : 1); // PAIR: both issuers pass every stage
      mbar_init(&sm->tail[s], 1);
    }
    ring_init(&sm->ring, kReaders);
    sm->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp0) {
    tmem_alloc(&sm->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if constexpr (!PAIR) sum_chunks<HD, N>(sm, args);
  // the join may be set up from here on; it waits for this grid's end itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;

  if (warp == kProducerWarp) {
    if constexpr (PAIR) produce_pair<HD, N>(sm, args, maps);
    else produce_split<HD, N>(sm, args, maps);
  } else if (warp == kMmaWarp0 || warp == kMmaWarp0 + 1) {
    if (lane == 0) issue<HD, PAIR, N>(sm, args, tmem, warp - kMmaWarp0);
  } else if (warp == kAuxWarp) {
    assist<HD, PAIR, N>(sm, args, maps);
  } else if constexpr (PAIR) {
    softmax_pair<HD, N>(sm, args, maps, tmem);
  } else {
    softmax_split<HD, N>(sm, args, tmem);
  }

  __syncwarp();
  if (*reinterpret_cast<volatile int*>(&sm->abort_flag)) drain_delay(2000000ull);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp0) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ joining the splits
//     lse = log sum_i exp(lse_i),  o = sum_i exp(lse_i - lse) o_i
// over the n parts of one row, part i at row part(i) of o_part and lse_part.
// The warps of the block take the parts in turn, so that few rows with many
// parts still have their loads in flight together.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 16;                  // SPLIT: blocks that share a unit's rows

template <int HD, typename F>
__device__ __forceinline__ void join_row(const PagedAttnHead& a, int n, F part, int64_t o_row, float* lse_out) {
  constexpr int C = HD / 32;
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float sum_o[kWarps][HD];
  __shared__ float lse_s[kMaxParts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();                             // the row before has read its sums
  for (int i = threadIdx.x; i < n; i += kJoinThreads) lse_s[i] = a.lse_part[part(i)];
  __syncthreads();
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, lse_s[i]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const bool seen = m != -INFINITY;
  float sum = 0.f;
  for (int i = lane; i < n; i += 32) sum += seen ? expf(lse_s[i] - m) : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = seen ? 1.f / sum : 0.f;
  float acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int i = warp; i < n; i += kWarps) {
    const float wgt = seen ? expf(lse_s[i] - m) * inv : 0.f;
    const float* src = a.o_part + part(i) * HD + lane * C;
    if constexpr (C == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      acc[0] = fmaf(wgt, v.x, acc[0]); acc[1] = fmaf(wgt, v.y, acc[1]);
      acc[2] = fmaf(wgt, v.z, acc[2]); acc[3] = fmaf(wgt, v.w, acc[3]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      acc[0] = fmaf(wgt, v.x, acc[0]); acc[1] = fmaf(wgt, v.y, acc[1]);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) sum_o[warp][lane * C + c] = acc[c];
  __syncthreads();
  for (int c = threadIdx.x; c < HD; c += kJoinThreads) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) v += sum_o[q][c];
    static_cast<__nv_bfloat16*>(a.o)[o_row * HD + c] = __float2bfloat16_rn(v);
  }
  if (threadIdx.x == 0) *lse_out = seen ? m + logf(sum) : -INFINITY;
}

// PAIR: one block per (query, head) row; rows of one split were written in place.
template <int HD, int N>
__global__ void __launch_bounds__(kJoinThreads) join_pair_kernel(const __grid_constant__ PagedAttnArgs<N> a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t tok_all = blockIdx.x / a.num_heads;
  const int h = static_cast<int>(blockIdx.x - tok_all * a.num_heads);
  int lo = 0, hi = a.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.segs[mid].tok0 <= tok_all) lo = mid; else hi = mid - 1;
  }
  const PagedSeg& s = a.segs[lo];
  if (s.splits <= 1) return;
  const int tok = static_cast<int>(tok_all) - s.tok0;
  const int len = max(0, min(__ldg(a.kv_lens + s.seq), a.max_kv_len));
  const Range r = pair_blocks(a, len, s.q_len, tok / a.tile_tokens & ~1);
  const int n = (r.b1 - r.b0 + a.split_blocks - 1) / a.split_blocks;
  if (n <= 1) return;
  const int64_t row0 = (s.part0 + tok) * a.num_heads + h;
  const int64_t step = static_cast<int64_t>(s.q_len) * a.num_heads;
  join_row<HD>(a, n, [&](int i) { return row0 + i * step; },
               static_cast<int64_t>(s.q_row0 + tok) * a.num_heads + h,
               a.lse + static_cast<int64_t>(h) * a.lse_stride + s.q_row0 + tok);
}

// SPLIT: block x looks after the unit that begins in CTA x and goes on in the
// CTAs behind it; kJoinRows blocks share its rows.
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) join_split_kernel(const __grid_constant__ PagedAttnHead a) {
  const int c = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedJoin j = a.joins[c];
  if (j.last < 0) return;
  for (int r = blockIdx.y; r < j.q_len * a.group; r += kJoinRows) {
    const int tok = r / a.group, h = j.hk * a.group + r - tok * a.group;
    join_row<HD>(a, j.last - c + 1,
                 [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.slot_rows + r; },
                 static_cast<int64_t>(j.q_row0 + tok) * a.num_heads + h,
                 a.lse + static_cast<int64_t>(h) * a.lse_stride + j.q_row0 + tok);
  }
}

// The first n_segs of N.
template <int N>
PagedAttnArgs<N> cut(const PagedAttnArgs<kMaxSegs>& a) {
  PagedAttnArgs<N> r;
  static_cast<PagedAttnHead&>(r) = a;
  for (int i = 0; i < a.n_segs; ++i) r.segs[i] = a.segs[i];
  return r;
}

template <int HD, bool PAIR, int N>
cudaError_t launch_attn(const PagedMaps& maps, const PagedAttnArgs<N>& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(PagedSmem<HD, PAIR>);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  // once per device
  static std::atomic<uint64_t> done[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<uint64_t>& word = done[(dev >> 6) & 1];
  if (!(word.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<HD, PAIR, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    word.fetch_or(uint64_t(1) << (dev & 63));
  }
  paged_attn_kernel<HD, PAIR, N><<<a.n_items, kThreads, smem, stream>>>(maps, a);
  return cudaGetLastError();
}

template <int HD, bool PAIR>
cudaError_t attn_kind(const PagedMaps& maps, const PagedAttnArgs<kMaxSegs>& a, cudaStream_t stream) {
  return a.n_segs <= kFewSegs ? launch_attn<HD, PAIR, kFewSegs>(maps, cut<kFewSegs>(a), stream)
                              : launch_attn<HD, PAIR, kMaxSegs>(maps, a, stream);
}

// The join's launch overlaps the attention's last CTAs (programmatic dependent
// launch); its blocks wait for their results.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int HD>
cudaError_t join_kind(bool pair, const PagedAttnArgs<kMaxSegs>& a, cudaStream_t stream) {
  const dim3 blocks(static_cast<unsigned>(static_cast<int64_t>(a.tokens) * a.num_heads));
  if (!pair)
    return launch_after(join_split_kernel<HD>, dim3(a.n_items, std::min(a.slot_rows, kJoinRows)), stream,
                        static_cast<const PagedAttnHead&>(a));
  return a.n_segs <= kFewSegs ? launch_after(join_pair_kernel<HD, kFewSegs>, blocks, stream, cut<kFewSegs>(a))
                              : launch_after(join_pair_kernel<HD, kMaxSegs>, blocks, stream, a);
}

}  // namespace

cudaError_t launch_paged_attn(int head_dim, bool pair, const PagedMaps& maps, const PagedAttnArgs<kMaxSegs>& a,
                              cudaStream_t stream) {
  if (head_dim == 64) return pair ? attn_kind<64, true>(maps, a, stream) : attn_kind<64, false>(maps, a, stream);
  return pair ? attn_kind<128, true>(maps, a, stream) : attn_kind<128, false>(maps, a, stream);
}

cudaError_t launch_paged_join(int head_dim, bool pair, const PagedAttnArgs<kMaxSegs>& a, cudaStream_t stream) {
  return head_dim == 64 ? join_kind<64>(pair, a, stream) : join_kind<128>(pair, a, stream);
}

uint32_t paged_attn_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_paged_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
