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
//               TMA box of its page.  The items are the CTA's equal share of
//               all key blocks of the call, or, of few short units, one whole
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
// Key blocks of a CTA at least (SPLIT: one for each group).  With three, a token
// over 1,000 keys (24 / 8 heads, pages of 64; a call repeated on the same inputs)
// takes 12.8 us instead of 11.7, a chunk of 200 over 1,536 21.7 instead of 20.6.
constexpr int kMinBlocks = 2;
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
  int seg;            // segment; -1: no item left
  int len;            // keys of its sequence
  int hk;             // key head
  int tile0;          // first query tile
  int s0, s1;         // key blocks
  int slot;           // slot of partial rows, or -1: the rows are final
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
  // At the start the blocks of every segment (PAIR) or of every 32 (SPLIT);
  // then SPLIT's m and l of every group's rows.
  int64_t scratch[PAIR ? kMaxSegs : 2 * kBlockM];
};

// Block ranges [b0, b1) of 128 keys.
struct Range {
  int b0, b1;
};

// Keys [lo, hi) that the query at position p of a sequence of `len` sees.
__device__ __forceinline__ void keys_of(const PagedAttnHead& a, int len, int p, int* lo, int* hi) {
  *hi = a.causal ? max(0, min(len, p + 1)) : len;
  *lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;   // p may be far below zero
}

// Blocks that queries [t0, t1) of the sequence see.
__device__ __forceinline__ Range blocks_of(const PagedAttnHead& a, int len, int q_len, int t0, int t1) {
  int lo, hi, x;
  keys_of(a, len, len - q_len + t0, &lo, &x);
  keys_of(a, len, len - q_len + t1 - 1, &x, &hi);
  if (hi <= lo) return {0, 0};
  return {lo / kBlockN, (hi + kBlockN - 1) / kBlockN};
}

__device__ __forceinline__ Range cut(Range r, int s0, int s1) {
  const int b0 = max(r.b0, s0), b1 = min(r.b1, s1);
  return b1 > b0 ? Range{b0, b1} : Range{s0, s0};
}

// The blocks that a unit (PAIR: two tiles from `tile0` on, SPLIT: the one
// tile) sees: the union of its tiles'.
template <bool PAIR>
__device__ __forceinline__ Range unit_blocks(const PagedAttnHead& a, int len, int q_len, int tile0) {
  const int t0 = tile0 * a.tile_tokens;
  Range r = blocks_of(a, len, q_len, t0, min(q_len, t0 + a.tile_tokens));
  if (PAIR && t0 + a.tile_tokens < q_len) {
    const Range s = blocks_of(a, len, q_len, t0 + a.tile_tokens, min(q_len, t0 + 2 * a.tile_tokens));
    if (r.b1 <= r.b0) return s;
    if (s.b1 > s.b0) r = {min(r.b0, s.b0), max(r.b1, s.b1)};
  }
  return r;
}

// One work item, as every role sees it.
struct Work {
  int seq, q_row0, q_len, len;
  int hk;
  int tile0;        // first query tile
  int s0, s1;       // the item's key blocks
  bool final;       // its rows are final: they go to o and lse
  int64_t part;     // else: their first row in o_part and lse_part
  bool has1;        // PAIR: the second tile exists
  Range r0, r1;     // each tile's blocks within [s0, s1)

  // by selection: an array indexed by the group would live in local memory
  __device__ __forceinline__ bool has(int t) const { return t == 0 || has1; }
  __device__ __forceinline__ int b0(int t) const { return t == 0 ? r0.b0 : r1.b0; }
  __device__ __forceinline__ int b1(int t) const { return t == 0 ? r0.b1 : r1.b1; }
  // Tile t has a block in the item.  One that has none takes no part in its
  // queries' coming and going: its softmax group would release them without
  // having waited for its issuer, twice before a slow one came by.
  __device__ __forceinline__ bool uses_q(int t) const { return has(t) && b1(t) > b0(t); }
};

template <bool PAIR, int N>
__device__ __forceinline__ Work decode(const PagedAttnArgs<N>& a, const Item& item) {
  const PagedSeg& s = a.segs[item.seg];
  Work w;
  w.seq = s.seq;
  w.q_row0 = s.q_row0;
  w.q_len = s.q_len;
  w.len = item.len;
  w.hk = item.hk;
  w.tile0 = item.tile0;
  w.s0 = item.s0;
  w.s1 = item.s1;
  w.final = item.slot < 0;
  w.part = static_cast<int64_t>(item.slot) * a.slot_rows;
  w.has1 = false;
  w.r0 = w.r1 = {item.s0, item.s1};
  if constexpr (PAIR) {
    const int t0 = w.tile0 * a.tile_tokens, t1 = t0 + a.tile_tokens;
    w.has1 = t1 < s.q_len;
    w.r0 = cut(blocks_of(a, w.len, s.q_len, t0, min(s.q_len, t1)), w.s0, w.s1);
    if (w.has1)
      w.r1 = cut(blocks_of(a, w.len, s.q_len, t1, min(s.q_len, t1 + a.tile_tokens)), w.s0, w.s1);
  }
  return w;
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
  item->seg = i->seg;
  item->len = i->len;
  item->hk = i->hk;
  item->tile0 = i->tile0;
  item->s0 = i->s0;
  item->s1 = i->s1;
  item->slot = i->slot;
  if (warp_wide) __syncwarp();
  if (!warp_wide || (threadIdx.x & 31) == 0) mbar_arrive(&sm->ring.empty[s]);
  return item->seg >= 0;
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

// Brings an item's K/V blocks into the rings.  uses0 / uses1: the rings' counts.
template <int HD, bool PAIR, int N>
__device__ __forceinline__ bool load_blocks(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps,
                                            const Work& w, uint32_t& uses0, uint32_t& uses1) {
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

// Key blocks that a unit counts for (one without keys still has rows to write),
// and what beginning and ending an item costs, in blocks: the cut is equal in
// time, not in blocks, when some CTAs get many short sequences.
__device__ __forceinline__ int weight_of(Range r) { return max(1, r.b1 - r.b0); }
template <int HD, bool PAIR>
__host__ __device__ constexpr int item_cost() { return PAIR ? 2 : HD == 128 ? 2 : 4; }

__device__ __forceinline__ int64_t div_nonneg(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

template <bool PAIR>
__device__ __forceinline__ int units_of(const PagedAttnHead& a, int q_len) {
  return PAIR ? (q_len + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens) : 1;
}

// All warps, at the start: the cost of one key head of every segment (PAIR),
// or the sum of 32 segments' (SPLIT, which has no room for more).
template <int HD, bool PAIR, int N>
__device__ __forceinline__ void sum_blocks(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (PAIR) {
    for (int s = warp; s < a.n_segs; s += kThreads / 32) {
      const int len = length_of(a, s), q_len = a.segs[s].q_len;
      int64_t sum = 0;
      for (int u = lane; u < units_of<true>(a, q_len); u += 32)
        sum += item_cost<HD, PAIR>() + weight_of(unit_blocks<true>(a, len, q_len, 2 * u));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) sm->scratch[s] = sum;
    }
  } else {
    for (int chunk = warp * 32; chunk < a.n_segs; chunk += kThreads) {
      int64_t sum = 0;
      if (chunk + lane < a.n_segs)
        sum = item_cost<HD, PAIR>() +
              weight_of(unit_blocks<false>(a, length_of(a, chunk + lane), a.segs[chunk + lane].q_len, 0));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) sm->scratch[chunk / 32] = sum;
    }
  }
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (static_cast<int>(threadIdx.x & 31) >= d) x += y;
  }
  return x;
}

// WHOLE, a launch of few units with few blocks each: CTA c takes the c-th whole,
// and neither the sums before nor the join behind it is needed.  (Both ways in
// one kernel cost the other launches 0.5 to 1.7 us of instruction fetches.)
template <int HD, bool PAIR, int N>
__device__ void produce_whole(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps) {
  const int nk = a.num_kv_heads;
  int seg = 0, x = blockIdx.x;
  if constexpr (PAIR) {
    for (; x >= units_of<true>(a, a.segs[seg].q_len) * nk; ++seg) x -= units_of<true>(a, a.segs[seg].q_len) * nk;
  } else {
    seg = x / nk;
    x -= seg * nk;
  }
  const int unit = x / nk, len = length_of(a, seg);
  const Range r = unit_blocks<PAIR>(a, len, a.segs[seg].q_len, PAIR ? 2 * unit : 0);
  const Item item = {seg, len, x - unit * nk, PAIR ? 2 * unit : 0, r.b0, max(r.b0, r.b1), -1};
  if (!publish(sm, 0, item)) return;
  uint32_t uses0 = 0, uses1 = 0;
  if (!load_blocks<HD, PAIR, N>(sm, a, maps, decode<PAIR>(a, item), uses0, uses1)) return;
  publish(sm, 1, Item{-1, 0, 0, 0, 0, 0, -1});
}

// Otherwise the blocks of all units (sequence, key head, query tiles) stand in
// one line, each unit's behind a gap of its item cost, and the line is cut into
// equal pieces, one per CTA: every SM has the same work whatever the lengths, and only
// units that a cut goes through are joined afterwards.  A CTA's piece of the
// unit that its range starts inside goes to slot 2c, of the unit that goes on
// behind its range to 2c + 1, and joins[c] tells the join what begins in slot
// 2c + 1.
template <int HD, bool PAIR, int N>
__device__ void produce(PagedSmem<HD, PAIR>* sm, const PagedAttnArgs<N>& a, const PagedMaps& maps) {
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const int nk = a.num_kv_heads;
  uint32_t uses0 = 0, uses1 = 0, n = 0;
  int64_t total = 0;
  for (int i = lane; i < (PAIR ? a.n_segs : (a.n_segs + 31) / 32); i += 32) total += sm->scratch[i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  total *= nk;
  const int64_t per = max(static_cast<int64_t>(kMinBlocks), div_nonneg(total + gridDim.x - 1, gridDim.x));
  constexpr int kCost = item_cost<HD, PAIR>();
  int64_t g = c * per;
  const int64_t end = min(total, g + per);
  PagedJoin join = {0, 0, 0, 0, -1};
  if (g < end) {
    // where block g lies: its segment, 32 at a time ...
    int64_t base = 0;          // blocks before the chunk of segments
    int chunk = 0, seg = 0;
    int64_t seg_blocks = 0, off = 0;
    for (;; chunk += 32) {
      if constexpr (!PAIR) {
        if (base + sm->scratch[chunk / 32] * nk <= g) {
          base += sm->scratch[chunk / 32] * nk;
          continue;
        }
      }
      int64_t w = 0;
      if (chunk + lane < a.n_segs) {
        if constexpr (PAIR) w = sm->scratch[chunk + lane];
        else w = kCost + weight_of(unit_blocks<false>(a, length_of(a, chunk + lane), a.segs[chunk + lane].q_len, 0));
      }
      const int64_t incl = base + warp_scan(w * nk);
      const uint32_t past = __ballot_sync(0xffffffffu, incl > g);
      if (past != 0) {
        const int k = __ffs(past) - 1;
        seg = chunk + k;
        seg_blocks = __shfl_sync(0xffffffffu, w, k);
        off = g - (__shfl_sync(0xffffffffu, incl, k) - seg_blocks * nk);
        break;
      }
      base = __shfl_sync(0xffffffffu, incl, 31);
    }
    // ... the key head in it, and the unit, 32 at a time
    int len = length_of(a, seg), q_len = a.segs[seg].q_len;
    int hk = static_cast<int>(div_nonneg(off, seg_blocks)), unit = 0;
    off -= hk * seg_blocks;
    if constexpr (PAIR) {
      int64_t before = 0;
      for (int u0 = 0;; u0 += 32) {
        const int u = u0 + lane;
        const int64_t w = u < units_of<true>(a, q_len) ? kCost + weight_of(unit_blocks<true>(a, len, q_len, 2 * u)) : 0;
        const int64_t incl = before + warp_scan(w);
        const uint32_t past = __ballot_sync(0xffffffffu, incl > off);
        if (past != 0) {
          const int k = __ffs(past) - 1;
          unit = u0 + k;
          off -= __shfl_sync(0xffffffffu, incl, k) - __shfl_sync(0xffffffffu, w, k);
          break;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    while (true) {
      const int tile0 = PAIR ? 2 * unit : 0;
      const Range r = unit_blocks<PAIR>(a, len, q_len, tile0);
      const int weight = weight_of(r);
      const int64_t avail = min(kCost + weight - off, end - g);
      const int first = static_cast<int>(max(off - kCost, int64_t(0)));          // the piece's blocks of the unit
      const int last = static_cast<int>(max(off + avail - kCost, int64_t(0)));
      if (last > first) {
        Item item = {seg, len, hk, tile0, 0, 0, -1};
        if (r.b1 > r.b0) {
          item.s0 = r.b0 + first;
          item.s1 = r.b0 + last;
        }
        if (last - first < weight) {
          item.slot = first > 0 ? 2 * c : 2 * c + 1;
          if (first == 0)
            join = {a.segs[seg].q_row0, q_len, hk, tile0, static_cast<int>(div_nonneg(g - off + kCost + weight - 1, per))};
        }
        if (!publish(sm, n++, item)) return;
        const Work w = decode<PAIR>(a, item);
        if (!load_blocks<HD, PAIR, N>(sm, a, maps, w, uses0, uses1)) return;
      }
      g += avail;
      if (g >= end) break;
      off = 0;
      if (++unit < units_of<PAIR>(a, q_len)) continue;
      unit = 0;
      if (++hk < nk) continue;
      hk = 0;
      ++seg;
      len = length_of(a, seg);
      q_len = a.segs[seg].q_len;
    }
  }
  if (lane == 0) a.joins[c] = join;
  publish(sm, n, Item{-1, 0, 0, 0, 0, 0, -1});
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
    const bool uses = PAIR ? w.uses_q(t) : true;
    if (uses && !mbar_wait(&sm->q_full[qt], q_it & 1u, abort_flag, &g_paged_err, code)) return;
    bool first = true;
    // PAIR: both issuers pass every stage, and each uses the blocks that its
    // tile sees; SPLIT: issuer t's blocks alternate with the other's, in its
    // own ring
    const int mine0 = w.b0(t), mine1 = uses ? w.b1(t) : 0;
    const int last_mine = PAIR ? mine1 - 1 : w.s1 - 1 - ((w.s1 - 1 - w.s0 - t) & 1);
    for (int j = PAIR ? w.s0 : w.s0 + t; j < w.s1; j += PAIR ? 1 : 2) {
      const bool mine = !PAIR || (j >= mine0 && j < mine1);
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
    if (uses) {
      // SPLIT's issuer without a block in this item does not wait for the
      // softmax group's work on the one before: it must not complete o_full, or
      // could complete it a second time before the group has seen the first.
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
        if (!w.uses_q(t)) continue;
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

// Scores of columns [col0, col0 + 32) outside [lo, hi) become -inf: one bit a
// column, so that an element costs a test and a select.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int col0, int lo, int hi) {
  const int first = min(max(lo - col0, 0), 32), last = min(max(hi - col0, 0), 32);
  const uint32_t below = first >= 32 ? 0xffffffffu : (1u << first) - 1u;
  const uint32_t seen = (last >= 32 ? 0xffffffffu : (1u << last) - 1u) & ~below;
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = (seen >> i) & 1u ? s[i] : __float_as_uint(-INFINITY);
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
  volatile int* abort_flag = &sm->abort_flag;
  const uint32_t code = ERR_TIMEOUT_SOFTMAX;
  const int row_tok = row / a.group, row_head = row - row_tok * a.group;
  uint32_t q_it = 0, sync_uses = 0;
  const float sl2 = a.scale_log2;
  uint32_t blk_it = 0, turn_it = 0;
  if (t == 1) mbar_arrive(&sm->turn[0]);         // the first turn is group 0's
  for (uint32_t n = 0;; ++n) {
    Item item;
    if (!take(sm, n, code, true, &item)) break;
    const Work w = decode<true>(a, item);
    const bool has = w.has(t);
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
      const int mine0 = w.b0(t), mine1 = has ? w.b1(t) : 0;
      bool ok = true;
      for (int j = w.s0; j < w.s1; ++j, ++turn_it) {
        const bool mine = j >= mine0 && j < mine1;
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
        float r[4];
        const int k0 = j * kBlockN;
#pragma unroll
        for (int c = 0; c < 4; ++c) r[c] = tmem_ld32_max(tS + c * 32, s[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          reg_fence(s[c]);
          reg_fence_f(r[c]);
        }
        if (k0 < lo_all || k0 + kBlockN > hi_all) {
          // the mask goes through this block
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mask32(s[c], k0 + c * 32, lo, hi);
            r[c] = max32(s[c]);
          }
        }
        float alpha;
        const bool need = raise_max(fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3])) * sl2, &m_run, &alpha);
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
        l_run = l_run * alpha + (ls0 + ls1);
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
    const bool seen = l_run != 0.f;             // (a NaN is handed on)
    const float inv_l = seen ? 1.f / l_run : 0.f;
    const float lse = seen ? (m_run + log2f(l_run)) * kLn2 : -INFINITY;
    const int h = w.hk * a.group + row_head;
    const bool loaded = !first;                 // the tile had a block: this item's Q is in q[t], and O was written
    const bool final_rows = w.final;
    // a full tile of final rows leaves by TMA through the tile's own Q buffer
    const bool by_tma = final_rows && loaded && tokens == a.tile_tokens;
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
          : w.part + t * kBlockM + row;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        if (loaded) {
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

// SPLIT: joins what the groups and copies have summed of each row, 2 * COPIES
// parts (part i: group i / COPIES, copy i % COPIES), through stage `st` of the
// rings: the item's last V stage, which its issuer leaves to this epilogue.
// There it stands as [part][row][width] floats, 16-byte pieces swizzled by the
// row, in as few passes over the columns as fit (one for eight rows or fewer).
// With many short sequences a CTA comes here every few microseconds: the loops
// have fixed lengths, and all TMEM loads of a pass are in flight at once.
template <int HD, int COPIES>
__device__ __forceinline__ bool join_parts(PagedSmem<HD, false>* sm, const PagedAttnHead& a, const Work& w,
                                           uint32_t tO, float m_run, float l_run, uint32_t st, uint32_t& sync_uses) {
  constexpr int kParts = 2 * COPIES;
  constexpr int kSpan = kBlockM / COPIES;        // rows of a copy
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = warp >> 2, row = threadIdx.x & 127;
  const int rows = w.q_len * a.group;
  const int r = row & (kSpan - 1);
  const int part = t * COPIES + row / kSpan;
  const uint32_t code = ERR_TIMEOUT_SOFTMAX;
  float2* ml = reinterpret_cast<float2*>(sm->scratch);
  ml[threadIdx.x] = make_float2(m_run, l_run);
  if (!warps_sync(&sm->all_sync, sync_uses, &sm->abort_flag, code)) return false;
  float2 v[kParts];
#pragma unroll
  for (int i = 0; i < kParts; ++i) v[i] = ml[i * kSpan + r];
  float m_all = v[0].x;
#pragma unroll
  for (int i = 1; i < kParts; ++i) m_all = fmaxf(m_all, v[i].x);
  float l_all = 0.f;
#pragma unroll
  for (int i = 0; i < kParts; ++i) l_all += v[i].y == 0.f ? 0.f : v[i].y * fast_exp2(v[i].x - m_all);
  // a part has seen something if its sum is not zero; one of NaN (whose maximum
  // may be -inf: NaN scores do not raise it) makes the row NaN
  const float scale = l_run == 0.f ? 0.f : fast_exp2(m_run - m_all) / l_all;
  if (t == 0 && row < kSpan && r < rows) {       // the first copy's threads know the row's LSE
    const int tok = a.row_token(r), h = w.hk * a.group + r - tok * a.group;
    const float lse = l_all != 0.f ? (m_all + log2f(l_all)) * kLn2 : -INFINITY;
    if (w.final)
      a.lse[static_cast<int64_t>(h) * a.lse_stride + w.q_row0 + tok] = lse;
    else
      a.lse_part[w.part + r] = lse;
  }
  float4* stage = reinterpret_cast<float4*>(sm->kv[st]);
  const int log_passes = COPIES * rows <= 32 ? 0 : COPIES * rows <= 64 ? 1 : 2;
  const int width = HD >> log_passes;            // columns of a pass
  const int log_f4 = (HD == 128 ? 5 : 4) - log_passes;            // 16-byte pieces of a row, 4 at least
  const int swz_mask = min(7, (1 << log_f4) - 1);
  const bool warp_rows = (r & ~31) < rows;
#pragma unroll 1
  for (int c = 0; c < 1 << log_passes; ++c) {
    if (warp_rows) {
      float4* dst = stage + ((part * rows + r) << log_f4);
#pragma unroll 1
      for (int x0 = 0; x0 < width; x0 += 32) {   // (a pass of 16 columns loads 16 it does not use)
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(tO + (c * width + x0 & HD - 32), o);
        tmem_wait_ld();
        reg_fence(o);
        const int odd = c * width + x0 & 16;     // of HD 64 in passes of 16: the upper half
        if (r < rows) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (4 * i + x0 >= width) continue;
            const int e = 4 * i;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (scale != 0.f)                    // else O may never have been written
              y = odd ? make_float4(__uint_as_float(o[(e + 16) & 31]) * scale, __uint_as_float(o[(e + 17) & 31]) * scale,
                                    __uint_as_float(o[(e + 18) & 31]) * scale, __uint_as_float(o[(e + 19) & 31]) * scale)
                      : make_float4(__uint_as_float(o[e]) * scale, __uint_as_float(o[e + 1]) * scale,
                                    __uint_as_float(o[e + 2]) * scale, __uint_as_float(o[e + 3]) * scale);
            dst[(x0 / 4 + i) ^ (r & swz_mask)] = y;
          }
        }
      }
    }
    if (!warps_sync(&sm->all_sync, sync_uses, &sm->abort_flag, code)) return false;
    for (int y = threadIdx.x; y < rows << log_f4; y += 2 * kBlockM) {
      const int rr = y >> log_f4, f = y & ((1 << log_f4) - 1);
      float4 u[kParts];
#pragma unroll
      for (int i = 0; i < kParts; ++i) u[i] = stage[((i * rows + rr) << log_f4) + (f ^ (rr & swz_mask))];
      float4 sum = u[0];
#pragma unroll
      for (int i = 1; i < kParts; ++i) {
        sum.x += u[i].x; sum.y += u[i].y; sum.z += u[i].z; sum.w += u[i].w;
      }
      const int col = c * width + 4 * f;
      if (w.final) {
        const int tk = a.row_token(rr), h = w.hk * a.group + rr - tk * a.group;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) +
                                  (static_cast<int64_t>(w.q_row0 + tk) * a.num_heads + h) * HD + col) =
            make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
      } else {
        *reinterpret_cast<float4*>(a.o_part + (w.part + rr) * HD + col) = sum;
      }
    }
    fence_proxy_async_smem();                    // TMA may write the stage after this
    if (!warps_sync(&sm->all_sync, sync_uses, &sm->abort_flag, code)) return false;
  }
  if (threadIdx.x == 0) mbar_arrive(&sm->kv_empty[st]);
  return true;
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
    const Work w = decode<false>(a, item);
    const int rows = w.q_len * a.group;
    const int copies = row_copies(rows);
    const int span = kBlockM / copies;           // rows of a copy
    const int r = row & (span - 1);              // the row it stands for
    const int nch = 4 / copies;                  // 32-column pieces of a block that are this warp's,
    const int ch0 = (quad / nch) * nch;          // from this one on
    const bool warp_rows = (r & ~31) < rows;     // the warp has a row at all
    const int tok = a.row_token(r);
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
    const int blocks = w.s1 - w.s0;
    const int ring = (blocks - 1) & 1;
    const uint32_t st = Ring::stage(ring, (ring ? base1 : base0) + 2u * static_cast<uint32_t>((blocks - 1) >> 1) + 1u);
    base0 += 2u * static_cast<uint32_t>((blocks + 1) / 2);
    base1 += 2u * static_cast<uint32_t>(blocks / 2);
    bool ok;
    if (copies == 4) ok = join_parts<HD, 4>(sm, a, w, tO, m_run, l_run, st, sync_uses);
    else if (copies == 2) ok = join_parts<HD, 2>(sm, a, w, tO, m_run, l_run, st, sync_uses);
    else ok = join_parts<HD, 1>(sm, a, w, tO, m_run, l_run, st, sync_uses);
    if (!ok) return;
  }
}

template <int HD, bool PAIR, bool WHOLE, int N>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedAttnArgs<N> args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  auto* sm = reinterpret_cast<PagedSmem<HD, PAIR>*>(smem_raw);
  if (!WHOLE && threadIdx.x == 0) args.joins[blockIdx.x].last = -1;   // also when this CTA gives up a wait
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
  if constexpr (!WHOLE) {
    sum_blocks<HD, PAIR, N>(sm, args);
    // the join may be set up from here on; it waits for this grid's end itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;

  if (warp >= kProducerWarp) {
    // 384 threads are launched with 168 registers each, 64,512 in all: PAIR's
    // softmax groups take 208 and leave these warps 88 (at 168 the block loop
    // spills, or not, with any change of the code around it).
    if constexpr (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kProducerWarp) {
      if constexpr (WHOLE) produce_whole<HD, PAIR, N>(sm, args, maps);
      else produce<HD, PAIR, N>(sm, args, maps);
    } else if (warp == kAuxWarp) {
      assist<HD, PAIR, N>(sm, args, maps);
    } else {
      if (lane == 0) issue<HD, PAIR, N>(sm, args, tmem, warp - kMmaWarp0);
    }
  } else if constexpr (PAIR) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_pair<HD>(sm, args, maps, tmem);
  } else {
    softmax_split<HD>(sm, args, tmem);
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
constexpr int kJoinRows = 16;                  // blocks that share a unit's rows
constexpr int kFewParts = 4;                   // parts of a row that one warp joins

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
  bool any = false;                            // a part that has seen a key, or is NaN
  for (int i = lane; i < n; i += 32) {
    any = any || lse_s[i] != -INFINITY;
    m = fmaxf(m, lse_s[i]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const bool seen = __any_sync(0xffffffffu, any);
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

// The same by one warp, for few parts.
template <int HD, typename F>
__device__ __forceinline__ void join_row_warp(const PagedAttnHead& a, int n, F part, int64_t o_row, float* lse_out) {
  constexpr int C = HD / 32;
  const int lane = threadIdx.x & 31;
  float l[kFewParts], x[kFewParts][C];
#pragma unroll
  for (int i = 0; i < kFewParts; ++i) {
    l[i] = -INFINITY;
    if (i < n) {
      l[i] = a.lse_part[part(i)];
      const float* src = a.o_part + part(i) * HD + lane * C;
      if constexpr (C == 4) *reinterpret_cast<float4*>(x[i]) = *reinterpret_cast<const float4*>(src);
      else *reinterpret_cast<float2*>(x[i]) = *reinterpret_cast<const float2*>(src);
    }
  }
  float m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kFewParts; ++i) m = fmaxf(m, l[i]);
  float acc[C] = {};
#pragma unroll
  for (int i = 0; i < kFewParts; ++i) {
    if (l[i] == -INFINITY) continue;             // nothing seen in this part
    const float wgt = expf(l[i] - m);
    sum += wgt;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(wgt, x[i][c], acc[c]);
  }
  const bool seen = sum != 0.f;                // (a NaN is handed on)
  const float inv = seen ? 1.f / sum : 0.f;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + o_row * HD + lane * C;
  if constexpr (C == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) *lse_out = seen ? m + logf(sum) : -INFINITY;
}

// And for many parts: the lanes take the parts' lse, then the warp goes through
// them with kManyLoads rows in flight.  (A block to a row, for hundreds of rows,
// took twice as long as the attention: 35 us for 200 queries over 1,536 keys.)
constexpr int kManyLoads = 8;
template <int HD, typename F>
__device__ __forceinline__ void join_row_many(const PagedAttnHead& a, int n, F part, int64_t o_row, float* lse_out) {
  constexpr int C = HD / 32;
  constexpr int kLane = (kMaxParts + 31) / 32;
  const int lane = threadIdx.x & 31;
  float l[kLane], m = -INFINITY, sum = 0.f;
  bool any = false;
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int i = 32 * k + lane;
    l[k] = i < n ? a.lse_part[part(i)] : -INFINITY;
    any = any || l[k] != -INFINITY;
    m = fmaxf(m, l[k]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const bool seen = __any_sync(0xffffffffu, any);
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    l[k] = l[k] == -INFINITY ? 0.f : expf(l[k] - m);             // the part's weight
    sum += l[k];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  float acc[C] = {};
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    for (int i0 = 32 * k; i0 < min(n, 32 * k + 32); i0 += kManyLoads) {
      float x[kManyLoads][C];
#pragma unroll
      for (int u = 0; u < kManyLoads; ++u) {
        const float* src = a.o_part + part(min(i0 + u, n - 1)) * HD + lane * C;
        if constexpr (C == 4) *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(src);
      }
#pragma unroll
      for (int u = 0; u < kManyLoads; ++u) {
        const float wgt = __shfl_sync(0xffffffffu, l[k], (i0 + u) & 31);   // 0 behind the last part
        if (wgt == 0.f) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = fmaf(wgt, x[u][c], acc[c]);
      }
    }
  }
  const float inv = seen ? 1.f / sum : 0.f;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + o_row * HD + lane * C;
  if constexpr (C == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) *lse_out = seen ? m + logf(sum) : -INFINITY;
}

// Block x looks after the unit that begins in CTA x and goes on in the CTAs
// behind it; kJoinRows blocks share its rows, a warp to a row or, where that
// leaves one for each block, a whole block.  Four blocks an SM (64 registers):
// at two, most of the time is blocks that find nothing to join (48 units of a
// chunk over 2,048 keys: 30 against 33 us with the attention).
// FEW_ROWS: slot_rows <= kJoinRows.
template <int HD, bool PAIR, bool FEW_ROWS>
__global__ void __launch_bounds__(kJoinThreads, 4) paged_join_kernel(const __grid_constant__ PagedAttnHead a) {
  const int c = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedJoin j = a.joins[c];
  if (j.last < 0) return;
  const int n = j.last - c + 1;
  const bool few = n <= kFewParts, by_warp = few || !FEW_ROWS;
  constexpr int kWarps = kJoinThreads / 32;
  for (int r = by_warp ? blockIdx.y * kWarps + threadIdx.x / 32 : blockIdx.y; r < a.slot_rows;
       r += by_warp ? kJoinRows * kWarps : kJoinRows) {
    const int row = PAIR ? r % kBlockM : r;                       // of its tile
    const int tok_t = row / a.group, tok = (j.tile0 + (PAIR ? r / kBlockM : 0)) * a.tile_tokens + tok_t;
    if (tok_t >= a.tile_tokens || tok >= j.q_len) continue;
    const int h = j.hk * a.group + row - tok_t * a.group;
    const auto part = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.slot_rows + r; };
    const int64_t o_row = static_cast<int64_t>(j.q_row0 + tok) * a.num_heads + h;
    float* lse = a.lse + static_cast<int64_t>(h) * a.lse_stride + j.q_row0 + tok;
    if (few) join_row_warp<HD>(a, n, part, o_row, lse);
    else if constexpr (FEW_ROWS) join_row<HD>(a, n, part, o_row, lse);
    else join_row_many<HD>(a, n, part, o_row, lse);
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

template <int HD, bool PAIR, bool WHOLE, int N>
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
    e = cudaFuncSetAttribute(paged_attn_kernel<HD, PAIR, WHOLE, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    word.fetch_or(uint64_t(1) << (dev & 63));
  }
  paged_attn_kernel<HD, PAIR, WHOLE, N><<<WHOLE ? a.whole : kPagedCtas, kThreads, smem, stream>>>(maps, a);
  return cudaGetLastError();
}

template <int HD, bool PAIR>
cudaError_t attn_kind(const PagedMaps& maps, const PagedAttnArgs<kMaxSegs>& a, cudaStream_t stream) {
  if (a.whole > 0) return launch_attn<HD, PAIR, true, kFewSegs>(maps, cut<kFewSegs>(a), stream);
  return a.n_segs <= kFewSegs ? launch_attn<HD, PAIR, false, kFewSegs>(maps, cut<kFewSegs>(a), stream)
                              : launch_attn<HD, PAIR, false, kMaxSegs>(maps, a, stream);
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

}  // namespace

cudaError_t launch_paged_attn(int head_dim, bool pair, const PagedMaps& maps, const PagedAttnArgs<kMaxSegs>& a,
                              cudaStream_t stream) {
  if (head_dim == 64) return pair ? attn_kind<64, true>(maps, a, stream) : attn_kind<64, false>(maps, a, stream);
  return pair ? attn_kind<128, true>(maps, a, stream) : attn_kind<128, false>(maps, a, stream);
}

cudaError_t launch_paged_join(int head_dim, bool pair, const PagedAttnHead& a, cudaStream_t stream) {
  const dim3 grid(kPagedCtas, static_cast<unsigned>(std::min(a.slot_rows, kJoinRows)));
  const bool few = a.slot_rows <= kJoinRows;   // never of a chunk: its slots are two tiles
  if (head_dim == 64)
    return pair  ? launch_after(paged_join_kernel<64, true, false>, grid, stream, a)
           : few ? launch_after(paged_join_kernel<64, false, true>, grid, stream, a)
                 : launch_after(paged_join_kernel<64, false, false>, grid, stream, a);
  return pair  ? launch_after(paged_join_kernel<128, true, false>, grid, stream, a)
         : few ? launch_after(paged_join_kernel<128, false, true>, grid, stream, a)
               : launch_after(paged_join_kernel<128, false, false>, grid, stream, a);
}

uint32_t paged_attn_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_paged_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
