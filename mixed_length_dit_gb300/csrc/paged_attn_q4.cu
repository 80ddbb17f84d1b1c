// Attention of few rows (single tokens, drafts) over a paged cache held in 4
// bits.
//
//     S = q K^T scale,  o = softmax(S) V,   K = c_k s_k,  V = c_v s_v
//
// with a step s for every 32 columns (a group) of a token's head.  The codes
// n = c + 8 are not made into values: the products run over n itself,
//
//     S = scale sum_g s_k[g] (sum_(i in g) q_i n_i - 8 sum_(i in g) q_i)
//     o_i = sum_j (p_j s_v[j, g]) (n_ji - 8)
//
// so that a key's steps multiply four sums instead of 128 codes, and a value's
// steps the probability before it is rounded to bf16 (the one rounding, as in the
// bf16 attention: the tensor cores take P in V's type).
//
// Bound by HBM at best, by the way from codes to operands otherwise: an SM's share
// of HBM is 43 codes a clock.  So K and V are the A operands of warp-level products
// (16 keys, or 16 columns, by the 8 rows of a query tile), unpacked in registers
// where they are used.  The 5th-generation tensor cores take B from shared memory
// only, and A from there or from TMEM: at HBM's rate unpacked codes would cross
// shared memory twice, 170 bytes a clock of its 128, so three quarters of that rate
// at best.  For few rows that is little more than what follows reaches; for 32 rows
// and more, whose codes are unpacked here again for every 16, it would be several
// times faster, and is not built.
//
// The codes become operands by masks alone.  A 16-bit pattern below 256 is, as a
// bf16, its number times 2^-133 (subnormal, or with the lowest exponent), and the
// products take such numbers as they are.  So a code in bits 0 to 3 is n, one in
// bits 4 to 7 is 16 n, and the other factor brings the size: a row of q is scaled
// by a power of two so that its largest element lies at 2^120 (columns whose codes
// come 16 times over by 1/16 of it), a key's step by 2^40 and a value's by 2^60.  All of
// it is exact.
// A word's codes are four operands after five logical operations; two tokens' codes
// of a column, as V wants them, take a byte permutation more for each.
//
// A unit is (sequence, key head, tile of 8 NT rows: queries times the heads that
// share the key head).  The tiles of 32 keys of all units stand in one line that
// is cut into equal pieces, one a CTA, as in the bf16 attention; the warps of a
// CTA take a unit's tiles in turn and are joined in shared memory; units that a cut
// goes through are joined by a second launch.  Few short units have a CTA each, or a
// cluster, whose CTAs share the tiles and join them through distributed shared
// memory.  One warp of a CTA copies the tiles of all others.
//
// Measured: 48 tokens over caches to 16,384 keys (40 / 8 heads, pages of 16) in 120 us,
// 483 MB at 4.0 TB/s; the same cache in bf16 takes 290.  Copies alone took 84 us there,
// everything but the copies 103.  Nothing is saturated: issue slots 52%, logical unit
// 50%, shared memory's data path 46%, tensor pipe 22%, HBM 55%; a tile is one chain of
// products, exponentials and products, and an SM has 14 warps to overlap them.  8-bit
// products (e4m3 codes, q in two parts) are made of two 16-bit ones and conversions on
// this GPU and gained nothing; codes as 128 + n with their offset taken off took 179 us,
// masks alone 141.
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "paged.h"
#include "paged_q4.cuh"

namespace zl {
namespace {

__device__ uint32_t g_attn_q4_err;

constexpr int kTile = 32;                      // keys of a warp's step
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;                // the running maximum lags by this much (base 2) at most
constexpr uint32_t kLow = 0x000f000fu;         // of codes: n, and 16 n
constexpr uint32_t kHigh = 0x00f000f0u;
constexpr uint32_t kMinus8 = 0x80088008u;      // -8 n's unit, twice, and 16 times that
constexpr uint32_t kMinus128 = 0x80808080u;
constexpr int kKeyExp = 40;                    // keys' steps, and so scores before the row's scale, come 2^40 times over
constexpr float kKeyScale = 0x1p40f;
constexpr float kValueScale = 0x1p60f;         // of values' steps, and so of P
constexpr float kOutScale = 0x1p73f;           // from sums of codes to the output

template <int HD, int NT>
struct Cfg {
  static constexpr int G = HD / kQ4Group;
  static constexpr int RT = 8 * NT;            // rows of a unit
  // Warps of a CTA that compute; one more copies.  128 registers a thread hold 8 rows'
  // sums, 168 hold 16's: 5 warps for 8 rows take 119 us (above), 7 for 16 rows 56 instead
  // of 53 (16 drafts of 3 to 8 tokens, 32 / 8 heads, 4,096 keys each); one CTA of 8 warps
  // and 255 registers took 150 instead of 128.  Units of 32 rows spill: 68 instead of 53.
  static constexpr int W = NT == 1 ? 7 : 5;
  static constexpr int kThreads = 32 * (W + 1);
  static constexpr int kCtasPerSm = 2;
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kRegion = kTile * kQ4Row<HD>;           // keys, or values, of a stage
  static_assert(W <= 8, "a warp's lanes look at 8 warps");
  static constexpr int kPad = HD + 4;          // floats of a row to be joined (rows 2c of four lanes in different banks)
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const uint8_t* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// d = a b + c.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint2& b, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int G>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[G]) {
  if constexpr (G == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  }
}
template <int G>
__device__ __forceinline__ void load_floats(const float* p, float (&w)[G]) {
  if constexpr (G == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    const float2 u = *reinterpret_cast<const float2*>(p);
    w[0] = u.x; w[1] = u.y;
  }
}

// A token's steps from its bytes to floats, times `by`.
template <int G>
__device__ __forceinline__ void spread_steps(float* to, const uint8_t* p, float by, bool there = true) {
  const uint64_t by2 = f2_pack(by, by);
  const auto scaled = [&](float2 x) {
    f2_unpack(f2_mul(f2_pack(x.x, x.y), by2), x.x, x.y);
    return x;
  };
  if constexpr (G == 4) {
    const uint32_t w = there ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    const float2 a = scaled(q4_steps01(w)), b = scaled(q4_steps23(w));
    *reinterpret_cast<float4*>(to) = make_float4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<float2*>(to) = scaled(q4_steps01(there ? *reinterpret_cast<const uint16_t*>(p) : 0u));
  }
}

// ------------------------------------------------------------------ the line of units
// Tiles [t0, t1) of 32 keys that rows [r0, r1) of a sequence see; none: t1 = t0.
struct Tiles {
  int t0, t1;
};

__device__ __forceinline__ void keys_of(const AttnQ4Head& a, int len, int p, int* lo, int* hi) {
  *hi = a.causal ? max(0, min(len, p + 1)) : len;
  *lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;   // p may be far below zero
}

__device__ __forceinline__ Tiles tiles_of(const AttnQ4Head& a, int len, int q_len, int r0, int r1) {
  int lo, hi, x;
  keys_of(a, len, len - q_len + a.row_token(r0), &lo, &x);
  keys_of(a, len, len - q_len + a.row_token(r1 - 1), &x, &hi);
  if (hi <= lo) return {0, 0};
  return {lo / kTile, (hi + kTile - 1) / kTile};
}

template <int N>
__device__ __forceinline__ int length_of(const AttnQ4Args<N>& a, int seg) {
  const int len = __ldg(a.kv_lens + a.segs[seg].seq);
  if (len >= 0 && len <= a.max_kv_len) return len;
  atomicOr(&g_attn_q4_err, ERR_BAD_PAGE);
  return len < 0 ? 0 : a.max_kv_len;
}

// Row tiles of a segment; what a unit weighs (in waves, a tile for every warp),
// with the cost of beginning and ending it.
template <int RT>
__device__ __forceinline__ int row_tiles(const AttnQ4Head& a, int q_len) { return (q_len * a.group + RT - 1) / RT; }

constexpr int kUnitCost = 1;                   // as long as a wave: queries in, warps joined
template <int W>
__device__ __forceinline__ int waves_of(Tiles t) { return max(1, (t.t1 - t.t0 + W - 1) / W); }

template <int W, int RT>
__device__ __forceinline__ int unit_weight(const AttnQ4Head& a, int len, int q_len, int rt) {
  const int rows = q_len * a.group;
  return kUnitCost + waves_of<W>(tiles_of(a, len, q_len, rt * RT, min(rows, rt * RT + RT)));
}

// The weight of a segment's row tiles for one key head.
template <int W, int RT>
__device__ __forceinline__ int seg_weight(const AttnQ4Head& a, int len, int q_len) {
  int sum = 0;
  for (int rt = 0; rt < row_tiles<RT>(a, q_len); ++rt) sum += unit_weight<W, RT>(a, len, q_len, rt);
  return sum;
}

__device__ __forceinline__ int64_t div_nonneg(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The CTA's piece of the line, by all threads.  weights: room for every segment's.
template <int W, int RT, int N>
__device__ void find_piece(const AttnQ4Args<N>& a, int32_t* weights, Q4Piece* out) {
  const int lane = threadIdx.x & 31;
  const int nk = a.num_kv_heads;
  Q4Piece p = {0, 0, 0, 0, 0, 1};
  if (a.whole > 0) {                           // few short units: each CTA, or cluster, has one to itself
    if (threadIdx.x < 32) {
      int x = blockIdx.x / a.share;
      for (;; ++p.seg) {
        const int units = row_tiles<RT>(a, a.segs[p.seg].q_len) * nk;
        if (x < units) break;
        x -= units;
      }
      const int rts = row_tiles<RT>(a, a.segs[p.seg].q_len);
      p.hk = x / rts;
      p.rt = x - p.hk * rts;
      p.left = 1;                              // any piece ends within its first unit
      if (lane == 0) *out = p;
    }
    __syncthreads();
    return;
  }
  for (int s = threadIdx.x; s < a.n_segs; s += blockDim.x)
    weights[s] = seg_weight<W, RT>(a, length_of(a, s), a.segs[s].q_len);
  __syncthreads();
  if (threadIdx.x < 32) {
    int64_t total = 0;
    for (int s = lane; s < a.n_segs; s += 32) total += weights[s];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    total *= nk;
    p.per = max(int64_t(1 + kUnitCost), div_nonneg(total + gridDim.x - 1, gridDim.x));
    const int64_t g = blockIdx.x * p.per;
    p.left = max(int64_t(0), min(total - g, p.per));
    if (p.left > 0) {
      int64_t base = 0;
      for (int chunk = 0;; chunk += 32) {
        const int64_t w = chunk + lane < a.n_segs ? weights[chunk + lane] : 0;
        int64_t incl = w * nk;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += y;
        }
        incl += base;
        const uint32_t past = __ballot_sync(0xffffffffu, incl > g);
        if (past != 0) {
          const int k = __ffs(past) - 1;
          const int64_t one = __shfl_sync(0xffffffffu, w, k);
          int64_t off = g - (__shfl_sync(0xffffffffu, incl, k) - one * nk);
          p.seg = chunk + k;
          p.hk = static_cast<int>(div_nonneg(off, one));
          off -= p.hk * one;
          const int q_len = a.segs[p.seg].q_len;
          if (row_tiles<RT>(a, q_len) > 1) {
            const int len = length_of(a, p.seg);
            for (;; ++p.rt) {
              const int weight = unit_weight<W, RT>(a, len, q_len, p.rt);
              if (off < weight) break;
              off -= weight;
            }
          }
          p.off = static_cast<int>(off);
          break;
        }
        base = __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) *out = p;
  }
  __syncthreads();
}

// One item: the tiles [s0, s1) of a unit that the CTA has.
struct Item {
  int seg, hk, rt;
  int len, q_len, rows;                        // rows of the unit
  int s0, s1;
  int slot;                                    // slot of partial rows; -1: the rows are final
  int behind;                                  // of a unit that begins here: what it weighs behind the piece, else 0
};

// Walks a CTA's items; every warp for itself, once for its copies and once for
// its products.
struct Walk {
  int seg, hk, rt;
  int off;                                     // into the unit
  int64_t left;                                // of the piece
  int len, q_len;

  template <int N>
  __device__ __forceinline__ void start(const AttnQ4Args<N>& a, const Q4Piece& p) {
    seg = p.seg; hk = p.hk; rt = p.rt; off = p.off; left = p.left;
    if (left > 0) {
      len = length_of(a, seg);
      q_len = a.segs[seg].q_len;
    }
  }

  // The next item; false: none left.
  template <int W, int RT, int N>
  __device__ __forceinline__ bool next(const AttnQ4Args<N>& a, Item* it) {
    while (left > 0) {
      const int rows = q_len * a.group, r0 = rt * RT;
      it->seg = seg; it->hk = hk; it->rt = rt;
      it->len = len; it->q_len = q_len;
      it->rows = min(RT, rows - r0);
      const Tiles t = tiles_of(a, len, q_len, r0, r0 + it->rows);
      it->s0 = t.t0;
      it->s1 = t.t1;
      it->slot = -1;
      it->behind = 0;
      if (a.whole > 0) {
        left = 0;
        return true;
      }
      const int waves = waves_of<W>(t), rest = kUnitCost + waves - off;
      const int avail = left < rest ? static_cast<int>(left) : rest;
      const int w0 = max(off - kUnitCost, 0), w1 = max(off + avail - kUnitCost, 0);      // the piece's waves of the unit
      if (w1 - w0 < waves) {
        it->slot = w0 == 0 ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
        if (w0 == 0) it->behind = rest - avail;
        it->s0 = t.t0 + w0 * W;
        it->s1 = min(t.t1, t.t0 + w1 * W);
      }
      left -= avail;
      off = 0;
      if (++rt * RT >= rows) {
        rt = 0;
        if (++hk >= a.num_kv_heads) {
          hk = 0;
          ++seg;
          if (left > 0) {
            len = length_of(a, seg);
            q_len = a.segs[seg].q_len;
          }
        }
      }
      if (w1 > w0) return true;
    }
    return false;
  }
};

template <int HD, int NT>
struct Smem {
  using C = Cfg<HD, NT>;
  alignas(128) uint8_t stage[C::W][C::kStages][2][C::kRegion];
  alignas(16) float part[C::W][8][C::kPad];    // 8 rows of every warp
  float m[C::W][C::RT], l[C::W][C::RT], lse[C::RT];
  // Of the item's queries: fragments of q^T for a group's two products, and their first
  // sums, -8 sum q of rows 2c, 2c + 1 for keys g and g + 8.
  uint4 q[NT][C::G][32];
  float4 q_sum[NT][C::G][4];
  float q_scale[C::RT];                        // a row's scores from its sums: scale and log2 e, its own scale
  alignas(8) uint64_t full[C::W][C::kStages], empty[C::W][C::kStages];
  Q4Piece piece;
  Walk walk[C::W];                             // of the warps that compute: it changes once in many tiles
  Item item[C::W];
  int abort_flag;
  int32_t weights[kMaxSegs];
};

// The next item of a warp, by all its lanes; false: none left.
template <int W, int RT, int N>
__device__ __forceinline__ bool next_item(const AttnQ4Args<N>& a, Walk* walk, Item* item) {
  Walk w = *walk;
  Item it;
  const bool ok = w.next<W, RT>(a, &it);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    *walk = w;
    *item = it;
  }
  __syncwarp();
  return ok;
}

// ------------------------------------------------------------------ copies
// Where the 16 keys of half a tile lie in a region: pages of 16 tokens are copied
// with their steps behind their codes, larger pages' codes and steps apart.
struct Layout {
  int codes_half, steps, steps_half;
};

template <int HD>
__device__ __forceinline__ Layout layout_of(const AttnQ4Head& a) {
  if (a.page_shift == 4) return {16 * kQ4Row<HD>, 16 * kQ4Codes<HD>, 16 * kQ4Row<HD>};
  return {16 * kQ4Codes<HD>, kTile * kQ4Codes<HD>, 16 * kQ4Steps<HD>};
}

// The first tile of an item for the CTA's first warp; the others' follow, and a
// warp's next one is W tiles on, or, of a unit that a cluster of `share` CTAs has, W
// tiles times that.
template <int W>
__device__ __forceinline__ int first_tile(const AttnQ4Head& a, const Item& it) {
  return it.s0 + (a.share > 1 ? static_cast<int>(blockIdx.x) % a.share * W : 0);
}

// The warp that copies (TMA bulk): a tile for each warp of the CTA at a time, by four
// lanes a tile.  They bring keys' codes and steps and values' codes and steps, or of
// pages of 16 each one's two pages, or of pages of 32 each one's page.  (Where every
// warp copied for itself the first tile came 3 us later, behind the copies of later
// stages; one thread that issues all copies took as long.)
template <int HD, int NT, int N>
__device__ void produce(const AttnQ4Args<N>& a, Smem<HD, NT>* sm, const Q4Piece& piece) {
  using C = Cfg<HD, NT>;
  const int lane = threadIdx.x & 31, w = lane >> 2, part = lane & 1;
  const int ps = 1 << a.page_shift;
  const bool small = a.page_shift == 4, values = lane & 2;
  uint32_t stage = 0, parity = 1;              // of warp w's stages
  Walk walk;
  walk.start(a, piece);
  Item it;
  while (walk.next<C::W, C::RT>(a, &it)) {
    const uint8_t* block = (values ? a.v_pages : a.k_pages) + ((static_cast<int64_t>(it.hk) * kQ4Row<HD>) << a.page_shift);
    const int32_t* entries = a.page_table + static_cast<int64_t>(a.segs[it.seg].seq) * a.table_cols;
    int tile = first_tile<C::W>(a, it) + w;
    const auto fetch = [&]() {                 // the page of the lane's copy
      const int pos = tile * kTile + (small ? 16 * part : 0);
      return w < C::W && tile < it.s1 && pos < it.len ? __ldg(entries + (pos >> a.page_shift)) : 0;
    };
    int page = fetch();
    while (true) {
      const bool mine = w < C::W && tile < it.s1;
      if (!__any_sync(0xffffffffu, mine)) break;
      const int pos = tile * kTile, row = pos & (ps - 1);
      const bool both = !small || pos + 16 < it.len;             // else the second page is not there
      uint32_t bytes = 0, from = 0, to = 0;
      if (mine) {
        if (small) {
          bytes = part == 0 || both ? 16 * kQ4Row<HD> : 0;
          to = part * 16 * kQ4Row<HD>;
        } else if (ps == kTile) {
          bytes = part ? 0 : C::kRegion;
        } else {
          bytes = part ? kTile * kQ4Steps<HD> : kTile * kQ4Codes<HD>;
          from = part ? ps * kQ4Codes<HD> + row * kQ4Steps<HD> : row * kQ4Codes<HD>;
          to = part ? kTile * kQ4Codes<HD> : 0;
        }
        if (bytes > 0 && static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) {
          atomicOr(&g_attn_q4_err, ERR_BAD_PAGE);                // reads page 0 in its place
          page = 0;
        }
      }
      const uint8_t* src = block + static_cast<int64_t>(page) * a.page_bytes + from;
      tile += C::W * a.share;
      page = fetch();
      // (after a wait that ran out nothing is read any more)
      const bool ok = !mine || mbar_wait(&sm->empty[w][stage], parity, &sm->abort_flag, &g_attn_q4_err, ERR_TIMEOUT_PRODUCER);
      if (!__all_sync(0xffffffffu, ok)) return;
      uint64_t* bar = &sm->full[mine ? w : 0][stage];
      if (mine && (lane & 3) == 0) mbar_arrive_expect_tx(bar, both ? 2 * C::kRegion : C::kRegion);
      __syncwarp();
      if (bytes > 0) bulk_load(smem_u32(sm->stage[w][stage][values]) + to, src, bytes, bar);
      if (mine && ++stage == C::kStages) {
        stage = 0;
        parity ^= 1u;
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ products
// A warp's share of a unit: lane (g, c) = (lane / 4, lane % 4) of the products'
// fragments.  Scores are S^T (keys g, g + 8 by rows 2c, 2c + 1), the output o^T
// (columns 32 q + 4 g + (0 .. 3) by rows 2c, 2c + 1; 2^-73 of it, of the odd
// columns 2^-69).
template <int HD, int NT>
struct Rows {
  using C = Cfg<HD, NT>;
  static constexpr int G = C::G;
  float o[NT][G][2][4];                        // [tile of 16 columns][fragment]
  float m[NT][2], l[NT][2];                    // of rows 2c, 2c + 1; l: the lane's keys alone
  float f[NT][2];                              // their q_scale

  template <int N>
  __device__ __forceinline__ void start(const AttnQ4Args<N>& a, const Item& it, Smem<HD, NT>* sm) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // the warps make the fragments of a group of 8 rows each
#pragma unroll 1
    for (int i = threadIdx.x >> 5; i < NT * G; i += C::W) {
      const int n = i / G, x = i % G, r = 8 * n + g;
      const int row = it.rt * C::RT + r, tok = a.row_token(row);
      const __nv_bfloat16* src = a.q + (a.segs[it.seg].q_row0 + static_cast<int64_t>(tok)) * a.q_stride +
                                 (it.hk * a.group + row - tok * a.group) * HD + 8 * c;
      uint4 u = make_uint4(0, 0, 0, 0);
      uint32_t top = 0;
      if (r < it.rows) {
        u = __ldg(reinterpret_cast<const uint4*>(src + 32 * x));
#pragma unroll
        for (int y = 0; y < G; ++y) top = __vmaxu2(top, q4_top(__ldg(reinterpret_cast<const uint4*>(src + 32 * y))));
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // The row's scale, 2^(up_exp - 127): its largest element goes to 2^120, or is
      // below 2^-7 and goes up by 2^127.  Codes are n 2^-133.
      const int up_exp = min(374 - static_cast<int>(top >> 7), 254);
      const float up = __uint_as_float(static_cast<uint32_t>(up_exp) << 23);
      // 2^133 of the codes and 2^-40 of the keys' steps, back by the row's scale: 2^-34 to
      // 2^101, for the largest queries too.  Finite and above zero whatever the softmax
      // scale, and for a row of NaN or infinities as well, whose products are NaN by
      // themselves: sums of zero stay zero, and keys that are not seen at -inf.
      const float down = __uint_as_float(static_cast<uint32_t>(387 - kKeyExp - up_exp) << 23) * a.scale_log2;
      if (c == 0 && x == 0) sm->q_scale[r] = fminf(fmaxf(down, FLT_MIN), FLT_MAX);
      const float2 x0 = bf16x2_to_float2(u.x), x1 = bf16x2_to_float2(u.y), x2 = bf16x2_to_float2(u.z), x3 = bf16x2_to_float2(u.w);
      // columns j and j + 4 beside one another, as a word's codes are taken; the odd ones' codes come 16 times over
      const float odd = up * 0.0625f;
      sm->q[n][x][lane] = make_uint4(pack_bf16x2(x0.x * up, x2.x * up), pack_bf16x2(x0.y * odd, x2.y * odd),
                                     pack_bf16x2(x1.x * up, x3.x * up), pack_bf16x2(x1.y * odd, x3.y * odd));
      // of scaled elements: 32 of the largest bf16 do not fit a float
      float sum = ((x0.x * up + x0.y * up) + (x1.x * up + x1.y * up)) + ((x2.x * up + x2.y * up) + (x3.x * up + x3.y * up));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum = sum * (-8.f * 0x1p-66f) * 0x1p-67f;
      const float s0 = __shfl_sync(0xffffffffu, sum, 8 * c), s1 = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
      if (g == 0) sm->q_sum[n][x][c] = make_float4(s0, s1, s0, s1);
    }
    named_bar_sync(1, 32 * C::W);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[n][e] = sm->q_scale[8 * n + 2 * c + e];
        m[n][e] = -INFINITY;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < G; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][x][t][i] = 0.f;
    }
  }

  // A tile of 32 keys from position `pos` on.  edge: some row does not see all of
  // them.  `steps`: room for 64 tokens' steps.
  __device__ __forceinline__ void tile(const AttnQ4Head& a, const Item& it, const Smem<HD, NT>* sm, const uint8_t* kr,
                                       const uint8_t* vr, const Layout& lay, float* steps, int pos, bool edge) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // the key of rows g, and 8 on: four lanes' values of a column are in different banks
    const int key_g = g ^ ((g >> 1) & 1);
    const int held = lay.steps + (lane >> 4) * lay.steps_half + (lane & 15) * G;
    spread_steps<G>(steps + lane * G, kr + held, kKeyScale);
    // (past the sequence anything may be held)
    spread_steps<G>(steps + (kTile + lane) * G, vr + held, kValueScale, pos + lane < it.len);
    __syncwarp();
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {              // 16 keys
      uint32_t wa[G], wb[G];
      float sa[G], sb[G];
      const uint8_t* codes = kr + h * lay.codes_half + key_g * kQ4Codes<HD> + c * (4 * G);
      load_words<G>(codes, wa);
      load_words<G>(codes + 8 * kQ4Codes<HD>, wb);
      load_floats<G>(steps + (16 * h + key_g) * G, sa);
      load_floats<G>(steps + (16 * h + 8 + key_g) * G, sb);
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const uint32_t w0[4] = {wa[x] & kLow, wb[x] & kLow, wa[x] & kHigh, wb[x] & kHigh};
        const uint32_t ua = wa[x] >> 8, ub = wb[x] >> 8;
        const uint32_t w1[4] = {ua & kLow, ub & kLow, ua & kHigh, ub & kHigh};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float d[4];
          const float4 z = sm->q_sum[n][x][c];
          const float first[4] = {z.x, z.y, z.z, z.w};
          const uint4 b = sm->q[n][x][lane];
          mma(d, w0, make_uint2(b.x, b.y), first);
          mma(d, w1, make_uint2(b.z, b.w), d);
#pragma unroll
          for (int k = 0; k < 2; ++k) {        // keys g, g + 8
            const float st = k ? sb[x] : sa[x];
            float* to = &s[h][n][2 * k];
            const uint64_t st2 = f2_pack(st, st), d2 = f2_pack(d[2 * k], d[2 * k + 1]);
            f2_unpack(x == 0 ? f2_mul(st2, d2) : f2_fma(st2, d2, f2_pack(to[0], to[1])), to[0], to[1]);
          }
        }
      }
    }
    if (edge) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = a.row_token(min(it.rt * C::RT + 8 * n + 2 * c + e, it.rt * C::RT + it.rows - 1));
          int lo, hi;
          keys_of(a, it.len, it.len - it.q_len + tok, &lo, &hi);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int key = pos + 16 * h + 8 * k + key_g;
              if (key < lo || key >= hi) s[h][n][2 * k + e] = -INFINITY;
            }
        }
    }
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // (a mask's -inf stays -inf: f is above zero)
        const float top = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
        raise = raise || top * f[n][e] > m[n][e] + kRescale;
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e])) * f[n][e];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          // a row's own scores decide, so that its bits do not depend on the rows beside it
          const float to = top > m[n][e] + kRescale ? top : m[n][e];
          const float alpha = to == m[n][e] ? 1.f : fast_exp2(m[n][e] - to);
          m[n][e] = to;
          l[n][e] *= alpha;
#pragma unroll
          for (int x = 0; x < G; ++x)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              o[n][x][t][e] *= alpha;
              o[n][x][t][2 + e] *= alpha;
            }
        }
    }
    // The scaled score is rounded as the maximum was, so that the largest one's difference
    // is zero whatever its size: a fused product would leave the maximum's rounding, 2^8
    // for scores of 2^32, in the exponent.  (The compiler fuses products and sums that
    // are both packed.)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint64_t neg2 = f2_pack(m[n][0] == -INFINITY ? 0.f : -m[n][0], m[n][1] == -INFINITY ? 0.f : -m[n][1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float* p = &s[h][n][2 * k];
          f2_unpack(f2_add(f2_pack(__fmul_rn(p[0], f[n][0]), __fmul_rn(p[1], f[n][1])), neg2), p[0], p[1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[e] = fast_exp2(p[e]);
            l[n][e] += p[e];
          }
        }
    }
    uint32_t w[2][4];
    float2 st[2][2];
#pragma unroll
    for (int x = 0; x < G; ++x) {
      // the codes of the keys of rows 2c, 2c + 1 and 2c + 8, 2c + 9 of each 16, and the steps
      // of those of rows g, g + 8, for two groups: four columns of a group are half a word
      if ((x & 1) == 0) {
        asm volatile("" ::: "memory");         // not loaded further ahead: registers
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = ((2 * c + (k & 1)) ^ (c & 1)) + 8 * (k >> 1);
            w[h][k] = *reinterpret_cast<const uint32_t*>(vr + h * lay.codes_half + row * kQ4Codes<HD> + 2 * G * g + 2 * x);
          }
          st[h][0] = *reinterpret_cast<const float2*>(steps + (kTile + 16 * h + key_g) * G + x);
          st[h][1] = *reinterpret_cast<const float2*>(steps + (kTile + 16 * h + 8 + key_g) * G + x);
        }
      }
      uint2 b[2][NT];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float t[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float step = x & 1 ? st[h][k].y : st[h][k].x;
            f2_unpack(f2_mul(f2_pack(s[h][n][2 * k], s[h][n][2 * k + 1]), f2_pack(step, step)), t[2 * k], t[2 * k + 1]);
          }
          b[h][n] = make_uint2(transpose8(pack_bf16x2(t[0], t[1])), transpose8(pack_bf16x2(t[2], t[3])));
        }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int byte = 2 * (x & 1) + t;      // of each word: the codes of rows g and (16 times) g + 8 of the tile
        uint32_t v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t u = __byte_perm(w[h][2 * k], w[h][2 * k + 1], byte | (4 + byte) << 8);
            v[h][2 * k] = add_bf16x2(u & kLow, kMinus8);
            v[h][2 * k + 1] = add_bf16x2(u & kHigh, kMinus128);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma(o[n][x][t], v[0], b[0][n], o[n][x][t]);
          mma(o[n][x][t], v[1], b[1][n], o[n][x][t]);
        }
      }
    }
  }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What the cluster's CTA `rank` has at p of its shared memory.
__device__ __forceinline__ uint32_t in_cluster(const void* p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(in_cluster(p, rank)) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(const float* p, int rank) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(in_cluster(p, rank)) : "memory");
  return x;
}

__device__ __forceinline__ void add4(float4& o, float f, const float4& u) {
  o.x = fmaf(f, u.x, o.x);
  o.y = fmaf(f, u.y, o.y);
  o.z = fmaf(f, u.z, o.z);
  o.w = fmaf(f, u.w, o.w);
}

// Four columns of a row of the item's sequence.
template <int HD, int N>
__device__ __forceinline__ void put_row(const AttnQ4Args<N>& a, const Item& it, int row, int col, const float4& o, float lse) {
  const int tok = a.row_token(row), h = it.hk * a.group + row - tok * a.group;
  const int64_t q_row = a.segs[it.seg].q_row0 + static_cast<int64_t>(tok);
  *reinterpret_cast<uint2*>(a.o + (q_row * a.num_heads + h) * HD + col) =
      make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (col == 0) a.lse[h * a.lse_stride + q_row] = lse;
}

// Joins the warps' shares of an item and writes its rows: every warp weights its
// sums by what it has of a row, and threads add them up, 8 rows at a time.
template <int HD, int NT, int N>
__device__ __forceinline__ void finish(const AttnQ4Args<N>& a, const Item& it, Smem<HD, NT>* sm, Rows<HD, NT>& r) {
  using C = Cfg<HD, NT>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = r.l[n][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (g == 0) {
        sm->m[warp][8 * n + 2 * c + e] = r.m[n][e];
        sm->l[warp][8 * n + 2 * c + e] = l;
      }
    }
  named_bar_sync(1, 32 * C::W);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // lane g looks at warp g; the rows' maximum, sum and this warp's weight
      const int i = 8 * n + 2 * c + e;
      const float m = g < C::W ? sm->m[g][i] : -INFINITY;
      float top = m;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = top == -INFINITY ? 0.f : top;
      float l = g < C::W ? fast_exp2(m - top) * sm->l[g][i] : 0.f;             // 0 of a warp that has seen no key
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      const bool seen = l != 0.f;              // (a NaN is handed on)
      const float f = seen ? fast_exp2(r.m[n][e] - top) / l * kOutScale : 0.f;
      if (warp == 0 && g == 0) sm->lse[i] = seen ? (top + log2f(l)) * kLn2 : -INFINITY;
#pragma unroll
      for (int x = 0; x < C::G; ++x)
        *reinterpret_cast<float4*>(&sm->part[warp][2 * c + e][32 * x + 4 * g]) =
            make_float4(r.o[n][x][0][e] * f, r.o[n][x][0][2 + e] * (f * 0.0625f), r.o[n][x][1][e] * f,
                        r.o[n][x][1][2 + e] * (f * 0.0625f));
    }
    named_bar_sync(1, 32 * C::W);
    constexpr int F4 = HD / 4;
    for (int y = threadIdx.x; y < 8 * F4; y += 32 * C::W) {
      const int k = y / F4, col = 4 * (y % F4), i = 8 * n + k;
      if (i >= it.rows) break;                 // rows come in order
      float4 o = *reinterpret_cast<const float4*>(&sm->part[0][k][col]);
#pragma unroll
      for (int w = 1; w < C::W; ++w) add4(o, 1.f, *reinterpret_cast<const float4*>(&sm->part[w][k][col]));
      if (a.share > 1) {                       // the cluster's CTAs join theirs below
        *reinterpret_cast<float4*>(&sm->part[0][k][col]) = o;
      } else if (it.slot >= 0) {
        const int64_t at = static_cast<int64_t>(it.slot) * C::RT + i;
        *reinterpret_cast<float4*>(a.o_part + at * HD + col) = o;
        if (col == 0) a.lse_part[at] = sm->lse[i];
      } else {
        put_row<HD>(a, it, it.rt * C::RT + i, col, o, sm->lse[i]);
      }
    }
    if (a.share > 1) {
      cluster_sync();
      const int rank = blockIdx.x % a.share;
      for (int y = threadIdx.x + 32 * C::W * rank; y < 8 * F4; y += 32 * C::W * a.share) {
        const int k = y / F4, col = 4 * (y % F4), i = 8 * n + k;
        if (i >= it.rows) break;
        float top = -INFINITY;
        for (int r2 = 0; r2 < a.share; ++r2) top = fmaxf(top, ld_cluster(&sm->lse[i], r2));
        top = top == -INFINITY ? 0.f : top;
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r2 = 0; r2 < a.share; ++r2) {
          const float lse = ld_cluster(&sm->lse[i], r2);
          if (lse == -INFINITY) continue;      // a CTA that has seen no key
          const float f = expf(lse - top);
          l += f;
          add4(o, f, ld_cluster4(&sm->part[0][k][col], r2));
        }
        const bool seen = l != 0.f;
        const float inv = seen ? 1.f / l : 0.f;
        put_row<HD>(a, it, it.rt * C::RT + i, col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv),
                    seen ? top + logf(l) : -INFINITY);
      }
      cluster_sync();                          // the others have read
    }
    named_bar_sync(1, 32 * C::W);
  }
}

template <int HD, int NT, int N>
__global__ void __launch_bounds__(Cfg<HD, NT>::kThreads, Cfg<HD, NT>::kCtasPerSm)
paged_attn_q4_kernel(const __grid_constant__ AttnQ4Args<N> a) {
  using C = Cfg<HD, NT>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto* sm = reinterpret_cast<Smem<HD, NT>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.whole == 0 && threadIdx.x == 0) a.joins[blockIdx.x].last = -1;
  if (warp < C::W && lane < C::kStages) {
    mbar_init(&sm->full[warp][lane], 1);
    mbar_init(&sm->empty[warp][lane], 1);
  }
  if (threadIdx.x == 0) sm->abort_flag = 0;
  fence_mbar_init();
  find_piece<C::W, C::RT, N>(a, sm->weights, &sm->piece);
  // the join may be set up from here on; it waits for this grid's end itself
  if (a.whole == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Q4Piece piece = sm->piece;

  if (warp == C::W) {
    produce<HD, NT, N>(a, sm, piece);
    if (a.share > 1)                           // as often as the other warps, below
      for (int i = 0; i < 2 * NT; ++i) cluster_sync();
  } else {
    Walk* walk = &sm->walk[warp];
    if (lane == 0) walk->start(a, piece);
    __syncwarp();
    Rows<HD, NT> rows;
    const Item& it = sm->item[warp];
    const Layout lay = layout_of<HD>(a);
    uint32_t stage = 0, parity = 0;
    float* steps = &sm->part[warp][0][0];      // free until the unit's end
    while (next_item<C::W, C::RT>(a, walk, &sm->item[warp])) {
      rows.start(a, it, sm);
      // keys that every row sees
      int lo, hi, x;
      const int last = it.rt * C::RT + it.rows - 1;
      keys_of(a, it.len, it.len - it.q_len + a.row_token(it.rt * C::RT), &x, &hi);
      keys_of(a, it.len, it.len - it.q_len + a.row_token(last), &lo, &x);
#pragma unroll 1
      for (int t = first_tile<C::W>(a, it) + warp; t < it.s1; t += C::W * a.share) {
        // (a wait that runs out is recorded, and the rows' values are wrong)
        mbar_wait(&sm->full[warp][stage], parity, &sm->abort_flag, &g_attn_q4_err, ERR_TIMEOUT_OTHER);
        __syncwarp();
        const int pos = t * kTile;
        rows.tile(a, it, sm, sm->stage[warp][stage][0], sm->stage[warp][stage][1], lay, steps, pos,
                  pos < lo || pos + kTile > hi);
        __syncwarp();                          // the stage has been read
        if (lane == 0) mbar_arrive(&sm->empty[warp][stage]);
        if (++stage == C::kStages) {
          stage = 0;
          parity ^= 1u;
        }
      }
      finish<HD, NT, N>(a, it, sm, rows);
      if (it.behind > 0 && threadIdx.x == 0)   // the CTAs behind have a whole piece each
        a.joins[blockIdx.x] = {a.segs[it.seg].q_row0, it.rt * C::RT, it.rows, it.hk,
                               static_cast<int32_t>(blockIdx.x + div_nonneg(it.behind + piece.per - 1, piece.per))};
    }
  }
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&sm->abort_flag)) {       // copies may still be on their way
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
}

// ------------------------------------------------------------------ joining the cut units
//     lse = log sum_i exp(lse_i),  o = sum_i exp(lse_i - lse) o_i
// over a row's parts in the CTAs from c to joins[c].last.  A warp takes a row of
// few parts; of many, the block's warps take its parts in turn.
constexpr int kJoinThreads = 256;
constexpr int kFewParts = 8;

template <int HD>
struct Acc {
  static constexpr int C = HD / 32;
  float x[C];
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (C == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(p);
    else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(p);
  }
};

template <int HD>
__device__ __forceinline__ void put_joined(const AttnQ4Head& a, const Q4Join& j, int r, const float (&x)[HD / 32], float inv,
                                        float lse) {
  const int lane = threadIdx.x & 31;
  const int row = j.row0 + r, tok = a.row_token(row), h = j.hk * a.group + row - tok * a.group;
  const int64_t q_row = j.q_row0 + static_cast<int64_t>(tok);
  __nv_bfloat16* dst = a.o + (q_row * a.num_heads + h) * HD + lane * (HD / 32);
  if constexpr (HD == 128)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(x[0] * inv, x[1] * inv);
  if (lane == 0) a.lse[h * a.lse_stride + q_row] = lse;
}

template <int HD>
__global__ void __launch_bounds__(kJoinThreads) join_q4_kernel(const __grid_constant__ AttnQ4Head a, int slot_rows) {
  constexpr int C = HD / 32, kWarps = kJoinThreads / 32;
  __shared__ float sum_o[kWarps][HD], sum_l[kWarps], max_l[kWarps];
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Q4Join j = a.joins[c];
  if (j.last < 0) return;
  const int n = j.last - c + 1;
  const auto part = [&](int i, int r) { return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_rows + r; };
  const bool few = n <= kFewParts;
  const int step = few ? 1 : kWarps, first = few ? 0 : warp;
  for (int r = few ? blockIdx.y * kWarps + warp : blockIdx.y; r < j.rows; r += few ? gridDim.y * kWarps : gridDim.y) {
    // the lanes take the parts' lse, then the warp goes through its parts
    float m = -INFINITY, sum = 0.f;
    Acc<HD> acc;
#pragma unroll
    for (int k = 0; k < C; ++k) acc.x[k] = 0.f;
    for (int i0 = first; i0 < n; i0 += 32 * step) {
      const int mine = i0 + lane * step;
      const float lse = mine < n ? a.lse_part[part(mine, r)] : -INFINITY;
      float top = lse;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float to = fmaxf(m, top);
      const float old = m == -INFINITY ? 0.f : expf(m - to);
      const float wgt = lse == -INFINITY ? 0.f : expf(lse - (to == -INFINITY ? 0.f : to));
      m = to;
      float s = wgt;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      sum = sum * old + s;
#pragma unroll
      for (int k = 0; k < C; ++k) acc.x[k] *= old;
      const int count = min(32, (n - i0 + step - 1) / step);
      for (int u0 = 0; u0 < count; u0 += 8) {
        Acc<HD> x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          x[u].load(a.o_part + part(i0 + min(u0 + u, count - 1) * step, r) * HD + lane * C);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float f = __shfl_sync(0xffffffffu, wgt, (u0 + u) & 31);
          if (u0 + u >= count || f == 0.f) continue;
#pragma unroll
          for (int k = 0; k < C; ++k) acc.x[k] = fmaf(f, x[u].x[k], acc.x[k]);
        }
      }
    }
    if (!few) {
      __syncthreads();                         // the row before has read its sums
#pragma unroll
      for (int k = 0; k < C; ++k) sum_o[warp][lane * C + k] = acc.x[k];
      if (lane == 0) {
        sum_l[warp] = sum;
        max_l[warp] = m;
      }
      __syncthreads();
      if (warp > 0) continue;
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, max_l[w]);
      sum = 0.f;
#pragma unroll
      for (int k = 0; k < C; ++k) acc.x[k] = 0.f;
      for (int w = 0; w < kWarps; ++w) {
        const float f = max_l[w] == -INFINITY ? (sum_l[w] != 0.f ? 1.f : 0.f) : expf(max_l[w] - m);
        sum = fmaf(f, sum_l[w], sum);
#pragma unroll
        for (int k = 0; k < C; ++k) acc.x[k] = fmaf(f, sum_o[w][lane * C + k], acc.x[k]);
      }
    }
    const bool seen = sum != 0.f;              // (a NaN is handed on)
    put_joined<HD>(a, j, r, acc.x, seen ? 1.f / sum : 0.f, seen ? (m == -INFINITY ? 0.f : m) + logf(sum) : -INFINITY);
  }
}

template <int N>
AttnQ4Args<N> cut(const AttnQ4Args<kMaxSegs>& a) {
  AttnQ4Args<N> r;
  static_cast<AttnQ4Head&>(r) = a;
  for (int i = 0; i < a.n_segs; ++i) r.segs[i] = a.segs[i];
  return r;
}

template <int HD, int NT, int N>
cudaError_t launch_kind(const AttnQ4Args<N>& a, cudaStream_t stream) {
  using C = Cfg<HD, NT>;
  constexpr size_t smem = sizeof(Smem<HD, NT>);
  static_assert(smem * C::kCtasPerSm <= 226 * 1024, "shared memory of an SM");
  // once per device
  static std::atomic<uint64_t> done[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<uint64_t>& word = done[(dev >> 6) & 1];
  if (!(word.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(paged_attn_q4_kernel<HD, NT, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    word.fetch_or(uint64_t(1) << (dev & 63));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.whole > 0 ? a.whole * a.share : attn_q4_ctas());
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.share;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.share > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_attn_q4_kernel<HD, NT, N>, a);
}

template <int HD, int NT>
cudaError_t launch_segs(const AttnQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  return a.n_segs <= kFewSegs ? launch_kind<HD, NT, kFewSegs>(cut<kFewSegs>(a), stream)
                              : launch_kind<HD, NT, kMaxSegs>(a, stream);
}

template <int HD>
cudaError_t launch_tiles(int nt, const AttnQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  return nt == 1 ? launch_segs<HD, 1>(a, stream) : launch_segs<HD, 2>(a, stream);
}

}  // namespace

int attn_q4_ctas() { return kPagedCtas * Cfg<128, 1>::kCtasPerSm; }

cudaError_t launch_attn_q4(int head_dim, int nt, const AttnQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  return head_dim == 64 ? launch_tiles<64>(nt, a, stream) : launch_tiles<128>(nt, a, stream);
}

// Its launch overlaps the attention's last CTAs (programmatic dependent launch).
cudaError_t launch_join_q4(int head_dim, int nt, const AttnQ4Head& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attn_q4_ctas(), nt == 1 ? 4 : 8);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return head_dim == 64 ? cudaLaunchKernelEx(&cfg, join_q4_kernel<64>, a, 8 * nt)
                        : cudaLaunchKernelEx(&cfg, join_q4_kernel<128>, a, 8 * nt);
}

uint32_t attn_q4_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_q4_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_attn_q4_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
