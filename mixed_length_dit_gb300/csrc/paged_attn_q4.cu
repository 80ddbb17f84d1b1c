// Attention of few rows (single tokens, drafts) over a paged cache held in 4
// bits.
//
//     S = q K^T scale,  o = softmax(S) V,   K = c_k s_k,  V = c_v s_v
//
// with a step s for every 32 columns (a group) of a token's head.  The codes are
// not made into bf16 values: a code n = c + 8 becomes the bf16 128 + n by one
// logical operation (its last four bits), and the products go
//
//     S = scale sum_g s_k[g] (sum_(i in g) q_i (128 + n_i) - 136 sum_(i in g) q_i)
//     o_i = sum_j (p_j s_v[j, g]) ((128 + n_ji) - 136)
//
// so that a key's steps multiply four sums instead of 128 codes, and a value's
// steps the probability before it is rounded to bf16 (the one rounding, as in the
// bf16 attention: the tensor cores take P in V's type).
//
// Bound by HBM at best, by instructions otherwise: an SM's share of HBM is 43
// codes a clock.  So K and V are the A operands of warp-level products
// (mma.m16n8k16: 16 keys, or 16 columns, by the 8 rows of a query tile by 16),
// unpacked in registers where they are used.  The 5th-generation tensor cores
// take B from shared memory only, and A from there or from TMEM: unpacked codes
// would cross shared memory twice, 170 bytes a clock of its 128.
//
// A unit is (sequence, key head, tile of 8 NT rows: queries times the heads that
// share the key head).  The tiles of 32 keys of all units stand in one line that
// is cut into equal pieces, one a CTA, as in the bf16 attention; the warps of a
// CTA take a unit's tiles in turn, each with copies (TMA bulk) of its own in
// flight, and are joined in shared memory; units that a cut goes through are
// joined by a second launch.
#include <algorithm>
#include <atomic>

#include "paged.h"
#include "paged_q4.cuh"

namespace zl {
namespace {

__device__ uint32_t g_attn_q4_err;

constexpr int kTile = 32;                      // keys of a warp's step
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;                // the running maximum lags by this much (base 2) at most
constexpr uint32_t kMagic = 0x43004300u;       // 128 as bf16, twice

template <int HD, int NT>
struct Cfg {
  static constexpr int G = HD / kQ4Group;
  static constexpr int RT = 8 * NT;            // rows of a unit
  static constexpr int W = 8;                  // warps of a CTA
  static constexpr int kCtasPerSm = NT == 1 ? 2 : 1;
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kRegion = kTile * kQ4Row<HD>;           // keys, or values, of a stage
  static constexpr bool kQInSmem = NT > 2;
  static constexpr int kPad = HD + 4;          // floats of a row to be joined (rows 2c of four lanes in different banks)
};

template <int HD, int NT>
struct Smem {
  using C = Cfg<HD, NT>;
  alignas(128) uint8_t stage[C::W][C::kStages][2][C::kRegion];
  alignas(16) float part[C::W][8][C::kPad];    // 8 rows of every warp
  float m[C::W][C::RT], l[C::W][C::RT];
  uint2 q[C::kQInSmem ? C::W : 1][C::kQInSmem ? NT : 1][C::G][2][32];
  float2 q_sum[C::kQInSmem ? C::W : 1][C::kQInSmem ? NT : 1][C::G][4];
  alignas(8) uint64_t full[C::W][C::kStages];
  int64_t sums[32];
  Q4Piece piece;
  int abort_flag;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint2& b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes j and j + 4 of a word, as 128 + n each.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int j) { return ((w >> (4 * j)) & 0x000f000fu) | kMagic; }

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

// The steps of a token's groups.
template <int G>
__device__ __forceinline__ void load_steps(const uint8_t* p, float (&s)[G]) {
  uint32_t w;
  if constexpr (G == 4) w = *reinterpret_cast<const uint32_t*>(p);
  else w = *reinterpret_cast<const uint16_t*>(p);
  const float2 a = q4_steps01(w);
  s[0] = a.x;
  s[1] = a.y;
  if constexpr (G == 4) {
    const float2 b = q4_steps23(w);
    s[2] = b.x;
    s[3] = b.y;
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
  keys_of(a, len, len - q_len + r0 / a.group, &lo, &x);
  keys_of(a, len, len - q_len + (r1 - 1) / a.group, &x, &hi);
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

constexpr int kUnitCost = 1;
template <int W>
__device__ __forceinline__ int waves_of(Tiles t) { return max(1, (t.t1 - t.t0 + W - 1) / W); }

template <int W, int RT>
__device__ __forceinline__ int unit_weight(const AttnQ4Head& a, int len, int q_len, int rt) {
  const int rows = q_len * a.group;
  return kUnitCost + waves_of<W>(tiles_of(a, len, q_len, rt * RT, min(rows, rt * RT + RT)));
}

// The weight of a segment's row tiles for one key head.
template <int W, int RT>
__device__ __forceinline__ int64_t seg_weight(const AttnQ4Head& a, int len, int q_len) {
  int64_t sum = 0;
  for (int rt = 0; rt < row_tiles<RT>(a, q_len); ++rt) sum += unit_weight<W, RT>(a, len, q_len, rt);
  return sum;
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// The CTA's piece of the line, by warp 0 (all of it; the others wait).
template <int W, int RT, int N>
__device__ void find_piece(const AttnQ4Args<N>& a, Q4Piece* out) {
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x, nk = a.num_kv_heads;
  Q4Piece p = {0, 0, 0, 0, 0, 0, 0};
  if (a.whole > 0) {                           // few short units: each CTA has one to itself
    int x = c;
    for (;; ++p.seg) {
      const int units = row_tiles<RT>(a, a.segs[p.seg].q_len) * nk;
      if (x < units) break;
      x -= units;
    }
    const int rts = row_tiles<RT>(a, a.segs[p.seg].q_len);
    p.hk = x / rts;
    p.rt = x - p.hk * rts;
    p.end = 1;                                 // any piece ends within its first unit
    p.per = 0;
    if (lane == 0) *out = p;
    return;
  }
  int64_t total = 0;
  for (int s = lane; s < a.n_segs; s += 32) total += seg_weight<W, RT>(a, length_of(a, s), a.segs[s].q_len);
  total = warp_sum(total) * nk;
  p.per = max(int64_t(1 + kUnitCost), (total + gridDim.x - 1) / gridDim.x);
  p.g = c * p.per;
  p.end = min(total, p.g + p.per);
  if (p.g < p.end) {
    int64_t base = 0;
    for (int chunk = 0;; chunk += 32) {
      int64_t w = 0;
      if (chunk + lane < a.n_segs) w = seg_weight<W, RT>(a, length_of(a, chunk + lane), a.segs[chunk + lane].q_len);
      int64_t incl = w * nk;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      incl += base;
      const uint32_t past = __ballot_sync(0xffffffffu, incl > p.g);
      if (past != 0) {
        const int k = __ffs(past) - 1;
        const int64_t one = __shfl_sync(0xffffffffu, w, k);
        p.seg = chunk + k;
        p.off = p.g - (__shfl_sync(0xffffffffu, incl, k) - one * nk);
        p.hk = static_cast<int>(p.off / one);
        p.off -= p.hk * one;
        break;
      }
      base = __shfl_sync(0xffffffffu, incl, 31);
    }
    const int len = length_of(a, p.seg), q_len = a.segs[p.seg].q_len;
    for (;; ++p.rt) {
      const int w = unit_weight<W, RT>(a, len, q_len, p.rt);
      if (p.off < w) break;
      p.off -= w;
    }
  }
  if (lane == 0) *out = p;
}

// One item: the tiles [s0, s1) of a unit that the CTA has.
struct Item {
  int seg, hk, rt;
  int len, q_len, rows;                        // rows of the unit
  int s0, s1;
  int slot;                                    // slot of partial rows; -1: the rows are final
  bool first;                                  // slot >= 0: the unit begins here
  int64_t behind;                              // and where the line's next unit begins
};

// Walks a CTA's items; every warp for itself, once for its copies and once for
// its products.
template <int W, int RT, int N>
struct Walk {
  int seg, hk, rt;
  int64_t off, g, end;
  int len, q_len;

  __device__ __forceinline__ void start(const AttnQ4Args<N>& a, const Q4Piece& p) {
    seg = p.seg; hk = p.hk; rt = p.rt; off = p.off; g = p.g; end = p.end;
    if (g < end) {
      len = length_of(a, seg);
      q_len = a.segs[seg].q_len;
    }
  }

  // The next item; false: none left.
  __device__ __forceinline__ bool next(const AttnQ4Args<N>& a, Item* it) {
    while (g < end) {
      const int rows = q_len * a.group, r0 = rt * RT;
      it->seg = seg; it->hk = hk; it->rt = rt;
      it->len = len; it->q_len = q_len;
      it->rows = min(RT, rows - r0);
      const Tiles t = tiles_of(a, len, q_len, r0, r0 + it->rows);
      it->s0 = t.t0;
      it->s1 = t.t1;
      it->slot = -1;
      if (a.whole > 0) {
        g = end;
        return true;
      }
      const int waves = waves_of<W>(t);
      const int64_t avail = min(kUnitCost + waves - off, end - g);
      const int w0 = static_cast<int>(max(off - kUnitCost, int64_t(0)));       // the piece's waves of the unit
      const int w1 = static_cast<int>(max(off + avail - kUnitCost, int64_t(0)));
      it->behind = g - off + kUnitCost + waves;
      if (w1 - w0 < waves) {
        it->first = w0 == 0;
        it->slot = it->first ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
        it->s0 = t.t0 + w0 * W;
        it->s1 = min(t.t1, t.t0 + w1 * W);
      }
      g += avail;
      off = 0;
      if (++rt >= row_tiles<RT>(a, q_len)) {
        rt = 0;
        if (++hk >= a.num_kv_heads) {
          hk = 0;
          ++seg;
          if (g < end) {
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

// A warp's tiles, one after another: a copy is set off as soon as a stage is free,
// with the page number that was fetched when the one before was.
template <int HD, int NT, int N>
struct Loader {
  using C = Cfg<HD, NT>;
  Walk<C::W, C::RT, N> walk;
  Item it;
  int tile;                                    // of the item; >= it.s1: none left
  int page;                                    // lane's page number of that tile
  uint32_t stage = 0;

  __device__ __forceinline__ void settle(const AttnQ4Args<N>& a) {
    while (tile >= it.s1) {
      if (!walk.next(a, &it)) return;
      tile = it.s0 + (threadIdx.x >> 5);
    }
    const int lane = threadIdx.x & 31;
    const int pos = tile * kTile + (a.page_shift == 4 ? (lane & 1) * 16 : 0);
    page = -1;
    if (lane < 4 && pos < it.len && (pos >> a.page_shift) < a.table_cols)
      page = __ldg(a.page_table + static_cast<int64_t>(a.segs[it.seg].seq) * a.table_cols + (pos >> a.page_shift));
  }

  __device__ __forceinline__ void start(const AttnQ4Args<N>& a, const Q4Piece& p) {
    walk.start(a, p);
    it.s1 = 0;
    tile = 0;
    settle(a);
  }

  // Lanes 0-3: keys' codes and steps, values' codes and steps (pages of 16: the
  // first and second page of each; of 32: one copy of each).
  __device__ __forceinline__ void issue(const AttnQ4Args<N>& a, Smem<HD, NT>* sm) {
    if (tile >= it.s1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = lane & 1, ps = 1 << a.page_shift;
    const int pos = tile * kTile;
    uint64_t* bar = &sm->full[warp][stage];
    uint32_t bytes = 0, from = 0, to = 0;
    if (a.page_shift == 4) {
      if (lane < 4 && pos + 16 * part < it.len) bytes = 16 * kQ4Row<HD>;
      to = part * 16 * kQ4Row<HD>;
    } else if (a.page_shift == 5) {
      if (lane < 4 && part == 0) bytes = kTile * kQ4Row<HD>;
    } else if (lane < 4) {
      const int row = pos & (ps - 1);
      bytes = part ? kTile * kQ4Steps<HD> : kTile * kQ4Codes<HD>;
      from = part ? ps * kQ4Codes<HD> + row * kQ4Steps<HD> : row * kQ4Codes<HD>;
      to = part ? kTile * kQ4Codes<HD> : 0;
    }
    int pg = page;
    if (bytes > 0 && (pg < 0 || pg >= a.num_pages)) {
      atomicOr(&g_attn_q4_err, ERR_BAD_PAGE);  // reads page 0 in its place
      pg = 0;
    }
    const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) mbar_arrive_expect_tx(bar, all);
    __syncwarp();
    if (bytes > 0) {
      const int64_t block = static_cast<int64_t>(pg) * a.num_kv_heads + it.hk;
      const uint8_t* src = (lane < 2 ? a.k_pages : a.v_pages) + ((block * kQ4Row<HD>) << a.page_shift) + from;
      bulk_load(smem_u32(sm->stage[warp][stage][lane >> 1]) + to, src, bytes, bar);
    }
    if (++stage == C::kStages) stage = 0;
    tile += C::W;
    settle(a);
  }
};

// ------------------------------------------------------------------ products
// A warp's share of a unit: lane (g, c) = (lane / 4, lane % 4) of the products'
// fragments.  Scores are S^T (keys g, g + 8 by rows 2c, 2c + 1), the output o^T
// (columns 32 q + 4 g + (0 .. 3) by rows 2c, 2c + 1).
template <int HD, int NT>
struct Rows {
  using C = Cfg<HD, NT>;
  static constexpr int G = C::G;
  float o[NT][G][2][4];                        // [tile of 16 columns][fragment]
  float m[NT][2], l[NT][2];                    // of rows 2c, 2c + 1; l: the lane's keys alone
  uint2 q[C::kQInSmem ? 1 : NT][G][2];         // fragments of q^T
  float q_sum[C::kQInSmem ? 1 : NT][G][2];     // -136 times the sum of a group's q

  template <int N>
  __device__ __forceinline__ void start(const AttnQ4Args<N>& a, const Item& it, Smem<HD, NT>* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
      const int row = it.rt * C::RT + r, tok = row / a.group;
      const __nv_bfloat16* src = a.q + (a.segs[it.seg].q_row0 + static_cast<int64_t>(tok)) * a.q_stride +
                                 (it.hk * a.group + row - tok * a.group) * HD + 8 * c;
#pragma unroll
      for (int x = 0; x < G; ++x) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (r < it.rows) u = __ldg(reinterpret_cast<const uint4*>(src + 32 * x));
        // columns j and j + 4 of the 8 beside one another, as a word's codes are taken
        const uint2 b0 = make_uint2(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632));
        const uint2 b1 = make_uint2(__byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
        float2 f = bf16x2_to_float2(u.x);
        float sum = f.x + f.y;
        f = bf16x2_to_float2(u.y); sum += f.x + f.y;
        f = bf16x2_to_float2(u.z); sum += f.x + f.y;
        f = bf16x2_to_float2(u.w); sum += f.x + f.y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -136.f;
        const float s0 = __shfl_sync(0xffffffffu, sum, 8 * c), s1 = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
        if constexpr (C::kQInSmem) {
          sm->q[warp][n][x][0][lane] = b0;
          sm->q[warp][n][x][1][lane] = b1;
          if (g == 0) sm->q_sum[warp][n][x][c] = make_float2(s0, s1);
        } else {
          q[n][x][0] = b0;
          q[n][x][1] = b1;
          q_sum[n][x][0] = s0;
          q_sum[n][x][1] = s1;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][x][t][i] = 0.f;
      }
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    __syncwarp();
  }

  // A tile of 32 keys from position `pos` on.  EDGE: some row does not see all of them.
  template <bool EDGE>
  __device__ __forceinline__ void tile(const AttnQ4Head& a, const Item& it, const Smem<HD, NT>* sm, const uint8_t* kr,
                                       const uint8_t* vr, const Layout& lay, int pos) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {              // 16 keys
      uint32_t wa[G], wb[G];
      float sa[G], sb[G];
      const uint8_t* codes = kr + h * lay.codes_half + c * (4 * G);
      load_words<G>(codes + g * kQ4Codes<HD>, wa);
      load_words<G>(codes + (g + 8) * kQ4Codes<HD>, wb);
      const uint8_t* steps = kr + lay.steps + h * lay.steps_half;
      load_steps<G>(steps + g * G, sa);
      load_steps<G>(steps + (g + 8) * G, sb);
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const uint32_t a0[4] = {pair_of(wa[x], 0), pair_of(wb[x], 0), pair_of(wa[x], 1), pair_of(wb[x], 1)};
        const uint32_t a1[4] = {pair_of(wa[x], 2), pair_of(wb[x], 2), pair_of(wa[x], 3), pair_of(wb[x], 3)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float s0, s1;
          uint2 b0, b1;
          if constexpr (C::kQInSmem) {
            const float2 f = sm->q_sum[warp][n][x][c];
            s0 = f.x;
            s1 = f.y;
            b0 = sm->q[warp][n][x][0][lane];
            b1 = sm->q[warp][n][x][1][lane];
          } else {
            s0 = q_sum[n][x][0];
            s1 = q_sum[n][x][1];
            b0 = q[n][x][0];
            b1 = q[n][x][1];
          }
          float d[4] = {s0, s1, s0, s1};
          mma(d, a0, b0);
          mma(d, a1, b1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float st = i < 2 ? sa[x] : sb[x];
            s[h][n][i] = x == 0 ? st * d[i] : fmaf(st, d[i], s[h][n][i]);
          }
        }
      }
    }
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (EDGE) {
          const int tok = min(it.rt * C::RT + 8 * n + 2 * c + e, it.rt * C::RT + it.rows - 1) / a.group;
          int lo, hi;
          keys_of(a, it.len, it.len - it.q_len + tok, &lo, &hi);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int key = pos + 16 * h + 8 * k + g;
              if (key < lo || key >= hi) s[h][n][2 * k + e] = -INFINITY;
            }
        }
        const float top = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e])) * a.scale_log2;
        raise = raise || top > m[n][e] + kRescale;
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e])) * a.scale_log2;
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
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float neg = m[n][e] == -INFINITY ? 0.f : -m[n][e];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float& p = s[h][n][2 * k + e];
            p = fast_exp2(fmaf(p, a.scale_log2, neg));
            l[n][e] += p;
          }
      }
    const __nv_bfloat162 off = __float2bfloat162_rn(136.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the codes of keys 2c, 2c + 1 and 2c + 8, 2c + 9: four columns of each group
      uint32_t w[4][G / 2];
      const uint8_t* codes = vr + h * lay.codes_half + g * (2 * G);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* p = codes + (2 * c + (k & 1) + 8 * (k >> 1)) * kQ4Codes<HD>;
        if constexpr (G == 4) {
          const uint2 u = *reinterpret_cast<const uint2*>(p);
          w[k][0] = u.x;
          w[k][1] = u.y;
        } else {
          w[k][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
      float sa[G], sb[G];
      const uint8_t* steps = vr + lay.steps + h * lay.steps_half;
      load_steps<G>(steps + g * G, sa);
      load_steps<G>(steps + (g + 8) * G, sb);
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const uint32_t sel = x & 1 ? 0x7632 : 0x5410;
        const uint32_t u = __byte_perm(w[0][x / 2], w[1][x / 2], sel), v = __byte_perm(w[2][x / 2], w[3][x / 2], sel);
        uint2 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float st = i < 2 ? sa[x] : sb[x];
            // a key that is not seen may have any step
            t[i] = EDGE && s[h][n][i] == 0.f ? 0.f : s[h][n][i] * st;
          }
          b[n] = make_uint2(transpose8(pack_bf16x2(t[0], t[1])), transpose8(pack_bf16x2(t[2], t[3])));
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t f[4] = {pair_of(u, 2 * t), pair_of(u, 2 * t + 1), pair_of(v, 2 * t), pair_of(v, 2 * t + 1)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 z = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&f[i]), off);
            f[i] = *reinterpret_cast<const uint32_t*>(&z);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(o[n][x][t], f, b[n]);
        }
      }
    }
  }
};

// Joins the warps' shares of an item and writes its rows.
template <int HD, int NT, int N>
__device__ __forceinline__ void finish(const AttnQ4Args<N>& a, const Item& it, Smem<HD, NT>* sm, Rows<HD, NT>& r) {
  using C = Cfg<HD, NT>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int n_warps = min(C::W, max(1, it.s1 - it.s0));        // the others had no tile
#pragma unroll
  for (int n = 0; n < NT; ++n) {
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
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (warp < n_warps) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 0; x < C::G; ++x)
          *reinterpret_cast<float4*>(&sm->part[warp][2 * c + e][32 * x + 4 * g]) =
              make_float4(r.o[n][x][0][e], r.o[n][x][0][2 + e], r.o[n][x][1][e], r.o[n][x][1][2 + e]);
    }
    __syncthreads();
    constexpr int F4 = HD / 4;
    for (int y = threadIdx.x; y < 8 * F4; y += 32 * C::W) {
      const int k = y / F4, col = 4 * (y % F4), i = 8 * n + k;
      if (i >= it.rows) break;                 // rows come in order
      float top = -INFINITY;
      for (int w = 0; w < n_warps; ++w) top = fmaxf(top, sm->m[w][i]);
      const float ref = top == -INFINITY ? 0.f : top;
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < n_warps; ++w) {
        const float f = fast_exp2(sm->m[w][i] - ref);          // 0 for a warp that has seen no key
        const float4 u = *reinterpret_cast<const float4*>(&sm->part[w][k][col]);
        l = fmaf(f, sm->l[w][i], l);
        o.x = fmaf(f, u.x, o.x);
        o.y = fmaf(f, u.y, o.y);
        o.z = fmaf(f, u.z, o.z);
        o.w = fmaf(f, u.w, o.w);
      }
      const bool seen = l != 0.f;              // (a NaN is handed on)
      const float inv = seen ? 1.f / l : 0.f;
      const float lse = seen ? (ref + log2f(l)) * kLn2 : -INFINITY;
      if (it.slot >= 0) {
        const int64_t at = static_cast<int64_t>(it.slot) * C::RT + i;
        *reinterpret_cast<float4*>(a.o_part + at * HD + col) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (col == 0) a.lse_part[at] = lse;
      } else {
        const int row = it.rt * C::RT + i, tok = row / a.group, h = it.hk * a.group + row - tok * a.group;
        const int64_t q_row = a.segs[it.seg].q_row0 + static_cast<int64_t>(tok);
        *reinterpret_cast<uint2*>(a.o + (q_row * a.num_heads + h) * HD + col) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (col == 0) a.lse[h * a.lse_stride + q_row] = lse;
      }
    }
    __syncthreads();
  }
}

template <int HD, int NT, int N>
__global__ void __launch_bounds__(32 * Cfg<HD, NT>::W, Cfg<HD, NT>::kCtasPerSm)
paged_attn_q4_kernel(const __grid_constant__ AttnQ4Args<N> a) {
  using C = Cfg<HD, NT>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto* sm = reinterpret_cast<Smem<HD, NT>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.whole == 0 && threadIdx.x == 0) a.joins[blockIdx.x].last = -1;
  if (lane == 0)
    for (int s = 0; s < C::kStages; ++s) mbar_init(&sm->full[warp][s], 1);
  if (threadIdx.x == 0) sm->abort_flag = 0;
  fence_mbar_init();
  if (warp == 0) find_piece<C::W, C::RT, N>(a, &sm->piece);
  // the join may be set up from here on; it waits for this grid's end itself
  if (a.whole == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  const Q4Piece piece = sm->piece;
  const Layout lay = layout_of<HD>(a);

  Loader<HD, NT, N> load;
  load.start(a, piece);
#pragma unroll 1
  for (int s = 0; s < C::kStages; ++s) load.issue(a, sm);

  Walk<C::W, C::RT, N> walk;
  walk.start(a, piece);
  Item it;
  Rows<HD, NT> rows;
  uint32_t stage = 0, parity = 0;
  while (walk.next(a, &it)) {
    rows.start(a, it, sm);
    // keys that every row sees
    int lo, hi, x;
    const int last = it.rt * C::RT + it.rows - 1;
    keys_of(a, it.len, it.len - it.q_len + it.rt * C::RT / a.group, &x, &hi);
    keys_of(a, it.len, it.len - it.q_len + last / a.group, &lo, &x);
#pragma unroll 1
    for (int t = it.s0 + warp; t < it.s1; t += C::W) {
      // (a wait that runs out is recorded, and the rows' values are wrong)
      mbar_wait(&sm->full[warp][stage], parity, &sm->abort_flag, &g_attn_q4_err, ERR_TIMEOUT_OTHER);
      __syncwarp();
      const uint8_t* kr = sm->stage[warp][stage][0];
      const uint8_t* vr = sm->stage[warp][stage][1];
      const int pos = t * kTile;
      if (pos >= lo && pos + kTile <= hi) rows.template tile<false>(a, it, sm, kr, vr, lay, pos);
      else rows.template tile<true>(a, it, sm, kr, vr, lay, pos);
      __syncwarp();                            // the stage has been read
      load.issue(a, sm);
      if (++stage == C::kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }
    finish<HD, NT, N>(a, it, sm, rows);
    if (it.slot >= 0 && it.first && threadIdx.x == 0)
      a.joins[blockIdx.x] = {a.segs[it.seg].q_row0, it.rt * C::RT, it.rows, it.hk,
                             static_cast<int32_t>((it.behind - 1) / piece.per)};
  }
  // after a wait that ran out, copies may still be on their way
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&sm->abort_flag)) {
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
__device__ __forceinline__ void put_row(const AttnQ4Head& a, const Q4Join& j, int r, const float (&x)[HD / 32], float inv,
                                        float lse) {
  const int lane = threadIdx.x & 31;
  const int row = j.row0 + r, tok = row / a.group, h = j.hk * a.group + row - tok * a.group;
  const int64_t q_row = j.q_row0 + static_cast<int64_t>(tok);
  __nv_bfloat16* dst = a.o + (q_row * a.num_heads + h) * HD + lane * (HD / 32);
  if constexpr (HD == 128)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(x[0] * inv, x[1] * inv);
  if (lane == 0) a.lse[h * a.lse_stride + q_row] = lse;
}

// The weights exp2((lse - m) / ln 2) of parts first, first + by, ... below n, and their rows' sum.
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
    put_row<HD>(a, j, r, acc.x, seen ? 1.f / sum : 0.f, seen ? (m == -INFINITY ? 0.f : m) + logf(sum) : -INFINITY);
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
  paged_attn_q4_kernel<HD, NT, N><<<a.whole > 0 ? a.whole : attn_q4_ctas(NT), 32 * C::W, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int HD, int NT>
cudaError_t launch_segs(const AttnQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  return a.n_segs <= kFewSegs ? launch_kind<HD, NT, kFewSegs>(cut<kFewSegs>(a), stream)
                              : launch_kind<HD, NT, kMaxSegs>(a, stream);
}

template <int HD>
cudaError_t launch_tiles(int nt, const AttnQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  return nt == 1 ? launch_segs<HD, 1>(a, stream) : nt == 2 ? launch_segs<HD, 2>(a, stream) : launch_segs<HD, 4>(a, stream);
}

}  // namespace

int attn_q4_ctas(int nt) { return kPagedCtas * (nt == 1 ? Cfg<128, 1>::kCtasPerSm : Cfg<128, 2>::kCtasPerSm); }

cudaError_t launch_attn_q4(int head_dim, int nt, const AttnQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  return head_dim == 64 ? launch_tiles<64>(nt, a, stream) : launch_tiles<128>(nt, a, stream);
}

// Its launch overlaps the attention's last CTAs (programmatic dependent launch).
cudaError_t launch_join_q4(int head_dim, int nt, const AttnQ4Head& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attn_q4_ctas(nt), nt == 1 ? 4 : 8);
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
