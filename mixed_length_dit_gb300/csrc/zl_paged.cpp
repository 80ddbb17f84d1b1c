// Host side of rotary positions and the paged key/value cache: argument checks
// and kernel launches behind the zl_rope_*, zl_paged_* and zl_pages_* entries
// of include/zl_attn.h.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "host.h"
#include "paged.h"
#include "zl_attn.h"

namespace {

using zl::aligned16;
using zl::device_sms;
using zl::launch_counted;
using RopeArgs = zl::RopeArgs<zl::kMaxSegs>;

bool page_size_ok(int32_t p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }

int shift_of(int32_t p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// A plan as zl_rope_init leaves it (a caller's struct is read by the kernel).
bool plan_ok(const zl_rope_t& p) {
  if (p.head_dim != 64 && p.head_dim != 128) return false;
  if (p.rot_dim < 2 || p.rot_dim > p.head_dim || (p.rot_dim & 1)) return false;
  if (p.n_axes < 1 || p.n_axes > ZL_ROPE_MAX_AXES) return false;
  int32_t last = 0;
  for (int32_t a = 0; a < p.n_axes; ++a) {
    if (p.pair_end[a] <= last) return false;
    last = p.pair_end[a];
  }
  return last == p.rot_dim / 2 && std::isfinite(p.magnitude);
}

// A [tokens][heads * d] operand whose tokens are `stride` elements apart.
zl_status check_rows(const void* p, int64_t stride, int32_t heads, int32_t hd, int64_t tokens, int elem) {
  if (!p) return ZL_EINVAL;
  if (stride < int64_t(heads) * hd || stride > (int64_t(1) << 40) / std::max<int64_t>(tokens, 1)) return ZL_EINVAL;
  if (!aligned16(p) || (stride * elem) % 16 != 0) return ZL_EALIGN;
  return ZL_OK;
}

zl_status rope(const zl_rope_t* plan, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
               const int32_t* positions, int64_t pos_stride, int64_t tokens, int32_t nq, int32_t nk, int32_t dtype,
               void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream, bool inverse) {
  if (!plan || !plan_ok(*plan)) return ZL_EINVAL;
  if (dtype != ZL_BF16 && dtype != ZL_FP32) return ZL_EUNSUPPORTED;
  if (tokens < 0 || tokens > zl::kMaxTokens || nq < 1 || nq > 4096 || nk < 0 || nk > 4096) return ZL_EINVAL;
  if (pos_stride < (plan->n_axes > 1 ? tokens : 0)) return ZL_EINVAL;
  if (tokens == 0) return ZL_OK;
  if (!positions) return ZL_EINVAL;
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return ZL_EALIGN;
  const int elem = dtype == ZL_BF16 ? 2 : 4;
  const int32_t hd = plan->head_dim;
  zl_status st = check_rows(q, q_stride, nq, hd, tokens, elem);
  if (st == ZL_OK) st = check_rows(q_out, q_out_stride, nq, hd, tokens, elem);
  if (st == ZL_OK && nk > 0) st = check_rows(k, k_stride, nk, hd, tokens, elem);
  if (st == ZL_OK && nk > 0) st = check_rows(k_out, k_out_stride, nk, hd, tokens, elem);
  if (st != ZL_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  static thread_local RopeArgs a;
  static_cast<zl::RopeHead&>(a) = zl::RopeHead();
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.tokens = tokens;
  a.nq = nq;
  a.nk = nk;
  a.head_dim = hd;
  a.inverse = inverse ? 1 : 0;
  a.elem_bytes = elem;
  a.skip_kept = q == q_out && q_stride == q_out_stride && (nk == 0 || (k == k_out && k_stride == k_out_stride));
  a.rope = *plan;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_counted(inverse ? "rope_bwd" : "rope_fwd", s, [&] { return zl::launch_rope(a, sms, s); });
}

// The checks every call on a cache applies to its description.
zl_status check_cache(const zl_paged_cache_t* c) {
  if (!c || c->reserved != 0) return ZL_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return ZL_EUNSUPPORTED;
  if (!page_size_ok(c->page_size)) return ZL_EUNSUPPORTED;
  if (c->table_cols < 1 || c->num_pages < 1 || c->num_kv_heads < 1 || c->num_kv_heads > 4096) return ZL_EINVAL;
  // rows of a pool are numbered in int32 (the tensor maps' coordinates)
  if (int64_t(c->num_pages) * c->num_kv_heads * c->page_size > INT32_MAX) return ZL_EINVAL;
  if (int64_t(c->table_cols) * c->page_size > INT32_MAX) return ZL_EINVAL;
  return ZL_OK;
}

zl_status check_cache_pointers(const zl_paged_cache_t* c) {
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->kv_lens) return ZL_EINVAL;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return ZL_EALIGN;
  if ((reinterpret_cast<uintptr_t>(c->page_table) & 3u) || (reinterpret_cast<uintptr_t>(c->kv_lens) & 3u))
    return ZL_EALIGN;
  return ZL_OK;
}

zl_status check_cu(const int32_t* cu, int32_t b, int64_t* total) {
  if (b < 0 || !cu || cu[0] != 0) return ZL_EINVAL;
  for (int32_t s = 0; s < b; ++s)
    if (cu[s + 1] < cu[s]) return ZL_EINVAL;
  *total = cu[b];
  return *total > zl::kMaxTokens ? ZL_EINVAL : ZL_OK;
}

zl_status check_attn(const int32_t* cu_q, int32_t num_seqs, int32_t max_kv_len, int32_t nh, int32_t nk, int32_t hd,
                     int64_t* tq) {
  if (hd != 64 && hd != 128) return ZL_EUNSUPPORTED;
  if (nk < 1 || nh < nk || nh > 4096 || nh % nk != 0) return ZL_EINVAL;
  if (max_kv_len < 0 || max_kv_len > zl::kMaxTokens) return ZL_EINVAL;   // the last block's end stays in int32
  if (nh / nk > zl::kBlockM) return ZL_EUNSUPPORTED;
  const zl_status st = check_cu(cu_q, num_seqs, tq);
  if (st != ZL_OK) return st;
  if ((*tq + zl::kBlockM) * int64_t(nh) * hd > (int64_t(1) << 40)) return ZL_EINVAL;
  return ZL_OK;
}

// ------------------------------------------------------------------ the attention's launches
// A call runs its sequences of one query tile (single tokens, drafts) and its
// longer chunks by two kernels, each as often as its sequences fill launches.
// The kernels split the work on the device; the workspace holds what a cut
// through a unit leaves in every CTA, whatever the lengths and the window.
struct Launch {
  int32_t segs = 0;
  int32_t slot_rows = 0;
};

int32_t tile_tokens(int32_t group) { return zl::kBlockM / group; }

// The sequences of a call that a launch takes: of [first, end) those with more
// than `above` rows (queries times the heads of a key head).
struct Chosen {
  int32_t first, end;
  int64_t above;
};

// The next launch of a kind: as many sequences from *i on as it holds.
Launch next_launch(const int32_t* cu, const Chosen& from, int32_t group, bool pair, int32_t* i) {
  Launch l;
  for (; *i < from.end && l.segs < zl::kMaxSegs; ++*i) {
    const int32_t n = cu[*i + 1] - cu[*i];
    if (n == 0 || int64_t(n) * group <= from.above || (n > tile_tokens(group)) != pair) continue;
    ++l.segs;
    l.slot_rows = pair ? 2 * zl::kBlockM : std::max(l.slot_rows, n * group);
  }
  return l;
}

// The launches run one after another and share the workspace.
size_t attn_workspace(const int32_t* cu, const Chosen& from, int32_t group, int32_t hd) {
  size_t need = 0;
  for (const bool pair : {false, true})
    for (int32_t i = from.first; i < from.end;) {
      const Launch l = next_launch(cu, from, group, pair, &i);
      if (l.segs == 0) continue;
      const size_t rows = static_cast<size_t>(2) * zl::kPagedCtas * l.slot_rows;
      need = std::max(need, zl::kPagedCtas * sizeof(zl::PagedJoin) + rows * (hd + 1) * sizeof(float));
    }
  return need;
}

// The launch's units if each is left whole, one CTA to a unit; 0 if they are cut
// into equal shares.  Whole units do without the sums over all lengths and
// without the join, equal shares finish earlier when there are fewer units than
// SMs or lengths differ.  L key blocks bound a unit (the lengths themselves are
// on the device), half of them is taken for the mean, so a share is about
// `share`; whole is taken while L is at most 4 blocks (chunks: 5), and one for
// every 16 units to be joined, above it.  Measured, whole and cut (us of the
// GPU, a call repeated on the same inputs; d = 128, pages of 64; L = 2, 4, 8, 16,
// every length at its bound):
//   8 units of a token       7.9 10.6    9.8 11.2   13.2 11.7   21.9 13.6
//   32 units of a token      8.0 11.1   10.2 12.7   14.3 14.4   22.0 16.7
//   128 units of 5 rows      8.9 11.9   11.0 14.4   15.0 21.7   27.3 32.2
//   8 units of a chunk      10.1 14.5   13.5 18.5   20.2 18.7   33.5 21.3
//   48 units of a chunk     10.1 14.6   13.6 22.8   20.3 26.5   33.6 30.1
// With pages of 16 a token's whole units are slower (eight boxes to a block), and
// at 32 units and L = 8 the rule takes the slower way:
//   8 units of a token       8.8 11.4   11.4 12.2   17.0 12.1   28.3 13.5
//   32 units of a token      9.0 11.7   12.1 12.7   17.6 14.7   29.1 17.0
//   128 units of 5 rows      9.5 12.3   12.6 15.0   18.1 23.0   30.8 33.7
// It goes by the bound alone: a captured call whose bound is its table's width
// is cut whatever the lengths come to.
int32_t whole_units(const zl::PagedAttnArgs<zl::kMaxSegs>& a, bool pair) {
  const int32_t span = pair ? 2 * a.tile_tokens : a.tile_tokens;     // queries of a unit, at most
  int64_t units = 0;
  for (int32_t i = 0; i < a.n_segs; ++i)
    units += int64_t(pair ? (a.segs[i].q_len + span - 1) / span : 1) * a.num_kv_heads;
  if (units > zl::kPagedCtas || a.n_segs > zl::kFewSegs) return 0;
  int64_t blocks = (int64_t(a.max_kv_len) + zl::kBlockN - 1) / zl::kBlockN;
  if (a.window > 0 && a.causal) blocks = std::min(blocks, (int64_t(a.window) + span) / zl::kBlockN + 2);
  const int64_t share = std::max<int64_t>(2, units * (blocks / 2 + 2) / zl::kPagedCtas);
  return blocks - share <= (pair ? 5 : 4) + units / 16 ? static_cast<int32_t>(units) : 0;
}

zl_status check_tables(const zl_page_tables_t* t, zl::PageTable* out) {
  if (!t) return ZL_EINVAL;
  if (!page_size_ok(t->page_size)) return ZL_EUNSUPPORTED;
  if (t->slots < 1 || t->slots > zl::kMaxSlots || t->table_cols < 1 || t->num_pages < 1) return ZL_EINVAL;
  if (int64_t(t->table_cols) * t->page_size > INT32_MAX) return ZL_EINVAL;
  if (!t->page_table || !t->kv_lens || !t->page_refs) return ZL_EINVAL;
  for (const void* p : {t->page_table, t->kv_lens, t->page_refs})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return ZL_EALIGN;
  *out = zl::PageTable{t->page_table, t->kv_lens, t->page_refs, t->slots,
                       t->table_cols, t->num_pages, shift_of(t->page_size)};
  return ZL_OK;
}

zl_status check_pool(const zl_page_pool_t* p, zl::PagePool* out) {
  if (!p || p->groups < 1 || p->num_pages < 1 || p->page_bytes < 16 || p->page_bytes % 16 != 0) return ZL_EINVAL;
  if (p->page_bytes > (int64_t(1) << 40) / p->num_pages) return ZL_EINVAL;
  if (p->group_stride % 16 != 0 || (p->groups > 1 && p->group_stride < p->page_bytes * p->num_pages)) return ZL_EINVAL;
  if (!p->base) return ZL_EINVAL;
  if (!aligned16(p->base)) return ZL_EALIGN;
  *out = zl::PagePool{static_cast<uint8_t*>(p->base), p->page_bytes, p->group_stride, p->groups, p->num_pages};
  return ZL_OK;
}

zl_status check_workspace(int32_t num_pages, const void* ws, size_t bytes) {
  if (!ws || bytes < zl::pages_workspace_words(num_pages) * sizeof(int32_t)) return ZL_EWORKSPACE;
  return aligned16(ws) ? ZL_OK : ZL_EALIGN;
}

// Appends to a cache in bf16, or in 4 bits.
zl_status append(const zl_paged_cache_t* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 const int32_t* cu_seqlens, int32_t num_seqs, const zl_rope_t* plan, const int32_t* positions,
                 int64_t pos_stride, const void* q, int64_t q_stride, int32_t num_heads, void* q_out,
                 int64_t q_out_stride, const int32_t* status, void* stream, bool q4) {
  zl_status st = check_cache(cache);
  if (st != ZL_OK) return st;
  int64_t tokens = 0;
  st = check_cu(cu_seqlens, num_seqs, &tokens);
  if (st != ZL_OK) return st;
  if (plan && (!plan_ok(*plan) || plan->head_dim != cache->head_dim)) return ZL_EINVAL;
  if (plan && plan->n_axes > 1 && !positions) return ZL_EINVAL;
  if (positions && (!plan || pos_stride < (plan->n_axes > 1 ? tokens : 0))) return ZL_EINVAL;
  if (num_heads < 0 || num_heads > 4096 || (num_heads > 0) != (q != nullptr)) return ZL_EINVAL;
  if (tokens == 0) return ZL_OK;
  st = check_cache_pointers(cache);
  if (st != ZL_OK) return st;
  if (misaligned4(positions) || misaligned4(status)) return ZL_EALIGN;
  const int32_t hd = cache->head_dim;
  st = check_rows(k, k_stride, cache->num_kv_heads, hd, tokens, 2);
  if (st == ZL_OK) st = check_rows(v, v_stride, cache->num_kv_heads, hd, tokens, 2);
  if (st == ZL_OK && q) st = check_rows(q, q_stride, num_heads, hd, tokens, 2);
  if (st == ZL_OK && q) st = check_rows(q_out, q_out_stride, num_heads, hd, tokens, 2);
  if (st != ZL_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  static thread_local RopeArgs a;
  static_cast<zl::RopeHead&>(a) = zl::RopeHead();
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_out = cache->k_pages;
  a.v_out = cache->v_pages;
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.nq = num_heads;
  a.nk = cache->num_kv_heads;
  a.head_dim = hd;
  a.elem_bytes = 2;
  a.append = 1;
  a.skip_kept = q && q == q_out && q_stride == q_out_stride;
  a.page_table = cache->page_table;
  a.kv_lens = cache->kv_lens;
  a.status = status;
  a.table_cols = cache->table_cols;
  a.num_pages = cache->num_pages;
  a.page_shift = shift_of(cache->page_size);
  if (plan) a.rope = *plan;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t s0 = 0; s0 < num_seqs; s0 += zl::kMaxSegs) {
    a.seq0 = s0;
    a.n_seqs = std::min(num_seqs - s0, zl::kMaxSegs);
    for (int32_t i = 0; i <= a.n_seqs; ++i) a.cu[i] = cu_seqlens[s0 + i];
    a.token0 = a.cu[0];
    a.tokens = a.cu[a.n_seqs] - a.cu[0];
    if (a.tokens == 0) continue;
    st = q4 ? launch_counted("paged_append_q4", s, [&] { return zl::launch_append_q4(a, sms, s); })
            : launch_counted("paged_append", s, [&] { return zl::launch_rope(a, sms, s); });
    if (st != ZL_OK) return st;
  }
  return ZL_OK;
}

// The arguments of an attention over a cache, and the checks of a call.
struct Attend {
  const zl_paged_cache_t* cache;
  const void* q;
  int64_t q_stride;
  const int32_t* cu;
  int32_t num_seqs;
  int32_t max_kv_len;
  int32_t num_heads;
  float scale;
  int32_t causal;
  int32_t window;
  void* o;
  float* lse;
  cudaStream_t stream;
  int64_t tq = 0;

  int32_t group() const { return num_heads / cache->num_kv_heads; }
  int32_t queries(int32_t s) const { return cu[s + 1] - cu[s]; }
  zl_status check();
};

zl_status Attend::check() {
  zl_status st = check_cache(cache);
  if (st != ZL_OK) return st;
  st = check_attn(cu, num_seqs, max_kv_len, num_heads, cache->num_kv_heads, cache->head_dim, &tq);
  if (st != ZL_OK) return st;
  if (max_kv_len > int64_t(cache->table_cols) * cache->page_size) return ZL_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ZL_EINVAL;
  if ((causal != 0 && causal != 1) || window < 0) return ZL_EINVAL;
  if (tq == 0) return ZL_OK;
  st = check_cache_pointers(cache);
  if (st != ZL_OK) return st;
  if (!o || !lse) return ZL_EINVAL;
  if (!aligned16(o) || misaligned4(lse)) return ZL_EALIGN;
  return check_rows(q, q_stride, num_heads, cache->head_dim, tq, 2);
}

// The bf16 attention's launches over `cache`, the call's own or one that has been
// unpacked from it.
zl_status launch_attn(const Attend& c, const zl_paged_cache_t& cache, const Chosen& from, void* workspace) {
  const int32_t hd = cache.head_dim, group = c.group();
  cudaStream_t s = c.stream;
  static thread_local zl::PagedAttnArgs<zl::kMaxSegs> a;      // ~21 KB: kept off the stack
  static_cast<zl::PagedAttnHead&>(a) = zl::PagedAttnHead();
  a.page_table = cache.page_table;
  a.kv_lens = cache.kv_lens;
  a.o = c.o;
  a.lse = c.lse;
  a.lse_stride = c.tq;
  a.num_heads = c.num_heads;
  a.num_kv_heads = cache.num_kv_heads;
  a.group = group;
  a.group_inv = (65536 + group - 1) / group;
  a.tile_tokens = tile_tokens(group);
  a.table_cols = cache.table_cols;
  a.num_pages = cache.num_pages;
  a.page_shift = shift_of(cache.page_size);
  a.max_kv_len = c.max_kv_len;
  a.causal = c.causal;
  a.window = c.window < c.max_kv_len ? c.window : 0;   // one that reaches over every key is none (and stays in 32 bits)
  a.scale_log2 = c.scale * 1.4426950408889634f;

  // the maps that the call's kinds of sequences use
  bool copies[3] = {false, false, false}, pairs = false;
  for (int32_t i = from.first; i < from.end; ++i) {
    const int64_t n = c.queries(i);
    if (n == 0 || n * a.group <= from.above) continue;
    pairs = pairs || n > a.tile_tokens;
    const int64_t tile_rows = n * a.group;
    copies[n > a.tile_tokens || tile_rows > 64 ? 0 : tile_rows > 32 ? 1 : 2] = true;
  }
  zl::PagedMaps maps;
  const int64_t pool_rows = int64_t(cache.num_pages) * cache.num_kv_heads * cache.page_size;
  const int box_rows = std::min(cache.page_size, zl::kBlockN);
  bool ok = zl::make_map(&maps.k, cache.k_pages, pool_rows, 1, hd, box_rows) &&
            zl::make_map(&maps.v, cache.v_pages, pool_rows, 1, hd, box_rows);
  if (pairs)
    ok = ok && zl::make_map_heads(&maps.o, c.o, c.tq, c.num_heads, hd, int64_t(c.num_heads) * hd, a.group, a.tile_tokens);
  for (int i = 0; i < 3; ++i)
    if (copies[i])
      ok = ok && zl::make_map_heads(&maps.q[i], c.q, c.tq, c.num_heads, hd, c.q_stride, a.group,
                                    zl::kBlockM / (1 << i) / a.group);
  if (!ok) return ZL_ECUDA;

  a.joins = static_cast<zl::PagedJoin*>(workspace);
  a.o_part = reinterpret_cast<float*>(a.joins + zl::kPagedCtas);
  for (const bool pair : {false, true}) {
    for (int32_t i = from.first; i < from.end;) {
      const int32_t first = i;
      const Launch l = next_launch(c.cu, from, group, pair, &i);
      if (l.segs == 0) continue;
      a.slot_rows = l.slot_rows;
      a.lse_part = a.o_part + int64_t(2) * zl::kPagedCtas * l.slot_rows * hd;
      a.n_segs = 0;
      for (int32_t x = first; x < i; ++x) {
        const int32_t n = c.queries(x);
        if (n > 0 && int64_t(n) * group > from.above && (n > a.tile_tokens) == pair)
          a.segs[a.n_segs++] = zl::PagedSeg{x, c.cu[x], n};
      }
      a.whole = whole_units(a, pair);
      zl_status st = launch_counted("paged_attn", s, [&] { return zl::launch_paged_attn(hd, pair, maps, a, s); });
      if (st != ZL_OK) return st;
      if (a.whole > 0) continue;
      st = launch_counted("paged_join", s, [&] { return zl::launch_paged_join(hd, pair, a, s); });
      if (st != ZL_OK) return st;
    }
  }
  return ZL_OK;
}

// ------------------------------------------------------------------ attention over 4 bits
// Sequences of at most kQ4Rows rows (queries times the heads of a key head) run
// over the codes as they are, a single token of more than 64 heads to a key head not
// among them.  Longer ones are unpacked to bf16, once for all of
// their queries, and handed to the bf16 attention, a batch at a time: as many as
// kScratchBytes hold, or one.
constexpr int64_t kQ4Rows = 64;
static_assert(kQ4Rows < 512, "row_token");
constexpr int64_t kScratchBytes = int64_t(1) << 30;

struct Q4Plan {
  int32_t chunks = 0;      // sequences that are unpacked
  int32_t batch = 0;       // of them at a time
  int32_t seg_pages = 0;   // pages of each
  int32_t cols = 0;        // of the scratch table
  size_t attn = 0;         // bytes of what the attentions leave to their joins
  size_t table = 0;        // bytes of the scratch table
  size_t pool = 0;         // bytes of the scratch keys, and of the values
  size_t bytes() const { return attn + table + 2 * pool; }
};

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The next launch over codes: sequences from *i on, units of nt tiles of 8 rows.  The
// longest sequence decides for all: 47 single tokens and one draft of 15 rows over long
// caches take 169 us, 48 single tokens 117.
struct Few {
  int32_t segs = 0;
  int32_t nt = 1;
  int64_t row_tiles = 0;   // of one key head
};

Few next_few(const int32_t* cu, int32_t num_seqs, int32_t group, int32_t* i) {
  Few f;
  const int32_t first = *i;
  int64_t most = 0;
  for (; *i < num_seqs && f.segs < zl::kMaxSegs; ++*i) {
    const int64_t rows = int64_t(cu[*i + 1] - cu[*i]) * group;
    if (rows == 0 || rows > kQ4Rows) continue;
    ++f.segs;
    most = std::max(most, rows);
  }
  f.nt = most <= 8 ? 1 : 2;
  for (int32_t x = first; x < *i; ++x) {
    const int64_t rows = int64_t(cu[x + 1] - cu[x]) * group;
    if (rows <= kQ4Rows) f.row_tiles += (rows + 8 * f.nt - 1) / (8 * f.nt);
  }
  return f;
}

size_t few_workspace(int32_t nt, int32_t hd) {
  const size_t ctas = zl::attn_q4_ctas();
  return up256(ctas * sizeof(zl::Q4Join)) + 2 * ctas * 8 * nt * (hd + 1) * sizeof(float);
}

// Whether the launch's units are left whole: each has a CTA, or a cluster of up to 8,
// to itself (no sums over the lengths, no join).  Sets whole (0: they are cut into
// equal shares) and share.  Measured (us of the GPU, a call repeated; d = 128, pages
// of 64, every length at its bound): whole with one CTA, whole with clusters, cut
//   keys                  256              512             1024             2048             4096             8192
//   8 units     6.0  6.9  9.1    7.4  7.0  9.5   10.5  7.4 10.7   16.9  8.8 10.5   28.7  9.9 11.4   52.8 12.7 12.7
//   32 units    6.4  7.4  9.9    7.8  7.6 10.0   10.9  8.6 11.0   17.1 10.5 12.6   29.1 12.2 14.4   53.1 16.0 17.1
//   96 units    6.8  8.4 10.9    8.4  9.6 11.5   11.3 11.9 12.4   17.5 16.1 16.3   29.4 24.4 22.2   56.4 42.7 32.9
//   288 units   9.3  9.4 10.7   11.3 11.3 12.7   15.2 15.2 16.7   24.7 24.7 26.1   42.6 42.6 45.9   77.3 77.3 78.9
// A cluster's CTAs need two waves of keys each to gain (eight where they make a second
// CTA on an SM).  The lengths themselves are on the device; half the bound is taken for
// their mean, so that equal shares have units * keys / 2 / ctas, and may begin three
// waves later.  Of the table the rule takes the slower way at 32 units of 4,096 keys
// (cut 14.4, clusters 12.2), at 96 of 1,024 (cut 12.4, whole 11.3) and 2,048 (16.3,
// 16.1), and at 288 of 2,048 and more (cut, 2 to 8% slower); with lengths spread from an
// eighth of the bound to it, cut against whole:  32 units of 4,096 14.8 12.7,  96 of
// 1,024 12.7 10.7,  288 of 2,048 23.0 21.7, but 288 of 4,096 32.8 37.8 and of 8,192 50.6
// 68.4, which is what the cut is for.  It was measured for 8 rows, d = 128 and pages of
// 64 alone; other units go by the same constants.
void whole_q4(zl::AttnQ4Head* a, const Few& f, int ctas) {
  a->whole = 0;
  a->share = 1;
  const int64_t units = f.row_tiles * a->num_kv_heads;
  if (units > ctas) return;
  int64_t keys = a->max_kv_len;
  if (a->window > 0 && a->causal) keys = std::min(keys, int64_t(a->window) + 64);
  const int64_t wave = f.nt == 1 ? 224 : 160;      // keys that a CTA's warps have at a time
  int32_t share = 1;
  while (share < 8 && units * share * 2 <= ctas && keys >= (units * share * 2 <= ctas / 2 ? 2 : 8) * share * wave) share *= 2;
  if (keys / share - units * keys / (2 * ctas) > 3 * wave) return;
  a->whole = static_cast<int32_t>(units);
  a->share = share;
}

zl_status plan_q4(const int32_t* cu, int32_t num_seqs, int32_t max_kv_len, int32_t nh, int32_t nk, int32_t hd,
                  int32_t window, Q4Plan* p) {
  const int32_t group = nh / nk;
  int32_t most = 0;
  for (int32_t i = 0; i < num_seqs; ++i) {
    const int32_t n = cu[i + 1] - cu[i];
    if (int64_t(n) * group <= kQ4Rows) continue;
    ++p->chunks;
    most = std::max(most, n);
  }
  if (p->chunks > 0) {
    const int64_t page = zl::kScratchPage;
    const int64_t cols = (int64_t(max_kv_len) + page - 1) / page;
    int64_t pages = cols;
    if (window > 0) pages = std::min(pages, (int64_t(most) + window) / page + 2);
    pages = std::max<int64_t>(pages, 1);
    if (pages * nk * page > INT32_MAX) return ZL_EUNSUPPORTED;     // the pool's rows are numbered in int32
    const int64_t each = pages * nk * page * hd * 2;               // keys, or values
    p->seg_pages = static_cast<int32_t>(pages);
    p->cols = static_cast<int32_t>(std::max<int64_t>(cols, 1));
    p->batch = static_cast<int32_t>(std::min<int64_t>({kScratchBytes / (2 * each), INT32_MAX / (pages * nk * page),
                                                       zl::kMaxSegs, p->chunks}));
    p->batch = std::max(p->batch, 1);
    p->table = up256(size_t(num_seqs) * p->cols * sizeof(int32_t));
    p->pool = up256(size_t(p->batch) * each);
  }
  p->attn = attn_workspace(cu, Chosen{0, num_seqs, kQ4Rows}, group, hd);
  for (int32_t i = 0; i < num_seqs;) {
    const Few f = next_few(cu, num_seqs, group, &i);
    if (f.segs > 0) p->attn = std::max(p->attn, few_workspace(f.nt, hd));
  }
  p->attn = up256(p->attn);
  return ZL_OK;
}

// The launches over codes.
zl_status launch_few_q4(const Attend& c, void* workspace) {
  const zl_paged_cache_t& cache = *c.cache;
  static thread_local zl::AttnQ4Args<zl::kMaxSegs> a;
  static_cast<zl::AttnQ4Head&>(a) = zl::AttnQ4Head();
  a.q = static_cast<const __nv_bfloat16*>(c.q);
  a.k_pages = static_cast<const uint8_t*>(cache.k_pages);
  a.v_pages = static_cast<const uint8_t*>(cache.v_pages);
  a.page_table = cache.page_table;
  a.kv_lens = cache.kv_lens;
  a.o = static_cast<__nv_bfloat16*>(c.o);
  a.lse = c.lse;
  a.q_stride = c.q_stride;
  a.lse_stride = c.tq;
  a.page_bytes = cache.num_kv_heads * cache.page_size * (cache.head_dim * 17 / 32);   // at most 4096 * 256 * 68
  a.num_heads = c.num_heads;
  a.num_kv_heads = cache.num_kv_heads;
  a.group = c.group();
  a.group_inv = (65536 + a.group - 1) / a.group;
  a.table_cols = cache.table_cols;
  a.num_pages = cache.num_pages;
  a.page_shift = shift_of(cache.page_size);
  a.max_kv_len = c.max_kv_len;
  a.causal = c.causal;
  a.window = c.window < c.max_kv_len ? c.window : 0;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  for (int32_t i = 0; i < c.num_seqs;) {
    const int32_t first = i;
    const Few f = next_few(c.cu, c.num_seqs, a.group, &i);
    if (f.segs == 0) continue;
    a.n_segs = 0;
    for (int32_t x = first; x < i; ++x) {
      const int32_t n = c.queries(x);
      if (n > 0 && int64_t(n) * a.group <= kQ4Rows) a.segs[a.n_segs++] = zl::PagedSeg{x, c.cu[x], n};
    }
    const int ctas = zl::attn_q4_ctas();
    a.joins = static_cast<zl::Q4Join*>(workspace);
    a.o_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up256(ctas * sizeof(zl::Q4Join)));
    a.lse_part = a.o_part + int64_t(2) * ctas * 8 * f.nt * cache.head_dim;
    whole_q4(&a, f, ctas);
    zl_status st = launch_counted("paged_attn_q4", c.stream,
                                  [&] { return zl::launch_attn_q4(cache.head_dim, f.nt, a, c.stream); });
    if (st == ZL_OK && a.whole == 0)
      st = launch_counted("paged_join_q4", c.stream,
                          [&] { return zl::launch_join_q4(cache.head_dim, f.nt, a, c.stream); });
    if (st != ZL_OK) return st;
  }
  return ZL_OK;
}

zl_status launch_attn_q4(const Attend& c, const Q4Plan& p, void* workspace) {
  const zl_paged_cache_t& cache = *c.cache;
  zl_status few = launch_few_q4(c, workspace);
  if (few != ZL_OK || p.chunks == 0) return few;
  auto* at = static_cast<uint8_t*>(workspace) + p.attn;
  zl_paged_cache_t scratch = cache;
  scratch.page_table = reinterpret_cast<int32_t*>(at);
  scratch.k_pages = at + p.table;
  scratch.v_pages = at + p.table + p.pool;
  scratch.table_cols = p.cols;
  scratch.page_size = zl::kScratchPage;
  static thread_local zl::UnpackQ4Args<zl::kMaxSegs> a;
  static_cast<zl::UnpackQ4Head&>(a) = zl::UnpackQ4Head();
  a.k_pages = static_cast<const uint8_t*>(cache.k_pages);
  a.v_pages = static_cast<const uint8_t*>(cache.v_pages);
  a.page_table = cache.page_table;
  a.kv_lens = cache.kv_lens;
  a.k_out = scratch.k_pages;
  a.v_out = scratch.v_pages;
  a.table = reinterpret_cast<int32_t*>(at);
  a.nk = cache.num_kv_heads;
  a.table_cols = cache.table_cols;
  a.num_pages = cache.num_pages;
  a.page_shift = shift_of(cache.page_size);
  a.max_kv_len = c.max_kv_len;
  a.window = c.window < c.max_kv_len ? c.window : 0;
  a.seg_pages = p.seg_pages;
  a.scratch_cols = p.cols;
  for (int32_t i = 0; i < c.num_seqs;) {
    Chosen part{i, i, kQ4Rows};
    a.n_segs = 0;
    for (; i < c.num_seqs; ++i) {
      if (int64_t(c.queries(i)) * c.group() <= kQ4Rows) continue;
      if (a.n_segs == p.batch) break;
      a.segs[a.n_segs++] = zl::PagedSeg{i, c.cu[i], c.queries(i)};
    }
    part.end = i;
    if (a.n_segs == 0) break;
    scratch.num_pages = a.n_segs * p.seg_pages;
    zl_status st = launch_counted("paged_unpack_q4", c.stream,
                                  [&] { return zl::launch_unpack_q4(cache.head_dim, a, c.stream); });
    if (st == ZL_OK) st = launch_attn(c, scratch, part, workspace);
    if (st != ZL_OK) return st;
  }
  return ZL_OK;
}

}  // namespace

namespace zl {

uint32_t paged_take_error() {
  const uint32_t a = rope_take_error();
  const uint32_t b = pages_take_error();
  const uint32_t c = paged_attn_take_error();
  const uint32_t d = pages_q4_take_error();
  const uint32_t e = attn_q4_take_error();
  for (const uint32_t x : {a, b, c, d, e})
    if (x == 0xFFFFFFFFu) return x;
  return a | b | c | d | e;
}

}  // namespace zl

extern "C" {

// ------------------------------------------------------------------ rotary positions
zl_status zl_rope_init(zl_rope_t* plan, int32_t head_dim, int32_t interleaved, int32_t n_axes,
                       const int32_t* axis_dims, double base, double factor, const double* ramp, double magnitude) {
  if (!plan || !axis_dims) return ZL_EINVAL;
  if (head_dim != 64 && head_dim != 128) return ZL_EUNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return ZL_EINVAL;
  if (n_axes < 1 || n_axes > ZL_ROPE_MAX_AXES) return ZL_EINVAL;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor)) return ZL_EINVAL;
  const float m = static_cast<float>(magnitude);     // what the kernels multiply by
  if (!std::isfinite(m) || m == 0.f) return ZL_EINVAL;
  if (ramp) {
    for (int i = 0; i < 3; ++i)
      if (!std::isfinite(ramp[i])) return ZL_EINVAL;
    if (!(ramp[0] >= 0.0) || !(ramp[1] > ramp[0]) || !(ramp[2] > 0.0)) return ZL_EINVAL;
  }
  int64_t rot = 0;
  for (int32_t a = 0; a < n_axes; ++a) {
    if (axis_dims[a] < 2 || (axis_dims[a] & 1)) return ZL_EINVAL;
    rot += axis_dims[a];
  }
  if (rot > head_dim) return ZL_EINVAL;
  zl_rope_t p;
  std::memset(&p, 0, sizeof(p));
  p.head_dim = head_dim;
  p.rot_dim = static_cast<int32_t>(rot);
  p.interleaved = interleaved;
  p.n_axes = n_axes;
  p.magnitude = m;
  const double two_pi = 6.283185307179586476925;
  int32_t pair = 0;
  for (int32_t a = 0; a < n_axes; ++a) {
    for (int32_t j = 0; j < axis_dims[a] / 2; ++j, ++pair) {
      double f = std::pow(base, -2.0 * j / axis_dims[a]);
      if (ramp) {
        const double turns = ramp[2] * f / two_pi;
        const double w = std::min(1.0, std::max(0.0, (turns - ramp[0]) / (ramp[1] - ramp[0])));
        f *= w + (1.0 - w) / factor;
      } else {
        f /= factor;
      }
      if (!std::isfinite(f)) return ZL_EINVAL;         // a factor near zero
      // turns per position, whole turns dropped, as a 64-bit fraction
      double t = f / two_pi;
      t -= std::floor(t);
      const double scaled = std::ldexp(t, 64);
      p.step[pair] = scaled < 18446744073709551615.0 ? static_cast<uint64_t>(scaled) : 0;
    }
    p.pair_end[a] = pair;
  }
  *plan = p;
  return ZL_OK;
}

zl_status zl_rope_fwd(const zl_rope_t* plan, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const int32_t* positions, int64_t pos_stride, int64_t tokens, int32_t num_heads,
                      int32_t num_kv_heads, int32_t dtype, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream) {
  return rope(plan, q, q_stride, k, k_stride, positions, pos_stride, tokens, num_heads, num_kv_heads, dtype, q_out,
              q_out_stride, k_out, k_out_stride, stream, false);
}

zl_status zl_rope_bwd(const zl_rope_t* plan, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const int32_t* positions, int64_t pos_stride, int64_t tokens, int32_t num_heads,
                      int32_t num_kv_heads, int32_t dtype, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream) {
  return rope(plan, q, q_stride, k, k_stride, positions, pos_stride, tokens, num_heads, num_kv_heads, dtype, q_out,
              q_out_stride, k_out, k_out_stride, stream, true);
}

// ------------------------------------------------------------------ append
zl_status zl_paged_append(const zl_paged_cache_t* cache, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* cu_seqlens, int32_t num_seqs, const zl_rope_t* plan,
                          const int32_t* positions, int64_t pos_stride, const void* q, int64_t q_stride,
                          int32_t num_heads, void* q_out, int64_t q_out_stride, void* stream) {
  return zl_paged_append_ex(cache, k, k_stride, v, v_stride, cu_seqlens, num_seqs, plan, positions, pos_stride, q,
                            q_stride, num_heads, q_out, q_out_stride, nullptr, stream);
}

zl_status zl_paged_append_ex(const zl_paged_cache_t* cache, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const int32_t* cu_seqlens, int32_t num_seqs, const zl_rope_t* plan,
                             const int32_t* positions, int64_t pos_stride, const void* q, int64_t q_stride,
                             int32_t num_heads, void* q_out, int64_t q_out_stride, const int32_t* status,
                             void* stream) {
  return append(cache, k, k_stride, v, v_stride, cu_seqlens, num_seqs, plan, positions, pos_stride, q, q_stride,
                num_heads, q_out, q_out_stride, status, stream, false);
}

zl_status zl_paged_append_q4(const zl_paged_cache_t* cache, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const int32_t* cu_seqlens, int32_t num_seqs, const zl_rope_t* plan,
                             const int32_t* positions, int64_t pos_stride, const void* q, int64_t q_stride,
                             int32_t num_heads, void* q_out, int64_t q_out_stride, const int32_t* status,
                             void* stream) {
  return append(cache, k, k_stride, v, v_stride, cu_seqlens, num_seqs, plan, positions, pos_stride, q, q_stride,
                num_heads, q_out, q_out_stride, status, stream, true);
}

zl_status zl_paged_read_q4(const zl_paged_cache_t* cache, const int32_t* cu_seqlens, int32_t num_seqs, void* k,
                           int64_t k_stride, void* v, int64_t v_stride, void* stream) {
  zl_status st = check_cache(cache);
  if (st != ZL_OK) return st;
  int64_t tokens = 0;
  st = check_cu(cu_seqlens, num_seqs, &tokens);
  if (st != ZL_OK || tokens == 0) return st;
  st = check_cache_pointers(cache);
  if (st == ZL_OK) st = check_rows(k, k_stride, cache->num_kv_heads, cache->head_dim, tokens, 2);
  if (st == ZL_OK) st = check_rows(v, v_stride, cache->num_kv_heads, cache->head_dim, tokens, 2);
  if (st != ZL_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  static thread_local zl::ReadQ4Args<zl::kMaxSegs> a;
  static_cast<zl::ReadQ4Head&>(a) = zl::ReadQ4Head();
  a.k_pages = static_cast<const uint8_t*>(cache->k_pages);
  a.v_pages = static_cast<const uint8_t*>(cache->v_pages);
  a.page_table = cache->page_table;
  a.kv_lens = cache->kv_lens;
  a.k_out = k;
  a.v_out = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.nk = cache->num_kv_heads;
  a.head_dim = cache->head_dim;
  a.table_cols = cache->table_cols;
  a.num_pages = cache->num_pages;
  a.page_shift = shift_of(cache->page_size);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t s0 = 0; s0 < num_seqs; s0 += zl::kMaxSegs) {
    a.seq0 = s0;
    a.n_seqs = std::min(num_seqs - s0, zl::kMaxSegs);
    for (int32_t i = 0; i <= a.n_seqs; ++i) a.cu[i] = cu_seqlens[s0 + i];
    a.token0 = a.cu[0];
    a.tokens = a.cu[a.n_seqs] - a.cu[0];
    if (a.tokens == 0) continue;
    st = launch_counted("paged_read_q4", s, [&] { return zl::launch_read_q4(a, sms, s); });
    if (st != ZL_OK) return st;
  }
  return ZL_OK;
}

// ------------------------------------------------------------------ attention
zl_status zl_paged_attn_workspace_size(const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t max_kv_len,
                                       int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, size_t* bytes) {
  if (!bytes) return ZL_EINVAL;
  int64_t tq = 0;
  const zl_status st = check_attn(cu_seqlens_q, num_seqs, max_kv_len, num_heads, num_kv_heads, head_dim, &tq);
  if (st != ZL_OK) return st;
  *bytes = attn_workspace(cu_seqlens_q, Chosen{0, num_seqs, 0}, num_heads / num_kv_heads, head_dim);
  return ZL_OK;
}

zl_status zl_paged_attn(const zl_paged_cache_t* cache, const void* q, int64_t q_stride, const int32_t* cu_seqlens_q,
                        int32_t num_seqs, int32_t max_kv_len, int32_t num_heads, float softmax_scale, int32_t causal,
                        int32_t window, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  Attend c{cache, q, q_stride, cu_seqlens_q, num_seqs, max_kv_len, num_heads, softmax_scale, causal, window, o, lse,
           static_cast<cudaStream_t>(stream)};
  zl_status st = c.check();
  if (st != ZL_OK || c.tq == 0) return st;
  const Chosen all{0, num_seqs, 0};
  const size_t need = attn_workspace(cu_seqlens_q, all, c.group(), cache->head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return ZL_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  return st != ZL_OK ? st : launch_attn(c, *cache, all, workspace);
}

zl_status zl_paged_attn_q4_workspace_size(const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t max_kv_len,
                                          int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t window,
                                          size_t* bytes) {
  if (!bytes || window < 0) return ZL_EINVAL;
  int64_t tq = 0;
  zl_status st = check_attn(cu_seqlens_q, num_seqs, max_kv_len, num_heads, num_kv_heads, head_dim, &tq);
  if (st != ZL_OK) return st;
  Q4Plan p;
  st = plan_q4(cu_seqlens_q, num_seqs, max_kv_len, num_heads, num_kv_heads, head_dim, window, &p);
  if (st == ZL_OK) *bytes = p.bytes();
  return st;
}

zl_status zl_paged_attn_q4(const zl_paged_cache_t* cache, const void* q, int64_t q_stride, const int32_t* cu_seqlens_q,
                           int32_t num_seqs, int32_t max_kv_len, int32_t num_heads, float softmax_scale,
                           int32_t causal, int32_t window, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  Attend c{cache, q, q_stride, cu_seqlens_q, num_seqs, max_kv_len, num_heads, softmax_scale, causal, window, o, lse,
           static_cast<cudaStream_t>(stream)};
  zl_status st = c.check();
  if (st != ZL_OK || c.tq == 0) return st;
  Q4Plan p;
  st = plan_q4(cu_seqlens_q, num_seqs, max_kv_len, num_heads, cache->num_kv_heads, cache->head_dim, window, &p);
  if (st != ZL_OK) return st;
  if (p.bytes() > 0 && (!workspace || workspace_bytes < p.bytes())) return ZL_EWORKSPACE;
  if (p.bytes() > 0 && !aligned16(workspace)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  return st != ZL_OK ? st : launch_attn_q4(c, p, workspace);
}

// ------------------------------------------------------------------ pages
zl_status zl_pages_workspace_size(int32_t num_pages, size_t* bytes) {
  if (!bytes || num_pages < 1) return ZL_EINVAL;
  *bytes = zl::pages_workspace_words(num_pages) * sizeof(int32_t);
  return ZL_OK;
}

zl_status zl_pages_extend(const zl_page_tables_t* tables, const int32_t* counts, int32_t* status, void* stream) {
  zl::PageTable t;
  zl_status st = check_tables(tables, &t);
  if (st != ZL_OK) return st;
  if (!counts || !status) return ZL_EINVAL;
  if (misaligned4(counts) || misaligned4(status)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_counted("pages_extend", s, [&] { return zl::launch_pages_extend(t, counts, status, s); });
}

zl_status zl_pages_fork(const zl_page_pool_t* pool, const zl_page_tables_t* tables, const int32_t* parents,
                        const int32_t* children, int32_t n, int32_t* status, void* workspace, size_t workspace_bytes,
                        void* stream) {
  zl::PageTable t;
  zl::PagePool p;
  zl_status st = check_tables(tables, &t);
  if (st == ZL_OK) st = check_pool(pool, &p);
  if (st != ZL_OK) return st;
  if (p.num_pages != t.num_pages || n < 0 || n > zl::kMaxSlots || !status) return ZL_EINVAL;
  if (n > 0 && (!parents || !children)) return ZL_EINVAL;
  if (misaligned4(parents) || misaligned4(children) || misaligned4(status)) return ZL_EALIGN;
  st = check_workspace(t.num_pages, workspace, workspace_bytes);
  if (st != ZL_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t* ws = static_cast<int32_t*>(workspace);
  st = launch_counted("pages_fork_plan", s,
                      [&] { return zl::launch_pages_fork_plan(t, parents, children, n, ws, status, s); });
  if (st != ZL_OK || n == 0) return st;
  return launch_counted("pages_fork_move", s,
                        [&] { return zl::launch_pages_fork_move(p, t, parents, children, n, ws, sms, s); });
}

zl_status zl_pages_free(const zl_page_tables_t* tables, const int32_t* slots, int32_t n, void* stream) {
  zl::PageTable t;
  zl_status st = check_tables(tables, &t);
  if (st != ZL_OK) return st;
  if (n < 0 || n > (1 << 20)) return ZL_EINVAL;
  if (n == 0) return ZL_OK;
  if (!slots) return ZL_EINVAL;
  if (misaligned4(slots)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_counted("pages_free", s, [&] { return zl::launch_pages_free(t, slots, n, s); });
}

zl_status zl_pages_truncate(const zl_page_tables_t* tables, const int32_t* lens, void* stream) {
  zl::PageTable t;
  zl_status st = check_tables(tables, &t);
  if (st != ZL_OK) return st;
  if (!lens) return ZL_EINVAL;
  if (misaligned4(lens)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_counted("pages_truncate", s, [&] { return zl::launch_pages_truncate(t, lens, s); });
}

zl_status zl_pages_compact(const zl_page_pool_t* pool, const zl_page_tables_t* tables, int32_t* live, void* workspace,
                           size_t workspace_bytes, void* stream) {
  zl::PageTable t;
  zl::PagePool p;
  zl_status st = check_tables(tables, &t);
  if (st == ZL_OK) st = check_pool(pool, &p);
  if (st != ZL_OK) return st;
  if (p.num_pages != t.num_pages || !live) return ZL_EINVAL;
  if (misaligned4(live)) return ZL_EALIGN;
  st = check_workspace(t.num_pages, workspace, workspace_bytes);
  if (st != ZL_OK) return st;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t* ws = static_cast<int32_t*>(workspace);
  st = launch_counted("pages_compact_plan", s, [&] { return zl::launch_pages_compact_plan(t, ws, live, s); });
  if (st != ZL_OK) return st;
  return launch_counted("pages_compact_move", s, [&] { return zl::launch_pages_compact_move(p, t, ws, sms, s); });
}

zl_status zl_pages_copy(const zl_page_pool_t* pool, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  zl::PagePool p;
  zl_status st = check_pool(pool, &p);
  if (st != ZL_OK) return st;
  if (n < 0) return ZL_EINVAL;
  if (n == 0) return ZL_OK;
  if (!src || !dst) return ZL_EINVAL;
  if (misaligned4(src) || misaligned4(dst)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_counted("pages_copy", s, [&] { return zl::launch_pages_copy(p, src, dst, n, sms, s); });
}

}  // extern "C"
