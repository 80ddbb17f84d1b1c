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

// The next launch of a kind: as many sequences from *i on as it holds.
Launch next_launch(const int32_t* cu, int32_t num_seqs, int32_t group, bool pair, int32_t* i) {
  Launch l;
  for (; *i < num_seqs && l.segs < zl::kMaxSegs; ++*i) {
    const int32_t n = cu[*i + 1] - cu[*i];
    if (n == 0 || (n > tile_tokens(group)) != pair) continue;
    ++l.segs;
    l.slot_rows = pair ? 2 * zl::kBlockM : std::max(l.slot_rows, n * group);
  }
  return l;
}

// The launches run one after another and share the workspace.
size_t attn_workspace(const int32_t* cu, int32_t num_seqs, int32_t group, int32_t hd) {
  size_t need = 0;
  for (const bool pair : {false, true})
    for (int32_t i = 0; i < num_seqs;) {
      const Launch l = next_launch(cu, num_seqs, group, pair, &i);
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

}  // namespace

namespace zl {

uint32_t paged_take_error() {
  const uint32_t a = rope_take_error();
  const uint32_t b = pages_take_error();
  const uint32_t c = paged_attn_take_error();
  if (a == 0xFFFFFFFFu || b == 0xFFFFFFFFu || c == 0xFFFFFFFFu) return 0xFFFFFFFFu;
  return a | b | c;
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
    st = launch_counted("paged_append", s, [&] { return zl::launch_rope(a, sms, s); });
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
  *bytes = attn_workspace(cu_seqlens_q, num_seqs, num_heads / num_kv_heads, head_dim);
  return ZL_OK;
}

zl_status zl_paged_attn(const zl_paged_cache_t* cache, const void* q, int64_t q_stride, const int32_t* cu_seqlens_q,
                        int32_t num_seqs, int32_t max_kv_len, int32_t num_heads, float softmax_scale, int32_t causal,
                        int32_t window, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  zl_status st = check_cache(cache);
  if (st != ZL_OK) return st;
  int64_t tq = 0;
  st = check_attn(cu_seqlens_q, num_seqs, max_kv_len, num_heads, cache->num_kv_heads, cache->head_dim, &tq);
  if (st != ZL_OK) return st;
  if (max_kv_len > int64_t(cache->table_cols) * cache->page_size) return ZL_EINVAL;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return ZL_EINVAL;
  if ((causal != 0 && causal != 1) || window < 0) return ZL_EINVAL;
  if (tq == 0) return ZL_OK;
  st = check_cache_pointers(cache);
  if (st != ZL_OK) return st;
  if (!o || !lse) return ZL_EINVAL;
  if (!aligned16(o) || misaligned4(lse)) return ZL_EALIGN;
  const int32_t hd = cache->head_dim;
  st = check_rows(q, q_stride, num_heads, hd, tq, 2);
  if (st != ZL_OK) return st;

  const int32_t group = num_heads / cache->num_kv_heads;
  const size_t need = attn_workspace(cu_seqlens_q, num_seqs, group, hd);
  if (need > 0 && (!workspace || workspace_bytes < need)) return ZL_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return ZL_EALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != ZL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  static thread_local zl::PagedAttnArgs<zl::kMaxSegs> a;      // ~21 KB: kept off the stack
  static_cast<zl::PagedAttnHead&>(a) = zl::PagedAttnHead();
  a.page_table = cache->page_table;
  a.kv_lens = cache->kv_lens;
  a.o = o;
  a.lse = lse;
  a.lse_stride = tq;
  a.num_heads = num_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = group;
  a.group_inv = (65536 + group - 1) / group;
  a.tile_tokens = tile_tokens(group);
  a.table_cols = cache->table_cols;
  a.num_pages = cache->num_pages;
  a.page_shift = shift_of(cache->page_size);
  a.max_kv_len = max_kv_len;
  a.causal = causal;
  a.window = window < max_kv_len ? window : 0;   // one that reaches over every key is none (and stays in 32 bits)
  a.scale_log2 = softmax_scale * 1.4426950408889634f;

  // the maps that the call's kinds of sequences use
  bool copies[3] = {false, false, false}, pairs = false;
  for (int32_t i = 0; i < num_seqs; ++i) {
    const int64_t n = cu_seqlens_q[i + 1] - cu_seqlens_q[i];
    if (n == 0) continue;
    pairs = pairs || n > a.tile_tokens;
    const int64_t tile_rows = n * a.group;
    copies[n > a.tile_tokens || tile_rows > 64 ? 0 : tile_rows > 32 ? 1 : 2] = true;
  }
  zl::PagedMaps maps;
  const int64_t pool_rows = int64_t(cache->num_pages) * cache->num_kv_heads * cache->page_size;
  const int box_rows = std::min(cache->page_size, zl::kBlockN);
  bool ok = zl::make_map(&maps.k, cache->k_pages, pool_rows, 1, hd, box_rows) &&
            zl::make_map(&maps.v, cache->v_pages, pool_rows, 1, hd, box_rows);
  if (pairs)
    ok = ok && zl::make_map_heads(&maps.o, o, tq, num_heads, hd, int64_t(num_heads) * hd, a.group, a.tile_tokens);
  for (int i = 0; i < 3; ++i)
    if (copies[i])
      ok = ok && zl::make_map_heads(&maps.q[i], q, tq, num_heads, hd, q_stride, a.group, zl::kBlockM / (1 << i) / a.group);
  if (!ok) return ZL_ECUDA;

  a.joins = static_cast<zl::PagedJoin*>(workspace);
  a.o_part = reinterpret_cast<float*>(a.joins + zl::kPagedCtas);
  for (const bool pair : {false, true}) {
    for (int32_t i = 0; i < num_seqs;) {
      const int32_t first = i;
      const Launch l = next_launch(cu_seqlens_q, num_seqs, group, pair, &i);
      if (l.segs == 0) continue;
      a.slot_rows = l.slot_rows;
      a.lse_part = a.o_part + int64_t(2) * zl::kPagedCtas * l.slot_rows * hd;
      a.n_segs = 0;
      for (int32_t x = first; x < i; ++x) {
        const int32_t n = cu_seqlens_q[x + 1] - cu_seqlens_q[x];
        if (n > 0 && (n > a.tile_tokens) == pair) a.segs[a.n_segs++] = zl::PagedSeg{x, cu_seqlens_q[x], n};
      }
      a.whole = whole_units(a, pair);
      st = launch_counted("paged_attn", s, [&] { return zl::launch_paged_attn(hd, pair, maps, a, s); });
      if (st != ZL_OK) return st;
      if (a.whole > 0) continue;
      st = launch_counted("paged_join", s, [&] { return zl::launch_paged_join(hd, pair, a, s); });
      if (st != ZL_OK) return st;
    }
  }
  return ZL_OK;
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
