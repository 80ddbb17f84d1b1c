// Whole-page operations of the paged key/value cache: extending, truncating,
// forking, freeing and compacting sequences, and copying pages.
//
// The tables live on the device, so that a generation loop (or a captured
// graph) never waits for the host.  What must be decided in one order, which
// free page goes to whom, is decided by one CTA that scans the reference counts
// (each warp owns a run of pages, read 32 at a time and ranked by ballots; with a
// run per thread, whose loads do not coalesce, planning 27,500 pages took 12 us
// more), and a prefix sum over the warps ranks the runs: results are the same
// on every run, lowest page number first, and an operation that lacks pages
// changes nothing.  The plan is a list of page moves in the workspace; a second
// launch over the whole GPU then moves the pages and rewrites the tables.  That
// launch is bound by HBM (each moved byte is read and written once: 6.4 GB in
// 944 us, 6.8 TB/s); the plan is bound by the latency of its few dependent
// passes over the counts (27 us for 27,500 pages).
#include "common.cuh"
#include "paged.h"

namespace zl {
namespace {

__device__ uint32_t g_pages_err;

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;

// Workspace words.
constexpr int kHdrOk = 0;          // the plan stands: move pages
constexpr int kHdrMoves = 1;       // page moves in the list
constexpr int kHdrLive = 2;        // compact: pages in use
__host__ __device__ inline int64_t ws_len() { return kPageHeader; }                       // fork: parents' lengths
__host__ __device__ inline int64_t ws_src() { return kPageHeader + kMaxSlots; }
__host__ __device__ inline int64_t ws_dst(int64_t np) { return ws_src() + np; }
__host__ __device__ inline int64_t ws_map(int64_t np) { return ws_src() + 2 * np; }

// Exclusive prefix sum of one value per thread over the CTA; *total gets the
// sum.  Every thread calls it.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int warp_sum[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = warp_sum[lane];
    int s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    warp_sum[lane] = s - w;
    if (lane == 31) *total = s;
  }
  __syncthreads();
  const int base = warp_sum[warp];
  __syncthreads();
  return base + x - v;
}

__device__ __forceinline__ int pages_of(int64_t len, int shift) {
  return static_cast<int>((len + (int64_t(1) << shift) - 1) >> shift);
}

// A warp's run of pages [first, last), a multiple of 32 apart.
__device__ __forceinline__ void page_run(int num_pages, int* first, int* last) {
  constexpr int kWarps = kPlanThreads / 32;
  const int64_t per = ((static_cast<int64_t>(num_pages) + kWarps - 1) / kWarps + 31) & ~int64_t(31);
  const int64_t f = per * (threadIdx.x >> 5);
  *first = static_cast<int>(f < num_pages ? f : num_pages);
  *last = static_cast<int>(f + per < num_pages ? f + per : num_pages);
}

// Pages of the warp's run that `pred` (of a page and its count) holds for.
template <typename P>
__device__ __forceinline__ int count_run(const PageTable& t, int first, int last, P pred) {
  int n = 0;
#pragma unroll 4
  for (int p0 = first; p0 < last; p0 += 32) {
    const int p = p0 + static_cast<int>(threadIdx.x & 31);
    n += __popc(__ballot_sync(0xffffffffu, p < last && pred(p, t.refs[p])));
  }
  return n;
}

// Calls `take(page, rank)` for those pages in order, ranks from `rank` on, as
// long as they are below `end`.
template <typename P, typename F>
__device__ __forceinline__ void rank_run(const PageTable& t, int first, int last, int rank, int end, P pred, F take) {
  const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
#pragma unroll 4
  for (int p0 = first; p0 < last && rank < end; p0 += 32) {
    const int p = p0 + static_cast<int>(threadIdx.x & 31);
    const bool is = p < last && pred(p, t.refs[p]);
    const uint32_t m = __ballot_sync(0xffffffffu, is);
    const int r = rank + __popc(m & below);
    if (is && r < end) take(p, r);
    rank += __popc(m);
  }
}

// Exclusive prefix sum of one value per warp (lane 0's) over the CTA.
__device__ __forceinline__ int warps_scan(int v, int* total) {
  return __shfl_sync(0xffffffffu, block_scan((threadIdx.x & 31) == 0 ? v : 0, total), 0);
}

__device__ __forceinline__ bool is_free(int, int refs) { return refs == 0; }

// ------------------------------------------------------------------ extend
__global__ void __launch_bounds__(kPlanThreads)
extend_kernel(PageTable t, const int32_t* counts, int32_t* status) {
  __shared__ int start[kMaxSlots];             // first rank of each slot's new pages
  __shared__ int bad, shared_end, total_need, total_free;
  __shared__ unsigned long long wanted;        // 64 bits: more than there are pages may be asked for
  if (threadIdx.x == 0) {
    bad = shared_end = 0;
    wanted = 0;
  }
  __syncthreads();
  // each thread owns a run of slots
  const int per = (t.slots + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(t.slots, static_cast<int>(threadIdx.x) * per), s1 = min(t.slots, s0 + per);
  int64_t need = 0;
  bool ok = true, own_end = true;
  for (int s = s0; s < s1; ++s) {
    const int64_t len = t.kv_lens[s], c = counts[s];
    if (len < 0 || c < 0 || len + c > INT32_MAX || pages_of(len + c, t.page_shift) > t.cols) {
      ok = false;
      continue;
    }
    need += pages_of(len + c, t.page_shift) - pages_of(len, t.page_shift);
    // a slot that was truncated inside a page which another one holds too: new
    // tokens would be written over the other's
    if (c > 0 && (len & ((1 << t.page_shift) - 1)) != 0) {
      const int p = t.table[static_cast<int64_t>(s) * t.cols + (len >> t.page_shift)];
      if (p >= 0 && p < t.num_pages && t.refs[p] > 1) own_end = false;
    }
  }
  if (!ok) atomicExch(&bad, 1);
  if (!own_end) atomicExch(&shared_end, 1);
  atomicAdd(&wanted, static_cast<unsigned long long>(need));
  int first, last;
  page_run(t.num_pages, &first, &last);
  const int rank0 = warps_scan(count_run(t, first, last, is_free), &total_free);
  if (bad || shared_end || wanted > static_cast<unsigned long long>(total_free)) {
    const unsigned long long lacking = wanted - total_free;
    if (threadIdx.x == 0)
      *status = bad ? -1 : shared_end ? -2 : static_cast<int>(lacking < INT32_MAX ? lacking : INT32_MAX);
    return;
  }
  int at = block_scan(static_cast<int>(need), &total_need);
  for (int s = s0; s < s1; ++s) {
    start[s] = at;
    at += pages_of(static_cast<int64_t>(t.kv_lens[s]) + counts[s], t.page_shift) - pages_of(t.kv_lens[s], t.page_shift);
  }
  __syncthreads();
  rank_run(t, first, last, rank0, total_need, is_free, [&](int p, int rank) {
    int lo = 0, hi = t.slots - 1;              // the last slot whose new pages start at or before rank
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= rank) lo = mid; else hi = mid - 1;
    }
    t.table[static_cast<int64_t>(lo) * t.cols + pages_of(t.kv_lens[lo], t.page_shift) + rank - start[lo]] = p;
    t.refs[p] = 1;
  });
  __syncthreads();                             // the old lengths were read above
  for (int s = s0; s < s1; ++s) t.kv_lens[s] += counts[s];
  if (threadIdx.x == 0) *status = 0;
}

// ------------------------------------------------------------------ free, truncate
// A CTA takes the pages behind length `keep` from slot s, whose length was
// `len`: each loses a reference.
__device__ __forceinline__ void drop_pages(const PageTable& t, int s, int len, int keep) {
  const int64_t used = len > 0 ? pages_of(len, t.page_shift) : 0;
  if (used > t.cols && threadIdx.x == 0) atomicOr(&g_pages_err, ERR_BAD_PAGE);
  for (int j = pages_of(keep, t.page_shift) + threadIdx.x; j < used && j < t.cols; j += kMoveThreads) {
    int32_t* e = t.table + static_cast<int64_t>(s) * t.cols + j;
    const int p = *e;
    *e = -1;
    if (p < 0 || p >= t.num_pages) {
      atomicOr(&g_pages_err, ERR_BAD_PAGE);
    } else if (atomicSub(&t.refs[p], 1) <= 0) {
      atomicAdd(&t.refs[p], 1);
      atomicOr(&g_pages_err, ERR_BAD_PAGE);
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) free_kernel(PageTable t, const int32_t* slots, int32_t n) {
  __shared__ int len;
  const int s = slots[blockIdx.x];
  if (s < 0 || s >= t.slots) {
    if (threadIdx.x == 0) atomicOr(&g_pages_err, ERR_BAD_PAGE);
    return;
  }
  // a slot that is named twice: whoever takes its length frees its pages
  if (threadIdx.x == 0) len = atomicExch(&t.kv_lens[s], 0);
  __syncthreads();
  drop_pages(t, s, len, 0);
}

__global__ void __launch_bounds__(kMoveThreads) truncate_kernel(PageTable t, const int32_t* lens) {
  const int s = blockIdx.x;
  const int len = t.kv_lens[s], keep = lens[s];
  if (keep < 0) {
    if (threadIdx.x == 0) atomicOr(&g_pages_err, ERR_BAD_PAGE);
    return;
  }
  if (keep >= len) return;
  __syncthreads();                             // every thread has read the length
  if (threadIdx.x == 0) t.kv_lens[s] = keep;
  drop_pages(t, s, len, keep);
}

// ------------------------------------------------------------------ fork
__global__ void __launch_bounds__(kPlanThreads)
fork_plan_kernel(PageTable t, const int32_t* parents, const int32_t* children, int32_t n, int32_t* ws,
                 int32_t* status) {
  __shared__ int bad, total_need, total_free;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int32_t* plen = ws + ws_len();
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(n, static_cast<int>(threadIdx.x) * per), i1 = min(n, i0 + per);
  const int mask = (1 << t.page_shift) - 1;
  // every parent's length as it was before the call
  int need = 0;
  bool ok = true;
  for (int i = i0; i < i1; ++i) {
    const int p = parents[i], c = children[i];
    int len = 0;
    if (p < 0 || p >= t.slots || c < 0 || c >= t.slots || p == c) {
      ok = false;
    } else {
      len = t.kv_lens[p];
      if (len < 0 || pages_of(len, t.page_shift) > t.cols) {
        ok = false;
        len = 0;
      } else if (len & mask) {
        const int e = t.table[static_cast<int64_t>(p) * t.cols + (len >> t.page_shift)];
        ok = ok && e >= 0 && e < t.num_pages;
        ++need;
      }
    }
    plen[i] = len;
  }
  if (!ok) atomicExch(&bad, 1);
  __syncthreads();
  const bool in_range = bad == 0;
  // children are empty and distinct: mark each by a length of its own
  __syncthreads();
  if (in_range) {
    for (int i = i0; i < i1; ++i)
      if (atomicCAS(&t.kv_lens[children[i]], 0, -1 - i) != 0) atomicExch(&bad, 1);
  }
  int first, last;
  page_run(t.num_pages, &first, &last);
  const int need0 = block_scan(need, &total_need);
  const int rank0 = warps_scan(count_run(t, first, last, is_free), &total_free);
  if (bad || total_need > total_free) {
    if (in_range)
      for (int i = i0; i < i1; ++i) atomicCAS(&t.kv_lens[children[i]], -1 - i, 0);
    if (threadIdx.x == 0) {
      *status = bad ? -1 : total_need - total_free;
      ws[kHdrOk] = 0;
    }
    return;
  }
  int32_t* src = ws + ws_src();
  int32_t* dst = ws + ws_dst(t.num_pages);
  rank_run(t, first, last, rank0, total_need, is_free, [&](int p, int rank) { dst[rank] = p; });
  __syncthreads();
  int at = need0;
  for (int i = i0; i < i1; ++i) {
    const int len = plen[i];
    if (len & mask) {
      const int64_t col = len >> t.page_shift;
      src[at] = t.table[static_cast<int64_t>(parents[i]) * t.cols + col];
      t.table[static_cast<int64_t>(children[i]) * t.cols + col] = dst[at];
      t.refs[dst[at]] = 1;
      ++at;
    }
    t.kv_lens[children[i]] = len;
  }
  if (threadIdx.x == 0) {
    *status = 0;
    ws[kHdrMoves] = total_need;
    ws[kHdrOk] = 1;
  }
}

// ------------------------------------------------------------------ compact
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PageTable t, int32_t* ws, int32_t* live_out) {
  __shared__ int live, holes, movers;
  int first, last;
  page_run(t.num_pages, &first, &last);
  warps_scan(count_run(t, first, last, [](int, int refs) { return refs > 0; }), &live);
  int32_t* src = ws + ws_src();
  int32_t* dst = ws + ws_dst(t.num_pages);
  int32_t* map = ws + ws_map(t.num_pages);
  const int n = live;
  const auto hole = [n](int p, int refs) { return p < n && refs <= 0; };
  const auto mover = [n](int p, int refs) { return p >= n && refs > 0; };
  const int rh = warps_scan(count_run(t, first, last, hole), &holes);
  const int rm = warps_scan(count_run(t, first, last, mover), &movers);
  rank_run(t, first, last, rh, INT32_MAX, hole, [&](int p, int rank) { dst[rank] = p; });
  rank_run(t, first, last, rm, INT32_MAX, mover, [&](int p, int rank) { src[rank] = p; });
  for (int p = threadIdx.x; p < t.num_pages; p += kPlanThreads) map[p] = p;
  __syncthreads();
  // four moves of a thread at once: their reads depend on one another
  for (int i0 = threadIdx.x; i0 < movers; i0 += 4 * kPlanThreads) {
    int s[4], d[4], r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kPlanThreads;
      s[u] = i < movers ? src[i] : -1;
      d[u] = i < movers ? dst[i] : 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u] = s[u] >= 0 ? t.refs[s[u]] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s[u] < 0) continue;
      map[s[u]] = d[u];
      t.refs[d[u]] = r[u];
      t.refs[s[u]] = 0;
    }
  }
  if (threadIdx.x == 0) {
    ws[kHdrOk] = 1;
    ws[kHdrMoves] = movers;
    ws[kHdrLive] = live;
    *live_out = live;
  }
}

// ------------------------------------------------------------------ moving pages
// Copies page src[i] to dst[i] in every group, in pieces of 16 KB that the
// blocks take in turn: four 16-byte loads of a thread are in flight at once.
constexpr int kPieceBytes = kMoveThreads * 16 * 4;

__device__ __forceinline__ void copy_pages(const PagePool& pool, const int32_t* src, const int32_t* dst, int n,
                                           int64_t block, int64_t blocks) {
  const int64_t pieces = (pool.page_bytes + kPieceBytes - 1) / kPieceBytes;
  const int64_t total = static_cast<int64_t>(n) * pool.groups * pieces;
  for (int64_t w = block; w < total; w += blocks) {
    const int64_t piece = w % pieces;
    const int64_t ig = w / pieces;
    const int64_t g = ig % pool.groups;
    const int64_t i = ig / pool.groups;
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= pool.num_pages || d < 0 || d >= pool.num_pages) {
      if (threadIdx.x == 0) atomicOr(&g_pages_err, ERR_BAD_PAGE);
      continue;
    }
    const uint8_t* from = pool.base + g * pool.group_stride + s * pool.page_bytes + piece * kPieceBytes;
    uint8_t* to = pool.base + g * pool.group_stride + d * pool.page_bytes + piece * kPieceBytes;
    const int64_t left = pool.page_bytes - piece * kPieceBytes;
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t o = (static_cast<int64_t>(u) * kMoveThreads + threadIdx.x) * 16;
      if (o < left) x[u] = *reinterpret_cast<const uint4*>(from + o);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t o = (static_cast<int64_t>(u) * kMoveThreads + threadIdx.x) * 16;
      if (o < left) *reinterpret_cast<uint4*>(to + o) = x[u];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads)
copy_kernel(PagePool pool, const int32_t* src, const int32_t* dst, int32_t n) {
  copy_pages(pool, src, dst, n, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kMoveThreads)
fork_move_kernel(PagePool pool, PageTable t, const int32_t* parents, const int32_t* children, int32_t n,
                 const int32_t* ws) {
  if (!ws[kHdrOk]) return;
  const int32_t* plen = ws + ws_len();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int full = plen[i] >> t.page_shift;
    const int32_t* from = t.table + static_cast<int64_t>(parents[i]) * t.cols;
    int32_t* to = t.table + static_cast<int64_t>(children[i]) * t.cols;
    for (int j = threadIdx.x; j < full; j += kMoveThreads) {
      const int p = from[j];
      to[j] = p;
      if (p >= 0 && p < t.num_pages)
        atomicAdd(&t.refs[p], 1);
      else
        atomicOr(&g_pages_err, ERR_BAD_PAGE);
    }
  }
  copy_pages(pool, ws + ws_src(), ws + ws_dst(t.num_pages), ws[kHdrMoves], blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(PagePool pool, PageTable t, const int32_t* ws) {
  const int live = ws[kHdrLive];
  const int32_t* map = ws + ws_map(t.num_pages);
  for (int s = blockIdx.x; s < t.slots; s += gridDim.x) {
    const int len = t.kv_lens[s];
    const int used = len > 0 ? min(pages_of(len, t.page_shift), t.cols) : 0;
    int32_t* row = t.table + static_cast<int64_t>(s) * t.cols;
    for (int j = threadIdx.x; j < used; j += kMoveThreads) {
      const int p = row[j];
      if (p < 0 || p >= t.num_pages)
        atomicOr(&g_pages_err, ERR_BAD_PAGE);
      else if (p >= live)
        row[j] = map[p];
    }
  }
  copy_pages(pool, ws + ws_src(), ws + ws_dst(t.num_pages), ws[kHdrMoves], blockIdx.x, gridDim.x);
}

}  // namespace

cudaError_t launch_pages_copy(const PagePool& pool, const int32_t* src, const int32_t* dst, int32_t n, int num_sms,
                              cudaStream_t stream) {
  copy_kernel<<<num_sms * 8, kMoveThreads, 0, stream>>>(pool, src, dst, n);
  return cudaGetLastError();
}

cudaError_t launch_pages_extend(const PageTable& t, const int32_t* counts, int32_t* status, cudaStream_t stream) {
  extend_kernel<<<1, kPlanThreads, 0, stream>>>(t, counts, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageTable& t, const int32_t* slots, int32_t n, cudaStream_t stream) {
  free_kernel<<<n, kMoveThreads, 0, stream>>>(t, slots, n);
  return cudaGetLastError();
}

cudaError_t launch_pages_truncate(const PageTable& t, const int32_t* lens, cudaStream_t stream) {
  truncate_kernel<<<t.slots, kMoveThreads, 0, stream>>>(t, lens);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork_plan(const PageTable& t, const int32_t* parents, const int32_t* children, int32_t n,
                                   int32_t* ws, int32_t* status, cudaStream_t stream) {
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(t, parents, children, n, ws, status);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork_move(const PagePool& pool, const PageTable& t, const int32_t* parents,
                                   const int32_t* children, int32_t n, const int32_t* ws, int num_sms,
                                   cudaStream_t stream) {
  fork_move_kernel<<<num_sms * 8, kMoveThreads, 0, stream>>>(pool, t, parents, children, n, ws);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact_plan(const PageTable& t, int32_t* ws, int32_t* live, cudaStream_t stream) {
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(t, ws, live);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact_move(const PagePool& pool, const PageTable& t, const int32_t* ws, int num_sms,
                                      cudaStream_t stream) {
  compact_move_kernel<<<num_sms * 8, kMoveThreads, 0, stream>>>(pool, t, ws);
  return cudaGetLastError();
}

uint32_t pages_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_pages_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_pages_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
