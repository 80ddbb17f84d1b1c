// Attention of a chunk of new tokens over a paged key/value cache.
//
// One warp per (query token, head) row: the row's keys are walked once with a
// running maximum and sum (base 2), each lane owning d/32 columns of q, k, v
// and the output.
#include "common.cuh"
#include "paged.h"

namespace zl {
namespace {

__device__ uint32_t g_paged_err;

constexpr int kSimpleThreads = 256;

template <int HD>
__global__ void __launch_bounds__(kSimpleThreads) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int C = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kSimpleThreads / 32) + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.tokens) * a.num_heads) return;
  const int64_t t = a.token0 + row / a.num_heads;
  const int h = static_cast<int>(row % a.num_heads);
  int lo = 0, hi = a.n_segs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.segs[mid].q_row0 <= t) lo = mid; else hi = mid - 1;
  }
  const PagedSeg sg = a.segs[lo];
  const int hk = h / a.group;
  int len = a.kv_lens[sg.seq];
  if (len < 0 || len > a.max_kv_len) {
    if (lane == 0) atomicOr(&g_paged_err, ERR_BAD_PAGE);
    len = len < 0 ? 0 : a.max_kv_len;
  }
  const int p = len - sg.q_len + static_cast<int>(t - sg.q_row0);
  const int k_end = a.causal ? min(len, p + 1) : len;
  const int k_begin = a.window > 0 ? max(0, p - a.window + 1) : 0;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + static_cast<int64_t>(h) * HD;
  float x[C], acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    x[c] = __bfloat162float(q[lane * C + c]) * a.scale_log2;
    acc[c] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = k_begin; j < k_end; ++j) {
    const int page = a.page_table[static_cast<int64_t>(sg.seq) * a.table_cols + (j >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(&g_paged_err, ERR_BAD_PAGE);
      continue;
    }
    const int64_t off = (((static_cast<int64_t>(page) * a.num_kv_heads + hk) << a.page_shift) +
                         (j & ((1 << a.page_shift) - 1))) * HD + lane * C;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k_pages) + off;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_pages) + off;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s = fmaf(x[c], __bfloat162float(k[c]), s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float m_new = fmaxf(m, s);
    const float alpha = m_new == -INFINITY ? 1.f : exp2f(m - m_new);
    const float w = m_new == -INFINITY ? 0.f : exp2f(s - m_new);
    l = l * alpha + w;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(w, __bfloat162float(v[c]), acc[c] * alpha);
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (t * a.num_heads + h) * HD;
#pragma unroll
  for (int c = 0; c < C; ++c) o[lane * C + c] = __float2bfloat16_rn(acc[c] * inv);
  if (lane == 0) a.lse[static_cast<int64_t>(h) * a.lse_stride + t] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attn(int head_dim, const PagedAttnArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.num_heads;
  const int64_t blocks = (rows + kSimpleThreads / 32 - 1) / (kSimpleThreads / 32);
  if (head_dim == 64)
    paged_attn_kernel<64><<<static_cast<unsigned>(blocks), kSimpleThreads, 0, stream>>>(a);
  else
    paged_attn_kernel<128><<<static_cast<unsigned>(blocks), kSimpleThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

uint32_t paged_attn_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_paged_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
