// The turn of rotary positions (zl_rope_t) and the place of a new token in a
// paged cache, as the kernels of rope.cu and pages_q4.cu compute them.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.h"
#include "zl_attn.h"

namespace zl {

// The axis whose position turns pair i.
__device__ __forceinline__ int rope_axis(const zl_rope_t& r, int i) {
  int axis = 0;
  while (axis < r.n_axes - 1 && i >= r.pair_end[axis]) ++axis;
  return axis;
}

// Cosine and sine, times the magnitude, of pair i at position p.  The angle is
// a 64-bit fixed-point fraction of a turn, p * step mod 2^64.
__device__ __forceinline__ float2 rope_turn(const zl_rope_t& r, int64_t p, int i, bool inverse) {
  const uint64_t phase = static_cast<uint64_t>(p) * r.step[i];
  // signed fraction of a turn in the top 32 bits; in half turns for sincospi
  const float x2 = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;
  float s, c;
  sincospif(x2, &s, &c);
  return make_float2(c * r.magnitude, (inverse ? -s : s) * r.magnitude);
}

// Whether a plan's pairs do not fill 16-byte pieces of elements of that size.
__host__ __device__ __forceinline__ bool rope_alone(const zl_rope_t& r, int elem_bytes) {
  return (r.rot_dim / 2) % (16 / elem_bytes) != 0;
}

// A pair by its cosine and sine.  The roundings are spelled out, so that every kernel
// gives the same bits: ALONE for plans whose pairs do not fill 16-byte pieces
// (rope_alone), where the fused product of the second element is the other one.
__device__ __forceinline__ float rope_first(float a, float b, float c, float s) {
  return __fmaf_rn(a, c, -__fmul_rn(b, s));
}
template <bool ALONE>
__device__ __forceinline__ float rope_second(float a, float b, float c, float s) {
  return ALONE ? __fmaf_rn(b, c, __fmul_rn(a, s)) : __fmaf_rn(a, s, __fmul_rn(b, c));
}

// Where a batch's packed token t lies in the cache: its position in the sequence
// (below zero where the length does not count it) and its page, or -1.  A holds
// the batch's sequences and the tables: RopeArgs, ReadQ4Args.
struct Place {
  int64_t pos;
  int32_t page;
};

template <typename A>
__device__ __forceinline__ Place place_of(const A& a, int64_t t) {
  int lo = 0, hi = a.n_seqs - 1;             // the last sequence that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int64_t seq = a.seq0 + lo;
  const int n = a.cu[lo + 1] - a.cu[lo];
  Place r = {static_cast<int64_t>(a.kv_lens[seq]) - n + (t - a.cu[lo]), -1};
  if (r.pos >= 0 && (r.pos >> a.page_shift) < a.table_cols) {
    const int page = a.page_table[seq * a.table_cols + (r.pos >> a.page_shift)];
    if (page >= 0 && page < a.num_pages) r.page = page;
  }
  return r;
}

}  // namespace zl
