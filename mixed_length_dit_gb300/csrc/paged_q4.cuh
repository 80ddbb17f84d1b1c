// The 4-bit form of a cache's tokens (include/zl_attn.h has its definition).
//
// Every 32 columns of a token's head share a step s; a value x is held as
// c = floor(x / s + 1/2) in [-8, 7] and reads c s.  A step is a byte 8 e + m:
// the top five and next three bits of a half below its sign, so (byte << 7) is
// the step as a half.  c has three bits beside its sign and s four, so c s is
// exact in bf16.
//
// A thread's piece of a token's head is 8 columns of each of its d / 32 groups,
// columns 32 q + 8 c + (0 .. 7) for piece c of four.  Its codes are one word for
// each group q, and the words of a piece stand together: one load of d / 8 bytes.
// For keys that is what a thread of the attention multiplies with.  For values
// a thread there wants four columns of each group, so the piece is two half
// pieces, the lower 16 bits of its words and the upper ones.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace zl {

constexpr int kQ4Group = 32;
constexpr uint32_t kQ4NaN = 0xffu;           // the step of a group that held a value that is not finite

// Bytes of a token's codes and steps.
template <int HD> constexpr int kQ4Codes = HD / 2;
template <int HD> constexpr int kQ4Steps = HD / kQ4Group;
template <int HD> constexpr int kQ4Row = kQ4Codes<HD> + kQ4Steps<HD>;

__device__ __forceinline__ float q4_step(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// The steps of bytes 0, 1 (2, 3) of a word: the bytes become the upper halves
// of 16 bits each, one to the right of where a half has them.
__device__ __forceinline__ float2 q4_steps01(uint32_t w) {
  const uint32_t h = __byte_perm(w, 0, 0x1404) >> 1;
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 q4_steps23(uint32_t w) {
  const uint32_t h = __byte_perm(w, 0, 0x3424) >> 1;
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The larger magnitudes of two pairs of bf16; a NaN is handed on.
__device__ __forceinline__ uint32_t q4_max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The largest magnitude among 8 bf16, as two of them.  Their patterns order as
// integers, with what is not finite above all others.
__device__ __forceinline__ uint32_t q4_top(const uint4& x) { return q4_max2(q4_max2(x.x, x.y), q4_max2(x.z, x.w)); }

// The byte of the step for a group whose largest magnitude is the bf16 `top`:
// top / 7 with four significant bits, halves up.  top has 8 bits, so a quotient
// that is no half lies at least 2^-8 of itself from one (below 2^-14, where steps
// are multiples of 2^-17, at least 2^-9 of such a unit); the product with
// 1 / 7 is off by 2^-23 of itself, and 2^-13 (2^-10) added before cutting puts
// the halves, and nothing else, on the upper side.
__device__ __forceinline__ uint32_t q4_step_byte(uint32_t top) {
  if (top >= 0x7f80u) return kQ4NaN;
  const float want = __uint_as_float(top << 16) * (1.f / 7.f);
  const uint32_t normal = min(((__float_as_uint(want) + 0x80400u) >> 20) - (112u << 3), 0xf7u);
  const uint32_t small = static_cast<uint32_t>(want * 131072.f + (0.5f + 0x1p-10f));
  return want >= 0x1p-14f ? normal : small;
}

// What a value is multiplied by: 1 / s, or 0 where the group reads as zero or NaN.
__device__ __forceinline__ float q4_inverse(uint32_t byte) {
  return byte == 0 || byte == kQ4NaN ? 0.f : __fdividef(1.f, q4_step(byte));
}

// The codes of 8 bf16, c + 8 in four bits each.  A half between two codes is a
// bf16 itself (two times c + 1/2 and a step of four bits have eight), and its
// neighbours lie 2^-10 steps away at least: 2^-12 added before cutting puts the
// halves on the upper side although the inverse and the product are rounded.  A
// step rounded to four bits is at least 16/17 of the seventh, so that x / s stays below
// 7.5: only steps below 2^-14 and the largest one need clamping.
template <bool CLAMP>
__device__ __forceinline__ uint32_t q4_codes_of(const uint4& x, float inv) {
  if (CLAMP && inv == 0.f) return 0x88888888u;   // zero, or not finite
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(w[i]);
    float a = fmaf(f.x, inv, 8.5f + 0x1p-12f), b = fmaf(f.y, inv, 8.5f + 0x1p-12f);
    if (CLAMP) {
      a = fminf(fmaxf(a, 0.f), 15.5f);
      b = fminf(fmaxf(b, 0.f), 15.5f);
    }
    // cut to whole numbers in the float's low bits
    r += __float_as_uint(__fadd_rd(a, 8388608.f)) << (8 * i);
    r += __float_as_uint(__fadd_rd(b, 8388608.f)) << (8 * i + 4);
  }
  return r - ((0x4b000000u) + (0x4b000000u << 4));   // the float's upper bits (what was shifted further is gone)
}
__device__ __forceinline__ uint32_t q4_codes(const uint4& x, float inv, bool clamp) {
  return clamp ? q4_codes_of<true>(x, inv) : q4_codes_of<false>(x, inv);
}
__device__ __forceinline__ bool q4_clamps(uint32_t byte) { return byte - 8u >= 0xf7u - 8u; }

// A piece's words, one for each group, as they are held, and back.
template <int G>
__device__ __forceinline__ void q4_order_values(uint32_t (&w)[G]) {
  if constexpr (G == 4) {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5410), b = __byte_perm(w[2], w[3], 0x5410);
    const uint32_t c = __byte_perm(w[0], w[1], 0x7632), d = __byte_perm(w[2], w[3], 0x7632);
    w[0] = a; w[1] = b; w[2] = c; w[3] = d;
  } else {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5410), b = __byte_perm(w[0], w[1], 0x7632);
    w[0] = a; w[1] = b;
  }
}
template <int G>
__device__ __forceinline__ void q4_natural_values(uint32_t (&w)[G]) {
  if constexpr (G == 4) {
    const uint32_t a = __byte_perm(w[0], w[2], 0x5410), b = __byte_perm(w[0], w[2], 0x7632);
    const uint32_t c = __byte_perm(w[1], w[3], 0x5410), d = __byte_perm(w[1], w[3], 0x7632);
    w[0] = a; w[1] = b; w[2] = c; w[3] = d;
  } else {
    q4_order_values(w);                        // its own inverse
  }
}

// The values of a word's 8 codes with a step: 128 + n is a bf16 whose last four
// bits are n, so c = (128 + n) - 136; exact, and so is the product.
__device__ __forceinline__ uint4 q4_values(uint32_t w, float step) {
  const __nv_bfloat162 s = __float2bfloat162_rn(step), off = __float2bfloat162_rn(136.f);
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {                // codes 2j and 2j + 1
    const uint32_t x = w >> (8 * j);
    const uint32_t b = (x & 0xfu) | ((x & 0xf0u) << 12) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), off), s);
    r[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace zl
