// Rotary positions of packed queries and keys, and the append of new tokens
// to a paged cache, which turns them on the way.
//
//     angle = pos * f,   (a, b) -> m (a cos - b sin, a sin + b cos)
//
// Memory-bound: every element is read and written once, with three float32
// operations in between.  Measured 7.1 TB/s on the backward of 190,288 tokens x
// 80 heads (1,097 us) and 6.9 on the image mix's 28,672 x 48 (102 us), where a
// plain copy reaches 6.8.  What would cost more than the traffic is the angle,
// so a block computes the cosines and sines of its tokens once, into shared
// memory, and all of their heads use them.  The angle itself is a 64-bit
// fixed-point fraction of a turn, pos * step mod 2^64, exact but for the rounding
// of step itself (made in float64: below 2^-54 of a turn, so 2^-34 at position
// 2^20).  A float32 product pos * f would be off by 2^-24 of all the turns so
// far, and float64 runs on a unit that this GPU has few of.  The top 32 bits go
// to sincospi as a float32, off by 2^-26 of a turn at most.
//
// A thread's unit is 16 columns for bf16, 8 for float32, as two 16-byte loads
// and stores (the two halves' pieces, or two neighbours), so a head's units are
// consecutive threads and a token's heads are one run.  Two units of a thread
// are in flight, the first two while the block makes its cosines.
// Plans whose pairs do not fill such units take units of one pair.
#include "common.cuh"
#include "paged.h"
#include "rope.cuh"

namespace zl {
namespace {

__device__ uint32_t g_rope_err;

constexpr int kRopeThreads = 256;
constexpr int kTokensMax = 2;                  // tokens of a block (4: 1-2% slower, 8: 1-5%)

template <typename T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Where the cosine and sine of pair i stand in their row: units of N pairs are
// read as 16-byte pieces (two pairs) by consecutive threads, whose pieces are
// 8 N bytes apart; swizzled by the unit, eight threads' pieces fall into
// different banks (unswizzled, conflicts filled two thirds of the cycles).
template <int N>
__device__ __forceinline__ int cs_at(int i) {
  if constexpr (N == 1) return i;
  const int unit = i / N, piece = i % N / 2;
  const int swz = N == 8 ? (unit >> 1) & 3 : (unit >> 2) & 1;
  return 2 * (unit * (N / 2) + (piece ^ swz)) + (i & 1);
}

// One unit of a head: N pairs turned, or 2N columns kept (past rot_dim).
// Loading and finishing are apart, so that a thread has two units' loads in
// flight.  VECTOR: N = 8 for bf16, 4 for float32; else one pair.
template <typename T, bool VECTOR, bool INTERLEAVED>
struct Unit {
  static constexpr int N = VECTOR ? Vec16<T>::N : 1;
  T* dst;
  int tl;                    // token of the block
  int unit, half;            // half: pairs that turn, of the whole head
  uint4 x, y;                // VECTOR: the unit's two 16-byte pieces
  float a, b;                // else: its two columns

  __device__ __forceinline__ bool kept() const { return unit * N >= half; }
  __device__ __forceinline__ int first() const { return kept() || INTERLEAVED ? 2 * N * unit : N * unit; }
  __device__ __forceinline__ int second() const { return kept() || INTERLEAVED ? first() + N : first() + half; }

  __device__ __forceinline__ void load(const T* src) {
    if constexpr (VECTOR) {
      x = *reinterpret_cast<const uint4*>(src + first());
      y = *reinterpret_cast<const uint4*>(src + second());
    } else {
      a = as_float(src[first()]);
      b = as_float(src[second()]);
    }
  }

  __device__ __forceinline__ void finish(const float2* cs) {
    if constexpr (VECTOR) {
      if (!kept()) {
        float u[N], v[N];
        Vec16<T>::unpack(x, u);
        Vec16<T>::unpack(y, v);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          // cos, sin of two pairs
          const float4 w = *reinterpret_cast<const float4*>(cs + cs_at<N>(N * unit + i));
          if constexpr (INTERLEAVED) {
            // pairs i, i+1 of the unit: columns 2i .. 2i+3 of the 2N loaded ones
            float* z = 2 * i < N ? u + 2 * i : v + 2 * i - N;
            const float z0 = z[0], z1 = z[1], z2 = z[2], z3 = z[3];
            z[0] = rope_first(z0, z1, w.x, w.y);
            z[1] = rope_second<!VECTOR>(z0, z1, w.x, w.y);
            z[2] = rope_first(z2, z3, w.z, w.w);
            z[3] = rope_second<!VECTOR>(z2, z3, w.z, w.w);
          } else {
            const float a0 = u[i], b0 = v[i], a1 = u[i + 1], b1 = v[i + 1];
            u[i] = rope_first(a0, b0, w.x, w.y);
            v[i] = rope_second<!VECTOR>(a0, b0, w.x, w.y);
            u[i + 1] = rope_first(a1, b1, w.z, w.w);
            v[i + 1] = rope_second<!VECTOR>(a1, b1, w.z, w.w);
          }
        }
        x = Vec16<T>::pack(u);
        y = Vec16<T>::pack(v);
      }
      *reinterpret_cast<uint4*>(dst + first()) = x;
      *reinterpret_cast<uint4*>(dst + second()) = y;
    } else {
      const float2 w = kept() ? make_float2(1.f, 0.f) : cs[unit];
      put(dst + first(), kept() ? a : rope_first(a, b, w.x, w.y));
      put(dst + second(), kept() ? b : rope_second<!VECTOR>(a, b, w.x, w.y));
    }
  }
};

// SEQS: sequences of an append's parameters; 0: no append.  The append of
// 29,764 tokens x 72 heads takes 161 us, 6.8 TB/s.  Five blocks an SM: 1,097 us
// on the backward above, 6 blocks 1,117, 4 the same.
template <typename T, bool VECTOR, bool INTERLEAVED, int SEQS>
__global__ void __launch_bounds__(kRopeThreads, 5)
rope_kernel(const __grid_constant__ RopeArgs<SEQS> a, int tokens_per_block, int heads_per_block) {
  __shared__ __align__(16) float2 cs[kTokensMax][ZL_ROPE_MAX_PAIRS];
  __shared__ int32_t pos_of[kTokensMax];       // append: position in the sequence
  __shared__ int64_t page_row[kTokensMax];     // append: first row of the token's page, + its row; -1: left out
  constexpr bool APPEND = SEQS > 0;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), a.tokens - t0));
  const int half = a.rope.rot_dim / 2;

  if constexpr (APPEND) {
    if (threadIdx.x < nt) {
      const Place at = place_of(a, a.token0 + t0 + threadIdx.x);
      const bool room = !a.status || *a.status == 0;   // else the lengths do not count the new tokens
      const int64_t row = room && at.page >= 0 ? ((static_cast<int64_t>(at.page) * a.nk) << a.page_shift) +
                                                     (at.pos & ((1 << a.page_shift) - 1))
                                               : -1;
      if (row < 0) atomicOr(&g_rope_err, ERR_BAD_PAGE);
      page_row[threadIdx.x] = row;
      pos_of[threadIdx.x] = static_cast<int32_t>(at.pos);
    }
    __syncthreads();
  }
  // The block's units: its tokens' heads [h0, h1), token by token.  A thread
  // takes every kRopeThreads-th and keeps two in flight, the first two over the
  // making of the cosines.
  using U = Unit<T, VECTOR, INTERLEAVED>;
  const int units = a.head_dim / (2 * U::N);   // of a head; a power of two
  const int ushift = 31 - __clz(units);
  const int heads = a.nq + (APPEND ? 2 : 1) * a.nk;
  const int h0 = blockIdx.y * heads_per_block;
  const int per_token = (min(heads, h0 + heads_per_block) - h0) << ushift;
  int tl = 0, x = threadIdx.x;                 // the next unit: of token tl, the x-th
  const auto fetch = [&](U& u) -> bool {
    while (true) {
      while (x >= per_token) {
        x -= per_token;
        ++tl;
      }
      if (tl >= nt) return false;
      const int64_t t = a.token0 + t0 + tl;
      const int h = h0 + (x >> ushift), hk = h - a.nq;
      u.tl = tl;
      u.unit = x & (units - 1);
      u.half = half;
      x += kRopeThreads;
      const T* src;
      if (h < a.nq) {
        if (a.skip_kept && u.kept()) continue;
        src = static_cast<const T*>(a.q) + t * a.q_stride + h * a.head_dim;
        u.dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + h * a.head_dim;
      } else if constexpr (!APPEND) {
        if (a.skip_kept && u.kept()) continue;
        src = static_cast<const T*>(a.k) + t * a.k_stride + hk * a.head_dim;
        u.dst = static_cast<T*>(a.k_out) + t * a.k_out_stride + hk * a.head_dim;
      } else {
        const int64_t row = page_row[u.tl];
        if (row < 0) continue;
        const bool is_v = hk >= a.nk;
        const int hr = is_v ? hk - a.nk : hk;
        if (is_v) u.half = 0;                  // values are copied
        src = is_v ? static_cast<const T*>(a.v) + t * a.v_stride + hr * a.head_dim
                   : static_cast<const T*>(a.k) + t * a.k_stride + hr * a.head_dim;
        u.dst = static_cast<T*>(is_v ? a.v_out : a.k_out) +
                (row + (static_cast<int64_t>(hr) << a.page_shift)) * a.head_dim;
      }
      u.load(src);
      return true;
    }
  };
  U u0, u1;
  bool has0 = fetch(u0);
  bool has1 = fetch(u1);

  for (int y = threadIdx.x; y < nt * half; y += kRopeThreads) {
    const int tp = y / half, i = y - tp * half;
    int64_t p;
    if (APPEND && !a.positions)
      p = pos_of[tp];
    else
      p = a.positions[rope_axis(a.rope, i) * a.pos_stride + a.token0 + t0 + tp];
    cs[tp][cs_at<U::N>(i)] = rope_turn(a.rope, p, i, a.inverse != 0);
  }
  __syncthreads();
  while (has0) {                               // units come in order: no u1 without a u0
    u0.finish(cs[u0.tl]);
    has0 = fetch(u0);
    if (has1) u1.finish(cs[u1.tl]);
    has1 = has0 && fetch(u1);
  }
}

template <int SEQS>
RopeArgs<SEQS> cut(const RopeArgs<kMaxSegs>& a) {
  RopeArgs<SEQS> r;
  static_cast<RopeHead&>(r) = a;
  for (int i = 0; i <= SEQS && i <= a.n_seqs; ++i) r.cu[i] = a.cu[i];
  return r;
}

template <typename T, bool VECTOR, bool INTERLEAVED>
void launch_kind(const RopeArgs<kMaxSegs>& a, dim3 grid, int tpb, int hpb, cudaStream_t stream) {
  if (!a.append) {
    rope_kernel<T, VECTOR, INTERLEAVED, 0><<<grid, kRopeThreads, 0, stream>>>(cut<0>(a), tpb, hpb);
  } else if constexpr (sizeof(T) == 2) {
    if (a.n_seqs <= kFewSegs)
      rope_kernel<T, VECTOR, INTERLEAVED, kFewSegs><<<grid, kRopeThreads, 0, stream>>>(cut<kFewSegs>(a), tpb, hpb);
    else
      rope_kernel<T, VECTOR, INTERLEAVED, kMaxSegs><<<grid, kRopeThreads, 0, stream>>>(a, tpb, hpb);
  }
}

template <typename T>
void launch_type(const RopeArgs<kMaxSegs>& a, bool vec, dim3 grid, int tpb, int hpb, cudaStream_t stream) {
  if (vec && a.rope.interleaved) launch_kind<T, true, true>(a, grid, tpb, hpb, stream);
  else if (vec) launch_kind<T, true, false>(a, grid, tpb, hpb, stream);
  else if (a.rope.interleaved) launch_kind<T, false, true>(a, grid, tpb, hpb, stream);
  else launch_kind<T, false, false>(a, grid, tpb, hpb, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs<kMaxSegs>& a, int num_sms, cudaStream_t stream) {
  const int heads = a.nq + (a.append ? 2 : 1) * a.nk;
  if (a.tokens == 0 || heads == 0) return cudaSuccess;
  const int per_unit = a.elem_bytes == 2 ? 8 : 4;
  const bool vec = !rope_alone(a.rope, a.elem_bytes);
  const int units = a.head_dim / (vec ? 2 * per_unit : 2);
  // Few tokens: one a block, and its heads dealt out to more blocks (each
  // block makes the token's cosines again) until the SMs have a block or two.
  const int tpb = a.tokens >= int64_t(num_sms) * 4 * kTokensMax ? kTokensMax : 1;
  const int64_t blocks = (a.tokens + tpb - 1) / tpb;
  const int fill = (kRopeThreads + units - 1) / units;       // heads that fill a block's threads once
  int hpb = heads;
  while (hpb > fill && blocks * ((heads + hpb - 1) / hpb) < 2 * num_sms) hpb = (hpb + 1) / 2;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + hpb - 1) / hpb));
  if (a.elem_bytes == 2) launch_type<__nv_bfloat16>(a, vec, grid, tpb, hpb, stream);
  else launch_type<float>(a, vec, grid, tpb, hpb, stream);
  return cudaGetLastError();
}

uint32_t rope_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_rope_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_rope_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
