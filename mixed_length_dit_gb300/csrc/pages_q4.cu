// A paged cache held in 4 bits: the append of new tokens, which quantises them
// on the way, and reading tokens back (paged_q4.cuh has the arithmetic).
//
// Memory-bound, like the bf16 append: an append reads 2 bytes a value and writes
// 17/32, reading back the other way round.  A token's head is four threads, each
// with the piece of it that stands together in the pages (8 columns of every
// group of 32), so that a thread has d / 32 loads of 16 bytes in flight, writes
// its codes in one store, finds a group's largest value with two exchanges among
// the four, and (heads of equal halves) turns its columns without asking others.
#include <algorithm>

#include "paged_q4.cuh"
#include "paged.h"
#include "rope.cuh"

namespace zl {
namespace {

__device__ uint32_t g_q4_err;

constexpr int kThreads = 256;
constexpr int kHeads = kThreads / 4;           // heads that a block takes at a time
constexpr int kTokensMax = 8;                  // tokens of a block

template <int HD>
struct Piece {
  static constexpr int G = HD / kQ4Group;
  uint4 x[G];                                  // 8 columns of each group

  __device__ __forceinline__ void load(const __nv_bfloat16* head, int c) {
#pragma unroll
    for (int q = 0; q < G; ++q) x[q] = *reinterpret_cast<const uint4*>(head + 32 * q + 8 * c);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* head, int c) const {
#pragma unroll
    for (int q = 0; q < G; ++q) *reinterpret_cast<uint4*>(head + 32 * q + 8 * c) = x[q];
  }
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// a and b: first and second elements of the pairs with cosines and sines cs[0 .. 7].
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const float2* cs) {
  float u[8], v[8];
  unpack8(a, u);
  unpack8(b, v);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 w = *reinterpret_cast<const float4*>(cs + i);
    const float a0 = u[i], b0 = v[i], a1 = u[i + 1], b1 = v[i + 1];
    u[i] = rope_first(a0, b0, w.x, w.y);
    v[i] = rope_second<false>(a0, b0, w.x, w.y);
    u[i + 1] = rope_first(a1, b1, w.z, w.w);
    v[i + 1] = rope_second<false>(a1, b1, w.z, w.w);
  }
  a = pack8(u);
  b = pack8(v);
}

// Four neighbouring pairs, those with an element at or behind `pairs` kept.
template <bool ALONE>
__device__ __forceinline__ void turn_neighbours(uint4& x, const float2* cs, int pairs) {
  float u[8];
  unpack8(x, u);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < pairs) {
      const float2 w = cs[i];
      const float a = u[2 * i], b = u[2 * i + 1];
      u[2 * i] = rope_first(a, b, w.x, w.y);
      u[2 * i + 1] = rope_second<ALONE>(a, b, w.x, w.y);
    }
  x = pack8(u);
}

// Turns the piece by the token's cosines and sines.  Four threads hold the head,
// `src` is where they loaded it from.
template <int HD>
__device__ __forceinline__ void turn(Piece<HD>& p, const zl_rope_t& r, const float2* cs, const __nv_bfloat16* src,
                                     int c) {
  constexpr int G = Piece<HD>::G;
  const int half = r.rot_dim / 2;
  const bool alone = rope_alone(r, 2);
  if (r.interleaved) {
#pragma unroll
    for (int q = 0; q < G; ++q) {
      const int first = 16 * q + 4 * c;        // pair
      if (first >= half) continue;
      if (alone) turn_neighbours<true>(p.x[q], cs + first, half - first);
      else turn_neighbours<false>(p.x[q], cs + first, half - first);
    }
  } else if (half == 32) {                     // groups q and q + 1
    turn_halves(p.x[0], p.x[1], cs + 8 * c);
  } else if (G == 4 && half == 64) {
#pragma unroll
    for (int q = 0; q < G / 2; ++q) turn_halves(p.x[q], p.x[q + G / 2], cs + 32 * q + 8 * c);
  } else {                                     // the other element is in another piece
#pragma unroll
    for (int q = 0; q < G; ++q) {
      const int j0 = 32 * q + 8 * c;
      if (j0 >= r.rot_dim) continue;
      float u[8];
      unpack8(p.x[q], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i;
        if (j >= r.rot_dim) continue;
        const bool is_first = j < half;
        const float2 w = cs[is_first ? j : j - half];
        const float other = __bfloat162float(src[is_first ? j + half : j - half]);
        u[i] = is_first ? rope_first(u[i], other, w.x, w.y)
               : alone  ? rope_second<true>(other, u[i], w.x, w.y)
                        : rope_second<false>(other, u[i], w.x, w.y);
      }
      p.x[q] = pack8(u);
    }
  }
}

// Quantises a head that four threads hold, and stores it in its row of the block
// of a page's head.
template <int HD>
__device__ __forceinline__ void keep(const Piece<HD>& p, uint8_t* block, int page_size, int row, int c, bool values,
                                     bool store) {
  constexpr int G = Piece<HD>::G;
  // The groups' largest magnitudes, two in a word, over the four threads; thread c
  // then finds the step of group c for all of them.
  uint32_t t[G / 2];
#pragma unroll
  for (int y = 0; y < G / 2; ++y) {
    const uint32_t u = q4_top(p.x[2 * y]), v = q4_top(p.x[2 * y + 1]);
    t[y] = q4_max2(__byte_perm(u, v, 0x5410), __byte_perm(u, v, 0x7632));
    t[y] = q4_max2(t[y], __shfl_xor_sync(0xffffffffu, t[y], 1));
    t[y] = q4_max2(t[y], __shfl_xor_sync(0xffffffffu, t[y], 2));
  }
  const int q0 = c & (G - 1);
  const uint32_t pair = G == 4 && q0 >= 2 ? t[G / 2 - 1] : t[0];
  const uint32_t byte = q4_step_byte(q0 & 1 ? pair >> 16 : pair & 0xffffu);
  const float inv = q4_inverse(byte);
  uint32_t steps = c < G ? byte << (8 * q0) : 0u;
  steps |= __shfl_xor_sync(0xffffffffu, steps, 1);
  steps |= __shfl_xor_sync(0xffffffffu, steps, 2);
  const bool clamp = __any_sync(0xffffffffu, q4_clamps(byte));
  uint32_t w[G];
#pragma unroll
  for (int q = 0; q < G; ++q) w[q] = q4_codes(p.x[q], __shfl_sync(0xffffffffu, inv, q, 4), clamp);
  if (!store) return;
  if (values) q4_order_values(w);
  uint8_t* codes = block + static_cast<int64_t>(row) * kQ4Codes<HD> + c * (4 * G);
  uint8_t* step = block + static_cast<int64_t>(page_size) * kQ4Codes<HD> + row * kQ4Steps<HD>;
  if constexpr (G == 4) {
    *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
    if (c == 0) *reinterpret_cast<uint32_t*>(step) = steps;
  } else {
    *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    if (c == 0) *reinterpret_cast<uint16_t*>(step) = static_cast<uint16_t>(steps);
  }
}

// ------------------------------------------------------------------ append
// TURN: keys and queries are turned, or there are queries to hand on.  The append and
// reading back of 29,764 tokens x 48 heads take 154 us together, 926 MB that a copy
// moves in 136; with the turn's registers in the same kernel, four blocks an SM, 166,
// and with three 180.
template <int HD, bool TURN, int SEQS>
__global__ void __launch_bounds__(kThreads, TURN ? 4 : 6)
append_q4_kernel(const __grid_constant__ RopeArgs<SEQS> a, int tokens_per_block, int heads_per_block,
                 uint32_t heads_inv) {
  __shared__ __align__(16) float2 cs[TURN ? kTokensMax : 1][HD / 2];
  __shared__ int32_t pos_of[kTokensMax];
  __shared__ int32_t page_of[kTokensMax];      // -1: left out
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), a.tokens - t0));
  const int half = TURN ? a.rope.rot_dim / 2 : 0;
  const int nq = TURN ? a.nq : 0;
  const int page_size = 1 << a.page_shift;

  if (threadIdx.x < nt) {
    const Place at = place_of(a, a.token0 + t0 + threadIdx.x);
    const bool room = !a.status || *a.status == 0;     // else the lengths do not count the new tokens
    if (!room || at.page < 0) atomicOr(&g_q4_err, ERR_BAD_PAGE);
    page_of[threadIdx.x] = room ? at.page : -1;
    pos_of[threadIdx.x] = static_cast<int32_t>(at.pos);
  }
  __syncthreads();
  if constexpr (TURN) {
    for (int y = threadIdx.x; y < nt * half; y += kThreads) {
      const int tp = y / half, i = y - tp * half;
      const int64_t p = a.positions ? a.positions[rope_axis(a.rope, i) * a.pos_stride + a.token0 + t0 + tp] : pos_of[tp];
      cs[tp][i] = rope_turn(a.rope, p, i, false);
    }
    __syncthreads();
  }

  const int h0 = blockIdx.y * heads_per_block;
  const int per_token = min(nq + 2 * a.nk, h0 + heads_per_block) - h0;
  const int c = threadIdx.x & 3;
  for (int x0 = 0; x0 < nt * per_token; x0 += kHeads) {        // whole warps: heads exchange among four threads
    const int x = x0 + (threadIdx.x >> 2);
    const bool any = x < nt * per_token;
    // x / heads_per_block (a block of fewer heads has one token); exact, as x times the heads is below 2^32
    const int tl = any && nt > 1 ? static_cast<int>(__umulhi(x, heads_inv)) : 0;
    const int h = any ? h0 + x - tl * per_token : 0;
    const int64_t t = a.token0 + t0 + tl;
    const int kind = h < nq ? 0 : h < nq + a.nk ? 1 : 2;   // query, key, value
    const int hk = h - nq - (kind == 2 ? a.nk : 0);
    const auto* src = static_cast<const __nv_bfloat16*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                      t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                      static_cast<int64_t>(kind == 0 ? h : hk) * HD;
    const int page = page_of[tl];
    const bool store = any && (kind == 0 || page >= 0);
    Piece<HD> p;
    if (store) {
      p.load(src, c);
      if (TURN && half > 0 && kind < 2) turn(p, a.rope, cs[TURN ? tl : 0], src, c);
    } else {
#pragma unroll
      for (int q = 0; q < Piece<HD>::G; ++q) p.x[q] = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();                              // a query turned in place has been read by all four
    if (store && kind == 0) p.store(static_cast<__nv_bfloat16*>(a.q_out) + t * a.q_out_stride + static_cast<int64_t>(h) * HD, c);
    if (__all_sync(0xffffffffu, kind == 0)) continue;
    const int64_t block = static_cast<int64_t>(max(page, 0)) * a.nk + max(hk, 0);
    keep(p, static_cast<uint8_t*>(kind == 2 ? a.v_out : a.k_out) + ((block * kQ4Row<HD>) << a.page_shift), page_size,
         pos_of[tl] & (page_size - 1), c, kind == 2, store && kind > 0);
  }
}

// ------------------------------------------------------------------ reading back
// A token's head is four threads again: d / 8 bytes of codes and all of its steps
// in, 8 columns of each group out.
template <int HD>
__device__ __forceinline__ void give(const uint8_t* block, int page_size, int row, int c, bool values,
                                     __nv_bfloat16* head) {
  constexpr int G = Piece<HD>::G;
  const uint8_t* codes = block + static_cast<int64_t>(row) * kQ4Codes<HD> + c * (4 * G);
  const uint8_t* step = block + static_cast<int64_t>(page_size) * kQ4Codes<HD> + row * kQ4Steps<HD>;
  uint32_t w[G], s;
  if constexpr (G == 4) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(codes));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    s = __ldg(reinterpret_cast<const uint32_t*>(step));
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(codes));
    w[0] = u.x; w[1] = u.y;
    s = __ldg(reinterpret_cast<const uint16_t*>(step));
  }
  if (values) q4_natural_values(w);
#pragma unroll
  for (int q = 0; q < G; ++q)
    *reinterpret_cast<uint4*>(head + 32 * q + 8 * c) = q4_values(w[q], q4_step((s >> (8 * q)) & 0xffu));
}

template <int HD, int SEQS>
__global__ void __launch_bounds__(kThreads)
read_q4_kernel(const __grid_constant__ ReadQ4Args<SEQS> a, int tokens_per_block) {
  __shared__ int32_t row_of[kTokensMax];
  __shared__ int32_t page_of[kTokensMax];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), a.tokens - t0));
  const int page_size = 1 << a.page_shift;
  if (threadIdx.x < nt) {
    const Place at = place_of(a, a.token0 + t0 + threadIdx.x);
    if (at.page < 0) atomicOr(&g_q4_err, ERR_BAD_PAGE);
    page_of[threadIdx.x] = at.page;
    row_of[threadIdx.x] = static_cast<int32_t>(at.pos & (page_size - 1));
  }
  __syncthreads();
  const int per_token = 2 * a.nk, c = threadIdx.x & 3;
  for (int x = threadIdx.x >> 2; x < nt * per_token; x += kHeads) {
    const int tl = x / per_token, h = x - tl * per_token;
    const bool values = h >= a.nk;
    const int hk = values ? h - a.nk : h;
    const int64_t t = a.token0 + t0 + tl;
    __nv_bfloat16* head = static_cast<__nv_bfloat16*>(values ? a.v_out : a.k_out) +
                          t * (values ? a.v_stride : a.k_stride) + static_cast<int64_t>(hk) * HD;
    const int page = page_of[tl];
    if (page < 0) {                            // not in the cache: zeros
#pragma unroll
      for (int q = 0; q < HD / 32; ++q) *reinterpret_cast<uint4*>(head + 32 * q + 8 * c) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint8_t* pool = values ? a.v_pages : a.k_pages;
    give<HD>(pool + (((static_cast<int64_t>(page) * a.nk + hk) * kQ4Row<HD>) << a.page_shift), page_size, row_of[tl], c,
             values, head);
  }
}

// ------------------------------------------------------------------ a chunk's keys and values in bf16
// The attention of many rows reads its sequences' keys and values again and again,
// from L2: they are unpacked once, into pages of kScratchPage tokens, and the bf16
// kernel runs over those.  Block (x, y, z): the x-th page that segment z sees, of
// key head y.
template <int HD, int SEGS>
__global__ void __launch_bounds__(kThreads) unpack_q4_kernel(const __grid_constant__ UnpackQ4Args<SEGS> a) {
  const PagedSeg seg = a.segs[blockIdx.z];
  int len = a.kv_lens[seg.seq];
  if (len < 0 || len > a.max_kv_len) {
    if (threadIdx.x == 0) atomicOr(&g_q4_err, ERR_BAD_PAGE);
    len = len < 0 ? 0 : a.max_kv_len;
  }
  // the first key that the first query sees
  const int first = len - seg.q_len;           // its position
  const int lo = a.window > 0 && first >= a.window ? first - a.window + 1 : 0;
  const int page = lo / kScratchPage + static_cast<int>(blockIdx.x);
  if (page * kScratchPage >= len) return;
  const int64_t to = static_cast<int64_t>(blockIdx.z) * a.seg_pages + blockIdx.x;
  if (threadIdx.x == 0 && blockIdx.y == 0)
    a.table[static_cast<int64_t>(seg.seq) * a.scratch_cols + page] = static_cast<int32_t>(to);
  const int hk = blockIdx.y, c = threadIdx.x & 3;
  const int n = min(kScratchPage, len - page * kScratchPage);
  const int page_size = 1 << a.page_shift;
  const int32_t* row = a.page_table + static_cast<int64_t>(seg.seq) * a.table_cols;
#pragma unroll 4
  for (int x = threadIdx.x >> 2; x < 2 * kScratchPage; x += kHeads) {
    const int i = x & (kScratchPage - 1);
    if (i >= n) continue;
    const int pos = page * kScratchPage + i;
    int from = pos >> a.page_shift < a.table_cols ? __ldg(row + (pos >> a.page_shift)) : -1;
    if (from < 0 || from >= a.num_pages) {     // reads page 0 in its place
      atomicOr(&g_q4_err, ERR_BAD_PAGE);
      from = 0;
    }
    const bool values = x >= kScratchPage;
    auto* head = static_cast<__nv_bfloat16*>(values ? a.v_out : a.k_out) +
                 ((to * a.nk + hk) * kScratchPage + i) * HD;
    give<HD>((values ? a.v_pages : a.k_pages) + (((static_cast<int64_t>(from) * a.nk + hk) * kQ4Row<HD>) << a.page_shift),
             page_size, pos & (page_size - 1), c, values, head);
  }
}

// The head and the first n sequences' entries of a launch's arguments.
template <int N, template <int> class A>
A<N> cut_cu(const A<kMaxSegs>& a) {
  A<N> r;
  static_cast<typename A<N>::Head&>(r) = a;
  for (int i = 0; i <= a.n_seqs; ++i) r.cu[i] = a.cu[i];
  return r;
}

// Tokens of a block: so many that its threads have a few heads each, once there
// are blocks for every SM several times over.
int tokens_of_block(int64_t tokens, int heads, int num_sms) {
  int n = 1;
  while (n < kTokensMax && n * heads < 2 * kHeads && tokens / (2 * n) >= 4 * num_sms) n *= 2;
  return n;
}

template <int HD, bool TURN>
void launch_append(const RopeArgs<kMaxSegs>& a, dim3 grid, int tpb, int hpb, cudaStream_t stream) {
  const uint32_t inv = static_cast<uint32_t>((uint64_t(1) << 32) / hpb + 1);
  if (a.n_seqs <= kFewSegs)
    append_q4_kernel<HD, TURN, kFewSegs><<<grid, kThreads, 0, stream>>>(cut_cu<kFewSegs>(a), tpb, hpb, inv);
  else
    append_q4_kernel<HD, TURN, kMaxSegs><<<grid, kThreads, 0, stream>>>(a, tpb, hpb, inv);
}

}  // namespace

cudaError_t launch_append_q4(const RopeArgs<kMaxSegs>& a, int num_sms, cudaStream_t stream) {
  const int heads = a.nq + 2 * a.nk;
  const int tpb = tokens_of_block(a.tokens, heads, num_sms);
  const int64_t blocks = (a.tokens + tpb - 1) / tpb;
  int hpb = heads;                             // few tokens: a token's heads are dealt out to more blocks
  while (hpb > kHeads && blocks * ((heads + hpb - 1) / hpb) < 2 * num_sms) hpb = (hpb + 1) / 2;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + hpb - 1) / hpb));
  const bool turn = a.rope.rot_dim > 0 || a.nq > 0;
  if (a.head_dim == 64)
    turn ? launch_append<64, true>(a, grid, tpb, hpb, stream) : launch_append<64, false>(a, grid, tpb, hpb, stream);
  else
    turn ? launch_append<128, true>(a, grid, tpb, hpb, stream) : launch_append<128, false>(a, grid, tpb, hpb, stream);
  return cudaGetLastError();
}

cudaError_t launch_read_q4(const ReadQ4Args<kMaxSegs>& a, int num_sms, cudaStream_t stream) {
  const int tpb = tokens_of_block(a.tokens, 2 * a.nk, num_sms);
  const unsigned grid = static_cast<unsigned>((a.tokens + tpb - 1) / tpb);
  const bool few = a.n_seqs <= kFewSegs;
  if (a.head_dim == 64) {
    if (few) read_q4_kernel<64, kFewSegs><<<grid, kThreads, 0, stream>>>(cut_cu<kFewSegs>(a), tpb);
    else read_q4_kernel<64, kMaxSegs><<<grid, kThreads, 0, stream>>>(a, tpb);
  } else {
    if (few) read_q4_kernel<128, kFewSegs><<<grid, kThreads, 0, stream>>>(cut_cu<kFewSegs>(a), tpb);
    else read_q4_kernel<128, kMaxSegs><<<grid, kThreads, 0, stream>>>(a, tpb);
  }
  return cudaGetLastError();
}

cudaError_t launch_unpack_q4(int head_dim, const UnpackQ4Args<kMaxSegs>& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.seg_pages), static_cast<unsigned>(a.nk), static_cast<unsigned>(a.n_segs));
  if (a.n_segs <= kFewSegs) {
    UnpackQ4Args<kFewSegs> r;
    static_cast<UnpackQ4Head&>(r) = a;
    for (int i = 0; i < a.n_segs; ++i) r.segs[i] = a.segs[i];
    if (head_dim == 64) unpack_q4_kernel<64><<<grid, kThreads, 0, stream>>>(r);
    else unpack_q4_kernel<128><<<grid, kThreads, 0, stream>>>(r);
  } else {
    if (head_dim == 64) unpack_q4_kernel<64><<<grid, kThreads, 0, stream>>>(a);
    else unpack_q4_kernel<128><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

uint32_t pages_q4_take_error() {
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_q4_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0) cudaMemcpyToSymbol(g_q4_err, &zero, sizeof(zero));
  return v;
}

}  // namespace zl
