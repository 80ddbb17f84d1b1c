// Internal interface between the host entries of the paged cache
// (zl_paged.cpp) and its kernels.  Not part of the public C ABI.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "zl_attn.h"

namespace zl {

// A launch carries its sequences by value.  Most calls have few, and a launch
// pays for every byte of its parameters, so each kernel exists for kFewSegs
// sequences and for kMaxSegs.
constexpr int kFewSegs = 64;

// One launch of rotary positions.  As rope_fwd / rope_bwd it turns `q` and
// `k` into `q_out` and `k_out` at given positions; as paged_append (`append`
// set) the keys go into the cache's pages, the values beside them, and the
// positions follow from the cache's lengths unless they are given.
struct RopeHead {
  const void* q;
  const void* k;
  const void* v;                // append only
  void* q_out;
  void* k_out;                  // append: the key pages
  void* v_out;                  // append: the value pages
  const int32_t* positions;     // [n_axes][pos_stride], or null (append)
  int64_t pos_stride;
  int64_t q_stride, k_stride, v_stride;          // elements between tokens
  int64_t q_out_stride, k_out_stride;
  int64_t token0;               // first token of this launch
  int64_t tokens;               // tokens of this launch
  int32_t nq, nk;               // query heads, key heads
  int32_t head_dim;
  int32_t inverse;              // turn by the negative angle (the transpose)
  int32_t elem_bytes;           // 2: bf16, 4: float32
  int32_t append;
  int32_t skip_kept;            // q and k are turned in place: unrotated columns stay
  // append: the cache
  const int32_t* page_table;    // [seqs][table_cols]
  const int32_t* kv_lens;       // [seqs]
  const int32_t* status;        // or null; not 0: nothing is appended
  int32_t table_cols;
  int32_t num_pages;
  int32_t page_shift;
  int32_t n_seqs;               // sequences of this launch
  int32_t seq0;                 // table row of the launch's first sequence
  zl_rope_t rope;
};

// N sequences; N = 0: no append.
template <int N>
struct RopeArgs : RopeHead {
  using Head = RopeHead;
  int32_t cu[N + 1];            // append: first token of each sequence of the launch
};
static_assert(sizeof(RopeArgs<kMaxSegs>) <= 32764, "rotary arguments exceed the kernel parameter space");

// CTAs of a paged attention launch, one for each of this GPU's SMs; each takes
// an equal share of the call's key blocks.  A row has a part from as many of
// them as its keys are spread over.
constexpr int kPagedCtas = 152;
constexpr int kMaxParts = kPagedCtas;

// One sequence's queries in a paged attention launch.
struct PagedSeg {
  int32_t seq;       // row of the page table and of the lengths
  int32_t q_row0;    // packed row of its first query
  int32_t q_len;     // queries, >= 1
};

// The unit (query tiles from tile0 on of a key head) that begins in a CTA and
// goes on in the CTAs up to `last` (-1: none).
struct PagedJoin {
  int32_t q_row0;
  int32_t q_len;
  int32_t hk;
  int32_t tile0;
  int32_t last;
};

struct PagedAttnHead {
  const int32_t* page_table;
  const int32_t* kv_lens;
  void* o;                      // [Tq][H][d] bf16
  float* lse;                   // [H][lse_stride]
  // parts of rows whose keys were split: 2 * CTAs slots of slot_rows rows (a
  // chunk's two tiles: 128 * tile + row; else token * group + head)
  float* o_part;                // [rows][d]
  float* lse_part;              // [rows]
  PagedJoin* joins;             // [CTAs]
  int64_t lse_stride;           // Tq
  int32_t num_heads;
  int32_t num_kv_heads;
  int32_t group;                // query heads of a key head
  int32_t group_inv;            // 65536 / group, rounded up
  int32_t tile_tokens;          // tokens of a query tile: 128 / group
  int32_t slot_rows;            // rows of a slot
  int32_t table_cols;
  int32_t num_pages;
  int32_t page_shift;
  int32_t max_kv_len;
  int32_t causal;
  int32_t window;
  float scale_log2;             // softmax scale * log2(e)
  int32_t n_segs;
  int32_t whole;                // > 0: the launch's units, of kFewSegs sequences at most; each has a CTA
                                // to itself and no join follows

#ifdef __CUDACC__
  // The token of a tile's row, row / group: exact for rows and groups up to
  // 128, because row * (group * group_inv - 65536) < 128 * 128 < 65536.
  __device__ __forceinline__ int row_token(int row) const { return (row * group_inv) >> 16; }
#endif
};

template <int N>
struct PagedAttnArgs : PagedAttnHead {
  PagedSeg segs[N];
};

// Tensor maps: q[i] takes the tokens of a tile that holds 1, 2 or 4 copies of
// its rows (boxes of 64 columns x group heads x 128 / copies / group tokens),
// o stores a tile like q[0]; k and v see a pool as rows of one head of one
// token (boxes of 64 columns x min(page, 128) rows).
struct PagedMaps {
  CUtensorMap q[3];
  CUtensorMap k, v, o;
};
static_assert(sizeof(PagedAttnArgs<kMaxSegs>) + sizeof(PagedMaps) <= 32764, "paged attention arguments exceed the kernel parameter space");

// Tokens read back from a cache held in 4 bits.
struct ReadQ4Head {
  const uint8_t* k_pages;       // [num_pages][nk] blocks of page_size tokens
  const uint8_t* v_pages;
  const int32_t* page_table;    // [seqs][table_cols]
  const int32_t* kv_lens;       // [seqs]
  void* k_out;                  // [T][nk][d] bf16
  void* v_out;
  int64_t k_stride, v_stride;   // elements between tokens
  int64_t token0;               // first token of this launch
  int64_t tokens;               // tokens of this launch
  int32_t nk;
  int32_t head_dim;
  int32_t table_cols;
  int32_t num_pages;
  int32_t page_shift;
  int32_t n_seqs;               // sequences of this launch
  int32_t seq0;                 // table row of the launch's first sequence
};

template <int N>
struct ReadQ4Args : ReadQ4Head {
  using Head = ReadQ4Head;
  int32_t cu[N + 1];            // first token of each sequence of the launch
};

// Sequences of a 4-bit cache unpacked for the bf16 attention: what each one's
// queries see goes to seg_pages pages of kScratchPage tokens of its own.
constexpr int kScratchPage = kBlockN;

struct UnpackQ4Head {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const int32_t* page_table;    // [seqs][table_cols]
  const int32_t* kv_lens;       // [seqs]
  void* k_out;                  // [segs * seg_pages][nk][kScratchPage][d] bf16
  void* v_out;
  int32_t* table;               // [seqs][scratch_cols]: the pages' numbers among those
  int32_t nk;
  int32_t table_cols;
  int32_t num_pages;
  int32_t page_shift;
  int32_t max_kv_len;
  int32_t window;
  int32_t seg_pages;
  int32_t scratch_cols;
  int32_t n_segs;
};

template <int N>
struct UnpackQ4Args : UnpackQ4Head {
  PagedSeg segs[N];
};

// A launch of the attention of few rows over a 4-bit cache.  A CTA's piece of the
// line of units: it begins `off` into the unit (seg, hk, rt).
struct Q4Piece {
  int32_t seg, hk, rt;
  int32_t off;
  int64_t left;                 // its length
  int64_t per;                  // of every CTA
};

// The unit (rows from row0 on) that begins in a CTA and goes on in the CTAs up to
// `last` (-1: none).
struct Q4Join {
  int32_t q_row0;
  int32_t row0;
  int32_t rows;
  int32_t hk;
  int32_t last;
};

struct AttnQ4Head {
  const __nv_bfloat16* q;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const int32_t* page_table;
  const int32_t* kv_lens;
  __nv_bfloat16* o;             // [Tq][H][d]
  float* lse;                   // [H][lse_stride]
  float* o_part;                // [2 * CTAs][rows of a unit][d]: slots of cut units
  float* lse_part;
  Q4Join* joins;                // [CTAs]
  int64_t q_stride;
  int64_t lse_stride;
  int32_t page_bytes;           // of a pool's page, all heads
  int32_t num_heads;
  int32_t num_kv_heads;
  int32_t group;                // query heads of a key head
  int32_t group_inv;            // 65536 / group, rounded up
  int32_t table_cols;
  int32_t num_pages;
  int32_t page_shift;
  int32_t max_kv_len;
  int32_t causal;
  int32_t window;
  float scale_log2;             // softmax scale * log2(e)
  int32_t n_segs;
  int32_t whole;                // > 0: the launch's units; each has `share` CTAs, a cluster, to itself, and no
                                // join follows
  int32_t share;                // else 1

#ifdef __CUDACC__
  // The token of a sequence's row, row / group: exact for rows below 512 and groups
  // up to 128, because row * (group * group_inv - 65536) < 512 * 128.
  __device__ __forceinline__ int row_token(int row) const { return (row * group_inv) >> 16; }
#endif
};

template <int N>
struct AttnQ4Args : AttnQ4Head {
  PagedSeg segs[N];
};

// A pool of pages seen by the kernels that move whole pages.
struct PagePool {
  uint8_t* base;                // groups x num_pages x page_bytes
  int64_t page_bytes;           // multiple of 16
  int64_t group_stride;         // bytes between groups
  int32_t groups;
  int32_t num_pages;
};

struct PageTable {
  int32_t* table;               // [slots][cols]
  int32_t* kv_lens;             // [slots]
  int32_t* refs;                // [num_pages]
  int32_t slots;
  int32_t cols;
  int32_t num_pages;
  int32_t page_shift;
};

// Most slots a page operation handles (their page counts are scanned in one
// CTA's shared memory).
constexpr int kMaxSlots = 8192;

// Scratch of fork and compact, in int32 words: a header, per-fork lengths,
// the list of page moves and, for compact, the page renumbering.
constexpr int kPageHeader = 64;
inline size_t pages_workspace_words(int64_t num_pages) {
  return kPageHeader + kMaxSlots + 3 * static_cast<size_t>(num_pages);
}

// Takes the head's sequences from args.cu when args.append is set.
cudaError_t launch_rope(const RopeArgs<kMaxSegs>& args, int num_sms, cudaStream_t stream);
// pair: sequences of more than one query tile each; else of one.
cudaError_t launch_paged_attn(int head_dim, bool pair, const PagedMaps& maps, const PagedAttnArgs<kMaxSegs>& args,
                              cudaStream_t stream);
// Joins the split rows of a launch_paged_attn with the same arguments.
cudaError_t launch_paged_join(int head_dim, bool pair, const PagedAttnHead& args, cudaStream_t stream);
// As launch_rope with args.append, into a cache held in 4 bits.
cudaError_t launch_append_q4(const RopeArgs<kMaxSegs>& args, int num_sms, cudaStream_t stream);
cudaError_t launch_read_q4(const ReadQ4Args<kMaxSegs>& args, int num_sms, cudaStream_t stream);
cudaError_t launch_unpack_q4(int head_dim, const UnpackQ4Args<kMaxSegs>& args, cudaStream_t stream);
// nt: tiles of 8 rows in a unit, 1 or 2; attn_q4_ctas: CTAs of such a launch.
int attn_q4_ctas();
cudaError_t launch_attn_q4(int head_dim, int nt, const AttnQ4Args<kMaxSegs>& args, cudaStream_t stream);
// Joins the cut units of a launch_attn_q4 with the same arguments.
cudaError_t launch_join_q4(int head_dim, int nt, const AttnQ4Head& args, cudaStream_t stream);
cudaError_t launch_pages_copy(const PagePool& pool, const int32_t* src, const int32_t* dst, int32_t n, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_pages_extend(const PageTable& t, const int32_t* counts, int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_free(const PageTable& t, const int32_t* slots, int32_t n, cudaStream_t stream);
cudaError_t launch_pages_truncate(const PageTable& t, const int32_t* lens, cudaStream_t stream);
cudaError_t launch_pages_fork_plan(const PageTable& t, const int32_t* parents, const int32_t* children, int32_t n,
                                   int32_t* ws, int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_fork_move(const PagePool& pool, const PageTable& t, const int32_t* parents,
                                   const int32_t* children, int32_t n, const int32_t* ws, int num_sms,
                                   cudaStream_t stream);
cudaError_t launch_pages_compact_plan(const PageTable& t, int32_t* ws, int32_t* live, cudaStream_t stream);
cudaError_t launch_pages_compact_move(const PagePool& pool, const PageTable& t, const int32_t* ws, int num_sms,
                                      cudaStream_t stream);

// Error words of these kernels (read and cleared; synchronous), and all of
// them in one (0xFFFFFFFF: a CUDA call failed).  kErrBadPage is the bit of
// page numbers, slots and lengths outside the cache.
constexpr uint32_t kErrBadPage = 32u;
uint32_t rope_take_error();
uint32_t pages_take_error();
uint32_t paged_attn_take_error();
uint32_t pages_q4_take_error();
uint32_t attn_q4_take_error();
uint32_t paged_take_error();

}  // namespace zl
