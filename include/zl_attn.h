/*
 * zl_attn.h -- C ABI of the coalesced varlen attention library (libzl_attn.so).
 *
 * The operation is the attention call of the Coalesced Attention Engine in
 * Zellige, "Moldable Sequence Placement for Mixed Image-Video DiT Training"
 * (arXiv 2608.01150v1), §IV-D: all whole sequences of one GPU are packed into
 * ONE block-diagonal softmax-attention call that keeps the sequences separate
 * and returns outputs in input order, and shards of split long sequences run
 * alongside them.  Per sequence s and head h (full bidirectional attention,
 * §II-A, no mask):
 *
 *     S   = Q_s K_s^T * scale
 *     O_s = softmax(S) V_s            (row-wise softmax)
 *     LSE = log(sum_j exp(S_ij))      (natural log, one value per query row)
 *
 * Conventions shared by every entry point
 *   - Packed token layout.  Q/O are [Tq, H, d] and K/V are [Tk, H, d],
 *     row-major, d contiguous.  Sequence s owns query rows
 *     [cu_seqlens_q[s], cu_seqlens_q[s+1]) and key rows
 *     [cu_seqlens_k[s], cu_seqlens_k[s+1]).  Tq = cu_seqlens_q[num_seqs].
 *   - LSE buffers are head-major: lse[h * Tq + row], float32.
 *   - cu_seqlens_* and tile tables are HOST arrays (int32, num_seqs + 1
 *     entries, cu[0] = 0, non-decreasing).  All other pointers are DEVICE
 *     pointers of the current CUDA device, 16-byte aligned.
 *   - Every device buffer must hold the size the batch implies (Tq or Tk
 *     rows of H * d elements, H * Tq LSE values, the queried workspace
 *     bytes).  The library sees pointers, not allocations, so it cannot
 *     check this: a shorter buffer is read or written past its end.  The
 *     Python binding checks it against the tensors' shapes before each call.
 *   - The caller owns every buffer.  The library never calls cudaMalloc and
 *     allocates no device memory per call: scratch comes from the caller's
 *     `workspace` (zl_varlen_attn_bwd_static alone uses a fixed 64 MiB
 *     array in the library's device image instead, reserved on each device
 *     the library is loaded on).  On the host, calls build small std::vector
 *     tables (the schedule, the tile grid) and, while zl_profile_begin is
 *     active, create two CUDA events per launch.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and return after enqueue.  Arguments are validated on the host
 *     before anything is enqueued; an invalid call returns an error and leaves
 *     every output untouched.  Device-side faults surface through
 *     zl_sync_check().
 *   - Every entry point returns a zl_status (0 = success, < 0 = error) and
 *     never aborts the process.
 *   - Thread-safe.  Global state: a per-device cache of device attributes
 *     (SM count, the merge kernels' resident blocks per SM), a process-wide
 *     launch counter, the optional profiling hook (zl_profile_*), one device
 *     error word per kernel family (set by a kernel that gave up a wait, read
 *     and cleared by zl_sync_check) and zl_varlen_attn_bwd_static's scratch
 *     array.
 */
#ifndef ZL_ATTN_H
#define ZL_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ZL_OK = 0,
  ZL_EINVAL = -1,        /* malformed arguments (sizes, cu_seqlens, tile table) */
  ZL_EUNSUPPORTED = -2,  /* valid but not implemented (head_dim, dtype, mode)   */
  ZL_EALIGN = -3,        /* a device pointer is not 16-byte aligned             */
  ZL_EWORKSPACE = -4,    /* workspace missing or smaller than required          */
  ZL_ECUDA = -5,         /* a CUDA runtime/driver call failed                   */
  ZL_ETIMEOUT = -6,      /* a kernel gave up a bounded wait (reported by
                            zl_sync_check)                                      */
  ZL_ENODEVICE = -7,     /* no usable sm_103 device                             */
  ZL_EPAGE = -8          /* a kernel met a page number, slot or length outside
                            the cache (reported by zl_sync_check)               */
} zl_status;

typedef enum {
  ZL_BF16 = 0,           /* bf16 inputs/outputs, float32 accumulation, tensor cores */
  ZL_FP32 = 1            /* float32 inputs/outputs, float32 SIMT arithmetic         */
} zl_dtype;

/*
 * One (query-chunk x head-range x KV-chunk) tile of a split sequence.
 * Zellige §IV-A gives every sequence a parallelism configuration (q, h, k):
 * split factors along the query axis (all-gather), the head axis (Ulysses) and
 * the key/value axis (ring), composable, (1, 1, 1) meaning whole; §IV-D runs
 * the shards of split sequences alongside whole ones, and §II-B / Table II
 * describe how a key-split sequence's attention is accumulated exactly from
 * its K/V blocks.  A tile is one shard of such a configuration.  Offsets are
 * relative to the sequence's own query and key ranges; heads are absolute.
 *
 * The tiles of a sequence must form a full grid: n_h_chunks x n_q_chunks x
 * n_kv_chunks tiles, one per (h_chunk, q_chunk, kv_chunk), whose head ranges
 * partition [0, H), whose query ranges partition the sequence's queries and
 * whose key ranges partition its keys (every tile with the same h_chunk has
 * the same head range, every tile with the same q_chunk the same query range,
 * every tile with the same kv_chunk the same key range; chunk ranges
 * contiguous, in chunk order, none empty).  A sequence listed in the tile
 * table is not also run whole.  A sequence with n_kv_chunks = 1 (a (q, h, 1)
 * configuration) needs no merge: its tiles write o and lse directly.
 *
 * h_len = 0 selects all H heads (h_start and h_chunk must then be 0), so a
 * zero-initialised head range means "not split by heads".
 */
typedef struct {
  int32_t seq;          /* index into cu_seqlens_q / cu_seqlens_k             */
  int32_t q_start;      /* first query of the chunk, relative to the sequence */
  int32_t q_len;        /* >= 1                                               */
  int32_t k_start;      /* first key of the chunk, relative to the sequence   */
  int32_t k_len;        /* >= 1                                               */
  int32_t q_chunk;      /* 0 .. n_q_chunks-1                                  */
  int32_t kv_chunk;     /* 0 .. n_kv_chunks-1: the partial slot it writes     */
  int32_t n_kv_chunks;  /* same for every tile of the sequence, 1 .. 64       */
  int32_t h_start;      /* first head of the tile's head range                */
  int32_t h_len;        /* heads in the range, 0 = all H heads                */
  int32_t h_chunk;      /* 0 .. n_h_chunks-1                                  */
} zl_tile_t;

/* Human-readable name of a status code (static string, never NULL). */
const char* zl_status_string(int32_t status);

/* ABI version of this header: (major << 16) | minor.  2.0: head-sharded
 * tiles; 2.1 adds ZL_FWD_BF16_PARTIALS, zl_lse_merge_ex and the schedule
 * queries; 2.2 adds rotary positions (zl_rope_*) and the paged key/value cache
 * (zl_paged_*, zl_pages_*); 2.3 adds zl_paged_append_ex (no existing entry
 * changed). */
int32_t zl_version(void);

/*
 * Workspace needed by zl_varlen_attn_fwd for this batch, in bytes (0 when no
 * sequence is split along its keys).  It holds the float32 shard partials:
 * for the sequences with n_kv_chunks > 1 (in sequence order, R = sum of their
 * query lengths, P = largest n_kv_chunks) an O partial [P][R][H][d] and an
 * LSE partial [P][H][R], then the fused-merge arrival counters.  Under
 * ZL_FWD_BF16_PARTIALS the O partial holds bf16 elements in the first half
 * of the same region; the size is the same.
 * Same argument rules as zl_varlen_attn_fwd.  Writes the size to *bytes.
 */
zl_status zl_varlen_attn_fwd_workspace_size(
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, const zl_tile_t* tiles, int32_t num_tiles,
    size_t* bytes);

/* One work item of the forward, as zl_varlen_attn_fwd_schedule reports it. */
typedef struct {
  int32_t launch;   /* forward launch of the call that runs it (a call with more
                       segments than one launch's parameters hold makes several) */
  int32_t seq;      /* sequence index                                          */
  int32_t tile;     /* index into the caller's tile table; -1: the whole sequence */
  int32_t head;     /* head                                                     */
  int32_t q_start;  /* first query row, relative to the sequence                */
  int32_t q_len;    /* query rows (up to 256 for ZL_BF16, 128 for ZL_FP32)      */
  int32_t k_start;  /* first key of the rows' key range, relative to the sequence */
  int32_t k_len;    /* keys every row of the item attends to                    */
} zl_work_item_t;

/*
 * The forward's work items for this batch, host only (no device work): the
 * tile scheduler of the Coalesced Attention Engine (Zellige §IV-D orders the
 * call's segments stably; §IV-C fills in decreasing price) as this library
 * applies it on one GPU.  Segments -- whole sequences and tiles -- are stably
 * ordered by decreasing key count (ties in input order); each splits into
 * items head by head, query block fastest; items run in this order, every SM
 * taking the next one when it is ready.  Writes the first max_items items to
 * `items` (host; may be NULL when max_items is 0) and their total to
 * *n_items.  Same argument rules and errors as zl_varlen_attn_fwd; `dtype`
 * selects the item size (256 query rows for ZL_BF16, 128 for ZL_FP32).
 */
zl_status zl_varlen_attn_fwd_schedule(
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, int32_t dtype,
    const zl_tile_t* tiles, int32_t num_tiles,
    zl_work_item_t* items, int64_t max_items, int64_t* n_items);

/*
 * Forward of the coalesced block-diagonal attention (Zellige §IV-D).
 *
 * q [Tq,H,d], k/v [Tk,H,d]     inputs, dtype `dtype`, device
 * cu_seqlens_q, cu_seqlens_k   host, num_seqs + 1 entries each
 * num_heads H >= 1, head_dim d in {64, 128}
 * softmax_scale                > 0; pass 1/sqrt(d) for the usual scaling
 * tiles, num_tiles             host tile table (may be NULL when 0)
 * o [Tq,H,d]                   output, same dtype as the inputs
 * lse [H,Tq]                   output, float32, natural log
 * workspace                    device, >= zl_varlen_attn_fwd_workspace_size
 *
 * Whole sequences and every tile run in one persistent launch whose work
 * items (sequence-or-tile x head of its range x query block) are ordered
 * longest first, ties in input order; each SM takes the next item of that
 * order when it is ready for one, so the launch balances itself.  It shares
 * the GPU safely with concurrent launches on other streams.  Tiles of key-split sequences write
 * float32 partials into the workspace, and a merge launch per such sequence
 * (zl_lse_merge's kernel) then combines each query row's partials into o and
 * lse exactly; tiles of sequences split only by queries and heads write o and
 * lse directly.  A sequence with queries but no keys is rejected (ZL_EINVAL);
 * zero-length sequences are skipped.
 */
zl_status zl_varlen_attn_fwd(
    const void* q, const void* k, const void* v,
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, int32_t dtype, float softmax_scale,
    const zl_tile_t* tiles, int32_t num_tiles,
    void* o, float* lse,
    void* workspace, size_t workspace_bytes, void* stream);

/* Flags of zl_varlen_attn_fwd_ex. */
enum {
  /* Merge the tile partials inside the forward launch: each tile counts
   * itself per (128-query block, head) after writing its partial, and the
   * tile that completes the set merges the partials of those rows (exact, as
   * zl_lse_merge; no waiting).  Saves the merge launch; measured slower than
   * the separate merge on the long-video batches, because the merging CTA's
   * tensor pipeline idles meanwhile.  bf16 only (ignored for ZL_FP32). */
  ZL_FWD_FUSED_MERGE = 1,
  /* Tiles of key-split sequences write their partial O rows in bf16 instead
   * of float32 (partial LSEs stay float32), which halves the bytes the
   * partials move through HBM, and the merge (separate or fused) reads them
   * back in bf16 and accumulates in float32.  Each partial row is rounded to
   * bf16 once before the merge: an added error of at most 2^-9 of each
   * partial's magnitude, inside the bf16 output's own rounding budget.  The
   * workspace is the same (its float32 size is an upper bound).  bf16 only
   * (ignored for ZL_FP32). */
  ZL_FWD_BF16_PARTIALS = 2
};

/*
 * zl_varlen_attn_fwd with option flags (a bitwise OR of ZL_FWD_* values; 0
 * gives exactly zl_varlen_attn_fwd).  Same arguments, layouts and workspace
 * otherwise.
 */
zl_status zl_varlen_attn_fwd_ex(
    const void* q, const void* k, const void* v,
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, int32_t dtype, float softmax_scale,
    const zl_tile_t* tiles, int32_t num_tiles,
    void* o, float* lse,
    void* workspace, size_t workspace_bytes, void* stream, uint32_t flags);

/*
 * Exact merge of partial attention results over disjoint key sets: the
 * accumulation step of block-wise (ring / all-gather) attention in Zellige
 * §II-B and Table II.  For every query row r and head h:
 *
 *     lse = log(sum_p exp(lse_p))
 *     o   = sum_p exp(lse_p - lse) * o_p
 *
 * A row whose partials all have lse_p = -inf gets o = 0, lse = -inf.
 *
 * o_partial    device float32, part p row r head h at
 *              ((p * part_stride_rows + r) * H + h) * d
 * lse_partial  device float32, at (p * H + h) * part_stride_rows + r
 * n_parts      1 .. 64;  rows >= 0;  part_stride_rows >= rows
 * o            device, [rows][H][d] in out_dtype (ZL_BF16: round to nearest
 *              even; ZL_FP32)
 * lse          device float32, at h * lse_head_stride + r; lse_head_stride
 *              >= rows
 * Memory-bound; one launch.
 */
zl_status zl_lse_merge(
    const float* o_partial, const float* lse_partial, int32_t n_parts,
    int64_t rows, int32_t num_heads, int32_t head_dim, int64_t part_stride_rows,
    void* o, int32_t out_dtype, float* lse, int64_t lse_head_stride, void* stream);

/*
 * zl_lse_merge with the partial O rows in part_dtype: ZL_FP32 (exactly
 * zl_lse_merge) or ZL_BF16 (the same layout in bf16 elements, as written by
 * the forward under ZL_FWD_BF16_PARTIALS).  lse_partial stays float32 and
 * the accumulation is float32 either way.  Other part_dtype values give
 * ZL_EUNSUPPORTED; the other arguments and errors are zl_lse_merge's.
 */
zl_status zl_lse_merge_ex(
    const void* o_partial, int32_t part_dtype, const float* lse_partial, int32_t n_parts,
    int64_t rows, int32_t num_heads, int32_t head_dim, int64_t part_stride_rows,
    void* o, int32_t out_dtype, float* lse, int64_t lse_head_stride, void* stream);

/*
 * Workspace needed by zl_varlen_attn_bwd, in bytes: a float32 dQ accumulator
 * [Tq][H][d] and the float32 row term D = rowsum(dO * O) [H][Tq].
 */
zl_status zl_varlen_attn_bwd_workspace_size(
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, size_t* bytes);

/* One work item of the backward, as zl_varlen_attn_bwd_schedule reports it. */
typedef struct {
  int32_t launch;   /* backward launch of the call that runs it                */
  int32_t seq;      /* sequence index                                          */
  int32_t head;     /* head                                                     */
  int32_t k_start;  /* first key of the item's key block, relative to the sequence */
  int32_t k_len;    /* keys of the block (up to 128)                            */
  int32_t q_len;    /* query rows the block visits: all of the sequence's       */
} zl_bwd_work_item_t;

/*
 * The backward's work items for this batch, host only (no device work).
 * The backward of a split sequence is the sum over its tiles, i.e. the
 * backward of the whole sequence, so every sequence runs whole; sequences
 * are stably ordered by decreasing query count (the rows each of their key
 * blocks visits), each splits into 128-key blocks head by head, key block
 * fastest, and the items run in this order, every SM taking the next one
 * when it is ready.  Writes the first max_items items to `items` (host; may
 * be NULL when max_items is 0) and their total to *n_items.  Same argument
 * rules and errors as zl_varlen_attn_bwd's batch description (cu_seqlens,
 * heads, head_dim, tiles).
 */
zl_status zl_varlen_attn_bwd_schedule(
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, const zl_tile_t* tiles, int32_t num_tiles,
    zl_bwd_work_item_t* items, int64_t max_items, int64_t* n_items);

/*
 * Backward of zl_varlen_attn_fwd: the analytic gradient of
 * O = softmax(Q K^T * scale) V per sequence and head (the paper trains with
 * exact backward, §V-A; the formula is plain calculus):
 *
 *     P  = exp(S - LSE)      (recomputed from the forward's LSE)
 *     D  = rowsum(dO * O)
 *     dV = P^T dO,   dS = P * (dO V^T - D),
 *     dQ = scale * dS K,   dK = scale * dS^T Q
 *
 * q, k, v, o, dout    device, dtype `dtype` (ZL_BF16 only), layouts as above
 * lse                 device float32 [H][Tq] from the forward
 * tiles               the forward's tile table: the backward of a split
 *                     sequence sums the contributions of all of its tiles,
 *                     which equals the backward of the whole sequence, so it
 *                     is computed that way (validated, then run whole)
 * dq [Tq,H,d], dk/dv [Tk,H,d]   outputs, dtype `dtype`
 * workspace           device, >= zl_varlen_attn_bwd_workspace_size
 */
zl_status zl_varlen_attn_bwd(
    const void* q, const void* k, const void* v, const void* o, const float* lse,
    const void* dout,
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, int32_t dtype, float softmax_scale,
    const zl_tile_t* tiles, int32_t num_tiles,
    void* dq, void* dk, void* dv,
    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward that needs no workspace.  The paper has no counterpart to this
 * entry point; it exists for callers that cannot allocate device memory at
 * the moment they need a gradient: a plugin inside an engine that owns all
 * device memory and forbids allocation while it executes, code between
 * stream-capture begin and end, where a new allocation would not be part of
 * the captured work, or a process whose memory a pooling allocator has
 * reserved and that may not call it.
 *
 * Same operation, arguments and layouts as zl_varlen_attn_bwd with
 * dtype = ZL_BF16, minus the tile table (tiles do not change a backward's
 * result) and the workspace.  Its scratch (float32 dQ accumulator and D) is a
 * 64 MiB array in the library's device image, reserved on every GPU the
 * library is loaded on until the process exits.  Limit: Tq * H * d (rounded
 * up to a multiple of 64) + Tq * H <= 16,777,216 float32 values, e.g.
 * Tq <= 3,250 tokens at H = 40, d = 128; a larger batch returns
 * ZL_EWORKSPACE before any GPU work.  The caller still owns and passes every
 * input and output.
 *
 * The first call on each device (with that device current) looks up the
 * array's device address; make that first call before any stream capture.
 * All calls on a device share the array: calls whose kernels may overlap on
 * the GPU (unordered streams) race on it and give undefined results; calls on
 * one stream are safe.  Each call clears the accumulator it uses, so results
 * do not depend on earlier calls.  Allocates no device memory and creates
 * no CUDA objects: its launches count in zl_launch_count but are not timed
 * by zl_profile_*, whose events it would have to create.  Batch rules and errors are
 * zl_varlen_attn_bwd's (token bounds included), checked before the scratch
 * limit.
 */
zl_status zl_varlen_attn_bwd_static(
    const void* q, const void* k, const void* v, const void* o, const float* lse,
    const void* dout,
    const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t num_seqs,
    int32_t num_heads, int32_t head_dim, float softmax_scale,
    void* dq, void* dk, void* dv, void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions.
 *
 * Each head's first rot_dim columns form rot_dim / 2 pairs (a, b), and every
 * pair i of a token turns by its own angle:
 *
 *     angle = position[axis_i] * f_i
 *     (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
 *
 * Pair i is columns (i, i + rot_dim/2), or (2i, 2i+1) when interleaved; the
 * columns from rot_dim on stay as they are.  The pairs are dealt out to
 * n_axes position axes in order (one axis for a text or packed token order;
 * frame, row and column for video latents); pair j of an axis that has d
 * columns has f = base^(-2j/d), scaled for long contexts by `factor`:
 *
 *     without a ramp   f / factor
 *     with a ramp      f * (w + (1 - w) / factor),
 *                      w = clamp((length * f / 2pi - low) / (high - low), 0, 1)
 *
 * so that with a ramp the pairs that turn more than `high` times over
 * `length` positions keep their frequency and those that turn less than `low`
 * times take the scaled one.  A frequency in turns is computed in float64, a few
 * roundings of 2^-53 of it each; beside that an angle is off by at most 2^-26 of
 * a turn at every int32 position (a fixed-point product, exact mod 1, whose
 * upper 32 bits become a float32).  Positions may be negative.
 */
#define ZL_ROPE_MAX_PAIRS 64
#define ZL_ROPE_MAX_AXES 4

/* A prepared plan: filled by zl_rope_init, then passed to any number of
 * calls.  Plain data; the caller owns it and may copy it. */
typedef struct {
  int32_t head_dim;                       /* 64 or 128                            */
  int32_t rot_dim;                        /* rotated columns, even, <= head_dim   */
  int32_t interleaved;                    /* 0: halves, 1: neighbours             */
  int32_t n_axes;                         /* 1 .. ZL_ROPE_MAX_AXES                */
  int32_t pair_end[ZL_ROPE_MAX_AXES];     /* pairs of axes 0 .. a, cumulative     */
  float magnitude;
  int32_t reserved;
  uint64_t step[ZL_ROPE_MAX_PAIRS];       /* f_i / 2pi turns, mod 1, times 2^64   */
} zl_rope_t;

/*
 * Fills *plan.  axis_dims (host, n_axes entries): the rotated columns of each
 * axis, even and >= 2, their sum rot_dim <= head_dim.  base > 1, factor > 0 (the
 * scaled frequencies must be finite), magnitude finite and not 0 in float32.
 * ramp: NULL, or {low, high, length} with 0 <= low < high and length > 0.  Host
 * only.
 */
zl_status zl_rope_init(zl_rope_t* plan, int32_t head_dim, int32_t interleaved, int32_t n_axes,
                       const int32_t* axis_dims, double base, double factor, const double* ramp,
                       double magnitude);

/*
 * Turns packed queries and keys: q [T, Hq, d] and k [T, Hk, d] in `dtype`
 * (ZL_BF16 or ZL_FP32; float32 arithmetic, one rounding), with *_stride
 * elements between tokens (>= heads * d, a multiple of 16 bytes; heads and
 * columns contiguous, so that q and k may be parts of one projection's rows).
 * num_kv_heads = 0 leaves k out.  positions: device int32, axis a of token t
 * at [a * pos_stride + t].  An output may be its own input (same pointer and
 * stride); otherwise no output may overlap an input.  One launch.
 */
zl_status zl_rope_fwd(const zl_rope_t* plan, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const int32_t* positions, int64_t pos_stride, int64_t tokens, int32_t num_heads,
                      int32_t num_kv_heads, int32_t dtype, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream);

/*
 * Gradient of zl_rope_fwd: the transposed (negative) turn, applied to the
 * gradients of its outputs.  Same arguments: q = the gradient of q_out, and so on.
 */
zl_status zl_rope_bwd(const zl_rope_t* plan, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const int32_t* positions, int64_t pos_stride, int64_t tokens, int32_t num_heads,
                      int32_t num_kv_heads, int32_t dtype, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream);

/* ------------------------------------------------------------------------
 * Paged key/value cache.
 *
 * One layer's cache is two pools of pages, k_pages and v_pages, each bf16
 * [num_pages][Hk][page_size][d]: a page holds page_size consecutive tokens of
 * one sequence, head by head.  Sequence s (a row of the tables, in the order
 * of the batch) owns the pages page_table[s][0 .. ceil(kv_lens[s]/page_size)),
 * and token j of it lies in page_table[s][j / page_size] at j % page_size.
 * Entries past a sequence's pages, and pool rows past its length, are never
 * used, whatever they hold.  page_refs[p] counts the sequences that hold page
 * p (0: free).  New tokens are never written into a page that another sequence
 * holds: forks share full pages only, and a sequence truncated inside a shared
 * page is not extended (see zl_pages_truncate).  All tables are DEVICE arrays:
 * a captured graph replays with the lengths and pages of the moment.
 *
 * Kernels check every page number, slot and length that they read from the
 * device, and never leave the buffers: a token or page move that is out of
 * range is left out, attention reads page 0 in place of a page that is not
 * there and a length within the call's bound (that sequence's outputs are then
 * undefined, other sequences' are right), and the next zl_sync_check reports
 * ZL_EPAGE.
 */
typedef struct {
  void* k_pages;               /* [num_pages][num_kv_heads][page_size][head_dim] bf16 */
  void* v_pages;
  const int32_t* page_table;   /* [num_seqs][table_cols]                              */
  const int32_t* kv_lens;      /* [num_seqs]: tokens, the call's new ones included    */
  int32_t table_cols;          /* >= 1                                                */
  int32_t num_pages;           /* >= 1                                                */
  int32_t page_size;           /* 16, 32, 64, 128 or 256                              */
  int32_t num_kv_heads;
  int32_t head_dim;            /* 64 or 128                                           */
  int32_t reserved;            /* 0                                                   */
} zl_paged_cache_t;

/*
 * Writes a batch's new tokens into the cache: sequence s's tokens
 * [cu_seqlens[s], cu_seqlens[s+1]) become its positions kv_lens[s] - n_s ..
 * kv_lens[s] - 1.  k and v: bf16 [T, Hk, d] with k_stride / v_stride elements
 * between tokens.  With a rope plan (NULL: none) the keys, and the queries
 * q [T, Hq, d] -> q_out (q may be NULL, then num_heads is 0), are turned on
 * the way, at the tokens' cache positions, or at `positions` (device, as for
 * zl_rope_fwd) when given; a plan of more than one axis needs them.  The
 * pages that the tokens go to must not be shared.  One launch per 640
 * sequences.
 *
 * The lengths have to count the new tokens.  Where zl_pages_extend lacked pages
 * they do not, and the tokens would be written over the sequences' last ones:
 * check its status before, or, where the host does not wait for it (a captured
 * graph), hand it to zl_paged_append_ex.
 */
zl_status zl_paged_append(const zl_paged_cache_t* cache, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* cu_seqlens, int32_t num_seqs, const zl_rope_t* plan,
                          const int32_t* positions, int64_t pos_stride, const void* q, int64_t q_stride,
                          int32_t num_heads, void* q_out, int64_t q_out_stride, void* stream);

/*
 * The same behind a zl_pages_extend whose status the host has not read: status
 * (device int32, or NULL) is read by the launch, and unless it is 0 no key or
 * value is written and the next zl_sync_check reports ZL_EPAGE.  (q_out is
 * written either way; of attention over the cache the call's outputs then mean
 * nothing, but the cache is as it was.)
 */
zl_status zl_paged_append_ex(const zl_paged_cache_t* cache, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const int32_t* cu_seqlens, int32_t num_seqs, const zl_rope_t* plan,
                             const int32_t* positions, int64_t pos_stride, const void* q, int64_t q_stride,
                             int32_t num_heads, void* q_out, int64_t q_out_stride, const int32_t* status,
                             void* stream);

/*
 * Workspace needed by zl_paged_attn for this batch, in bytes: what sequences
 * whose keys are spread over several SMs leave there until they are joined.
 * It depends on the queries, the heads and head_dim alone, at most 40 MiB, and
 * a call needs nothing of it from an earlier one: calls that are ordered (the
 * layers of a model, graphs replayed in turn) may share one workspace, calls
 * that may overlap must not.  Same argument rules as zl_paged_attn.
 */
zl_status zl_paged_attn_workspace_size(const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t max_kv_len,
                                       int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, size_t* bytes);

/*
 * Attention of a chunk of new tokens over the paged cache.  Sequence s has
 * n_s = cu_seqlens_q[s+1] - cu_seqlens_q[s] queries (any number from 0 on;
 * 1: a single new token) at positions p = kv_lens[s] - n_s + i.  Query p sees
 * the keys j with
 *
 *     j < kv_lens[s],   j <= p if causal,   j > p - window if window > 0
 *
 * A query that sees none gets o = 0 and lse = -inf.  Query head h reads key
 * head h / (num_heads / num_kv_heads).
 *
 * q [Tq, H, d] bf16, q_stride elements between tokens; o [Tq, H, d] bf16,
 * lse [H, Tq] float32 (natural log, as zl_varlen_attn_fwd's, so that results
 * over other keys can be joined with zl_lse_merge).  max_kv_len: an upper
 * bound of kv_lens, at most table_cols * page_size and 2^31 - 257 (a longer
 * sequence is cut there and reported as ZL_EPAGE).  num_heads is a multiple of num_kv_heads
 * and at most 128 times as many.  Scores, the running maximum and sum, and the
 * output accumulate in float32; the probabilities are rounded to bf16 once for
 * the tensor cores.  The values of a sequence's tokens must be finite: a
 * product of zero and infinity would reach queries that do not see them (its
 * keys may be anything where the mask hides them, and rows past its length
 * anything at all).  The work is spread over the SMs in equal shares whatever
 * the lengths (short ones, by max_kv_len and the window, are left whole); results
 * are the same on every run with the same lengths and arguments.  Where a
 * sequence's keys are cut follows from the whole batch, so its last bits may
 * change with the sequences beside it and with max_kv_len.  o and lse overlap no
 * other operand.  One or two
 * launches per 640 sequences of one query tile (up to 128 / (num_heads /
 * num_kv_heads) queries) and one or two per 640 longer ones.
 */
zl_status zl_paged_attn(const zl_paged_cache_t* cache, const void* q, int64_t q_stride, const int32_t* cu_seqlens_q,
                        int32_t num_seqs, int32_t max_kv_len, int32_t num_heads, float softmax_scale, int32_t causal,
                        int32_t window, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* The tables of a cache as the page operations change them. */
typedef struct {
  int32_t* page_table;         /* [slots][table_cols]                                 */
  int32_t* kv_lens;            /* [slots]                                             */
  int32_t* page_refs;          /* [num_pages]                                         */
  int32_t slots;               /* 1 .. 8192                                           */
  int32_t table_cols;          /* >= 1                                                */
  int32_t num_pages;           /* >= 1                                                */
  int32_t page_size;           /* 16, 32, 64, 128 or 256                              */
} zl_page_tables_t;

/*
 * The pools whose pages are moved: group g's page p is the page_bytes (a
 * multiple of 16) at base + g * group_stride + p * page_bytes.  The layers'
 * key and value pools of one allocation are its groups.
 */
typedef struct {
  void* base;
  int64_t page_bytes;
  int64_t group_stride;        /* bytes, >= num_pages * page_bytes                    */
  int32_t groups;              /* >= 1                                                */
  int32_t num_pages;           /* >= 1                                                */
} zl_page_pool_t;

/* Scratch of zl_pages_fork and zl_pages_compact, in bytes. */
zl_status zl_pages_workspace_size(int32_t num_pages, size_t* bytes);

/*
 * Makes room for counts[s] (device, >= 0) new tokens in every slot: kv_lens
 * grows by counts, and the pages that the new lengths need are taken from the
 * free ones, lowest number first, in the order of slots and positions.
 * *status (device): 0; or the number of pages that were lacking; or -1 for a
 * negative count or a length that does not fit a table row; or -2 for a slot
 * whose new tokens would begin inside a page that another slot holds (it was
 * truncated there).  Unless it is 0 nothing was changed.
 */
zl_status zl_pages_extend(const zl_page_tables_t* tables, const int32_t* counts, int32_t* status, void* stream);

/*
 * Makes slot children[i] a copy of slot parents[i] (device, n of each): the
 * child shares the parent's full pages, and a last page that is not full is
 * copied into a free page of its own (lowest number first, in the order of i),
 * in every group of the pool.  A parent may be forked any number of times; the
 * children are distinct empty slots.  *status as for zl_pages_extend (-1: a
 * slot out of range, a child that is not empty or named twice).
 */
zl_status zl_pages_fork(const zl_page_pool_t* pool, const zl_page_tables_t* tables, const int32_t* parents,
                        const int32_t* children, int32_t n, int32_t* status, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * Empties the slots (device, n of them; one that is named twice or is empty
 * already counts once): their pages lose a reference, their table entries
 * become -1 and their lengths 0.  A page that no slot holds any more is free.
 */
zl_status zl_pages_free(const zl_page_tables_t* tables, const int32_t* slots, int32_t n, void* stream);

/*
 * Shortens every slot that is longer than lens[s] (device, >= 0) to it, as when
 * drafted tokens are taken back: the pages behind lose a reference, their table
 * entries become -1.  (A caller that only lowered kv_lens would lose those
 * pages.)  A slot cut inside a page that another slot holds too cannot grow
 * (zl_pages_extend: -2) until it has a copy of that page of its own: fork it to
 * an empty slot and free it, or free the others.
 */
zl_status zl_pages_truncate(const zl_page_tables_t* tables, const int32_t* lens, void* stream);

/*
 * Packs the pool: with L pages in use, those numbered L and up move to the
 * free pages below L (both in ascending order), in every group of the pool,
 * and the tables and counts follow.  *live (device) = L.
 */
zl_status zl_pages_compact(const zl_page_pool_t* pool, const zl_page_tables_t* tables, int32_t* live, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Copies page src[i] over page dst[i] (device, n pairs) in every group.  No
 * page may be both a source and a target, nor a target twice.
 */
zl_status zl_pages_copy(const zl_page_pool_t* pool, const int32_t* src, const int32_t* dst, int32_t n, void* stream);

/*
 * Synchronizes `stream`, then reports (and clears) any error a kernel of this
 * library flagged on the current device: ZL_ETIMEOUT when a bounded wait
 * inside a kernel ran out (the kernel stopped early and its outputs are
 * undefined), ZL_EPAGE when a kernel of the paged cache left something out
 * that its tables misplaced, ZL_ECUDA for a CUDA error.  ZL_OK otherwise.
 */
zl_status zl_sync_check(void* stream);

/*
 * Self-test of failure detection.  The pages have no counterpart; what it
 * exercises is the rule every kernel here follows: no wait is unbounded, a
 * wait that runs out records an error and ends the CTA's other roles, and the
 * kernel returns so that the context stays usable.  It enqueues one small
 * kernel whose wait on an mbarrier that nothing arrives on gives up after
 * limit_ns nanoseconds (1 .. 1e9; else ZL_EINVAL), while a second warp of
 * the same CTA, waiting with the kernels' own limit, must leave as soon as the
 * first one has given up.  No copy or MMA is in flight and no memory is
 * touched.  The next zl_sync_check(stream) returns ZL_ETIMEOUT (and clears
 * the record); work enqueued afterwards runs normally.
 */
zl_status zl_selftest_wait_timeout(uint64_t limit_ns, void* stream);

/* Number of kernel launches this library has enqueued in this process. */
int64_t zl_launch_count(void);

/*
 * Per-kernel timing, the single-GPU counterpart of the paper's Hardware
 * Profiler, which measures execution time per configuration (Zellige §IV-B).
 * Between zl_profile_begin() and zl_profile_end() every kernel this library
 * launches is bracketed by two CUDA events on its stream.  zl_profile_end()
 * waits for those events, writes one entry per kernel name (launch count and
 * summed device time) into `entries` (up to max_entries; *n_entries gets the
 * number written), releases the events and stops recording.  Recording is
 * process-wide; begin while already recording returns ZL_EINVAL.
 */
typedef struct {
  char name[32];
  int64_t launches;
  double total_ms;
} zl_profile_entry_t;

zl_status zl_profile_begin(void);
zl_status zl_profile_end(zl_profile_entry_t* entries, int32_t max_entries, int32_t* n_entries);

#ifdef __cplusplus
}
#endif

#endif /* ZL_ATTN_H */
