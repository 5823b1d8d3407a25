/*
 * ringattn.h — C ABI of the single-GPU ring attention hot path (GB300, sm_103a).
 *
 * Ring attention splits one sequence of N tokens into D shards of N/D tokens. Rank r keeps
 * its query shard; the K/V shards travel around a ring, so at step s rank r holds the K/V
 * shard of rank (r - s) mod D, computes local attention against it and folds the block
 * result into its running (out, lse) with the log-sum-exp merge (Ring Attention concept
 * page, "Sequence sharding and the ring topology" and "Online softmax across ring steps";
 * nanotron how-to page, "Forward Pass Implementation"). On one GPU the D ranks are virtual:
 * all shards sit in HBM and a ring step is the choice of which K/V shard a query tile reads.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers owned by the caller. The library allocates no
 *   device memory and never synchronises the device (except ra_check_device_status); all
 *   work is enqueued on the caller's CUDA stream, passed as `void* stream` (a cudaStream_t,
 *   NULL = legacy default stream).
 * - Token tensors (q, k, v, out, dout, dq, dk, dv) are row-major with the head dimension
 *   innermost: batch mode [B, S, H, Dh], varlen mode packed [T, H, Dh].
 *   Their token axis is SHARD-MAJOR: the D local shard buffers concatenated. Batch mode:
 *   token (b, r, a) — local index a of rank r — is row b*S + r*(S/D) + a. Varlen mode:
 *   every sequence i is split on its own into D pieces of len_i/D tokens, and rank r's
 *   buffer (rows [r*T/D, (r+1)*T/D)) holds its pieces of all sequences in order, i.e.
 *   token (i, r, a) is row r*T/D + cu_seqlens[i]/D + a. ra_shard_tokens / ra_shard_lse
 *   convert from and to natural order.
 * - Which global position a local token holds depends on the layout (ring-flash-attn
 *   package card, "What it is and what it does"): BASIC: r*L + a; ZIGZAG (2D chunks of
 *   c = L/2, rank r holds chunks r and 2D-1-r): a < c ? r*c + a : (2D-1-r)*c + a - c;
 *   STRIPE (token t on rank t mod D): a*D + r. L = len/D is the local length.
 * - lse is float32, natural log: batch mode [B, Hq, S], varlen mode [Hq, T], with the
 *   token axis shard-major like the token tensors.
 * - Causal masking uses global positions: query at position p sees keys at positions
 *   <= p of the same sequence (concept page, "Watch Out For"). With the basic layout this
 *   is the pages' rule "attend only if step <= rank" plus a triangular diagonal block.
 * - Grouped-query attention: query head h reads K/V head h / (Hq/Hkv).
 * - Return value: RA_OK (0) or a negative ra_status. On error nothing was launched (except
 *   RA_ERR_CUDA, which reports a failed launch) and ra_last_error() returns a message.
 *
 * Supported: bf16 with head_dim 64 or 128 (tensor-core path; every token tensor but a backward's
 * `out` begins on 16 bytes); f32 with head_dim 1..128 (CUDA-core path). D >= 1 and every
 * sequence length divisible by D (2D for zigzag).
 * Up to RA_MAX_SEQS sequences (batch elements or varlen sequences) per call.
 */
#ifndef RINGATTN_H
#define RINGATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RA_VERSION 1
#define RA_MAX_SEQS 1024

typedef enum ra_status {
  RA_OK = 0,
  RA_ERR_INVALID_ARG = -1,   /* null pointer, negative size, bad enum                     */
  RA_ERR_UNSUPPORTED = -2,   /* dtype / head_dim / hq % hkv / option not implemented      */
  RA_ERR_SHAPE = -3,         /* a length not divisible by D (2D for zigzag), bad cu_seqlens */
  RA_ERR_WORKSPACE = -4,     /* workspace smaller than ra_workspace_bytes()               */
  RA_ERR_CUDA = -5,          /* a CUDA call or kernel launch failed                       */
  RA_ERR_DEVICE_TIMEOUT = -6, /* a kernel gave up a bounded wait (see ra_check_device_status) */
  RA_ERR_CACHE_INDEX = -7    /* a kernel met a page index, a length or a position outside the
                                paged cache it was given (see ra_check_device_status)      */
} ra_status;

typedef enum ra_dtype { RA_F32 = 0, RA_BF16 = 1 } ra_dtype;

typedef enum ra_layout {
  RA_LAYOUT_BASIC = 0,
  RA_LAYOUT_ZIGZAG = 1,
  RA_LAYOUT_STRIPE = 2
} ra_layout;

/* One ring-attention problem (nanotron how-to page, "Calling the Ring Attention Function
 * Directly": q, k, v, cu_seqlens, max_seqlen, scaling, causal, deterministic; ring-flash-attn
 * package card: batch and varlen modes, basic / zigzag / stripe). */
typedef struct ra_problem {
  int32_t dtype;              /* ra_dtype of q, k, v, out, dout, dq, dk, dv                  */
  int32_t layout;             /* ra_layout                                                  */
  int32_t causal;             /* 1: global-position causal mask; 0: full attention          */
  int32_t D;                  /* ring size: number of virtual shards                        */
  int32_t batch;              /* batch mode: B > 0.  Varlen mode: 0                          */
  int32_t seqlen;             /* batch mode: S (per batch element). Varlen mode: ignored     */
  int32_t n_seqs;             /* varlen mode: number of packed sequences                     */
  const int32_t* cu_seqlens;  /* varlen mode: HOST array of n_seqs+1 natural-order offsets,
                                 cu_seqlens[0] = 0, non-decreasing. NULL in batch mode.      */
  int32_t hq;                 /* query heads                                                */
  int32_t hkv;                /* K/V heads (hq % hkv == 0)                                   */
  int32_t head_dim;           /* Dh                                                         */
  float scale;                /* softmax scale; <= 0 selects 1/sqrt(head_dim) (the pages'
                                 default for scaling=None)                                  */
  int32_t deterministic;      /* 1: the backward must be run-to-run bit-identical (no
                                 floating-point atomics). 0: no such promise is asked for;
                                 the bf16 backward is atomic-free and deterministic anyway,
                                 the f32 one always is                                      */
} ra_problem;

/* Fused ring forward: every rank r, every step s = 0..D-1 against K/V shard (r-s) mod D,
 * with the log-sum-exp merge fused (running max and denominator kept across steps).
 * q [.., Hq, Dh], k/v [.., Hkv, Dh] in the problem dtype; out like q; lse float32.
 * The workspace is optional: NULL (any workspace_bytes) runs with a static work split;
 * a device buffer of >= ra_workspace_bytes(p, 0) bytes, 256-byte aligned, holds a counter
 * from which the CTAs take their work items (a CTA that finishes early takes more), and is
 * overwritten. (nanotron how-to page, "Forward Pass Implementation".) */
int ra_ring_attn_fwd(const ra_problem* p, const void* q, const void* k, const void* v,
                     void* out, float* lse, void* workspace, size_t workspace_bytes,
                     void* stream);

/* One ring step of the unfused path: rank `rank` (or every rank if rank < 0) attends with
 * its query shard to the K/V shard it holds at step `step`, i.e. shard (rank-step) mod D.
 * Writes the NORMALISED block_out (like q, in dtype `block_out_dtype` = RA_F32 or RA_BF16)
 * and block_lse (lse layout) for the rows of the selected rank(s) only. A row that sees no
 * key gets block_lse = -inf and block_out = 0. (How-to page, step 2: local attention of
 * the rank's queries against the received K/V slice.) */
int ra_block_attn_fwd(const ra_problem* p, int rank, int step, const void* q,
                      const void* k, const void* v, void* block_out, int block_out_dtype,
                      float* block_lse, void* stream);

/* The log-sum-exp merge of update_out_and_lse (how-to page, "Numerically-Stable Output
 * Fusion"), in place on float32 out / lse, for the rows of rank `rank` (all if < 0):
 *   lse' = log(exp(lse) + exp(block_lse))
 *   out' = exp(lse - lse') * out + exp(block_lse - lse') * block_out
 * lse = -inf with out = 0 is the identity (start state of a ring). block_out is float32 or
 * bf16 (block_out_dtype); out is always float32, in the token layout with Hq heads. */
int ra_update_out_and_lse(const ra_problem* p, int rank, float* out, float* lse,
                          const void* block_out, int block_out_dtype, const float* block_lse,
                          void* stream);

/* Bytes of device workspace: which = 0 for ra_ring_attn_fwd (optional there), which = 1
 * for ra_ring_attn_bwd, which = 2 for ra_block_attn_bwd, which = 3 for ra_qk_norm_rope_bwd; 0 for which = 0 on the f32 path. Returns 0 for an invalid problem as well;
 * call ra_validate to tell the two apart. */
size_t ra_workspace_bytes(const ra_problem* p, int which);

/* Ring backward (how-to page, "Backward Pass and Gradient Accumulation"): the blocks of
 * every (rank, step) pair again, each differentiated against the FINAL out and lse of the
 * forward (P recomputed from lse, never stored); dq accumulates per query rank, dk and dv
 * accumulate into the K/V shard that owns the block, summed over the query heads of a
 * group. Inputs: q, k, v, out, lse as from the forward, dout like out. Outputs dq (like q),
 * dk, dv (like k) in the problem dtype; every element is written. The bf16 path runs two
 * passes without atomics (K/V tiles: dk, dv; query tiles: dq), so results are run-to-run
 * bit-identical. The workspace (device, >= ra_workspace_bytes(p, 1), 256-byte aligned)
 * holds the per-row dot(dout, out), the counter from which the K/V-tile pass's CTAs take
 * their work items (and, only when the environment variable RA_BWD=fused selects the
 * single-pass variant with float reductions, float32 dq sums); it is overwritten. */
int ra_ring_attn_bwd(const ra_problem* p, const void* q, const void* k, const void* v,
                     const void* out, const float* lse, const void* dout, void* dq,
                     void* dk, void* dv, void* workspace, size_t workspace_bytes,
                     void* stream);

/* One ring step of the unfused backward (how-to page, "Backward Pass and Gradient
 * Accumulation": per step, the block is differentiated against the FINAL out and lse, then
 * dq += block_dq on the rank and block_dk / block_dv are added into the K/V shard's
 * gradients). Rank `rank` (every rank if rank < 0) at step `step` holds K/V shard
 * (rank - step) mod D; this call ADDS, in float32:
 *   dq_acc rows of rank `rank`                     += block_dq   (layout like q)
 *   dk_acc, dv_acc rows of shard (rank-step) mod D += block_dk, block_dv (layout like k)
 * Summing the calls of steps 0..D-1 into zeroed accumulators gives the full backward.
 * Inputs as for ra_ring_attn_bwd (out, lse: the final forward results). The workspace
 * (device, >= ra_workspace_bytes(p, 2), 256-byte aligned) receives the per-row
 * dot(dout, out) of the selected rank(s) and the passes' item counters; it is overwritten. Rows outside the selection are
 * not touched. Calls must not overlap on the GPU when they add into the same rows. The bf16
 * path runs the two atomic-free passes of ra_ring_attn_bwd restricted to the step (each
 * accumulator row is added by one thread), so results are run-to-run bit-identical;
 * RA_BWD=fused selects the single pass that adds block_dq with float reductions. */
int ra_block_attn_bwd(const ra_problem* p, int rank, int step, const void* q, const void* k,
                      const void* v, const void* out, const float* lse, const void* dout,
                      float* dq_acc, float* dk_acc, float* dv_acc, void* workspace,
                      size_t workspace_bytes, void* stream);

/* The same backward for callers that cannot allocate device memory (a plain-C plugin
 * handed only its input and output buffers, or a caller that must keep cudaMalloc and its
 * device-wide synchronisation out of a training step). The pages have no counterpart: on
 * the pages every rank allocates its own buffers. Instead of a caller workspace, the
 * scratch (the per-row dot(dout, out), plus float32 dq sums when RA_BWD=fused selects the
 * single-pass variant) lives in one static device
 * array of RA_NOALLOC_SCRATCH_BYTES that every GPU loading the library keeps until exit.
 * Arguments as for ra_ring_attn_bwd minus the workspace. Problems whose
 * ra_workspace_bytes(p, 1) exceeds the array are rejected with RA_ERR_WORKSPACE and nothing
 * is launched. The first call on a device looks the array's address up on that device
 * and keeps it for the life of the process (make that first call before any stream
 * capture; a cudaDeviceReset after it is not supported, since the kept address would then
 * be stale). Every call shares the array and the
 * backward clears what must start at zero, but calls that overlap on the GPU race on it:
 * order them on one stream. Allocates nothing. */
#define RA_NOALLOC_SCRATCH_BYTES (64u << 20)
int ra_ring_attn_bwd_noalloc(const ra_problem* p, const void* q, const void* k, const void* v,
                             const void* out, const float* lse, const void* dout, void* dq,
                             void* dk, void* dv, void* stream);

/* ---- sliding window --------------------------------------------------------------------- */

#define RA_MAX_SINKS 128

/* Ring attention with a sliding window: the query at position p of a sequence sees the keys at
 * positions k <= p with k > p - window or k < sinks (the first `sinks` tokens of every
 * sequence stay visible). The problem must be causal, with D <= 64 in bf16; window >= 1, 0 <=
 * sinks <= RA_MAX_SINKS. Tensors, layouts, lse and the optional workspace (now
 * ra_window_workspace_bytes(p, window, sinks, 0)) are as for ra_ring_attn_fwd; K/V tiles that
 * no query of a block sees are never loaded. With a window that no sequence is longer than,
 * this is ra_ring_attn_fwd. As there, k and v must be finite: hidden keys of a loaded tile
 * count with weight 0. */
int ra_window_attn_fwd(const ra_problem* p, int window, int sinks, const void* q, const void* k,
                       const void* v, void* out, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Its backward, arguments as for ra_ring_attn_bwd (as there, the row sums dO . O are formed from
 * `out` in its dtype, but for bf16 windows of up to 16 visible keys, where its rounding would tell;
 * dout must be finite as well). In bf16 dq and dk take a weight of less than 2^-39 for 0.
 * Run-to-run bit-identical. The workspace (device, >= ra_window_workspace_bytes(p, window, sinks,
 * 1), 256-byte aligned) is overwritten. It holds a sum of the sinks' gradients for every K/V head,
 * shard with sinks and piece of a shard's queries; a problem with 2^31 of them is refused
 * (RA_ERR_UNSUPPORTED). */
int ra_window_attn_bwd(const ra_problem* p, int window, int sinks, const void* q, const void* k,
                       const void* v, const void* out, const float* lse, const void* dout, void* dq,
                       void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of the two calls above: which = 0 forward (optional there), which = 1
 * backward; 0 for arguments that the calls refuse. */
size_t ra_window_workspace_bytes(const ra_problem* p, int window, int sinks, int which);

/* ---- head norms and position rotation ------------------------------------------------ */

#define RA_MAX_ROTARY_DIM 128
#define RA_MAX_CACHE_SEQS 8192 /* sequences of a paged cache in one call */

/* A rotation by position of the first `rotary_dim` elements of a head: pair i turns by
 * position * inv_freq[i] radians. The pairs are (i, i + rotary_dim/2), or (2i, 2i + 1) when
 * interleaved. Filled in by ra_rope_init, passed by value to the kernels. */
typedef struct ra_rope {
  int32_t rotary_dim;
  int32_t interleaved;
  uint64_t turns[RA_MAX_ROTARY_DIM / 2]; /* turns per position, in units of 2^-64 of a turn: the
                                            product with a position wraps at whole turns, so an
                                            angle is good to 2^-26 of a turn (the float that its
                                            sine and cosine are taken of) at any position */
} ra_rope;

/* Fills in `rope` from rotary_dim/2 HOST doubles (radians per position, finite). rotary_dim is
 * even, 2..RA_MAX_ROTARY_DIM. */
int ra_rope_init(ra_rope* rope, int rotary_dim, int interleaved, const double* inv_freq);

/* Per-head norm of queries and keys with the rotation in the same pass, before
 * ra_ring_attn_fwd: for every head x of every token of the problem
 *   y = R(position) (x * rsqrt(mean(x^2) + eps) * weight)
 * where the position is the token's global position in its sequence under the problem's
 * layout (the rows are shard-major). q_weight and k_weight hold head_dim elements of the
 * problem dtype; both NULL leaves the norm out (eps is then not looked at), rope NULL leaves
 * the rotation out, one of the two must be there. rope->rotary_dim <= head_dim; the rest of a
 * head is not rotated. q and k may be views into a wider tensor: q_row_stride and
 * k_row_stride are the elements from one token to the next (>= heads * head_dim); the heads
 * of a token are contiguous. q_out and k_out are contiguous; q_out may be q, and k_out k, when
 * that is contiguous too. */
int ra_qk_norm_rope_fwd(const ra_problem* p, const ra_rope* rope, float eps, const void* q,
                        int64_t q_row_stride, const void* k, int64_t k_row_stride,
                        const void* q_weight, const void* k_weight, void* q_out, void* k_out,
                        void* stream);

/* Its backward: from the gradients dq_out and dk_out (contiguous) of the outputs and the
 * INPUTS q and k of the forward, the gradients dq and dk of the inputs (contiguous, problem
 * dtype; dq may be dq_out, dk may be dk_out) and, in float32, dq_weight and dk_weight
 * (head_dim elements each, summed over every token and head in a fixed order: run-to-run
 * bit-identical). Without weights q, k, dq_weight and dk_weight are not used and may be NULL.
 * The workspace (device, >= ra_workspace_bytes(p, 3), 256-byte aligned) is overwritten. */
int ra_qk_norm_rope_bwd(const ra_problem* p, const ra_rope* rope, float eps, const void* dq_out,
                        const void* dk_out, const void* q, int64_t q_row_stride, const void* k,
                        int64_t k_row_stride, const void* q_weight, const void* k_weight,
                        void* dq, void* dk, float* dq_weight, float* dk_weight,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ---- positions on several axes ---------------------------------------------------------- */

#define RA_MAX_AXES 8

/* A rotation of tokens that have a position on each of n_axes axes (time, height and width of a
 * video's patches; text has the same on all): pair i turns by the token's position on axis axis[i]
 * times inv_freq[i] radians. Filled in by ra_axis_rope_init. */
typedef struct ra_axis_rope {
  ra_rope rope;
  int32_t n_axes;
  uint8_t axis[RA_MAX_ROTARY_DIM / 2];
} ra_axis_rope;

/* Fills in `rope`: rotary_dim, interleaved and inv_freq as for ra_rope_init, axis rotary_dim/2 HOST
 * integers in [0, n_axes), n_axes 1..RA_MAX_AXES. */
int ra_axis_rope_init(ra_axis_rope* rope, int rotary_dim, int interleaved, const double* inv_freq,
                      int n_axes, const int32_t* axis);

/* ra_qk_norm_rope_fwd, ra_qk_norm_rope_bwd (below: ra_kv_cache_append) with such a rotation, the
 * other arguments as there. positions (device, int32, any values) has n_axes elements for every row
 * of q and k, pos_row_stride (>= n_axes) elements from one row to the next, in the rows' own order:
 * shard-major like q and k (ra_shard_tokens with row_bytes 4 * n_axes brings them there). A row's
 * place in its sequence plays no part. Angles are as good as with one axis. */
int ra_qk_norm_axis_rope_fwd(const ra_problem* p, const ra_axis_rope* rope, const int32_t* positions,
                             int64_t pos_row_stride, float eps, const void* q, int64_t q_row_stride,
                             const void* k, int64_t k_row_stride, const void* q_weight,
                             const void* k_weight, void* q_out, void* k_out, void* stream);
int ra_qk_norm_axis_rope_bwd(const ra_problem* p, const ra_axis_rope* rope, const int32_t* positions,
                             int64_t pos_row_stride, float eps, const void* dq_out, const void* dk_out,
                             const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                             const void* q_weight, const void* k_weight, void* dq, void* dk,
                             float* dq_weight, float* dk_weight, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ---- serving: a paged key-value cache and the attention of one new token -------------- */

/* A cache of n_pages pages of page_size tokens; page p, place s, K/V head h starts at element
 * p*page_stride + s*slot_stride + h*head_stride of k_pages and of v_pages, head_dim elements
 * contiguous (so [n_pages, page_size, hkv, head_dim], [n_pages, hkv, page_size, head_dim] and
 * views of them are all fine). Token t of sequence b is in page
 * block_table[b*table_stride + t / page_size] at place t % page_size. All pointers are DEVICE
 * pointers; entries of the table beyond a sequence's length are not looked at. An entry
 * outside [0, n_pages), or a length beyond max_pages * page_size, is never followed: the
 * kernels record RA_ERR_CACHE_INDEX in the device status and leave out that token (append) or
 * read page 0 / the cache's part of the sequence in its place (decode, whose result for that
 * sequence then means nothing). */
typedef struct ra_paged_cache {
  int32_t dtype;      /* ra_dtype of the pages, and of the tokens that go with them */
  int32_t hkv;
  int32_t head_dim;   /* bf16: 64 or 128; f32: 1..128 */
  int32_t page_size;  /* >= 1 */
  int32_t n_pages;    /* >= 1 */
  int32_t n_seqs;     /* rows of the block table: the sequences of a batch */
  int32_t max_pages;  /* entries of a row; max_pages * page_size <= 2^31 - 64 */
  int64_t table_stride;
  int64_t page_stride, slot_stride, head_stride; /* elements */
  void* k_pages;
  void* v_pages;
  const int32_t* block_table;
} ra_paged_cache;

/* Puts new tokens into the cache: k (after norm and rotation, as in ra_qk_norm_rope_fwd) and v
 * (as it is) go to their places, q (after the same) to q_out. seq_lens [n_seqs] (device) are
 * the lengths WITH the new tokens, as ra_paged_attn_decode wants them. cu_new NULL: one new
 * token for each sequence, row b of q, k, v belongs to sequence b (n_tokens = n_seqs); a
 * sequence of length 0 is idle: nothing is stored for it and its row of q_out is 0. Else
 * cu_new [n_seqs + 1] (device): rows cu_new[b] .. cu_new[b+1]-1 are the last tokens of
 * sequence b; rows from cu_new[n_seqs] on are left as they are. No two rows may go to the
 * same place. q and q_out both NULL: k and v only (hq is then not looked at). Row strides as
 * above; q_out is contiguous. weights both NULL: no norm; rope NULL: no rotation. */
int ra_kv_cache_append(const ra_paged_cache* c, const ra_rope* rope, float eps, int n_tokens,
                       int hq, const void* q, int64_t q_row_stride, const void* k,
                       int64_t k_row_stride, const void* v, int64_t v_row_stride,
                       const void* q_weight, const void* k_weight, const int32_t* seq_lens,
                       const int32_t* cu_new, void* q_out, void* stream);

/* The same with positions on several axes: positions and pos_row_stride as for
 * ra_qk_norm_axis_rope_fwd, a row for each of the n_tokens rows. Where a token goes in the cache is
 * its place in its sequence, as before. */
int ra_kv_cache_append_axes(const ra_paged_cache* c, const ra_axis_rope* rope, const int32_t* positions,
                            int64_t pos_row_stride, float eps, int n_tokens, int hq, const void* q,
                            int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                            int64_t v_row_stride, const void* q_weight, const void* k_weight,
                            const int32_t* seq_lens, const int32_t* cu_new, void* q_out, void* stream);

/* Attention of the last token of every sequence: q and out [n_seqs, hq, head_dim] (contiguous,
 * cache dtype; hq % hkv == 0), lse [n_seqs, hq] (float32, natural log). The query sees the keys
 * 0 .. seq_lens[b]-1, and with window > 0 of these only the last `window` and the first
 * `sinks`. A sequence of length 0 gets out = 0, lse = -inf. scale <= 0 selects
 * 1/sqrt(head_dim). The keys of the batch are dealt out evenly over the SMs whatever the
 * lengths, and parts of a sequence are joined by the log-sum-exp merge, in a fixed order
 * (run-to-run bit-identical). bf16 wants q, out and the pages 16-byte aligned, and strides that
 * are multiples of 8 elements. The workspace (device, >= ra_paged_workspace_bytes(c, hq), 256-byte
 * aligned) is overwritten; nothing in it is kept from call to call, so calls and captured
 * graphs may share it as long as they do not run at the same time. */
int ra_paged_attn_decode(const ra_paged_cache* c, int hq, float scale, int window, int sinks,
                         const void* q, const int32_t* seq_lens, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of ra_paged_attn_decode; 0 for an invalid cache or hq. */
size_t ra_paged_workspace_bytes(const ra_paged_cache* c, int hq);

/* Prefixes that groups of sequences of a batch have in common: the sequences cu_groups[g] ..
 * cu_groups[g+1]-1 begin with the same prefix_lens[g] tokens (a document, instructions), so that
 * their keys and values there are equal; as a rule their rows of the block table name the same
 * pages. Sequences of no group, or with a prefix_lens of 0, share nothing. Both arrays are DEVICE
 * arrays, cu_groups [n_groups + 1] non-decreasing within 0 .. n_seqs, prefix_lens [n_groups].
 * Sharing changes how the keys are read, and the result by no more than its roundings (see
 * ra_paged_attn_extend on the weights): the whole key tiles (128 keys, in float32 64) of a prefix are read once for the group, by the block table row of its first sequence that has
 * new tokens, where that saves work, and where every sequence of the group has the prefix before its
 * new tokens; else each sequence reads its own. Offsets that decrease or leave 0 .. n_seqs are
 * recorded in the device status (RA_ERR_CACHE_INDEX) where the call looks at them, and then nothing is
 * shared. A decoding step over a cache whose block table has room for no more than 256 MB of keys and
 * values (n_seqs * max_pages pages) does not look: it reads every sequence apart, which is faster. */
typedef struct ra_shared_prefix {
  int32_t n_groups; /* <= n_seqs; 0: none */
  const int32_t* cu_groups;
  const int32_t* prefix_lens;
} ra_shared_prefix;

/* Causal attention of the last tokens of every sequence, which are in the cache already (see
 * ra_kv_cache_append): a question after a document, a prompt that comes in chunks, drafted tokens
 * to be checked. q and out [n_tokens, hq, head_dim] (contiguous, cache dtype; hq % hkv == 0), lse
 * [n_tokens, hq] (float32, natural log). seq_lens [n_seqs] (device) are the lengths WITH the new
 * tokens. cu_new [n_seqs + 1] (device): rows cu_new[b] .. cu_new[b+1]-1 are the last tokens of
 * sequence b; rows before cu_new[0] and from cu_new[n_seqs] on are left as they are. cu_new NULL: one
 * new token of every sequence (n_tokens = n_seqs), and a sequence of length 0 is idle: its row gets
 * out = 0, lse = -inf. The row at position p of its sequence sees the keys k <= p, with window > 0
 * only those with k > p - window or k < sinks (0 <= sinks <= RA_MAX_SINKS). shared may be NULL; with
 * a window it must be. Keys that no row of a sequence sees are not read; those that some row sees
 * must be finite (a key that a row does not see may count with weight 0). scale <= 0 selects
 * 1/sqrt(head_dim). A sequence with more new tokens than its length, offsets that decrease or pass
 * n_tokens, or a page index outside the cache is recorded in the device status
 * (RA_ERR_CACHE_INDEX), and never followed. bf16 wants q, out and the pages 16-byte aligned, and
 * strides that are multiples of 8 elements. In bf16 the softmax's weights, float32 numbers, go into the
 * product with v as two bf16 numbers (2^-16) in steps of one new token (cu_new NULL), for sequences of
 * at most 16 rows (new tokens x query heads of a K/V head), and, in calls of at most 16 rows a sequence on
 * average, for shared prefixes of whose rows at least half are of such sequences: out is then as far from
 * the definition as its own rounding, 0.0017 in relative L2. Elsewhere they go in as one (2^-8, as in
 * ra_ring_attn_fwd): 0.0023. Run-to-run
 * bit-identical. The workspace (device, >= ra_paged_extend_workspace_bytes, 256-byte aligned) is
 * overwritten; nothing in it is kept from call to call, so calls and captured graphs may share it as
 * long as they do not run at the same time. */
int ra_paged_attn_extend(const ra_paged_cache* c, const ra_shared_prefix* shared, int n_tokens, int hq,
                         float scale, int window, int sinks, const void* q, const int32_t* seq_lens,
                         const int32_t* cu_new, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Bytes of workspace of ra_paged_attn_extend (n_groups 0: nothing shared; with groups every row
 * has two float32 results in it); 0 for arguments that the call refuses. */
size_t ra_paged_extend_workspace_bytes(const ra_paged_cache* c, int n_groups, int n_tokens, int hq);

/* Natural order <-> shard-major order of a token tensor (row = one token, `row_bytes`
 * bytes: H*Dh*element size), bit-exact copy. direction 0: natural -> shard-major (shard);
 * 1: shard-major -> natural (unshard). src and dst must not overlap. */
int ra_shard_tokens(const ra_problem* p, int direction, const void* src, void* dst,
                    int64_t row_bytes, void* stream);

/* The same permutation for an lse tensor (float32, [B, Hq, S] or [Hq, T]). */
int ra_shard_lse(const ra_problem* p, int direction, const float* src, float* dst,
                 void* stream);

/* ---- host-side integer helpers (no GPU needed; the kernels use the same arithmetic) ---- */

/* 0 if the problem is valid, else the ra_status the compute calls would return. */
int ra_validate(const ra_problem* p);

/* Global positions of sequence `seq` (natural order index; batch element in batch mode):
 * pos_out[r*L + a] = global position of local token a of rank r, L = len/D. */
int ra_layout_positions(const ra_problem* p, int seq, int64_t* pos_out);

/* Per-row key counts of one (rank, step) block of sequence `seq`: the keys a local query
 * row may see in K/V shard (rank-step) mod D always form a prefix [0, count) of that
 * shard's local tokens (positions grow with the local index in every layout). Writes L
 * counts; count 0 = row sees nothing at this step, L = full row. *active_out (may be NULL)
 * is 1 if any row sees a key, i.e. the step is not skipped. */
int ra_step_counts(const ra_problem* p, int seq, int rank, int step, int32_t* count_out,
                   int32_t* active_out);

/* The work list the kernels run, in launch order. which = 0: forward (one item per
 * 256-query-row block of one rank and one query head); which = 1: backward (one item per
 * 128-row K/V tile of one rank and one K/V head). Each item is 4 int32: sequence, head,
 * rank, block index. Writes at most max_items items; returns the item count (or < 0). */
int ra_work_items(const ra_problem* p, int which, int32_t* items_out, int max_items);

/* ---- status ---- */

/* Synchronises the current device, then reports whether any kernel of this library gave
 * up a bounded wait since the last reset, or met an index outside a paged cache: RA_OK,
 * RA_ERR_DEVICE_TIMEOUT, else RA_ERR_CACHE_INDEX (RA_ERR_CUDA if the synchronisation itself
 * failed). reset != 0 clears the flags. */
int ra_check_device_status(int reset);

/* Test hook for the bounded-wait path: launches one CTA that waits, with a limit of
 * `timeout_ns` nanoseconds, on a shared-memory barrier that nothing completes, then gives
 * up, records RA_ERR_DEVICE_TIMEOUT in the device status and returns. */
int ra_test_wait_timeout(uint64_t timeout_ns, void* stream);

/* Test hook for the softmax's FMA-pipe exponential: y[i] = 2^x[i] for n device floats
 * x[i] <= 127, computed the way the forward kernel computes part of its exponentials
 * (range split and a degree-3 polynomial; relative error below 8e-5; inputs below -125
 * give 2^-125). */
int ra_test_exp2_poly(const float* x, float* y, int n, void* stream);

/* Profiling hook: while set (non-NULL), ra_ring_attn_fwd and ra_ring_attn_bwd record
 * `start_event` immediately before and `stop_event` immediately after their main kernels
 * (the fused forward; the backward's K/V-tile pass and query-tile dq pass, or its single
 * pass) on the call's stream, so a caller can time them alone with cudaEventElapsedTime.
 * Both are cudaEvent_t handles owned by the caller; pass NULL, NULL to switch the hook off.
 * Per calling thread. */
int ra_profile_events(void* start_event, void* stop_event);

/* Companion of ra_profile_events: while set (non-NULL), the two-pass backward records
 * `mid_event` between its K/V-tile pass and its dq pass. NULL switches it off. Per
 * calling thread. */
int ra_profile_split_event(void* mid_event);

/* Thread-local message describing the last error of this thread ("" if none). */
const char* ra_last_error(void);

/* RA_VERSION. */
int ra_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RINGATTN_H */
