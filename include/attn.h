/*
 * attn.h -- C ABI of the GB300 (sm_103a) fused exact-attention library.
 *
 * Exact scaled-dot-product attention, O = softmax(scale * Q K^T [+ causal
 * mask]) V, computed as one fused tiled kernel that keeps the running row
 * max m, running row sum l and an unnormalised O accumulator on chip, so the
 * N x N score and probability matrices never reach HBM.  The forward stores
 * O and the per-row log-sum-exp; the backward recomputes P from that LSE.
 *
 * Sources (web pages on FlashAttention):
 *   - FlashAttention (PKM page), "三招": 1 Tiling, 2 Online Softmax (the m / l /
 *     unnormalised-O recurrence and the final division by l), 3 Recomputation
 *     (store O and the softmax statistics, rebuild P in the backward).
 *   - FlashAttention深度攻略 (xiaohack page) §3 tiling into B_r query rows and
 *     B_c key/value rows, §4 online-softmax derivation, §6 recomputation
 *     backward, §7 kernel fusion, and the live-coding section whose module
 *     works on a (B*H, N, d) view after transposing (B, N, H, d) inputs.
 *   - "Flash Attention 到底做了什么？" (guanweilu page): exactness (differs from
 *     the plain computation only in floating-point rounding order).
 *
 * Conventions shared by every call
 *   - Tensors q, k, v, o, dO, dq, dk, dv are DEVICE pointers to contiguous
 *     row-major [B, H, N, d] arrays of the call's element type (bf16 for the
 *     unsuffixed calls, fp16 for the _f16 twins), 16-byte aligned.  This is
 *     the (B*H, N, d) view of the pages' module; a caller holding (B, N, H, d)
 *     tensors transposes first.
 *   - lse is a DEVICE pointer to fp32 [B, H, N]: LSE_i = ln sum_j
 *     exp(scale * q_i . k_j) over the keys visible to query i (natural log,
 *     in the same units as the scaled logits).
 *   - causal != 0 hides key j from query i iff j > i (square problem: query
 *     and key positions share one index).  scale multiplies Q K^T as given.
 *   - Supported: B, H, N >= 1; N <= 2^24; d in {32, 64, 128}; B*H <= 65535.
 *   - stream is a cudaStream_t (NULL = legacy default stream).  Every call
 *     only enqueues work on it and returns; results are ready when the
 *     stream is.  Calls on different streams that share outputs race.
 *   - All memory passed in is owned by the caller.  The library keeps no
 *     tensor between calls.  Outputs must not alias inputs.
 *   - Errors: argument errors are returned synchronously (nothing is
 *     enqueued).  A kernel that detects a problem on the device (a pipeline
 *     wait that exceeded its time limit) records a sticky status that
 *     attn_sync_status() returns; the kernel itself returns early instead of
 *     hanging, and its outputs are then unspecified.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, non-positive size, non-finite scale */
  ATTN_ERR_UNSUPPORTED = 2, /* head dim not in {32, 64, 128}, or sizes beyond the limits */
  ATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed (launch, allocation, ...) */
  ATTN_ERR_TIMEOUT = 4,     /* a device-side pipeline wait gave up (sticky, see attn_sync_status) */
  ATTN_ERR_ARCH = 5,        /* current device is not compute capability 10.3 (sm_103) */
  ATTN_ERR_DEVICE_CHECK = 6 /* a kernel's own device-side check failed (sticky): a page table, length or row
                               offset out of range (paged cache) */
} attn_status_t;

/*
 * Forward pass, bf16 inputs/outputs, fp32 accumulation.
 *   q, k, v : in,  [B, H, N, d] bf16
 *   o       : out, [B, H, N, d] bf16, O = softmax(scale Q K^T [+mask]) V
 *   lse     : out, [B, H, N] fp32, per-row log-sum-exp of the scaled logits
 * Tiling / online softmax / final 1/l division: FlashAttention (PKM page)
 * "三招" 1 and 2; FlashAttention深度攻略 §3-§4.
 * Returns an attn_status_t.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
             int N, int d, float scale, int causal, void* stream);

/*
 * Backward pass (recomputation), bf16.
 *   q, k, v, o, dO : in, [B, H, N, d] bf16 (o is attn_fwd's output for q, k, v)
 *   lse            : in, [B, H, N] fp32 from attn_fwd
 *   dq, dk, dv     : out, [B, H, N, d] bf16 gradients of L = <O, dO>:
 *                    P = exp(scale Q K^T - LSE) (rebuilt, never stored),
 *                    D_i = sum_k dO_ik O_ik, dS = P o (dO V^T - D),
 *                    dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO.
 * Recomputation: FlashAttention (PKM page) "三招" 3; FlashAttention深度攻略 §6.
 * Scratch: an fp32 dQ accumulator [B, H, N, d] and D [B, H, N] (plus, when
 * a non-causal grid's last partial wave is split over query halves, at most
 * (SMs / 2) x 4 fp32 128 x d tiles of partial dK/dV) are taken from the
 * stream-ordered allocator (cudaMallocAsync on `stream`) and freed on the
 * same stream before the call returns (the memory is released when the
 * stream reaches that point).
 */
int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
             const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
             float scale, int causal, void* stream);

/* fp16 twins: identical parameters and semantics with fp16 tensors. */
int attn_fwd_f16(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float scale, int causal, void* stream);
int attn_bwd_f16(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                 float scale, int causal, void* stream);

/*
 * Forward and backward with dropout fused into the softmax step (bf16, and
 * fp16 through the _f16 twins below;
 * FlashAttention深度攻略 §7, operator fusion: the softmax step of the fused
 * kernel also applies dropout).  Inverted dropout on P:
 *   t = floor((1 - p_drop) * 256 + 0.5) (in double), the keep probability
 *   rounded to a multiple of 1/256;
 *   keep_ij = [u_ij < t], u_ij = byte (j mod 4) of word (j mod 16) / 4 of
 *     Philox4x32-10(counter = (j / 16, i, b * H + h, offset),
 *                   key = (seed & 0xffffffff, seed >> 32))
 *     (Salmon, Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy as
 *     1, 2, 3", SC'11);
 *   O_i = (256 / t) sum_j keep_ij P_ij V_j; LSE is that of the undropped P.
 * The backward draws the same bytes again (nothing is stored) and returns the
 * gradients of L = <O, dO>: dV = (256/t) (keep o P)^T dO,
 * dS = P o ((256/t) keep o (dO V^T) - D), D_i = sum_k dO_ik O_ik,
 * dQ = scale dS K, dK = scale dS^T Q.  Pass the forward's p_drop, seed and
 * offset.  Other arguments, layouts, scratch and errors are those of
 * attn_fwd / attn_bwd; in addition ATTN_ERR_INVALID_ARG when p_drop is not in
 * [0, 1) or t would be 0 (p_drop > 1 - 1/512).  t = 256 (p_drop < 1/512) is
 * no dropout and runs attn_fwd / attn_bwd.
 */
int attn_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int H, int N, int d, float scale, int causal, float p_drop,
                     unsigned long long seed, unsigned int offset, void* stream);
int attn_bwd_dropout(const void* q, const void* k, const void* v, const void* o, const void* dO,
                     const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                     float scale, int causal, float p_drop, unsigned long long seed,
                     unsigned int offset, void* stream);
/* The same for fp16 q, k, v, o, dO, dq, dk, dv (the keep bytes are identical). */
int attn_fwd_dropout_f16(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int N, int d, float scale, int causal, float p_drop,
                         unsigned long long seed, unsigned int offset, void* stream);
int attn_bwd_dropout_f16(const void* q, const void* k, const void* v, const void* o, const void* dO,
                         const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                         float scale, int causal, float p_drop, unsigned long long seed,
                         unsigned int offset, void* stream);

/*
 * Block-sparse forward (bf16; fp16 through attn_fwd_blocksparse_f16): attn_fwd
 * where whole 128 x 128 tiles of the
 * score matrix are enabled or skipped by a block mask (FlashAttention深度攻略,
 * 进阶追问 "Sparse FlashAttention"; the tiles skipped are never loaded or
 * multiplied, generalising the causal tile skipping).
 *   block_mask : DEVICE pointer, [mask_heads][nb][nb] bytes, nb = ceil(N/128);
 *                head h uses mask (h % H) % mask_heads, mask_heads in {1, H}.
 *                Key j is visible to query i iff
 *                block_mask[..][i / 128][j / 128] != 0 (and j <= i if causal).
 *   A row that sees no key gets O = 0 and LSE = -inf.  N <= 262144 (else
 *   ATTN_ERR_UNSUPPORTED).
 */
int attn_fwd_blocksparse(const void* q, const void* k, const void* v, void* o, float* lse,
                         const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                         float scale, int causal, void* stream);
int attn_fwd_blocksparse_f16(const void* q, const void* k, const void* v, void* o, float* lse,
                             const unsigned char* block_mask, int mask_heads, int B, int H, int N,
                             int d, float scale, int causal, void* stream);

/*
 * Block-sparse backward (bf16; fp16 through attn_bwd_blocksparse_f16): the
 * gradients of attn_fwd_blocksparse's output
 * for the same block_mask, mask_heads and causal flag (o and lse from that
 * call).  The CTA of each 128-key tile visits only the query tiles whose mask
 * entry enables it; a key tile no query tile sees gets dK = dV = 0, and dQ
 * rows of a query block that sees no key are 0.  Scratch and errors as for
 * attn_bwd; the mask constraints as for attn_fwd_blocksparse.
 */
int attn_bwd_blocksparse(const void* q, const void* k, const void* v, const void* o, const void* dO,
                         const float* lse, void* dq, void* dk, void* dv,
                         const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                         float scale, int causal, void* stream);
int attn_bwd_blocksparse_f16(const void* q, const void* k, const void* v, const void* o,
                             const void* dO, const float* lse, void* dq, void* dk, void* dv,
                             const unsigned char* block_mask, int mask_heads, int B, int H, int N,
                             int d, float scale, int causal, void* stream);

/*
 * Block-sparse attention with dropout (both passes; bf16, fp16 through the
 * _f16 twins): the block mask of attn_fwd_blocksparse decides which keys a
 * query sees, and among those the keep rule of attn_fwd_dropout applies
 * unchanged -- keep_ij depends only on (i, j, b * H + h, seed, offset), not on
 * the mask (FlashAttention深度攻略 §7 fuses mask and dropout into the one
 * softmax step; 进阶追问 "Sparse FlashAttention" skips the masked tiles).
 * Arguments are those of attn_fwd_blocksparse / attn_bwd_blocksparse followed
 * by p_drop, seed and offset as for attn_fwd_dropout; the errors are the
 * union of both.  t = 256 runs the block-sparse kernels without dropout.
 */
int attn_fwd_blocksparse_dropout(const void* q, const void* k, const void* v, void* o, float* lse,
                                 const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                                 float scale, int causal, float p_drop, unsigned long long seed,
                                 unsigned int offset, void* stream);
int attn_fwd_blocksparse_dropout_f16(const void* q, const void* k, const void* v, void* o, float* lse,
                                     const unsigned char* block_mask, int mask_heads, int B, int H, int N,
                                     int d, float scale, int causal, float p_drop, unsigned long long seed,
                                     unsigned int offset, void* stream);
int attn_bwd_blocksparse_dropout(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                 const float* lse, void* dq, void* dk, void* dv,
                                 const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                                 float scale, int causal, float p_drop, unsigned long long seed,
                                 unsigned int offset, void* stream);
int attn_bwd_blocksparse_dropout_f16(const void* q, const void* k, const void* v, const void* o,
                                     const void* dO, const float* lse, void* dq, void* dk, void* dv,
                                     const unsigned char* block_mask, int mask_heads, int B, int H, int N,
                                     int d, float scale, int causal, float p_drop, unsigned long long seed,
                                     unsigned int offset, void* stream);

/*
 * Forward with FP8 (e4m3) inputs: q, k, v are [B, H, N, 128] e4m3 bytes whose
 * real values are descale_q*q, descale_k*k, descale_v*v (per-tensor factors,
 * finite and > 0); o is bf16 [B, H, N, 128], lse fp32 [B, H, N] in the units
 * of scale * Q_real K_real^T.  Same method as attn_fwd with 8-bit tensor-core
 * MMAs (FlashAttention (PKM page) 效果 table / FA3 note: FP8 as the further
 * gain); P is rounded to e4m3 for the P V product.  d must be 128 and
 * scale >= 0 (else ATTN_ERR_UNSUPPORTED).  Scratch: a transposed copy of V,
 * B*H*128*ceil(N/128)*128 bytes, from cudaMallocAsync on `stream` (freed on
 * it); launches 2 kernels.
 */
int attn_fwd_fp8(const void* q, const void* k, const void* v, float descale_q, float descale_k,
                 float descale_v, void* o, float* lse, int B, int H, int N, int d, float scale,
                 int causal, void* stream);

/*
 * Decode: exact attention of ONE query token per (batch, head) against a
 * key/value cache of L tokens (bf16), all L keys visible.
 *   q    : in,  [B, H, d] bf16 (the [B, H, 1, d] query of one decode step)
 *   k, v : in,  [B, H, L, d] bf16 cache
 *   o    : out, [B, H, d] bf16;  lse : out, [B, H] fp32
 * The keys of each (b, h) are split across CTAs and the partial results
 * (running max, sum, unnormalised output) merged exactly -- the decode
 * variant named in FlashAttention (PKM page), "注意" section, with the
 * online-softmax merge of "三招" 2.  Bound by reading the cache from HBM.
 * Scratch: B*H*splits*(d+2) floats from cudaMallocAsync on `stream`, freed
 * on it; launches 2 kernels.  Same conventions and errors as attn_fwd.
 */
int attn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                int L, int d, float scale, void* stream);

/*
 * Paged key/value cache: storage of ragged sequences for serving, filled by
 * attn_paged_append, read by attn_paged_decode and, in part, through
 * attn_paged_select.  The pages name decode as the case where no N x N matrix
 * exists and the cost is reading the cache (FlashAttention (PKM page), "注意");
 * the layout of the cache in pages is this library's.
 *
 * Sequence b's token at position p lies in page block_table[b][p / page_size],
 * slot p % page_size.  All arrays are caller-owned device memory; the struct
 * itself is host memory, read during the call only.
 *   k_pages, v_pages : [num_pages, kv_heads, page_size, head_dim] with strides
 *                (in elements) between pages, heads and tokens as given, the
 *                channels contiguous.  Strides are multiples of 16 bytes and
 *                such that no two rows overlap; an order of dimensions is not
 *                implied (pages of [page_size, kv_heads, head_dim], or K and V
 *                in turns in one array, are strides of their own).
 *   k_min, k_max : [num_pages, kv_heads, head_dim] contiguous, the cache's
 *                type: channelwise minimum and maximum of a page's keys as
 *                stored.  Both or neither; attn_paged_select needs them.
 *   block_table : [B, max_pages] int32, rows table_stride ints apart.  Entries
 *                behind a sequence's last page are never read.
 *   seq_lens   : [B] int32, tokens in the cache (0: the slot holds no sequence).
 *   type       : element type of the cache; bf16 and fp16 caches take rows of
 *                their own type, e4m3 either.  The value of an e4m3 element is
 *                k_scale (v_scale) times what is stored, finite and > 0; the
 *                scales of the other types are 1.
 *   Supported: head_dim in {32, 64, 128}; page_size a multiple of 8, at most
 *   1024; max_pages * page_size <= 2^30; B and kv_heads <= 65535, and B * kv_heads
 *   too (up to 8192 sequences: 2^20); query heads <= 65535, and B * query heads too
 *   where a key/value head has more than 1024.
 * Table entries and lengths are read on the device only, so a captured graph
 * may be replayed after they changed.  A page number outside [0, num_pages) or
 * a length outside [0, max_pages * page_size] is never followed: what it would
 * reach is left out, and attn_sync_status returns ATTN_ERR_DEVICE_CHECK.
 */
typedef enum { ATTN_TYPE_BF16 = 0, ATTN_TYPE_F16 = 1, ATTN_TYPE_E4M3 = 2 } attn_type_t;

typedef struct {
  void *k_pages, *v_pages;
  long long k_strides[3], v_strides[3]; /* page, head, token; elements */
  void *k_min, *k_max;                  /* or NULL */
  const int* block_table;
  const int* seq_lens;
  long long table_stride;
  int num_pages, page_size, kv_heads, head_dim, max_pages, B;
  int type; /* attn_type_t */
  float k_scale, v_scale;
} attn_paged_kv_t;

/* Token-major rows [rows, heads, head_dim], bf16 or fp16, channels contiguous:
 * strides in elements (multiples of 8; of no effect along an extent of 1), so
 * a slice of a projection's output needs no copy. */
typedef struct {
  void* data;
  long long row_stride, head_stride;
} attn_rows_t;

/*
 * Bookkeeping of a step: from the number of new tokens of each sequence the
 * block table's new entries, the lengths, token_start for attn_paged_append and
 * a slot for every new token.  Nothing is read on the host, so that a step can
 * be captured with the calls that use its results.
 *   kv   : block_table and seq_lens are written (the struct's other pointers are
 *          not followed).  Entries of pages that the sequence has are kept.
 *   n_new : in, [B] int32: new tokens of each sequence, 0 for none, or -1: the
 *          sequence is over, its pages are free again and its length 0.
 *   lens : in, [B] int32, tokens before the step; NULL: kv->seq_lens, in place.
 *   free_pages : in and out, [free_cap] int32: a ring of free page numbers;
 *          free_state : in, [2] int32: position of the first and number of them.
 *          New pages are taken from the front, for the sequences in ascending
 *          order and each one's pages in ascending order; pages of sequences that
 *          are over go behind the last (and can be taken from the next step on).
 *   free_out : out, [2] int32, free_state after the step; NULL: in place.
 *   token_start : out, [B + 1] int32: the sequences' first rows among the new
 *          tokens' rows, token_start[B] the number of all.
 *   slots : out, [rows] int64, or NULL: page * page_size + slot in the page of
 *          each new token; -1 for rows from token_start[B] on.
 *   rows : the most new tokens that the step may have; rows and free_cap at most 2^30.
 *   window, sinks : 0, 0, or those of attn_paged_decode_window.  A sequence then
 *          holds F = ceil(sinks / page_size) pages of sinks and
 *          R = ceil((window - 1) / page_size) + 1 others at most: entry j >= F + R
 *          repeats entry j - R, whose tokens have left the window.  Then at most
 *          R * page_size new tokens of one sequence in a step (they would share
 *          slots); of the calls that read a cache only attn_paged_decode_window, with
 *          that window or a narrower one and no more sinks, reads such a sequence rightly.
 * The step is done whole or not at all: lengths and free_state as before,
 * token_start 0, slots -1, and ATTN_ERR_DEVICE_CHECK through attn_sync_status.  It
 * is not done if
 *   - more pages are wanted than are free,
 *   - the pages that are free before the step and those that come back in it are
 *     more than free_cap, also where the step takes some, whose numbers the ring
 *     keeps (a ring of num_pages entries is never too small),
 *   - there are more new tokens than rows, or
 *   - a length, a count or free_state is out of range.
 * A page number outside [0, num_pages) in the ring or the table is handed on as
 * -1, with the same status.  With lens and free_out given the step can be taken
 * again from the same state (the ring and the table keep what it needs).
 *   workspace : attn_paged_assign_workspace() bytes, as for attn_paged_decode.
 * Launches 1 or 2 kernels.
 */
int attn_paged_assign(const attn_paged_kv_t* kv, const int* n_new, const int* lens, int* free_pages, int free_cap,
                      int* free_state, int* free_out, int* token_start, long long* slots, int rows, int window, int sinks,
                      void* workspace, void* stream);

/*
 * Appends new tokens' keys and values to the cache, with the position rotation
 * applied on the way.
 *   k, v    : in, [rows, kv_heads, head_dim] of x_type.
 *   q       : in, [rows, q_heads, head_dim], or NULL with q_heads = 0;
 *   q_out   : out, the rotated q; may be q itself (same strides) and must not
 *             overlap it otherwise.
 *   token_start : [B + 1] int32, ascending: rows token_start[b] .. token_start[b + 1] - 1
 *             are the last tokens of sequence b, at positions up to
 *             seq_lens[b] - 1 (seq_lens counts them already).  Rows outside
 *             [token_start[0], token_start[B]) are padding.  NULL: rows = B,
 *             row b is the last token of sequence b.
 *   cos, sin : [table_rows, rot_dim / 2] fp32, row p for position p; rot_dim a
 *             multiple of 16 up to head_dim (0: no rotation).  Channels (i,
 *             i + rot_dim / 2), or (2 i, 2 i + 1) if interleaved, turn by angle i
 *             in fp32: x1 cos - x2 sin, x2 cos + x1 sin; one rounding.
 * An e4m3 cache holds the fp32 quotient x / scale (x the row's element, or what
 * the rotation gives in fp32) rounded to nearest even, saturated at +-448 (NaN
 * stays NaN).  Summaries, where the cache has them: a page's is started by the
 * token in its first slot and widened by later ones (a NaN is passed over; a
 * channel of nothing but NaN keeps k_min = inf and k_max = -inf, in e4m3 NaN for
 * both, and so ranks its page first); after a sequence was cut back it still
 * covers the dropped tokens.
 * Slots with seq_lens[b] = 0 and rows of padding write nothing, nor do
 * positions at or past table_rows (ATTN_ERR_DEVICE_CHECK through
 * attn_sync_status, as for a token_start that is not ascending within rows
 * or gives a sequence more rows than tokens).  Two sequences must not append
 * to one page.  Launches 1 kernel (0 where rows = 0).
 */
int attn_paged_append(const attn_paged_kv_t* kv, const attn_rows_t* k, const attn_rows_t* v, const attn_rows_t* q,
                      const attn_rows_t* q_out, int q_heads, int rows, const int* token_start, const float* cos,
                      const float* sin, int table_rows, int rot_dim, int interleaved, int x_type, void* stream);

/*
 * Exact attention of one new token per sequence over the cache.
 *   q    : in,  [B, q_heads, head_dim] of x_type; query heads h * q_heads / kv_heads
 *          and following share key/value head h.
 *   o    : out, [B, q_heads, head_dim] contiguous, x_type
 *   lse  : out, [B, q_heads] fp32
 *   pages: NULL (all seq_lens[b] tokens), or [B, kv_heads, n_pages] int32 page
 *          indices within the sequence (attn_paged_select's output): attention
 *          over the tokens of those pages only, in any order, no page twice,
 *          negative entries behind the others (of a sequence of fewer than
 *          n_pages pages only as many entries are read as it has pages).
 *          Indices past the sequence's last page are skipped.
 *   scale : of the logits; finite, also times k_scale log2(e).
 * A sequence without visible tokens gets o = 0, lse = -inf.  Slots behind a
 * sequence's end may hold anything (NaN too).
 *   workspace : attn_paged_decode_workspace() bytes of device memory, 16-byte
 *          aligned, or NULL where that is 0; the call's own until it is done.
 * Launches at most 2 kernels.
 */
int attn_paged_decode(const attn_paged_kv_t* kv, const attn_rows_t* q, int q_heads, void* o, float* lse,
                      const int* pages, int n_pages, float scale, int x_type, void* workspace, void* stream);

/*
 * attn_paged_decode for a model with a sliding window: the new token, which is a
 * sequence's last, sees its last `window` tokens (itself among them) and its
 * first `sinks` ones, as a query of attn_fwd_window.  Only the pages that hold
 * those are looked up and read, so the table entries of others may be anything,
 * and pages of tokens that have left the window may be in use elsewhere.
 *   window >= 1, sinks >= 0, both at most 2^30.
 *   workspace : attn_paged_decode_window_workspace() bytes.
 * Everything else as for attn_paged_decode.
 */
int attn_paged_decode_window(const attn_paged_kv_t* kv, const attn_rows_t* q, int q_heads, void* o, float* lse,
                             int window, int sinks, float scale, int x_type, void* workspace, void* stream);

/*
 * For each sequence and key/value head the n_select pages on which the new
 * token's queries can have their largest logits (scale > 0):
 *   score(p) = max over the head's query heads g of
 *              sum_c max(q_gc k_min[p]_c, q_gc k_max[p]_c),
 * an upper bound of q_g . k over the page's keys.  The first keep_first and the
 * last keep_last pages (their sum at most n_select) are taken whatever their
 * score; of equal scores the lower index.  Scores count to 53 bits or more of
 * their terms' magnitude (not an fp32 sum's 20).  A NaN score ranks first.
 *   pages : out, [B, kv_heads, n_select] int32, ascending; a sequence of fewer
 *           pages gets all of them, then -1.
 *   workspace : attn_paged_select_workspace() bytes, as for attn_paged_decode.
 */
int attn_paged_select(const attn_paged_kv_t* kv, const attn_rows_t* q, int q_heads, int* pages, int n_select,
                      int keep_first, int keep_last, int x_type, void* workspace, void* stream);

/* Bytes of workspace (0 for sizes that the calls reject).  n_pages as for
 * attn_paged_decode, 0 for all pages.  They depend on the sizes only. */
long long attn_paged_decode_workspace(const attn_paged_kv_t* kv, int q_heads, int n_pages);
long long attn_paged_decode_window_workspace(const attn_paged_kv_t* kv, int q_heads, int window, int sinks);
long long attn_paged_select_workspace(const attn_paged_kv_t* kv);
long long attn_paged_assign_workspace(const attn_paged_kv_t* kv);

/* [B, heads, N, d] of bf16 or fp16 with contiguous channels, strides in elements:
 * multiples of 8 (of no effect along an extent of 1) and such that no two rows
 * overlap; an order of dimensions is not implied, so [B, N, heads, d] and slices
 * of a projection's output need no copy. */
typedef struct {
  void* data;
  long long batch_stride, head_stride, row_stride;
} attn_bhnd_t;

/*
 * Causal attention with a sliding window and sinks, the first tokens, which stay
 * visible; query heads may share key/value heads.
 *   q, o : in and out, [B, q_heads, Nq, d];  k, v : in, [B, kv_heads, Nk, d],
 *          Nk >= Nq; q_heads a multiple of kv_heads: query heads
 *          h * q_heads / kv_heads and following share key/value head h.
 *   lse  : out, [B, q_heads, Nq] fp32
 * The queries are the last Nq of Nk positions: query i stands at
 * p = i + Nk - Nq and sees key j iff j <= p and (j > p - window or j < sinks).
 *   window >= 1 (Nk or more: the causal mask), sinks >= 0.
 *   type : ATTN_TYPE_BF16 or ATTN_TYPE_F16, of all four tensors.
 * The tiles of keys that no query of a 128-row tile sees are neither loaded nor
 * multiplied (FlashAttention深度攻略, 进阶追问 "Sparse FlashAttention", for a
 * mask that is not made of tiles).  The inputs must be finite, also where the mask
 * hides them (padding at a sequence's end, say): inside a tile a hidden key has
 * weight 0, and 0 times inf is NaN.
 * Supported: d in {32, 64, 128}, Nk <= 2^24, B * q_heads <= 65535, finite scale.
 * The outputs must not overlap the inputs or one another; slices of one buffer
 * whose rows take turns do not.  Launches 1 kernel.
 */
int attn_fwd_window(const attn_bhnd_t* q, const attn_bhnd_t* k, const attn_bhnd_t* v, const attn_bhnd_t* o, float* lse,
                    int B, int q_heads, int kv_heads, int Nq, int Nk, int d, int window, int sinks, float scale, int type,
                    void* stream);

/*
 * The gradients of attn_fwd_window's output for the same window, sinks and scale
 * (o and lse from that call), as attn_bwd's; dk and dv are the sums over the
 * query heads that share a key/value head, and 0 for keys that no query sees.
 * A call repeats bit for bit.
 * With fp16 P and dS are operands of 16-bit products in a range of their own, by
 * powers of two taken from the largest rows of dO and v, so that gradients far below
 * or above 1 keep their bits: for dQ down to 2^-28 of 2 |dO row| |v row|, for dK of
 * that with the largest row of dO of the query heads that share the key.
 *   workspace : attn_bwd_window_workspace() bytes of device memory, 16-byte aligned,
 *          the call's own until it is done: two fp32 row vectors, fp32 partial tiles
 *          of dK and dV where a tile of keys has many more queries than others
 *          (the sinks) or there are few of them, and those largest rows.
 * Launches 2 or 3 kernels, with fp16 one more.
 */
int attn_bwd_window(const attn_bhnd_t* q, const attn_bhnd_t* k, const attn_bhnd_t* v, const attn_bhnd_t* o,
                    const attn_bhnd_t* dO, const float* lse, const attn_bhnd_t* dq, const attn_bhnd_t* dk,
                    const attn_bhnd_t* dv, int B, int q_heads, int kv_heads, int Nq, int Nk, int d, int window, int sinks,
                    float scale, int type, void* workspace, void* stream);

/* Bytes of workspace (0 for sizes that the call rejects).  They depend on the sizes only. */
long long attn_bwd_window_workspace(int B, int q_heads, int kv_heads, int Nq, int Nk, int d, int window, int sinks);

/*
 * attn_bwd without any memory allocation (bf16).  The pages have no
 * counterpart: this is a deployment variant of attn_bwd.
 *
 * For callers that may not allocate device memory inside the call: code that
 * runs while an allocator must not be re-entered, runtimes that freeze device
 * allocations once a fixed memory budget is set up, or hosts that give the
 * library only the tensors.  Parameters, layouts, ownership and results are
 * those of attn_bwd; the difference is where the scratch lives.  Instead of
 * the stream-ordered allocator it uses one fixed array of 34,078,720 bytes
 * (32.5 MiB) in device memory owned by the library (a GPU that loads the
 * array keeps it until the process exits).  The scratch a problem needs is
 *     align256(4*B*H*N*d) + 2 * align256(4*B*H*ceil(N/128)*128)   bytes;
 * B=1, H=8, N=8192, d=128 needs exactly the whole array.  A problem needing
 * more is rejected with ATTN_ERR_UNSUPPORTED before anything is enqueued
 * (use attn_bwd for it).
 *   - The first call on each device looks up the array's device address on
 *     that device and caches it for the life of the process; make that first
 *     call before any stream capture.  cudaDeviceReset discards the array
 *     together with the context: do not call attn_bwd_noalloc on a device
 *     after resetting it in the same process.
 *   - Every call on a device shares the one array.  A call rewrites all of
 *     the scratch it reads, so it does not depend on what an earlier call
 *     left there, but two calls that can run at the same time on the GPU
 *     (different streams, or different host threads) race on it and give
 *     wrong gradients: order them on one stream or synchronise in between.
 */
int attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                     const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                     float scale, int causal, void* stream);

/*
 * Synchronises `stream`, then returns and clears the sticky device status of
 * the current device (ATTN_OK, ATTN_ERR_TIMEOUT or ATTN_ERR_DEVICE_CHECK), or
 * ATTN_ERR_CUDA if the synchronisation itself failed.
 */
int attn_sync_status(void* stream);

/* Static, human-readable name of a status code (never NULL). */
const char* attn_status_string(int status);

/* Number of kernel launches the most recent successful attn_fwd* / attn_bwd* /
 * attn_decode / attn_paged_* call on this thread enqueued (forward 1, backward 3,
 * decode 2, window backward 2 to 4, paged append 1, paged decode 1 or 2, paged select 2,
 * paged assign 1 or 2). */
int attn_last_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
