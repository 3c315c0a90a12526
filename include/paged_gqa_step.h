/*
 * paged_gqa_step.h -- the operators one step of a model runs around paged
 * attention on a cache held in 8 bits with one scale for each block of tokens
 * and KV head.  paged_gqa.h has attention over FP16 caches and over E4M3
 * caches with one scale per tensor, and the top-k/top-p masking that ends a
 * step; its conventions (pointers, streams, status codes, err_flag, KV
 * layouts, head groups) hold here too.
 *
 * Further conventions
 * -------------------
 *  * PAGED_GQA_F16 / BF16 / F32 name element types of rows that are not in a
 *    cache.  Strides are in elements and not negative.
 *  * Where a tensor is written, its rows must not overlap one another, nor
 *    the tensors the call reads, except where in-place use is stated.
 *  * No entry point here keeps anything between calls but a per-device cache
 *    of device attributes; two calls on two streams are independent as long
 *    as their outputs (and a workspace, where there is one) are.
 */
#ifndef PAGED_GQA_STEP_H
#define PAGED_GQA_STEP_H

#include "paged_gqa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of q, k, v rows and logits. */
typedef enum {
    PAGED_GQA_F16 = 0,
    PAGED_GQA_BF16 = 1,
    PAGED_GQA_F32 = 2
} paged_gqa_float_dtype;

/* KV type of the block-scaled caches besides PAGED_GQA_KV_E4M3: signed bytes. */
#define PAGED_GQA_KV_INT8 2

/* Further bits ORed into *err_flag. */
#define PAGED_GQA_FLAG_BAD_VALUE  256  /* append: an element or a stored scale is not finite (or a scale negative) */
#define PAGED_GQA_FLAG_BAD_INDEX  512  /* logits: a token id >= V, or a mask row outside the masks: skipped */

/* Strides of the scale tensors in elements (floats).  The scale of rows
 * i * scale_block .. (i + 1) * scale_block - 1 of (page, kv_head) lies at
 *     scales + page * page_stride + i * block_stride + kv_head * head_stride,
 * and an element is code value * scale.  K and V have a scale tensor each, of
 * one layout. */
typedef struct {
    int64_t page_stride;
    int64_t block_stride;
    int64_t head_stride;
} paged_gqa_scale_layout;

/* ------------------------------------------------------------ rotary positions */

/* How the pairs of a rotated row lie: (i, i + rot/2), or (2i, 2i + 1). */
#define PAGED_GQA_ROPE_HALF        0
#define PAGED_GQA_ROPE_INTERLEAVED 1

/* Frequency scaling for long contexts (paged_gqa_rope_frequencies). */
#define PAGED_GQA_ROPE_SCALE_NONE   0
#define PAGED_GQA_ROPE_SCALE_LINEAR 1
#define PAGED_GQA_ROPE_SCALE_BASE   2
#define PAGED_GQA_ROPE_SCALE_RAMP   3

/* H heads of T tokens: row (t, h) starts at x + t * token_stride + h *
 * head_stride and is written at the same place of out with out's strides. */
typedef struct {
    const void* x;
    void* out;
    int64_t token_stride, head_stride;
    int64_t out_token_stride, out_head_stride;
    int heads;
} paged_gqa_rope_rows;

/*
 * Rotary positions of q and k.  With angle a = positions[t] * inv_freq[i],
 * pair i of every row of token t, (u, v), becomes
 *     scale * (u cos a - v sin a,  v cos a + u sin a),
 * or with inverse != 0 the rotation by -a (the transpose; with scale = 1 it
 * undoes the rotation, and it is the gradient's map).  Elements from rot_dim
 * on pass through unchanged and unscaled.
 *  q, k        k may be NULL.  out == x with equal strides rotates in place.
 *  dtype       PAGED_GQA_F16, BF16 or F32 (of x and out).
 *  D           1 .. 4096 elements per row.
 *  rot_dim     even, 0 .. D.
 *  layout      PAGED_GQA_ROPE_HALF or PAGED_GQA_ROPE_INTERLEAVED.
 *  positions   device int32 [T]; any value, negative ones included.
 *  inv_freq    device float64 [rot_dim / 2], radians per position.  Angles are
 *              reduced to a turn exactly (64-bit fixed point), so far
 *              positions lose nothing.
 * Arithmetic is float32, rounded once to dtype.  One kernel is launched.
 */
int paged_gqa_rope(const paged_gqa_rope_rows* q, const paged_gqa_rope_rows* k, int T, int D,
                   int dtype, const int32_t* positions, const double* inv_freq, int rot_dim,
                   int layout, float scale, int inverse, void* stream);

/*
 * inv_freq of rot_dim / 2 pairs into host memory: f_i = base^(-2i / rot_dim),
 * scaled for contexts longer than the trained one by
 *   NONE    f_i
 *   LINEAR  f_i / factor
 *   BASE    base replaced by base * factor^(rot_dim / (rot_dim - 2))
 *           (the slowest pair ends up at f / factor, the fastest unchanged)
 *   RAMP    f_i (g + (1 - g) / factor), g = clamp((r_i - low) / (high - low), 0, 1)
 *           with r_i = original_len * f_i / 2 pi, the turns of pair i over the
 *           trained context: pairs of many turns stay, those of few are
 *           stretched.
 * Host only.  Returns PAGED_GQA_ERR_SHAPE unless rot_dim is even and >= 2,
 * base and factor are finite and > 0, and for RAMP original_len > 0 and
 * high > low.
 */
int paged_gqa_rope_frequencies(double* inv_freq, int rot_dim, double base, int scaling,
                               double factor, double original_len, double low, double high);

/* ------------------------------------------------------------ quantising append */

/*
 * Quantises new K and V rows into the paged cache.  Sequence b's new tokens
 * are the rows new_offsets[b] .. new_offsets[b + 1] - 1 of k and v (row b
 * alone when new_offsets is NULL), and take its positions seq_starts[b],
 * seq_starts[b] + 1, ...; seq_starts[b] tokens are stored already.
 *
 * A scale block is scale_block consecutive tokens of a page.  For every
 * (block, KV head) that gets new rows, with m the largest magnitude of their
 * finite elements,
 *     E4M3   s_new = the smallest power of two with m <= 448 s_new (the code
 *            has its own exponent, so a power of two costs no precision, and
 *            stored rows change scale without loss until they turn subnormal)
 *     INT8   s_new = m / 127 in float32
 *     s      = s_new, or max(s_old, s_new) where the block holds stored rows
 *     code   = round to nearest even of x / s (0 where s = 0)
 * and where s > s_old the block's stored rows are coded again,
 * code' = round to nearest even of code * s_old / s.  Quotients are rounded
 * once.  Infinities saturate (0 where s = 0), NaN becomes the E4M3 NaN or INT8 0;
 * both are flagged and do not count for m (PAGED_GQA_FLAG_BAD_VALUE).  A stored scale
 * that is negative, infinite or NaN counts as 0, its rows as zeros (same flag).
 * Appending the same rows at the same positions again changes nothing.
 *
 *  k, v           device rows (t, head) of D elements of src_dtype at
 *                 t * token_stride + head * head_stride, 16-byte aligned
 *                 (strides too); K and V have strides of their own.
 *  T              rows of k and v; rows behind new_offsets[B] belong to no
 *                 sequence and are ignored.
 *  k_cache ...    pools as for decode, of kv_dtype PAGED_GQA_KV_E4M3 or
 *                 PAGED_GQA_KV_INT8; rows must not overlap.
 *  k_scales ...   device float32, see paged_gqa_scale_layout.
 *  scale_block    >= 1, divides page_size.
 *  block_table    device int32, rows of >= ceil(max_seq_len / page_size) entries.
 *  seq_starts     device int32 [B]; a negative one drops the sequence's rows
 *                 (PAGED_GQA_FLAG_EMPTY_ROW).
 *  new_offsets    device int32 [B + 1], not decreasing, from 0 to at most T; or NULL (then T = B).
 *  max_seq_len    rows at positions from here on are dropped
 *                 (PAGED_GQA_FLAG_SEQ_CLAMPED), rows on pages outside the
 *                 pool too (PAGED_GQA_FLAG_BAD_PAGE).
 * The pages written must belong to one sequence each, and to one place of its
 * table row: rows written to one block from two places race.  Results are deterministic.  One kernel is
 * launched; no workspace.
 */
int paged_gqa_append_scaled(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                            const void* v, int64_t v_token_stride, int64_t v_head_stride,
                            int src_dtype, int T, void* k_cache, void* v_cache,
                            paged_gqa_kv_layout kv_layout, int kv_dtype, float* k_scales,
                            float* v_scales, paged_gqa_scale_layout scale_layout, int scale_block,
                            const int32_t* block_table, int64_t bt_row_stride,
                            const int32_t* seq_starts, const int32_t* new_offsets, int B, int Hkv,
                            int D, int page_size, int num_pages, int max_seq_len, int* err_flag,
                            void* stream);

/* ------------------------------------------------------------ attention */

/*
 * Bytes of workspace paged_gqa_decode_scaled needs for this shape on the
 * current CUDA device: with its automatic split (splits = 0), or with
 * paged_gqa_workspace.force_splits = splits.  0 for invalid shapes and for
 * batches above 4096, which need none.  Host only.
 */
size_t paged_gqa_decode_scaled_workspace_size(int B, int Hq, int Hkv, int D, int splits);

/*
 * paged_gqa_decode over a block-scaled cache: with element = code * scale,
 *     out[b, h, :] = sum_{t < L} softmax_t(softmax_scale * <q[b,h,:], K_t>) V_t
 * over the tokens whose page is valid.  Arguments, flags and inert inputs as
 * for paged_gqa_decode, but for
 *  kv_dtype      PAGED_GQA_KV_E4M3 or PAGED_GQA_KV_INT8.
 *  k_scales,     device float32, finite and >= 0 for every block with an
 *  v_scales      attended token (others are not read).
 *  scale_block   >= 1, divides page_size.
 *  kv_layout     the pool spans fewer than 2^32 times the largest power of two
 *                that divides its three strides (1 TB where rows are contiguous;
 *                PAGED_GQA_ERR_UNSUPPORTED otherwise).
 *  ws            with a workspace (paged_gqa_decode_scaled_workspace_size
 *                bytes) the call may share all sequences' tokens among CTAs and
 *                merge their results in a second kernel, which long contexts
 *                need; it does so where that is the faster way for B, Hkv and
 *                max_seq_len, and always with force_splits.  Otherwise, and
 *                without a workspace or for a batch above 4096 whatever
 *                force_splits says, a cluster of up to 8 CTAs takes each
 *                (sequence, KV head) in one kernel.  A workspace shared by two
 *                calls in flight races.
 * Results are deterministic for a given device, shape and workspace choice.
 * Elements above binary16's range give infinities in out, NaN codes NaN.
 */
int paged_gqa_decode_scaled(const void* q, const void* k_cache, const void* v_cache,
                            paged_gqa_kv_layout kv_layout, int kv_dtype, const float* k_scales,
                            const float* v_scales, paged_gqa_scale_layout scale_layout,
                            int scale_block, const int32_t* block_table, int64_t bt_row_stride,
                            const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int page_size,
                            int num_pages, int max_seq_len, float softmax_scale, void* out,
                            const paged_gqa_workspace* ws, void* stream);

/*
 * paged_gqa_sparse_prefill over a block-scaled cache: the same rows, inert inputs
 * and flags, the cache as for paged_gqa_decode_scaled.  One kernel; where rows are
 * few, a cluster of up to 8 CTAs takes each (row, KV head).
 */
int paged_gqa_sparse_prefill_scaled(const void* q, const void* k_cache, const void* v_cache,
                                    paged_gqa_kv_layout kv_layout, int kv_dtype,
                                    const float* k_scales, const float* v_scales,
                                    paged_gqa_scale_layout scale_layout, int scale_block,
                                    const int32_t* block_table, int num_pages, int kv_len,
                                    const int32_t* sel_idx, int n_sel, const int32_t* q_pos, int R,
                                    int Hq, int Hkv, int D, int page_size, float softmax_scale,
                                    void* out, int* err_flag, void* stream);

/* ------------------------------------------------------------ logits */

/* What changes a step's logits; every part is optional (NULL pointers).
 *  history        device int32, row b of max_history entries at history +
 *                 b * history_stride: the token ids of sequence b so far,
 *                 history_lens[b] of them (device int32 [B], clamped to 0 ..
 *                 max_history; NULL: max_history).  Negative ids are padding.
 *                 The first prompt_lens[b] (NULL: 0) are the prompt's, the
 *                 others were generated.
 *  repetition     device float32 [B], > 0: logits of all tokens in the history
 *                 are divided by it where positive and multiplied where not.
 *  frequency,     device float32 [B]: logits lose frequency * count + presence
 *  presence       for tokens generated count > 0 times.
 *  bias_tokens,   device [B, n_bias] rows at bias_stride: bias_values[b, i]
 *  bias_values    (float32) is added to the logit of bias_tokens[b, i] (int32;
 *                 negative ones are padding); a token's entries are summed in
 *                 their order first.
 *  mask           device words, mask_rows rows at mask_stride: token v is
 *                 allowed where bit v % 32 of word v / 32 is set, otherwise its
 *                 logit is -infinity.  Row b takes mask row mask_index[b]
 *                 (device int32 [B]; negative: no mask), or row b when
 *                 mask_index is NULL (then mask_rows >= B). */
typedef struct {
    const int32_t* history;
    int64_t history_stride;
    int max_history;
    const int32_t* history_lens;
    const int32_t* prompt_lens;
    const float* repetition;
    const float* frequency;
    const float* presence;
    const int32_t* bias_tokens;
    const float* bias_values;
    int64_t bias_stride;
    int n_bias;
    const uint32_t* mask;
    int64_t mask_stride;
    int mask_rows;
    const int32_t* mask_index;
} paged_gqa_logit_rules;

/*
 * Penalties, biases and grammar masks on a step's logits, in this order:
 *     y = x / r or x * r (repetition);  y -= frequency * count + presence;
 *     y += bias;  y = -infinity where the mask forbids the token
 * in float32.  Its result is what paged_gqa_topk_topp_mask takes.
 *  logits      device rows of V elements of dtype at logits_stride.
 *  out         device float32 rows at out_stride; out == logits with equal
 *              strides and dtype PAGED_GQA_F32 works in place.
 *  rules       NULL: the logits as float32.
 *  B, V        0 .. 65535 rows, 1 .. 2^31 - 8193 columns; max_history and
 *              n_bias at most 2^28.
 * Tokens out of range are skipped (PAGED_GQA_FLAG_BAD_INDEX).  A row whose
 * mask allows nothing becomes -infinity throughout.  Results are
 * deterministic.  One kernel is launched; no workspace.
 */
int paged_gqa_logits_process(const void* logits, int64_t logits_stride, int dtype, float* out,
                             int64_t out_stride, int B, int V, const paged_gqa_logit_rules* rules,
                             int* err_flag, void* stream);

/* ------------------------------------------------------------ calls by structure */

/* The arguments of the functions above in their order, for callers to whom a call
 * of many arguments is dear (the Python binding packs them in one go).  Each
 * _call function does what its namesake does and returns the same status. */
typedef struct {
    paged_gqa_rope_rows q, k;      /* k.heads == 0: no k */
    const int32_t* positions;
    const double* inv_freq;
    void* stream;
    int T, D, dtype, rot_dim, layout;
    float scale;
    int inverse;
} paged_gqa_rope_args;

typedef struct {
    const void* k;
    int64_t k_token_stride, k_head_stride;
    const void* v;
    int64_t v_token_stride, v_head_stride;
    void *k_cache, *v_cache;
    paged_gqa_kv_layout kv_layout;
    float *k_scales, *v_scales;
    paged_gqa_scale_layout scale_layout;
    const int32_t* block_table;
    int64_t bt_row_stride;
    const int32_t *seq_starts, *new_offsets;
    int* err_flag;
    void* stream;
    int src_dtype, T, kv_dtype, scale_block, B, Hkv, D, page_size, num_pages, max_seq_len;
} paged_gqa_append_scaled_args;

typedef struct {
    const void *q, *k_cache, *v_cache;
    paged_gqa_kv_layout kv_layout;
    const float *k_scales, *v_scales;
    paged_gqa_scale_layout scale_layout;
    const int32_t* block_table;
    int64_t bt_row_stride;
    const int32_t* seq_lens;
    void* out;
    void* workspace;
    size_t workspace_bytes;
    int* err_flag;
    void* split_events[2];
    void* stream;
    int kv_dtype, scale_block, B, Hq, Hkv, D, page_size, num_pages, max_seq_len, force_splits;
    float softmax_scale;
} paged_gqa_decode_scaled_args;

typedef struct {
    const void *q, *k_cache, *v_cache;
    paged_gqa_kv_layout kv_layout;
    const float *k_scales, *v_scales;
    paged_gqa_scale_layout scale_layout;
    const int32_t *block_table, *sel_idx, *q_pos;
    void* out;
    int* err_flag;
    void* stream;
    int kv_dtype, scale_block, num_pages, kv_len, n_sel, R, Hq, Hkv, D, page_size;
    float softmax_scale;
} paged_gqa_sparse_prefill_scaled_args;

typedef struct {
    const void* logits;
    int64_t logits_stride;
    float* out;
    int64_t out_stride;
    paged_gqa_logit_rules rules;
    int* err_flag;
    void* stream;
    int dtype, B, V;
} paged_gqa_logits_process_args;

int paged_gqa_rope_call(const paged_gqa_rope_args* args);
int paged_gqa_append_scaled_call(const paged_gqa_append_scaled_args* args);
int paged_gqa_decode_scaled_call(const paged_gqa_decode_scaled_args* args);
int paged_gqa_sparse_prefill_scaled_call(const paged_gqa_sparse_prefill_scaled_args* args);
int paged_gqa_logits_process_call(const paged_gqa_logits_process_args* args);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_GQA_STEP_H */
