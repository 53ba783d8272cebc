/*
 * lsa_kv8.h - C ABI of the 8-bit K/V cache of the Lookahead Sparse Attention (LSA) decode step.
 *
 * The decode step is bound by reading the kept chunks' K/V. These calls keep that cache in 8 bits:
 * they prepare a new token's queries and keys, write K/V quantised, read it back, and attend over it.
 * The conventions are those of lsa.h (device pointers, 16-byte alignment, asynchronous on `stream`,
 * validation on the host before anything is launched, the sticky error word of the workspace, CUDA
 * graph capture); calls that share a workspace must not overlap on the GPU.
 *
 * The cache. A value is stored as float8_e4m3 times a float32 scale that a block of `scale_block`
 * consecutive tokens of one K/V head shares. Chunk i of the flattened chunk axis (lsa_dims) holds, for
 * each K/V head, its chunk_len token rows side by side, so that a (chunk, head) is one contiguous run:
 *   K8, V8           [sum N_b][n_kv_heads][chunk_len][Dh]         float8_e4m3 (1 byte a value)
 *   k_scale, v_scale [sum N_b][n_kv_heads][chunk_len/scale_block] float32
 * The scales that lsa_kv8_append writes are powers of two, so a block whose scale grows is rescaled
 * without a further rounding (but for values that become e4m3 subnormals). A cache written by other
 * means may hold any finite scale of 2^-126 or more.
 *
 * Grouped heads: lsa_dims.H query heads share n_kv_heads K/V heads; query head h reads K/V head
 * h / (H / n_kv_heads).
 *
 * Lengths: where a call takes seq_len ([B] int32, device, nullable), only the first seq_len[b] tokens of
 * sequence b's cache exist (clamped to 0..N_b * chunk_len; NULL: all of them). Rows behind them are
 * never used, whatever they hold.
 */
#ifndef LSA_KV8_H_
#define LSA_KV8_H_

#include "lsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache's shape and its device pointers. Host memory; copied by value into the launch. */
typedef struct {
    int32_t n_kv_heads;   /* a power of two that divides lsa_dims.H */
    int32_t scale_block;  /* tokens to a scale: 8, 16, 32 or 64, at most chunk_len */
    void *K8, *V8;        /* 16-byte aligned */
    float *k_scale, *v_scale;
} lsa_kv8_cache;

/* Preparation of queries and keys: RMS norm of each head's Dh values, then the position's rotation.
 *   y   = x / sqrt(mean(x^2) + eps) * weight        (weight == NULL: y = x)
 *   a_i = position * inv_freq[i], i < rot_dim/2     (the product and its reduction in 64 bits)
 *   (y_p, y_r) <- (y_p cos a_i - y_r sin a_i, y_r cos a_i + y_p sin a_i)
 * with the pair (p, r) = (i, i + rot_dim/2), or (2i, 2i + 1) if `interleaved`. Values from rot_dim on
 * are not rotated. Computed in fp32, the mean of squares too (values below 2^60), and rounded once to kv_dtype. */
typedef struct {
    int32_t rot_dim;         /* a multiple of 16, 0..Dh */
    int32_t interleaved;     /* 0 or 1 */
    float eps;               /* >= 0, finite */
    const float *inv_freq;   /* device [rot_dim/2]; may be NULL if rot_dim is 0 */
    const float *q_weight;   /* device [Dh], 16-byte aligned, or NULL: queries are not normed */
    const float *k_weight;   /* device [Dh], 16-byte aligned, or NULL: keys are not normed */
} lsa_qk_prep;

/* Bytes of device workspace that the calls below need for `dims` and `cache` (its pointers are not
 * looked at); at least lsa_workspace_size(dims), so that the workspace also serves the calls of lsa.h.
 * Initialise it with lsa_workspace_init. */
LSA_API lsa_status lsa_kv8_workspace_size(const lsa_dims *dims, const lsa_kv8_cache *cache, size_t *bytes);

/* Norm and rotation of a run of tokens' queries and keys in one pass (the prefill's form, and any call
 * that needs the prepared rows themselves). Of `dims` it uses H, Dh and kv_dtype.
 *   positions  [n_tok] int32
 *   q          n_tok rows of [H][Dh] kv_dtype, q_stride elements from one token to the next, or NULL
 *   k          n_tok rows of [n_kv_heads][Dh] kv_dtype, k_stride elements apart, or NULL
 *   q_out, k_out  the same shapes, *_out_stride elements apart; NULL where the input is NULL. May be
 *              the input itself (same pointer and stride), and must not overlap it in another way.
 * Strides are multiples of 16 bytes and at least a row, so that rows may lie inside a packed
 * projection [n_tok][(H + 2 n_kv_heads) * Dh]. n_tok == 0 does nothing. */
LSA_API lsa_status lsa_qk_norm_rope(const lsa_dims *dims, int32_t n_kv_heads, const lsa_qk_prep *prep,
                                    int64_t n_tok, const int32_t *positions, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, void *q_out, int64_t q_out_stride,
                                    void *k_out, int64_t k_out_stride, void *stream);

/* Write new token rows to the cache, quantised.
 *   prep       NULL: k is written as it is; else k is prepared first (k_weight, position start[b] + i)
 *              and rounded to kv_dtype, as lsa_qk_norm_rope would store it
 *   n_new      rows per sequence, >= 1
 *   k, v       [B][n_new] rows of [n_kv_heads][Dh] kv_dtype, k_stride / v_stride elements from one row
 *              to the next (a multiple of 16 bytes); sequence b's rows start at row b * n_new
 *   start      [B] int32 device: tokens that sequence b's cache holds already; row i becomes token
 *              start[b] + i. NULL: 0 for every sequence
 *   new_count  [B] int32 device: only the first new_count[b] rows are written (clamped to 0..n_new);
 *              NULL: all n_new
 * Per block of scale_block tokens and head, with amax the largest finite |x| of its new rows:
 *   scale = the least power of two >= 2^-120 with amax <= 448 * scale;
 *   a block that holds older tokens (below start) keeps the larger of its scale and that one, and if the
 *   scale grows its older codes are requantised: e4m3(code * old_scale / new_scale);
 *   code  = e4m3(x / scale), to nearest, ties to even.
 * Non-finite rows set LSA_ERR_NONFINITE: an infinity is stored as +-448 * scale, a NaN as NaN. Rows
 * past the cache's end (or start < 0) are not written and set LSA_ERR_BAD_ID. Nothing else of the cache
 * is touched. */
LSA_API lsa_status lsa_kv8_append(const lsa_dims *dims, const lsa_kv8_cache *cache, const lsa_qk_prep *prep,
                                  int32_t n_new, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                  const int32_t *start, const int32_t *new_count, void *ws, size_t ws_bytes,
                                  void *stream);

/* Read chunks back into resident buffers of the 16- or 32-bit cache's layout (as lsa_gather_kv).
 *   chunk_ids    [sum k_b] int32 local chunk indices, or NULL: every chunk of every sequence in order
 *   K_res, V_res [sum k_b * C][n_kv_heads][Dh] kv_dtype, out ([sum N_b * C] rows if chunk_ids is NULL):
 *                row j*C+t of sequence b's block = code * scale (fp32) of token ids[j]*C+t, rounded to kv_dtype
 * Rows of tokens at or behind seq_len[b], and of ids outside 0..N_b-1 (LSA_ERR_BAD_ID), are left as they
 * were. */
LSA_API lsa_status lsa_kv8_gather(const lsa_dims *dims, const lsa_kv8_cache *cache, const int32_t *chunk_ids,
                                  const int32_t *seq_len, void *K_res, void *V_res, void *ws, size_t ws_bytes,
                                  void *stream);

/* Sparse decode attention over the 8-bit cache: softmax(q.K^T / sqrt(Dh)) V of one decode query per
 * sequence over the tokens of its kept chunks.
 *   q          [B][H][Dh] kv_dtype
 *   chunk_ids  [sum k_b] int32 local chunk indices, or NULL: every chunk (attention over the whole cache).
 *              An id outside 0..N_b-1 sets LSA_ERR_BAD_ID and is left out
 *   kept_count [B] int32 device or NULL: attend over the first kept_count[b] ids only (with chunk_ids NULL,
 *              over the first kept_count[b] chunks)
 *   out        [B][H][Dh] float32;  lse [B][H] float32 natural-log sum of exp of the scaled logits, or NULL
 * A sequence with no token to attend to gets out = 0 and lse = -inf; a head with a NaN or an infinity in its q
 * gets NaN. fp32 softmax and sums; the codes are multiplied exactly (as f16) with q and with the softmax
 * weights times V's scales, both held as the sum of two f16 numbers. That is 22 bits, for q down to 2^-17 of
 * its row's largest value, for a weight times its scale down to 2^-16 of the head's largest such product (an
 * error of 2^-38 of the largest below that). A weight below 2^-126 of the largest counts as 0. */
LSA_API lsa_status lsa_kv8_decode_attn(const lsa_dims *dims, const lsa_kv8_cache *cache, const void *q,
                                       const int32_t *chunk_ids, const int32_t *kept_count,
                                       const int32_t *seq_len, float *out, float *lse, void *ws, size_t ws_bytes,
                                       void *stream);

/* A token's whole step over the 8-bit cache: write the new token's K/V (lsa_kv8_append, one row per
 * sequence at position seq_len[b]), prepare its queries (also at position seq_len[b]), score the chunks, keep
 * the top k, and attend over the kept chunks' tokens below seq_len[b] + 1. seq_len itself is not changed: the
 * caller adds one after the step.
 *   prep           NULL: q and k are taken as they are
 *   chunk_emb      the caller's, of every chunk that holds a token, the one being filled among them: a chunk is
 *                  kept by its score alone, also the one that the new token was written to
 *   q, k, v        [B] rows of [H][Dh] (q) and [n_kv_heads][Dh] (k, v) kv_dtype, *_stride elements apart.
 *                  k and v both NULL: nothing is written, and the attention reads tokens below seq_len[b]
 *   seq_len        [B] int32 device, tokens cached before the step; may be NULL only if k and v are NULL
 *                  and prep is NULL (every chunk is then full)
 * Chunks that hold no token yet (behind seq_len[b] and the new token) are not compared: their embeddings may be
 * anything, and they are named, lowest index first, only where fewer than k_b chunks hold tokens.
 * Other arguments as lsa_decode_step; without prep, q_stride must be H * Dh. */
LSA_API lsa_status lsa_decode_step_kv8(const lsa_dims *dims, const lsa_kv8_cache *cache, const lsa_qk_prep *prep,
                                       const void *q_emb, const void *chunk_emb, const void *q, int64_t q_stride,
                                       const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                       const int32_t *seq_len, int32_t *chunk_ids_out, float *out, float *lse,
                                       void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LSA_KV8_H_ */
