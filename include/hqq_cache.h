/*
 * hqq_cache.h -- C ABI of libhqq_cache.so: a key-value cache held in the
 * library's quantized format, and the attention of one new token a sequence
 * straight from its codes, on MI355X (gfx950).  It stands beside hqq_quantize,
 * hqq_dequantize_ex and hqq_linear (hqq.h), whose formats, conventions and
 * status codes it shares.
 *
 * The cache.  Keys and values are rows of `dim` values, one per token and
 * key-value head.  A page holds page_size consecutive tokens of one sequence
 * for all heads; either side (k, v) is one axis = 1 quantized matrix of hqq.h
 * with pages * heads * page_size rows and dim columns:
 *   packed  uint32 [pages, heads, page_size, dim * nbits / 32]
 *   scale, zero  fp32 [pages, heads, page_size, dim / group_size]
 * Slot s is token place s % page_size of page s / page_size.  A row's values
 * are (code - zero) / scale.
 *   nbits      2, 4 or 8 (HQQ_EINVAL_NBITS)
 *   dim        64, 96, 128, 192 or 256 (HQQ_EINVAL_SHAPE)
 *   group_size 32, 64, 128 or 256, dividing dim into at most 4 groups
 *              (HQQ_EINVAL_GROUP)
 *   page_size  a power of two, 16 to 1024; pages 1 to 2^31 - 1; heads 1 to 1024;
 *              pages * heads * page_size at most 2^40 (HQQ_EINVAL_SHAPE)
 *
 * Conventions of hqq.h hold: device pointers, 16-byte aligned unless said
 * otherwise; all arguments are checked on the host before anything is enqueued;
 * calls only enqueue work on `stream` of the current device; nothing is
 * allocated and no state is kept.  Outputs and the workspace must not overlap
 * inputs, the cache's arrays or one another (HQQ_EINVAL_PTR).  A call of no
 * tokens (no sequences) does nothing and needs no pointers but the cache's.
 *
 * Strides.  Keys, values and queries are rows of dim 16-bit values: row (t, h)
 * starts at t * token_stride + h * head_stride values, strides >= 0 and
 * multiples of 8 (HQQ_EINVAL_SHAPE), so that they can be a part of a wider
 * projection's output.  Other inputs and all outputs are contiguous.
 */
#ifndef HQQ_CACHE_H
#define HQQ_CACHE_H

#include "hqq.h"

#ifdef __cplusplus
extern "C" {
#endif

#ifndef HQQ_EWORKSPACE
#define HQQ_EWORKSPACE (-11) /* workspace smaller than the *_workspace function says */
#endif

/* One side of a cache: its arrays. */
typedef struct hqq_cache_side {
    uint32_t *packed;
    float *scale;
    float *zero;
} hqq_cache_side;

/* A cache: its arrays and their layout. */
typedef struct hqq_cache {
    hqq_cache_side k, v;
    int64_t pages;
    int32_t page_size, heads, dim, nbits, group_size;
} hqq_cache;

/* Quantize `tokens` tokens into the cache at their slots: each group with the
 * scale, zero and codes that hqq_quantize gives it at iters = 0,
 *   scale = qmax / (max - min), zero = -(min * scale)  (1, -min where max = min)
 *   code  = clamp(round_half_even(x * scale + zero), 0, qmax)
 *   K, V   rows [tokens, heads] of dtype (fp16 or bf16), read
 *   slots  int64 [tokens] (8-byte aligned).  A token whose slot lies outside
 *          [0, pages * page_size) is skipped.  The others' slots must differ:
 *          of two tokens with one slot, parts of either may stay.
 *   K_hat, V_hat  both NULL, or [tokens, heads, dim] of dtype: the values that
 *          the cache now stands for, as hqq_cache_read gives them
 * Other slots are left as they are.  Values are finite, as for hqq_quantize;
 * the difference of a group's largest and smallest is finite in fp32 and either
 * 0 or at least 2^-118 (fp16 values always are).
 * Limit of write and read (HQQ_EINVAL_SHAPE): tokens * heads at most 2^26. */
HQQ_API int hqq_cache_write(const hqq_cache *cache, const uint16_t *K, int64_t k_token_stride,
                            int64_t k_head_stride, const uint16_t *V, int64_t v_token_stride,
                            int64_t v_head_stride, int64_t tokens, const int64_t *slots, int dtype,
                            uint16_t *K_hat, uint16_t *V_hat, void *stream);

/* Read tokens back: K and V [tokens, heads, dim] of dtype receive the values
 * (code - zero) / scale at the slots (fp32, rounded once: what
 * hqq_dequantize_ex gives the rows).  A slot may be named more than once.  A
 * token whose slot lies outside [0, pages * page_size) gets zeros. */
HQQ_API int hqq_cache_read(const hqq_cache *cache, const int64_t *slots, int64_t tokens, int dtype, uint16_t *K,
                           uint16_t *V, void *stream);

/* Attention of one new token for each of `batch` sequences.  With the
 * sequence's keys k_t and values v_t (not rounded to 16 bits),
 *   s_t = softmax_scale * q . k_t,  lse = log sum_t exp(s_t),
 *   out = sum_t exp(s_t - lse) v_t
 * over its tokens t < length, of which only the last `window` count where
 * window > 0.  q_heads is a multiple of the cache's heads; q heads i * G to
 * i * G + G - 1, G = q_heads / heads, read key-value head i.
 *   Q        rows [batch, q_heads] of dtype
 *   table    int32 [batch, table_width] (4-byte aligned): page table[b][i] holds
 *            the tokens i * page_size and up of sequence b.  A page outside
 *            [0, pages) holds none: its tokens do not count.  Entries past a
 *            sequence's length (or before its window) are not used.
 *   lengths  int32 [batch] (4-byte aligned), the new token's own keys and values
 *            included; below 0 counts as 0, above table_width * page_size as that
 *   out      [batch, q_heads, dim] of dtype;  lse fp32 [batch, q_heads] (4-byte
 *            aligned), or NULL.  A sequence in which no token counts gives 0 and
 *            -infinity.
 * Scores, exponentials' sums and outputs are formed in fp32; besides the
 * output, each weight exp(s_t - max) times its group's 1 / scale is rounded for
 * the second product: to 22 bits, or by at most 2^-39 of the largest 1 / scale
 * that the group has among the sequence's tokens, whatever their weights (22
 * bits down to 2^-17 of it, then fewer), or 2^-145 where that is more.
 * Keys, values and queries are taken to be of magnitude 2^64 at most,
 * softmax_scale times the largest of a query 2^100 and a score, summed by
 * magnitudes, 2^120 (with fp16 values and a scale below 2^80 they are; with bf16
 * ones they need not be): beyond, a finite result can come out infinite or NaN.
 * softmax_scale is > 0 and at most 2^100, window >= 0 (HQQ_EINVAL_PARAM); batch
 * at most 2^15, q_heads 2^16, batch * q_heads 2^28, table_width at least 1 (also
 * where there are no sequences), table_width * page_size at most 2^30 and batch
 * times that 2^37 (HQQ_EINVAL_SHAPE).
 * The result does not depend on what else runs: sums are added in an order
 * that sizes and lengths set.
 *
 * The workspace holds the parts of sequences that are split over their length,
 * and how many sequences are shared out; nothing in it has to be set before a
 * call or kept after it.  Calls that may run at the same time (two streams, two
 * captured graphs) need one each. */
HQQ_API int64_t hqq_cache_attention_workspace(const hqq_cache *cache, int64_t batch, int64_t q_heads,
                                              int64_t table_width);
HQQ_API int hqq_cache_attention(const hqq_cache *cache, const uint16_t *Q, int64_t q_batch_stride,
                                int64_t q_head_stride, int64_t batch, int64_t q_heads, const int32_t *table,
                                int64_t table_width, const int32_t *lengths, float softmax_scale,
                                int64_t window, int dtype, uint16_t *out, float *lse, void *workspace,
                                int64_t workspace_bytes, void *stream);

/* Static description of a status code of this header or of hqq.h. */
HQQ_API const char *hqq_cache_strerror(int status);

#ifdef __cplusplus
}
#endif
#endif /* HQQ_CACHE_H */
