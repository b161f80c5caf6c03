/*
 * kda_cache.h -- paged 8-bit key/value cache and the attention that reads it (gfx950).
 *
 * Models that mix the recurrence of kda.h with layers of softmax attention serve
 * both kinds from the same batch: one token per sequence (kda_decode), a few draft
 * tokens (kda_verify_ucache_flush) or packed documents (kda_prefill_varlen). These
 * calls are the attention layers' side of such a step: kda_cache_write quantises the
 * new tokens' keys and values into the sequences' pages, kda_cache_attention
 * attends to all of them, kda_cache_read gives tokens back in bf16.
 *
 * Cache. A pool of num_pages pages of page_size tokens (16, 32, 64, 128 or 256) for
 * the keys and one for the values. Page p, head h, token slot s, channel c is the
 * byte at p * page_stride + (h * page_size + s) * 128 + c; k_scale and v_scale hold
 * one fp32 per page and head at p * H + h, and a byte stands for code * scale:
 *  - KDA_CACHE_FP8: OCP fp8 e4m3 ("e4m3fn", largest code 448),
 *  - KDA_CACHE_INT8: signed integers from -127 to 127.
 * The scales that kda_cache_write makes are powers of two, so that dividing by one
 * is exact, the values read back are exact in bf16, and an e4m3 value keeps its
 * relative step whatever the scale. (The largest bf16 values, from 3.3e38 on, round to
 * a code that stands for 2^128: it reads back as infinity.) kda_cache_read and
 * kda_cache_attention take any finite scale.
 *
 * Sequences. Sequence b has kv_lens[b] tokens, those of this call included; token
 * position i lies in slot i mod page_size of page page_table[b * table_row_stride +
 * i / page_size]. The call's tokens are the last ones: with n_b of them, positions
 * kv_lens[b] - n_b .. kv_lens[b] - 1. In the packed tensors they are rows
 * cu_seqlens[b] .. cu_seqlens[b + 1] - 1; cu_seqlens NULL: n_b = total_tokens / n_seqs
 * for every sequence (n_seqs must divide total_tokens). Rows behind the last
 * sequence are neither read nor written. The packed tensors are bf16, head h at
 * element h * 128 of a row.
 *
 * Device-visible bad values never fault. A sequence with kv_lens[b] < n_b or
 * > table_width * page_size is inactive: nothing is written to the cache, rows that
 * a call would have written are zeros (lse: -infinity). A page index outside [0,
 * num_pages) is a page that does not exist: its tokens are not written, read back
 * as zeros, and attention leaves them out. cu_seqlens is clamped to [0,
 * total_tokens]. Bytes and scales of slots and pages behind a sequence's end are
 * never looked at: they may hold anything, NaN codes among it.
 *
 * Other conventions are those of kda.h: device pointers unless the name ends in
 * _host, strides in elements, nothing allocated or synchronised, work enqueued on
 * `stream` only, host-visible errors returned before a launch. bf16 pointers and
 * strides need no alignment beyond 2 bytes; k_cache and v_cache are 16-byte aligned
 * and their page strides multiples of 16, else KDA_ERR_UNSUPPORTED.
 *
 * Errors common to the calls. KDA_ERR_BAD_SHAPE: negative sizes, H < 1,
 * num_pages < 0, table_width < 1, total_tokens no multiple of n_seqs without
 * cu_seqlens, tokens without sequences. KDA_ERR_UNSUPPORTED: D other than 128,
 * cache_dtype, page_size, H over 2^13, more than 2^30 tokens, table_width * page_size
 * over 2^28 or n_seqs times that over 2^35, or more than the 2^24 - 1 workgroups of a
 * launch (a page that gets or gives tokens, or 32 or 128 query rows of a key/value
 * head). KDA_ERR_BAD_STRIDE: a negative stride, a page stride below H * page_size *
 * 128, output rows or the pages' rows that overlap, a table_row_stride below
 * table_width. num_pages = 0 needs no cache pointers; total_tokens = 0 is a no-op that
 * needs no pointers. No output may overlap an input or another output.
 */
#ifndef KDA_CACHE_H_
#define KDA_CACHE_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  KDA_CACHE_FP8 = 0, /* cache_dtype: fp8 e4m3 codes */
  KDA_CACHE_INT8 = 1 /* cache_dtype: int8 codes */
};

/*
 * kda_cache_write -- quantise the call's keys and values into their pages.
 *
 *  k, v               bf16 [total_tokens, H * 128]
 *  k_cache, v_cache, k_scale, v_scale   updated in place
 * Per page, head and side, with amax the largest finite magnitude among the page's
 * new tokens and M = 448 (fp8) or 127 (int8):
 *   need  = 2^e, e the smallest integer >= -100 with amax <= M 2^e
 *   scale = need where the call writes slot 0 of the page, else max(need, old scale)
 *   code  = value / scale, rounded to nearest even; beyond +-M (infinities) +-M;
 *           NaN: the e4m3 NaN, or 0 in int8. (Behind an old scale that is no power of
 *           two and stays: value * (1 / scale), both in fp32.)
 * Where the scale grows, the codes of the sequence's earlier tokens in that page
 * become code * (old scale / scale), rounded the same way: with powers of two an
 * e4m3 value changes only where it falls below 2^-6 of the new scale. Other slots
 * keep their bytes. Tokens of one call are written at once: the result depends on
 * how a document was cut into calls only where a page's scale grew.
 * A page that receives tokens belongs to one sequence of the call; pages shared by
 * several (a common prefix) are whole, and only read.
 */
kda_status kda_cache_write(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t D,
                           const int32_t* cu_seqlens,
                           const void* k, int64_t k_row_stride,
                           const void* v, int64_t v_row_stride,
                           int32_t cache_dtype, int32_t page_size, int64_t num_pages,
                           void* k_cache, int64_t k_page_stride,
                           void* v_cache, int64_t v_page_stride,
                           float* k_scale, float* v_scale,
                           const int32_t* page_table, int32_t table_width,
                           int64_t table_row_stride, const int32_t* kv_lens,
                           hipStream_t stream);

/*
 * kda_cache_read -- the last n_b tokens of each sequence in bf16 (with cu_seqlens
 * and kv_lens of its first m tokens, any range of them).
 *
 *  k, v               bf16 [total_tokens, H * 128] out: code * scale in fp32, rounded to
 *                     bf16 (the product is exact where the scale is a power of two)
 */
kda_status kda_cache_read(int32_t n_seqs, int64_t total_tokens, int32_t H, int32_t D,
                          const int32_t* cu_seqlens,
                          void* k, int64_t k_row_stride, void* v, int64_t v_row_stride,
                          int32_t cache_dtype, int32_t page_size, int64_t num_pages,
                          const void* k_cache, int64_t k_page_stride,
                          const void* v_cache, int64_t v_page_stride,
                          const float* k_scale, const float* v_scale,
                          const int32_t* page_table, int32_t table_width,
                          int64_t table_row_stride, const int32_t* kv_lens,
                          hipStream_t stream);

/*
 * kda_cache_attention_workspace_size -- bytes that kda_cache_attention needs for these
 * sizes (0 for invalid ones). Pure host arithmetic.
 */
size_t kda_cache_attention_workspace_size(int32_t n_seqs, int64_t total_tokens, int32_t H_q,
                                          int32_t H_kv);

/*
 * kda_cache_attention -- causal softmax attention of the call's tokens over the cache.
 *
 *  H_q, H_kv          query heads and key/value heads; H_q is a multiple of H_kv, and
 *                     query head h reads key/value head h / (H_q / H_kv)
 *  cu_seqlens_host    HOST copy of cu_seqlens (the plan of the launch); both or neither
 *  q                  bf16 [total_tokens, H_q * 128]
 *  scale              multiplies q . k; finite, also times log2(e)
 *  out                bf16 [total_tokens, H_q * 128]
 *  lse                fp32 [total_tokens, H_q] with lse_row_stride, or NULL
 *  workspace          >= kda_cache_attention_workspace_size(...) bytes, 256-byte
 *                     aligned; written before it is read in every call, so calls
 *                     that do not overlap in time may share one
 * Token i of sequence b sees the keys at positions 0 .. kv_lens[b] - n_b + i:
 *   s_j = scale q . k_j,  lse = log sum_j exp(s_j),  out = sum_j exp(s_j - lse) v_j
 * with fp32 sums and maxima, and products of exact q and codes. The weights exp(s_j - ref)
 * are off by 2^-16 of themselves at most where a sequence has at most 128 query rows per
 * key/value head (n_b * H_q / H_kv); with more rows, multiplied by the values' scale, they are
 * rounded to fp16: by 2^-11 of themselves, or 2^-31 of the largest such product that a row has
 * seen. A token that sees no key has out = 0 and lse = -infinity. The cache has to hold
 * the call's own tokens (kda_cache_write).
 * Values may be of any size with code * scale below 2^128: no sum leaves fp32's range, and
 * out is infinite only where the definition's value rounds to infinity in bf16. Scores have
 * to stay inside fp32's range, as sums of |q| |code| and multiplied by scale * log2(e) and
 * the keys' scale. Beyond, and where a query is not finite, a row (a token's head) is NaN or
 * what infinite scores give; no other row is touched by it.
 * The result does not depend on other sequences' contents, and is the same in every
 * call with the same lengths.
 * KDA_ERR_BAD_SEQLENS: cu_seqlens_host does not run from 0 upwards to at most
 * total_tokens. KDA_ERR_WORKSPACE_TOO_SMALL; KDA_ERR_UNSUPPORTED for an unaligned
 * workspace, or more than 256 query heads for a key/value head.
 */
kda_status kda_cache_attention(int32_t n_seqs, int64_t total_tokens, int32_t H_q, int32_t H_kv,
                               int32_t D, const int32_t* cu_seqlens_host,
                               const int32_t* cu_seqlens,
                               const void* q, int64_t q_row_stride,
                               int32_t cache_dtype, int32_t page_size, int64_t num_pages,
                               const void* k_cache, int64_t k_page_stride,
                               const void* v_cache, int64_t v_page_stride,
                               const float* k_scale, const float* v_scale,
                               const int32_t* page_table, int32_t table_width,
                               int64_t table_row_stride, const int32_t* kv_lens, float scale,
                               void* out, int64_t out_row_stride,
                               float* lse, int64_t lse_row_stride,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_CACHE_H_ */
