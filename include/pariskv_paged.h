/* pariskv_paged.h -- a K/V cache in pages: written chunk by chunk as a prompt comes in, read by
 * the attention of each chunk of new tokens (or of single tokens while decoding), and read back
 * into the dense slabs that the rest of the library takes.
 *
 * "Technical Summary: ParisKV" starts from a prefilled KV cache (Normalization and Rotation:
 * calibration is "precomputed during the prefill phase"). These calls cover the way there: a
 * serving program writes each chunk of a prompt (pariskv_paged_write), attends it over all the
 * pages so far (pariskv_paged_attend), and hands the finished prompt to the retrieval path as
 * slabs [batch][num_kv_heads][ld_tok][d] (pariskv_paged_read), the layout of
 * pariskv_build_index, pariskv_append, pariskv_dense_attend, pariskv_sparse_attend and
 * pariskv_cache_prefill. Pages may hold 8 bits an element, which halves what the cache takes
 * and what an attention over it reads.
 *
 * Conventions as in pariskv.h: plain pointers, caller-owned buffers, asynchronous on `stream`,
 * argument errors reported synchronously with nothing enqueued. All device buffers of a call
 * must lie on the current device. Calls may be captured into CUDA graphs; lengths, tables and
 * starts are read from device memory when the work runs, so a captured call follows them. */
#ifndef PARISKV_PAGED_H_
#define PARISKV_PAGED_H_

#include "pariskv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a page holds.
 *   PARISKV_PAGES_BF16: bf16 rows.
 *   PARISKV_PAGES_E4M3: one byte an element (e4m3: 1 sign, 4 exponent and 3 mantissa bits, no
 *     infinities, at most 448) and one scale byte b per row of 128 elements. An element stands
 *     for code * 2^(b - 127). A row is stored with the least e in [-120, 119] for which its
 *     largest magnitude is <= 448 * 2^e (e = -120 for a row of zeros), b = e + 127, and
 *     code = x / 2^e rounded to nearest even, saturating at 448. The division is exact, so the
 *     codes are the same however they are computed, and code * 2^e is exact in bf16 and fp32.
 *     A row that holds an infinity or a NaN is stored with b = 255 and codes 0x7f; it reads back
 *     as NaN. Rows that the caller fills in keep to the same: b in [7, 246] and codes other than
 *     0x7f and 0xff, or b = 255 and codes 0x7f. */
enum { PARISKV_PAGES_BF16 = 0, PARISKV_PAGES_E4M3 = 1 };

/* A pool of pages (caller's device memory). Row r of KV head h in page p is the 128 elements
 * from k + p * page_stride + (h * page_size + r) * 128 on (elements of 2 or 1 bytes), its scale
 * byte k_scale[p * scale_stride + h * page_size + r]; v likewise. */
typedef struct {
    void* k;
    void* v;
    uint8_t* k_scale;      /* E4M3 only (NULL for BF16); 16-byte aligned */
    uint8_t* v_scale;
    int64_t num_pages;     /* 1 .. 2^31 - 1 */
    int64_t page_stride;   /* elements; >= num_kv_heads * page_size * 128, a multiple of 16 bytes */
    int64_t scale_stride;  /* bytes; >= num_kv_heads * page_size, a multiple of 16 (E4M3) */
    int32_t page_size;     /* tokens in a page: 16, 32, 64, 128 or 256 */
    int32_t format;        /* PARISKV_PAGES_BF16 or PARISKV_PAGES_E4M3 */
} pariskv_pages;

/* The new tokens of a batch of sequences and where each sequence's pages are (device memory).
 * Sequence s brings q_len = q_start[s + 1] - q_start[s] new tokens, rows q_start[s] ... of the
 * per-token arrays; it has kv_len[s] tokens once they are in the cache, so its new token j is
 * at position kv_len[s] - q_len + j. Position t lies in page page_table[s * table_stride +
 * t / page_size], row t % page_size. Lengths may differ and may be zero. A page id outside
 * [0, num_pages), or a position past table_width * page_size, stands for tokens that are not
 * there (given back, or never taken): they are not written, not read and not attended.
 * Positions below zero (kv_len < q_len) are not written and attend nothing. Rows at or past
 * q_start[batch] belong to no sequence; their outputs stay as they are. */
typedef struct {
    const int32_t* page_table;  /* [batch][table_stride] */
    const int32_t* kv_len;      /* [batch] */
    const int32_t* q_start;     /* [batch + 1], ascending, within [0, total_q] */
    int64_t total_q;            /* rows of the per-token arrays; 0 .. 2^31 - 1 */
    int32_t table_width;        /* entries of each sequence's table, >= 1 */
    int32_t table_stride;       /* >= table_width */
    int32_t max_q;              /* at least every q_len: a sequence's rows past max_q are left out.
                                 * It also chooses the attention's kernel, for the whole call (see
                                 * pariskv_paged_attend), so it should not be larger than need be. */
} pariskv_chunk;

/* Writes the new tokens' K and V rows into their pages.
 *   cfg:  batch, num_kv_heads and dtype (of k_new and v_new: F32 or BF16) are used.
 *   k_new, v_new: device pointers, element (row, h, j) at [row * ld + h * 128 + j] with token
 *     strides k_ld, v_ld (>= num_kv_heads * 128, whole 16-byte words); 16-byte aligned.
 * fp32 rows go into BF16 pages rounded to nearest even. No two tokens of a call may share a
 * slot: which of them it then holds, or parts of which, is not defined. One launch.
 * Errors: EINVAL, ECUDA. */
PARISKV_API pariskv_status pariskv_paged_write(const pariskv_config* cfg,
                                               const pariskv_pages* pages,
                                               const pariskv_chunk* chunk, const void* k_new,
                                               const void* v_new, int64_t k_ld, int64_t v_ld,
                                               void* stream);

/* Reads positions [first, first + n) of every sequence back into dense slabs of cfg->dtype
 * (F32 or BF16): position first + r of sequence s, KV head h, goes to
 * K[((s * num_kv_heads + h) * ld_tok + r) * 128 ...], V likewise. Rows whose tokens are not
 * there (at or past kv_len, or on a page that is not there) stay as they are.
 *   K, V: device or pinned host pointers, 16-byte aligned; either may be NULL (not read back).
 *   chunk: page_table and kv_len are used (q_start, total_q and max_q are not).
 * One launch. Errors: EINVAL, ECUDA. */
PARISKV_API pariskv_status pariskv_paged_read(const pariskv_config* cfg,
                                              const pariskv_pages* pages,
                                              const pariskv_chunk* chunk, int64_t first, int64_t n,
                                              void* K, void* V, int64_t ld_tok, void* stream);

/* Attention of the new tokens over the pages (their own rows among them: write first):
 *   out[row][head] = sum_t softmax_t(scale * <q[row][head], K[head / group][t]>) V[head / group][t]
 *   lse[row][head] = ln sum_t exp(scale * <q[row][head], K[head / group][t]>)
 * over the tokens t < kv_len that are there and, with causal != 0, t <= the row's own position.
 * A row that attends nothing gets out = 0 and lse = -infinity.
 *   cfg:   batch, num_kv_heads, group (1..128) and dtype (PARISKV_BF16 only) are used.
 *   q:     device pointer bf16, element (row, head, j) at [row * q_ld + head * 128 + j], token
 *          stride q_ld >= num_kv_heads * group * 128 and a multiple of 8; 16-byte aligned.
 *   out:   device pointer [total_q][num_kv_heads * group][128] of out_dtype, 16-byte aligned.
 *          PARISKV_BF16: the probabilities enter the second product with at least bf16's 8
 *          bits; PARISKV_F32: with 24 bits, so that the result is as exact as fp32 sums are (the
 *          tensor cores truncate theirs, which is bounded to some 2^-20 of sum_t p_t |V_t|, however
 *          many tokens there are). Over E4M3 pages with max_q * group <= 16 this holds for weights
 *          p_t * 2^(V's scale) down to 2^-24 (BF16) or 2^-30 (F32) of the row's largest; smaller ones
 *          are off by at most 2^-32 or 2^-54 of it.
 *   lse:   device pointer [total_q][num_kv_heads * group] fp32, or NULL.
 * Sums, maxima and accumulators are fp32; the accumulators are relative to maxima that may lag by
 * a factor of 2^8, so sums of V's magnitudes over the attended tokens past 2^119 can overflow to
 * infinity. A K or V row with an infinity or a NaN in it makes the
 * rows that attend it infinite or NaN (V: in the elements concerned) and no others; but a token
 * whose score is minus infinity weighs nothing. The same call on the same data gives the same bits.
 * Calls with max_q * group <= 16 stream K and V once for up to 16 rows a sequence and KV head; with
 * more rows, every sequence of the call goes by tiles of 128 or 256 rows. Each rounds its weights
 * differently, so a sequence's last bits can depend on what else is in the call, and one long chunk
 * among single tokens (or a max_q that is not reached) makes those slower: 32 of them over 32768
 * tokens 1.3 times over BF16 pages and 2.8 times over E4M3 ones. Two calls avoid that.
 * The workspace comes from the library's per-device memory pool, stream-ordered on `stream`. Two or
 * three launches.
 * Errors: EINVAL, ENOMEM, ECUDA; ETIMEOUT from pariskv_paged_sync. */
PARISKV_API pariskv_status pariskv_paged_attend(const pariskv_config* cfg,
                                                const pariskv_pages* pages,
                                                const pariskv_chunk* chunk, const void* q,
                                                int64_t q_ld, float scale, int32_t causal,
                                                void* out, int32_t out_dtype, float* lse,
                                                void* stream);

/* Waits for the work on `stream` and reports whether a device-side wait of a paged attention on
 * the current device has run out since the last report (PARISKV_ETIMEOUT: the outputs of that
 * call are not complete; never seen while the device works). The report is the device's, not the
 * stream's: of several threads that ask at once, one gets it. Not to be captured. */
PARISKV_API pariskv_status pariskv_paged_sync(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PARISKV_PAGED_H_ */
