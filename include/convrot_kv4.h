/*
 * convrot_kv4.h -- C ABI of the rotated INT4 cache of keys and values and the
 * attention that reads it (library libconvrot_kv4.so).
 *
 * The cache.  A row is one token's key (or value) of one head, D = 64, 128 or
 * 256 values.  It is rotated by R = I (x) H_group (convrot.h; group = 64, or
 * 256 with D = 256) and quantised like a row of the W4A4 layer, with a bf16
 * scale:
 *      y = row R,  a = max|y|,  s = bf16_rne(a / 7)  (0 where below 2^-100),
 *      q = clamp(round_half_away(y * (1 / s)), -7, 7)   (fp32; s = 0: 0).
 * The scale is rounded before the codes are chosen.  A row that holds a NaN
 * or an infinity, or whose sums over a group are not finite (of values beyond
 * 2^119 they may not be), gets a scale that is not finite, and so do the
 * results that read it.  Rows live in pages of `page` tokens (16, 32, 64, 128
 * or 256):
 *      codes  uint8 [num_pages][kv_heads][page][D/2]  (low nibble = even
 *             channel, 4-bit two's complement),
 *      scales bf16  [num_pages][kv_heads][page],
 * once for keys and once for values.  A token's slot is
 * page id * page + its place in the page.  A request's block table row lists
 * the page ids of its tokens in order.
 *
 * Attention.  Because R is orthogonal, q . (k^ R^T) = (q R) . k^ and
 * sum p (v^ R^T) = (sum p v^) R^T: the queries and the outputs are rotated,
 * the cache never is.
 *
 * Conventions are those of convrot.h (device pointers on the current device,
 * 16-byte aligned, caller-owned buffers, arguments validated before any
 * launch, deterministic results), but whole-number arrays (slots, lengths,
 * tables, counts) begin anywhere that their type allows, so that parts of
 * longer arrays can be given; only the plan's `cached` and `result` begin on 16
 * bytes.  A buffer that a call writes overlaps no
 * other that it writes or reads (CONVROT_ERR_OVERLAP).  What lies in device
 * memory cannot be validated by the host: a slot or page id outside the cache,
 * where a call reads one, is skipped as if the token were not there, and
 * recorded as CONVROT_ERR_PAGE, which convrot_kv4_check_device_error reports.
 */
#ifndef CONVROT_KV4_H_
#define CONVROT_KV4_H_

#include "convrot.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CONVROT_KV4_MAX_REQUESTS 8192

/* A cache as every entry point takes it (host struct, device pointers). */
typedef struct {
    uint8_t *k_codes;
    void *k_scales;      /* bf16 */
    uint8_t *v_codes;
    void *v_scales;      /* bf16 */
    int64_t num_pages;   /* num_pages * page < 2^31 */
    int kv_heads;        /* 1 .. 1024 */
    int page;
    int head_dim;
    int group;
} convrot_kv4_cache;

/*
 * The bookkeeping of one step, on the GPU.  Request b holds cached[b] tokens
 * and brings new_tokens[b] more (0: none; negative: it is finished and gives
 * its pages back).  block_table int32 [B][max_pages] holds the page ids of the
 * cached tokens; the ids of the pages that the new tokens need are added to
 * it.  free_pages int32 [capacity] is a stack of *free_count page ids: first
 * the pages of finished requests are pushed (in the order of the requests and
 * of their tables), then the step's pages are popped (in the order of the
 * requests, the top first).  Outputs, none of them an input:
 *   seq_lens int32 [B]        cached + new (0: finished),
 *   cu_q int32 [B + 1]        prefix sums of the new tokens,
 *   slots int64 [max_tokens]  slot of each new token, requests in order,
 *   positions int32 [max_tokens]  its position in its request; both -1 behind
 *                             the last new token,
 *   result int32 [4]          {free pages left, pages taken, new tokens, status}.
 * result[3] = 0 when the step was laid out.  Otherwise nothing is, no page
 * changes hands, seq_lens = cached, cu_q = 0, slots and positions = -1,
 * result[0] = *free_count, and result[3] says why: 1 too few free pages;
 * 2 a request is longer than its block table row or 2^31 - 1; 3 more new
 * tokens than max_tokens; 4 a negative cached length, or a free list or table
 * whose numbers cannot be (free_count outside [0, capacity], more pages come
 * back than fit).  Running the call again on the same inputs gives the same
 * outputs: only entries that it does not read have changed.  References are not
 * counted: a page that several requests share must not be in the table row of a
 * request that finishes.  B is at most
 * CONVROT_KV4_MAX_REQUESTS, page as above.  One kernel.
 */
convrot_status convrot_kv4_plan(const int32_t *cached, const int32_t *new_tokens, int64_t B,
                                int page, int32_t *block_table, int64_t max_pages,
                                int32_t *free_pages, int64_t capacity, const int32_t *free_count,
                                int64_t max_tokens, int32_t *seq_lens, int32_t *cu_q,
                                int64_t *slots, int32_t *positions, int32_t *result,
                                convrot_stream_t stream);

/*
 * Quantise the keys and values of T tokens into the cache: k_bf16 and v_bf16
 * are [T][kv_heads][D] with ldk and ldv values between tokens (multiples of 8,
 * at least kv_heads * D: columns of a fused projection's rows can be given as
 * they are).  Tokens whose slot is negative are skipped.  The slots of a call
 * must differ.  One kernel.
 */
convrot_status convrot_kv4_append(const convrot_kv4_cache *cache, const void *k_bf16, int64_t ldk,
                                  const void *v_bf16, int64_t ldv, const int64_t *slots, int64_t T,
                                  convrot_stream_t stream);

/*
 * The rows of T slots as the attention sees them: k_bf16 and v_bf16
 * [T][kv_heads][D] = bf16_rne((q s) R^T).  Zeros where the slot is negative
 * (or outside the cache).  One kernel.
 */
convrot_status convrot_kv4_read(const convrot_kv4_cache *cache, const int64_t *slots, int64_t T,
                                void *k_bf16, void *v_bf16, convrot_stream_t stream);

/* Bytes of workspace convrot_kv4_attention needs (host-only; 0 for sizes that
 * it refuses): partial results of requests whose keys are split. */
size_t convrot_kv4_attention_workspace_size(int64_t T, int64_t B, int heads, int kv_heads,
                                            int head_dim, int64_t max_keys);

/*
 * out[t][h] = sum_j softmax_j(scale q[t][h] . k^_j) v^_j over the cache.
 * q_bf16 [T][heads][D] with ldq values between tokens; heads a multiple of
 * kv_heads, query head h reads head h / (heads / kv_heads).  Request b's
 * queries are the tokens cu_q[b] .. cu_q[b+1] - 1, the last ones of its
 * seq_lens[b] tokens, whose rows are in the cache: with n queries, query i
 * sees the positions j <= seq_lens[b] - n + i.  A query that sees nothing
 * gives zeros.  block_table int32 [B][max_pages]; entries behind a request's
 * last page are not read.  out_bf16 [T][heads][D]; rows from cu_q[B] on are
 * left as they were.  workspace: at least
 * convrot_kv4_attention_workspace_size(T, B, heads, kv_heads, D,
 * max_pages * page) bytes, 256-byte aligned (CONVROT_ERR_WORKSPACE); calls that
 * use one workspace must be ordered on the GPU; it needs no initialisation.
 * -2^100 <= scale <= 2^100.  Queries are held as 16-bit whole numbers, off by
 * at most 2^-16 of their row's largest rotated value; rows below 2^-100 count
 * as 0, rows with a NaN or an infinity give NaN, rows of values beyond 2^119
 * may.  The products of softmax weights and values' scales are rounded to f16
 * relative to the largest that the query has met among the keys it sees: off by
 * 2^-11 of each, or by 2^-30 of that largest where they are below 2^-19 of it.
 * Softmax weights below 2^-110 of the query's largest may count as 0, and scores
 * have to stay in fp32's range.  Lengths and queries beyond what block_table and
 * q_bf16 hold are cut.  Two kernels.
 */
convrot_status convrot_kv4_attention(const convrot_kv4_cache *cache, const void *q_bf16,
                                     int64_t ldq, int64_t T, int heads, const int32_t *block_table,
                                     int64_t max_pages, const int32_t *seq_lens,
                                     const int32_t *cu_q, int64_t B, float scale, void *workspace,
                                     size_t ws_bytes, void *out_bf16, convrot_stream_t stream);

/* Failure detection.  Synchronise `stream`, then return and clear this
 * library's device error word: CONVROT_OK, or CONVROT_ERR_PAGE after a slot or
 * page id outside the cache was met. */
convrot_status convrot_kv4_check_device_error(convrot_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_KV4_H_ */
