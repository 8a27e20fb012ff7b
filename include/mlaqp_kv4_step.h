/*
 * mlaqp_kv4_step.h -- C ABI of what a decode step over the paged 4-bit latent
 * cache (mlaqp_kv4.h) needs around its attention:
 *
 *   mlaqp_kv4_append_rope  normalises the latents, rotates the key parts and
 *                          the queries' parts by their positions and writes
 *                          the tokens into the cache
 *   mlaqp_kv4_digest       bounds of every channel over the tokens of a page
 *   mlaqp_kv4_select       the pages that each query token attends to, chosen
 *                          by those bounds: a block table and lengths for
 *                          mlaqp_kv4_attend
 *
 * With them a sparse decode step of a layer is
 *
 *   append_rope -> digest -> mlaqp_run (q) -> select -> mlaqp_kv4_attend
 *
 * on k pages a query token instead of all: 40 us for the last two instead of 149
 * for 64 sequences of 16K to 32K tokens at k = 32 pages of 64, and nothing gained
 * up to some 3K tokens a sequence.  Caches, slots, block tables and
 * the device status word are those of mlaqp_kv4.h, and so are the conventions:
 * every call launches on `stream` of the current device, allocates nothing,
 * never synchronises, can be captured into a CUDA graph, and touches no memory
 * before the previous kernel on the stream has finished.
 */
#ifndef MLAQP_KV4_STEP_H_
#define MLAQP_KV4_STEP_H_

#include <stdint.h>

#include "mlaqp.h"
#include "mlaqp_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MLAQP_ROPE_INTERLEAVED = 0,  /* pair j: elements 2j and 2j+1 */
  MLAQP_ROPE_HALVES = 1        /* pair j: elements j and j+32  */
} mlaqp_rope_style;

/*
 * Write T tokens into a layer's cache as mlaqp_kv4_append does, with what
 * comes before it, and rotate the same tokens' queries:
 *
 *   y[t,c]   = latent[t,c] * r_t * norm_weight[c],
 *              r_t = 1/sqrt(mean_c latent[t,c]^2 + norm_eps)
 *              (y = latent where norm_weight is NULL)
 *   cached latents = y as mlaqp_kv4_append quantises it, straight from FP32
 *   pair (a, b) of k_pe and of each head's q_pe -> (a*cos - b*sin, b*cos + a*sin),
 *              cos, sin those of pair j at positions[t], rounded once to BF16;
 *              elements stay where they are
 *
 * The sum of squares is the FP32 number next to the exact one (it is summed in two
 * floats), so r and y do not depend on an order of summation; the root, its
 * reciprocal and both products are rounded to FP32 each, in this order.  Where the
 * sum is beyond FP32 (2^128; magnitudes of some 2^59.5 in all latents, or of 2^64 in
 * one) r is 0; squares below FP32's normal range (magnitudes below 2^-63) lose bits,
 * which matters without norm_eps.
 *
 *   latent, k_pe, their strides, cache, slots  as mlaqp_kv4_append
 *   norm_weight  BF16[512], 16-byte aligned, or NULL (norm_eps is then not used);
 *                norm_eps finite and >= 0
 *   q_pe         BF16, element (t,h,j) at q_pe[t*q_token_stride + h*q_head_stride + j],
 *                strides >= 0 and multiples of 8 elements, 16-byte aligned; NULL
 *                with H = 0: no queries
 *   q_pe_out     the rotated queries, likewise; q_out_head_stride >= 64 where
 *                H > 1, q_out_token_stride >= (H-1)*q_out_head_stride + 64 where T > 1.
 *                May be q_pe with the same strides; otherwise what is written may
 *                not overlap what is read (rows of the same token stride may lie
 *                side by side, as views into one projection output do)
 *   H            0..128 (the heads of a whole model's prompt)
 *   positions    int32[T]; a token at a negative position is left out (nothing
 *                of it is written), one at num_positions or above is left out
 *                and reported
 *   cos_sin      FP32 [num_positions][64], 16-byte aligned: the 32 pairs'
 *                cosines, then their sines
 *   rope_style   mlaqp_rope_style
 * A negative slot, or one out of range (reported), leaves out the cached token
 * alone; its queries are rotated.  T = 0 launches nothing.
 */
int mlaqp_kv4_append_rope(const void* latent, int64_t latent_token_stride, const void* norm_weight, float norm_eps,
                          const void* k_pe, int64_t k_pe_token_stride, const void* q_pe, int64_t q_token_stride,
                          int64_t q_head_stride, void* q_pe_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                          int H, const int32_t* positions, const float* cos_sin, int num_positions, int rope_style,
                          void* cache, int64_t page_stride, int num_pages, int page_size, const int32_t* slots, int T,
                          mlaqp_stream_t stream);

/*
 * A page's digest is 1168 bytes at digests + page*digest_stride bytes
 * (digest_stride >= 1168, a multiple of 16; digests 16-byte aligned), int8 but
 * for the exponents:
 *   0     largest[512]   latents        1024  largest[64]   rope elements
 *   512   smallest[512]  latents        1088  smallest[64]  rope elements
 *   1152  exponent bytes of the latents and of the rope part, 14 zeros
 * largest[c] = ceil(max_t v[t,c] / 2^e) and smallest[c] = floor(min_t v[t,c] / 2^e)
 * over the page's tokens, v what mlaqp_kv4_gather reads, e the smallest
 * exponent >= -60 with all |v| of the part <= 127 * 2^e, byte e + 127.  A part
 * with a NaN, an infinity or an e above 60 has byte 255 and zeros.
 */
#define MLAQP_KV4_DIGEST_BYTES 1168

/*
 * Digests of the pages of one layer that have filled up: for i < n, those of
 * sequence s = seqs[i] whose last token is among its last new_tokens[i] ones
 * (0 <= new_tokens[i] <= max_new; more than the sequence has: all of them).  The
 * call looks up n * min(ceil(max_new/page_size), block_table_stride, num_pages)
 * table entries, whatever new_tokens says (half a million of them take 4 us).
 * Call it behind mlaqp_kv4_append with the lists given to mlaqp_kv4_extend,
 * and for every token a page's contents were written anew otherwise (a page
 * copied or moved by mlaqp_kv4_compact or mlaqp_kv4_copy_pages; the pages that
 * mlaqp_kv4_fork shares keep theirs).  Pages that are not full need none.
 * Several sequences may share a page.  From the first to the last of num_pages the
 * digests may overlap neither the cache nor another input.  A sequence index or
 * length out of range, or new_tokens[i] outside 0..max_new, is reported and the item
 * left out; a page out of range is reported and left out.  n = 0 launches nothing.
 */
int mlaqp_kv4_digest(const void* cache, int64_t page_stride, int num_pages, int page_size, const int32_t* block_table,
                     int64_t block_table_stride, int num_seqs, const int32_t* seq_lens, const int32_t* seqs,
                     const int32_t* new_tokens, int n, int max_new, void* digests, int64_t digest_stride,
                     mlaqp_stream_t stream);

/*
 * Choose the pages of query tokens.  For sequence b < B (row s = seqs[b], s = b
 * where seqs is NULL) and its query token i < q_len (row m = b*q_len+i), n =
 * seq_lens[s] - (q_len-1-i) tokens are visible, in N = ceil(n/page_size) pages.
 * Where N <= k all are taken, else k: the first `first`, the last `last`, and
 * of those between the ones of the highest scores, of equal scores the ones
 * that come first.  In the order of the sequence:
 *
 *   sel_table[m*sel_stride + r]  the r-th page taken, -1 behind them, r < k
 *   sel_lens[m]                  visible tokens in them, 0 where n <= 0
 *
 * which mlaqp_kv4_attend takes as block table and lengths of B*q_len sequences
 * with q_len = 1 (num_seqs = B*q_len, seqs = NULL).
 *
 * The score of a page bounds from above, up to the rounding of q, the sum over
 * the heads of q . latent + q . rope of any of its tokens:
 *
 *   qi[h,c] = q[m,h,c] / 2^f rounded to the nearest integer, ties to even, f the
 *             smallest exponent >= -100 with all |q[m]| <= 2047 * 2^f (all 0
 *             where q[m] holds a NaN or an infinity)
 *   up[c] = sum_h max(qi[h,c], 0)     down[c] = sum_h min(qi[h,c], 0)
 *   A = sum over the latents of up[c]*largest[c] + down[c]*smallest[c],
 *   B' = the same over the rope elements, both exact
 *   score = fl(A) * 2^e_latent + fl(B') * 2^e_rope, in FP32, rounded to nearest
 *             (+infinity where an exponent byte is 255, or where what lies there is
 *             no digest and the sum no number)
 *
 * so the choice depends on no order of summation.  One power of two holds for all
 * heads of a query token: a head much smaller than the largest counts in coarse
 * steps.  And one choice holds for all of them: it follows the pages that the heads
 * want together.  Where each wants another page, the spread of the bounds, which
 * grows with H, hides them: of 400 pages of 64 tokens, 32 taken, 16 heads whose
 * queries lean towards one page together keep all of their attention weight, 16
 * heads with a page of their own each keep 47% on average, some of them none (8
 * heads 87%; the best 32 pages hold all of it).  Only digests of full pages
 * that lie between the first and the last ones taken are read; a page out of
 * range there is reported and scores least.
 *
 *   q, q_token_stride, q_dtype  as mlaqp_kv4_attend (a common scale does not
 *                               matter here: there is no q_scale)
 *   workspace                   16-byte aligned device memory of
 *                               mlaqp_kv4_select_workspace() bytes for this call
 *                               alone while it runs
 * sel_table, sel_lens and workspace may overlap neither one another nor an input (of
 * a table's row: its first min(block_table_stride, num_pages) entries).
 * 1 <= H <= 16, 1 <= q_len <= 16, B*q_len <= 256; 1 <= k <= 2^20, first >= 0,
 * last >= 1, first + last <= k <= sel_stride.  A sequence index or a length out of
 * range is reported and its rows are empty.  B = 0 launches nothing.
 */
int mlaqp_kv4_select(const void* q, int64_t q_token_stride, int q_dtype, const void* digests, int64_t digest_stride,
                     int num_pages, int page_size, const int32_t* block_table, int64_t block_table_stride, int num_seqs,
                     const int32_t* seq_lens, const int32_t* seqs, int B, int q_len, int H, int k, int first, int last,
                     int32_t* sel_table, int64_t sel_stride, int32_t* sel_lens, void* workspace,
                     int64_t workspace_bytes, mlaqp_stream_t stream);

/* Workspace bytes of mlaqp_kv4_select, or -1 for sizes outside the domain. */
int64_t mlaqp_kv4_select_workspace(int B, int q_len, int64_t block_table_stride, int num_pages);

/* Loads every kernel of this header on `device` (< 0: current); call before
 * graph capture. */
int mlaqp_kv4_step_prewarm(int device);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* MLAQP_KV4_STEP_H_ */
