/*
 * mlaqp_kv4.h -- C ABI of the paged 4-bit latent cache and the MLA decode
 * attention over it: what lies between the query projection of mlaqp.h
 * (whose [M,H,576] output is `q` here) and its V up-projection (which takes
 * `x`).
 *
 * One cached token of one layer is 400 bytes:
 *   - 512 latents as E2M1 codes (OCP MX: 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a
 *     sign) and one E8M0 byte s per 32 consecutive latents, value =
 *     code * 2^(s-127); s is 87..167, or 255 for a block that held a NaN or
 *     an infinity (all 32 values then read as NaN).  Other bytes are read as
 *     the nearer of 87 and 167;
 *   - 64 rope elements in BF16.
 *
 * A page holds page_size = P in {16, 32, 64, 128} tokens of one layer in
 * 400*P bytes: codes [P][256], rope [P][128], scales [P][16].  The order
 * inside the rows is what the attention kernel wants to find in shared
 * memory:
 *   codes   16 bytes per block of 32 latents, four 32-bit words of 8.  In a
 *           word the magnitude of element e is at bits 4e..4e+2, its sign at
 *           bit 8e+7 (e < 4) or 8(e-4)+3 (e >= 4).  Blocks j with j & 4 hold
 *           their two 8-byte halves in swapped order;
 *   rope    16-byte chunk c of the token at position t of the page is at
 *           chunk c ^ (t & 7).
 * A cache of one layer is num_pages pages, page p at cache + p*page_stride
 * bytes (page_stride >= 400*P, a multiple of 16; cache 16-byte aligned).
 * A slot is page*P + position.
 *
 * Sequences live in rows of a block table: int32 block_table[num_seqs] with
 * block_table_stride entries per row, entry j of row s the page of tokens
 * [j*P, (j+1)*P) of sequence s (-1: none), and int32 seq_lens[num_seqs].
 * int32 ref_count[num_pages] counts the rows that hold a page; a page with
 * count 0 is free.  All of it is device memory, all of it read and written
 * by the kernels in stream order, nothing of it by the host.
 *
 * Every call launches on `stream`, allocates nothing, never synchronises and
 * can be captured into a CUDA graph.  All launches use programmatic
 * dependent launch and touch no memory before the previous kernel on the
 * stream has finished, so they may follow any kernel.  Status codes and
 * mlaqp_last_error() as in mlaqp.h.  What only the device can see is recorded
 * in the word of mlaqp_device_status():
 *   MLAQP_DEVSTATUS_BAD_INDEX     a page, slot or sequence index out of range,
 *                                 a length beyond its table row or the pool's
 *                                 num_pages*page_size tokens, a child that is
 *                                 not empty: that item was left out
 *   MLAQP_DEVSTATUS_OUT_OF_PAGES  a fork or extension found no free page: that
 *                                 sequence was left as it was
 *   MLAQP_DEVSTATUS_WAIT_TIMEOUT  (as in mlaqp.h) the attention kernel waited
 *                                 a second for one of its own copies or
 *                                 products and gave up: that call's x and lse
 *                                 mean nothing
 */
#ifndef MLAQP_KV4_H_
#define MLAQP_KV4_H_

#include <stdint.h>

#include "mlaqp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLAQP_DEVSTATUS_BAD_INDEX 2u
#define MLAQP_DEVSTATUS_OUT_OF_PAGES 4u

#define MLAQP_KV4_TOKEN_BYTES 400
#define MLAQP_KV4_MAX_HEADS 16
#define MLAQP_KV4_MAX_Q_LEN 16
#define MLAQP_KV4_MAX_PAGES (1 << 20)

/* Bytes of one page (400*page_size), or 0 for an unsupported page_size. */
int64_t mlaqp_kv4_page_bytes(int page_size);

/*
 * Write T tokens into a layer's cache.  latent: BF16, token t at
 * latent + t*latent_token_stride, 512 elements; k_pe: BF16, 64 elements,
 * likewise (strides in elements, >= 0, multiples of 8; both 16-byte
 * aligned), so the two halves of a [T,576] projection can be passed as
 * views.  slots: int32[T]; a negative slot leaves its token out, a slot >=
 * num_pages*page_size is left out and reported.  Slots must be distinct.
 * The scale byte of a block is the smallest s (within 87..167) with
 * amax <= 7 * 2^(s-127): 7 is half way from the top code 6 to the next step,
 * so no element is off by more than half a step; codes round to nearest
 * even.  T = 0 launches nothing.
 */
int mlaqp_kv4_append(const void* latent, int64_t latent_token_stride, const void* k_pe,
                     int64_t k_pe_token_stride, void* cache, int64_t page_stride, int num_pages,
                     int page_size, const int32_t* slots, int T, mlaqp_stream_t stream);

/*
 * Read T cached tokens back as BF16: out + t*out_token_stride receives the
 * 512 latents (exact in BF16) and the 64 rope elements of slots[t]; a
 * negative slot gives a row of zeros, one out of range a row of zeros and a
 * report.  out_token_stride >= 576, a multiple of 8; out 16-byte aligned.
 */
int mlaqp_kv4_gather(const void* cache, int64_t page_stride, int num_pages, int page_size,
                     const int32_t* slots, int T, void* out, int64_t out_token_stride,
                     mlaqp_stream_t stream);

/*
 * MLA decode attention.  For sequence b < B (row s = seqs[b] of the table,
 * s = b when seqs is NULL), its query tokens i < q_len (q row m = b*q_len+i)
 * and heads h < H, with n = seq_lens[s] - (q_len-1-i) visible tokens:
 *
 *   S[t]       = softmax_scale * ( sum_{c<512} q[m,h,c] * latent[t,c]
 *                                + sum_{j<64}  q[m,h,512+j] * rope[t,j] )   t < n
 *   x[m,h,:]   = sum_t softmax(S)[t] * latent[t,:]          BF16
 *   lse[m,h]   = log(sum_t exp(S[t]))                       FP32, lse may be NULL
 *
 * so the last query token sees the whole sequence and the ones before it one
 * token less each (the cache already holds the query tokens' own entries).
 * A row that sees nothing (n <= 0, or all of its tokens left out, see below)
 * gets x = 0 and lse = -infinity.  Scores
 * are summed, and softmax, sums and lse held, in FP32, from operands of fewer
 * bits:
 *   - latents exactly where the block's scale byte is at most 14 below the
 *     largest of its token, in steps of 2^-15 of that largest scale where it is
 *     further below (mlaqp_kv4_gather reads those exactly);
 *   - BF16 queries exactly down to 2^-13 of the row's largest magnitude among
 *     its 512 (or 2^-40 of the largest among its last 64, if that is more), in
 *     steps of 2^-20 of it below; E4M3 queries and rope parts exactly;
 *   - probabilities p_t, where they weigh latents, with 11 bits while p_t times
 *     the token's largest scale is at least 2^-18 of what that product comes to
 *     in any of the row's tokens, in steps of 2^-28 of that below.  lse is of
 *     the probabilities in FP32.
 * A NaN anywhere in a row's visible tokens, or a NaN or an infinity in its q,
 * makes that row NaN; what lies beyond the visible tokens is never used.
 *   q          BF16 (MLAQP_OUT_BF16) or E4M3 (MLAQP_OUT_E4M3, value =
 *              code * *q_scale, q_scale one FP32 in device memory, NULL for
 *              BF16): element (m,h,j) at q[m*q_token_stride + h*576 + j];
 *              16-byte aligned, q_token_stride >= 576*H and a multiple of 16
 *              bytes -- the layout mlaqp_run writes
 *   x          element (m,h,c) at x[m*x_token_stride + h*512 + c], x_token_stride
 *              >= 512*H, a multiple of 8; 16-byte aligned -- what
 *              mlaqp_v_up_run(x, x_token_stride, 512, ...) reads
 *   workspace  16-byte aligned device memory of mlaqp_kv4_attend_workspace()
 *              bytes for this call alone while it runs; its contents mean
 *              nothing before and after
 * 1 <= H <= 16, 1 <= q_len <= 16, B*q_len <= 256, softmax_scale finite and
 * > 0.  B = 0 launches nothing.  A page index outside 0..num_pages-1 within
 * a sequence's length is reported and its tokens are left out.  Results do
 * not depend on what else runs: the work is split by the lengths alone and
 * joined in a fixed order.
 */
int mlaqp_kv4_attend(const void* q, int64_t q_token_stride, int q_dtype, const float* q_scale,
                     const void* cache, int64_t page_stride, int num_pages, int page_size,
                     const int32_t* block_table, int64_t block_table_stride, int num_seqs,
                     const int32_t* seq_lens, const int32_t* seqs, int B, int q_len, int H,
                     float softmax_scale, void* x, int64_t x_token_stride, float* lse,
                     void* workspace, int64_t workspace_bytes, mlaqp_stream_t stream);

/* Workspace bytes of mlaqp_kv4_attend for these sizes on `device` (< 0:
 * current), or -1 with a message. */
int64_t mlaqp_kv4_attend_workspace(int B, int q_len, int H, int device);

/*
 * Test hook for the attention kernel's bounded waits: as mlaqp_kv4_attend,
 * with their limit set to wait_limit_ns (1..10^9) and, for held > 0, one of the
 * hand-overs between the kernel's warps never taking place: 1 copies landed,
 * 2 copy units free, 3 scales, 4 rope rows landed, 5 rope rows free, 6 codes
 * converted, 7 their tiles free, 8 scores, 9 scores read, 10 probabilities,
 * 11 output products, 12 queries, 13 output read (2, 5, 7, 9 and 13 matter to
 * CTAs with more than one tile or row group).  The kernel records
 * MLAQP_DEVSTATUS_WAIT_TIMEOUT, waits for its own copies and products and
 * returns; x, lse and the workspace hold nothing of use.  Not for production.
 */
#define MLAQP_KV4_ATTEND_STAGES 13
int mlaqp_debug_kv4_attend_bounded_wait(const void* q, int64_t q_token_stride, int q_dtype, const float* q_scale,
                                        const void* cache, int64_t page_stride, int num_pages, int page_size,
                                        const int32_t* block_table, int64_t block_table_stride, int num_seqs,
                                        const int32_t* seq_lens, const int32_t* seqs, int B, int q_len, int H,
                                        float softmax_scale, void* x, int64_t x_token_stride, float* lse,
                                        void* workspace, int64_t workspace_bytes, unsigned int wait_limit_ns, int held,
                                        mlaqp_stream_t stream);

/*
 * Page operations.  They work on the table rows named by a list of n
 * sequences (device int32, distinct) and, where pages are copied, on all
 * `layers` layers of the cache: page p of layer l is at
 * cache + l*layer_stride + p*page_stride.  Free pages are taken lowest index
 * first, in list order, so the outcome is determined by the inputs.
 * num_pages <= 2^20.  n = 0 launches nothing (but for compact).
 */

/*
 * Grow sequences by new_tokens[i] (>= 0) tokens: take the pages this needs
 * and write the new tokens' slots to slots[i*max_new + k], k <
 * new_tokens[i] (-1 behind them).  new_tokens[i] > max_new, a row too short,
 * or new tokens that would begin in a page out of range, is reported and
 * leaves the sequence as it was (its slots: -1).  Item i takes the
 * free pages behind those that the items before it ask for, so where pages
 * run out the items that still fit are the first ones.
 */
int mlaqp_kv4_extend(int32_t* block_table, int64_t block_table_stride, int num_seqs,
                     int32_t* seq_lens, int32_t* ref_count, int num_pages, int page_size,
                     const int32_t* seqs, const int32_t* new_tokens, int n, int32_t* slots,
                     int max_new, mlaqp_stream_t stream);

/*
 * Fork: children[i] (an empty sequence) becomes a copy of parents[i].  Full
 * pages are shared (their counts rise); of a partly filled last page the
 * tokens are copied into a new page in every layer, so parent and child can
 * both grow.  A parent may occur several times.  Lengths count as they were
 * before the call, so a child is an empty parent to the other items.  An item
 * whose parent holds a page out of range is left out: its child stays empty and
 * it takes no free page.
 */
int mlaqp_kv4_fork(int32_t* block_table, int64_t block_table_stride, int num_seqs, int32_t* seq_lens,
                   int32_t* ref_count, int num_pages, int page_size, const int32_t* parents,
                   const int32_t* children, int n, void* cache, int64_t page_stride,
                   int64_t layer_stride, int layers, void* workspace, int64_t workspace_bytes,
                   mlaqp_stream_t stream);

/* Release: the sequences become empty, their pages' counts fall. */
int mlaqp_kv4_release(int32_t* block_table, int64_t block_table_stride, int num_seqs,
                      int32_t* seq_lens, int32_t* ref_count, int num_pages, int page_size,
                      const int32_t* seqs, int n, mlaqp_stream_t stream);

/*
 * Compact: with n pages live, the k-th free page below index n receives the
 * k-th live page at or above n, in every layer; tables and counts follow,
 * *n_live = n.  Afterwards pages n and above are free.  A table entry at or
 * above n whose page is out of range or counts 0 is reported and stays.
 */
int mlaqp_kv4_compact(int32_t* block_table, int64_t block_table_stride, int num_seqs,
                      int32_t* seq_lens, int32_t* ref_count, int num_pages, int page_size, void* cache,
                      int64_t page_stride, int64_t layer_stride, int layers, int32_t* n_live,
                      void* workspace, int64_t workspace_bytes, mlaqp_stream_t stream);

/*
 * Copy whole pages src[i] -> dst[i] in every layer (tables and counts are
 * the caller's).  No dst may occur twice or be a src.
 */
int mlaqp_kv4_copy_pages(void* cache, int64_t page_stride, int64_t layer_stride, int layers,
                         int num_pages, int page_size, const int32_t* src, const int32_t* dst, int n,
                         mlaqp_stream_t stream);

/* Workspace bytes of mlaqp_kv4_fork (lists of n) and mlaqp_kv4_compact for
 * num_pages pages; -1 for sizes outside the domain. */
int64_t mlaqp_kv4_pages_workspace(int num_pages, int n);

/* Loads every kernel of this header on `device` (< 0: current); call before
 * graph capture. */
int mlaqp_kv4_prewarm(int device);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* MLAQP_KV4_H_ */
