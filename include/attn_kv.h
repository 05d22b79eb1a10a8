/*
 * attn_kv.h -- C ABI of the operators around paged attention: rotary
 * positions, page plans, cache appends, page sketches and attention over the
 * pages that a sketch selects.
 *
 * The conventions of attn.h hold here too: device pointers owned by the
 * caller and 16-byte aligned (index arrays: 4-byte aligned), asynchronous
 * calls on `stream`, nothing enqueued when an argument is refused, no memory
 * allocated, the device status word for lengths, slots and page ids that are
 * out of range on the device (ATTN_ERR_DEVICE_DATA: the kernels skip or clamp
 * them, touch nothing outside the buffers, and the call's results are
 * undefined).  Every call can be captured into a CUDA graph and replayed.
 * Outputs must not overlap inputs unless a call says that it works in place.
 *
 * A serving step over a paged cache strings them together:
 *   attn_paged_plan          lengths -> offsets, positions, slots, table rows
 *   attn_paged_append        q, k, v -> rotated q; K and V in their slots
 *   attn_page_sketch         the pages just written -> their 8-bit sketches
 *   attn_paged_fwd (attn.h)  or attn_paged_sparse_fwd: the attention itself
 */
#ifndef ATTN_GB300_ATTN_KV_H
#define ATTN_GB300_ATTN_KV_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How attn_rope_inv_freq stretches the rotation to longer contexts. */
typedef enum {
    ATTN_ROPE_PLAIN = 0,  /* f_i = base^(-2i / rot) */
    ATTN_ROPE_LINEAR = 1, /* f_i / factor: positions interpolated */
    ATTN_ROPE_NTK = 2,    /* base * factor^(rot / (rot - 2)): the slowest pair stretched by factor, the fastest kept */
    ATTN_ROPE_BANDS = 3,  /* by turns over orig_len, n_i = orig_len f_i / 2 pi: n_i >= high kept, n_i <= low divided by
                             factor, between them (1 - t) f_i / factor + t f_i, t = (n_i - low) / (high - low) */
    ATTN_ROPE_YARN = 4    /* the same two ends, blended along the pair index i: pairs up to floor(c(high)) kept, from
                             ceil(c(low)) on divided, linear between them, with c(n) = rot ln(orig_len / (2 pi n)) /
                             (2 ln base), both ends clamped to [0, rot - 1]; amplitude 0.1 ln(factor) + 1 */
} attn_rope_scaling_t;

/* Host function: the angle per position of each rotated pair, float64.
 *   inv_freq: HOST array of rot / 2 doubles (written); amplitude: HOST double
 *   or NULL (written: the factor on rotated vectors, 1 except for YARN).
 *   rot even, in [2, 1024]; base > 1; factor >= 1 (read by the four stretched
 *   kinds); orig_len >= 1 and 0 < low < high (read by BANDS and YARN;
 *   their published ends are 1 and 4 turns for BANDS, 1 and 32 for YARN).
 * Errors: ATTN_ERR_INVALID_ARG. */
attn_status_t attn_rope_inv_freq(double* inv_freq, double* amplitude, int rot, double base, int scaling,
                                 double factor, int orig_len, double low, double high);

/* Rotary positions.  Each pair (a, b) of the first `rot` dims of a head
 * vector at position P turns by the angle t = P f_i and is scaled:
 *   a' = amplitude (a cos t - b sin t),   b' = amplitude (a sin t + b cos t).
 * interleaved = 0: pair i is dims (i, i + rot / 2); 1: dims (2i, 2i + 1).
 * Dims rot .. d - 1 pass through.  inverse = 1 turns by -t with the same
 * amplitude: the transpose, which is the gradient of the forward call (dq and
 * dk in, the gradients of the unrotated q and k out).
 *   q, k: [B, H, N, d] and [B, H_k, N, d] through element strides, the head
 *   dim dense; k and k_out may both be NULL (H_k ignored).  q_out, k_out: the
 *   same shapes, own strides; either may be its input (same pointer and
 *   strides) for a rotation in place.
 *   elem_bytes: 2 (bf16) or 4 (fp32), for inputs and outputs alike.
 *   strides: HOST array of 12: (b, h, n) of q, q_out, k, k_out, in elements,
 *   multiples of 16 / elem_bytes; input strides may be 0 (broadcast), output
 *   strides of dims longer than 1 are at least d.
 *   positions: int32, position of token n of batch entry b at
 *   positions[b * pos_stride_b + n] (pos_stride_b 0: shared by the batch);
 *   any int32 value; NULL: position n.
 *   inv_freq: DEVICE array of rot / 2 float64 (freq_bits 64) or fp32 (32).
 *   d in {64, 128}; rot a multiple of 16 in [16, d]; B, H, N >= 1;
 *   B * N < 2^31, H and H_k at most 65535; amplitude finite.
 * P f_i / 2 pi is taken modulo 1 in 64-bit fixed point, good to |P| 2^-63 turns
 * (|f_i| < 2^63), and its cosine and sine are fp32, good to 2 ulp (or 2^-44) at any
 * position; the rotation is fp32 and rounds once to the output type.
 * Errors: ATTN_ERR_INVALID_ARG / ATTN_ERR_UNSUPPORTED before the launch;
 * ATTN_ERR_CUDA when it fails. */
attn_status_t attn_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* positions,
                        long long pos_stride_b, const void* inv_freq, int freq_bits, int elem_bytes, int B, int H,
                        int H_k, int N, int d, int rot, const long long* strides, int interleaved, int inverse,
                        float amplitude, void* stream);

/* Page plan of a step: from the requests' cached and new lengths, the
 * offsets, positions and cache slots of the new tokens, and the table entries
 * of the pages they start, taken from a stack of free pages.
 *   ctx_lens: int32 [B] keys already cached; new_lens: int32 [B] new tokens
 *   per request, or NULL for one each.
 *   block_table: int32 [B, max_pages]: entries of the pages that the new
 *   tokens start are written, entries of the cached pages are read.
 *   free_pages: int32 [n_free], free_count: int32 [1]: entries
 *   0 .. count - 1 are free; pages are taken from the top, in request order
 *   and page order.  free_left: int32 [1] (written): the count after the call.
 *   Outputs: cu_seqlens_q int32 [B + 1]; seq_lens int32 [B] = ctx + new;
 *   positions, slots int32 [total_q]: token cu[r] + i of request r has
 *   position P = ctx_r + i and slot page(P) * page_size + P % page_size.
 *   Tokens from cu[B] on (padding) get position 0 and slot -1.
 *   seq_lens may be ctx_lens (or new_lens) and free_left may be free_count: they
 *   are read before they are written, so a captured step can advance itself.
 *   1 <= B <= 16384, total_q >= 1, page_size a multiple of 8 in [8, 1024],
 *   n_free >= 1 (the array; count may be 0).
 * On the device, reported as ATTN_ERR_DEVICE_DATA: a negative length, or one
 * past max_pages * page_size (clamped); more tokens than total_q; a count
 * outside [0, n_free]; too few free pages (the tokens without a page get slot
 * -1 and their table entry is -1); a page id outside [0, num_pages) (slot -1). */
attn_status_t attn_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int32_t* block_table,
                              const int32_t* free_pages, const int32_t* free_count, int B, int total_q,
                              int page_size, int max_pages, int num_pages, int n_free, int32_t* cu_seqlens_q,
                              int32_t* seq_lens, int32_t* positions, int32_t* slots, int32_t* free_left,
                              void* stream);

/* Cache append: q and k rotated as by attn_rope, k and v written to their
 * cache slots, in one pass over the new tokens.
 *   q [T, H, d], k, v [T, H_kv, d], bf16, through element strides (views of a
 *   fused projection), head dim dense; q_out [T, H, d], which may be q.
 *   q and q_out may both be NULL (H ignored): only K and V.
 *   k_cache, v_cache: bf16 [num_pages, page_size, H_kv, d].
 *   slots: int32 [T], page * page_size + row.  A negative slot marks a token
 *   that is skipped: nothing of it is read or written.  A slot past the cache
 *   is skipped and sets ATTN_ERR_DEVICE_DATA.  Two tokens with the same slot
 *   leave either's values there, or a mixture.
 *   positions: int32 [T]; inv_freq, freq_bits as for attn_rope.  rot = 0 (both
 *   may be NULL) stores k as it is and copies q.
 *   strides: HOST array of 8: (t, h) of q, q_out, k, v, in elements, multiples
 *   of 8; input strides may be 0; q_out strides are at least d.
 *   d in {64, 128}; rot 0 or a multiple of 16 up to d; page_size a multiple of
 *   8 in [8, 1024]; T >= 1.  Errors as attn_rope. */
attn_status_t attn_paged_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                                void* v_cache, const int32_t* slots, const int32_t* positions,
                                const void* inv_freq, int freq_bits, int T, int H, int H_kv, int d, int rot,
                                int page_size, int num_pages, const long long* strides, int interleaved,
                                float amplitude, void* stream);

/* Page sketches: what attn_page_select scores instead of the keys.  For each
 * page and KV head, with max_c and min_c the extremes of channel c over the
 * page's valid keys and amp = max over c of |max_c|, |min_c|:
 *   sketch: int8 [num_pages, H_kv, 2 d]: round(max_c / amp * 127) for c < d,
 *   then round(min_c / amp * 127) (nearest, ties to even; 0 where amp = 0);
 *   amp: fp32 [num_pages, H_kv].  A page that holds an infinity or NaN gets
 *   amp = +inf and codes 0, and is always worth selecting.
 * The call renews the sketches of the pages that hold each request's newest
 * keys: the last cu_seqlens_q[r + 1] - cu_seqlens_q[r] of its seq_lens[r]
 * keys, or the last max_q_len of them where cu_seqlens_q is NULL.  So
 * max_q_len = 1 follows a decode step, and max_q_len = max_pages * page_size
 * rebuilds every page.
 *   k_cache as attn_paged_fwd reads it; block_table int32 [B, max_pages].
 *   With cu_seqlens_q, max_q_len bounds the tokens of a request (more are cut
 *   to the last max_q_len and set ATTN_ERR_DEVICE_DATA).
 *   d in {64, 128}; page_size a power of two in [8, 1024].
 * Rows of a page past the request's last key are not read.  Requests that
 * share a page (a common prefix) renew it alike as long as the page is full;
 * one that is still being filled belongs to one request. */
attn_status_t attn_page_sketch(const void* k_cache, const int32_t* block_table, const int32_t* cu_seqlens_q,
                               const int32_t* seq_lens, int B, int max_q_len, int H_kv, int d, int page_size,
                               int max_pages, int num_pages, int8_t* sketch, float* amp, void* stream);

/* Page selection.  Query token t of request r (q and cu_seqlens_q as for
 * attn_paged_fwd, causal: position P = seq_lens[r] - q_len + i) sees the n =
 * P / page_size + 1 pages that hold keys 0 .. P.  If n <= budget all of them
 * are taken.  Otherwise, per KV head, the first `first` pages, the last `last`
 * pages (the query's own page is the last) and, of the rest, those with the
 * highest scores, ties to the earlier page, budget pages in all:
 *   c_h = round(q_h / |q_h|max * 127)   (8-bit codes of query head h)
 *   I_h(p) = sum_c max(c_h, 0) max8_c(p) + min(c_h, 0) min8_c(p)
 *   score(p) = max over the group's heads of (|q_h|max I_h(p)) * amp(p)
 * an 8-bit estimate of the largest q.k that a key of the page can have.  I_h
 * is an integer sum, exact in any order, and each product above is one fp32
 * rounding, so the choice does not depend on how the work is split.  (NaN
 * scores and non-finite sketches count as +inf; |q_h|max infinite or NaN makes
 * that head's score +inf.)
 *   tables: int32 [total_q, H_kv, budget], the chosen pages' physical ids in
 *   the order of their keys (-1 for one out of range), -1 behind them; sel_lens: int32 [total_q], the
 *   keys they hold for the token: the same for every KV head, since a token's
 *   own page, the only one that may be partial, is always chosen.  Tokens
 *   behind the last request, and tokens that see no key, get 0 and -1.
 *   H / H_kv <= 128; budget >= 1; first >= 0, last >= 1, first + last <=
 *   budget; total_q * H_kv * max(max_pages, budget) < 2^31.
 *   workspace: attn_page_select_workspace_size bytes, 16-byte aligned, no
 *   initialisation; where that is 256 (budget >= max_pages) none is used and
 *   NULL will do. */
size_t attn_page_select_workspace_size(int total_q, int H_kv, int max_pages, int budget);
attn_status_t attn_page_select(const void* q, const int8_t* sketch, const float* amp, const int32_t* block_table,
                               const int32_t* cu_seqlens_q, const int32_t* seq_lens, int B, int total_q, int H,
                               int H_kv, int d, int page_size, int max_pages, int num_pages, int budget, int first,
                               int last, int32_t* tables, int32_t* sel_lens, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Page-sparse attention: attn_page_select, then attention of each query
 * token over the keys of its chosen pages, per KV head; LSE over those keys.
 * With budget >= the pages in use it is attn_paged_fwd with causal = 1.
 *   k_cache, v_cache, block_table, seq_lens, q, o, lse (or NULL), scale,
 *   cu_seqlens_q (NULL: one token per request, total_q = B) as for
 *   attn_paged_fwd; sketch, amp, budget, first, last as for attn_page_select;
 *   tables, sel_lens: the selection, written when not NULL (both or neither).
 * A token that sees no key gets O = 0 and lse = -inf, one with a NaN among the
 * scores of its chosen keys NaN in both; rows behind the last request are left
 * as they were.
 * Each token gathers its own pages: meant for decode steps and the few tokens
 * per request of a drafted continuation; a long prompt is better served by
 * attn_paged_fwd, whose tiles share the keys among 128 rows.
 * Groups of up to 24 heads (d = 64: 32) with a budget of up to 1024 pages and
 * tables of up to 22000 pages run as one kernel that keeps everything on chip;
 * the others as a selection and the kernel of attn_paged_fwd.  Scores, maxima
 * and sums are fp32 on both.  The one kernel takes the probabilities to 2^-16
 * (as two bf16 numbers each), so O is off by little more than its own rounding
 * to bf16; the other rounds them to bf16 before the product with V, as
 * attn_paged_fwd does.
 *   workspace: attn_paged_sparse_fwd_workspace_size bytes, 16-byte aligned,
 *   no initialisation; calls that may overlap need distinct workspaces.  Where
 *   the size is 256 (one kernel) none is used and NULL will do. */
size_t attn_paged_sparse_fwd_workspace_size(int total_q, int H, int H_kv, int d, int page_size, int max_pages,
                                            int budget);
attn_status_t attn_paged_sparse_fwd(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_table, const int32_t* cu_seqlens_q,
                                    const int32_t* seq_lens, const int8_t* sketch, const float* amp, int B,
                                    int total_q, int H, int H_kv, int d, int page_size, int max_pages,
                                    int num_pages, int budget, int first, int last, float scale, void* o,
                                    float* lse, int32_t* tables, int32_t* sel_lens, void* workspace,
                                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_GB300_ATTN_KV_H */
