/*
 * attn_kv8.h -- C ABI of a paged KV cache held in 8 bits: appends that
 * quantise, reading back, and attention over it.
 *
 * The conventions of attn.h and attn_kv.h hold here too: device pointers owned
 * by the caller and 16-byte aligned (index arrays, scales and lse: 4-byte
 * aligned), asynchronous calls on `stream`, nothing enqueued when an argument
 * is refused, no memory allocated, ATTN_ERR_DEVICE_DATA in the device status
 * word for lengths, slots and page ids that are out of range on the device.
 * Every call can be captured into a CUDA graph and replayed.
 *
 * The cache.  Codes and scales, for K and for V:
 *   k_cache, v_cache: e4m3fn [num_pages, page_size, H_kv, d]
 *   k_scale, v_scale: fp32 [num_pages, H_kv, page_size / block]
 * The value of a code is decode(code) * scale of its block: `block` consecutive
 * rows of a page, of one KV head.  block is a power of two from 1 (a scale for
 * every token) to page_size (one for the page); page_size a power of two in
 * [8, 1024]; d in {64, 128}.  Scales are positive and finite (0 reads as 0);
 * those that attn_paged_append_fp8 writes are powers of two, so that a change
 * of scale moves codes without rounding them again, but for the smallest.
 * e4m3 numbers keep 4 significant bits at any scale, so a power of two costs
 * them nothing but the last of 15 binades.
 *
 * A serving step:
 *   attn_paged_plan (attn_kv.h)  lengths -> offsets, positions, slots, table rows
 *   attn_paged_append_fp8        q, k, v -> rotated q; K and V as codes in their slots
 *   attn_paged_fwd_fp8           the attention itself
 * and for a long prompt over a cached prefix:
 *   attn_paged_read_fp8          the requests' keys and values, packed, in 16 bits
 *   attn_varlen_fwd (attn.h)     the attention over them
 */
#ifndef ATTN_GB300_ATTN_KV8_H
#define ATTN_GB300_ATTN_KV8_H

#include "attn_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache append: q and k rotated as by attn_rope, k and v quantised into their
 * cache slots.
 *   q, q_out, k, v, slots, positions, inv_freq, freq_bits, rot, strides,
 *   interleaved, amplitude: as for attn_paged_append; q and q_out may both be
 *   NULL (H ignored).
 * For every block of a page that the call's tokens enter, and every KV head,
 * with r the first row they take in it:
 *   need = 2^e, e the smallest integer in [-126, 120] with amax <= 448 * 2^e,
 *          amax the largest magnitude among the block's new (rotated) rows;
 *   scale = need where r = 0, else max(the block's scale before, need);
 *   code = x / scale, rounded to the nearest e4m3 (ties to even), straight from
 *          the fp32 result of the rotation; an infinity or NaN becomes the
 *          code of NaN and does not count towards amax;
 *   rows 0 .. r - 1, where the scale grew: code * (before / scale), rounded.
 * Rows behind the last that the call writes in a block are no longer valid:
 * rows of a block are filled in order, from 0, or again from an earlier row.
 * Tokens of one block follow one another in the call, in the order of their
 * slots and without gaps (as attn_paged_plan numbers them); where they do not,
 * or where two tokens have the same slot, that block's contents and scale are
 * undefined.  A negative slot marks a token that is skipped: nothing of it is
 * read or written.  A slot past the cache is skipped and sets
 * ATTN_ERR_DEVICE_DATA.
 *   T >= 1; rot 0 or a multiple of 16 up to d; H and H_kv at most 65535;
 *   num_pages * page_size < 2^31.  Errors as attn_paged_append. */
attn_status_t attn_paged_append_fp8(const void* q, void* q_out, const void* k, const void* v, void* k_cache,
                                    void* v_cache, float* k_scale, float* v_scale, const int32_t* slots,
                                    const int32_t* positions, const void* inv_freq, int freq_bits, int T, int H,
                                    int H_kv, int d, int rot, int page_size, int block, int num_pages,
                                    const long long* strides, int interleaved, float amplitude, void* stream);

/* Reading back: the keys and values of B requests, packed one after another.
 *   cu_seqlens_k: int32 [B + 1], row offsets: request r's keys 0 .. n_r - 1,
 *   n_r = cu[r + 1] - cu[r], become rows cu[r] ..; rows from cu[B] on are left
 *   as they were.  block_table: int32 [B, max_pages].
 *   k, v: [total_k, H_kv, d], bf16 (elem_bytes 2) or fp32 (4): code * scale in
 *   fp32, rounded once to bf16 (which is exact for scales that are powers of
 *   two).  Either of k and v may be NULL, with its cache and scales.
 *   B, total_k, H_kv, max_pages >= 1; H_kv at most 65535.
 * On the device, reported as ATTN_ERR_DEVICE_DATA: offsets that are not
 * 0 <= cu[r] <= cu[r + 1] <= total_k, or more keys than the table holds (such
 * a request is skipped, and where offsets are not in order, rows of others may
 * be left as they were too); a page id out of range (its rows become 0).
 * Errors: ATTN_ERR_INVALID_ARG / ATTN_ERR_UNSUPPORTED before the launch;
 * ATTN_ERR_CUDA when it fails. */
attn_status_t attn_paged_read_fp8(const void* k_cache, const void* v_cache, const float* k_scale,
                                  const float* v_scale, const int32_t* block_table, const int32_t* cu_seqlens_k,
                                  int B, int total_k, int H_kv, int d, int page_size, int block, int max_pages,
                                  int num_pages, void* k, void* v, int elem_bytes, void* stream);

/* Attention over the cache: attn_paged_fwd on the values of the codes.
 *   s_j = scale * ks_j (q . kc_j),  O = sum_j softmax(s)_j vs_j vc_j,  LSE of s,
 * kc, vc the codes of key j and ks, vs the scales of its block.
 *   q, o: bf16 [total_q, H, d]; lse: fp32 [total_q, H] or NULL; block_table,
 *   cu_seqlens_q (NULL: one token per request, total_q = B and max_q_len = 1),
 *   seq_lens, max_q_len, scale, causal: as for attn_paged_fwd.  H a multiple
 *   of H_kv, H / H_kv at most 128; B at most 2^30.
 * Precision: the matrix units take the codes as they are, e4m3 by e4m3 with
 * fp32 sums.  q enters as two e4m3 numbers for each element over a power of two of its
 * head vector: exact where it is above 2^-12 of the vector's largest, off by less than 2^-21
 * of that below.  Probabilities (times their block's scale) enter
 * the second product as fp16 numbers, in four e5m2 numbers each: off by at most 2^-11 of themselves and
 * 2^-33 of the row's largest (2^-19 of it, if every scale of V that the row sees is below
 * 2^-112), so that a long tail of small ones counts in O as it does in the sum. Those below
 * 2^-126 of the largest are zero.  O is summed in fp32 before it is divided by the sum of probabilities.
 * Maxima, sums and exponentials are fp32; O is rounded once.
 * A token that sees no key gets O = 0 and lse = -inf; one with a NaN among its
 * scores NaN in both; rows behind the last request are left as they were.
 * Keys past a request's length are not part of any result, whatever their rows
 * hold.
 * Each run of up to 32 query rows (tokens times the heads of a group) streams
 * the request's keys: meant for decode steps and the few tokens per request of
 * a drafted continuation.  From about 80 rows of a KV head on (d = 128; 50 for
 * d = 64) attn_paged_read_fp8 and attn_varlen_fwd are faster: 16 requests of 8192
 * keys and 8 KV heads of 128 take 118 us for 32 rows, where those take 230, 210
 * and 245 for 64, 394 and 269 for 128.
 *   workspace: attn_paged_fwd_fp8_workspace_size bytes (0 on invalid sizes),
 *   16-byte aligned, no initialisation; calls that may overlap need distinct
 *   workspaces.
 * On the device, reported as ATTN_ERR_DEVICE_DATA: as for attn_paged_fwd. */
size_t attn_paged_fwd_fp8_workspace_size(int B, int total_q, int max_q_len, int H, int H_kv, int d, int page_size,
                                         int max_pages);
attn_status_t attn_paged_fwd_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                 const float* v_scale, const int32_t* block_table, const int32_t* cu_seqlens_q,
                                 const int32_t* seq_lens, int B, int total_q, int max_q_len, int H, int H_kv, int d,
                                 int page_size, int block, int max_pages, int num_pages, float scale, int causal,
                                 void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ATTN_GB300_ATTN_KV8_H */
