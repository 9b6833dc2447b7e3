/*
 * qsa_layer.h -- the operators around the selected-slot attention in a serving layer
 * (part of libqsa.so, B200 / sm_100a):
 *
 *   qsa_qk_norm_rope      per-head norm and position rotation of queries and keys in one
 *                         pass, keys and values stored to their cache slots
 *   qsa_pack_index_keys   int8 codes of the keys of the cheap score, one per micro-block
 *   qsa_select_slots      the cheap score and the choice of every query row's slots: writes
 *                         the slot_idx / width that qsa_sparse_prefill takes
 *   qsa_paged_decode      attention of one new token per sequence over its whole paged
 *                         cache, split over the cache's length and joined
 *
 * The conventions are those of qsa.h: device pointers owned by the caller, strides in
 * elements of the tensor's own type with an innermost stride of 1, nothing is allocated
 * or synchronised, errors are returned before any launch and leave the outputs untouched,
 * values that the host cannot see are checked on the device and reported through
 * *err_word (QSA_ERRBIT_*, may be NULL).  Sizes of zero are no-ops that return QSA_OK.
 * Results are deterministic: the same inputs give bitwise the same outputs.  Outputs and the
 * workspace must not overlap the inputs, except where an argument says so; a workspace is
 * in use until the call's work on the stream is done.
 */
#ifndef QSA_LAYER_H_
#define QSA_LAYER_H_

#include "qsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most position axes of qsa_qk_norm_rope, most heads of the cheap score, and the largest
 * numbers of selected blocks and of selected slots (blocks times block) of a row. */
#define QSA_MAX_ROPE_AXES 4
#define QSA_MAX_INDEX_HEADS 64
#define QSA_MAX_TOP_BLOCKS 8192

/* A further bit of *err_word: a bounded wait (one second) of qsa_select_slots for its own
 * copies or products ran out (the device was stopped or is failing).  The rows whose scores
 * were computed with those come out empty: a width of 0, and -1 for every slot. */
#define QSA_ERRBIT_TIMEOUT 0x10u

/*
 * qsa_qk_norm_rope -- norms of queries and keys for each head, with the position rotation
 * and the store to the cache in the same pass.
 *
 * For every token t and head h of q (and of k):
 *   n = x * 1/sqrt(mean(x^2) + eps) * (weight + weight_offset)      (x without a weight)
 *   pair i < rot / 2: a = positions[axis(i), t] * inv_freq[i],  (c, s) = rope_scale (cos a, sin a)
 *     (u, v) = dimensions (i, i + rot / 2), or (2 i, 2 i + 1) with interleaved = 1
 *     (u, v) -> (u c - v s, v c + u s);   dimensions >= rot pass unrotated
 * The angle is reduced in 64 bits, so far positions lose nothing; everything else is
 * 32-bit, rounded once at the store.
 *
 *   q, k, v       bf16 [T, Hq | Hkv, D], strides (t, h).  q (with Hq = 0), k and v may be
 *                 absent (NULL); v needs k.  v is not normed or rotated, only stored.
 *   q_weight, k_weight   bf16 [D], or NULL: not normed.
 *   positions     int32 [axes, T], axis stride pos_stride; inv_freq float [rot / 2].
 *   sections      HOST array of `axes` pair counts whose sum is rot / 2: the first
 *                 sections[0] pairs turn by axis 0, the next sections[1] by axis 1, ...
 *                 NULL with axes = 1.
 *   q_out         bf16 [T, Hq, D].  May be q itself (same pointer and strides).
 *   k_dst, v_dst  [rows, Hkv, D], strides (row, h): token t goes to row slots[t], or to
 *                 row t when slots is NULL (then rows must be >= T; k_dst may be k).
 *                 bf16, or with kv_fp8 E4M3 codes of x * (1 / k_scale) (x * (1 / v_scale)),
 *                 saturated (strides in bytes).  slots[t] = -1 stores nothing; another value outside
 *                 [0, rows) stores nothing and sets QSA_ERRBIT_SLOT_RANGE.  When two tokens
 *                 name one slot, what it holds is unspecified.  With slots and rows = 0 the
 *                 destinations may be NULL.
 *   D is 64, 128 or 256; rot is a multiple of 16, at most D (0: no rotation).
 * Pointers are 16-byte aligned (positions, inv_freq, slots: 4) and strides multiples of 16
 * bytes (8 bytes for E4M3 destinations).
 */
qsa_status_t qsa_qk_norm_rope(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                              int64_t k_stride_t, int64_t k_stride_h, const void* v,
                              int64_t v_stride_t, int64_t v_stride_h, const void* q_weight,
                              const void* k_weight, float weight_offset, float eps,
                              const int32_t* positions, int64_t pos_stride, const float* inv_freq,
                              int32_t rot, int32_t interleaved, const int32_t* sections,
                              int32_t axes, float rope_scale, int32_t T, int32_t Hq, int32_t Hkv,
                              int32_t D, void* q_out, int64_t q_out_stride_t,
                              int64_t q_out_stride_h, void* k_dst, int64_t k_dst_stride_s,
                              int64_t k_dst_stride_h, void* v_dst, int64_t v_dst_stride_s,
                              int64_t v_dst_stride_h, const int32_t* slots, int64_t rows,
                              int32_t kv_fp8, float k_scale, float v_scale, uint32_t* err_word,
                              void* stream);

/*
 * qsa_pack_index_keys -- the cheap score's key of each named micro-block.
 *
 * For every i < n with b = blocks[i] >= 0:
 *   m = (keys[b block] + ... + keys[b block + block - 1]) / block     (32-bit, in slot order)
 *   scales[b] = max |m| / 127,   codes[b] = round-half-even(m / scales[b])   (0 when the scale is 0;
 *   held to 127 in magnitude, which a quotient over a subnormal scale, itself rounded, may exceed)
 * A block whose keys hold a non-finite value gets codes 0 and a NaN scale, which the
 * selection ranks last.
 *
 *   keys    bf16 [S, Di], row stride key_stride_s (multiple of 8): one index key per slot.
 *   blocks  int32 [n] physical micro-blocks (slot / block); -1 is skipped, another value
 *           outside [0, floor(S / block)) is skipped and sets QSA_ERRBIT_SLOT_RANGE.
 *   codes   int8 [floor(S / block), Di], row stride code_stride (multiple of 16);
 *   scales  float [floor(S / block)].  Blocks that are not named keep what they hold.
 *   Di is 64 or 128; block is 1..16.
 */
qsa_status_t qsa_pack_index_keys(const void* keys, int64_t key_stride_s, const int32_t* blocks,
                                 int32_t n, int32_t block, int32_t Di, int64_t S, int8_t* codes,
                                 int64_t code_stride, float* scales, uint32_t* err_word,
                                 void* stream);

/*
 * qsa_select_slots -- the cheap score of every query row against the micro-blocks of its
 * sequence, and the slots of the blocks that score best.
 *
 * Row t is the i-th of the n_b rows of sequence b (cu_q[b] <= t < cu_q[b + 1]; with cu_q
 * NULL every sequence has one row).  It sees p = seq_lens[b] - (n_b - 1 - i) tokens, i.e.
 * f = floor(p / block) complete micro-blocks and p mod block slots of an incomplete one.
 *   query codes: as the keys' (scale s_h, integers c_h) for every head;  g_h = weight[t, h] s_h
 *   score(j) = scales[j] * sum_h g_h * max(0, c_h . codes[j]),   j < f
 * The products of codes are exact integers; every other product and sum is rounded to 32
 * bits, the heads added in order, so the score, and with it the choice, does not depend
 * on how the work is laid out.  The row takes min(top_blocks, f) blocks: first blocks
 * j < sink_blocks, j >= f - local_blocks, then those of the largest score; a NaN score
 * counts as -infinity and equal ones go to the lower j.
 *
 *   slot_idx  int32 [Tq, W], W = top_blocks * block + block - 1: the slots of the taken
 *             blocks in ascending j, then those of the incomplete micro-block, then -1.
 *   width     int32 [Tq]: how many of them there are.
 * Rows of no sequence (before cu_q[0], from cu_q[B] on) keep what they hold.
 *
 *   q           bf16 [Tq, Hi, Di], strides (t, h); weight float [Tq, Hi], row stride weight_stride.
 *   codes, scales   what qsa_pack_index_keys makes, `pages` * page_size / block of them.
 *   page_table  int32 [B, P], row stride page_stride: the sequence's tokens
 *               [page_size m, page_size (m + 1)) lie in the slots of page page_table[b, m].
 *               page_size is a multiple of block.  A page outside [0, pages) sets
 *               QSA_ERRBIT_SLOT_RANGE; its blocks score -infinity and its slots come out
 *               as -1.
 *   seq_lens    int32 [B]; values outside [0, P page_size] are clamped and set
 *               QSA_ERRBIT_WIDTH_RANGE, as do values of cu_q outside [0, Tq].
 *   cu_q        int32 [B + 1], non-decreasing.  One that decreases sets
 *               QSA_ERRBIT_WIDTH_RANGE, and the rows are not valid: slots of the pool, or -1.
 *   1 <= Hi <= 64, Di 64 or 128, block 1..16, top_blocks >= 1 with top_blocks * block <= 8192,
 *   sink_blocks + local_blocks <= top_blocks.
 *   workspace   qsa_select_slots_workspace_bytes(...) bytes, 256-byte aligned.  They hold the
 *               32-bit scores of a chunk of rows (512 MiB, or 64 rows where those are more)
 *               and, with many rows per sequence and at most 32 heads, the codes of all
 *               query rows: about Tq H (Di + 4) bytes, H the heads rounded up to a power of
 *               two, and 256 (Di + 4) more for each sequence of each chunk.
 */
size_t qsa_select_slots_workspace_bytes(int32_t Tq, int32_t B, int32_t P, int32_t page_size,
                                        int32_t Hi, int32_t Di, int32_t block);
qsa_status_t qsa_select_slots(const void* q, int64_t q_stride_t, int64_t q_stride_h,
                              const float* weight, int64_t weight_stride, const int8_t* codes,
                              int64_t code_stride, const float* scales, const int32_t* page_table,
                              int64_t page_stride, const int32_t* seq_lens, const int32_t* cu_q,
                              int32_t Tq, int32_t B, int32_t P, int64_t pages, int32_t page_size,
                              int32_t Hi, int32_t Di, int32_t block, int32_t top_blocks,
                              int32_t sink_blocks, int32_t local_blocks, int32_t* slot_idx,
                              int64_t idx_stride_t, int32_t* width, void* workspace,
                              size_t workspace_bytes, uint32_t* err_word, void* stream);

/*
 * qsa_paged_decode -- attention of one new token per sequence over its paged cache.
 *
 * For every sequence b, head h and KV head j = floor(h / (Hq / Hkv)), over the seq_lens[b]
 * tokens i whose slots the page table names (slot = page_table[b, i / page_size] * page_size
 * + i mod page_size):
 *   s_i = scale * q[b, h] . k_cache[slot_i, j];   out[b, h] = sum_i softmax(s)_i v_cache[slot_i, j]
 * or exactly +0 when the sequence has no token, and NaN (out and lse) when a score is NaN.
 * The tokens of all sequences are shared out evenly over the thread blocks; pieces of one
 * sequence are joined by their log-sum-exp.
 *
 *   q            bf16 [B, Hq, D], strides (b, h);  out bf16 [B, Hq, D].
 *   k_cache, v_cache   [pages * page_size, Hkv, D] (fewer than 2^31 slots, their strides
 *                below 2^30 elements): bf16, or E4M3 codes with kv_fp8 (strides in bytes), dequantised as code * k_scale (v_scale).
 *   page_table   int32 [B, P], row stride page_stride.  A page outside [0, pages) sets
 *                QSA_ERRBIT_SLOT_RANGE; its tokens are masked.
 *   seq_lens     int32 [B]; values outside [0, P page_size] are clamped and set
 *                QSA_ERRBIT_WIDTH_RANGE.
 *   lse          float [B, Hq] (contiguous), or NULL: the base-2 log-sum-exp of the scaled
 *                scores (-infinity without a token).
 *   blocks       0 = automatic, else the number of thread blocks, at most 65536 (the plan makes it
 *                a multiple of Hkv, and smaller when there is less work); the order of the
 *                sums, and with it the last bits, depend on it.
 *   workspace    as planned, 16-byte aligned (fp32 partial outputs and log-sum-exp).
 *   The weights are rounded to 16 bits for their product with V, in numerator and denominator
 *   alike (bf16, 2^-8 of each; with kv_fp8 16-bit floats, 2^-11, or 2^-32 of the largest weight
 *   where that is more); scores, sums and joins are 32-bit.
 *   D must be 256 and 1 <= Hq / Hkv <= 16.  With kv_fp8 the products run on 16-bit floats:
 *   a query element of 65536 or more sets QSA_ERRBIT_Q_RANGE (that row is not valid), and one
 *   below 2^-17 is rounded to a multiple of 2^-24.
 */
int32_t qsa_paged_decode_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                              int32_t page_size, int32_t kv_fp8, int32_t num_sms,
                              int32_t blocks_request, size_t* workspace_bytes);
qsa_status_t qsa_paged_decode(const void* q, int64_t q_stride_b, int64_t q_stride_h,
                              const void* k_cache, int64_t k_stride_s, int64_t k_stride_h,
                              const void* v_cache, int64_t v_stride_s, int64_t v_stride_h,
                              const int32_t* page_table, int64_t page_stride,
                              const int32_t* seq_lens, int32_t B, int32_t Hq, int32_t Hkv,
                              int32_t D, int32_t P, int64_t pages, int32_t page_size, float scale,
                              int32_t kv_fp8, float k_scale, float v_scale, void* out,
                              int64_t out_stride_b, int64_t out_stride_h, float* lse,
                              int32_t blocks, void* workspace, size_t workspace_bytes,
                              uint32_t* err_word, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* QSA_LAYER_H_ */
