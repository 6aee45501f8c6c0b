/*
 * pkv_ops.h -- operators beside the decode path of pkv.h: the position rotation
 * on the way into the cache, a cache in 8 bits with one scale for each block and
 * kv head, attention over it, and attention with capped scores, a distance bias
 * or a sliding window.
 *
 * The conventions are those of pkv.h: device buffers owned by the caller, work
 * enqueued on `stream`, host arguments checked before anything is enqueued (an
 * error enqueues nothing), values in device memory never faulting.
 *
 * Block-scaled E4M3 pools
 * -----------------------
 * k_cache, v_cache: uint8 [num_blocks][16][num_kv_heads][head_dim] of E4M3 codes
 * (as pkv.h describes them). k_scale, v_scale: uint8 [num_blocks][num_kv_heads];
 * a byte b stands for the scale 2^(b - 127), so a code c of block p and kv head h
 * is the value e4m3(c) * 2^(scale[p][h] - 127). Byte 0 marks a block that holds
 * nothing yet; 255 is not used. A power of two costs at most one bit of E4M3's
 * range against a free scale, and lets a block's codes move to a larger scale
 * without a second rounding (short of the smallest codes).
 * pkv_copy_blocks serves such a pool too (a copy is a copy: pass head_dim / 2 for
 * its bf16 elements); the scale rows of the same blocks go with it.
 */
#ifndef PKV_OPS_H
#define PKV_OPS_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pkv_rotary_turns -- host: the rotation frequencies of rotary positions, as
 * 64-bit fixed point: turns[i] = f_i * 2^64 (modulo 2^64), f_i the turns (of a
 * full circle) per position of pair i,
 *     f_i = base^(-2 i / rotary_dim) / (2 pi),   0 <= i < rotary_dim / 2.
 * In this form position * turns wraps exactly where the angle does, so far
 * positions lose no accuracy. For contexts beyond those a model was trained on:
 *   PKV_ROPE_PLAIN   f_i as above (factor, original_length, low and high unused)
 *   PKV_ROPE_LINEAR  f_i / factor (positions interpolated)
 *   PKV_ROPE_BASE    base * factor^(rotary_dim / (rotary_dim - 2)) in place of
 *                    base: the slowest pair is slowed by factor, the fastest
 *                    hardly at all (rotary_dim >= 4)
 *   PKV_ROPE_RAMP    pairs that turn at least `high` times within
 *                    original_length positions keep f_i, those that turn at most
 *                    `low` times get f_i / factor, those between a linear blend
 *                    by their number of turns.
 * turns: host, uint64 [rotary_dim / 2]. PKV_ERR_NULL without it, PKV_ERR_SHAPE
 * for an odd or non-positive rotary_dim (or 2 with PKV_ROPE_BASE), PKV_ERR_RANGE
 * for a base <= 0, a factor <= 0, or (RAMP) original_length <= 0 or high <= low,
 * not finite numbers among them, PKV_ERR_UNSUPPORTED for another kind.
 */
enum { PKV_ROPE_PLAIN = 0, PKV_ROPE_LINEAR = 1, PKV_ROPE_BASE = 2, PKV_ROPE_RAMP = 3 };
pkv_status pkv_rotary_turns(int32_t rotary_dim, double base, int32_t kind, double factor,
                            double original_length, double low, double high, uint64_t *turns);

/*
 * pkv_rope_kv_append -- rotate the step's queries and keys by their positions
 * and write keys and values into their slots of a bf16 pool, in one launch.
 *
 * For row i, head h and pair j (0 <= j < rotary_dim / 2), with
 *     a = 2 pi * (positions[i] * turns[j] mod 2^64) / 2^64,
 *     x' = rotary_scale * (x cos a - y sin a),
 *     y' = rotary_scale * (y cos a + x sin a),
 * where (x, y) are dims (j, j + rotary_dim / 2) of the head, or with `interleaved`
 * dims (2 j, 2 j + 1); dims from rotary_dim on are copied. q' goes to q_out for
 * every row; k' and v go to the pool row of slot_mapping[i] as pkv_kv_append
 * writes it (negative or past the pool: that row writes no K and V). Computed in
 * fp32 (the angle in 64-bit fixed point), rounded once to bf16, nearest even; v
 * is copied bit for bit.
 *
 *   q             device, bf16, row i at q + i * q_stride, [num_q_heads][head_dim]
 *                 within a row; NULL (with q_out NULL and num_q_heads 0): keys and
 *                 values only
 *   k_new, v_new  device, bf16, rows k_stride / v_stride apart,
 *                 [num_kv_heads][head_dim] within a row
 *   strides       in elements; multiples of 8, at least the row's elements (the
 *                 three may be slices of one projection's output)
 *   positions     device, int64 [n_new]; any value (a negative one turns back)
 *   turns         device, uint64 [rotary_dim / 2] (pkv_rotary_turns)
 *   slot_mapping  device, int64 [n_new], as pkv_kv_append
 *   q_out         device, bf16 [n_new][num_q_heads][head_dim]; may be q itself
 *                 (then q_stride must be num_q_heads * head_dim), else no overlap
 *   k_cache, v_cache  device, bf16 [num_blocks][16][num_kv_heads][head_dim]
 *   head_dim      a multiple of 8, <= 1024; rotary_dim even, 2 .. head_dim
 *   rotary_scale  finite (1 for plain rotation)
 * q, k_new, v_new, q_out and the pools 16-byte aligned, positions, turns and
 * slot_mapping 8-byte. n_new == 0 is a no-op returning PKV_OK.
 */
pkv_status pkv_rope_kv_append(const void *q, int64_t q_stride, const void *k_new,
                              int64_t k_stride, const void *v_new, int64_t v_stride,
                              const int64_t *positions, const uint64_t *turns,
                              const int64_t *slot_mapping, int64_t n_new, void *q_out,
                              void *k_cache, void *v_cache, int64_t num_blocks,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t rotary_dim, int32_t interleaved, float rotary_scale,
                              void *stream);

/*
 * pkv_rope_kv_append_fp8_block -- the same into a block-scaled E4M3 pool.
 *
 * The scale of a block and head follows its contents. With A the largest finite
 * magnitude among the rows this call writes there (k' or v, in fp32) and e the
 * smallest integer (at least -126) with A <= 448 * 2^e:
 *  - a block that this call starts (it writes the block's row 0) gets the scale
 *    2^e; its other rows are left as they are;
 *  - a block that it continues gets the larger of 2^e and its scale so far; when
 *    that grew, all 16 rows of codes are first rounded to the new scale;
 * then each new element is E4M3(x / scale): nearest, ties to even, magnitudes
 * beyond 448 (infinities) saturated, NaN kept. Blocks and heads without a new
 * row are untouched.
 *
 * The rows of one block must follow one another in slot_mapping (a token run of
 * one sequence does) and name distinct slots; rows of one block that come apart,
 * or twice the same slot, leave that block unspecified.
 *
 *   k_scale, v_scale  device, uint8 [num_blocks][num_kv_heads]; zero before a
 *                     pool's first use
 *   head_dim          a multiple of 8, <= 256
 * Caches 8-byte aligned; everything else as pkv_rope_kv_append.
 */
pkv_status pkv_rope_kv_append_fp8_block(
    const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
    int64_t v_stride, const int64_t *positions, const uint64_t *turns,
    const int64_t *slot_mapping, int64_t n_new, void *q_out, void *k_cache, void *v_cache,
    uint8_t *k_scale, uint8_t *v_scale, int64_t num_blocks, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
    float rotary_scale, void *stream);

/*
 * pkv_paged_decode_attention_scored -- pkv_paged_decode_attention with its scores
 * capped, biased by distance, or limited to a window, over bf16 or block-scaled
 * E4M3 pools.
 *
 * With p = T - n_query_per_seq + j the position of query j (T as there), query
 * head qh and every visible position t <= p:
 *     x_t = scale * <q, K_s[t]>
 *     x_t = softcap * tanh(x_t / softcap)            if softcap > 0
 *     x_t = x_t + alibi_slopes[qh] * (t - p)          if alibi_slopes is given
 *     visible only if t > p - window                  if window > 0
 *     out = sum_t softmax(x)_t * V_s[t]
 * A query that sees nothing (p < 0) gives zeros. Blocks wholly before every
 * query's window are not read: their table entries may be anything. K and V of
 * positions that no query of the sequence sees may hold anything, NaN included.
 *
 *   k_scale, v_scale  uint8 [num_blocks][num_kv_heads] for block-scaled E4M3
 *                     pools (head_dim 128); both NULL for bf16 pools (head_dim 64
 *                     or 128); one alone is PKV_ERR_NULL
 *   softcap           finite, >= 0; 0: no cap (PKV_ERR_RANGE otherwise, or where
 *                     3 scale / softcap is beyond float)
 *   alibi_slopes      device, float [num_q_heads], finite, or NULL
 *   window            >= 0; 0: no window (PKV_ERR_RANGE otherwise)
 *   max_blocks_per_seq  how long a sequence may be: tables no wider than the batch
 *                     needs let few or short sequences be finished in one launch
 *                     (the results' rounding may differ with the width)
 *   workspace         >= pkv_workspace_size_scored(...) bytes, used as
 *                     pkv_paged_decode_attention uses its own
 * Other arguments, limits, errors and the error word as
 * pkv_paged_decode_attention; scores, softmax statistics and sums are fp32, the
 * result deterministic. Over bf16 pools a softmax weight is held as two bf16 terms
 * (2^-16). Over E4M3 pools a query row is scaled by a power of two and held in
 * f16 (exact but for elements below 2^-28 of its largest), and a weight as one f16
 * term (2^-11): before the output's rounding the error is at most 2^-11 of
 * sum p |V_s| / sum p beside the scores' own fp32 rounding.
 */
size_t pkv_workspace_size_scored(int32_t num_seqs, int32_t n_query_per_seq, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim);

pkv_status pkv_paged_decode_attention_scored(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
    int32_t n_query_per_seq, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    float scale, float softcap, const float *alibi_slopes, int32_t window, void *out,
    int32_t out_dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * pkv_paged_decode_attention_fp8_block -- pkv_paged_decode_attention over
 * block-scaled E4M3 pools: pkv_paged_decode_attention_scored without a cap, a bias
 * or a window, k_scale and v_scale required.
 */
pkv_status pkv_paged_decode_attention_fp8_block(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
    int32_t n_query_per_seq, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    float scale, void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
    void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_OPS_H */
