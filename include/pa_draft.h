/*
 * pa_draft.h -- one speculative-decoding step over the paged KV cache (C ABI).
 *
 * A small drafter proposes several continuations of each sequence as a TREE of tokens;
 * the large model scores the whole tree in one pass and keeps one branch of it
 * (deeplearn.tn, "Les leviers d'optimisation en production": several drafted tokens are
 * verified in one pass of the large model).  The calls of this header are the pieces of
 * that pass that touch the cache or decide what enters it:
 *
 *   pa_rotary_and_cache   rotate queries and keys to their positions and, for tokens that
 *                         are certain (a prompt chunk, plain decode), append to the cache;
 *   pa_tree_attention     the tree's rows attend the cached context and their ancestors;
 *   pa_verify_tree        accept or reject the drafted tokens, draw the next one, and give
 *                         every row its cache slot (-1 where it is not kept).
 *
 * The tree's keys and values stay outside the cache until the verification has spoken:
 * pa_tree_attention takes them as [T][Hkv][D] tensors beside the cache, and the kept rows
 * are then appended by pa_reshape_and_cache / pa_quantize_kv(_fp8) with the slot_mapping
 * that pa_verify_tree wrote (negative slots are skipped).  No cache row is ever taken back.
 *
 * Rows: T rows packed by sequence, sequence s owning rows query_start[s] ..
 * query_start[s + 1] - 1.  Within a sequence, row 0 is the tree's root -- the newest token
 * that is certain, whose keys are not cached yet -- and parents[row] is the in-sequence
 * index of the row a token was drafted after: -1, or an index below the row's own.  A chain
 * of drafts has parents -1, 0, 1, 2, ...  At most PA_TREE_MAX_NODES rows per sequence.
 *
 * Conventions (streams, alignment, device-side checks, err_flag) as in pa.h.
 */
#ifndef PA_DRAFT_H
#define PA_DRAFT_H

#include <stddef.h>
#include <stdint.h>

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_TREE_MAX_NODES 256

enum { PA_PROB_F32 = 0, PA_PROB_BF16 = 1 };

/* How pa_rotary_frequencies scales the frequencies for contexts longer than trained on. */
enum {
    PA_ROTARY_PLAIN = 0,      /* f_j = base^(-2j / rot_dim)                                    */
    PA_ROTARY_LINEAR = 1,     /* f_j / factor: positions interpolated                          */
    PA_ROTARY_BASE = 2,       /* base grown to base * factor^(rot_dim / (rot_dim - 2))         */
    PA_ROTARY_RAMP = 3,       /* f_j kept for pairs that turn more than p0 times within
                                 original_context, f_j / factor below p1 turns, a linear ramp
                                 over the pair index between ("by parts" interpolation of the
                                 YaRN paper); attention factor 0.1 ln(factor) + 1              */
    PA_ROTARY_WAVELENGTH = 4  /* f_j kept where the wavelength 2 pi / f_j is below
                                 original_context / p1, f_j / factor above original_context /
                                 p0, blended linearly in original_context / wavelength between */
};

/*
 * Angular frequencies (radians per position) of the rot_dim / 2 rotated pairs: a host
 * computation.
 *   rot_dim            even, >= 2 (PA_ROTARY_BASE: >= 4).
 *   base               > 1.
 *   factor             >= 1; ignored by PA_ROTARY_PLAIN.
 *   original_context, p0, p1   PA_ROTARY_RAMP (p0 > p1 > 0 turns, 32 and 1 in the paper) and
 *                      PA_ROTARY_WAVELENGTH (0 < p0 < p1) only; ignored otherwise.
 *   inv_freq           host, rot_dim / 2 doubles (written).
 *   attention_factor   host, nullable: what queries and keys are scaled by (1 except for
 *                      PA_ROTARY_RAMP).
 */
pa_status pa_rotary_frequencies(int rot_dim, double base, int scaling, double factor,
                                double original_context, double p0, double p1, double *inv_freq,
                                double *attention_factor);

/*
 * The table pa_rotary_and_cache reads: table[j] = inv_freq[j] / (2 pi) turns per position
 * as a 64-bit fraction of a turn (units of 2^-64, rounded; whole turns drop out).  A
 * position times an entry, modulo 2^64, is the angle with every whole turn removed
 * exactly, so far positions lose nothing.  Host arrays of n entries; any finite inv_freq.
 */
pa_status pa_rotary_table(const double *inv_freq, int n, uint64_t *table);

/*
 * Rotary positions, fused with the append.  For token t at position p = positions[t], pair
 * j < rot_dim / 2, angle a = p * inv_freq[j], c = attention_factor cos a, s =
 * attention_factor sin a, every query head and key head is rotated:
 *   y[i] = x[i] c - x[i'] s,   y[i'] = x[i'] c + x[i] s,
 *   (i, i') = (j, j + rot_dim / 2), or (2j, 2j + 1) when interleaved;
 * elements from rot_dim on are left as they are (and not scaled).
 *   query, key, value  [T][heads][D] bf16, device: the heads of a token dense, tokens
 *                      query_stride / key_stride / value_stride elements apart (multiples of
 *                      8, at least heads * D), so slices of one projection's output will do.
 *   positions          [T] int64, device (any value; negative ones rotate backwards).
 *   table              [rot_dim / 2] uint64, device (pa_rotary_table).
 *   rot_dim            even, 2 .. D.
 *   query_out          [T][Hq][D] bf16, dense.  May be query itself when that is dense.
 *   key_out            [T][Hkv][D] bf16, dense, or NULL.  May be key itself when that is
 *                      dense.  Outputs must not overlap inputs in any other way.
 *   k_cache, v_cache   the paged cache, or both NULL: no append, and value, slot_mapping and
 *                      the scales are ignored (then key_out must be given).  Layouts,
 *                      kv_dtype, scales and slot_mapping (negative: not appended; the
 *                      others of a call must differ) as in pa_reshape_and_cache and
 *                      pa_quantize_kv(_fp8).
 * Products and sums are fp32 with one rounding to bf16.  An 8-bit cache quantises the
 * rotated fp32 key by pa_quantize_kv(_fp8)'s rule directly, without rounding it to bf16
 * first; value rows are bit-identical to those calls.  D in {64, 128}, bs in {16, 32}.
 */
pa_status pa_rotary_and_cache(pa_bf16 *query_out, pa_bf16 *key_out, const pa_bf16 *query,
                              int64_t query_stride, const pa_bf16 *key, int64_t key_stride,
                              const pa_bf16 *value, int64_t value_stride, void *k_cache,
                              void *v_cache, float *k_scale, float *v_scale, int kv_dtype,
                              const int64_t *slot_mapping, const int64_t *positions,
                              const uint64_t *table, int rot_dim, int interleaved,
                              float attention_factor, int T, int Hq, int Hkv, int D, int bs, int N,
                              int *err_flag, void *stream);

/* Bytes of device workspace pa_tree_attention needs (0 for invalid arguments as well). */
size_t pa_tree_workspace_size(int S, int T, int Hq, int Hkv, int D, int bs, int kv_dtype,
                              int max_context_len, int max_query_len);

/*
 * Attention of a tree of drafted tokens.  Row i of sequence s attends all context_lens[s]
 * cached tokens and, among its sequence's own rows, itself and its ancestors:
 *   out[i][h] = sum_t softmax_t(scale * q[i][h] . k_t) v_t.
 *   query, out         [T][Hq][D] bf16, dense.
 *   key, value         [T][Hkv][D] bf16: the rows' own keys (rotated) and values; heads
 *                      dense, rows key_stride / value_stride elements apart (multiples of 8,
 *                      at least Hkv * D).
 *   context_lens       [S] int32, device: cached tokens, the tree's rows not included; may
 *                      be 0 (max_context_len too).
 *   query_start        [S + 1] int32, device; parents [T] int32, device (see above; several
 *                      rows of a sequence may have parent -1).
 *   max_query_len      host bound of the rows of a sequence, 1 .. min(T, PA_TREE_MAX_NODES).
 *   workspace          pa_tree_workspace_size(...) bytes, 256-byte aligned; nothing in it is kept from
 *                      one call to the next, but calls that may run at the same time (streams,
 *                      replayed graphs) need one each.
 * A sequence whose offsets are outside [0, T], decreasing or longer than max_query_len is
 * left out (PA_FLAG_QUERY_OUT_OF_RANGE), as is one with a parent that is neither -1 nor
 * below its row (PA_FLAG_TREE_PARENT): its rows of out are not written.  Other arguments,
 * cache types and device-side checks as in pa_multi_token_attention.  Scores, softmax
 * statistics and weighted sums are fp32, the weights of cached tokens bf16 (fp16 with 8-bit
 * caches); the result is rounded once to bf16.  Values of an 8-bit cache with D = 128 are
 * taken as fp16(code * fp16(scale)), within 2^-10 of code * scale, or 2^-31 of the largest
 * scale of the 128 tokens they are read with where that is more.
 */
pa_status pa_tree_attention(pa_bf16 *out, const pa_bf16 *query, const pa_bf16 *key,
                            int64_t key_stride, const pa_bf16 *value, int64_t value_stride,
                            const void *k_cache, const void *v_cache, const float *k_scale,
                            const float *v_scale, int kv_dtype, const int32_t *block_tables, int M,
                            const int32_t *context_lens, const int32_t *query_start,
                            const int32_t *parents, int S, int T, int Hq, int Hkv, int D, int bs,
                            int N, float scale, int max_context_len, int max_query_len,
                            void *workspace, size_t workspace_bytes, int *err_flag, void *stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given random
 * numbers; the tokens kept and the next one are distributed as if the target had been
 * sampled token by token.  The walk starts at row 0 of each sequence.  At row c with
 * target distribution p = target_probs[c] and, with draft_probs, the distribution q =
 * draft_probs[c] that c's children were independently drawn from, the children x_1, x_2,
 * .. are tried in row order, with R_k(v) = max(p(v) - C_k q(v), 0), C_0 = 0, Z_0 = 1:
 *   child x of row r is accepted if uniforms[r] * Z_k * q(x) < R_k(x), and the walk moves
 *   to it; otherwise C_{k+1} = C_k + Z_k and Z_{k+1} = sum_v R_{k+1}(v)
 * (k counts the rejected children: R_k / Z_k is the residual distribution
 * norm(max(R - q, 0)) taken k times).  Without draft_probs the children are the drafter's
 * fixed choices: q(x) = 1, and a rejected token's R becomes 0.  Where no child is
 * accepted the next token is drawn from R: the first v whose running sum of R exceeds
 * final_uniforms[s] * sum(R) (from p itself if R has no mass left).
 *   draft_tokens       [T] int32: the rows' tokens (row 0's is not read).  A token outside
 *                      [0, V) is never accepted (PA_FLAG_TOKEN_OUT_OF_RANGE).
 *   target_probs, draft_probs  [T] rows of V probabilities, fp32 or bf16 (prob_dtype), rows
 *                      target_stride / draft_stride elements (>= V) apart; draft_probs may be
 *                      NULL.  Negative and NaN entries count as 0.  A row that has to be drawn
 *                      from and sums to 0 or not to a finite number gives token -1
 *                      (PA_FLAG_PROBABILITY).
 *   uniforms [T], final_uniforms [S]   fp32 in [0, 1) (row 0's is not read).
 *   tokens_out, path   [S][max_query_len] int32 (written): the rows walked, as indices into
 *                      [0, T), root first, and the token that follows each: the accepted
 *                      drafts, then the token drawn; -1 behind them.
 *   n_out              [S] int32 (written): how many, 1 + accepted drafts; 0 for a sequence
 *                      that is empty or left out.
 *   slot_mapping       [T] int64 (written for the rows of sequences), or NULL: the cache slot
 *                      of each row walked, position context_lens[s] + place on the path
 *                      through block_tables [S][M]; -1 for the others.  A slot whose table
 *                      entry is missing or outside [0, N) is -1 (PA_FLAG_BLOCK_OUT_OF_RANGE).
 *                      Ignored when NULL: block_tables, M, context_lens, bs, N.
 * A sequence with bad offsets or parents is left out as in pa_tree_attention.  Sums,
 * products and the borders drawn at are carried in pairs of fp32 (about 48 bits), always in
 * the same order for the same shapes.  V <= 2^30, max_query_len <= min(T, PA_TREE_MAX_NODES).
 */
pa_status pa_verify_tree(int32_t *tokens_out, int32_t *path, int32_t *n_out, int64_t *slot_mapping,
                         const int32_t *draft_tokens, const void *target_probs,
                         int64_t target_stride, const void *draft_probs, int64_t draft_stride,
                         int prob_dtype, const int32_t *query_start, const int32_t *parents,
                         const float *uniforms, const float *final_uniforms, int S, int T, int V,
                         int max_query_len, const int32_t *block_tables, int M,
                         const int32_t *context_lens, int bs, int N, int *err_flag, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_DRAFT_H */
