/*
 * specverify_step.h -- C ABI of libspecverify: the serving step around the
 * cached pass of specverify_lowbit.h.
 *
 * In the order of a step: pages are reserved for each sequence's new tokens,
 * queries and keys are normalised and rotated by their positions, keys and
 * values go into the cache (spec_cache4_write), and the new tokens attend to
 * it: through a window with a few first tokens that stay visible, or, for
 * branches of one prompt, to a prefix that is read once for all of them.
 *
 * Memory, streams, status codes and workspaces are those of
 * specverify_lowbit.h: array arguments are DEVICE pointers, the caller owns
 * every buffer, a call only enqueues work on `stream`, a workspace is plain
 * scratch of one call at a time.
 */
#ifndef SPECVERIFY_STEP_H
#define SPECVERIFY_STEP_H

#include "specverify_lowbit.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Norms of queries and keys for each head, and their rotation by position, in
 * one pass.
 *
 * A head x [D] of new token i of sequence b becomes
 *   y = x / sqrt(mean_d x[d]^2 + eps) * weight    (norm != 0; weight NULL: ones)
 *   y = x                                         (norm == 0; weights NULL)
 * and then, of its first rotary_dim values, n = rotary_dim / 2 pairs are turned:
 *   (y[c], y[c + n]), interleaved: (y[2c], y[2c + 1]),  c < n, by the angle
 *   (start[b] + depth[b][i]) * inv_freq[c],
 * (u, v) to (u cos - v sin, v cos + u sin); the others stay.  The angle is
 * taken in 64 bits and reduced there, so that positions of any size keep their
 * angles; the rest is F32, rounded once to the output's type. */
typedef struct {
  int32_t head_dim;     /* 16 .. 256, a multiple of 16 */
  int32_t rotary_dim;   /* 0 .. head_dim, a multiple of 16 */
  int32_t interleaved;  /* 0 or 1 */
  int32_t norm;         /* 0 or 1 */
  float eps;            /* finite, >= 0 (norm) */
  int32_t weight_dtype; /* spec_dtype_t */
  const void* q_weight; /* [head_dim] or NULL, 16-byte aligned */
  const void* k_weight;
  const float* inv_freq; /* [rotary_dim / 2]; NULL when rotary_dim is 0 */
  const int32_t* depth;  /* [T] of sequence b at depth + b * depth_stride, or NULL: i */
  int64_t depth_stride;  /* 0 shares one */
} spec_rotate_t;

/* q [B][T][q_heads][head_dim] to q_out, k [B][T][heads][head_dim] to k_out,
 * each F32 or BF16 (spec_heads_t).  An output may be its own input (same data,
 * type and strides); any other overlap is not allowed.  q_heads or heads may be
 * 0, at most 16384 together; the pair is then not looked at.
 *   start [B], any value;  count [B], or NULL: T new tokens each
 * Rows i >= count[b] are not read and their outputs stay as they were; all
 * T rows of a sequence whose count lies outside 0 .. T become NaN. */
int spec_norm_rotate(spec_heads_t q, spec_heads_t q_out, int32_t q_heads, spec_heads_t k,
                     spec_heads_t k_out, int32_t heads, const spec_rotate_t* how, int32_t B,
                     int32_t T, const int32_t* start, const int32_t* count, void* stream);

/* ---------------------------------------------------------------------------
 * spec_attention_cache4 through a window.  New token i stands at
 * start[b] + depth[b][i] and sees, of the cached positions x < start[b], those
 * with x > start[b] + depth[b][i] - window and those with x < sinks.  Of the new
 * tokens it sees those that its mask words name, whatever their distance; where
 * mask is NULL, those at j <= i with i - j < window or start[b] + j < sinks.
 *   window >= 1, sinks >= 0
 *   depth  [T] of sequence b at depth + b * depth_stride (0 shares one), a tree's
 *          depths, each in 0 .. T - 1 (others are taken as the nearer end); NULL:
 *          i.  Only with a mask.
 * Pages no position of which is below sinks or above start[b] - window are not
 * read, and their table entries may hold anything.  For all else
 * spec_attention_cache4's words hold.
 * workspace: spec_attention_cache4_window_workspace bytes, 256-byte aligned. */
size_t spec_attention_cache4_window_workspace(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                              int32_t head_dim);
int spec_attention_cache4_window(spec_cache4_t cache, spec_heads_t q, int32_t B, int32_t T,
                                 int32_t q_heads, const int32_t* start, const int32_t* count,
                                 const uint32_t* mask, int64_t mask_seq_stride,
                                 int64_t mask_pos_stride, const int32_t* depth,
                                 int64_t depth_stride, int32_t window, int32_t sinks, float scale,
                                 spec_heads_t out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * spec_attention_cache4 behind shared prefixes.  Sequences fan g .. fan g +
 * fan - 1 (those below B) are branches of prefix g, whose prefix_len[g] tokens
 * stand in pages prefix_table[g][0 ..] of the same pool.  A new token sees its
 * whole prefix, and of its own sequence (start, count, mask, cache.table) what
 * spec_attention_cache4 says.  Either a prefix's pages are read and converted once
 * for each block of the rows of all its branches, or each branch reads them before
 * its own, where that costs less (short prefixes, few branches): the sizes and the
 * tables' widths decide, not prefix_len, so that tables serve best that are no
 * wider than need be.  The results of both differ by roundings within the bounds
 * of spec_attention_cache4.
 *   prefix_table  [ceil(B / fan)][prefix_cols], row g at + g * prefix_stride
 *   prefix_len    [ceil(B / fan)], 0 .. 64 prefix_cols; the rows i < count[b] of
 *                 branches whose prefix has a length outside, or a page outside
 *                 the pool, become NaN
 *   fan >= 1; min(fan, B) T q_heads at most 2^30
 * For all else spec_attention_cache4's words hold.
 * workspace: spec_attention_cache4_shared_workspace bytes, 256-byte aligned: by
 * these sizes alone, with room for a record of each row (4 head_dim + 16 bytes)
 * also where branches read their prefix themselves. */
size_t spec_attention_cache4_shared_workspace(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                              int32_t head_dim, int32_t fan);
int spec_attention_cache4_shared(spec_cache4_t cache, const int32_t* prefix_table,
                                 int64_t prefix_stride, int32_t prefix_cols,
                                 const int32_t* prefix_len, int32_t fan, spec_heads_t q, int32_t B,
                                 int32_t T, int32_t q_heads, const int32_t* start,
                                 const int32_t* count, const uint32_t* mask,
                                 int64_t mask_seq_stride, int64_t mask_pos_stride, float scale,
                                 spec_heads_t out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The pages of each sequence, from lengths that stand in device memory.
 *
 * Sequence b holds pages table[b][0 .. held[b] - 1]; free_pages[0 .. n - 1],
 * n = free_count[0], are nobody's.  The call brings every sequence to
 * w = ceil(need[b] / 64) pages:
 *   - pages behind w go back: all of them, in the order of (b, page), are put
 *     on the end of free_pages from the last to the first, and their entries
 *     become -1;
 *   - then missing pages are taken from the end of free_pages, in the order of
 *     (b, page), for one sequence after the other, until one finds too few:
 *     it and all after it that miss pages stay as they are.
 * held[b] and free_count[0] are brought up to date (held[b] < w tells a
 * sequence that was left out).  A second call with the former lengths undoes
 * the first, page for page.
 *   table       [B][table_cols], row b at table + b * table_stride
 *   free_pages  [free_capacity]
 * Data faults: a sequence with held[b] or w outside 0 .. table_cols, or need[b]
 * < 0, stays as it is; where free_count[0], or what it would be before the first
 * page is taken, lies outside 0 .. free_capacity, nothing is changed.
 * B at most 65536.
 * workspace: spec_cache4_reserve_workspace bytes, 256-byte aligned; where that
 * is 0 (B at most 128) there need be none. */
size_t spec_cache4_reserve_workspace(int32_t B);
int spec_cache4_reserve(int32_t* table, int64_t table_stride, int32_t table_cols, int32_t* held,
                        const int32_t* need, int32_t B, int32_t* free_pages,
                        int32_t free_capacity, int32_t* free_count, void* workspace,
                        size_t workspace_bytes, void* stream);

/* slots[b][i] = 64 table[b][x / 64] + x % 64, x = start[b] + i: where new token i
 * stands in a pool of n_pages pages; -1 for i >= count[b] (NULL: T), for a page
 * outside the pool, and for every token of an ill-formed sequence.
 *   slots [B][T] contiguous */
int spec_cache4_slots(const int32_t* table, int64_t table_stride, int32_t table_cols,
                      int32_t n_pages, int32_t B, int32_t T, const int32_t* start,
                      const int32_t* count, int64_t* slots, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPECVERIFY_STEP_H */
