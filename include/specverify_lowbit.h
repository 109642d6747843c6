/*
 * specverify_lowbit.h -- C ABI of libspecverify: the target's pass over the
 * candidates in few bits.
 *
 * The verify calls of specverify.h take the target's logits at every drafted
 * position.  Two operators of the pass that makes them depend on the
 * candidates: the attention of a sequence's new positions (the last accepted
 * token and its drafts, a chain or a candidate tree) over the cached keys and
 * values, whose tail the next step overwrites behind the accepted length, and
 * the LM head.  These calls hold the cache in 4 bits and the head in 8.
 *
 * Memory, streams and status codes are those of specverify.h: array arguments
 * are DEVICE pointers, the caller owns every buffer, a call only enqueues work
 * on `stream`.  One difference: a workspace of these calls is plain scratch.
 * It need not be cleared, its contents mean nothing between calls, and calls
 * that may overlap (other streams, captured graphs that may replay at the
 * same time) need one each.
 */
#ifndef SPECVERIFY_LOWBIT_H
#define SPECVERIFY_LOWBIT_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * A key/value cache in 4 bits: pages of SPEC_CACHE4_PAGE tokens from a pool.
 *
 * Format.  The D values of a token's key (value) in one kv head form D / 32
 * groups.  A group is held as 4-bit e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives, the OCP microscaling element) and one exponent byte e; code
 * c stands for c 2^(e-127).  2^(e-127) is the smallest power of two, at least
 * 2^-126 and at most 2^125, whose 6-fold holds the group's largest magnitude;
 * values round to the nearest code, ties to the even one, and what passes
 * 3 x 2^126, the largest such value that is finite in F32 and BF16, is held
 * as it.  A (token, head) whose key or value holds
 * a NaN or an infinity is held as NaN: every key exponent byte is 255 and all
 * codes are 0.
 *
 * A page's record of one kv head has 68 D bytes (t = token of the page):
 *   key codes        [64 t][D / 2], the even element in a byte's low half
 *   key exponents    [D / 32 groups][16][4], token t at [t % 16][t / 16]
 *   value codes      [4][4][16][4][D / 32], token t at [t / 16][t % 16 / 4][.]
 *                    [t % 4], the third axis over sixteenths of D
 *   value exponents  [4][4][D / 32 groups][4], token t at
 *                    [t / 16][t % 16 / 4][.][t % 4]
 * (the order in which the attention's matrix instructions take them).
 *
 * Positions.  Sequence b has start[b] cached tokens and count[b] new ones (T of
 * them where count is NULL) at positions start[b] .. start[b] + count[b] - 1;
 * position x lives in page table[b][x / 64].  Pages may be shared by sequences
 * as long as no call writes a position of theirs twice.
 *
 * Data faults.  A sequence is ill-formed when start[b] < 0, count[b] < 0,
 * count[b] > T or start[b] + count[b] > 64 table_cols; a position is ill-formed
 * when its page lies outside the pool.  Nothing is written for them, and what
 * is read of them is NaN. */
#define SPEC_CACHE4_PAGE 64

typedef struct {
  void* pages;           /* [n_pages][heads][68 head_dim] bytes, 16-byte aligned */
  const int32_t* table;  /* [B][table_cols], row b at table + b * table_stride */
  int64_t table_stride;  /* >= table_cols */
  int32_t n_pages;
  int32_t table_cols;
  int32_t heads;         /* kv heads, 1 .. SPEC_CACHE4_MAX_HEADS */
  int32_t head_dim;      /* 64, 128 or 256 */
} spec_cache4_t;
#define SPEC_CACHE4_MAX_HEADS 1024

/* Heads of positions: element (b, i, h, x) at
 *   data[b * seq_stride + i * pos_stride + h * head_stride + x]
 * (strides in elements).  data and the byte sizes of all strides are
 * multiples of 16; the stride of an axis of one step is not used.  Rows that a
 * call writes lie apart: with the axes in the order of their strides, each
 * steps over all that the ones before it cover. */
typedef struct {
  void* data;
  int32_t dtype; /* spec_dtype_t */
  int32_t reserved;
  int64_t seq_stride;
  int64_t pos_stride;
  int64_t head_stride;
} spec_heads_t;

/* Bytes of one page's record of one kv head: 68 head_dim (0 if unsupported). */
size_t spec_cache4_record_bytes(int32_t head_dim);

/* Quantises the new keys and values k, v [B][T][heads][head_dim] (F32 or BF16,
 * both the same) into the cache.  Tokens i >= count[b] are not read. */
int spec_cache4_write(spec_cache4_t cache, spec_heads_t k, spec_heads_t v, int32_t B, int32_t T,
                      const int32_t* start, const int32_t* count, void* stream);

/* Reads positions start[b] .. start[b] + count[b] - 1 back: the values the
 * codes stand for, as F32 or BF16 (exact in both) into k, v
 * [B][T][heads][head_dim].  Rows i >= count[b] are left as they were. */
int spec_cache4_read(spec_cache4_t cache, spec_heads_t k, spec_heads_t v, int32_t B, int32_t T,
                     const int32_t* start, const int32_t* count, void* stream);

/* Attention of the new positions over the cache:
 *   s(i, x) = scale sum_d q[b][i][h][d] K[x][h / (q_heads / heads)][d]
 *   out[b][i][h] = sum_x softmax_x(s(i, x)) V[x],  lse = log sum_x exp(s(i, x))
 * over the positions x that new token i sees: every x < start[b], and new
 * token j (position start[b] + j, j < count[b]) when bit j % 32 of
 * mask word j / 32 of row (b, i) is set, or, where mask is NULL, when j <= i.
 * The new tokens' own keys and values are written before the call.  A token
 * that sees nothing gets out = 0 and lse = -inf; one that sees a position held
 * as NaN, and every one of an ill-formed sequence or of one with an
 * ill-formed position below start[b] + count[b], gets NaN.
 *   q     [B][T][q_heads][head_dim] BF16
 *   mask  words [T][ceil(T / 32)] of sequence b at mask + b * mask_seq_stride,
 *         row i at + i * mask_pos_stride (words; seq stride 0 shares one mask)
 *   scale finite, > 0
 *   out   [B][T][q_heads][head_dim] BF16, rounded once; the products and the
 *         normaliser take the same probabilities, in BF16 relative to the
 *         running maximum, so that out is a weighted mean of the values seen;
 *         scores, sums and lse are F32: a row whose scores times scale log2 e,
 *         or whose sums of up to 2^8 |V| a position, pass its range gets no
 *         meaningful result, and no other row is touched
 *   lse   [B][T][q_heads] F32 or NULL
 * Rows i >= count[b] of out and lse are left as they were.
 * Limits: q_heads a multiple of heads, at most 16384; T <= SPEC_CACHE4_MAX_T;
 * B (table_cols + 8) heads ceil(T q_heads / heads / 16) below 2^40.
 * workspace: spec_attention_cache4_workspace bytes, 256-byte aligned. */
#define SPEC_CACHE4_MAX_T 256
size_t spec_attention_cache4_workspace(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                       int32_t head_dim);
int spec_attention_cache4(spec_cache4_t cache, spec_heads_t q, int32_t B, int32_t T,
                          int32_t q_heads, const int32_t* start, const int32_t* count,
                          const uint32_t* mask, int64_t mask_seq_stride, int64_t mask_pos_stride,
                          float scale, spec_heads_t out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The LM head in 8-bit floating point (OCP e4m3) with one scale per block of
 * 128.
 *
 * Quantises weight [V][d] (F32 or BF16, row v at v * weight_stride elements) to
 * q [V][d] (contiguous e4m3 bytes) and scale [ceil(V/128)][ceil(d/128)] F32: a
 * block's scale is the smallest power of two, at least 2^-126, whose 448-fold
 * holds its largest finite magnitude; values round to nearest, ties to even; a
 * NaN or an infinity becomes NaN.
 * 32 <= d <= 65536, a multiple of 32; rows 16-byte aligned. */
int spec_quantize_fp8(const void* weight, int32_t dtype, int64_t weight_stride, int32_t V,
                      int32_t d, void* q, float* scale, void* stream);

/* logits[b][j][v] = sum_c h8[b][j][c] weight[v][c] scale[v / 128][c / 128]
 * where h8 is the hidden row rounded to e4m3 in blocks of 128 with a
 * power-of-two scale each, by the rule of spec_quantize_fp8.
 *   hidden  [B][rows][d] F32 or BF16, strides in elements; rows 16-byte aligned
 *   weight  [V][d] e4m3, row v at v * weight_stride bytes (a multiple of 16, at
 *           most 2^22)
 *   scale   [ceil(V/128)][ceil(d/128)] F32, contiguous, any finite values whose
 *           products with the hidden rows' scales are in F32's range
 *   logits  [B][rows][V] F32 or BF16 (spec_logits_t addressing, written; its
 *           rows lie apart)
 * F32 logits, and BF16 ones of up to 16 rows (B rows) of d up to 8192, are sums
 * held in F32.  Other BF16 logits are summed by the 8-bit matrix instructions:
 * of each product of eight neighbouring columns (8 g .. 8 g + 7), what lies below
 * 2^-13 of the largest of the eight is dropped (a factor below e4m3's normal range
 * counts as 2^-6 there), so that a logit is off by the sum over all eights of
 * 7 x 2^-13 of their largest |h8 weight scale| at most.  For normal data that is
 * 1.5e-5 in the 2-norm, far below BF16's rounding; a logit that is much smaller
 * than its terms loses more by it than by its rounding.  Callers who need its F32
 * sum take F32 logits.
 * 1 <= rows <= 2 SPEC_MAX_K + 1; d as above.
 * workspace: spec_lmhead_fp8_workspace bytes, 256-byte aligned. */
size_t spec_lmhead_fp8_workspace(int32_t B, int32_t rows, int32_t d);
int spec_lmhead_fp8(spec_logits_t hidden, int32_t B, int32_t rows, int32_t d, const void* weight,
                    int64_t weight_stride, const float* scale, int32_t V, spec_logits_t logits,
                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPECVERIFY_LOWBIT_H */
