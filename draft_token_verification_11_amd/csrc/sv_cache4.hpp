// sv_cache4.hpp -- the 4-bit key/value cache: writing, reading back, and the
// attention of a sequence's new positions over it (gfx950, wave64).  The
// format of a page's record is stated in include/specverify_lowbit.h.
#pragma once

#include "sv_device.hpp"

namespace sv {

typedef __bf16 c4_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 c4_bf16x8 __attribute__((ext_vector_type(8)));
typedef float c4_f32x2 __attribute__((ext_vector_type(2)));
typedef float c4_f32x4 __attribute__((ext_vector_type(4)));

constexpr int kC4Page = 64;

// Byte offsets in a record of head dimension D (NG = D / 32 groups).
template <int D>
struct C4 {
  static constexpr int NG = D / 32;
  static constexpr int kRecord = 68 * D;
  static constexpr int kKeyExp = 32 * D;               // after 64 rows of D / 2
  static constexpr int kVal = kKeyExp + 64 * NG;
  static constexpr int kValExp = kVal + 32 * D;
};

// A value that every lane of a wave needs, read by the scalar unit, so that
// waiting for it is no wait for the vector loads under way.
__device__ __forceinline__ int32_t c4_scalar(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(p);
}

struct C4View {
  uint8_t* pages;
  const int32_t* table;
  int64_t table_stride;
  int32_t n_pages, table_cols, heads;

  // Whether `n` tokens from `s` on fit the sequence's table.
  __host__ __device__ __forceinline__ bool fits(int32_t s, int32_t n, int32_t T) const {
    return s >= 0 && n >= 0 && n <= T && (int64_t)s + n <= (int64_t)table_cols * kC4Page;
  }
  // The pool page of the sequence's page `p` (0 <= p < table_cols), or -1.
  __host__ __device__ __forceinline__ int32_t page(int64_t b, int32_t p) const {
    const int32_t x = table[b * table_stride + p];
    return (uint32_t)x < (uint32_t)n_pages ? x : -1;
  }
  template <int D>
  __host__ __device__ __forceinline__ uint8_t* record(int32_t page, int32_t h) const {
    return pages + ((int64_t)page * heads + h) * C4<D>::kRecord;
  }
};

struct C4Heads {
  void* data;
  int64_t seq, pos, head;  // strides in elements
};

// ---------------------------------------------------------------------------
// Writing and reading back.  A thread holds 8 values of a token's key and the
// same 8 of its value; D / 8 threads hold a token, a wave 512 / D tokens of
// one head whose positions start at a multiple of their number, so that the
// value codes of four tokens, which stand side by side in the record, leave
// the wave together.  Bound by memory: each value is read once and written
// once, and only the exponent bytes (1 of 17 stored) are scattered.  4 x 8,191
// tokens of 8 heads of 128, BF16 (170 MB in and out): written in 46 us (3.7 TB/s),
// read back in 29.7 us (5.7 TB/s); 4 x 4,095 tokens F32 35 and 29 us, heads of 256
// BF16 49 and 31; 64 x 6 tokens: 4 us each.  A wave over all four
// sixteens of a page, which stores key exponents as dwords, took 51 us.
struct C4MoveArgs {
  C4View cache;
  C4Heads k, v;
  const int32_t* start;
  const int32_t* count;  // or null: T
  int64_t waves;
  int32_t T, runs;       // runs: position runs of a wave's length a sequence may touch
};

__device__ __forceinline__ float c4_exp_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Exponent byte of a group with the largest magnitude `amax` (finite).  252 at
// most: 6 x 2^125 is the largest code times a power of two that fp32 and bf16
// hold (4 x 2^126 would be 2^128), and the conversion holds what lies past it
// as 6.
__device__ __forceinline__ uint32_t c4_exponent(float amax) {
  const int32_t e = (int32_t)((__float_as_uint(amax) + 0x3FFFFFu) >> 23) - 2;
  return (uint32_t)(e < 1 ? 1 : e > 252 ? 252 : e);
}

__device__ __forceinline__ uint32_t c4_pack8(const float* x, float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
}

// Where the thread's 8 value codes (elements 8u .. 8u + 7 of token t) stand:
// 4 bytes for D >= 128, two runs of 2 bytes 8 apart for D = 64.
template <int D>
__host__ __device__ __forceinline__ int c4_val_off(int t, int u) {
  constexpr int NG = C4<D>::NG;
  const int byte = 4 * u;
  return C4<D>::kVal + (t >> 2) * (2 * D) + (byte / NG) * (4 * NG) + (t & 3) * NG + byte % NG;
}

template <int D>
__host__ __device__ __forceinline__ int c4_key_exp_off(int t, int g) {
  return C4<D>::kKeyExp + g * 64 + (t & 15) * 4 + (t >> 4);
}
template <int D>
__host__ __device__ __forceinline__ int c4_val_exp_off(int t, int g) {
  return C4<D>::kValExp + (t >> 2) * (4 * C4<D>::NG) + g * 4 + (t & 3);
}

// The token of this thread: its sequence, head, index among the new tokens
// and position, or false if it has none (out of the call, or ill-formed).
struct C4Token {
  int64_t b;
  int32_t h, i, pos;
  bool live;  // belongs to a well-formed sequence's new tokens
};
template <int D>
__device__ __forceinline__ bool c4_token(const C4MoveArgs& A, int lane, C4Token& x) {
  constexpr int kTokens = 512 / D;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= A.waves) return false;
  x.h = (int32_t)(w % A.cache.heads);
  const int64_t r = w / A.cache.heads;
  x.b = r / A.runs;
  const int32_t s = A.start[x.b], n = A.count ? A.count[x.b] : A.T;
  const bool ok = A.cache.fits(s, n, A.T);
  // ill-formed: the tokens are named by their index alone, so that a reader
  // can mark them
  const int32_t s0 = ok ? s : 0, n0 = ok ? n : A.T;
  x.pos = (int32_t)(s0 / kTokens + r % A.runs) * kTokens + lane / (D / 8);
  x.i = x.pos - s0;
  x.live = ok;
  return x.i >= 0 && x.i < n0;
}

template <typename T, int D>
__global__ __launch_bounds__(256) void k_cache4_write(C4MoveArgs A) {
  const int lane = threadIdx.x & 63;
  constexpr int kLanes = D / 8;  // threads of a token
  C4Token x;
  bool have = c4_token<D>(A, lane, x) && x.live;
  int32_t page = -1;
  if (have) page = A.cache.page(x.b, x.pos / kC4Page);
  have = have && page >= 0;
  const int u = lane % kLanes;
  float kf[8] = {}, vf[8] = {};
  if (have) {
    const int64_t ko = x.b * A.k.seq + x.i * A.k.pos + x.h * A.k.head + 8 * u;
    const int64_t vo = x.b * A.v.seq + x.i * A.v.pos + x.h * A.v.head + 8 * u;
    load8<T, true>(reinterpret_cast<const T*>(A.k.data) + ko, 0, 8, kf);
    load8<T, true>(reinterpret_cast<const T*>(A.v.data) + vo, 0, 8, vf);
  }
  float ka = 0.f, va = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ka = fmaxf(ka, __builtin_fabsf(kf[e]));
    va = fmaxf(va, __builtin_fabsf(vf[e]));
    bad |= !__builtin_isfinite(kf[e]) || !__builtin_isfinite(vf[e]);
  }
  // a group is held by four neighbouring threads
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    ka = fmaxf(ka, __shfl_xor(ka, off));
    va = fmaxf(va, __shfl_xor(va, off));
  }
  const uint64_t mine = (kLanes == 64 ? ~0ull : ((1ull << kLanes) - 1)) << (lane / kLanes * kLanes);
  const bool nan = (__ballot(bad) & mine) != 0;
  if (!have) return;
  const uint32_t ke = nan ? 255u : c4_exponent(ka), ve = nan ? 1u : c4_exponent(va);
  const uint32_t kw = nan ? 0u : c4_pack8(kf, c4_exp_scale(ke));
  const uint32_t vw = nan ? 0u : c4_pack8(vf, c4_exp_scale(ve));
  uint8_t* rec = A.cache.record<D>(page, x.h);
  const int t = x.pos % kC4Page;
  *reinterpret_cast<uint32_t*>(rec + t * (D / 2) + 4 * u) = kw;
  uint8_t* vp = rec + c4_val_off<D>(t, u);
  if constexpr (D == 64) {
    *reinterpret_cast<uint16_t*>(vp) = (uint16_t)vw;
    *reinterpret_cast<uint16_t*>(vp + 4 * C4<D>::NG) = (uint16_t)(vw >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(vp) = vw;
  }
  if (u % 4 == 0) {
    rec[c4_key_exp_off<D>(t, u / 4)] = (uint8_t)ke;
    rec[c4_val_exp_off<D>(t, u / 4)] = (uint8_t)ve;
  }
}

__device__ __forceinline__ void c4_unpack8(uint32_t w, float scale, uint16_t* out) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  *reinterpret_cast<uint4*>(out) = r;
}
__device__ __forceinline__ void c4_unpack8(uint32_t w, float scale, float* out) {
  const c4_f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const c4_f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const c4_f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const c4_f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  *reinterpret_cast<float4*>(out) = make_float4(a[0], a[1], b[0], b[1]);
  *reinterpret_cast<float4*>(out + 4) = make_float4(c[0], c[1], d[0], d[1]);
}
__device__ __forceinline__ void c4_fill_nan(uint16_t* out) {
  *reinterpret_cast<uint4*>(out) = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
}
__device__ __forceinline__ void c4_fill_nan(float* out) {
  const float n = __builtin_nanf("");
  *reinterpret_cast<float4*>(out) = make_float4(n, n, n, n);
  *reinterpret_cast<float4*>(out + 4) = make_float4(n, n, n, n);
}

template <typename T, int D>
__global__ __launch_bounds__(256) void k_cache4_read(C4MoveArgs A) {
  const int lane = threadIdx.x & 63;
  constexpr int kLanes = D / 8;
  C4Token x;
  if (!c4_token<D>(A, lane, x)) return;
  const int u = lane % kLanes;
  T* ko = reinterpret_cast<T*>(A.k.data) + x.b * A.k.seq + x.i * A.k.pos + x.h * A.k.head + 8 * u;
  T* vo = reinterpret_cast<T*>(A.v.data) + x.b * A.v.seq + x.i * A.v.pos + x.h * A.v.head + 8 * u;
  const int32_t page = x.live ? A.cache.page(x.b, x.pos / kC4Page) : -1;
  if (page < 0) {
    c4_fill_nan(ko);
    c4_fill_nan(vo);
    return;
  }
  const uint8_t* rec = A.cache.record<D>(page, x.h);
  const int t = x.pos % kC4Page;
  const uint32_t kw = *reinterpret_cast<const uint32_t*>(rec + t * (D / 2) + 4 * u);
  const uint8_t* vp = rec + c4_val_off<D>(t, u);
  uint32_t vw;
  if constexpr (D == 64)
    vw = *reinterpret_cast<const uint16_t*>(vp) |
         ((uint32_t)*reinterpret_cast<const uint16_t*>(vp + 4 * C4<D>::NG) << 16);
  else
    vw = *reinterpret_cast<const uint32_t*>(vp);
  const uint32_t ke = rec[c4_key_exp_off<D>(t, u / 4)], ve = rec[c4_val_exp_off<D>(t, u / 4)];
  if (ke == 255u) {
    c4_fill_nan(ko);
    c4_fill_nan(vo);
    return;
  }
  c4_unpack8(kw, c4_exp_scale(ke), ko);
  c4_unpack8(vw, c4_exp_scale(ve), vo);
}

// ---------------------------------------------------------------------------
// Attention of the new positions over the cache.
//
// The T new tokens' query heads that share a kv head are the rows of one
// product: row r = i G + g (token i, head g of the G heads).  For a page of 64
// tokens a wave computes
//   S' = K Q'   (tokens x rows; K from its codes, converted to bf16 exactly)
//   P' = exp2(c S' - m), m the row's running maximum, c = scale log2 e
//   O' += V' P' (head dimension x rows)
// with v_mfma_f32_16x16x32_bf16, whose lane l holds A[l % 16][8 (l / 16) .. +8],
// Bt[l % 16][8 (l / 16) .. +8] and C[4 (l / 16) + r][l % 16].  The order of a
// product's inner index is free, and it is chosen so that no value changes
// lanes between the two products:
//   - S': inner index d; lane group q = l / 16 holds d = q D / 4 .. + D / 4, 8
//     at a time, a contiguous run of one token's key codes;
//   - a lane then holds S' of row l % 16 at tokens 16 tile + 4 q + 0..3, which
//     is the B operand of the second product if its inner index runs over
//     tokens 4 q .. 4 q + 3 of one tile and then of the next;
//   - V' has to come in that order: the record stores the values of tokens
//     4 q .. 4 q + 3 of a tile side by side for each sixteenth of D;
//   - a lane ends with O' of row l % 16 at d = q D / 4 .. + D / 4.
// Row statistics belong to a lane (and its three partners of the other lane
// groups), so rescaling O' by a new maximum is one factor per lane.  The
// maximum is raised only when a score passes it by 2^8 (P' stays below 2^8,
// far from any limit of bf16 or fp32), so most pages skip the rescaling.  P' is
// rounded to bf16 for the product (2^-8 relative at most, the size of the
// output's own rounding).  The normaliser sums the rounded values, so that the
// output is a weighted mean of what the row sees: values that agree come out as
// they are, and the rounding of a probability that outweighs all others cancels.
// The log-sum-exp takes the sum of the unrounded ones.  The second sum costs 1 to
// 6 % (64 x 6 rows 62.6 us, so 63.9; trees of 168 rows 86.9, so 90.0; 64 rows of
// heads of 64 39.3, so 41.6; summed by a matrix instruction 63.7, 89.4 and, spilled,
// 42.6).  P' as the sum of two bf16 would bring the error against 64 bits
// from 0.0017 to 0.0024 down to the output's own rounding, 0.0014 to 0.0017, in
// another half of the matrix instructions: 67.5, 107 and 46.4 us, and 131,003
// tokens x 36 rows 57.2 instead of 48.9.
//
// What bounds it (times of this kernel; where two times are compared elsewhere in
// this file, both are of the build that the choice was made in).
//   - Few rows, long sequences of one length: the cache's bytes (64 x 8 heads of
//     128, 24 rows over 4,090 tokens, 292 MB: 65 us, 4.5 TB/s).
//   - The same with ragged lengths: the ends of segments as well, about 5 us of a
//     workgroup each, and workgroups that end at different times (1,500 to 4,091
//     tokens, 201 MB: 58 us, 3.5 TB/s).
//   - Many rows: the vector unit, which converts and permutes a page's codes anew
//     for each block of rows, and the products that wait for it (16 x 8 heads, 168
//     rows over 37 to 8,155 tokens: 90 to 93 us; vector instructions in 57 % of the
//     busy cycles, matrix units in 28 %).
//   - One short sequence: a chain of loads that wait for each other (lengths, table,
//     pages) and few workgroups that go through its pages (777 tokens: 11 us, on 8 of
//     768; a launch that does less, such as the cache write's, takes under 4).
//   - Very many sequences: finding the shares, for which every wave reads all
//     lengths (65,536 sequences: 0.67 ms, without any page; 1,000: nothing that shows).
//
// Work split: the pages of all (sequence, kv head, block of rows) are laid end
// to end and cut into one equal range per workgroup, whatever the sequences'
// lengths; the four waves of a workgroup take the range's pages in turn.  A
// workgroup whose range cuts one of them leaves its rows' maximum, sum and
// unnormalised output in the workspace, and k_attention_cache4_join adds those
// up in order, so that results do not depend on the order of workgroups.
// Of the workgroups of a call (as many as are in flight at once, see C4Shape)
// those that its pages do not need end at once.
struct C4AttnArgs {
  C4View cache;
  const uint16_t* q;
  int64_t q_seq, q_pos, q_head;
  uint16_t* out;
  int64_t o_seq, o_pos, o_head;
  float* lse;             // [B][T][q_heads] or null
  const int32_t* start;
  const int32_t* count;   // or null: T
  const uint32_t* mask;   // or null: chain
  int64_t mask_seq, mask_pos;
  int32_t B, T, G, row_blocks;
  float c;                // scale log2 e
  int32_t split;          // 0: no segment is cut, and there is nothing to join
  struct C4Cut* cuts;     // [workgroups] the segment that a workgroup begins and others end
  float* parts;           // [2 x workgroups] records of a workgroup's first and last cut segment
};

struct C4Cut {
  int32_t b, hr, nnew;  // its sequence, head and block of rows, and the sequence's new tokens
  int32_t parts, slot;  // workgroups that hold it, from this one on (0: none); its record in this one
  int32_t pad[3];
};

// Pages of sequence b that its new tokens attend to; 0 when it has no rows.
// `bad`: ill-formed (one page then stands for the sequence, so that its rows
// are visited).
template <bool UNIFORM>
__device__ __forceinline__ int32_t c4_pages(const C4AttnArgs& A, int64_t b, bool& bad) {
  const int32_t s = UNIFORM ? c4_scalar(A.start + b) : A.start[b];
  const int32_t n = !A.count ? A.T : UNIFORM ? c4_scalar(A.count + b) : A.count[b];
  bad = !A.cache.fits(s, n, A.T);
  if (bad) return 1;
  return n == 0 ? 0 : (s + n + kC4Page - 1) / kC4Page;
}

// Beginning and ending a segment (its rows, the first loads, joining the four
// waves) costs a workgroup as much time as about this many pages; without it
// in the shares a batch with short sequences waits for the workgroups that
// hold many of them (16 sequences of 37 to 8,155 tokens, 8 heads of 128, 168 rows:
// 124 us at 3 pages, 93 at 6, 92 at 8, 94 at 12; 96 x 16 heads of 64 over 0 to 2,045,
// 48 rows: 85 at 6, 75 at 8; 7 x 8 heads over 5,000 to 9,000: 23.6 and 24.3).
constexpr int32_t kC4SegCost = 8;

// Weight of a segment of `pages`.
__device__ __forceinline__ int64_t c4_weight(int32_t pages) {
  return pages ? pages + kC4SegCost : 0;
}

// floor(x / y) for 0 <= x < 2^42, 0 < y < 2^42, from a reciprocal r of y good to
// 2^-14: two Newton steps bring it to 2^-51, so that the product is less than
// one off and its whole part at most one.  Shares and places among all
// segments pass 32 bits in large calls.
__host__ __device__ __forceinline__ int64_t c4_quotient(int64_t x, int64_t y, double r) {
  const double d = (double)y;
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  const int64_t q = (int64_t)((double)x * r), rest = x - q * y;
  return q - (rest < 0) + (rest >= y);
}
__device__ __forceinline__ int64_t c4_div(int64_t x, int64_t y) {
  return c4_quotient(x, y, __builtin_amdgcn_rcp((double)y));
}

// Sum over the lanes up to and with this one.
__device__ __forceinline__ int64_t c4_prefix(int64_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(x, off);
    if (lane >= off) x += o;
  }
  return x;
}
__device__ __forceinline__ int64_t c4_lane(int64_t x, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((int32_t)x, l);
  const uint32_t hi = __builtin_amdgcn_readlane((int32_t)(x >> 32), l);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Weight of all sequences' segments (of one head and row block): a lane sums a
// run of `per` sequences; `before`: the weight before its run.
__device__ __forceinline__ int64_t c4_plan(const C4AttnArgs& A, int lane, int32_t per, int64_t& before) {
  int64_t sum = 0;
  for (int32_t j = 0; j < per; ++j) {
    const int64_t b = (int64_t)lane * per + j;
    bool bad;
    if (b < A.B) sum += c4_weight(c4_pages<false>(A, b, bad));
  }
  const int64_t incl = c4_prefix(sum, lane);
  before = incl - sum;
  return c4_lane(incl, 63);
}
// The sequence in which weight x (below the total) lies, and the weight before
// it: the lane's run, then 64 sequences of it at a time.
__device__ __forceinline__ int64_t c4_find(const C4AttnArgs& A, int lane, int32_t per, int64_t before,
                                           int64_t x, int64_t& at) {
  const int run = 63 - __builtin_clzll(__ballot(before <= x));
  at = c4_lane(before, run);
  if (per == 1) return run;
  for (int64_t b0 = (int64_t)run * per;; b0 += 64) {
    const int64_t b = b0 + lane;
    bool bad;
    const int64_t wt = b < A.B ? c4_weight(c4_pages<false>(A, b, bad)) : 0;
    const int64_t incl = c4_prefix(wt, lane);
    const uint64_t past = __ballot(at + incl > x);
    if (past) {
      const int l = __builtin_ctzll(past);
      at += c4_lane(incl - wt, l);
      return b0 + l;
    }
    at += c4_lane(incl, 63);
  }
}

// The weight of each workgroup's range: an equal share, at least one page per
// wave and a segment's cost.
template <int GRID>
__device__ __forceinline__ int64_t c4_share(int64_t weight) {
  const int64_t s = (weight + GRID - 1) / GRID;
  return s < 4 + kC4SegCost ? 4 + kC4SegCost : s;
}
// Page of a segment of `pages` at which weight `x` from its begin lies.
__device__ __forceinline__ int32_t c4_cut(int64_t x, int32_t pages) {
  x -= kC4SegCost;
  return x <= 0 ? 0 : (x >= pages ? pages : (int32_t)x);
}

template <int D, int RT>
struct C4Rec {  // one cut segment: O [RT * 16][D], m, l and n [RT * 16]
  static constexpr int kRows = RT * 16;
  static constexpr int kFloats = kRows * (D + 3);
};

__device__ __forceinline__ float c4_max_quads(float x) {  // over the four lane groups
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float c4_sum_quads(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// s c - m, the product rounded as the maximum's is.
__device__ __forceinline__ float c4_scaled_less(float s, float c, float m) {
#pragma clang fp contract(off)
  const float x = s * c;
  return x - m;
}

constexpr float kC4Low = -3.402823466e38f;  // a maximum before any score: no finite one is below it
constexpr float kC4Raise = 8.0f;     // a score passes the maximum by 2^8 before it is raised
constexpr float kC4Exact = 0x1p24f;  // up to here half a step of a maximum is 1/2 at most

// What a row's new token sees of the 32 positions from `base` on (relative to
// start): bit x for position base + x.
__device__ __forceinline__ uint32_t c4_sees(const C4AttnArgs& A, int64_t b, int32_t i, int32_t n,
                                            int64_t base) {
  if (i >= n) return 0;
  if (!A.mask) {
    const int64_t seen = (int64_t)i + 1 - base;  // positions below base + seen
    return seen <= 0 ? 0 : (seen >= 32 ? ~0u : (1u << seen) - 1u);
  }
  const uint32_t* row = A.mask + b * A.mask_seq + i * A.mask_pos;
  const int32_t words = (A.T + 31) / 32;
  auto word = [&](int64_t k) -> uint32_t {
    if (k < 0) return ~0u;                // cached tokens
    if (k >= words) return 0;
    const int64_t left = n - 32 * k;      // new tokens of this word
    return left >= 32 ? row[k] : row[k] & (left <= 0 ? 0u : (1u << left) - 1u);
  };
  const int64_t k = base >> 5;            // floor: base may be negative
  const int sh = (int)(base & 31);
  return sh == 0 ? word(k) : (word(k) >> sh) | (word(k + 1) << (32 - sh));
}

typedef uint32_t C4U2 __attribute__((ext_vector_type(2)));
typedef uint32_t C4U4 __attribute__((ext_vector_type(4)));

// The codes and exponents of a pair of 16-token tiles in a lane's registers.
template <int D>
struct C4Unit {
  static constexpr int W = D / 32;    // dwords of codes per tile, keys and values each
  uint32_t k[2][W];                   // D / 4 elements of one token
  uint32_t v[2][W];                   // 4 tokens x D / 16 elements
  uint32_t ke[D == 256 ? 2 : 1];      // byte `tile`: this lane's token
  uint32_t ve[2];                     // byte j: token 4 q + j of the tile
};

__device__ __forceinline__ uint32_t c4_cvt(uint32_t w, float scale, int byte) {
  // the byte select is an immediate; `byte` is constant at every call
  switch (byte) {
    case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
}

// A conversion's scale operand with exponent byte `i` of w as its exponent
// field: 2^(e - 127), 255 for NaN.  The conversions take nothing but that
// field, so the other bytes may stand around it: one shift.
__device__ __forceinline__ float c4_byte_scale(uint32_t w, int i) {
  return __uint_as_float(i < 3 ? w << (23 - 8 * i) : w >> 1);
}

template <int D, int RT>
struct C4State {
  c4_f32x4 o[RT][D / 16];
  float m[RT], l[RT], n[RT];  // maximum, sum of P' and of P' rounded
  float less[RT];             // what a score's product is taken less: m, or 0 for rows that are far
  uint64_t far;               // lanes of rows whose maximum has passed kC4Exact
};

// Takes the keys, and the values, of pair `half` of a page out of its buffer, by
// instructions that the compiler does not know to read LDS: it would wait for
// every load under way at each, for along some branches it cannot tell which of
// them they need (131,003 tokens, 36 rows: 55.8 us, so 50.7).
template <int D>
__device__ __forceinline__ void c4_take_keys(const uint8_t* from, int half, int lane, C4Unit<D>& R) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)from;
  const uint32_t at4 = base + lane * 4;
  if constexpr (D == 64) {
    C4U2 k0, k1;
    asm volatile(
        "ds_read_b64 %0, %3\n\tds_read_b64 %1, %3 offset:512\n\tds_read_b32 %2, %4 offset:2048\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(k0), "=&v"(k1), "=&v"(R.ke[0])
        : "v"(base + (lane & 15) * 32 + (lane >> 4) * 8), "v"(at4)
        : "memory");
#pragma unroll
    for (int x = 0; x < 2; ++x) R.k[0][x] = k0[x], R.k[1][x] = k1[x];
  } else if constexpr (D == 128) {
    C4U4 k0, k1;
    asm volatile(
        "ds_read_b128 %0, %3\n\tds_read_b128 %1, %3 offset:1024\n\tds_read_b32 %2, %4 offset:4096\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(k0), "=&v"(k1), "=&v"(R.ke[0])
        : "v"(base + lane * 16), "v"(at4)
        : "memory");
#pragma unroll
    for (int x = 0; x < 4; ++x) R.k[0][x] = k0[x], R.k[1][x] = k1[x];
  } else {
    C4U4 k[4];
    asm volatile(
        "ds_read_b128 %0, %6\n\tds_read_b128 %1, %6 offset:1024\n\t"
        "ds_read_b128 %2, %6 offset:2048\n\tds_read_b128 %3, %6 offset:3072\n\t"
        "ds_read_b32 %4, %7 offset:8192\n\tds_read_b32 %5, %7 offset:8448\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(k[0]), "=&v"(k[1]), "=&v"(k[2]), "=&v"(k[3]), "=&v"(R.ke[0]), "=&v"(R.ke[1])
        : "v"(base + lane * 16), "v"(at4)
        : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 0; x < 8; ++x) R.k[i][x] = k[2 * i + x / 4][x % 4];
  }
#pragma unroll
  for (int x = 0; x < (D == 256 ? 2 : 1); ++x) R.ke[x] >>= 16 * half;
#endif
}
template <int D>
__device__ __forceinline__ void c4_take_values(const uint8_t* from, int lane, C4Unit<D>& R) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)from;
  const uint32_t at4 = base + lane * 4;
  if constexpr (D == 64) {
    C4U2 v0, v1;
    asm volatile(
        "ds_read_b64 %0, %4 offset:1024\n\tds_read_b64 %1, %4 offset:1536\n\t"
        "ds_read_b32 %2, %5 offset:2304\n\tds_read_b32 %3, %5 offset:2560\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(R.ve[0]), "=&v"(R.ve[1])
        : "v"(base + lane * 8), "v"(at4)
        : "memory");
#pragma unroll
    for (int x = 0; x < 2; ++x) R.v[0][x] = v0[x], R.v[1][x] = v1[x];
  } else if constexpr (D == 128) {
    C4U4 v0, v1;
    asm volatile(
        "ds_read_b128 %0, %4 offset:2048\n\tds_read_b128 %1, %4 offset:3072\n\t"
        "ds_read_b32 %2, %5 offset:4352\n\tds_read_b32 %3, %5 offset:4608\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v0), "=&v"(v1), "=&v"(R.ve[0]), "=&v"(R.ve[1])
        : "v"(base + lane * 16), "v"(at4)
        : "memory");
#pragma unroll
    for (int x = 0; x < 4; ++x) R.v[0][x] = v0[x], R.v[1][x] = v1[x];
  } else {
    C4U4 v[4];
    asm volatile(
        "ds_read_b128 %0, %6 offset:4096\n\tds_read_b128 %1, %6 offset:5120\n\t"
        "ds_read_b128 %2, %6 offset:6144\n\tds_read_b128 %3, %6 offset:7168\n\t"
        "ds_read_b32 %4, %7 offset:8704\n\tds_read_b32 %5, %7 offset:8960\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(R.ve[0]), "=&v"(R.ve[1])
        : "v"(base + lane * 16), "v"(at4)
        : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 0; x < 8; ++x) R.v[i][x] = v[2 * i + x / 4][x % 4];
  }
#endif
}

// One pair of tiles, from its buffer.  masked (of the wave): some of its 32 positions are not
// seen by some row; sees[] then has this lane's rows' bits, and `valid` those
// of the positions that hold tokens.  rows_of(j, qf): part j of the rows' operand.
template <int D, int RT, typename Q>
__device__ __forceinline__ void c4_unit(const uint8_t* from, int half, Q rows_of, C4State<D, RT>& S, float c, int lane,
                                        bool masked, const uint32_t (&sees)[RT], uint32_t valid) {
  const int q = lane >> 4;
  C4Unit<D> R;
  c4_take_keys<D>(from, half, lane, R);
  c4_f32x4 s[RT][2];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 2; ++i) s[rt][i] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    c4_bf16x8 kf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sc = c4_byte_scale(R.ke[D == 256 ? j / 4 : 0], i);
      uint4 a;
      a.x = c4_cvt(R.k[i][j], sc, 0);
      a.y = c4_cvt(R.k[i][j], sc, 1);
      a.z = c4_cvt(R.k[i][j], sc, 2);
      a.w = c4_cvt(R.k[i][j], sc, 3);
      kf[i] = __builtin_bit_cast(c4_bf16x8, a);
    }
    c4_bf16x8 qf[RT];
    rows_of(j, qf);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        s[rt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i], qf[rt], s[rt][i], 0, 0, 0);
  }
  c4_take_values<D>(from, lane, R);
  if (masked) {  // what stands past the last token is not a value: zeros with an exponent of 1
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!((valid >> (16 * i + 4 * q + j)) & 1)) {
          R.ve[i] = (R.ve[i] & ~(0xFFu << (8 * j))) | (127u << (8 * j));
#pragma unroll
          for (int x = 0; x < (D + 127) / 128; ++x) {
            // token j's D / 32 bytes of this lane's codes
            if constexpr (D == 64) R.v[i][j / 2] &= j % 2 ? 0xFFFFu : 0xFFFF0000u;
            else R.v[i][D / 128 * j + x] = 0u;
          }
        }
  }
  c4_bf16x8 p[RT];  // P' of the pair, the second product's operand
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (masked) {
      const uint32_t mine = sees[rt] >> (4 * q);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!((mine >> (16 * i + r)) & 1)) s[rt][i][r] = -__builtin_inff();
    }
    float top = fmaxf(fmaxf(s[rt][0][0], s[rt][0][1]), fmaxf(s[rt][0][2], s[rt][0][3]));
#pragma unroll
    for (int r = 0; r < 4; ++r) top = fmaxf(top, s[rt][1][r]);
    // rare, but for a wave with far rows; the lanes of a row agree on it here
    if (__ballot(top * c > S.less[rt] + kC4Raise) | S.far) {
      const float m = fmaxf(S.m[rt], c4_max_quads(top) * c);
      const float f = __builtin_amdgcn_exp2f(S.m[rt] - m);
      S.m[rt] = S.less[rt] = m;
      S.l[rt] *= f;
      S.n[rt] *= f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) S.o[rt][i] *= f;
      // Below, the exact product less the maximum, which is a rounded one: where
      // scores are equal, off by half a step of the maximum, which P' and its sums
      // have in common.  For far rows that would leave their range: they round the
      // products as they did the maximum.
      const bool far = __builtin_fabsf(m) > kC4Exact && m > kC4Low;
      S.far |= __ballot(far);
      if (far) {
        const float back = 1.0f / c;  // c is above 2^-104 where a row is far
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[rt][i][r] = c4_scaled_less(s[rt][i][r], c, m) * back;
        S.less[rt] = 0.f;
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][i][r], c, -S.less[rt]));
        sum += e;
        p[rt][4 * i + r] = (__bf16)e;
      }
    S.l[rt] += sum;
    constexpr c4_bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
    for (int r = 0; r < 8; r += 2)
      S.n[rt] = __builtin_amdgcn_fdot2_f32_bf16(c4_bf16x2{p[rt][r], p[rt][r + 1]}, one, S.n[rt], false);
  }
  // V' of the pair: byte y of token j's codes gives that token's values of two
  // neighbouring d; tokens are paired for each d by a byte permutation
  constexpr int NB = D / 32;  // bytes of a lane's codes of one token
  float sc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sc[i][j] = c4_byte_scale(R.ve[i], j);
#pragma unroll
  for (int y = 0; y < NB; ++y) {
    uint32_t a[2][4];  // [tile][token]: bf16 of d = 2 y, 2 y + 1
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[i][j] = c4_cvt(R.v[i][(j * NB + y) / 4], sc[i][j], (j * NB + y) % 4);
      }
    uint4 lo, hi;
    lo.x = __builtin_amdgcn_perm(a[0][1], a[0][0], 0x05040100u);
    lo.y = __builtin_amdgcn_perm(a[0][3], a[0][2], 0x05040100u);
    lo.z = __builtin_amdgcn_perm(a[1][1], a[1][0], 0x05040100u);
    lo.w = __builtin_amdgcn_perm(a[1][3], a[1][2], 0x05040100u);
    hi.x = __builtin_amdgcn_perm(a[0][1], a[0][0], 0x07060302u);
    hi.y = __builtin_amdgcn_perm(a[0][3], a[0][2], 0x07060302u);
    hi.z = __builtin_amdgcn_perm(a[1][1], a[1][0], 0x07060302u);
    hi.w = __builtin_amdgcn_perm(a[1][3], a[1][2], 0x07060302u);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      S.o[rt][2 * y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(c4_bf16x8, lo), p[rt], S.o[rt][2 * y], 0, 0, 0);
      S.o[rt][2 * y + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(c4_bf16x8, hi), p[rt], S.o[rt][2 * y + 1], 0, 0, 0);
    }
  }
}

// Writes N values of a finished row, normalised, or NaN; with the first ones
// the row's lse.
template <int N>
__device__ __forceinline__ void c4_finish(const C4AttnArgs& A, int64_t b, int32_t i, int32_t head,
                                          int d0, const float* x, float m, float l, float n) {
  const float inv = n == 0.f ? 0.f : 1.0f / n;  // a NaN sum stays NaN
  typedef __bf16 Out __attribute__((ext_vector_type(N)));
  Out y;
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = (__bf16)(x[e] * inv);
  *reinterpret_cast<Out*>(A.out + b * A.o_seq + i * A.o_pos + head * A.o_head + d0) = y;
  if (d0 == 0 && A.lse) {
    constexpr float kLn2 = 0.6931471805599453f;
    const int64_t at = (b * A.T + i) * ((int64_t)A.G * A.cache.heads) + head;
    A.lse[at] = l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// How the cached pages come: each wave fills two LDS buffers of its own with
// pairs of tiles, straight from memory (buffer_load ... lds), and takes them out
// in the order it put them in.  Nothing is shared, so the only wait is the
// wave's own, and what is on its way costs no registers, which belong to the
// accumulators.  A buffer holds kPairs pairs of 4.75 KiB (at D = 128): with 8
// waves a CU 70 KiB or more are in flight, while the code of a pair, which the
// instruction cache has to bring at every launch, stands twice and no more.
template <int D, int RT>
struct C4Shape {
  // whether the rows' operand stays in registers (else LDS, read per pair)
  static constexpr bool kQRegs = D * RT <= 256;
  static_assert(kQRegs || (D == 128 && RT == 3), "what c4_take_rows reads");
  // Waves a SIMD, or workgroups a compute unit: as many as registers and LDS
  // hold, for a wave waits much on itself (scores, exponentials, their sum and
  // the second product follow each other).  Three where 168 registers do without
  // spills: 96 x 16 heads of 64, 5 rows over 0 to 2,045 tokens 41 us with two,
  // 36 with three; 25 rows 58 and 46; 64 x 8 heads of 128 in tiles of 16 rows 84
  // and 70 (32 rows a tile: 62 and, 11 registers spilled, 66).  Workgroups of a
  // call: that many for each of 256 compute units.
  static constexpr int kWaves = D * RT <= 128 ? 3 : 2;
  static constexpr int kGrid = 256 * kWaves;
  static constexpr int kPairs = D == 64 || (D == 128 && RT == 2) ? 2 : 1;
  static_assert(kPairs <= 2, "as many waits");
  static constexpr int kCodes = 2 * 16 * D / 2;        // bytes of a pair's keys, or values
  static constexpr int kKeyExps = (D == 256 ? 2 : 1) * 256;
  static constexpr int kUnit = 2 * kCodes + kKeyExps + 512;
  static constexpr int kBuf = kPairs * kUnit;           // a wave's part of a buffer
  // memory instructions of a pair
  static constexpr int kLoads = 2 * kCodes / 1024 + kKeyExps / 256 + 2;
};

// Starts the loads of pair `half` of the record into `to`.
template <int D>
__device__ __forceinline__ void c4_fetch(const uint8_t* rec, int half, int lane, uint8_t* to) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host's pass does not know the buffer resource's type
  constexpr int NG = C4<D>::NG, kCodes = 16 * D;
  typedef __attribute__((address_space(3))) void* Lds;
  const int n = lane & 15, q = lane >> 4;
  const auto src = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(rec), 0, C4<D>::kRecord, 0x00020000);
  // D = 64: as the bytes stand; else 16 bytes a lane, the ones it will take
  const int ko = D == 64 ? lane * 16 : n * (D / 2) + q * (D / 8);
  const int vo = C4<D>::kVal + (D == 64 ? lane * 16 : lane * (D / 8));
  constexpr int kTiles = D == 64 ? 1 : 2, kParts = D == 256 ? 2 : 1;
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
      const int at = (i * kParts + x) * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (Lds)(to + at), 16, ko, (2 * half + i) * (8 * D) + 16 * x, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (Lds)(to + kCodes + at), 16, vo,
                                               (2 * half + i) * (8 * D) + 16 * x, 0, 0);
    }
  uint8_t* ex = to + 2 * kCodes;
#pragma unroll
  for (int x = 0; x < kParts; ++x)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (Lds)(ex + 256 * x), 4,
                                             C4<D>::kKeyExp + (q * NG / 4) * 64 + n * 4, 64 * x, 0, 0);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (Lds)(ex + 256 * (kParts + i)), 4,
                                             C4<D>::kValExp + q * (4 * NG) + (n * NG / 16) * 4,
                                             (2 * half + i) * (16 * NG), 0, 0);
#endif
}

// Takes part j of the rows' operand, at p and two further tiles of 4 KiB, in the
// same way.
__device__ __forceinline__ void c4_take_rows(const uint4* p, c4_bf16x8 (&qf)[3]) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("ds_read_b128 %0, %3\n\tds_read_b128 %1, %3 offset:4096\n\tds_read_b128 %2, %3 offset:8192\n\t"
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(qf[0]), "=&v"(qf[1]), "=&v"(qf[2])
               : "v"((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint4*)p)
               : "memory");
#endif
}

// Waits until at most n vector memory operations are under way.
template <int N>
__device__ __forceinline__ void c4_wait() {
  static_assert(N < 64, "six bits");
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4 | 15 << 8);  // the other counters as they are
#endif
}

template <int D, int RT>
__global__ __launch_bounds__(256, (C4Shape<D, RT>::kWaves)) void k_attention_cache4(C4AttnArgs A) {
  using Sh = C4Shape<D, RT>;
  constexpr int kRows = RT * 16, N = Sh::kPairs;
  // Two arrays, each named where it is used, so that the compiler does not wait
  // for the other's loads when it reads one.
  __shared__ __attribute__((aligned(16))) uint8_t ring0[4 * Sh::kBuf], ring1[4 * Sh::kBuf];
  __shared__ uint4 qs[Sh::kQRegs ? 1 : RT][Sh::kQRegs ? 1 : D / 32][Sh::kQRegs ? 1 : 64];
  __shared__ float ms[4][kRows], ls[4][kRows], ns[4][kRows];
  // After a segment the buffers hold O of 16 rows x kCols columns of each wave, in turn.
  constexpr int kCols = D == 64 ? 64 : N == 2 ? 128 : 64, kPad = kCols + 4, kRun = kCols / 16;
  static_assert(4 * 16 * kPad * 4 <= sizeof(ring0), "room");

  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, q = lane >> 4;
  // every wave for itself: no barrier before the first loads
  const int32_t per = (A.B + 63) / 64;
  const int32_t HR = A.cache.heads * A.row_blocks;
  int64_t before;
  const int64_t all = c4_plan(A, lane, per, before) * HR;  // weight of all segments
  const int64_t share = c4_share<Sh::kGrid>(all);
  const int64_t lo = (int64_t)blockIdx.x * share;
  const int64_t hi = min(lo + share, all);
  int32_t cut_b = 0, cut_hr = 0, cut_new = 0, cut_parts = 0, cut_slot = 0;
  auto note = [&] {
    if (A.split && tid == 0) A.cuts[blockIdx.x] = {cut_b, cut_hr, cut_new, cut_parts, cut_slot, {0, 0, 0}};
  };
  if (lo >= hi) {
    note();
    return;
  }

  // the segment of weight `lo`: its sequence, then its head and block of rows
  int64_t seq_at;
  int64_t b = c4_find(A, lane, per, before, c4_div(lo, HR), seq_at);
  bool bad;
  int32_t pages = c4_pages<true>(A, b, bad);
  int32_t hr = (int32_t)c4_div(lo - seq_at * HR, c4_weight(pages));
  int64_t seg = seq_at * HR + hr * c4_weight(pages);  // where it begins
  const int32_t R = A.T * A.G;
  for (; seg < hi; seg += c4_weight(pages), ++hr) {
    if (hr == HR) {  // the next sequence with pages (seg is its begin)
      do pages = c4_pages<true>(A, ++b, bad);
      while (pages == 0);
      hr = 0;
    }
    int32_t p0 = c4_cut(lo - seg, pages), p1 = c4_cut(hi - seg, pages);
    if (!A.split) p0 = 0, p1 = seg < lo ? 0 : pages;  // whole, where it begins
    if (p0 == p1) continue;  // its pages are another workgroup's
    const int32_t h = hr / A.row_blocks, r0 = hr % A.row_blocks * kRows;
    const int32_t s0 = c4_scalar(A.start + b);
    const int32_t nnew = bad || !A.count ? A.T : c4_scalar(A.count + b);
    if (p0 == 0 && p1 < pages) {
      cut_b = (int32_t)b, cut_hr = hr, cut_new = nnew, cut_slot = seg > lo ? 1 : 0;
      cut_parts = (int32_t)c4_div(seg + kC4SegCost + pages - 1, share) - blockIdx.x + 1;
    }

    // The waves take the segment's pairs of tiles in turn, so that a wave's are
    // all first or all second ones of their pages.  A page outside the pool
    // stands for page 0 and marks the rows.
    bool faulty = bad;
    const int half = w & 1;
    const int32_t end = bad ? p0 : p1, pw = p0 + (w >> 1);  // this wave's pages: pw, pw + 2, ..
    int32_t nu = end > pw ? (end - pw + 1) / 2 : 0;
    // the last page may hold no token in its second half
    if (nu && (pw + 2 * (nu - 1)) * (int64_t)kC4Page + 32 * half >= (int64_t)s0 + nnew) --nu;
    auto page_of = [&](int32_t u) { return u < nu ? c4_scalar(A.cache.table + b * A.cache.table_stride + pw + 2 * u) : 0; };
    auto fetch = [&](int32_t page, uint8_t* buf, int k) {
      if ((uint32_t)page >= (uint32_t)A.cache.n_pages) {
        faulty = true;
        page = 0;
      }
      c4_fetch<D>(A.cache.record<D>(page, h), half, lane, buf + w * Sh::kBuf + k * Sh::kUnit);
    };
    int32_t first[2 * N];  // all on their way before the first is needed
#pragma unroll
    for (int k = 0; k < 2 * N; ++k) first[k] = page_of(k);

    // The rows' operand, all on its way at once, before the first pairs.
    constexpr int kQ = Sh::kQRegs ? D / 32 : D / 128;  // chunks a wave loads of a tile
    uint4 qx[RT][kQ];
    int32_t tok[RT];  // this lane's rows' tokens; T past the last row
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int32_t r = r0 + 16 * rt + n16;
      const int32_t i = r / A.G, g = r - i * A.G;
      tok[rt] = r < R ? i : A.T;
      const uint16_t* qp = A.q + b * A.q_seq + i * A.q_pos + ((int64_t)h * A.G + g) * A.q_head;
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        qx[rt][j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < R && i < nnew) qx[rt][j] = load16(qp + q * (D / 4) + 8 * (Sh::kQRegs ? j : 4 * j + w));
      }
    }
    // Waited for here, by an instruction that the compiler knows: at their first use,
    // among the pairs, its wait would be for those too (64 x 8 heads of 128, 24 rows:
    // 66.0 us, so 62.8).  Heads of 64 do better with the pairs sooner under way (96 x
    // 16 heads, 60 rows: 109 us, so 105).
    if constexpr (D > 64) c4_wait<0>();
#pragma unroll
    for (int k = 0; k < 2 * N; ++k)
      if (k < nu) fetch(first[k], k < N ? ring0 : ring1, k % N);
    int32_t ahead = page_of(2 * N);  // the page of the next fetch
    if constexpr (!Sh::kQRegs) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < kQ; ++j) qs[rt][4 * j + w][lane] = qx[rt][j];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // __syncthreads would wait for the pairs too
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    auto rows_of = [&](int j, c4_bf16x8(&qf)[RT]) {
      if constexpr (Sh::kQRegs) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) qf[rt] = __builtin_bit_cast(c4_bf16x8, qx[rt][j]);
      } else {
        c4_take_rows(&qs[0][j][lane], qf);
      }
    };
    C4State<D, RT> S;
    S.far = 0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      S.m[rt] = S.less[rt] = kC4Low;
      S.l[rt] = S.n[rt] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) S.o[rt][i] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // the pairs u .. u + N - 1 of one buffer
    auto work = [&](int32_t u, uint8_t* buf) {
#pragma unroll 1
      for (int k = 0; k < N; ++k, ++u) {
        if (u >= nu) return;
        // this pair has arrived when no more than the later ones' loads are left
        // (loads return in order)
        const int32_t later = nu - 1 - u;
        if (later >= 2 * N - 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((2 * N - 1) * Sh::kLoads) : "memory");
        else if (N == 2 && later == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * Sh::kLoads) : "memory");
        else if (N == 2 && later == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Sh::kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        // the first of its positions relative to the new tokens'
        const int64_t base = (int64_t)(pw + 2 * u) * kC4Page + 32 * half - s0;
        const bool masked = base + 32 > 0;
        uint32_t sees[RT] = {}, valid = 0;
        if (masked) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) sees[rt] = c4_sees(A, b, tok[rt], nnew, base);
          const int64_t have = nnew - base;
          valid = have >= 32 ? ~0u : (1u << have) - 1u;
        }
        c4_unit<D, RT>(buf + w * Sh::kBuf + k * Sh::kUnit, half, rows_of, S, A.c, lane, masked, sees, valid);
        if (u + 2 * N < nu) {
          fetch(ahead, buf, k);
          ahead = page_of(u + 2 * N + 1);
        }
      }
    };
    for (int32_t u = 0; u < nu; u += 2 * N) {
      work(u, ring0);
      work(u + N, ring1);
    }
    if (faulty) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S.l[rt] = S.n[rt] = __builtin_nanf("");
    }
    // The four waves' rows together, a tile of 16 rows x kCols columns at a
    // time: column group 4 q + y of a lane holds D / 16 columns, of which a run
    // of kRun goes each time.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float l = c4_sum_quads(S.l[rt]), n = c4_sum_quads(S.n[rt]);
      if (q == 0) {
        ms[w][16 * rt + n16] = S.m[rt];
        ls[w][16 * rt + n16] = l;
        ns[w][16 * rt + n16] = n;
      }
    }
    __syncthreads();  // also: every wave has emptied its buffers
    const bool whole = p0 == 0 && p1 == pages;
    float* part = A.parts + ((int64_t)blockIdx.x * 2 + (seg > lo ? 1 : 0)) * C4Rec<D, RT>::kFloats;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int mine = 16 * rt + n16;
      const float f = __builtin_amdgcn_exp2f(
          S.m[rt] - fmaxf(fmaxf(ms[0][mine], ms[1][mine]), fmaxf(ms[2][mine], ms[3][mine])));
      const int rr = tid >> 4, row = 16 * rt + rr;  // this thread's row of the sums
      const float top = fmaxf(fmaxf(ms[0][row], ms[1][row]), fmaxf(ms[2][row], ms[3][row]));
      float l = 0.f, n = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float g = __builtin_amdgcn_exp2f(ms[x][row] - top);
        l += ls[x][row] * g;
        n += ns[x][row] * g;
      }
      const int32_t r = r0 + row, i = r / A.G, head = h * A.G + (r - i * A.G);
      const bool live = r < R && i < nnew;
#pragma unroll
      for (int x = 0; x < D / kCols; ++x) {
        // the buffers in turn: one barrier a time
        float* const oacc = reinterpret_cast<float*>((rt * (D / kCols) + x) & 1 ? ring1 : ring0);
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int e = 0; e < kRun; e += 4)
            *reinterpret_cast<float4*>(&oacc[(w * 16 + n16) * kPad + (4 * q + y) * kRun + e]) =
                make_float4(S.o[rt][x * kRun + e][y] * f, S.o[rt][x * kRun + e + 1][y] * f,
                            S.o[rt][x * kRun + e + 2][y] * f, S.o[rt][x * kRun + e + 3][y] * f);
        __syncthreads();
        const int grp = tid & 15, d0 = grp * (D / 16) + x * kRun;
        float v[kRun] = {};
#pragma unroll
        for (int ww = 0; ww < 4; ++ww)
#pragma unroll
          for (int e = 0; e < kRun; ++e) v[e] += oacc[(ww * 16 + rr) * kPad + grp * kRun + e];
        if (!live) continue;
        if (whole) {
          c4_finish<kRun>(A, b, i, head, d0, v, top, l, n);
        } else {
#pragma unroll
          for (int e = 0; e < kRun; ++e) part[row * D + d0 + e] = v[e];
          if (d0 == 0) {
            part[kRows * D + row] = top;
            part[kRows * D + kRows + row] = l;
            part[kRows * D + 2 * kRows + row] = n;
          }
        }
      }
    }
    __syncthreads();  // the buffers, ms, ls and ns are free
  }
  note();
}

// Sums the records x0 .. x1 - 1 of a row, eight of them under way at a time.
template <int D>
__device__ __forceinline__ void c4_gather(const float* first, const float* rest, int64_t floats, int rows,
                                          int row, int32_t x0, int32_t x1, int lane, float& m, float& l,
                                          float& n, float (&v)[D / 64]) {
  constexpr int E = D / 64, N = 8;
  m = kC4Low;
  l = n = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.f;
  for (int32_t base = x0; base < x1; base += N) {
    float pm[N], pl[N], pn[N], o[N][E];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int32_t x = min(base + k, x1 - 1);
      const float* p = x == 0 ? first : rest + x * floats;
      pm[k] = p[rows * D + row];
      pl[k] = p[rows * D + rows + row];
      pn[k] = p[rows * D + 2 * rows + row];
#pragma unroll
      for (int e = 0; e < E; ++e) o[k][e] = p[row * D + lane * E + e];
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (base + k < x1) {
        const float top = fmaxf(m, pm[k]);
        const float f = __builtin_amdgcn_exp2f(m - top), g = __builtin_amdgcn_exp2f(pm[k] - top);
        m = top;
        l = l * f + pl[k] * g;
        n = n * f + pn[k] * g;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] * f + o[k][e] * g;
      }
  }
}

// Joins the cut segments of calls with many of them, of few records each: four
// rows a workgroup, a wave each, for the segment that workgroup blockIdx.x of
// the attention began, if others end it.
template <int D, int RT>
__global__ __launch_bounds__(256) void k_attention_cache4_join(C4AttnArgs A) {
  constexpr int kRows = RT * 16, E = D / 64;  // E columns a lane
  constexpr int64_t kFloats = C4Rec<D, RT>::kFloats;
  const auto* cp = A.cuts + blockIdx.x;
  const int32_t parts = c4_scalar(&cp->parts);
  if (parts == 0) return;
  const int32_t b = c4_scalar(&cp->b), hr = c4_scalar(&cp->hr), slot = c4_scalar(&cp->slot);
  const int32_t nnew = c4_scalar(&cp->nnew);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t row = blockIdx.y * 4 + w, h = hr / A.row_blocks;
  const int32_t r = hr % A.row_blocks * kRows + row, i = r / A.G;
  if (r >= A.T * A.G || i >= nnew) return;
  const float* rest = A.parts + (int64_t)blockIdx.x * 2 * kFloats;
  float m, l, n, v[E];
  c4_gather<D>(rest + slot * kFloats, rest, 2 * kFloats, kRows, row, 0, parts, lane, m, l, n, v);
  c4_finish<E>(A, b, i, h * A.G + (r - i * A.G), lane * E, v, m, l, n);
}

// Joins those of calls with few segments of many records: a row a workgroup, a
// quarter of the records a wave.  Where the records stand follows from the
// lengths alone, as in the attention.
template <int D, int RT>
__global__ __launch_bounds__(256) void k_attention_cache4_join_long(C4AttnArgs A) {
  constexpr int kRows = RT * 16, E = D / 64;
  constexpr int64_t kFloats = C4Rec<D, RT>::kFloats;
  __shared__ float vs[4][D], ms[4], ls[4], ns[4];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t per = (A.B + 63) / 64, HR = A.cache.heads * A.row_blocks;
  const int32_t b = blockIdx.x / HR, hr = blockIdx.x % HR, row = blockIdx.y;
  const int32_t h = hr / A.row_blocks, r = hr % A.row_blocks * kRows + row, i = r / A.G;
  int64_t before;
  const int64_t share = c4_share<C4Shape<D, RT>::kGrid>(c4_plan(A, lane, per, before) * HR);
  bool bad;
  int64_t at = c4_lane(before, b / per);
  for (int32_t x = b / per * per; x < b; ++x) at += c4_weight(c4_pages<true>(A, x, bad));
  const int32_t pages = c4_pages<true>(A, b, bad);
  const int32_t nnew = bad || !A.count ? A.T : c4_scalar(A.count + b);
  if (pages == 0 || r >= A.T * A.G || i >= nnew) return;
  const int64_t seg = at * HR + hr * c4_weight(pages);
  // the workgroups that hold its first and last page
  const int32_t w0 = (int32_t)c4_div(seg + kC4SegCost, share);
  const int32_t parts = (int32_t)c4_div(seg + kC4SegCost + pages - 1, share) - w0 + 1;
  if (parts == 1) return;  // written whole
  const float* rest = A.parts + (int64_t)w0 * 2 * kFloats;
  const float* first = rest + (seg > w0 * share ? kFloats : 0);
  float m, l, n, v[E];
  const int32_t quarter = (parts + 3) / 4;
  c4_gather<D>(first, rest, 2 * kFloats, kRows, row, w * quarter, min(parts, w * quarter + quarter), lane, m, l, n, v);
#pragma unroll
  for (int e = 0; e < E; ++e) vs[w][lane * E + e] = v[e];
  if (lane == 0) {
    ms[w] = m;
    ls[w] = l;
    ns[w] = n;
  }
  __syncthreads();
  if (w) return;
  m = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
  l = n = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const float f = __builtin_amdgcn_exp2f(ms[x] - m);
    l += ls[x] * f;
    n += ns[x] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += vs[x][lane * E + e] * f;
  }
  c4_finish<E>(A, b, i, h * A.G + (r - i * A.G), lane * E, v, m, l, n);
}

}  // namespace sv
