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
// once, and only the exponent bytes (1 of 17 stored) are scattered.
struct C4MoveArgs {
  C4View cache;
  C4Heads k, v;
  const int32_t* start;
  const int32_t* count;  // or null: T
  int64_t waves;
  int32_t T, runs;       // runs: position runs of a wave's length a sequence may touch
};

__device__ __forceinline__ float c4_exp_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Exponent byte of a group with the largest magnitude `amax` (finite).
__device__ __forceinline__ uint32_t c4_exponent(float amax) {
  const int32_t e = (int32_t)((__float_as_uint(amax) + 0x3FFFFFu) >> 23) - 2;
  return (uint32_t)(e < 1 ? 1 : e);
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
// rounded to bf16 for the product (2^-9 relative, the size of the output's
// own rounding); the normaliser sums the unrounded fp32 values.
//
// Work split: the pages of all (sequence, kv head, block of rows) are laid end
// to end and cut into one equal range per workgroup, whatever the sequences'
// lengths; the four waves of a workgroup take the range's pages in turn.  A
// workgroup whose range ends inside a sequence leaves its rows' maximum, sum
// and unnormalised output in the workspace, and k_attention_cache4_join adds
// those up in order, so that results do not depend on the order of workgroups.
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
  float* parts;           // [2 grid] records of a workgroup's first and last cut segment
  int32_t grid;
};

// Pages of sequence b that its new tokens attend to; 0 when it has no rows.
// `bad`: ill-formed (one page then stands for the sequence, so that its rows
// are visited).
__device__ __forceinline__ int32_t c4_pages(const C4AttnArgs& A, int64_t b, bool& bad) {
  const int32_t s = A.start[b], n = A.count ? A.count[b] : A.T;
  bad = !A.cache.fits(s, n, A.T);
  if (bad) return 1;
  return n == 0 ? 0 : (s + n + kC4Page - 1) / kC4Page;
}

// Prefix sums of the sequences' pages over a workgroup: thread t owns
// sequences t * per .. + per.
struct C4Plan {
  int64_t before[256];
  int64_t wave[4];
  int64_t total;
};
__device__ __forceinline__ int32_t c4_plan(const C4AttnArgs& A, C4Plan& P) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int32_t per = (A.B + 255) / 256;
  int64_t sum = 0;
  for (int32_t j = 0; j < per; ++j) {
    const int64_t b = (int64_t)tid * per + j;
    bool bad;
    if (b < A.B) sum += c4_pages(A, b, bad);
  }
  int64_t incl = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 63) P.wave[w] = incl;
  __syncthreads();
  int64_t base = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < w) base += P.wave[i];
  P.before[tid] = base + incl - sum;
  if (tid == 255) P.total = base + incl;
  __syncthreads();
  return per;
}

// Pages of each workgroup's range: an equal share, at least one page per wave.
__device__ __forceinline__ int64_t c4_share(int64_t pages, int32_t grid) {
  const int64_t s = (pages + grid - 1) / grid;
  return s < 4 ? 4 : s;
}

template <int D, int RT>
struct C4Rec {  // one cut segment: O [RT * 16][D], m and l [RT * 16]
  static constexpr int kRows = RT * 16;
  static constexpr int kFloats = kRows * (D + 2);
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

constexpr float kC4Low = -3.0e38f;  // a maximum before any score
constexpr float kC4Raise = 8.0f;    // a score passes the maximum by 2^8 before it is raised

// What a row's new token sees of the 64 positions from `base` on (relative to
// start): bit x for position base + x.
__device__ __forceinline__ uint64_t c4_sees(const C4AttnArgs& A, int64_t b, int32_t i, int32_t n,
                                            int64_t base) {
  if (i >= n) return 0;
  if (!A.mask) {
    const int64_t seen = (int64_t)i + 1 - base;  // positions below base + seen
    return seen <= 0 ? 0 : (seen >= 64 ? ~0ull : (1ull << seen) - 1);
  }
  const uint32_t* row = A.mask + b * A.mask_seq + i * A.mask_pos;
  const int32_t words = (A.T + 31) / 32;
  auto word = [&](int64_t k) -> uint64_t {
    if (k < 0) return 0xFFFFFFFFull;      // cached tokens
    if (k >= words) return 0;
    uint32_t w = row[k];
    const int64_t left = n - 32 * k;      // new tokens of this word
    if (left < 32) w &= left <= 0 ? 0u : (1u << left) - 1u;
    return w;
  };
  const int64_t k0 = base >> 5;           // floor: base may be negative
  const int sh = (int)(base & 31);
  const uint64_t lo = word(k0) | (word(k0 + 1) << 32);
  return sh == 0 ? lo : (lo >> sh) | (word(k0 + 2) << (64 - sh));
}

// The codes and exponents of one page in a lane's registers.
template <int D>
struct C4PageRegs {
  static constexpr int NG = C4<D>::NG;
  static constexpr int KW = D / 32;            // dwords of key codes per tile
  uint32_t k[4][KW];                           // 4 tiles: D / 8 bytes of one token
  uint32_t v[4][D / 32];                       // 4 tiles: 4 tokens x D / 32 bytes
  uint32_t ke[D == 256 ? 2 : 1];               // byte `tile`: this lane's token
  uint32_t ve[4];                              // byte j: token 4 q + j of the tile
};

template <int N>
__device__ __forceinline__ void c4_load_words(const uint8_t* p, uint32_t* out) {
  if constexpr (N == 2) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    out[0] = a.x, out[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 a = *reinterpret_cast<const uint4*>(p + 16 * i);
      out[4 * i] = a.x, out[4 * i + 1] = a.y, out[4 * i + 2] = a.z, out[4 * i + 3] = a.w;
    }
  }
}

template <int D>
__device__ __forceinline__ void c4_load_page(const uint8_t* rec, int lane, C4PageRegs<D>& R) {
  constexpr int NG = C4<D>::NG;
  const int n = lane & 15, q = lane >> 4;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    c4_load_words<D / 32>(rec + (16 * t + n) * (D / 2) + q * (D / 8), R.k[t]);
    c4_load_words<D / 32>(rec + C4<D>::kVal + (t * 64 + lane) * (D / 8), R.v[t]);
    R.ve[t] = *reinterpret_cast<const uint32_t*>(rec + C4<D>::kValExp + (4 * t + q) * (4 * NG) +
                                                 (n * NG / 16) * 4);
  }
  const int g = q * NG / 4;
  R.ke[0] = *reinterpret_cast<const uint32_t*>(rec + C4<D>::kKeyExp + g * 64 + n * 4);
  if constexpr (D == 256)
    R.ke[1] = *reinterpret_cast<const uint32_t*>(rec + C4<D>::kKeyExp + (g + 1) * 64 + n * 4);
}

__device__ __forceinline__ uint32_t c4_cvt(uint32_t w, float scale, int byte) {
  // the byte select is an immediate; `byte` is constant at every call
  switch (byte) {
    case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
}

// Scale 2^(e - 127) of exponent byte `i` of w; 255 stands for NaN.
__device__ __forceinline__ float c4_byte_scale(uint32_t w, int i) {
  return __uint_as_float(((w >> (8 * i)) & 0xFFu) << 23);
}

template <int D, int RT>
struct C4State {
  c4_f32x4 o[RT][D / 16];
  float m[RT], l[RT];
};

// One page.  MASKED: some of its positions are not seen by some row (sees[]:
// this lane's rows; `valid`: positions that hold tokens, as bits).
template <int D, int RT, bool MASKED>
__device__ __forceinline__ void c4_page(const C4PageRegs<D>& R, const c4_bf16x8 (&qf)[RT][D / 32],
                                        C4State<D, RT>& S, float c, int lane,
                                        const uint64_t (&sees)[RT], uint64_t valid) {
  const int q = lane >> 4;
  c4_f32x4 s[RT][4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][t] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
    float scale[D == 256 ? 2 : 1];
    scale[0] = c4_byte_scale(R.ke[0], t);
    if constexpr (D == 256) scale[1] = c4_byte_scale(R.ke[1], t);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      uint4 a;
      const float sc = scale[D == 256 ? j / 4 : 0];
      a.x = c4_cvt(R.k[t][j], sc, 0);
      a.y = c4_cvt(R.k[t][j], sc, 1);
      a.z = c4_cvt(R.k[t][j], sc, 2);
      a.w = c4_cvt(R.k[t][j], sc, 3);
      const c4_bf16x8 kf = __builtin_bit_cast(c4_bf16x8, a);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        s[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[rt][j], s[rt][t], 0, 0, 0);
    }
  }
  uint4 p[RT][2];  // P' of tile pairs, the B operands
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if constexpr (MASKED) {
      const uint64_t mine = sees[rt] >> (4 * q);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!((mine >> (16 * t + r)) & 1)) s[rt][t][r] = -__builtin_inff();
    }
    float top = fmaxf(fmaxf(s[rt][0][0], s[rt][0][1]), fmaxf(s[rt][0][2], s[rt][0][3]));
#pragma unroll
    for (int t = 1; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, s[rt][t][r]);
    top = c4_max_quads(top) * c;
    if (__any(top > S.m[rt] + kC4Raise)) {
      const float m = fmaxf(S.m[rt], top);
      const float f = __builtin_amdgcn_exp2f(S.m[rt] - m);
      S.m[rt] = m;
      S.l[rt] *= f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) S.o[rt][i] *= f;
    }
    float e[4][4];
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        e[t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][t][r], c, -S.m[rt]));
        sum += e[t][r];
      }
    S.l[rt] += sum;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c4_bf16x8 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = (__bf16)e[2 * h][r];
        x[4 + r] = (__bf16)e[2 * h + 1][r];
      }
      p[rt][h] = __builtin_bit_cast(uint4, x);
    }
  }
  // V' of a tile pair: byte y of token j's codes gives that token's values of
  // two neighbouring d; tokens are paired for each d by a byte permutation
  constexpr int NB = D / 32;  // bytes of a lane's codes of one token
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int y = 0; y < NB; ++y) {
      uint32_t a[2][4];  // [tile of the pair][token]: bf16 of d = 2 y, 2 y + 1
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w = R.v[2 * h + t][(j * NB + y) / 4];
          float sc = c4_byte_scale(R.ve[2 * h + t], j);
          if constexpr (MASKED) {  // what stands past the last token is not a value
            const bool have = (valid >> (16 * (2 * h + t) + 4 * q + j)) & 1;
            w = have ? w : 0u;
            sc = have ? sc : 1.0f;
          }
          a[t][j] = c4_cvt(w, sc, (j * NB + y) % 4);
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
        const c4_bf16x8 pf = __builtin_bit_cast(c4_bf16x8, p[rt][h]);
        S.o[rt][2 * y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(c4_bf16x8, lo), pf, S.o[rt][2 * y], 0, 0, 0);
        S.o[rt][2 * y + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(c4_bf16x8, hi), pf, S.o[rt][2 * y + 1], 0, 0, 0);
      }
    }
  }
}

// Eight output values of a row as bf16.
__device__ __forceinline__ void c4_store8(uint16_t* p, const float* x) {
  c4_bf16x8 y;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (__bf16)x[i];
  *reinterpret_cast<uint4*>(p) = __builtin_bit_cast(uint4, y);
}

// Writes a finished row's eighth-of-... values: normalised, or NaN.
__device__ __forceinline__ void c4_finish8(const C4AttnArgs& A, int64_t b, int32_t i, int32_t head,
                                           int d0, float* x, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a NaN sum stays NaN
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  c4_store8(A.out + b * A.o_seq + i * A.o_pos + head * A.o_head + d0, x);
  if (d0 == 0 && A.lse) {
    constexpr float kLn2 = 0.6931471805599453f;
    const int64_t at = (b * A.T + i) * ((int64_t)A.G * A.cache.heads) + head;
    A.lse[at] = l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

template <int D, int RT>
__global__ __launch_bounds__(256) void k_attention_cache4(C4AttnArgs A) {
  constexpr int kRows = RT * 16;
  constexpr int kPad = D + 4;  // an LDS row of O: the 16 rows of a tile on different banks
  __shared__ C4Plan plan;
  __shared__ float oacc[4][16 * kPad];
  __shared__ float ms[4][kRows], ls[4][kRows];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, q = lane >> 4;
  const int32_t per = c4_plan(A, plan);
  const int64_t HR = (int64_t)A.cache.heads * A.row_blocks;
  const int64_t share = c4_share(plan.total * HR, A.grid);
  const int64_t lo = (int64_t)blockIdx.x * share;
  const int64_t hi = min(lo + share, plan.total * HR);
  if (lo >= hi) return;

  // the sequence of page `lo`: its thread's run of sequences, then within it
  int64_t b = 0, seq_at = 0;  // seq_at: pages before b, over all heads and row blocks
  {
    int t0 = 0, t1 = 255;
    while (t0 < t1) {  // last thread whose first page is at or before lo
      const int mid = (t0 + t1 + 1) / 2;
      if (plan.before[mid] * HR <= lo) t0 = mid;
      else t1 = mid - 1;
    }
    b = (int64_t)t0 * per;
    seq_at = plan.before[t0] * HR;
  }
  bool bad;
  int32_t pages = c4_pages(A, b, bad);
  while (seq_at + pages * HR <= lo) {
    seq_at += pages * HR;
    pages = c4_pages(A, ++b, bad);
  }
  int64_t at = lo;
  const int32_t R = A.T * A.G;
  while (at < hi) {
    if (at >= seq_at + pages * HR) {  // the next sequence with pages
      do {
        seq_at += pages * HR;
        pages = c4_pages(A, ++b, bad);
      } while (pages == 0);
    }
    const int64_t hr = (at - seq_at) / pages;
    const int64_t seg = seq_at + hr * pages;  // the segment's first page
    const int32_t p0 = (int32_t)(at - seg);
    const int32_t p1 = (int32_t)min((int64_t)pages, hi - seg);
    at = seg + p1;
    const int32_t h = (int32_t)(hr / A.row_blocks), r0 = (int32_t)(hr % A.row_blocks) * kRows;
    const int32_t s0 = A.start[b], nnew = bad ? A.T : (A.count ? A.count[b] : A.T);

    c4_bf16x8 qf[RT][D / 32];
    int32_t tok[RT];  // this lane's rows' tokens; T past the last row
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int32_t r = r0 + 16 * rt + n16;
      const int32_t i = r / A.G, g = r - i * A.G;
      tok[rt] = r < R ? i : A.T;
      const uint16_t* qp = A.q + b * A.q_seq + i * A.q_pos + ((int64_t)h * A.G + g) * A.q_head;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < R && i < nnew) x = load16(qp + q * (D / 4) + 8 * j);
        qf[rt][j] = __builtin_bit_cast(c4_bf16x8, x);
      }
    }
    C4State<D, RT> S;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      S.m[rt] = kC4Low;
      S.l[rt] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) S.o[rt][i] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
    }
    bool faulty = bad;
    if (!bad) {
      for (int32_t p = p0 + w; p < p1; p += 4) {
        const int32_t page = A.cache.page(b, p);
        if (page < 0) {
          faulty = true;
          continue;
        }
        C4PageRegs<D> regs;
        c4_load_page<D>(A.cache.record<D>(page, h), lane, regs);
        const int64_t base = (int64_t)p * kC4Page - s0;
        uint64_t sees[RT];
        if (base + kC4Page <= 0) {
          c4_page<D, RT, false>(regs, qf, S, A.c, lane, sees, ~0ull);
        } else {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) sees[rt] = c4_sees(A, b, tok[rt], nnew, base);
          const int64_t have = nnew - base;  // tokens of this page
          const uint64_t valid = have >= 64 ? ~0ull : (1ull << have) - 1;
          c4_page<D, RT, true>(regs, qf, S, A.c, lane, sees, valid);
        }
      }
    }
    if (faulty) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S.l[rt] = __builtin_nanf("");
    }
    // the four waves' rows together
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float l = c4_sum_quads(S.l[rt]);
      if (q == 0) {
        ms[w][16 * rt + n16] = S.m[rt];
        ls[w][16 * rt + n16] = l;
      }
    }
    __syncthreads();
    const bool whole = p0 == 0 && p1 == pages;
    float* part = A.parts + ((int64_t)blockIdx.x * 2 + (seg > lo ? 1 : 0)) * C4Rec<D, RT>::kFloats;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = 16 * rt + n16;
      const float top = fmaxf(fmaxf(ms[0][row], ms[1][row]), fmaxf(ms[2][row], ms[3][row]));
      const float f = __builtin_amdgcn_exp2f(S.m[rt] - top);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
          *reinterpret_cast<float4*>(&oacc[w][n16 * kPad + (4 * q + r) * (D / 16) + i]) =
              make_float4(S.o[rt][i][r] * f, S.o[rt][i + 1][r] * f, S.o[rt][i + 2][r] * f,
                          S.o[rt][i + 3][r] * f);
      __syncthreads();
      // 16 rows x D: eight values of a row per step
      for (int x = tid; x < 2 * D; x += 256) {
        const int rr = x / (D / 8), d0 = (x % (D / 8)) * 8;
        const int row2 = 16 * rt + rr;
        float v[8] = {};
#pragma unroll
        for (int ww = 0; ww < 4; ++ww)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += oacc[ww][rr * kPad + d0 + e];
        const float mt = fmaxf(fmaxf(ms[0][row2], ms[1][row2]), fmaxf(ms[2][row2], ms[3][row2]));
        float l = 0.f;
#pragma unroll
        for (int ww = 0; ww < 4; ++ww) l += ls[ww][row2] * __builtin_amdgcn_exp2f(ms[ww][row2] - mt);
        if (whole) {
          const int32_t r = r0 + row2, i = r / A.G;
          if (r < R && i < nnew)
            c4_finish8(A, b, i, h * A.G + (r - i * A.G), d0, v, mt, l);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + row2 * D + d0);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (d0 == 0) {
            part[kRows * D + row2] = mt;
            part[kRows * D + kRows + row2] = l;
          }
        }
      }
      __syncthreads();
    }
  }
}

// Joins the cut segments of each (sequence, kv head, block of rows), in order.
template <int D, int RT>
__global__ __launch_bounds__(256) void k_attention_cache4_join(C4AttnArgs A) {
  constexpr int kRows = RT * 16, kFloats = C4Rec<D, RT>::kFloats;
  __shared__ C4Plan plan;
  const int tid = threadIdx.x;
  const int32_t per = c4_plan(A, plan);
  const int64_t HR = (int64_t)A.cache.heads * A.row_blocks;
  const int64_t share = c4_share(plan.total * HR, A.grid);
  const int64_t b = blockIdx.x / HR, hr = blockIdx.x % HR;
  bool bad;
  int64_t before = plan.before[b / per];
  for (int64_t x = b / per * per; x < b; ++x) before += c4_pages(A, x, bad);
  const int32_t pages = c4_pages(A, b, bad);
  if (pages == 0) return;
  const int64_t seg = before * HR + hr * pages, end = seg + pages;
  const int64_t w0 = seg / share, w1 = (end - 1) / share;
  if (w0 == w1) return;  // written whole
  const int32_t h = (int32_t)(hr / A.row_blocks), r0 = (int32_t)(hr % A.row_blocks) * kRows;
  const int32_t nnew = bad ? A.T : (A.count ? A.count[b] : A.T), R = A.T * A.G;
  auto rec = [&](int64_t wg) {
    return A.parts + (wg * 2 + (wg == w0 && seg > wg * share ? 1 : 0)) * kFloats;
  };
  for (int x = tid; x < kRows * D / 8; x += 256) {
    const int row = x / (D / 8), d0 = (x % (D / 8)) * 8;
    const int32_t r = r0 + row, i = r / A.G;
    if (r >= R || i >= nnew) continue;
    float m = kC4Low, l = 0.f, v[8] = {};
    for (int64_t wg = w0; wg <= w1; ++wg) {
      const float* p = rec(wg);
      const float pm = p[kRows * D + row], pl = p[kRows * D + kRows + row];
      const float top = fmaxf(m, pm);
      const float f = __builtin_amdgcn_exp2f(m - top), g = __builtin_amdgcn_exp2f(pm - top);
      m = top;
      l = l * f + pl * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * f + p[row * D + d0 + e] * g;
    }
    c4_finish8(A, b, i, h * A.G + (r - i * A.G), d0, v, m, l);
  }
}

}  // namespace sv
