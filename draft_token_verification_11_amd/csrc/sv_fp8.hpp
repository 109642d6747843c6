// sv_fp8.hpp -- the LM head in 8-bit floating point (OCP e4m3) with one scale
// per block of 128: the weights' quantiser, the hidden rows' rounding and the
// product (gfx950, wave64).
#pragma once

#include "sv_device.hpp"

namespace sv {

typedef __bf16 f8_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 f8_bf16x8 __attribute__((ext_vector_type(8)));
typedef float f8_f32x4 __attribute__((ext_vector_type(4)));
typedef short f8_s16x2 __attribute__((ext_vector_type(2)));

// Exponent field of a block's scale: the smallest power of two whose 448-fold
// (1.75 x 2^8) holds `amax`.
__device__ __forceinline__ uint32_t f8_exponent(float amax) {
  const int32_t e = (int32_t)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)(e < 1 ? 1 : e);
}

// 2^(e - 127) of an exponent field e in [1, 254].
__device__ __forceinline__ float f8_scale(uint32_t e) { return __uint_as_float(e << 23); }

// A uniform scale's power of two as the matrix instructions' operand, 2^(e - 127), and
// what is left of it: 1 to 2, or the whole of one below F32's normal range.
__device__ __forceinline__ float f8_part(float s, int& e) {
  const uint32_t x = __float_as_uint(s);
  e = (int)(x >> 23 & 255u);
  const uint32_t part = e ? (x & 0x807FFFFFu) | 0x3F800000u : __float_as_uint(s * 0x1p127f);
  return __uint_as_float(__builtin_amdgcn_readfirstlane(part));
}

// |x| for a block's maximum: finite magnitudes only.
__device__ __forceinline__ float f8_mag(float x) {
  const float a = __builtin_fabsf(x);
  return __builtin_isfinite(a) ? a : 0.f;
}

// Four values over 2^(e - 127) as e4m3; infinities and NaN become NaN.
__device__ __forceinline__ uint32_t f8_pack4(const float* x, float scale) {
  f8_s16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

// Weights: a workgroup takes one 128 x 128 block, 16 threads to a row of 128.
// The block's values stay in registers between the maximum and the rounding,
// so each is read once.  Bound by memory: 151,936 x 4,096 BF16 (1.87 GB in and out)
// in 342 us, 5.5 TB/s; 32,003 x 1,056 F32 (169 MB) in 34 us, 5.0 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_fp8(const T* __restrict__ weight, int64_t stride,
                                                      int64_t V, int32_t d, int32_t d_blocks,
                                                      uint8_t* __restrict__ out,
                                                      float* __restrict__ scale) {
  __shared__ float slots[4];
  const int64_t vb = blockIdx.x / d_blocks;
  const int32_t db = (int32_t)(blockIdx.x % d_blocks);
  const int32_t c = db * 128 + (threadIdx.x & 15) * 8;
  float x[8][8];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t v = vb * 128 + (threadIdx.x >> 4) + 16 * k;
    if (v < V && c < d) {  // d is a multiple of 32: whole groups of 8
      load8<T, true>(weight + v * stride + c, 0, 8, x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, f8_mag(x[k][i]));
    }
  }
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(slots[0], slots[1]), fmaxf(slots[2], slots[3]));
  const float s = f8_scale(f8_exponent(amax));
  if (threadIdx.x == 0) scale[vb * d_blocks + db] = s;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t v = vb * 128 + (threadIdx.x >> 4) + 16 * k;
    if (v < V && c < d)
      *reinterpret_cast<uint2*>(out + v * d + c) = make_uint2(f8_pack4(x[k], s), f8_pack4(x[k] + 4, s));
  }
}

// Hidden rows rounded to e4m3 in blocks of 128, a block's exponent byte beside
// them.  16 threads to a block; columns past d up to a multiple of 128 are zero,
// which makes whatever the head's partial last block is multiplied with vanish.
// 2,560 rows of 4,096: 11 us; nine: 5 us, a launch.
struct F8HiddenArgs {
  const void* hidden;
  int64_t seq, pos;
  int32_t rows;
  int64_t M;
  int32_t d, dp;     // dp: d rounded up to 128
  uint8_t* out;      // [M][dp]
  uint8_t* exps;     // [dp / 128][m_pitch]
  int64_t m_pitch;   // M rounded up to 256
};
template <typename T>
__global__ __launch_bounds__(256) void k_hidden_fp8(F8HiddenArgs A) {
  const int64_t blocks = A.dp / 128;
  const int64_t x = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (x >= A.M * blocks) return;  // whole groups of 16 threads
  const int64_t m = x / blocks, b = m / A.rows;
  const int32_t c = (int32_t)(x % blocks) * 128 + (threadIdx.x & 15) * 8;
  float v[8] = {};
  if (c < A.d)
    load8<T, true>(reinterpret_cast<const T*>(A.hidden) + b * A.seq + (m - b * A.rows) * A.pos + c, 0, 8, v);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, f8_mag(v[i]));
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 16));
  const uint32_t e = f8_exponent(amax);
  const float s = f8_scale(e);
  *reinterpret_cast<uint2*>(A.out + m * A.dp + c) = make_uint2(f8_pack4(v, s), f8_pack4(v + 4, s));
  if ((threadIdx.x & 15) == 0) A.exps[(x % blocks) * A.m_pitch + m] = (uint8_t)e;
}

// ---------------------------------------------------------------------------
// The product.  A operand the weights, Bt the hidden rows, so that a lane of a
// 16 x 16 tile holds four neighbouring vocabulary entries of one hidden row.
// The products of a block of 128 are summed by the matrix instructions from
// zero and added to the running F32 sum (one FMA per value), with both scales or
// without either, for with one of them a block may leave F32's range where its part
// of the logit does not.  Two ways to sum a block:
//   F8   v_mfma_scale_f32_16x16x128_f8f6f4 on the e4m3 bytes, the scales' powers of
//        two as its scale operands.  Of eight neighbouring columns it drops what lies
//        below 2^-13 of their largest product (2-norm error 1.5e-5 on normal data,
//        7 x 2^-13 of the eights' largest products at most), which a logit much
//        smaller than its terms feels, so it serves BF16 logits only: it takes half
//        the time of the other (2,560 rows 1.51 ms and, to F32, 3.03).
//   BF16 four v_mfma_f32_16x16x32_bf16 on the bytes widened to bf16, exact for
//        e4m3; sums as exact as F32's, from 2^-18 to 2^25, and the FMA takes them
//        times the product of the scales.
// Both take a lane's inner index in the same order: lane group q = l / 16 holds
// columns 16 q .. + 16 and 64 + 16 q .. + 16 of the block, two 16-byte loads.
struct F8HeadArgs {
  const uint8_t* hidden;   // [M][dp] e4m3
  const uint8_t* exps;     // [dp / 128][m_pitch]
  int64_t m_pitch, M, V;
  int32_t d, dp, rows;
  const uint8_t* weight;
  int64_t w_stride;
  const float* scale;
  void* out;
  int64_t o_seq, o_pos;
  int32_t v_tiles, m_tiles;
};

typedef int f8_i32x4 __attribute__((ext_vector_type(4)));
typedef int f8_i32x8 __attribute__((ext_vector_type(8)));

// Bytes 8 h .. 8 h + 7 of a lane's 16 as bf16.
__device__ __forceinline__ f8_bf16x8 f8_widen(const uint4& w, int h) {
  const uint32_t a = h ? w.z : w.x, b = h ? w.w : w.y;
  uint4 f;
  f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false));
  f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true));
  f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false));
  f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true));
  return __builtin_bit_cast(f8_bf16x8, f);
}
__device__ __forceinline__ f8_i32x8 f8_join(const uint4& a, const uint4& b) {
  return f8_i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

template <typename TO>
__device__ __forceinline__ TO* f8_out_row(const F8HeadArgs& A, int64_t m) {
  const int64_t b = m / A.rows;
  return reinterpret_cast<TO*>(A.out) + b * A.o_seq + (m - b * A.rows) * A.o_pos;
}
__device__ __forceinline__ uint2 f8_bf16x4(const f8_f32x4& x) {
  typedef __bf16 V __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, V{(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]});
}

// Four neighbouring logits of a row; `vec`: the row's fours are aligned.
template <typename TO>
__device__ __forceinline__ void f8_store4(TO* row, int64_t v, int64_t V, const f8_f32x4& x, bool vec) {
  if constexpr (sizeof(TO) == 4) {
    if (vec && v + 4 <= V) {
      *reinterpret_cast<float4*>(row + v) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (v + r < V) row[v + r] = x[r];
    }
  } else {
    const uint2 h = f8_bf16x4(x);
    if (vec && v + 4 <= V) {
      *reinterpret_cast<uint2*>(row + v) = h;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (v + r < V) row[v + r] = (uint16_t)((r < 2 ? h.x : h.y) >> (16 * (r & 1)));
    }
  }
}
template <typename TO>
__device__ __forceinline__ bool f8_vec_out(const F8HeadArgs& A) {
  constexpr size_t n = 4 * sizeof(TO);
  return ((uintptr_t)A.out % n | (uintptr_t)(A.o_seq * sizeof(TO)) % n | (uintptr_t)(A.o_pos * sizeof(TO)) % n) == 0;
}

// Up to 16 hidden rows: bound by the weights' bytes.  The hidden rows stand in
// LDS whole, in the order in which lanes take them; a wave goes through units of
// 16 vocabulary entries, their blocks of 128 columns straight from memory to
// registers, kFly blocks in flight also from one unit into the next.  Nine rows
// over 151,936 x 4,096, F32 logits: 120 us, 5.2 TB/s of weights and logits.
template <typename TO, int BLOCKS>  // BLOCKS: the most blocks a row may have
__global__ __launch_bounds__(512, 2) void k_lmhead_fp8_rows(F8HeadArgs A) {
  constexpr int kFly = 6;
  __shared__ __attribute__((aligned(16))) uint8_t hs[BLOCKS * 2048];
  __shared__ uint8_t es[BLOCKS * 16];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, q = lane >> 4;
  const int32_t blocks = A.dp / 128;
  const int32_t units = (int32_t)((A.V + 15) / 16), waves = gridDim.x * 8;  // V is at most 2^24
  const int32_t mine = blockIdx.x * 8 + w;

  // This wave's blocks: all of unit `mine`, then of `mine` + waves, ..  Where rows
  // lie a multiple of 4 KiB apart, a unit's begin at column block unit % blocks:
  // waves side by side would read the same columns of their rows at one time, and
  // those share few memory channels (nine rows, 151,936 x 4,096: 137 us from
  // column 0, 124 so; 32,000 x 8,192: 64 and 55; at pitches of 1,024 to 3,584
  // bytes it would cost 2 to 8 %).  Past the last block the loads repeat it, unused: no branch makes the compiler wait
  // for all of them.
  struct Block {
    uint4 w[2];
    float s;
  };
  const bool turn = A.w_stride % 4096 == 0;
  int32_t lu = min(mine, units - 1);  // where the loads are
  int32_t lk = turn ? lu % blocks : 0, left = blocks;
  auto load = [&](Block& B) {
    const int64_t v = min((int64_t)lu * 16 + n16, A.V - 1);  // entries past V are not stored
    const uint8_t* lw = A.weight + v * A.w_stride;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // a column past d meets zeros of the hidden rows: column 0 stands in
      const int32_t col = lk * 128 + x * 64 + q * 16;
      B.w[x] = load16(lw + (col < A.d ? col : 0));
    }
    B.s = A.scale[(int64_t)(lu / 8) * blocks + lk];  // a unit lies in one block of 128 entries
    if (--left > 0) {
      lk = lk + 1 == blocks ? 0 : lk + 1;
    } else if (lu + waves < units) {
      left = blocks;
      lu += waves;
      lk = turn ? lu % blocks : 0;
    }
  };
  Block ring[kFly];
#pragma unroll
  for (int k = 0; k < kFly; ++k) load(ring[k]);

  for (int32_t i = w; i < 2 * blocks; i += 8) {
    const int64_t m = min((int64_t)n16, A.M - 1);
    *reinterpret_cast<uint4*>(hs + i * 1024 + lane * 16) =
        load16(A.hidden + m * A.dp + (i >> 1) * 128 + (i & 1) * 64 + q * 16);
  }
  for (int32_t i = threadIdx.x; i < blocks * 16; i += 512)
    es[i] = A.exps[(i >> 4) * A.m_pitch + min((int64_t)(i & 15), A.M - 1)];
  __syncthreads();

  const bool vec = f8_vec_out<TO>(A);
  int32_t u = mine, kb = turn ? mine % blocks : 0, todo = blocks;
  f8_f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  while (u < units) {
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      if (u >= units) break;
      const float s = ring[k].s * f8_scale(es[kb * 16 + n16]);
      f8_f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 h = *reinterpret_cast<const uint4*>(hs + (2 * kb + x) * 1024 + lane * 16);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_widen(ring[k].w[x], y), f8_widen(h, y), c, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(c[r], s, acc[r]);
      load(ring[k]);
      kb = kb + 1 == blocks ? 0 : kb + 1;
      if (--todo == 0) {
        if (n16 < A.M) f8_store4<TO>(f8_out_row<TO>(A, n16), (int64_t)u * 16 + 4 * q, A.V, acc, vec);
        acc = f8_f32x4{0.f, 0.f, 0.f, 0.f};
        todo = blocks;
        u += waves;
        kb = turn ? u % blocks : 0;
      }
    }
  }
}

// More rows: a matrix product in tiles of BV entries x BM rows, WAVES waves in
// WV x WM, the operands' blocks of 128 columns (one row of 128 bytes each)
// through two LDS buffers each that the memory pipeline fills by itself
// (buffer_load ... lds, 16 bytes a lane) while the matrix instructions work on
// the other.  A row's eight 16-byte chunks are stored in the order
// c ^ (row / 2 % 8), by permuting the addresses that the lanes load from, so that
// the 16 rows a quarter of a fragment read touches (256 bytes) fall on the 64
// banks without conflict.  2,560 rows over 151,936 x 4,096 to BF16 logits: 1.50 ms,
// 2.1 PFLOP/s (the matrix units busy for 52 % of it, vector instructions for 57 %;
// LDS reads and fills take as many cycles, and the chip's clock falls to 2.0 GHz);
// 240 rows over 128,003 x 2,080 to F32: 0.17 ms, 0.20 where the weights come from
// memory (matrix units busy for 40 %, vector instructions, which widen, for 51 %), of
// which rows that do not start at multiples of 16 bytes cost a tenth or more (over
// 128,000 entries: 0.16 to 0.18).
template <typename TO, bool F8, int BV, int BM, int WV, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void k_lmhead_fp8_tile(F8HeadArgs A) {
  constexpr int WM = WAVES / WV, TV = BV / WV / 16, TM = BM / WM / 16;  // a wave's tiles of 16
  static_assert(TV * WV * 16 == BV && TM * WM * 16 == BM, "whole tiles");
  constexpr int kStep = 8 * WAVES;  // rows that one load of each wave brings
  static_assert(BV % kStep == 0 && BM % kStep == 0, "whole loads");
  static_assert(128 % (BV / WV) == 0, "a wave's entries lie in one block of 128");
  static_assert(TV <= 4, "a column's tiles are added in four steps");
  constexpr int kExps = 256;  // before the hidden rows' bytes: their exponents
  static_assert(BM <= kExps, "room");
  // arrays of their own, each named where it is used, so that the compiler can
  // tell a fragment read of one from the fill of another and does not wait for it
  __shared__ __attribute__((aligned(16))) uint8_t w0[BV * 128], w1[BV * 128];
  __shared__ __attribute__((aligned(16))) uint8_t h0[kExps + BM * 128], h1[kExps + BM * 128];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, q = lane >> 4;
  // the workgroups of one XCD (blockIdx % 8) take neighbouring tiles, rows
  // fastest, so that they share the head's tiles and the rows in its L2
  const int64_t tiles = (int64_t)A.v_tiles * A.m_tiles, per = (tiles + 7) / 8;
  const int64_t at = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || at >= tiles) return;
  const int64_t v0 = at / A.m_tiles * BV, m0 = at % A.m_tiles * BM;
  const int32_t blocks = A.dp / 128;

  // The tile's part of each operand as a buffer: 32-bit offsets, and rows past
  // its end read as zeros.
  const int32_t vr = (int32_t)min((int64_t)BV, A.V - v0), mr = (int32_t)min((int64_t)BM, A.M - m0);
  const int32_t ws = (int32_t)A.w_stride;
  const auto wsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A.weight + v0 * A.w_stride), 0,
                                                      (vr - 1) * ws + A.d, 0x00020000);
  const auto hsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A.hidden + m0 * A.dp), 0,
                                                      mr * A.dp, 0x00020000);
  const auto esrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A.exps + m0), 0,
                                                      (int32_t)min(A.m_pitch * blocks - m0, (int64_t)0x7FFFFFFF), 0x00020000);
  const int row = 8 * w + lane / 8, chunk = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
  const int32_t woff = row * ws + chunk, hoff = row * A.dp + chunk;
  typedef __attribute__((address_space(3))) void* Lds;
  // Load x of block kb's weights, and of its hidden rows, eight rows a wave; with
  // the last one the first wave's load of the exponents.  The rows' offsets are
  // added here, not kept in a register each.
  constexpr int kWLoads = BV / kStep, kHLoads = BM / kStep;
  auto stage_w = [&](int32_t kb, uint8_t* to, int x) {
    int32_t wo = woff;
    asm volatile("" : "+v"(wo));
    // a column past d: the hidden row's zeros meet a zero
    const bool in = kb * 128 + chunk < A.d;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wsrc, (Lds)(to + (kStep * x + 8 * w) * 128), 16,
                                             in ? wo + (kb * 128 + kStep * x * ws) : 0x7FFFFFFF, 0, 0, 0);
  };
  auto stage_h = [&](int32_t kb, uint8_t* to, int x) {
    int32_t ho = hoff;
    asm volatile("" : "+v"(ho));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(hsrc, (Lds)(to + kExps + (kStep * x + 8 * w) * 128), 16,
                                             ho + (kb * 128 + kStep * x * A.dp), 0, 0, 0);
    if (x == kHLoads - 1 && w == 0)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(esrc, (Lds)to, 4, (int32_t)(kb * A.m_pitch) + 4 * lane, 0, 0, 0);
  };
  auto chunk_of = [&](const uint8_t* from, int r, int c) {
    return *reinterpret_cast<const uint4*>(from + r * 128 + ((c ^ ((r >> 1) & 7)) * 16));
  };

  f8_f32x4 acc[TV][TM];
#pragma unroll
  for (int i = 0; i < TV; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
  const int vw = (w / WM) * (BV / WV), mw = (w % WM) * (BM / WM);  // this wave's corner
  // uniform, and read by the scalar unit: a wait on it is no wait for the tiles
  const auto* sp = (const __attribute__((address_space(4))) float*)(
      A.scale + min((v0 + vw) / 128, (A.V - 1) / 128) * blocks);

  // A barrier behind this wave's reads of LDS (__syncthreads would wait for all
  // loads that are on their way to LDS too).
  auto meet = [] {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // Computes block kb from wa and ha and starts the loads of the next one's
  // hidden rows (into hb) and, when every wave has its weights in registers, of
  // the weights of the one after that (into wa): spread over the columns, for
  // issued together they hold the wave (and, after a barrier, all of them) for
  // 700 to 1,200 cycles of a block's 4,000.
  constexpr int kH = TM / 2;  // columns with the hidden rows' loads
  float next = sp[0];  // the scale of the block to come: the first product takes it
  auto compute = [&](int32_t kb, uint8_t* wa, const uint8_t* ha, uint8_t* hn) {
    const float s = next;
    next = sp[min(kb + 1, blocks - 1)];
    uint4 wf[TV][2];
#pragma unroll
    for (int i = 0; i < TV; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) wf[i][y] = chunk_of(wa, vw + 16 * i + n16, 4 * y + q);
    f8_bf16x8 wb[F8 ? 1 : TV][4];
    if constexpr (!F8)
#pragma unroll
      for (int i = 0; i < TV; ++i)
#pragma unroll
        for (int y = 0; y < 4; ++y) wb[i][y] = f8_widen(wf[i][y / 2], y & 1);
    // a tile is added to the running sums while the matrix unit works on the one
    // in its place of the next column
    f8_f32x4 c[2][TV];
    // F8: the powers of two go to the instruction, and what is left of the weights'
    // scale to the sum (2,560 rows 1,511 us; with a factor of both scales for each
    // column 1,537); else that factor
    int we = 0;
    float both[2];
    if constexpr (F8) both[0] = both[1] = f8_part(s, we);
    auto add = [&](int i, int j) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(c[j & 1][i][r], both[j & 1], acc[i][j][r]);
      // keeps the products here: without a use they may move past the barrier
      asm volatile("" : "+v"(acc[i][j]));
    };
    uint4 hf[2][2];
    uint32_t e[2];
    auto rows = [&](int j) {
#pragma unroll
      for (int y = 0; y < 2; ++y) hf[j & 1][y] = chunk_of(ha + kExps, mw + 16 * j + n16, 4 * y + q);
      e[j & 1] = ha[mw + 16 * j + n16];
    };
    rows(0);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      if (j == 1) meet();  // every wave has its weights
      if (j + 1 < TM) rows(j + 1);
      if (j < kH) {
#pragma unroll
        for (int x = kHLoads * j / kH; x < kHLoads * (j + 1) / kH; ++x) stage_h(kb + 1, hn, x);
      }
      if (j >= kH) {
#pragma unroll
        for (int x = kWLoads * (j - kH) / (TM - kH); x < kWLoads * (j + 1 - kH) / (TM - kH); ++x)
          stage_w(kb + 2, wa, x);
      }
      if constexpr (F8) {
        const f8_i32x8 hb = f8_join(hf[j & 1][0], hf[j & 1][1]);
#pragma unroll
        for (int i = 0; i < TV; ++i) {
          c[j & 1][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              f8_join(wf[i][0], wf[i][1]), hb, f8_f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, we, 0, (int)e[j & 1]);
          __builtin_amdgcn_sched_barrier(0);  // the order here is the one meant
          if (j) add(i, j - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        both[j & 1] = f8_scale(e[j & 1]) * s;
        f8_bf16x8 hb[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) hb[y] = f8_widen(hf[j & 1][y / 2], y & 1);
#pragma unroll
        for (int i = 0; i < TV; ++i) c[j & 1][i] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
#pragma unroll
          for (int i = 0; i < TV; ++i) {
            c[j & 1][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[i][y], hb[y], c[j & 1][i], 0, 0, 0);
            if (i == 0) __builtin_amdgcn_sched_barrier(0);
          }
          if (j && y < TV) add(y, j - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TV; ++i) add(i, TM - 1);
    __builtin_amdgcn_sched_barrier(0);
  };

  // At each barrier the block to compute has arrived for every wave (each waits
  // for its own loads first, but for those of the next block's weights, which
  // are the last), and every wave is done with the buffers that are filled next.
  // Loads past the last block read zeros or a row's next bytes and are not used:
  // with a branch around them the compiler would wait for all.
  auto arrive = [&] {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWLoads) : "memory");
    meet();
  };
#pragma unroll
  for (int x = 0; x < kWLoads; ++x) stage_w(0, w0, x);
#pragma unroll
  for (int x = 0; x < kHLoads; ++x) stage_h(0, h0, x);
#pragma unroll
  for (int x = 0; x < kWLoads; ++x) stage_w(1, w1, x);
  int32_t kb = 0;
  for (; kb + 1 < blocks; kb += 2) {
    arrive();
    compute(kb, w0, h0, h1);
    arrive();
    compute(kb + 1, w1, h1, h0);
  }
  if (kb < blocks) {
    arrive();
    compute(kb, w0, h0, h1);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // The tile leaves through LDS, so that a row's entries leave together: kOut
  // rows at a time, 512 bytes of a row (its 16-byte chunks in the order
  // c ^ (row % 32), for the banks), then 16 bytes a lane, or one entry a lane
  // where the rows do not start at multiples of 16 bytes (of 240 rows of
  // 128,003 F32 entries over 2,080, stores from the registers took 8 % more).  BF16
  // logits go past the caches: with the verify call that reads them 240 rows of
  // 128,000 over 4,096 take 178 us, else 185, and 2,560 rows of 151,936 1.69 and
  // 1.72 ms; for F32 ones of 240 rows of 151,936 over 2,080 it would be 274 and 266.
  constexpr int kRowBytes = BV * sizeof(TO), kChunks = kRowBytes / 16;
  constexpr int kOut = 256 / (int)sizeof(TO) < BM ? 256 / (int)sizeof(TO) : BM;
  static_assert(kOut / 2 * kRowBytes <= BV * 128, "room");
  auto out_chunk = [&](int r, int c) { return (r & 1 ? w1 : w0) + r / 2 * kRowBytes + (c ^ (r & (kChunks - 1))) * 16; };
  constexpr int kRound = kOut / WM / 16;  // a wave's columns of tiles each time
  static_assert(TM % kRound == 0, "whole rounds");
  const bool vec = ((uintptr_t)A.out | (uintptr_t)(A.o_seq * sizeof(TO)) | (uintptr_t)(A.o_pos * sizeof(TO))) % 16 == 0;
#pragma unroll
  for (int g = 0; g < TM / kRound; ++g) {
    __syncthreads();  // every wave is done with the buffers
#pragma unroll
    for (int j = 0; j < kRound; ++j) {
      const int r = (w % WM) * (kRound * 16) + 16 * j + n16;
#pragma unroll
      for (int i = 0; i < TV; ++i) {
        const f8_f32x4 x = acc[i][g * kRound + j];
        const int at = (vw + 16 * i + 4 * q) * (int)sizeof(TO);  // 8 or 16 bytes
        uint8_t* to = out_chunk(r, at / 16) + at % 16;
        if constexpr (sizeof(TO) == 4) *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<uint2*>(to) = f8_bf16x4(x);
      }
    }
    __syncthreads();
    if (vec) {
      const int c = threadIdx.x % kChunks;
      constexpr int kPass = 64 * WAVES / kChunks;
#pragma unroll
      for (int k = 0; k < kOut / kPass; ++k) {
        const int r = kPass * k + threadIdx.x / kChunks;
        const int64_t m = m0 + (r / (kRound * 16)) * (BM / WM) + g * kRound * 16 + r % (kRound * 16);
        constexpr int kPer = 16 / sizeof(TO);
        const int64_t v = v0 + c * kPer;
        if (m >= A.M || v >= A.V) continue;
        TO* row = f8_out_row<TO>(A, m);
        const uint8_t* from = out_chunk(r, c);
        if (v + kPer <= A.V) {
          const f8_i32x4 x = *reinterpret_cast<const f8_i32x4*>(from);
          if constexpr (sizeof(TO) == 2) __builtin_nontemporal_store(x, reinterpret_cast<f8_i32x4*>(row + v));
          else *reinterpret_cast<f8_i32x4*>(row + v) = x;
        } else {
          for (int e = 0; v + e < A.V; ++e) row[v + e] = reinterpret_cast<const TO*>(from)[e];
        }
      }
    } else {
      for (int r = w; r < kOut; r += WAVES) {
        const int64_t m = m0 + (r / (kRound * 16)) * (BM / WM) + g * kRound * 16 + r % (kRound * 16);
        if (m >= A.M) continue;
        TO* row = f8_out_row<TO>(A, m);
#pragma unroll
        for (int k = 0; k < BV / 64; ++k) {
          const int x = 64 * k + lane, at = x * (int)sizeof(TO);
          if (v0 + x < A.V)
            row[v0 + x] = *reinterpret_cast<const TO*>(out_chunk(r, at / 16) + at % 16);
        }
      }
    }
  }
}

}  // namespace sv
