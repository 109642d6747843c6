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
// so each is read once.
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
// zero and added to the running F32 sum times the block's scale (one FMA per
// value).  Two ways to sum a block:
//   F8   v_mfma_scale_f32_16x16x128_f8f6f4 on the e4m3 bytes, the hidden
//        row's power of two as its scale operand.  It adds neighbouring
//        products to about 14 bits (2-norm error 1.5e-5 on normal data), so it
//        serves BF16 logits only.
//   BF16 four v_mfma_f32_16x16x32_bf16 on the bytes widened to bf16, exact for
//        e4m3 and for e4m3 times a power of two; sums as exact as F32's.
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

typedef int f8_i32x8 __attribute__((ext_vector_type(8)));

// Bytes 8 h .. 8 h + 7 of a lane's 16 as bf16 times `scale` (a power of two).
__device__ __forceinline__ f8_bf16x8 f8_widen(const uint4& w, int h, float scale) {
  const uint32_t a = h ? w.z : w.x, b = h ? w.w : w.y;
  uint4 f;
  f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false));
  f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
  f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
  f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
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
    const uint16_t h[4] = {__builtin_bit_cast(uint16_t, (__bf16)x[0]), __builtin_bit_cast(uint16_t, (__bf16)x[1]),
                           __builtin_bit_cast(uint16_t, (__bf16)x[2]), __builtin_bit_cast(uint16_t, (__bf16)x[3])};
    if (vec && v + 4 <= V) {
      *reinterpret_cast<uint2*>(row + v) = make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (v + r < V) row[v + r] = h[r];
    }
  }
}
template <typename TO>
__device__ __forceinline__ bool f8_vec_out(const F8HeadArgs& A) {
  constexpr size_t n = 4 * sizeof(TO);
  return ((uintptr_t)A.out % n | (uintptr_t)(A.o_seq * sizeof(TO)) % n | (uintptr_t)(A.o_pos * sizeof(TO)) % n) == 0;
}

// Few hidden rows: bound by the weights' bytes.  A wave takes 16 NB vocabulary
// entries and every row (16 MB of them), its fragments straight from memory to
// registers, the blocks of 128 ahead of the one being summed in flight.
template <typename TO, int MB, int NB>
__global__ __launch_bounds__(64) void k_lmhead_fp8_rows(F8HeadArgs A) {
  const int lane = threadIdx.x, n16 = lane & 15, q = lane >> 4;
  const int64_t v0 = (int64_t)blockIdx.x * (16 * NB);
  const int32_t blocks = A.dp / 128;
  const uint8_t* wp[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int64_t v = v0 + 16 * nb + n16;
    wp[nb] = A.weight + (v < A.V ? v : A.V - 1) * A.w_stride;  // rows past V are not stored
  }
  const uint8_t* hp[MB];
  const uint8_t* ep[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = 16 * mb + n16, row = m < A.M ? m : A.M - 1;
    hp[mb] = A.hidden + row * A.dp + q * 16;
    ep[mb] = A.exps + row;
  }
  const float* sp = A.scale + (v0 / 128) * blocks;  // 16 NB entries lie in one block of 128

  struct Block {
    uint4 w[NB][2], h[MB][2];
    uint32_t e[MB];
    float s;
  };
  auto load = [&](int32_t kb, Block& B) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // a column past d meets zeros of the hidden row: any byte of the same
      // head row does
      const int32_t col = kb * 128 + x * 64 + q * 16, c = col < A.d ? col : 0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) B.w[nb][x] = load16(wp[nb] + c);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) B.h[mb][x] = load16(hp[mb] + kb * 128 + x * 64);
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) B.e[mb] = ep[mb][kb * A.m_pitch];
    B.s = sp[kb];
  };
  f8_f32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
  auto add = [&](const Block& B) {
    f8_f32x4 c[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) c[mb][nb] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f8_bf16x8 hf[MB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) hf[mb] = f8_widen(B.h[mb][x], h, f8_scale(B.e[mb]));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const f8_bf16x8 wf = f8_widen(B.w[nb][x], h, 1.0f);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            c[mb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, hf[mb], c[mb][nb], 0, 0, 0);
        }
      }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[mb][nb][r] = __builtin_fmaf(c[mb][nb][r], B.s, acc[mb][nb][r]);
  };
  // three blocks in flight while one is summed
  Block b0, b1, b2;
  const int32_t last = blocks - 1;
  load(0, b0);
  load(min(1, last), b1);
  load(min(2, last), b2);
  int32_t kb = 0;
  for (; kb + 3 <= blocks; kb += 3) {  // reloads past the end repeat the last block, unused
    add(b0);
    load(min(kb + 3, last), b0);
    add(b1);
    load(min(kb + 4, last), b1);
    add(b2);
    load(min(kb + 5, last), b2);
  }
  if (kb < blocks) add(b0);
  if (kb + 1 < blocks) add(b1);

  const bool vec = f8_vec_out<TO>(A);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = 16 * mb + n16;
    if (m >= A.M) continue;
    TO* row = f8_out_row<TO>(A, m);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) f8_store4<TO>(row, v0 + 16 * nb + 4 * q, A.V, acc[mb][nb], vec);
  }
}

// More rows: a matrix product in tiles of BV entries x BM rows, eight waves in
// WV x WM, the operands' blocks of 128 columns (one row of 128 bytes each)
// through two LDS buffers that the memory pipeline fills by itself
// (buffer_load ... lds, 16 bytes a lane) while the matrix instructions work on
// the other.  A row's eight 16-byte chunks are stored in the order c ^ (row % 8),
// by permuting the addresses that the lanes load from, so that the eight rows a
// quarter of a fragment read touches fall on different banks.
template <typename TO, bool F8, int BV, int BM, int WV>
__global__ __launch_bounds__(512, 2) void k_lmhead_fp8_tile(F8HeadArgs A) {
  constexpr int WM = 8 / WV, TV = BV / WV / 16, TM = BM / WM / 16;  // a wave's tiles of 16
  static_assert(TV * WV * 16 == BV && TM * WM * 16 == BM, "whole tiles");
  static_assert(BV % 64 == 0 && BM % 64 == 0, "8 rows a wave and load");
  static_assert(128 % (BV / WV) == 0, "a wave's entries lie in one block of 128");
  constexpr int kTiles = BM;  // a buffer: the rows' exponents, then the bytes of [weights | hidden]
  constexpr int kBuf = kTiles + (BV + BM) * 128;
  // two arrays, each named where it is used, so that the compiler can tell a
  // fragment read of one from the fill of the other and does not wait for it
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kBuf];
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
  const int row = 8 * w + lane / 8, chunk = ((lane & 7) ^ (lane >> 3)) * 16;  // row % 8 is lane / 8
  const int32_t woff = row * ws + chunk, hoff = row * A.dp + chunk;
  typedef __attribute__((address_space(3))) void* Lds;
  auto stage = [&](int32_t kb, uint8_t* to) {
    // one register per operand: the rows' offsets are added here, not kept
    int32_t wo = woff, ho = hoff;
    asm volatile("" : "+v"(wo), "+v"(ho));
    // a column past d: the hidden row's zeros meet a zero
    const bool in = kb * 128 + chunk < A.d;
#pragma unroll
    for (int i = 0; i < BV / 64; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wsrc, (Lds)(to + kTiles + (64 * i + 8 * w) * 128), 16,
                                               in ? wo + (kb * 128 + 64 * i * ws) : 0x7FFFFFFF, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < BM / 64; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(hsrc, (Lds)(to + kTiles + (BV + 64 * i + 8 * w) * 128), 16,
                                               ho + (kb * 128 + 64 * i * A.dp), 0, 0, 0);
    if (w < BM / 256)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(esrc, (Lds)(to + 256 * w), 4,
                                               (int32_t)(kb * A.m_pitch) + 256 * w + 4 * lane, 0, 0, 0);
  };
  auto chunk_of = [&](const uint8_t* from, int r, int c) {
    return *reinterpret_cast<const uint4*>(from + kTiles + r * 128 + ((c ^ (r & 7)) * 16));
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

  auto compute = [&](int32_t kb, const uint8_t* from) {
    const float s = sp[kb];
    uint4 wf[TV][2];
#pragma unroll
    for (int i = 0; i < TV; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) wf[i][y] = chunk_of(from, vw + 16 * i + n16, 4 * y + q);
    f8_bf16x8 wb[F8 ? 1 : TV][4];
    if constexpr (!F8)
#pragma unroll
      for (int i = 0; i < TV; ++i)
#pragma unroll
        for (int y = 0; y < 4; ++y) wb[i][y] = f8_widen(wf[i][y / 2], y & 1, 1.0f);
    // a column of tiles is added to the running sums while the next one's
    // products are under way
    f8_f32x4 c[2][TV];
    auto add = [&](int j) {
#pragma unroll
      for (int i = 0; i < TV; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(c[j & 1][i][r], s, acc[i][j][r]);
      // keeps the products here: without a use they may move past the barrier
#pragma unroll
      for (int i = 0; i < TV; ++i) asm volatile("" : "+v"(acc[i][j]));
    };
    uint4 hf[2][2];
    uint32_t e[2];
    auto rows = [&](int j) {
#pragma unroll
      for (int y = 0; y < 2; ++y) hf[j & 1][y] = chunk_of(from, BV + mw + 16 * j + n16, 4 * y + q);
      e[j & 1] = from[mw + 16 * j + n16];
    };
    rows(0);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      if (j + 1 < TM) rows(j + 1);
#pragma unroll
      for (int i = 0; i < TV; ++i) c[j & 1][i] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (F8) {
        const f8_i32x8 hb = f8_join(hf[j & 1][0], hf[j & 1][1]);
#pragma unroll
        for (int i = 0; i < TV; ++i)
          c[j & 1][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              f8_join(wf[i][0], wf[i][1]), hb, c[j & 1][i], 0, 0, 0, 127, 0, (int)e[j & 1]);
      } else {
        const float sh = f8_scale(e[j & 1]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const f8_bf16x8 hb = f8_widen(hf[j & 1][y / 2], y & 1, sh);
#pragma unroll
          for (int i = 0; i < TV; ++i)
            c[j & 1][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[i][y], hb, c[j & 1][i], 0, 0, 0);
        }
      }
      if (j) add(j - 1);
      // the order above is the one meant: fragments one column ahead, no more
      __builtin_amdgcn_sched_barrier(0);
    }
    add(TM - 1);
    __builtin_amdgcn_sched_barrier(0);
  };

  // At each barrier the block to compute has arrived for every wave (each
  // waits for its own loads first), and every wave is done with the buffer
  // that the next one goes to.
  auto arrive = [] {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  stage(0, buf0);
  int32_t kb = 0;
  for (; kb + 1 < blocks; kb += 2) {
    arrive();
    stage(kb + 1, buf1);
    compute(kb, buf0);
    arrive();
    if (kb + 2 < blocks) stage(kb + 2, buf0);
    compute(kb + 1, buf1);
  }
  if (kb < blocks) {
    arrive();
    compute(kb, buf0);
  }

  const bool vec = f8_vec_out<TO>(A);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m = m0 + mw + 16 * j + n16;
    if (m >= A.M) continue;
    TO* row = f8_out_row<TO>(A, m);
#pragma unroll
    for (int i = 0; i < TV; ++i) f8_store4<TO>(row, v0 + vw + 16 * i + 4 * q, A.V, acc[i][j], vec);
  }
}

}  // namespace sv
