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
  const float s = __uint_as_float(f8_exponent(amax) << 23);
  if (threadIdx.x == 0) scale[vb * d_blocks + db] = s;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t v = vb * 128 + (threadIdx.x >> 4) + 16 * k;
    if (v < V && c < d)
      *reinterpret_cast<uint2*>(out + v * d + c) = make_uint2(f8_pack4(x[k], s), f8_pack4(x[k] + 4, s));
  }
}

// Hidden rows rounded to e4m3 in blocks of 128 and kept as bf16, which holds
// every e4m3 value times its power of two exactly (down to bf16's own range).
// 16 threads to a block; columns past d up to a multiple of 128 are zero.
struct F8HiddenArgs {
  const void* hidden;
  int64_t seq, pos;
  int32_t rows;
  int64_t M;
  int32_t d, dp;     // dp: d rounded up to 128
  uint16_t* out;     // [M][dp]
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
  const float s = __uint_as_float(f8_exponent(amax) << 23);
  const uint32_t w0 = f8_pack4(v, s), w1 = f8_pack4(v + 4, s);
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true));
  *reinterpret_cast<uint4*>(A.out + m * A.dp + c) = o;
}

// The product, a wave to 16 MB hidden rows x 16 NB vocabulary entries, with
// fragments straight from memory: A operand the weights (their 8 bits widened
// to bf16, exactly), Bt the hidden rows.  The products of a block of 128 are
// summed by four matrix instructions from zero and added to the running sum
// with the block's scale.
struct F8HeadArgs {
  const uint16_t* hidden;  // [M][dp] bf16
  int64_t M, V;
  int32_t d, dp, rows;
  const uint8_t* weight;
  int64_t w_stride;
  const float* scale;
  void* out;
  int64_t o_seq, o_pos;
};
template <typename TO, int MB, int NB>
__global__ __launch_bounds__(256) void k_lmhead_fp8(F8HeadArgs A) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n16 = lane & 15, q = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + w) * (16 * NB);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MB);
  if (v0 >= A.V) return;
  const int32_t blocks = A.dp / 128;
  f8_f32x4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
  const float* sp = A.scale + (v0 / 128) * blocks;  // 16 NB entries lie in one block of 128
  for (int32_t kb = 0; kb < blocks; ++kb) {
    f8_f32x4 c[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) c[mb][nb] = f8_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t col = kb * 128 + h * 64 + q * 16;
      uint4 wr[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int64_t v = v0 + 16 * nb + n16;
        wr[nb] = make_uint4(0u, 0u, 0u, 0u);
        if (v < A.V && col < A.d) wr[nb] = load16(A.weight + v * A.w_stride + col);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f8_bf16x8 hf[MB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const int64_t m = m0 + 16 * mb + n16;
          hf[mb] = __builtin_bit_cast(f8_bf16x8, load16(A.hidden + (m < A.M ? m : 0) * A.dp + col + 8 * s));
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t a = s ? wr[nb].z : wr[nb].x, b = s ? wr[nb].w : wr[nb].y;
          uint4 f;
          f.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false));
          f.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true));
          f.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false));
          f.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true));
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            c[mb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(f8_bf16x8, f), hf[mb],
                                                                c[mb][nb], 0, 0, 0);
        }
      }
    }
    const float s = sp[kb];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[mb][nb][r] = __builtin_fmaf(c[mb][nb][r], s, acc[mb][nb][r]);
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = m0 + 16 * mb + n16;
    if (m >= A.M) continue;
    const int64_t b = m / A.rows;
    TO* row = reinterpret_cast<TO*>(A.out) + b * A.o_seq + (m - b * A.rows) * A.o_pos;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t v = v0 + 16 * nb + 4 * q + r;
        if (v < A.V) {
          if constexpr (sizeof(TO) == 4) row[v] = acc[mb][nb][r];
          else row[v] = __builtin_bit_cast(uint16_t, (__bf16)acc[mb][nb][r]);
        }
      }
  }
}

}  // namespace sv
