// sv_rotate.hpp -- norms of queries and keys for each head with their rotation
// by position (gfx950, wave64).
#pragma once

#include "sv_device.hpp"

namespace sv {

struct RotHeads {
  const void* in;
  void* out;
  const void* weight;                       // or null
  int64_t seq, pos, head;                   // strides of `in`, in elements
  int64_t out_seq, out_pos, out_head;
  int32_t heads;
};

struct RotateArgs {
  RotHeads x[2];          // queries, keys
  const float* inv_freq;
  const int32_t* start;
  const int32_t* count;   // or null: T
  const int32_t* depth;   // or null: i
  int64_t depth_seq;
  int64_t tokens;         // B T
  int32_t T, D, rot, interleaved, norm;
  int32_t weight_f32;
  float eps;
  int32_t chunks, per;    // waves of a token, and each one's rounds of 64 / LANES heads
};

// cos and sin of `angle` whole turns: what passes a turn is dropped in 64 bits.
__device__ __forceinline__ void rot_turn(double turns, float& c, float& s) {
  const float part = (float)(turns - __builtin_rint(turns));
  sincospif(2.0f * part, &s, &c);
}

__device__ __forceinline__ void rot_load(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void rot_load(const uint16_t* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void rot_store(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void rot_store(uint16_t* p, const float (&x)[8]) {
  typedef __bf16 B8 __attribute__((ext_vector_type(8)));
  B8 y;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = (__bf16)x[e];
  *reinterpret_cast<B8*>(p) = y;
}

template <int LANES>
__device__ __forceinline__ float rot_sum(float x) {
#pragma unroll
  for (int off = 1; off < LANES; off <<= 1) x += __shfl_xor(x, off);
  return x;
}
template <int LANES>
__device__ __forceinline__ float rot_max(float x) {
#pragma unroll
  for (int off = 1; off < LANES; off <<= 1) x = fmaxf(x, __shfl_xor(x, off));
  return x;
}

// y = x / sqrt(mean x^2 + eps) w for each head, then pairs (a, b) of its first `rot`
// values become (a cos t - b sin t, b cos t + a sin t), t = (start + depth) inv_freq.
// All of it is F32, but for the angle: a product of 2^30 and a frequency needs more
// bits than F32 has, so that it is taken in 64 bits and brought into one turn there.
// The one rounding to fewer bits is that of a BF16 output.
// Bound by memory for prompts (4 x 8,191 tokens of 32 + 8 heads of 128, BF16: 671 MB
// in 141 us, 4.7 TB/s, where a copy reaches 5.1), by its launch and one chain of
// loads for a step (64 x 6 tokens 6.8 us, one token 4.0).
// A thread holds 8 neighbouring values of a head, LANES of them a head (those past
// D / 8 none), a wave 64 / LANES heads of one token, whose angles it makes
// once for all the heads that it goes through, queries first.
template <typename TI, typename TO, int LANES>
__global__ __launch_bounds__(256) void k_norm_rotate(RotateArgs A) {
  constexpr int kHeads = 64 / LANES;
  const int lane = threadIdx.x & 63, u = lane % LANES;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t token = wave / A.chunks;
  if (token >= A.tokens) return;
  const int64_t b = token / A.T;
  const int32_t i = (int32_t)(token - b * A.T);
  const int32_t n = A.count ? A.count[b] : A.T;
  const bool bad = n < 0 || n > A.T;
  if (!bad && i >= n) return;

  // Angles of this thread's pairs: where pairs are neighbours 4, else 8, the
  // other halves being those of the thread rot / 16 further on or back.
  const int half = A.rot / 2, d = 8 * u;
  const bool turned = d < A.rot, second = d >= half;
  const int far = A.rot / 16;  // threads to the other half
  float cs[8], sn[8];
  if (turned) {
    const double at = (double)((int64_t)A.start[b] + (A.depth ? A.depth[b * A.depth_seq + i] : i));
    const float* f = A.inv_freq + (A.interleaved ? 4 * u : second ? d - half : d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e >= 4 && A.interleaved) break;
      rot_turn(at * ((double)f[e] * 0.15915494309189535), cs[e], sn[e]);  // 1 / (2 pi)
    }
  }
  const int partner = lane + (second ? -far : far);

  // rounds of kHeads heads, the queries' before the keys'
  const int32_t rounds_q = (A.x[0].heads + kHeads - 1) / kHeads;
  const int32_t rounds = rounds_q + (A.x[1].heads + kHeads - 1) / kHeads;
  const int32_t first = (int32_t)(wave - token * A.chunks) * A.per;
  const int32_t last = min(first + A.per, rounds);
  for (int32_t r = first; r < last; ++r) {
    const RotHeads& X = r < rounds_q ? A.x[0] : A.x[1];
    const int32_t h = (r < rounds_q ? r : r - rounds_q) * kHeads + lane / LANES;
    const bool live = h < X.heads && d < A.D;
    float x[8] = {};
    if (live) rot_load(reinterpret_cast<const TI*>(X.in) + b * X.seq + i * X.pos + h * X.head + d, x);
    if (A.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
      ss = rot_sum<LANES>(ss);
      // the squares' sum in F32's range: as a rule
      float scale = 1.0f, inv = __builtin_amdgcn_rsqf(ss * (1.0f / (float)A.D) + A.eps);
      if (!(ss < 0x1p120f) || ss < 0x1p-90f) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_fabsf(x[e]));
        top = rot_max<LANES>(top);
        // a power of two that brings the largest value to [1, 2), as far as one of F32's does
        const int32_t ex = min(max(127 - (int32_t)(__float_as_uint(top) >> 23), -126), 126);
        scale = top > 0.f ? __uint_as_float((uint32_t)(127 + ex) << 23) : 1.0f;
        ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = x[e] * scale;
          ss = __builtin_fmaf(y, y, ss);
        }
        ss = rot_sum<LANES>(ss);
        // eps scale^2 has room in 64 bits
        const double mean = (double)ss / A.D + (double)A.eps * scale * scale;
        inv = (float)(1.0 / sqrt(mean));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * inv;
      if (X.weight && live) {
        float w[8];
        if (A.weight_f32) rot_load(reinterpret_cast<const float*>(X.weight) + d, w);
        else rot_load(reinterpret_cast<const uint16_t*>(X.weight) + d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= w[e];
      }
    }
    if (A.rot) {
      if (A.interleaved) {
        if (turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = p * cs[e] - q * sn[e];
            x[2 * e + 1] = q * cs[e] + p * sn[e];
          }
        }
      } else {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl(x[e], partner);
        if (turned) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = second ? x[e] * cs[e] + o[e] * sn[e] : x[e] * cs[e] - o[e] * sn[e];
        }
      }
    }
    if (bad) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __builtin_nanf("");
    }
    if (live) rot_store(reinterpret_cast<TO*>(X.out) + b * X.out_seq + i * X.out_pos + h * X.out_head + d, x);
  }
}

}  // namespace sv
