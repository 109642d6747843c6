// sv_cache4_short.hpp -- attention over the 4-bit cache for many short sequences
// (gfx950, wave64).
#pragma once

#include "sv_cache4.hpp"

namespace sv {

// The mathematics and the operands' layout are those of k_attention_cache4.  That one
// gives the pages of a (sequence, kv head, block of rows) to the four waves of a
// workgroup, whose rows have then to be joined.  Where there are as many such
// segments as waves in flight, a wave goes through all of one's pages by itself, with nothing to
// share or to join: rows and their statistics stay in its registers, and its
// pages come through LDS buffers of its own, a page's two pairs of tiles at a time.
// 512 branches of up to 5 tokens, 32 heads on 8 of 128, up to 105 own tokens each and a
// record of F32 to take in: 30.8 us, 77 MB fetched; bound by a wave's chain of loads,
// products and exponentials (vector instructions in 41 % of the busy cycles).
template <int D, int RT>
struct C4Short {
  using Sh = C4Shape<D, RT>;
  static constexpr int kBuf = 2 * Sh::kUnit;  // of a wave
};

template <int D, int RT, typename Args>
__global__ __launch_bounds__(256, 2) void k_attention_cache4_short(Args A) {
  using Sh = C4Shape<D, RT>;
  constexpr int kRows = RT * 16, kRun = D / 16, NG = D / 32;
  __shared__ __attribute__((aligned(16))) uint8_t buffers[4][C4Short<D, RT>::kBuf];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, q = lane >> 4;
  const int32_t HR = A.cache.heads * A.row_blocks;
  const int64_t x = (int64_t)blockIdx.x * 4 + w;
  const int64_t b = x / HR;
  if (b >= A.B) return;
  const int32_t hr = (int32_t)(x - b * HR), h = hr / A.row_blocks, r0 = hr % A.row_blocks * kRows;
  bool bad;
  const int32_t pages = c4_pages<true>(A, b, bad);
  if (pages == 0) return;
  const int32_t s0 = c4_scalar(A.start + b);
  const int32_t nnew = c4_new(A, b, bad);
  bool faulty = bad;
  const int32_t ps = kC4Behind<Args> && !bad ? c4_behind<true>(A, b) : 0, np = c4_pages_of(ps);
  // pairs of tiles; the last page may hold no token in its second half
  const int32_t pairs = bad ? 0 : 2 * np + (int32_t)(((int64_t)s0 + nnew + 31) / 32);
  uint8_t* const buf = buffers[w];
  int32_t page = 0;
  auto fetch = [&](int32_t u) {
    if (u >= pairs) return;
    if (!(u & 1)) {
      const int32_t p = u / 2;
      if constexpr (kC4Behind<Args>)
        page = p < np ? c4_scalar(A.prefix.table + (b / A.fan) * A.prefix.table_stride + p)
                      : c4_scalar(A.cache.table + b * A.cache.table_stride + (p - np));
      else page = c4_scalar(A.cache.table + b * A.cache.table_stride + p);
      if ((uint32_t)page >= (uint32_t)A.cache.n_pages) {
        faulty = true;
        page = 0;
      }
    }
    c4_fetch<D>(A.cache.template record<D>(page, h), u & 1, lane, buf + (u & 1) * Sh::kUnit);
  };
  uint4 qx[RT][NG];
  int32_t tok[RT], heads[RT];  // this lane's rows: tokens, T past the last one
  int64_t seqs[RT];
  uint32_t live = 0;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    seqs[rt] = b;
    const bool have = c4_row(A, h, r0 + 16 * rt + n16, nnew, seqs[rt], tok[rt], heads[rt]);
    live |= (uint32_t)have << rt;
    const uint16_t* qp = A.q + b * A.q_seq + tok[rt] * A.q_pos + (int64_t)heads[rt] * A.q_head;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      qx[rt][j] = make_uint4(0u, 0u, 0u, 0u);
      if (have) qx[rt][j] = load16(qp + q * (D / 4) + 8 * j);
    }
  }
  c4_wait<0>();  // here, and not among the pages' loads at their first use
  fetch(0);
  fetch(1);
  C4State<D, RT> S;
  S.far = 0;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    S.m[rt] = S.less[rt] = kC4Low;
    S.l[rt] = S.n[rt] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) S.o[rt][i] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
  }
  auto rows_of = [&](int j, c4_bf16x8(&qf)[RT]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) qf[rt] = __builtin_bit_cast(c4_bf16x8, qx[rt][j]);
  };
#pragma unroll 1
  for (int32_t u = 0; u < pairs; ++u) {
    if (u + 1 < pairs) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Sh::kLoads) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const bool before = kC4Behind<Args> && u < 2 * np;  // a prefix has no new tokens
    const int64_t base = before ? (int64_t)32 * u - ps : (int64_t)32 * (u - 2 * np) - s0;
    const bool masked = base + 32 > 0;
    uint32_t sees[RT] = {}, valid = 0;
    if (masked) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        sees[rt] = !(live >> rt & 1) ? 0u : before ? c4_below(-base) : c4_sees(A, b, tok[rt], nnew, base);
      valid = c4_below((before ? 0 : nnew) - base);
    }
    c4_unit<D, RT>(buf + (u & 1) * Sh::kUnit, u & 1, rows_of, S, A.c, lane, masked, sees, valid);
    fetch(u + 2);
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float nan = __builtin_nanf("");
    const float sum = c4_sum_quads(S.l[rt]), rounded = c4_sum_quads(S.n[rt]);
    const float l = faulty ? nan : sum, n = faulty ? nan : rounded;
    if (!(live >> rt & 1)) continue;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float v[kRun];
#pragma unroll
      for (int e = 0; e < kRun; ++e) v[e] = S.o[rt][e][y];
      c4_finish<kRun>(A, seqs[rt], tok[rt], heads[rt], (4 * q + y) * kRun, v, S.m[rt], l, n);
    }
  }
}

}  // namespace sv
