// sv_cache4_wide.hpp -- attention over the 4-bit cache for many rows of a kv
// head: the waves of a workgroup share each page's converted keys and values
// (gfx950, wave64).
#pragma once

#include "sv_cache4.hpp"

namespace sv {

// The mathematics, the operands' layout and the split into equal shares are those
// of k_attention_cache4.  There each wave converts the codes of its own pages
// for the rows of one block; with rows for several blocks that is the same
// conversion several times.  Here the waves of a workgroup hold up to RT tiles
// of 16 rows each and go through the same pages together: each converts its part
// of a page's codes to bf16 and puts them into LDS, as the operands that every
// wave then reads, while the page before is attended to.
// 4 prefixes of up to 8,155 tokens, 378 rows on each of 4 heads of 256: 55 us, matrix
// units 25 % and vector instructions 34 % of the busy cycles, 78 MB fetched; a page
// takes its workgroup about 3 us, the ends of a segment 17.  What bounds it is the
// barrier after each page, behind which converting, scores, exponentials and the
// second product follow each other; scores of the next page begun before it gained
// nothing.
template <int D>
struct C4Wide {
  static_assert(D == 128 || D == 256, "heads of 64 gain nothing by it");
  static constexpr int RT = D == 256 ? 1 : 3;
  static constexpr int kWaves = D == 256 ? 8 : 4;
  static constexpr int kTiles = kWaves * RT, kRows = 16 * kTiles;  // of a block at most
  static constexpr int kPerCu = 8 / kWaves;                        // workgroups a compute unit: two waves a SIMD
  static constexpr int kGrid = 256 * kPerCu;
  static constexpr int kKeys = 64 * D * 2;                         // bytes of a page's keys, or values, in bf16
  static constexpr int kCost = 8;   // pages that a segment's ends cost
  // Whether calls whose live rows are counted through come here: of heads of 128 they
  // gain nothing (64 x 8 heads, 96 of 160 rows live: 185 us by k_attention_cache4, 190).
  static constexpr bool kCounted = D == 256;
  // What a pair of waves with the same rows hands over: float4s of O, floats of m, l, n.
  static constexpr int kHandO = RT * (D / 16) * 64, kHandStats = 3 * RT * 64;
  static constexpr int kStats = kWaves / 2 * kHandStats;
  static_assert(kWaves / 2 * kHandO * 16 <= 4 * kKeys, "in two pages' buffers");
  // A cut segment: O [kRows][D], m, l, n [kRows], and what the rows are.
  static constexpr int64_t kFloats = kRows * (D + 5);
};
// What a row is: its sequence (-1: none) and token.
struct C4RowMap {
  int32_t seq, tok;
};
// A wave's tiles of a block's rows.
struct C4Share {
  int32_t tiles, mine, row0;  // of the block; this wave's, and the first row of them
  bool half;                  // two waves have the same rows
};
// Neighbouring tiles to a wave; where half the waves hold them all, two waves
// have the same.
template <int D>
__host__ __device__ __forceinline__ C4Share c4_wave_share(int32_t rows, int w) {
  using Sh = C4Wide<D>;
  C4Share x;
  x.tiles = (rows + 15) / 16;
  x.half = x.tiles <= Sh::kTiles / 2;
  const int W = x.half ? Sh::kWaves / 2 : Sh::kWaves, v = x.half ? w >> 1 : w;
  const int more = x.tiles % W;  // waves that have a tile more
  x.mine = x.tiles / W + (v < more);
  x.row0 = 16 * (x.tiles / W * v + (v < more ? v : more));
  return x;
}
// Where wave w's pair of waves with the same rows hands them over: its float4s of O
// in the pages' buffers, and its floats of m, l and n.  Each pair has room for as many
// tiles as one can have, however many it has: of a block of 3 or 5 tiles one pair has
// one more than the other.
struct C4HandOver {
  int32_t o, stats;
};
template <int D>
__host__ __device__ constexpr C4HandOver c4_hand_over(int w) {
  using Sh = C4Wide<D>;
  return {(w >> 1) * Sh::kHandO, (w >> 1) * Sh::kHandStats};
}
// Finds a wave's rows in the block of `rows` rows whose first one is r0, and puts
// down what they are.
template <int D, typename Args>
__device__ __forceinline__ C4Share c4_map_rows(const Args& A, int32_t rows, int64_t b, int32_t r0, int32_t nnew, int w,
                                               int lane, C4RowMap* map) {
  const int32_t upto = c4_rows_upto(A, b, lane);
  int32_t all = c4_rows(A);
  if constexpr (kC4Prefix<Args>)
    if (A.compact) all = __builtin_amdgcn_readlane(upto, 63);
  const C4Share x = c4_wave_share<D>(min(max(all - r0, 0), rows), w);
#pragma unroll
  for (int r = 0; r < 16 * C4Wide<D>::RT; r += 64) {
    int64_t bb = b;
    int32_t i = 0, head;
    const bool live = c4_any_row(A, upto, 0, r0 + x.row0 + r + lane, nnew, bb, i, head);
    if (r + lane < 16 * x.mine) map[r + lane] = {live ? (int32_t)bb : -1, i};
  }
  return x;
}

// A thread's part of a page's codes.  Of the keys a wave has a tile, lane (n, q)
// elements of token n from q D / 4 on, D / 4 of them; of the values four tokens
// in a sixteenth of D.  With eight waves two have a tile, and half of each lane's.
template <int D>
struct C4Codes {
  uint32_t k[4], v[4], ke, ve;
};

__device__ __forceinline__ void c4_load_dwords(const uint8_t* p, uint32_t (&x)[4]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}

// Where a thread's values stand: its tile of 16 tokens and, of it, the four, in
// which sixteenth of D.
struct C4ValuePlace {
  int tile, quad, part;
};
__device__ __forceinline__ C4ValuePlace c4_value_place(int w, int lane) {
  // neighbouring lanes: the same four of a pair of tiles, so that their halves of
  // an operand's 16 bytes stand side by side
  return {(w & 2) + (lane & 1), 2 * (w & 1) + (lane >> 5), (lane >> 1) & 15};
}

template <int D>
__device__ __forceinline__ void c4_load_keys(const uint8_t* rec, int w, int lane, C4Codes<D>& R) {
  constexpr int NG = D / 32;
  const int n = lane & 15, q = lane >> 4, half = w >> 2;
  c4_load_dwords(rec + (16 * (w & 3) + n) * (D / 2) + q * (D / 8) + 16 * half, R.k);
  R.ke = *reinterpret_cast<const uint32_t*>(rec + C4<D>::kKeyExp + (q * NG / 4 + half) * 64 + n * 4);
}
template <int D>
__device__ __forceinline__ void c4_load_values(const uint8_t* rec, int w, int lane, C4Codes<D>& R) {
  constexpr int NG = D / 32;
  const C4ValuePlace V = c4_value_place(w, lane);
  const int four = 4 * V.tile + V.quad;
  const uint8_t* const p = rec + C4<D>::kVal + (four * 16 + V.part) * (4 * NG);
  if constexpr (D == 256) {
#pragma unroll
    for (int j = 0; j < 4; ++j) R.v[j] = *reinterpret_cast<const uint32_t*>(p + 8 * j + 4 * (w >> 2));
  } else {
    c4_load_dwords(p, R.v);
  }
  R.ve = *reinterpret_cast<const uint32_t*>(rec + C4<D>::kValExp + four * (4 * NG) + (V.part * NG / 16) * 4);
}

// Converts them into a page's operands: keys [4 tiles][D / 32][64 lanes] and
// values [2 pairs of tiles][D / 16][64 lanes], 16 bytes each.
template <int D>
__device__ __forceinline__ void c4_convert_keys(const C4Codes<D>& R, int w, int lane, uint8_t* keys) {
  constexpr int NG = D / 32, N = 4;
  const float sc = __uint_as_float(((R.ke >> (8 * (w & 3))) & 0xFFu) << 23);
  uint8_t* const to = keys + (((w & 3) * NG + N * (w >> 2)) * 64 + lane) * 16;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint4 a;
    a.x = c4_cvt(R.k[j], sc, 0);
    a.y = c4_cvt(R.k[j], sc, 1);
    a.z = c4_cvt(R.k[j], sc, 2);
    a.w = c4_cvt(R.k[j], sc, 3);
    *reinterpret_cast<uint4*>(to + j * 1024) = a;
  }
}
// `have`: tokens of the page; what stands past them are no values: zeros with an
// exponent of 1.
template <int D>
__device__ __forceinline__ void c4_convert_values(C4Codes<D>& R, int w, int lane, int have, uint8_t* values) {
  constexpr int N = 4;  // bytes of a token's values here
  const C4ValuePlace V = c4_value_place(w, lane);
  if (have < 64) {
    const int left = have - 16 * V.tile - 4 * V.quad;  // of the four
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j >= left) {
        R.ve = (R.ve & ~(0xFFu << (8 * j))) | (127u << (8 * j));
        R.v[j] = 0u;
      }
  }
  float sc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sc[j] = c4_byte_scale(R.ve, j);
  uint8_t* const to = values + (((w >> 1 & 1) * (D / 16) + 2 * N * (w >> 2)) * 64 + V.quad * 16 + V.part) * 16 + (lane & 1) * 8;
#pragma unroll
  for (int y = 0; y < N; ++y) {
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = c4_cvt(R.v[(j * N + y) / 4], sc[j], (j * N + y) % 4);
    uint2 lo, hi;
    lo.x = __builtin_amdgcn_perm(a[1], a[0], 0x05040100u);
    lo.y = __builtin_amdgcn_perm(a[3], a[2], 0x05040100u);
    hi.x = __builtin_amdgcn_perm(a[1], a[0], 0x07060302u);
    hi.y = __builtin_amdgcn_perm(a[3], a[2], 0x07060302u);
    *reinterpret_cast<uint2*>(to + (2 * y) * 1024) = lo;
    *reinterpret_cast<uint2*>(to + (2 * y + 1) * 1024) = hi;
  }
}

// A barrier behind the wave's own LDS writes; __syncthreads would wait for the
// loads under way too.
__device__ __forceinline__ void c4_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The query head of row r of kv head h: rows stand token by token.
__device__ __forceinline__ int32_t c4_head(const C4AttnArgs& A, int32_t h, int32_t r) { return h * A.G + r % A.G; }

// A page's record; one outside the pool stands for page 0 and marks the rows.
template <int D>
__device__ __forceinline__ const uint8_t* c4_page_record(const C4AttnArgs& A, int32_t page, int32_t h, bool& faulty) {
  if ((uint32_t)page >= (uint32_t)A.cache.n_pages) {
    faulty = true;
    page = 0;
  }
  return A.cache.record<D>(page, h);
}

// A segment's work: the pages p0 .. end - 1 of sequence (or prefix) b in kv head h.
struct C4Segment {
  int64_t b;
  int32_t h, r0, s0, nnew;
  int32_t p0, p1, pages, end;
  C4Gap gap;
  bool faulty;
};

// Has N parts of an operand read from LDS, FEW ahead of the NT products that each
// of them goes into.
template <int N, int FEW, int NT>
__device__ __forceinline__ void c4_in_turn() {
  __builtin_amdgcn_sched_group_barrier(0x100, FEW, 0);  // LDS reads
#pragma unroll
  for (int x = 0; x < N - FEW; ++x) {
    __builtin_amdgcn_sched_group_barrier(0x8, NT, 0);   // matrix instructions
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x8, NT * FEW, 0);
}

// The segment's pages for a wave's NT tiles of rows, the first of them row
// `row0` of the block.  HALF: two waves have the same rows, one the first pair of
// tiles of each page, the other the second.
template <int D, int NT, bool HALF, typename Args>
__device__ __forceinline__ void c4_wide_run(const Args& A, C4Segment G, uint8_t (&pagebuf)[2][2][C4Wide<D>::kKeys],
                                            const C4RowMap* map, int32_t row0, C4Codes<D>& R4, int32_t ahead, int w, int lane, float* part, float* stats) {
  using Sh = C4Wide<D>;
  constexpr int NG = D / 32, kRun = D / 16, RT = NT ? NT : 1;
  // An operand's parts wait in registers while the work before them is done,
  // where there are registers for that.
  constexpr bool kAhead = NT > 0 && D * NT <= 256;
  constexpr int kFew = 4;  // else so many parts
  const int n16 = lane & 15, q = lane >> 4;
  auto place = [&](int32_t p) { return kC4Window<Args> && p >= G.gap.keep ? p + G.gap.skip : p; };
  bool faulty = G.faulty;
  auto page_of = [&](int32_t p) {
    return p < G.end ? c4_scalar(A.cache.table + G.b * A.cache.table_stride + place(p)) : 0;
  };
  auto record = [&](int32_t page) { return c4_page_record<D>(A, page, G.h, faulty); };
  const C4RowMap* const mine = map + n16;  // this lane's rows, 16 apart
  uint4 qx[RT][NG];
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    const int32_t head = c4_head(A, G.h, G.r0 + row0 + 16 * rt + n16);
    const C4RowMap x = mine[16 * rt];
    const uint16_t* qp = A.q + x.seq * A.q_seq + x.tok * A.q_pos + (int64_t)head * A.q_head;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      qx[rt][j] = make_uint4(0u, 0u, 0u, 0u);
      if (x.seq >= 0) qx[rt][j] = load16(qp + q * (D / 4) + 8 * j);
    }
  }
  C4State<D, RT> S;
  S.far = 0;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    S.m[rt] = S.less[rt] = kC4Low;
    S.l[rt] = S.n[rt] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) S.o[rt][i] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // The position of page p's first token relative to the new ones', and its tokens.
  auto base_of = [&](int32_t p) { return (int64_t)place(p) * kC4Page - G.s0; };
  auto have_of = [&](int32_t p) {
    const int64_t have = G.nnew - base_of(p);
    return have < 64 ? (int)have : 64;
  };
  // What the rows see of the 32 positions from `at` on, if that is not all of them.
  auto seen = [&](int64_t at, uint32_t (&sees)[RT]) -> bool {
    bool masked = at + 32 > 0;
    if constexpr (kC4Window<Args>)  // or the last token's window ends behind, and these are not all sinks
      masked |= at <= (int64_t)A.T - 1 - A.window && at + G.s0 + 32 > A.sinks;
    if (!masked) return false;
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      if constexpr (kC4Prefix<Args>) {
        sees[rt] = c4_below(-at);
      } else {
        const C4RowMap x = mine[16 * rt];
        sees[rt] = x.seq < 0 ? 0u : c4_sees(A, G.b, x.tok, G.nnew, at);
        if constexpr (kC4Window<Args>)
          if (x.seq >= 0) sees[rt] &= c4_in_window(A, G.s0, (int64_t)c4_depth(A, G.b, x.tok) - A.window + 1, at);
      }
    }
    return true;
  };
  // The last page is converted again where there is none behind it.
  const int32_t last = G.end - 1;
  if (G.p0 < G.end) {
    c4_convert_keys<D>(R4, w, lane, pagebuf[0][0]);
    c4_convert_values<D>(R4, w, lane, have_of(G.p0), pagebuf[0][1]);
    const uint8_t* const rec = record(ahead);
    c4_load_keys<D>(rec, w, lane, R4);
    c4_load_values<D>(rec, w, lane, R4);
    ahead = page_of(min(G.p0 + 2, last));
  }
  c4_barrier();
  for (int32_t p = G.p0; p < G.end; ++p) {
    const uint8_t* const keys = pagebuf[(p - G.p0) & 1][0];
    const uint8_t* const values = keys + Sh::kKeys;
    uint8_t* const next = pagebuf[(p - G.p0 + 1) & 1][0];
    const int64_t base = base_of(p);
    // made anew each time: kept for the loop, the addresses below cost registers
    int at = lane;
    asm volatile("" : "+v"(at));
    auto pair_of = [&](int pair) {
      uint32_t sees[RT] = {};
      const bool masked = seen(base + 32 * pair, sees);
      auto key = [&](int i, int j) {
        return *reinterpret_cast<const c4_bf16x8*>(keys + (((2 * pair + i) * NG + j) * 64 + at) * 16);
      };
      auto value = [&](int e) {
        return *reinterpret_cast<const c4_bf16x8*>(values + ((pair * (D / 16) + e) * 64 + at) * 16);
      };
      c4_f32x4 s[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) s[rt][i] = c4_f32x4{0.f, 0.f, 0.f, 0.f};
      constexpr int kKeyParts = kAhead ? 2 * NG : kFew;  // in registers at a time
      c4_bf16x8 kf[kKeyParts];
#pragma unroll
      for (int x = 0; x < kKeyParts; ++x) kf[x] = key(x % 2, x / 2);
#pragma unroll
      for (int x = 0; x < 2 * NG; ++x) {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
          s[rt][x % 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              kf[x % kKeyParts], __builtin_bit_cast(c4_bf16x8, qx[rt][x / 2]), s[rt][x % 2], 0, 0, 0);
        if (x + kKeyParts < 2 * NG) kf[x % kKeyParts] = key((x + kKeyParts) % 2, (x + kKeyParts) / 2);
      }
      if constexpr (!kAhead) c4_in_turn<2 * NG, kFew, NT>();
      constexpr int kParts = kAhead ? D / 16 : kFew;
      c4_bf16x8 vf[kParts];
#pragma unroll
      for (int e = 0; e < kParts; ++e) vf[e] = value(e);
      __builtin_amdgcn_sched_barrier(0);
      c4_bf16x8 pr[RT];
      c4_probabilities<D, RT>(s, S, A.c, q, masked, sees, pr);
      if constexpr (kAhead) {
        // the next page's keys, or values, beside the products
        if (HALF || pair == 0) c4_convert_keys<D>(R4, w, at, next);
        if (HALF || pair == 1) c4_convert_values<D>(R4, w, at, have_of(min(p + 1, last)), next + Sh::kKeys);
      }
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
          S.o[rt][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[e % kParts], pr[rt], S.o[rt][e], 0, 0, 0);
        if (e + kParts < D / 16) vf[e % kParts] = value(e + kParts);
      }
      if constexpr (!kAhead) c4_in_turn<D / 16, kFew, NT>();
    };
    if constexpr (NT > 0 && HALF) {
      pair_of(w & 1);
    } else if constexpr (NT > 0 && kAhead) {
      pair_of(0);
      pair_of(1);
    } else if constexpr (NT > 0) {
#pragma unroll 1
      for (int pair = 0; pair < 2; ++pair) pair_of(pair);
    }
    if constexpr (!kAhead) {
      c4_convert_keys<D>(R4, w, at, next);
      c4_convert_values<D>(R4, w, at, have_of(min(p + 1, last)), next + Sh::kKeys);
    }
    const uint8_t* const rec = record(ahead);
    c4_load_keys<D>(rec, w, at, R4);
    c4_load_values<D>(rec, w, at, R4);
    ahead = page_of(min(p + 3, last));
    c4_barrier();
  }
  if constexpr (HALF) {  // the two waves of the same rows: the second's go to the first
    const C4HandOver to = c4_hand_over<D>(w);
    float4* const o = reinterpret_cast<float4*>(pagebuf) + to.o + lane;
    float* const st = stats + to.stats + lane;
    if (w & 1) {
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
          o[(rt * (D / 16) + e) * 64] = make_float4(S.o[rt][e][0], S.o[rt][e][1], S.o[rt][e][2], S.o[rt][e][3]);
        st[(3 * rt) * 64] = S.m[rt];
        st[(3 * rt + 1) * 64] = S.l[rt];
        st[(3 * rt + 2) * 64] = S.n[rt];
      }
    }
    c4_barrier();
    if (w & 1) return;
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      const float m = st[(3 * rt) * 64], top = fmaxf(S.m[rt], m);
      const float f = __builtin_amdgcn_exp2f(S.m[rt] - top), g = __builtin_amdgcn_exp2f(m - top);
      S.m[rt] = top;
      S.l[rt] = S.l[rt] * f + st[(3 * rt + 1) * 64] * g;
      S.n[rt] = S.n[rt] * f + st[(3 * rt + 2) * 64] * g;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const float4 v = o[(rt * (D / 16) + e) * 64];
        S.o[rt][e] = S.o[rt][e] * f + c4_f32x4{v.x, v.y, v.z, v.w} * g;
      }
    }
  }
  const bool whole = G.p0 == 0 && G.p1 == G.pages;
  const float nan = __builtin_nanf("");
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    const float sum = c4_sum_quads(S.l[rt]), rounded = c4_sum_quads(S.n[rt]);
    const float l = faulty ? nan : sum, n = faulty ? nan : rounded;
    const int32_t row = row0 + 16 * rt + n16, head = c4_head(A, G.h, G.r0 + row);
    const C4RowMap x = mine[16 * rt];
    if (!whole && q == 0) {
      float* const p = part + Sh::kRows * D + row;
      p[0] = S.m[rt];
      p[Sh::kRows] = l;
      p[2 * Sh::kRows] = n;
      reinterpret_cast<int32_t*>(p)[3 * Sh::kRows] = x.seq;
      reinterpret_cast<int32_t*>(p)[4 * Sh::kRows] = x.tok;
    }
    if (x.seq < 0) continue;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int d0 = (4 * q + y) * kRun;
      float v[kRun];
#pragma unroll
      for (int e = 0; e < kRun; ++e) v[e] = S.o[rt][e][y];
      if (whole) {
        c4_finish<kRun>(A, x.seq, x.tok, head, d0, v, S.m[rt], l, n);
      } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e) part[row * D + d0 + e] = v[e];
      }
    }
  }
}

// EACH: a workgroup a segment, none of which is cut.
template <int D, typename Args, bool EACH>
__global__ __launch_bounds__(64 * C4Wide<D>::kWaves, C4Wide<D>::kPerCu) void k_attention_cache4_wide(Args A, int32_t block_rows) {
  using Sh = C4Wide<D>;
  __shared__ __attribute__((aligned(16))) uint8_t pagebuf[2][2][Sh::kKeys];
  __shared__ C4RowMap maps[Sh::kWaves][16 * Sh::RT];
  __shared__ float stats[Sh::kStats];

  if constexpr (kC4Prefix<Args> && !Sh::kCounted) A.compact = 0;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t per = (A.B + 63) / 64;
  const int32_t HR = c4_times(A);
  int64_t before = 0, share = 1, lo = 0, hi = 1;
  if (!EACH) {
    const int64_t all = c4_plan<Sh::kCost>(A, lane, per, before) * HR;  // weight of all segments
    share = c4_share<Sh::kGrid, Sh::kCost>(all);
    lo = (int64_t)blockIdx.x * share;
    hi = min(lo + share, all);
  }
  int32_t cut_b = 0, cut_hr = 0, cut_new = 0, cut_parts = 0, cut_slot = 0;
  auto note = [&] {
    if (A.split && tid == 0) A.cuts[blockIdx.x] = {cut_b, cut_hr, cut_new, cut_parts, cut_slot, {0, 0, 0}};
  };
  if (lo >= hi) {
    note();
    return;
  }
  int64_t seq_at = 0;
  C4Segment G;
  if (EACH) G.b = blockIdx.x / (uint32_t)(A.cache.heads * A.row_blocks);
  else G.b = c4_find<Sh::kCost>(A, lane, per, before, c4_div(lo, HR), seq_at);
  bool bad;
  G.pages = c4_pages<true>(A, G.b, bad);
  int32_t nb = c4_blocks<true>(A, G.b);
  int32_t hr = EACH ? (int32_t)(blockIdx.x % (uint32_t)(A.cache.heads * A.row_blocks))
                      : (int32_t)c4_div(lo - seq_at * HR, c4_weight<Sh::kCost>(G.pages));
  if (EACH && G.pages == 0) return;
  int64_t seg = EACH ? 0 : seq_at * HR + hr * c4_weight<Sh::kCost>(G.pages);  // where it begins
  for (; seg < hi; seg += c4_weight<Sh::kCost>(G.pages), ++hr) {
    if (hr == A.cache.heads * nb) {  // the next sequence with pages (seg is its begin)
      do {
        G.pages = c4_pages<true>(A, ++G.b, bad);
        nb = c4_blocks<true>(A, G.b);
      } while (G.pages == 0 || nb == 0);
      hr = 0;
    }
    G.p0 = c4_cut<Sh::kCost>(lo - seg, G.pages), G.p1 = c4_cut<Sh::kCost>(hi - seg, G.pages);
    if (!A.split) G.p0 = 0, G.p1 = seg < lo ? 0 : G.pages;  // whole, where it begins
    if (G.p0 == G.p1) continue;  // its pages are another workgroup's
    G.h = hr / nb;
    G.r0 = hr % nb * block_rows;
    G.s0 = c4_scalar(A.start + G.b);
    G.nnew = c4_new(A, G.b, bad);
    G.gap = C4Gap{0, 0};
    if constexpr (kC4Window<Args>)
      if (!bad) G.gap = c4_gap(A.window, A.sinks, G.s0, G.nnew);
    G.faulty = bad;
    G.end = bad ? G.p0 : G.p1;
    if (kC4Prefix<Args> && G.s0 == 0) G.end = G.p0;  // its page stands for none
    // The first page's codes are on their way while the rows are found.
    C4Codes<D> codes{};
    int32_t ahead = 0;
    if (G.p0 < G.end) {
      auto at = [&](int32_t p) {
        const int32_t x = kC4Window<Args> && p >= G.gap.keep ? p + G.gap.skip : p;
        return A.cache.table + G.b * A.cache.table_stride + x;
      };
      const uint8_t* const rec = c4_page_record<D>(A, c4_scalar(at(G.p0)), G.h, G.faulty);
      ahead = c4_scalar(at(min(G.p0 + 1, G.end - 1)));
      c4_load_keys<D>(rec, w, lane, codes);
      c4_load_values<D>(rec, w, lane, codes);
    }
    const C4Share W = c4_map_rows<D>(A, block_rows, G.b, G.r0, G.nnew, w, lane, maps[w]);
    const int32_t tiles = __builtin_amdgcn_readfirstlane(W.tiles);
    if (tiles == 0) continue;
    if (G.p0 == 0 && G.p1 < G.pages) {
      cut_b = (int32_t)G.b, cut_hr = G.h * A.row_blocks + hr % nb, cut_new = tiles, cut_slot = seg > lo ? 1 : 0;
      cut_parts = (int32_t)c4_div(seg + Sh::kCost + G.pages - 1, share) - blockIdx.x + 1;
    }
    const int32_t mine = __builtin_amdgcn_readfirstlane(W.mine), row0 = __builtin_amdgcn_readfirstlane(W.row0);
    const bool half = tiles <= Sh::kTiles / 2;
    float* const part = A.parts + ((int64_t)blockIdx.x * 2 + (seg > lo ? 1 : 0)) * Sh::kFloats;
    c4_barrier();  // the buffers are free
    auto run = [&](auto n) {
      if (half) c4_wide_run<D, n, true>(A, G, pagebuf, maps[w], row0, codes, ahead, w, lane, part, stats);
      else c4_wide_run<D, n, false>(A, G, pagebuf, maps[w], row0, codes, ahead, w, lane, part, stats);
    };
    if (mine == 0) run(std::integral_constant<int, 0>());
    else if (mine == 1) run(std::integral_constant<int, 1>());
    else if (mine == 2) run(std::integral_constant<int, Sh::RT >= 2 ? 2 : 0>());
    else run(std::integral_constant<int, Sh::RT >= 3 ? 3 : 0>());
  }
  note();
}

// Joins the cut segments: a workgroup a tile of 16 rows of the segment that
// workgroup blockIdx.x of the attention began.  Sixteen threads hold a row's
// columns, four in each 64; SHARE times as many share its records.
template <int D, int SHARE, typename Args>
__global__ __launch_bounds__(256 * SHARE) void k_attention_cache4_wide_join(Args A, int32_t block_rows) {
  using Sh = C4Wide<D>;
  constexpr int E = D / 16, N = 4;  // columns of a thread; records under way at a time
  __shared__ float vs[SHARE > 1 ? SHARE : 1][SHARE > 1 ? 16 : 1][SHARE > 1 ? D + 1 : 1], st[SHARE][3][16];
  const auto* cp = A.cuts + blockIdx.x;
  const int32_t parts = c4_scalar(&cp->parts);
  if (parts == 0 || (int32_t)blockIdx.y >= c4_scalar(&cp->nnew)) return;  // nnew: its tiles
  const int32_t hr = c4_scalar(&cp->hr), slot = c4_scalar(&cp->slot);
  const int part = threadIdx.x >> 8, r = (threadIdx.x >> 4) & 15, grp = threadIdx.x & 15;
  const int32_t row = blockIdx.y * 16 + r;
  const float* const rest = A.parts + (int64_t)blockIdx.x * 2 * Sh::kFloats;
  const float* const first = rest + slot * Sh::kFloats;
  const float* const what = first + Sh::kRows * (D + 3) + row;
  const int32_t seq = reinterpret_cast<const int32_t*>(what)[0], tok = reinterpret_cast<const int32_t*>(what)[Sh::kRows];
  const int32_t each = (parts + SHARE - 1) / SHARE, x0 = min(part * each, parts), x1 = min(x0 + each, parts);
  float m = kC4Low, l = 0.f, n = 0.f, v[E] = {};
  for (int32_t base = x0; base < x1; base += N) {
    float pm[N], pl[N], pn[N], o[N][E];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int32_t x = min(base + k, x1 - 1);
      const float* p = x == 0 ? first : rest + x * (2 * Sh::kFloats);
      pm[k] = p[Sh::kRows * D + row];
      pl[k] = p[Sh::kRows * (D + 1) + row];
      pn[k] = p[Sh::kRows * (D + 2) + row];
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(&o[k][e]) = *reinterpret_cast<const float4*>(p + row * D + 16 * e + 4 * grp);
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
  if constexpr (SHARE > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) vs[part][r][e * 16 + grp] = v[e];
    if (grp == 0) st[part][0][r] = m, st[part][1][r] = l, st[part][2][r] = n;
    __syncthreads();
    if (part) return;
    m = kC4Low;
#pragma unroll
    for (int x = 0; x < SHARE; ++x) m = fmaxf(m, st[x][0][r]);
    l = n = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll
    for (int x = 0; x < SHARE; ++x) {
      const float f = __builtin_amdgcn_exp2f(st[x][0][r] - m);
      l += st[x][1][r] * f;
      n += st[x][2][r] * f;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += vs[x][r][e * 16 + grp] * f;
    }
  }
  if (seq < 0) return;
  const int32_t head = c4_head(A, hr / A.row_blocks, hr % A.row_blocks * block_rows + row);
#pragma unroll
  for (int e = 0; e < E; e += 4) c4_finish<4>(A, seq, tok, head, 16 * e + 4 * grp, v + e, m, l, n);
}

}  // namespace sv
