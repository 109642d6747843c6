// sv_cache4_host.hpp -- what the C ABI calls over the 4-bit cache share on the
// host: argument checks, the attention's shapes and its launch.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "specverify_lowbit.h"
#include "sv_cache4.hpp"
#include "sv_cache4_wide.hpp"

namespace {

constexpr int64_t kMaxWorkItems = (int64_t(1) << 32) - 1;
constexpr int32_t kMaxB = 1 << 16;         // sequences of a cache call
constexpr int32_t kMaxNew = 1 << 24;       // new tokens of a sequence in a cache call
constexpr int32_t kMaxTableCols = 1 << 24;  // positions stay below 2^30
constexpr int32_t kMaxQHeads = 16384;

size_t elem_size(int dtype) { return dtype == SPEC_DTYPE_BF16 ? 2 : 4; }
bool dtype_ok(int dtype) { return dtype == SPEC_DTYPE_F32 || dtype == SPEC_DTYPE_BF16; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool grid_fits(int64_t blocks, int threads) { return blocks >= 1 && blocks * threads <= kMaxWorkItems; }
int finish_launch() { return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP; }

bool head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

int check_cache(const spec_cache4_t& c) {
  if (!c.pages || !c.table) return SPEC_ERR_INVALID_ARG;
  if (!aligned(c.pages, 16) || !aligned(c.table, 4)) return SPEC_ERR_INVALID_ARG;
  if (c.n_pages < 1 || c.table_cols < 1 || c.heads < 1 || c.table_stride < c.table_cols)
    return SPEC_ERR_INVALID_ARG;
  if (!head_dim_ok(c.head_dim) || c.heads > SPEC_CACHE4_MAX_HEADS || c.table_cols > kMaxTableCols)
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

int check_heads(const spec_heads_t& x) {
  if (!x.data) return SPEC_ERR_INVALID_ARG;
  if (!dtype_ok(x.dtype)) return SPEC_ERR_UNSUPPORTED;
  const int64_t per = int64_t(16 / elem_size(x.dtype));
  if (!aligned(x.data, 16)) return SPEC_ERR_INVALID_ARG;
  for (int64_t s : {x.seq_stride, x.pos_stride, x.head_stride})
    if (s < 0 || s % per) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

// Whether rows of `width` elements along axes of n steps lie apart: with the
// axes by stride, each steps over all that the ones before it cover.
struct Axis {
  int64_t n, stride;
};
template <int N>
bool apart(Axis (&x)[N], int64_t width) {
  std::sort(x, x + N, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
  __int128 covered = width;
  for (const Axis& a : x) {
    if (a.n == 1) continue;
    if (a.stride < covered) return false;
    covered += __int128(a.n - 1) * a.stride;
  }
  return true;
}

// Rows that are written must not share elements.
int check_written(const spec_heads_t& x, int64_t B, int64_t T, int64_t heads, int64_t d) {
  Axis axes[] = {{B, x.seq_stride}, {T, x.pos_stride}, {heads, x.head_stride}};
  return apart(axes, d) ? SPEC_OK : SPEC_ERR_INVALID_ARG;
}

int check_new(int32_t B, int32_t T, const int32_t* start) {
  if (B < 1 || T < 1 || !start || !aligned(start, 4)) return SPEC_ERR_INVALID_ARG;
  if (B > kMaxB || T > kMaxNew) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

sv::C4View view(const spec_cache4_t& c) {
  return {static_cast<uint8_t*>(c.pages), c.table, c.table_stride, c.n_pages, c.table_cols, c.heads};
}
sv::C4Heads heads(const spec_heads_t& x) {
  return {x.data, x.seq_stride, x.pos_stride, x.head_stride};
}

// Row tiles of 16 a workgroup keeps, and how many such blocks hold the rows of a
// kv head.  More tiles convert the cache's codes less often, but their
// accumulators leave room for fewer waves.  Times of the whole call:
//   heads of 128  48 rows, 16 x 8 heads over up to 8,155 tokens: 48 us in tiles
//                 of 1, 47 of 2, 39 of 3; 168 rows: 133, 100, 91; four leave one
//                 wave a SIMD (171 in an earlier build where three took 102)
//   heads of 64   48 rows, 96 x 16 heads over up to 2,045: 95, 95, 81; 64 rows:
//                 121, 100 and in a block of four 102; 176 rows, 16 x 8 heads
//                 over up to 8,155: 83, in blocks of 2 or 3 73, of 4 72
//   heads of 256  32 rows, 32 x 4 heads over up to 8,000: 60 in tiles of 1, 64 of
//                 2; 168 rows, 16 x 4 heads: 127 and 153 (both of an earlier
//                 build; now 60 and 123)
int max_tiles(int32_t d) { return d == 256 ? 1 : d == 128 ? 3 : 4; }
void row_blocks(int64_t rows, int32_t d, int* tiles, int64_t* blocks) {
  const int64_t t = (rows + 15) / 16;
  *blocks = (t + max_tiles(d) - 1) / max_tiles(d);
  *tiles = int((t + *blocks - 1) / *blocks);
}

// Tables of at most this many pages a sequence are not cut: the pass that joins
// cut ones costs 4 us where there are few (one sequence of 8 heads) and up to 13 (16
// x 8 heads, 168 rows).  Whole calls: 16 pages, 8 sequences of 8 heads 12.1 us whole,
// 14.6 cut, 96 of 16 26.3 and 28.6; 20 pages 13.3 and 14.7, 30.9 and 31.5; 24 pages
// 14.8 and 14.8, 35.2 and 34.2; 32 pages, one sequence of 8 heads 17.0 and 14.7.  The
// rule sees the table's width, not the lengths, which stand in device memory: 777
// tokens of one sequence take 11.9 us with a table of 13 columns, 14.0 with one of 512.
constexpr int32_t kAttnWhole = 20;
// Whether so many segments of so many pages at most are better not cut, where a
// segment can have a workgroup of its own (not in spec_attention_cache4, whose
// workgroups take what begins in their shares).  The GPU hands out the next one when
// one ends, there is nothing to find or to join, and a segment's pages take their
// time: four times as many segments as pages are enough to fill the rest of the GPU.
// Whole calls, us, cut and each (24 rows a kv head, 8 of them of 128, lengths up to
// 9,000):
//   window of 2,000   8 sequences 24.8 and 25.3, 16 28.2 and 25.7, 64 53 and 38
//   window of 4,000   16 sequences 33.9 and 41.1, 32 48.8 and 42.3, 64 81 and 65
//   window of 8,000   64 sequences 136 and 116, with lengths from 10 on 89 and 90
// Past 72 pages one long sequence among short ones would be waited for too long.
constexpr int64_t kEachCols = 72;
bool each_pays(int64_t segments, int64_t pages) {
  return pages <= kAttnWhole || (pages <= kEachCols && segments >= 4 * pages);
}
// Up to this many segments (sequences x heads x blocks of rows) each is in four
// records or more on average, and their rows are joined by a workgroup each (4 x 8
// heads over 4,000 to 16,000 tokens: 25.5 us, by a wave each 28.8; 8 x 8: 35.6 and
// 36.3; 16 x 8: it would be 57.2 and 52.3).
constexpr int64_t kAttnFew = 64;

int check_attention_sizes(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d) {
  if (B < 1 || T < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads) return SPEC_ERR_INVALID_ARG;
  if (B > kMaxB || T > SPEC_CACHE4_MAX_T || kv_heads > SPEC_CACHE4_MAX_HEADS ||
      q_heads > kMaxQHeads || !head_dim_ok(d))
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// Calls f with the shape of a head dimension and its row tiles.
template <int D, typename F>
void with_shape(int tiles, F f) {
  if (tiles == 1) f(std::integral_constant<int, D>(), std::integral_constant<int, 1>());
  else if constexpr (D < 256) {
    if (tiles == 2) f(std::integral_constant<int, D>(), std::integral_constant<int, 2>());
    else if (tiles == 3) f(std::integral_constant<int, D>(), std::integral_constant<int, 3>());
    else if constexpr (D == 64) f(std::integral_constant<int, D>(), std::integral_constant<int, 4>());
  }
}
template <typename F>
void with_shape(int32_t d, int tiles, F f) {
  if (d == 64) with_shape<64>(tiles, f);
  else if (d == 128) with_shape<128>(tiles, f);
  else with_shape<256>(tiles, f);
}

size_t shape_workspace(int32_t d, int tiles) {
  size_t bytes = 0;
  with_shape(d, tiles, [&](auto D, auto RT) {
    bytes = size_t(sv::C4Shape<D, RT>::kGrid) * (sizeof(sv::C4Cut) + 2 * sizeof(float) * size_t(sv::C4Rec<D, RT>::kFloats));
  });
  return bytes;
}
size_t attention_workspace(int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d) {
  int tiles;
  int64_t blocks;
  row_blocks(int64_t(T) * (q_heads / kv_heads), d, &tiles, &blocks);
  return shape_workspace(d, tiles);
}

template <int D, int RT, typename Args>
void launch_attention(Args& A, void* workspace, hipStream_t st) {
  constexpr int kGrid = sv::C4Shape<D, RT>::kGrid;
  A.cuts = static_cast<sv::C4Cut*>(workspace);
  A.parts = reinterpret_cast<float*>(A.cuts + kGrid);
  const int64_t segments = int64_t(A.B) * A.cache.heads * A.row_blocks;
  A.each = sv::kC4Each<Args> && !A.split && grid_fits(segments, 256);
  const unsigned grid = A.each ? unsigned(segments) : kGrid;
  hipLaunchKernelGGL((sv::k_attention_cache4<D, RT, Args>), dim3(grid), dim3(256), 0, st, A);
  if (!A.split) return;
  if (segments <= kAttnFew)
    hipLaunchKernelGGL((sv::k_attention_cache4_join_long<D, RT, Args>), dim3(unsigned(segments), RT * 16), dim3(256), 0, st, A);
  else
    hipLaunchKernelGGL((sv::k_attention_cache4_join<D, RT, Args>), dim3(kGrid, RT * 4), dim3(256), 0, st, A);
}

// The same for many rows of a kv head, whose pages the waves of a workgroup
// share: rows of a block, and blocks.  Heads of 128 and 256 only.
template <typename F>
void with_wide(int32_t d, F f) {
  if (d == 128) f(std::integral_constant<int, 128>());
  else f(std::integral_constant<int, 256>());
}
void wide_blocks(int64_t rows, int32_t d, int32_t* block_rows, int64_t* blocks) {
  with_wide(d, [&](auto D) {
    const int64_t t = (rows + 15) / 16, most = sv::C4Wide<D>::kTiles;
    *blocks = (t + most - 1) / most;
    *block_rows = int32_t((t + *blocks - 1) / *blocks * 16);
  });
}
// Whether sharing pays for `rows` rows of a kv head, so many (sequence, kv head)
// and pages of each at most (whole calls, us, without it and with it):
//   heads of 64   hardly: 192 rows, 16 heads over 16,384 tokens 51 and 64; 168 rows,
//                 32 x 8 heads through a window of 4,000 121 and 110, the best
//   heads of 128  where there is a sequence and head for each workgroup, so that few
//                 are cut: behind shared prefixes 64 x 8 heads over 2,048, 64 rows 77
//                 and 81, 160 rows 175 and 162, 256 rows 269 and 238; 168 rows through
//                 windows 64 x 8 of 1,000 104 and 82, of 4,000 276 and 231, 32 x 8 of
//                 2,000 84 and 98, 16 x 8 of 1,000 31 and 59
//   heads of 256  where its workgroups have some pages each, for they are half as
//                 many: 168 rows through windows 16 x 4 heads of 4,000 101 and 92, 64 x
//                 4 of 1,000 117 and 95, 8 x 4 of 1,000 25 and 45; 4 x 4 heads, 378
//                 rows, over 8,192 105 and 97, over 2,048 52 and 65
bool wide_rows(int64_t rows, int32_t d) { return d == 128 ? rows > 96 : d == 256 && rows > 64; }
bool wide_pays(int64_t rows, int32_t d, int64_t seqs_heads, int64_t pages) {
  if (!wide_rows(rows, d)) return false;
  if (d == 128) return seqs_heads >= sv::C4Wide<128>::kGrid;
  int32_t block_rows;
  int64_t blocks;
  wide_blocks(rows, d, &block_rows, &blocks);
  return seqs_heads * blocks >= (16 * sv::C4Wide<256>::kGrid + pages - 1) / pages;
}
size_t wide_workspace(int32_t d) {
  size_t bytes = 0;
  with_wide(d, [&](auto D) {
    bytes = size_t(sv::C4Wide<D>::kGrid) * (sizeof(sv::C4Cut) + 2 * sizeof(float) * size_t(sv::C4Wide<D>::kFloats));
  });
  return bytes;
}
// Segments up to which four times as many threads share a row's records, which are
// 32 or more (378 rows of heads of 256 over 131,072 tokens, 3 segments: 104 us and
// 139; 12 segments over 65,536: 158 and 159; 24 over 16,384: 98 and 95).
constexpr int64_t kWideFew = 8;
template <int D, typename Args>
void launch_wide(Args& A, int32_t block_rows, void* workspace, hipStream_t st) {
  using Sh = sv::C4Wide<D>;
  constexpr int kGrid = Sh::kGrid;
  A.cuts = static_cast<sv::C4Cut*>(workspace);
  A.parts = reinterpret_cast<float*>(A.cuts + kGrid);
  const int64_t segments = int64_t(A.B) * A.cache.heads * A.row_blocks;
  if constexpr (sv::kC4Each<Args>)
    if (!A.split && grid_fits(segments, 64 * Sh::kWaves)) {
      hipLaunchKernelGGL((sv::k_attention_cache4_wide<D, Args, true>), dim3(unsigned(segments)), dim3(64 * Sh::kWaves), 0, st, A, block_rows);
      return;
    }
  hipLaunchKernelGGL((sv::k_attention_cache4_wide<D, Args, false>), dim3(kGrid), dim3(64 * Sh::kWaves), 0, st, A, block_rows);
  if (!A.split) return;
  const dim3 grid{unsigned(kGrid), unsigned(block_rows / 16)};
  if constexpr (D == 256)  // of heads of 128 there are always more
    if (segments <= kWideFew) {
      hipLaunchKernelGGL((sv::k_attention_cache4_wide_join<D, 4, Args>), grid, dim3(1024), 0, st, A, block_rows);
      return;
    }
  hipLaunchKernelGGL((sv::k_attention_cache4_wide_join<D, 1, Args>), grid, dim3(256), 0, st, A, block_rows);
}

// Arguments of an attention call, checked, and its row tiles.
int attention_args(const spec_cache4_t& cache, const spec_heads_t& q, int32_t B, int32_t T, int32_t q_heads,
                   const int32_t* start, const int32_t* count, const uint32_t* mask, int64_t mask_seq_stride,
                   int64_t mask_pos_stride, float scale, const spec_heads_t& out, float* lse, void* workspace,
                   size_t workspace_bytes, sv::C4AttnArgs* A, int* tiles) {
  int rc;
  if ((rc = check_new(B, T, start)) != SPEC_OK) return rc;
  if ((rc = check_cache(cache)) != SPEC_OK) return rc;
  if ((rc = check_attention_sizes(B, T, q_heads, cache.heads, cache.head_dim)) != SPEC_OK) return rc;
  if ((rc = check_heads(q)) != SPEC_OK) return rc;
  if ((rc = check_heads(out)) != SPEC_OK) return rc;
  if (q.dtype != SPEC_DTYPE_BF16 || out.dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if ((rc = check_written(out, B, T, q_heads, cache.head_dim)) != SPEC_OK) return rc;
  if ((count && !aligned(count, 4)) || (lse && !aligned(lse, 4))) return SPEC_ERR_INVALID_ARG;
  if (mask && (!aligned(mask, 4) || mask_seq_stride < 0 || mask_pos_stride < 0))
    return SPEC_ERR_INVALID_ARG;
  const float c = float(double(scale) * 1.4426950408889634);
  if (!std::isfinite(scale) || !(scale > 0.0f) || !std::isfinite(c) || !(c > 0.0f))
    return SPEC_ERR_INVALID_ARG;
  const int32_t G = q_heads / cache.heads;
  int64_t blocks;
  row_blocks(int64_t(T) * G, cache.head_dim, tiles, &blocks);
  // the pages of all sequences, heads and blocks of rows are one sum
  if (int64_t(B) * (int64_t(cache.table_cols) + sv::kC4SegCost) * cache.heads >= (int64_t(1) << 40) / blocks)
    return SPEC_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < attention_workspace(T, q_heads, cache.heads, cache.head_dim))
    return SPEC_ERR_WORKSPACE;
  *A = {view(cache), static_cast<const uint16_t*>(q.data), q.seq_stride, q.pos_stride, q.head_stride,
        static_cast<uint16_t*>(out.data), out.seq_stride, out.pos_stride, out.head_stride, lse, start, count,
        mask, mask_seq_stride, mask_pos_stride, B, T, G, int32_t(blocks), c, cache.table_cols > kAttnWhole,
        nullptr, nullptr};
  return SPEC_OK;
}

}  // namespace
