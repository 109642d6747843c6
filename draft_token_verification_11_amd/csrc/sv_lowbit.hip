// sv_lowbit.hip -- the C ABI of the target's pass in few bits: argument
// validation and kernel launches for gfx950.  See
// include/specverify_lowbit.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "specverify_lowbit.h"
#include "sv_cache4.hpp"
#include "sv_fp8.hpp"

namespace {

constexpr int64_t kMaxWorkItems = (int64_t(1) << 32) - 1;
constexpr int32_t kMaxB = 1 << 16;         // sequences of a cache call
constexpr int32_t kMaxNew = 1 << 24;       // new tokens of a sequence in a cache call
constexpr int32_t kMaxTableCols = 1 << 24;  // positions stay below 2^30
constexpr int32_t kMaxQHeads = 16384;
constexpr int64_t kMaxWeightStride = 1 << 22;  // a tile's 256 rows have 32-bit offsets

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

// Arguments of the two moving calls, and their grid.
int move_args(const spec_cache4_t& c, const spec_heads_t& k, const spec_heads_t& v, int32_t B,
              int32_t T, const int32_t* start, const int32_t* count, sv::C4MoveArgs* A,
              unsigned* grid) {
  int rc;
  if ((rc = check_new(B, T, start)) != SPEC_OK) return rc;
  if ((rc = check_cache(c)) != SPEC_OK) return rc;
  if ((rc = check_heads(k)) != SPEC_OK) return rc;
  if ((rc = check_heads(v)) != SPEC_OK) return rc;
  if (k.dtype != v.dtype || (count && !aligned(count, 4))) return SPEC_ERR_INVALID_ARG;
  const int64_t per = 512 / c.head_dim;  // tokens of a wave
  const int64_t runs = (int64_t(T) + 2 * per - 2) / per;
  const int64_t waves = int64_t(B) * runs * c.heads;
  const int64_t blocks = (waves + 3) / 4;
  if (!grid_fits(blocks, 256)) return SPEC_ERR_UNSUPPORTED;
  *A = {view(c), heads(k), heads(v), start, count, waves, T, int32_t(runs)};
  *grid = unsigned(blocks);
  return SPEC_OK;
}

template <typename T>
void launch_write(int32_t d, unsigned grid, const sv::C4MoveArgs& A, hipStream_t st) {
  if (d == 64) hipLaunchKernelGGL((sv::k_cache4_write<T, 64>), dim3(grid), dim3(256), 0, st, A);
  else if (d == 128) hipLaunchKernelGGL((sv::k_cache4_write<T, 128>), dim3(grid), dim3(256), 0, st, A);
  else hipLaunchKernelGGL((sv::k_cache4_write<T, 256>), dim3(grid), dim3(256), 0, st, A);
}
template <typename T>
void launch_read(int32_t d, unsigned grid, const sv::C4MoveArgs& A, hipStream_t st) {
  if (d == 64) hipLaunchKernelGGL((sv::k_cache4_read<T, 64>), dim3(grid), dim3(256), 0, st, A);
  else if (d == 128) hipLaunchKernelGGL((sv::k_cache4_read<T, 128>), dim3(grid), dim3(256), 0, st, A);
  else hipLaunchKernelGGL((sv::k_cache4_read<T, 256>), dim3(grid), dim3(256), 0, st, A);
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

size_t attention_workspace(int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d) {
  int tiles;
  int64_t blocks;
  row_blocks(int64_t(T) * (q_heads / kv_heads), d, &tiles, &blocks);
  size_t bytes = 0;
  with_shape(d, tiles, [&](auto D, auto RT) {
    bytes = size_t(sv::C4Shape<D, RT>::kGrid) * (sizeof(sv::C4Cut) + 2 * sizeof(float) * size_t(sv::C4Rec<D, RT>::kFloats));
  });
  return bytes;
}

template <int D, int RT>
void launch_attention(sv::C4AttnArgs& A, void* workspace, hipStream_t st) {
  constexpr int kGrid = sv::C4Shape<D, RT>::kGrid;
  A.cuts = static_cast<sv::C4Cut*>(workspace);
  A.parts = reinterpret_cast<float*>(A.cuts + kGrid);
  hipLaunchKernelGGL((sv::k_attention_cache4<D, RT>), dim3(kGrid), dim3(256), 0, st, A);
  if (!A.split) return;
  const int64_t segments = int64_t(A.B) * A.cache.heads * A.row_blocks;
  if (segments <= kAttnFew)
    hipLaunchKernelGGL((sv::k_attention_cache4_join_long<D, RT>), dim3(unsigned(segments), RT * 16), dim3(256), 0, st, A);
  else
    hipLaunchKernelGGL((sv::k_attention_cache4_join<D, RT>), dim3(kGrid, RT * 4), dim3(256), 0, st, A);
}

int check_head(const void* weight, int64_t stride, int64_t elem, int32_t V, int32_t d) {
  if (!weight || V < 1 || d < 32 || d % 32) return SPEC_ERR_INVALID_ARG;
  if (V > SPEC_MAX_V || d > 65536) return SPEC_ERR_UNSUPPORTED;
  if (!aligned(weight, 16) || stride % (16 / elem)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

int64_t padded(int32_t d) { return (int64_t(d) + 127) / 128 * 128; }

template <typename TO, bool F8, int BV, int BM, int WV, int WAVES>
void launch_head_tile(sv::F8HeadArgs A, hipStream_t st) {
  A.v_tiles = int32_t((A.V + BV - 1) / BV);
  A.m_tiles = int32_t((A.M + BM - 1) / BM);
  const int64_t tiles = int64_t(A.v_tiles) * A.m_tiles;
  hipLaunchKernelGGL((sv::k_lmhead_fp8_tile<TO, F8, BV, BM, WV, WAVES>), dim3(unsigned((tiles + 7) / 8 * 8)),
                     dim3(64 * WAVES), 0, st, A);
}
// One workgroup per compute unit of the kernel for up to 16 rows.
constexpr unsigned kHeadGrid = 256;

// The kernel for M rows; times over 151,936 entries x 4,096.
template <typename TO>
void launch_head(const sv::F8HeadArgs& A, hipStream_t st) {
  constexpr bool f8 = sizeof(TO) == 2;  // BF16 logits: the 8-bit instructions' sums do
  // Up to 16 rows whose LDS image fits (rows of 8,192): 0.122 ms, in tiles 0.134.
  if (A.M <= 16 && A.dp <= 8192) {
    if (A.dp <= 4096)
      hipLaunchKernelGGL((sv::k_lmhead_fp8_rows<TO, 32>), dim3(kHeadGrid), dim3(512), 0, st, A);
    else
      hipLaunchKernelGGL((sv::k_lmhead_fp8_rows<TO, 64>), dim3(kHeadGrid), dim3(512), 0, st, A);
    return;
  }
  // Up to 64 rows (24 rows over 32,000 entries: 0.034 ms, in tiles of 128 0.045).
  if (A.M <= 64) {
    launch_head_tile<TO, f8, 128, 64, 2, 4>(A, st);
    return;
  }
  // Two workgroups of four waves a compute unit, which fill each other's waits
  // (120 rows, F32: 0.188 ms, one of eight waves 0.224), and where the matrix
  // instructions bind, one of eight with wave tiles of 64 x 128, which read LDS
  // less, unless it pads more rows.  Where it does, in tiles of 128 and of 256: 260
  // rows 266 and 304 us, 520 441 and 432, 1,300 978 and 875, 2,565 1,932 and 1,654;
  // over 32,003 x 2,080 520 rows 76 and 87, 1,300 146 and 138, 1,650 174 and 178.  So
  // from about 1,280 rows on the small tiles lose mostly: the rule does not see that.
  // (2,560 rows, which pad none: 1,510 to 1,530.)  F32 logits need four times the
  // instructions a block; there LDS does not bind (2,560 rows: 3.03 ms, in an earlier
  // build 3.12 either way).
  if constexpr (f8)
    if ((A.M + 255) / 256 * 256 == (A.M + 127) / 128 * 128) {
      launch_head_tile<TO, f8, 256, 256, 4, 8>(A, st);
      return;
    }
  launch_head_tile<TO, f8, 128, 128, 2, 4>(A, st);
}

}  // namespace

extern "C" {

size_t spec_cache4_record_bytes(int32_t head_dim) {
  return head_dim_ok(head_dim) ? size_t(68) * size_t(head_dim) : 0;
}

int spec_cache4_write(spec_cache4_t cache, spec_heads_t k, spec_heads_t v, int32_t B, int32_t T,
                      const int32_t* start, const int32_t* count, void* stream) {
  sv::C4MoveArgs A;
  unsigned grid;
  const int rc = move_args(cache, k, v, B, T, start, count, &A, &grid);
  if (rc != SPEC_OK) return rc;
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (k.dtype == SPEC_DTYPE_BF16) launch_write<uint16_t>(cache.head_dim, grid, A, st);
  else launch_write<float>(cache.head_dim, grid, A, st);
  return finish_launch();
}

int spec_cache4_read(spec_cache4_t cache, spec_heads_t k, spec_heads_t v, int32_t B, int32_t T,
                     const int32_t* start, const int32_t* count, void* stream) {
  sv::C4MoveArgs A;
  unsigned grid;
  int rc = move_args(cache, k, v, B, T, start, count, &A, &grid);
  if (rc != SPEC_OK) return rc;
  if ((rc = check_written(k, B, T, cache.heads, cache.head_dim)) != SPEC_OK) return rc;
  if ((rc = check_written(v, B, T, cache.heads, cache.head_dim)) != SPEC_OK) return rc;
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (k.dtype == SPEC_DTYPE_BF16) launch_read<uint16_t>(cache.head_dim, grid, A, st);
  else launch_read<float>(cache.head_dim, grid, A, st);
  return finish_launch();
}

size_t spec_attention_cache4_workspace(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                       int32_t head_dim) {
  if (check_attention_sizes(B, T, q_heads, heads, head_dim) != SPEC_OK) return 0;
  return attention_workspace(T, q_heads, heads, head_dim);
}

int spec_attention_cache4(spec_cache4_t cache, spec_heads_t q, int32_t B, int32_t T,
                          int32_t q_heads, const int32_t* start, const int32_t* count,
                          const uint32_t* mask, int64_t mask_seq_stride, int64_t mask_pos_stride,
                          float scale, spec_heads_t out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
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
  int tiles;
  int64_t blocks;
  row_blocks(int64_t(T) * G, cache.head_dim, &tiles, &blocks);
  // the pages of all sequences, heads and blocks of rows are one sum
  if (int64_t(B) * (int64_t(cache.table_cols) + sv::kC4SegCost) * cache.heads >= (int64_t(1) << 40) / blocks)
    return SPEC_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < attention_workspace(T, q_heads, cache.heads, cache.head_dim))
    return SPEC_ERR_WORKSPACE;
  sv::C4AttnArgs A{view(cache), static_cast<const uint16_t*>(q.data), q.seq_stride, q.pos_stride,
                   q.head_stride, static_cast<uint16_t*>(out.data), out.seq_stride, out.pos_stride,
                   out.head_stride, lse, start, count, mask, mask_seq_stride, mask_pos_stride, B, T, G,
                   int32_t(blocks), c, cache.table_cols > kAttnWhole, nullptr, nullptr};
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  with_shape(cache.head_dim, tiles, [&](auto D, auto RT) { launch_attention<D, RT>(A, workspace, st); });
  return finish_launch();
}

int spec_quantize_fp8(const void* weight, int32_t dtype, int64_t weight_stride, int32_t V,
                      int32_t d, void* q, float* scale, void* stream) {
  if (!dtype_ok(dtype)) return SPEC_ERR_UNSUPPORTED;
  int rc;
  if ((rc = check_head(weight, weight_stride, int64_t(elem_size(dtype)), V, d)) != SPEC_OK) return rc;
  if (weight_stride < d || !q || !scale || !aligned(q, 16) || !aligned(scale, 4))
    return SPEC_ERR_INVALID_ARG;
  const int64_t db = padded(d) / 128, blocks = (int64_t(V) + 127) / 128 * db;
  if (!grid_fits(blocks, 256)) return SPEC_ERR_UNSUPPORTED;
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == SPEC_DTYPE_BF16)
    hipLaunchKernelGGL((sv::k_quantize_fp8<uint16_t>), dim3(unsigned(blocks)), dim3(256), 0, st,
                       static_cast<const uint16_t*>(weight), weight_stride, int64_t(V), d, int32_t(db),
                       static_cast<uint8_t*>(q), scale);
  else
    hipLaunchKernelGGL((sv::k_quantize_fp8<float>), dim3(unsigned(blocks)), dim3(256), 0, st,
                       static_cast<const float*>(weight), weight_stride, int64_t(V), d, int32_t(db),
                       static_cast<uint8_t*>(q), scale);
  return finish_launch();
}

size_t spec_lmhead_fp8_workspace(int32_t B, int32_t rows, int32_t d) {
  if (B < 1 || rows < 1 || d < 32 || d % 32 || B > (1 << 24) || rows > 2 * SPEC_MAX_K + 1 || d > 65536)
    return 0;
  const size_t M = size_t(B) * size_t(rows);
  return align256(M * size_t(padded(d))) + align256(M) * size_t(padded(d) / 128);
}

int spec_lmhead_fp8(spec_logits_t hidden, int32_t B, int32_t rows, int32_t d, const void* weight,
                    int64_t weight_stride, const float* scale, int32_t V, spec_logits_t logits,
                    void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  if (B < 1 || rows < 1) return SPEC_ERR_INVALID_ARG;
  if (B > (1 << 24) || rows > 2 * SPEC_MAX_K + 1) return SPEC_ERR_UNSUPPORTED;
  if ((rc = check_head(weight, weight_stride, 1, V, d)) != SPEC_OK) return rc;
  if (weight_stride < d || !scale || !aligned(scale, 4)) return SPEC_ERR_INVALID_ARG;
  if (weight_stride > kMaxWeightStride) return SPEC_ERR_UNSUPPORTED;
  if (!dtype_ok(hidden.dtype) || !dtype_ok(logits.dtype)) return SPEC_ERR_UNSUPPORTED;
  const int64_t per = int64_t(16 / elem_size(hidden.dtype));
  if (!hidden.data || !aligned(hidden.data, 16) || hidden.seq_stride < 0 || hidden.pos_stride < 0 ||
      hidden.seq_stride % per || hidden.pos_stride % per)
    return SPEC_ERR_INVALID_ARG;
  // written rows must not share elements
  Axis axes[] = {{B, logits.seq_stride}, {rows, logits.pos_stride}};
  if (!logits.data || !aligned(logits.data, elem_size(logits.dtype)) || !apart(axes, V))
    return SPEC_ERR_INVALID_ARG;
  const int64_t M = int64_t(B) * rows, dp = padded(d);
  const int64_t rounding = (M * (dp / 128) + 15) / 16;
  const int64_t tiles = ((int64_t(V) + 127) / 128) * ((M + 63) / 64);  // of the smallest kind, and a round of 8
  if (!grid_fits(rounding, 256) || !grid_fits(tiles + 8, 256)) return SPEC_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < spec_lmhead_fp8_workspace(B, rows, d))
    return SPEC_ERR_WORKSPACE;
  auto st = static_cast<hipStream_t>(stream);
  sv::F8HiddenArgs H{hidden.data, hidden.seq_stride, hidden.pos_stride, rows, M, d, int32_t(dp),
                     static_cast<uint8_t*>(workspace),
                     static_cast<uint8_t*>(workspace) + align256(size_t(M) * size_t(dp)),
                     int64_t(align256(size_t(M)))};
  sv::F8HeadArgs A{H.out, H.exps, H.m_pitch, M, V, d, int32_t(dp), rows, static_cast<const uint8_t*>(weight),
                   weight_stride, scale, const_cast<void*>(logits.data), logits.seq_stride,
                   logits.pos_stride, 0, 0};
  (void)hipGetLastError();
  if (hidden.dtype == SPEC_DTYPE_BF16)
    hipLaunchKernelGGL((sv::k_hidden_fp8<uint16_t>), dim3(unsigned(rounding)), dim3(256), 0, st, H);
  else
    hipLaunchKernelGGL((sv::k_hidden_fp8<float>), dim3(unsigned(rounding)), dim3(256), 0, st, H);
  if (logits.dtype == SPEC_DTYPE_BF16) launch_head<uint16_t>(A, st);
  else launch_head<float>(A, st);
  return finish_launch();
}

}  // extern "C"
