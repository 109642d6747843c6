// sv_lowbit.hip -- the C ABI of the target's pass in few bits: argument
// validation and kernel launches for gfx950.  See
// include/specverify_lowbit.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "specverify_lowbit.h"
#include "sv_cache4_host.hpp"
#include "sv_fp8.hpp"

namespace {

constexpr int64_t kMaxWeightStride = 1 << 22;  // a tile's 256 rows have 32-bit offsets

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
  sv::C4AttnArgs A;
  int tiles;
  const int rc = attention_args(cache, q, B, T, q_heads, start, count, mask, mask_seq_stride, mask_pos_stride, scale,
                                out, lse, workspace, workspace_bytes, &A, &tiles);
  if (rc != SPEC_OK) return rc;
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
