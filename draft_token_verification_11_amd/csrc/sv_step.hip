// sv_step.hip -- the C ABI of the serving step but for shared prefixes:
// argument validation and kernel launches for gfx950.  See
// include/specverify_step.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "specverify_step.h"
#include "sv_cache4_host.hpp"
#include "sv_pages.hpp"
#include "sv_rotate.hpp"

namespace {

// Waves that a small rotation is cut into: as many as the compute units hold at once.
// 128 x 16 tokens of 32 + 8 heads of 128 take 15.1 us with it, 18.3 with 2,048 and
// 20.5 with 32,768, for each of which the angles are made again; 16 x 256 tokens 20.1,
// 22.1, 24.4; 64 x 6 6.8, 6.2, 6.7; one token 4.4 with any.
constexpr int64_t kRotateWaves = 8192;

// Workgroups that move the pages of a call of many sequences (4,093 sequences there and
// back with slots 40.1 us, with 256 43.9, with 4,096 40.1).
constexpr int64_t kReserveBlocks = 1024;

// New tokens from which on a workgroup has those of one sequence only (4,093 x 1,000 in
// such a call 40.1 us, by tokens 43.2; 512 x 400 32.2 both; 4,093 x 16 32.4 by
// sequences, 31.4 by tokens).
constexpr int32_t kSlotsLong = 256;

// One side of a rotation; a side without heads is not looked at.
int check_side(const spec_heads_t& in, const spec_heads_t& out, int32_t heads, const void* weight,
               const spec_rotate_t& how, int32_t B, int32_t T) {
  int rc;
  if (heads == 0) return SPEC_OK;
  if ((rc = check_heads(in)) != SPEC_OK) return rc;
  if ((rc = check_heads(out)) != SPEC_OK) return rc;
  if ((rc = check_written(out, B, T, heads, how.head_dim)) != SPEC_OK) return rc;
  if (weight && (!how.norm || !aligned(weight, 16))) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}
sv::RotHeads side(const spec_heads_t& in, const spec_heads_t& out, int32_t heads, const void* weight) {
  if (heads == 0) return {};
  return {in.data, out.data, weight, in.seq_stride, in.pos_stride, in.head_stride,
          out.seq_stride, out.pos_stride, out.head_stride, heads};
}

template <typename TI, typename TO>
int launch_rotate(sv::RotateArgs& A, hipStream_t st) {
  const int lanes = A.D <= 64 ? 8 : A.D <= 128 ? 16 : 32, per = 64 / lanes;
  const int64_t rounds = (A.x[0].heads + per - 1) / per + (A.x[1].heads + per - 1) / per;
  const int64_t want = std::min<int64_t>(rounds, (kRotateWaves + A.tokens - 1) / A.tokens);
  A.per = int32_t((rounds + want - 1) / want);
  A.chunks = int32_t((rounds + A.per - 1) / A.per);
  const int64_t blocks = (A.tokens * A.chunks + 3) / 4;
  if (!grid_fits(blocks, 256)) return SPEC_ERR_UNSUPPORTED;
  const dim3 grid{unsigned(blocks)}, block{256};
  (void)hipGetLastError();
  if (lanes == 8) hipLaunchKernelGGL((sv::k_norm_rotate<TI, TO, 8>), grid, block, 0, st, A);
  else if (lanes == 16) hipLaunchKernelGGL((sv::k_norm_rotate<TI, TO, 16>), grid, block, 0, st, A);
  else hipLaunchKernelGGL((sv::k_norm_rotate<TI, TO, 32>), grid, block, 0, st, A);
  return finish_launch();
}

// Scratch of either kernel that a window may take.
size_t window_workspace(int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d) {
  const bool many = wide_rows(int64_t(T) * (q_heads / kv_heads), d);
  return std::max(attention_workspace(T, q_heads, kv_heads, d), many ? wide_workspace(d) : size_t(0));
}

}  // namespace

extern "C" {

int spec_norm_rotate(spec_heads_t q, spec_heads_t q_out, int32_t q_heads, spec_heads_t k,
                     spec_heads_t k_out, int32_t heads, const spec_rotate_t* how, int32_t B,
                     int32_t T, const int32_t* start, const int32_t* count, void* stream) {
  int rc;
  if (!how || q_heads < 0 || heads < 0 || (q_heads == 0 && heads == 0)) return SPEC_ERR_INVALID_ARG;
  if (q_heads > kMaxQHeads || heads > kMaxQHeads - q_heads) return SPEC_ERR_UNSUPPORTED;
  if ((rc = check_new(B, T, start)) != SPEC_OK) return rc;
  if (count && !aligned(count, 4)) return SPEC_ERR_INVALID_ARG;
  if (how->head_dim < 16 || how->head_dim > 256 || how->head_dim % 16) return SPEC_ERR_UNSUPPORTED;
  if (how->rotary_dim < 0 || how->rotary_dim > how->head_dim) return SPEC_ERR_INVALID_ARG;
  if (how->rotary_dim % 16) return SPEC_ERR_UNSUPPORTED;
  if ((how->rotary_dim > 0) != (how->inv_freq != nullptr) || !aligned(how->inv_freq, 4)) return SPEC_ERR_INVALID_ARG;
  if (how->interleaved < 0 || how->interleaved > 1 || how->norm < 0 || how->norm > 1) return SPEC_ERR_INVALID_ARG;
  if (how->norm && (!std::isfinite(how->eps) || how->eps < 0.0f)) return SPEC_ERR_INVALID_ARG;
  if (!dtype_ok(how->weight_dtype)) return SPEC_ERR_UNSUPPORTED;
  if (how->depth && (!aligned(how->depth, 4) || how->depth_stride < 0)) return SPEC_ERR_INVALID_ARG;
  if ((rc = check_side(q, q_out, q_heads, how->q_weight, *how, B, T)) != SPEC_OK) return rc;
  if ((rc = check_side(k, k_out, heads, how->k_weight, *how, B, T)) != SPEC_OK) return rc;
  const spec_heads_t &in = q_heads ? q : k, &out = q_heads ? q_out : k_out;
  if (q_heads && heads && (q.dtype != k.dtype || q_out.dtype != k_out.dtype)) return SPEC_ERR_INVALID_ARG;
  sv::RotateArgs A{{side(q, q_out, q_heads, how->q_weight), side(k, k_out, heads, how->k_weight)},
                   how->inv_freq, start, count, how->depth, how->depth_stride, int64_t(B) * T, T, how->head_dim,
                   how->rotary_dim, how->interleaved, how->norm, how->weight_dtype == SPEC_DTYPE_F32, how->eps, 0, 0};
  auto st = static_cast<hipStream_t>(stream);
  const bool bf = in.dtype == SPEC_DTYPE_BF16, to_bf = out.dtype == SPEC_DTYPE_BF16;
  if (bf) return to_bf ? launch_rotate<uint16_t, uint16_t>(A, st) : launch_rotate<uint16_t, float>(A, st);
  return to_bf ? launch_rotate<float, uint16_t>(A, st) : launch_rotate<float, float>(A, st);
}

size_t spec_attention_cache4_window_workspace(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                              int32_t head_dim) {
  if (check_attention_sizes(B, T, q_heads, heads, head_dim) != SPEC_OK) return 0;
  return window_workspace(T, q_heads, heads, head_dim);
}

int spec_attention_cache4_window(spec_cache4_t cache, spec_heads_t q, int32_t B, int32_t T,
                                 int32_t q_heads, const int32_t* start, const int32_t* count,
                                 const uint32_t* mask, int64_t mask_seq_stride,
                                 int64_t mask_pos_stride, const int32_t* depth,
                                 int64_t depth_stride, int32_t window, int32_t sinks, float scale,
                                 spec_heads_t out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  sv::C4WindowArgs A;
  int tiles;
  if (window < 1 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  if (depth && (!mask || !aligned(depth, 4) || depth_stride < 0)) return SPEC_ERR_INVALID_ARG;
  const int rc = attention_args(cache, q, B, T, q_heads, start, count, mask, mask_seq_stride, mask_pos_stride, scale,
                                out, lse, workspace, workspace_bytes, &A, &tiles);
  if (rc != SPEC_OK) return rc;
  if (workspace_bytes < window_workspace(T, q_heads, cache.heads, cache.head_dim)) return SPEC_ERR_WORKSPACE;
  A.window = window;
  A.sinks = sinks;
  A.depth = depth;
  A.depth_seq = depth_stride;
  // pages that a sequence can have read at most
  const int64_t pages = (int64_t(window) + T + sv::kC4Page - 2) / sv::kC4Page + 1 + (int64_t(sinks) + sv::kC4Page - 1) / sv::kC4Page;
  const int64_t cols = std::min<int64_t>(pages, cache.table_cols);
  auto st = static_cast<hipStream_t>(stream);
  const int32_t d = cache.head_dim;
  const int64_t rows = int64_t(T) * A.G;
  (void)hipGetLastError();
  if (wide_pays(rows, d, int64_t(B) * cache.heads, cols)) {
    int32_t block_rows;
    int64_t blocks;
    wide_blocks(rows, d, &block_rows, &blocks);
    A.row_blocks = int32_t(blocks);
    A.split = !each_pays(int64_t(B) * cache.heads * blocks, cols);
    with_wide(d, [&](auto D) { launch_wide<D>(A, block_rows, workspace, st); });
  } else {
    A.split = !each_pays(int64_t(B) * cache.heads * A.row_blocks, cols);
    with_shape(d, tiles, [&](auto D, auto RT) { launch_attention<D, RT>(A, workspace, st); });
  }
  return finish_launch();
}

size_t spec_cache4_reserve_workspace(int32_t B) {
  return B <= sv::kResFew || B > kMaxB ? 0 : 256 + align256(size_t(B) * 8);
}

int spec_cache4_reserve(int32_t* table, int64_t table_stride, int32_t table_cols, int32_t* held,
                        const int32_t* need, int32_t B, int32_t* free_pages,
                        int32_t free_capacity, int32_t* free_count, void* workspace,
                        size_t workspace_bytes, void* stream) {
  for (const void* p : {static_cast<const void*>(table), static_cast<const void*>(held), static_cast<const void*>(need),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_count)})
    if (!p || !aligned(p, 4)) return SPEC_ERR_INVALID_ARG;
  if (B < 1 || table_cols < 1 || table_stride < table_cols || free_capacity < 1) return SPEC_ERR_INVALID_ARG;
  if (B > kMaxB || table_cols > kMaxTableCols) return SPEC_ERR_UNSUPPORTED;
  const size_t need_bytes = spec_cache4_reserve_workspace(B);
  if (need_bytes && (!workspace || !aligned(workspace, 256) || workspace_bytes < need_bytes)) return SPEC_ERR_WORKSPACE;
  const sv::ReserveArgs A{table, table_stride, held, need, free_pages, free_count, table_cols, B, free_capacity};
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (B <= sv::kResFew) {
    hipLaunchKernelGGL(sv::k_cache4_reserve, dim3(1), dim3(sv::kResThreads), 0, st, A);
    return finish_launch();
  }
  auto* const plan = static_cast<sv::ReservePlan*>(workspace);
  auto* const upto = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
  const int64_t most = std::min<int64_t>(int64_t(B) * table_cols, free_capacity);  // pages that a call can move
  const unsigned blocks = unsigned(std::min<int64_t>((most + 255) / 256, kReserveBlocks));
  hipLaunchKernelGGL(sv::k_cache4_reserve_plan, dim3(1), dim3(sv::kResThreads), 0, st, A, plan, upto);
  hipLaunchKernelGGL(sv::k_cache4_reserve_move, dim3(blocks), dim3(256), 0, st, A, plan, upto);
  return finish_launch();
}

int spec_cache4_slots(const int32_t* table, int64_t table_stride, int32_t table_cols,
                      int32_t n_pages, int32_t B, int32_t T, const int32_t* start,
                      const int32_t* count, int64_t* slots, void* stream) {
  int rc;
  if ((rc = check_new(B, T, start)) != SPEC_OK) return rc;
  if (!table || !aligned(table, 4) || !slots || !aligned(slots, 8) || (count && !aligned(count, 4)))
    return SPEC_ERR_INVALID_ARG;
  if (table_cols < 1 || table_stride < table_cols || n_pages < 1) return SPEC_ERR_INVALID_ARG;
  if (table_cols > kMaxTableCols) return SPEC_ERR_UNSUPPORTED;
  const int64_t tokens = int64_t(B) * T, blocks = (tokens + 255) / 256;
  if (!grid_fits(blocks, 256)) return SPEC_ERR_UNSUPPORTED;
  const sv::SlotArgs A{table, table_stride, start, count, slots, tokens, table_cols, n_pages, T};
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (T >= kSlotsLong)
    hipLaunchKernelGGL(sv::k_cache4_slots_run, dim3(unsigned(B), unsigned((T + sv::kSlotsRun - 1) / sv::kSlotsRun)), dim3(256), 0, st, A);
  else
    hipLaunchKernelGGL(sv::k_cache4_slots, dim3(unsigned(blocks)), dim3(256), 0, st, A);
  return finish_launch();
}

}  // extern "C"
