// sv_shared.hip -- the C ABI of attention behind shared prefixes: argument
// validation and kernel launches for gfx950.  See include/specverify_step.h for
// the contract.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "specverify_step.h"
#include "sv_cache4_host.hpp"
#include "sv_cache4_short.hpp"

namespace {

constexpr int64_t kMaxSharedRows = 1 << 30;  // of a prefix, over all heads

bool shared_sizes_ok(int32_t B, int32_t T, int32_t q_heads, int32_t fan) {
  return fan >= 1 && int64_t(std::min(fan, B)) * T <= kMaxSharedRows / q_heads;
}

// How the rows of a prefix are held.
struct PrefixShape {
  bool wide;           // many rows: the waves of a workgroup share the pages
  int tiles;           // not wide: tiles of a block
  int32_t block_rows;  // wide: rows of a block
  int64_t blocks;
};
PrefixShape prefix_shape(int64_t rows, int32_t d, int64_t prefixes_heads, int64_t cols, bool compact) {
  PrefixShape x{};
  // `rows` are far more than the live ones where those are counted through
  x.wide = wide_pays(rows, d, prefixes_heads, cols);
  if (x.wide && compact) with_wide(d, [&](auto D) { x.wide = sv::C4Wide<D>::kCounted; });
  if (x.wide) wide_blocks(rows, d, &x.block_rows, &x.blocks);
  else row_blocks(rows, d, &x.tiles, &x.blocks);
  return x;
}
// Whether a wave goes through the pages of a (branch, kv head, block of rows) by itself:
// where there are as many of those as waves in flight, or half as many and few
// pages.  Whole calls, us, four waves to each and one (16 rows a kv head):
//   256   of heads of 128, 2 pages 8.7 and 13.7, 4 9.6 and 16.6
//   512   2 pages 10.8 and 14.5, 8 14.0 and 23.1
//   1,024 2 pages 18.7 and 15.7, 8 23.9 and 23.8, 32 55 and 58
//   2,048 2 pages 27.7 and 19.7, 8 37.2 and 30.7, 32 95 and 95
//   2,048 of heads of 256, 8 pages 66 and 49, 32 147 and 130; 4,096 of heads of 64, 32
//         pages 143 and 123
bool short_pays(int64_t segments, int64_t cols) {
  return (segments >= 2048 && cols <= 32) || (segments >= 1024 && cols <= 8);
}
// Branches up to which their live rows are counted through: one a lane.  (64 x 8 branches
// of up to 5 tokens, on average 3: 180 us, 242 with all rows; all of them live: 256 and
// 257; 8 x 48 of up to 3: 98 and 111.)
constexpr int32_t kCompactFan = 64;

// What a page costs a block of rows, in those of a block of one tile: more tiles share
// the conversion of its codes, wide blocks (of up to 192 and 128 rows) yet more.
double block_cost(bool wide, int tiles, int32_t d) {
  if (wide) return d == 128 ? 4.2 : 3.8;
  return tiles == 1 ? 1.0 : tiles == 2 ? 1.2 : tiles == 3 ? 1.3 : 2.6;
}
// Whether a prefix's pages are read for all its branches at once, or by each branch
// before its own.  Sharing them saves the branches' blocks the pages, at 0.8, 1.3 or
// 1.6 ns each for the whole GPU, and costs a pass more, 9 us, another one where only
// the prefixes' segments are cut, and the rows' records: written and read at 4 TB/s, what
// is past 32 MB at a quarter of that.  Of counted branches some rows are taken not to
// be live.  Whole calls, us, by each branch and shared:
//   heads of 128  4 samples of one prompt of 777 tokens, 8 kv heads: 11.7 and 16.6; 16
//                 such prompts of 777 15.6 and 19.1, of 2,000 27.0 and 27.9, of 4,000 44
//                 and 33; 64 x 8 branches of 20 rows behind 512 tokens 61 and 88, 1,000
//                 105 and 114, 2,000 249 and 169
//   heads of 64   96 branches of 2 rows, 16 kv heads, 200 tokens 13.4 and 17.5, 500 23.1
//                 and 20.0, 2,000 50 and 35; 32 x 16 of 8 rows, 4 kv heads, 512 tokens
//                 20.8 and 26.1 (the rule reads them by each), 1,024 34.3 and 32.3
//   heads of 256  8 x 45 branches of 14 rows, 16 kv heads, 1,024 tokens 178 and 213; 4 x
//                 6 of 63 rows, 4 kv heads, 4,096 tokens 67 and 72, 8,155 116 and 95
// The rule sees the table's width and not the prefixes' lengths.
bool shared_pays(const PrefixShape& shape, const sv::C4AttnArgs& A, int tiles, int64_t each, int64_t prefixes,
                 int64_t cols, int64_t rows, int32_t d, bool compact) {
  const double blocks = double(shape.blocks) * block_cost(shape.wide, shape.tiles, d) * (compact ? 0.6 : 1.0);
  const double branches = double(each) * double(A.row_blocks) * block_cost(false, tiles, d);
  const double page = d == 64 ? 0.83e-3 : d == 128 ? 1.3e-3 : 1.6e-3;
  const double saved = (branches - blocks) * double(prefixes * A.cache.heads) * double(cols) * page;
  const bool cut = cols > kAttnWhole && each_pays(int64_t(A.B) * A.cache.heads * A.row_blocks, cols + A.cache.table_cols);
  const double mb = double(rows) * d * 8 / 1e6;
  return saved > 9.0 + (cut ? 10.0 : 0.0) + mb / 4 + std::max(mb - 32, 0.0) * 0.75;
}

// A call's workspace: the rows' records, and one attention's after the other.
// Its size does not go by the tables, of which a size query knows nothing.
struct SharedSpace {
  size_t rec, stat, scratch;
  size_t bytes() const { return rec + stat + scratch; }
};
SharedSpace shared_space(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t d, int32_t fan) {
  const size_t count = size_t(B) * size_t(T) * size_t(q_heads);
  const int64_t rows = int64_t(std::min(fan, B)) * T * (q_heads / kv_heads);
  int tiles;
  int64_t blocks;
  row_blocks(rows, d, &tiles, &blocks);
  const size_t prefix = std::max(shape_workspace(d, tiles), wide_rows(rows, d) ? wide_workspace(d) : 0);
  return {align256(count * size_t(d) * 4), align256(count * 16),
          std::max(attention_workspace(T, q_heads, kv_heads, d), prefix)};
}

// The branches' pass, over at most `cols` pages each.
template <typename Args>
void launch_own(Args& A, int32_t d, int tiles, int64_t cols, void* scratch, hipStream_t st) {
  const int64_t segments = int64_t(A.B) * A.cache.heads * A.row_blocks, grid = (segments + 3) / 4;
  A.split = !each_pays(segments, cols);
  if (short_pays(segments, cols) && grid_fits(grid, 256))
    with_shape(d, tiles, [&](auto D, auto RT) {
      hipLaunchKernelGGL((sv::k_attention_cache4_short<D, RT, Args>), dim3(unsigned(grid)), dim3(256), 0, st, A);
    });
  else
    with_shape(d, tiles, [&](auto D, auto RT) { launch_attention<D, RT>(A, scratch, st); });
}

}  // namespace

extern "C" {

size_t spec_attention_cache4_shared_workspace(int32_t B, int32_t T, int32_t q_heads, int32_t heads,
                                              int32_t head_dim, int32_t fan) {
  if (check_attention_sizes(B, T, q_heads, heads, head_dim) != SPEC_OK || !shared_sizes_ok(B, T, q_heads, fan)) return 0;
  return shared_space(B, T, q_heads, heads, head_dim, fan).bytes();
}

int spec_attention_cache4_shared(spec_cache4_t cache, const int32_t* prefix_table,
                                 int64_t prefix_stride, int32_t prefix_cols,
                                 const int32_t* prefix_len, int32_t fan, spec_heads_t q, int32_t B,
                                 int32_t T, int32_t q_heads, const int32_t* start,
                                 const int32_t* count, const uint32_t* mask,
                                 int64_t mask_seq_stride, int64_t mask_pos_stride, float scale,
                                 spec_heads_t out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  sv::C4AttnArgs base;
  int rc, tiles;
  if (fan < 1) return SPEC_ERR_INVALID_ARG;
  if ((rc = attention_args(cache, q, B, T, q_heads, start, count, mask, mask_seq_stride, mask_pos_stride, scale, out,
                           lse, workspace, workspace_bytes, &base, &tiles)) != SPEC_OK)
    return rc;
  if (!shared_sizes_ok(B, T, q_heads, fan)) return SPEC_ERR_UNSUPPORTED;
  spec_cache4_t prefix = cache;
  prefix.table = prefix_table;
  prefix.table_stride = prefix_stride;
  prefix.table_cols = prefix_cols;
  if ((rc = check_cache(prefix)) != SPEC_OK) return rc;
  if (!prefix_len || !aligned(prefix_len, 4)) return SPEC_ERR_INVALID_ARG;
  const int32_t d = cache.head_dim, each = std::min(fan, B), prefixes = (B + each - 1) / each;
  const bool compact = count && each <= kCompactFan;
  const PrefixShape shape = prefix_shape(int64_t(each) * T * (q_heads / cache.heads), d, int64_t(prefixes) * cache.heads, prefix_cols,
                                         compact);
  if (prefixes * (int64_t(prefix_cols) + sv::kC4SegCost) * cache.heads >= (int64_t(1) << 40) / shape.blocks)
    return SPEC_ERR_UNSUPPORTED;
  const int64_t rows = int64_t(B) * T * q_heads;
  if (!shared_pays(shape, base, tiles, each, prefixes, prefix_cols, rows, d, compact)) {
    const int64_t cols = int64_t(prefix_cols) + cache.table_cols;
    if (int64_t(B) * (cols + sv::kC4SegCost) * cache.heads < (int64_t(1) << 40) / base.row_blocks) {
      sv::C4BehindArgs A;
      static_cast<sv::C4AttnArgs&>(A) = base;
      A.prefix = view(prefix);
      A.prefix_len = prefix_len;
      A.fan = each;
      if (workspace_bytes < shared_space(B, T, q_heads, cache.heads, d, fan).bytes()) return SPEC_ERR_WORKSPACE;
      auto st = static_cast<hipStream_t>(stream);
      (void)hipGetLastError();
      launch_own(A, d, tiles, cols, workspace, st);
      return finish_launch();
    }
  }
  const SharedSpace space = shared_space(B, T, q_heads, cache.heads, d, fan);
  if (workspace_bytes < space.bytes()) return SPEC_ERR_WORKSPACE;
  auto* const rec = static_cast<float*>(workspace);
  auto* const stat = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + space.rec);
  void* const scratch = static_cast<uint8_t*>(workspace) + space.rec + space.stat;

  sv::C4PrefixArgs P;
  static_cast<sv::C4AttnArgs&>(P) = base;
  P.cache = view(prefix);
  P.start = prefix_len;
  P.B = prefixes;
  P.row_blocks = int32_t(shape.blocks);
  P.block_rows = shape.wide ? shape.block_rows : 16 * shape.tiles;
  P.compact = compact;
  P.split = prefix_cols > kAttnWhole;
  P.fan = each;
  P.seqs = B;
  P.dim = d;
  P.rec = rec;
  P.stat = stat;
  sv::C4OwnArgs O;
  static_cast<sv::C4AttnArgs&>(O) = base;
  O.dim = d;
  O.rec = rec;
  O.stat = stat;
  auto st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (shape.wide) with_wide(d, [&](auto D) { launch_wide<D>(P, P.block_rows, scratch, st); });
  else with_shape(d, shape.tiles, [&](auto D, auto RT) { launch_attention<D, RT>(P, scratch, st); });
  launch_own(O, d, tiles, cache.table_cols, scratch, st);
  return finish_launch();
}

}  // extern "C"
