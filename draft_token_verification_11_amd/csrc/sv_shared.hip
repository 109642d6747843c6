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
  // `rows` are far more than the live ones where those are counted through; heads of
  // 128 then gain nothing by wide blocks (64 x 8 heads, 96 of 160 rows live: 185 us
  // and 190)
  x.wide = wide_pays(rows, d, prefixes_heads, cols) && !(compact && d == 128);
  if (x.wide) wide_blocks(rows, d, &x.block_rows, &x.blocks);
  else row_blocks(rows, d, &x.tiles, &x.blocks);
  return x;
}
// Pages of a branch's own up to which a wave goes through them by itself.
constexpr int32_t kShortCols = 8;
// Branches up to which their live rows are counted through: one a lane.
constexpr int32_t kCompactFan = 64;

// Whether a prefix's pages are read for all its branches at once, or by each branch
// before its own.  Sharing them saves a block of rows of each branch the pages, at
// about 2.7 ns a page for the whole GPU (three blocks of 16 rows in one that shares
// the conversion cost a block of heads of 256 2.6 times as much), and costs further
// passes, 10 us, and the rows' records, written and read.  Whole calls, us, by each
// branch and shared:
//   heads of 128  4 branches of 4 rows, 8 kv heads, 777 tokens: 15 and 18; 16 such
//                 prefixes 21 and 18; 64 x 8 branches of 20 rows, 200 tokens 45 and 75,
//                 512 tokens 117 and 85
//   heads of 64   96 branches of 2 rows, 16 kv heads, 200 tokens 37 and 42 (the rule
//                 shares), 1,000 tokens 52 and 49; 32 x 16 branches of 8 rows, 256
//                 tokens 22 and 31 (the rule shares), 1,024 tokens 94 and 39
//   heads of 256  8 x 45 branches of 14 rows, 16 kv heads, 256 tokens 74 and 162, 1,024
//                 tokens 277 and 217; 4 x 6 of 63 rows, 4 kv heads, 2,048 tokens 46
//                 and 56, 8,155 tokens 127 and 80
// The rule sees the table's width and not the prefixes' lengths.
bool shared_pays(const PrefixShape& shape, int64_t each, int64_t prefixes, int64_t kv_heads, int64_t cols, int64_t rows,
                 int32_t d, int64_t branch_blocks) {
  const double blocks = shape.wide ? shape.blocks * 2.6 : double(shape.blocks);
  const double saved = (double(each) * double(branch_blocks) - blocks) * double(prefixes * kv_heads) * double(cols) * 0.0027;
  return saved > 10.0 + double(rows) * d * 8 / 4e6;
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
  const int64_t waves = int64_t(A.B) * A.cache.heads * A.row_blocks;
  if (cols <= kShortCols && grid_fits((waves + 3) / 4, 256))
    with_shape(d, tiles, [&](auto D, auto RT) {
      hipLaunchKernelGGL((sv::k_attention_cache4_short<D, RT, Args>), dim3(unsigned((waves + 3) / 4)), dim3(256), 0, st, A);
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
  if (!shared_pays(shape, each, prefixes, cache.heads, prefix_cols, rows, d, base.row_blocks)) {
    const int64_t cols = int64_t(prefix_cols) + cache.table_cols;
    if (int64_t(B) * (cols + sv::kC4SegCost) * cache.heads < (int64_t(1) << 40) / base.row_blocks) {
      sv::C4BehindArgs A;
      static_cast<sv::C4AttnArgs&>(A) = base;
      A.prefix = view(prefix);
      A.prefix_len = prefix_len;
      A.fan = each;
      A.split = cols > kAttnWhole;
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
