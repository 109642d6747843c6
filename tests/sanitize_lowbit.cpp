// Host code of the low-bit calls under sanitizers: every size query and every
// refusal, at the ends of the arguments' ranges.  No call here launches a kernel.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "specverify_lowbit.h"

static int bad = 0;
#define REFUSED(call) do { if ((call) == SPEC_OK) { ++bad; std::printf("accepted: %s\n", #call); } } while (0)

int main() {
  constexpr int32_t big = std::numeric_limits<int32_t>::max(), low = std::numeric_limits<int32_t>::min();
  constexpr int64_t wide = std::numeric_limits<int64_t>::max() - 15, under = std::numeric_limits<int64_t>::min();
  void* p = reinterpret_cast<void*>(uintptr_t(1) << 20);
  void* odd = reinterpret_cast<void*>((uintptr_t(1) << 20) + 2);
  auto* i32 = static_cast<const int32_t*>(p);
  auto* f32 = static_cast<float*>(p);
  const int32_t ends[] = {low, -1, 0, 1, 2, 63, 64, 65, 128, 129, 256, 257, 1024, 1 << 16, 1 << 24, big};
  for (int32_t a : ends) {
    bad += (spec_cache4_record_bytes(a) != 0) != (a == 64 || a == 128 || a == 256);
    for (int32_t b : ends)
      for (int32_t c : ends) {
        (void)spec_attention_cache4_workspace(a, b, c, 1, 128);
        (void)spec_attention_cache4_workspace(1, a, b, c, 64);
        (void)spec_attention_cache4_workspace(1, 1, a, b, c);
        (void)spec_lmhead_fp8_workspace(a, b, c);
      }
  }
  const spec_cache4_t good{p, i32, 4, 8, 4, 2, 128};
  const spec_heads_t x{p, SPEC_DTYPE_BF16, 0, 4096, 512, 128};
  auto heads = [&](void* d, int32_t t, int64_t s, int64_t i, int64_t h) { return spec_heads_t{d, t, 0, s, i, h}; };
  for (int32_t a : ends) {
    for (int32_t b : ends) {
      // no workspace: refused whatever else holds
      REFUSED(spec_attention_cache4(good, x, a, b, 2, i32, nullptr, nullptr, 0, 0, 1.0f, x, nullptr, nullptr, 0, nullptr));
      REFUSED(spec_attention_cache4({p, i32, wide, a, b, 2, 128}, x, 2, 3, 2, i32, nullptr, nullptr, 0, 0, 1.0f, x,
                                    nullptr, p, 0, nullptr));
      REFUSED(spec_attention_cache4({p, i32, wide, 8, 4, a, b}, x, 2, 3, 2, i32, nullptr, nullptr, 0, 0, 1.0f, x,
                                    nullptr, p, 0, nullptr));
      REFUSED(spec_lmhead_fp8({p, SPEC_DTYPE_F32, 0, 4096, 512}, a, b, 128, p, 128, f32, 300,
                              {p, SPEC_DTYPE_F32, 0, 1 << 20, 512}, nullptr, 0, nullptr));
      REFUSED(spec_lmhead_fp8({p, SPEC_DTYPE_F32, 0, 4096, 512}, 2, 3, a, p, wide, f32, b,
                              {p, SPEC_DTYPE_F32, 0, wide, wide}, p, 0, nullptr));
      if (a != big) REFUSED(spec_quantize_fp8(p, SPEC_DTYPE_F32, under, a, b, p, f32, nullptr));
    }
    if (a < 1 || a > 1 << 16) REFUSED(spec_cache4_write(good, x, x, a, 3, i32, nullptr, nullptr));
    if (a < 1 || a > 1 << 24) REFUSED(spec_cache4_read(good, x, x, 2, a, i32, nullptr, nullptr));
  }
  REFUSED(spec_quantize_fp8(p, SPEC_DTYPE_F32, wide - 1, 300, 128, p, f32, nullptr));
  REFUSED(spec_cache4_write(good, x, x, 1 << 16, 1 << 24, i32, nullptr, nullptr));
  for (int64_t s : {under, int64_t(-1), int64_t(-8), int64_t(4), wide}) {
    for (const spec_heads_t& y : {heads(p, SPEC_DTYPE_BF16, s, 512, 128), heads(p, SPEC_DTYPE_BF16, 4096, s, 128),
                                  heads(p, SPEC_DTYPE_BF16, 4096, 512, s)}) {
      if (s != wide) REFUSED(spec_cache4_write(good, y, x, 2, 3, i32, nullptr, nullptr));
      REFUSED(spec_attention_cache4(good, x, 2, 3, 2, i32, nullptr, nullptr, 0, 0, 1.0f, y, nullptr, p, 0, nullptr));
    }
    REFUSED(spec_attention_cache4(good, x, 2, 3, 2, i32, nullptr, static_cast<uint32_t*>(p), s, s, 1.0f, x, nullptr, p, 0,
                                  nullptr));
  }
  for (float c : {0.0f, -1.0f, -INFINITY, INFINITY, NAN, 3e38f, 1e-45f})
    REFUSED(spec_attention_cache4(good, x, 2, 3, 2, i32, nullptr, nullptr, 0, 0, c, x, nullptr, p, 0, nullptr));
  REFUSED(spec_cache4_read({odd, i32, 4, 8, 4, 2, 128}, x, x, 2, 3, i32, nullptr, nullptr));
  REFUSED(spec_cache4_read(good, heads(odd, SPEC_DTYPE_BF16, 4096, 512, 128), x, 2, 3, i32, nullptr, nullptr));
  std::printf(bad ? "bad %d\n" : "sanitized low-bit validation ok\n", bad);
  return bad != 0;
}
