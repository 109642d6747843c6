// Host code of the serving step's calls under sanitizers: every size query and
// refusal, at the ends of the arguments' ranges.  No call here launches a kernel.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "specverify_step.h"

static int bad = 0;
#define REFUSED(call) do { if ((call) == SPEC_OK) { ++bad; std::printf("accepted: %s\n", #call); } } while (0)

int main() {
  constexpr int32_t big = std::numeric_limits<int32_t>::max(), low = std::numeric_limits<int32_t>::min();
  constexpr int64_t wide = std::numeric_limits<int64_t>::max() - 15, under = std::numeric_limits<int64_t>::min();
  void* p = reinterpret_cast<void*>(uintptr_t(1) << 20);
  void* odd = reinterpret_cast<void*>((uintptr_t(1) << 20) + 2);
  auto* c32 = static_cast<const int32_t*>(p);
  auto* m32 = static_cast<int32_t*>(p);
  const int32_t ends[] = {low, -1, 0, 1, 2, 63, 64, 65, 128, 256, 257, 1024, 16384, 1 << 16, 1 << 24, 1 << 30, big};
  const spec_cache4_t good{p, c32, 4, 8, 4, 2, 128};
  const spec_heads_t x{p, SPEC_DTYPE_BF16, 0, 4096, 512, 128};
  for (int32_t a : ends)
    for (int32_t b : ends)
      for (int32_t c : ends) {
        (void)spec_attention_cache4_shared_workspace(a, b, c, 1, 128, c);
        (void)spec_attention_cache4_shared_workspace(1, a, b, c, 64, a);
        (void)spec_attention_cache4_shared_workspace(a, 256, 16384, 1, 256, b);
        // no workspace: refused whatever else holds
        REFUSED(spec_attention_cache4_shared(good, c32, 4, 4, c32, a, x, b, c, 2, c32, nullptr, nullptr, 0, 0, 1.0f, x,
                                             nullptr, nullptr, 0, nullptr));
        REFUSED(spec_attention_cache4_shared(good, c32, wide, a, c32, b, x, 2, 3, 2, c32, nullptr, nullptr, 0, 0, 1.0f, x,
                                             nullptr, p, 0, nullptr));
        REFUSED(spec_attention_cache4_window(good, x, 2, 3, 2, c32, nullptr, nullptr, 0, 0, nullptr, 0, a, b, 1.0f, x, nullptr,
                                             p, size_t(c < 0 ? 0 : c) & 1023, nullptr));
      }
  for (int32_t a : ends) {
    const spec_rotate_t how{128, 128, 0, 1, 1e-6f, SPEC_DTYPE_BF16, p, p, static_cast<const float*>(p), nullptr, 0};
    spec_rotate_t h = how;
    if (a < 16 || a > 256) {
      h.head_dim = a;
      REFUSED(spec_norm_rotate(x, x, 2, x, x, 1, &h, 2, 3, c32, nullptr, nullptr));
      h = how;
      h.rotary_dim = a;
      REFUSED(spec_norm_rotate(x, x, 2, x, x, 1, &h, 2, 3, c32, nullptr, nullptr));
      REFUSED(spec_cache4_reserve(m32, 4, a > 1 << 24 ? a : -1, m32, c32, 2, m32, 8, m32, p, 1 << 20, nullptr));
      REFUSED(spec_norm_rotate(x, x, 16384, x, x, a, &how, 2, 3, c32, nullptr, nullptr));
      REFUSED(spec_norm_rotate(x, x, a < 0 ? a : big, x, x, a, &how, 2, 3, c32, nullptr, nullptr));
    }
    if (a < 1 || a > 1 << 16) {
      REFUSED(spec_norm_rotate(x, x, 2, x, x, 1, &how, a, 3, c32, nullptr, nullptr));
      REFUSED(spec_cache4_reserve(m32, 4, 4, m32, c32, a, m32, 8, m32, p, 1 << 20, nullptr));
      REFUSED(spec_cache4_slots(c32, 4, 4, 8, a, 3, c32, nullptr, static_cast<int64_t*>(p), nullptr));
    }
    if (a < 1 || a > 1 << 24) REFUSED(spec_cache4_slots(c32, 4, 4, 8, 2, a, c32, nullptr, static_cast<int64_t*>(p), nullptr));
    if (a < 1) REFUSED(spec_cache4_reserve(m32, 4, 4, m32, c32, 2, m32, a, m32, p, 1 << 20, nullptr));
  }
  const spec_rotate_t how{128, 128, 0, 1, 1e-6f, SPEC_DTYPE_BF16, p, p, static_cast<const float*>(p), nullptr, 0};
  REFUSED(spec_norm_rotate(x, x, 2, x, x, 1, &how, 1 << 16, 1 << 24, c32, nullptr, nullptr));
  REFUSED(spec_cache4_slots(c32, 4, 4, 8, 1 << 16, 1 << 24, c32, nullptr, static_cast<int64_t*>(p), nullptr));
  for (int64_t s : {under, int64_t(-1), int64_t(-8), int64_t(4), wide})
    for (const spec_heads_t& y : {spec_heads_t{p, SPEC_DTYPE_BF16, 0, s, 512, 128}, spec_heads_t{p, SPEC_DTYPE_BF16, 0, 4096, s, 128},
                                  spec_heads_t{p, SPEC_DTYPE_BF16, 0, 4096, 512, s}}) {
      if (s != wide) REFUSED(spec_norm_rotate(y, x, 2, x, x, 2, &how, 2, 3, c32, nullptr, nullptr));
      if (s != wide) REFUSED(spec_norm_rotate(x, y, 2, x, x, 2, &how, 2, 3, c32, nullptr, nullptr));
      REFUSED(spec_attention_cache4_window(good, x, 2, 3, 2, c32, nullptr, nullptr, s, s, c32, s, 4, 4, 1.0f, y, nullptr, p, 0,
                                           nullptr));
    }
  for (float c : {0.0f, -1.0f, -INFINITY, INFINITY, NAN, 3e38f, 1e-45f})
    REFUSED(spec_attention_cache4_shared(good, c32, 4, 4, c32, 2, x, 2, 3, 2, c32, nullptr, nullptr, 0, 0, c, x, nullptr, p, 0,
                                         nullptr));
  REFUSED(spec_cache4_reserve(static_cast<int32_t*>(odd), 4, 4, m32, c32, 2, m32, 8, m32, p, 1 << 20, nullptr));
  std::printf(bad ? "bad %d\n" : "sanitized step validation ok\n", bad);
  return bad != 0;
}
