// sv_pages.hpp -- each sequence's pages reserved and given back from lengths in
// device memory, and the slots of its new tokens (gfx950, wave64).
#pragma once

#include "sv_cache4.hpp"

namespace sv {

struct ReserveArgs {
  int32_t* table;
  int64_t table_stride;
  int32_t* held;
  const int32_t* need;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t table_cols, B, capacity;
};

// Pages that sequence b holds and shall hold; both its own where it is
// ill-formed.
__device__ __forceinline__ void res_pages(const ReserveArgs& A, int32_t b, int32_t& held, int32_t& want) {
  held = A.held[b];
  const int32_t need = A.need[b];
  want = need > 0 ? (need - 1) / kC4Page + 1 : 0;
  if (need < 0 || held < 0 || held > A.table_cols || want > A.table_cols) want = held;
}

// Moves `pages` pages between a row of the table and the stack, whose ends are
// `row` (the first of them) and `top` (one past its place): page p stands at
// top - 1 - p.
template <bool GIVE>
__device__ __forceinline__ void res_move(int32_t* row, int32_t* top, int32_t p) {
  if constexpr (GIVE) {
    top[-1 - p] = row[p];
    row[p] = -1;
  } else {
    row[p] = top[-1 - p];
  }
}
constexpr int32_t kResOwn = 8;  // pages that a thread moves by itself; more are a wave's
template <bool GIVE>
__device__ __forceinline__ void res_run(int32_t* row, int32_t* top, int32_t pages) {
  const int lane = threadIdx.x & 63;
  if (pages <= kResOwn)
    for (int32_t p = 0; p < pages; ++p) res_move<GIVE>(row, top, p);
  for (uint64_t many = __ballot(pages > kResOwn); many; many &= many - 1) {
    const int l = __builtin_ctzll(many);
    int32_t* const r = reinterpret_cast<int32_t*>(c4_lane(reinterpret_cast<int64_t>(row), l));
    int32_t* const t = reinterpret_cast<int32_t*>(c4_lane(reinterpret_cast<int64_t>(top), l));
    const int32_t n = __builtin_amdgcn_readlane(pages, l);
    for (int32_t p = lane; p < n; p += 64) res_move<GIVE>(r, t, p);
  }
}

constexpr int kResThreads = 1024;

// One workgroup, a run of sequences a thread: both sums over the sequences, then
// the pages that go back, then those that are taken, which may be among them.
__global__ __launch_bounds__(kResThreads) void k_cache4_reserve(ReserveArgs A) {
  __shared__ int64_t gives[kResThreads / 64], takes[kResThreads / 64];
  __shared__ unsigned long long used;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int32_t per = (A.B + kResThreads - 1) / kResThreads;
  const int32_t b0 = min(tid * per, A.B), b1 = min(b0 + per, A.B);
  int64_t give = 0, take = 0;
  for (int32_t b = b0; b < b1; ++b) {
    int32_t held, want;
    res_pages(A, b, held, want);
    give += max(held - want, 0);
    take += max(want - held, 0);
  }
  const int64_t free0 = *A.free_count;
  const int64_t give_upto = c4_prefix(give, lane), take_upto = c4_prefix(take, lane);
  if (lane == 63) gives[w] = give_upto, takes[w] = take_upto;
  if (tid == 0) used = 0;
  __syncthreads();
  int64_t give_at = give_upto - give, take_at = take_upto - take, full = free0;
  for (int x = 0; x < kResThreads / 64; ++x) {
    if (x < w) give_at += gives[x], take_at += takes[x];
    full += gives[x];
  }
  if (free0 < 0 || full > A.capacity) return;  // free0 below its capacity too, then
  // The threads of a wave go through their runs together; past its run a thread
  // has no pages to move.
  for (int32_t j = 0; j < per; ++j) {
    const int32_t b = b0 + j;
    int32_t held = 0, want = 0;
    if (b < b1) res_pages(A, b, held, want);
    const int32_t n = max(held - want, 0);
    res_run<true>(A.table + b * A.table_stride + want, A.free_pages + (full - give_at), n);
    give_at += n;
    if (n) A.held[b] = want;
  }
  __syncthreads();
  int64_t most = 0;
  for (int32_t j = 0; j < per; ++j) {
    const int32_t b = b0 + j;
    int32_t held = 0, want = 0;
    if (b < b1) res_pages(A, b, held, want);
    const int32_t miss = max(want - held, 0);
    take_at += miss;
    const bool served = miss > 0 && take_at <= full;
    res_run<false>(A.table + b * A.table_stride + held, A.free_pages + (full - (take_at - miss)), served ? miss : 0);
    if (served) {
      A.held[b] = want;
      most = take_at;
    }
  }
  if (most) atomicMax(&used, (unsigned long long)most);
  __syncthreads();
  if (tid == 0) *A.free_count = (int32_t)(full - (int64_t)used);
}

struct SlotArgs {
  const int32_t* table;
  int64_t table_stride;
  const int32_t* start;
  const int32_t* count;  // or null: T
  int64_t* slots;
  int64_t tokens;        // B T
  int32_t table_cols, n_pages, T;
};

__global__ __launch_bounds__(256) void k_cache4_slots(SlotArgs A) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x >= A.tokens) return;
  const int64_t b = x / A.T;
  const int32_t i = (int32_t)(x - b * A.T);
  const C4View cache{nullptr, A.table, A.table_stride, A.n_pages, A.table_cols, 0};
  const int32_t s = A.start[b], n = A.count ? A.count[b] : A.T;
  int64_t slot = -1;
  if (cache.fits(s, n, A.T) && i < n) {
    const int32_t pos = s + i, page = cache.page(b, pos / kC4Page);
    if (page >= 0) slot = (int64_t)page * kC4Page + pos % kC4Page;
  }
  A.slots[x] = slot;
}

}  // namespace sv
