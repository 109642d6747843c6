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

// All pages that go back are counted through in the order of (sequence, page), and
// so are those that are taken.  Page j that goes back stands at full - 1 - j of
// the free pages, `full` being how many there are before the first is taken, and
// page j that is taken comes from there: with fewer than j + 1 pages going back
// from among those that were free before.  So index j alone says what is read
// and what is written, for both together, and no two write or read what the
// other writes.  Which sequence it is of follows from the sums over the
// sequences before: a search in those.
struct ReservePlan {
  int64_t full, gives, takes;  // takes: of the sequences that are served
};

// The first of n ascending sums (each with its own element) that passes j.
__device__ __forceinline__ int32_t res_find(const int32_t* upto, int32_t n, int32_t j) {
  int32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (upto[mid] > j) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Moves pages j, j + step, ..  held: as it is after the call.
__device__ __forceinline__ void res_move(const ReserveArgs& A, const ReservePlan& P, const int32_t* give_upto,
                                         const int32_t* take_upto, const int32_t* held, int64_t j, int64_t step) {
  for (const int64_t end = P.gives > P.takes ? P.gives : P.takes; j < end; j += step) {
    int32_t* const top = A.free_pages + (P.full - 1 - j);
    int32_t page;
    if (j < P.gives) {
      const int32_t b = res_find(give_upto, A.B, (int32_t)j), before = b ? give_upto[b - 1] : 0;
      int32_t* const at = A.table + b * A.table_stride + held[b] + ((int32_t)j - before);
      page = *at;
      *at = -1;
      *top = page;
    } else {
      page = *top;
    }
    if (j < P.takes) {
      const int32_t b = res_find(take_upto, A.B, (int32_t)j);
      A.table[b * A.table_stride + held[b] - (take_upto[b] - (int32_t)j)] = page;
    }
  }
}

constexpr int kResThreads = 1024;

// Integers only.  Bound by loads that wait for each other and by launches: lengths,
// sums, a search, a page (64 sequences 5.7 us; 4,093 7.6 for the sums and 7.9 for
// 24,000 pages, their 1,000 slots each 8.2, 33 MB at 4 TB/s).
// The sums, by one workgroup, a run of `per` sequences a thread: into give_upto
// and take_upto, with the lengths after the call in held (which may be A.held).
// False where nothing may change.  Sums of what is taken past what there is
// stand as one past the free pages: no page is searched for there.
__device__ __forceinline__ bool res_plan(const ReserveArgs& A, ReservePlan& P, int32_t* give_upto, int32_t* take_upto,
                                         int32_t* held_after) {
  __shared__ int64_t gives[kResThreads / 64], takes[kResThreads / 64];
  __shared__ unsigned long long used;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int32_t per = (A.B + kResThreads - 1) / kResThreads;
  const int32_t b0 = min(tid * per, A.B), b1 = min(b0 + per, A.B);
  int64_t give = 0, take = 0;
  // the first few stay in registers
  constexpr int kKeep = 4;
  int32_t held[kKeep] = {}, want[kKeep] = {};
#pragma unroll
  for (int x = 0; x < kKeep; ++x)
    if (b0 + x < b1) res_pages(A, b0 + x, held[x], want[x]);
#pragma unroll
  for (int x = 0; x < kKeep; ++x) {
    give += max(held[x] - want[x], 0);
    take += max(want[x] - held[x], 0);
  }
  for (int32_t b = b0 + kKeep; b < b1; ++b) {
    int32_t h, n;
    res_pages(A, b, h, n);
    give += max(h - n, 0);
    take += max(n - h, 0);
  }
  const int64_t free0 = *A.free_count;
  int64_t give_at = c4_prefix(give, lane), take_at = c4_prefix(take, lane);
  if (lane == 63) gives[w] = give_at, takes[w] = take_at;
  if (tid == 0) used = 0;
  __syncthreads();
  give_at -= give;
  take_at -= take;
  P.gives = 0;
#pragma unroll
  for (int x = 0; x < kResThreads / 64; ++x) {
    if (x < w) give_at += gives[x], take_at += takes[x];
    P.gives += gives[x];
  }
  P.full = free0 + P.gives;
  if (free0 < 0 || P.full > A.capacity) return false;
  int64_t most = 0;
  auto put = [&](int32_t b, int32_t h, int32_t n) {
    give_at += max(h - n, 0);
    take_at += max(n - h, 0);
    const bool served = take_at <= P.full;
    if (served) most = take_at;
    give_upto[b] = (int32_t)give_at;
    take_upto[b] = served ? (int32_t)take_at : 0x7FFFFFFF;
    held_after[b] = n < h || served ? n : h;
  };
#pragma unroll
  for (int x = 0; x < kKeep; ++x)
    if (b0 + x < b1) put(b0 + x, held[x], want[x]);
  for (int32_t b = b0 + kKeep; b < b1; ++b) {
    int32_t h, n;
    res_pages(A, b, h, n);
    put(b, h, n);
  }
  // sums ascend with the threads: the wave's last served one has its largest
  const uint64_t any = __ballot(most > 0);
  if (any && lane == 63 - __builtin_clzll(any)) atomicMax(&used, (unsigned long long)most);
  __syncthreads();
  P.takes = (int64_t)used;
  return true;
}

// Few sequences: all of it by one workgroup.  A second launch would cost a call 0.7
// us (100 sequences there and back with slots 15.3 us, with two launches 16.6), and
// pages that one workgroup moves by itself more and more (1,000 sequences 30 % of
// which end: 61.4, with two 25.3; 512: 30.5).  The rule sees the sequences, not their
// pages: 128 of 512 pages each, all taken and given back, 99.9 us, of 2,048 374; 129 of
// either 25.6.
constexpr int32_t kResFew = 128;
__global__ __launch_bounds__(kResThreads) void k_cache4_reserve(ReserveArgs A) {
  __shared__ int32_t give_upto[kResFew], take_upto[kResFew], held[kResFew];
  ReservePlan P;
  if (!res_plan(A, P, give_upto, take_upto, held)) return;
  res_move(A, P, give_upto, take_upto, held, threadIdx.x, kResThreads);
  if ((int32_t)threadIdx.x < A.B) A.held[threadIdx.x] = held[threadIdx.x];
  if (threadIdx.x == 0) *A.free_count = (int32_t)(P.full - P.takes);
}

// Many: the sums by one workgroup, into `scratch` [plan, give_upto, take_upto], and
// the pages by as many as it takes.
__global__ __launch_bounds__(kResThreads) void k_cache4_reserve_plan(ReserveArgs A, ReservePlan* plan, int32_t* upto) {
  ReservePlan P;
  const bool ok = res_plan(A, P, upto, upto + A.B, A.held);
  if (threadIdx.x) return;
  if (ok) *A.free_count = (int32_t)(P.full - P.takes);
  else P.full = P.gives = P.takes = 0;
  *plan = P;
}
__global__ __launch_bounds__(256) void k_cache4_reserve_move(ReserveArgs A, const ReservePlan* plan, const int32_t* upto) {
  res_move(A, *plan, upto, upto + A.B, A.held, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
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

__device__ __forceinline__ int64_t slot_of(const SlotArgs& A, int64_t b, int32_t s, int32_t n, int32_t i) {
  const C4View cache{nullptr, A.table, A.table_stride, A.n_pages, A.table_cols, 0};
  if (!cache.fits(s, n, A.T) || i >= n) return -1;
  const int32_t pos = s + i, page = cache.page(b, pos / kC4Page);
  return page < 0 ? -1 : (int64_t)page * kC4Page + pos % kC4Page;
}

// Few tokens a sequence: a token a thread, whatever its sequence.
__global__ __launch_bounds__(256) void k_cache4_slots(SlotArgs A) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x >= A.tokens) return;
  // as a rule all of it has 32 bits
  const int64_t b = A.tokens >> 31 ? x / A.T : (uint32_t)x / (uint32_t)A.T;
  A.slots[x] = slot_of(A, b, A.start[b], A.count ? A.count[b] : A.T, (int32_t)(x - b * A.T));
}
// Many: four tokens of one sequence a thread.
constexpr int kSlotsRun = 4 * 256;
__global__ __launch_bounds__(256) void k_cache4_slots_run(SlotArgs A) {
  const int64_t b = blockIdx.x;
  const int32_t s = c4_scalar(A.start + b), n = A.count ? c4_scalar(A.count + b) : A.T;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int32_t i = (int32_t)blockIdx.y * kSlotsRun + k * 256 + threadIdx.x;
    if (i < A.T) A.slots[b * A.T + i] = slot_of(A, b, s, n, i);
  }
}

}  // namespace sv
