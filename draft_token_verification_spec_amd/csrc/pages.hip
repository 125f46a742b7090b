// Pages of a cache taken and given back as requests' lengths say, and the slots
// of the new tokens.
//
// The free pages are a stack.  With need_b = ceil(kv_len[b] / page size) and
// held_b pages of request b,
//   give_b = max(held_b - need_b, 0),  take_b = max(need_b - held_b, 0),
// the k-th page given back over all requests goes to place
// count + sum(give) - 1 - k of the stack, and the k-th taken comes from place
// C - 1 - k of the C = count + sum(give) pages then on it: exclusive sums over
// the requests, and copies.  Taking right after is thus undone by giving back,
// to the entry.
//
// Bound by latency: a scan and three dependent copies.  Up to 1024 requests
// and kSmallRows rows one workgroup does it all, the copies shared evenly over
// its threads, each of which finds its item's request by a search in LDS.
// Otherwise two launches: the sums with the pages given back, by workgroups of
// 64 requests or more (several for one such part, where there are few), each of
// which adds up all requests for itself, and the pages taken with the slots, by
// workgroups of one request each.
//
// Measured: 256 requests that grow by 5 tokens 6.5 us; 1500 prompts of up to 1000
// tokens (55 thousand pages, 940 thousand rows) 7 + 7 us, and given back 10 + 4.
// The pages themselves do not choose the launch: where up to 1024 requests take or
// give back very many in a call of few rows, one workgroup moves them all (64
// requests of 131072 tokens, 524 thousand pages, 350 us either way).
// pages_give_kernel fills the 128 registers of 1024 threads and spills 17.
#include "sv_attn.hpp"

namespace sv {

namespace {

constexpr int kPagesThreads = 1024;
constexpr int kMoveThreads = 256;

struct Change {
  int held, need;  // pages; need is not below the shared ones that are held
  bool fits;       // the page table's row can hold `need` pages
  __device__ __forceinline__ int give() const { return fits && held > need ? held - need : 0; }
  __device__ __forceinline__ int take() const { return fits && need > held ? need - held : 0; }
};

__device__ __forceinline__ Change change_of(const PagesArgs& a, int b, int held) {
  Change c;
  c.held = min(max(held, 0), a.max_pages);
  const int len = max(a.kv_len[b], 0);
  c.need = int((int64_t(len) + (1 << a.page_shift) - 1) >> a.page_shift);
  c.fits = c.need <= a.max_pages;
  if (a.shared) c.need = max(c.need, min(a.shared[b], c.held));
  return c;
}

__device__ __forceinline__ int64_t pages_on_stack(const PagesArgs& a) {
  return min(max(*a.free_count, 0), a.num_pages);
}

__device__ __forceinline__ int64_t wave_total(int64_t x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(static_cast<long long>(x), o, 64);
  return x;
}

// Exclusive sums over the workgroup of two numbers per thread, and the sums of
// these and of three more over all threads.
struct Sums {
  longlong2 before, total;
  int64_t more[3];
};
struct SumsLds {
  longlong2 pairs[kPagesThreads / 64];
  int64_t more[3][kPagesThreads / 64];
};
template <int MORE>
__device__ __forceinline__ Sums sum_up(longlong2 x, const int64_t (&more)[3], SumsLds& lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  longlong2 upto = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t p = __shfl_up(static_cast<long long>(upto.x), o, 64), q = __shfl_up(static_cast<long long>(upto.y), o, 64);
    if (lane >= o) upto.x += p, upto.y += q;
  }
  if (lane == 63) lds.pairs[wave] = upto;
#pragma unroll
  for (int i = 0; i < MORE; ++i) {
    const int64_t t = wave_total(more[i]);
    if (lane == 0) lds.more[i][wave] = t;
  }
  __syncthreads();
  Sums s = {{upto.x - x.x, upto.y - x.y}, {0, 0}, {0, 0, 0}};
  for (int w = 0; w < kPagesThreads / 64; ++w) {
    const longlong2 p = lds.pairs[w];
    if (w < wave) s.before.x += p.x, s.before.y += p.y;
    s.total.x += p.x, s.total.y += p.y;
#pragma unroll
    for (int i = 0; i < MORE; ++i) s.more[i] += lds.more[i][w];
  }
  return s;
}

// The last of n ascending entries that is at most x (the first is).
template <typename E, typename X>
__device__ __forceinline__ int last_upto(const E* v, int n, X x) {
  int lo = 0;
  for (int step = n <= 64 ? 32 : 512; step > 0; step >>= 1)
    if (lo + step < n && v[lo + step] <= x) lo += step;
  return lo;
}

// The pages given back by n requests from b0 on: the k-th of `total`, of the last
// request r with from[r] <= k, to place top - k of the stack; by `slices`
// workgroups, four a thread at a time.
__device__ __forceinline__ void give_back(const PagesArgs& a, int b0, int n, const int64_t* from, const int* need,
                                          int64_t total, int64_t top, int slice, int slices) {
  constexpr int kAtATime = 4;
  for (int64_t k0 = int64_t(slice) * kAtATime * kPagesThreads + threadIdx.x; k0 < total;
       k0 += int64_t(slices) * kAtATime * kPagesThreads) {
    int32_t* entry[kAtATime];
    int page[kAtATime];
#pragma unroll
    for (int i = 0; i < kAtATime; ++i) {
      const int64_t k = min(k0 + i * kPagesThreads, total - 1);
      const int r = last_upto(from, n, k);
      entry[i] = a.table + (b0 + r) * a.table_stride + need[r] + (k - from[r]);
    }
#pragma unroll
    for (int i = 0; i < kAtATime; ++i) page[i] = *entry[i];
#pragma unroll
    for (int i = 0; i < kAtATime; ++i) {
      const int64_t k = k0 + i * kPagesThreads, at = top - k;
      if (k >= total) break;
      if (at >= 0 && at < a.num_pages) a.free_pages[at] = page[i];
      *entry[i] = -1;
    }
  }
}

// The slot of a row at `place` of a request that holds `held` pages, of which
// those from `old` on are the taken-th and following ones taken of `count`.
__device__ __forceinline__ void put_row(const PagesArgs& a, int t, int b, int64_t place, int held, int old, int64_t taken,
                                        int64_t count) {
  int64_t slot = -1;
  const int64_t i = place >> a.page_shift;
  if (place >= 0 && i < held) {
    const int page = i < old ? a.table[b * a.table_stride + i] : a.free_pages[count - 1 - (taken + i - old)];
    if (page >= 0 && page < a.num_pages) slot = (int64_t(page) << a.page_shift) + (place & ((1 << a.page_shift) - 1));
  }
  if (a.slots) a.slots[t] = slot;
  if (a.positions) a.positions[t] = place;
}

__global__ __launch_bounds__(kPagesThreads) void pages_small_kernel(PagesArgs a) {
  __shared__ SumsLds lds;
  __shared__ int64_t give_from[kPagesThreads], take_from[kPagesThreads];
  __shared__ int old[kPagesThreads], now[kPagesThreads], start[kPagesThreads + 1], length[kPagesThreads];
  const int b = threadIdx.x;
  const bool live = b < a.B;
  Change c = {0, 0, true};
  if (live) {
    c = change_of(a, b, a.held[b]);
    length[b] = max(a.kv_len[b], 0);
  }
  if (a.query_start)
    for (int i = b; i <= a.B; i += kPagesThreads) start[i] = a.query_start[i];
  const int64_t count0 = pages_on_stack(a);
  const Sums sums = sum_up<0>({c.give(), c.take()}, {0, 0, 0}, lds);
  const longlong2 from = sums.before, total = sums.total;
  const int64_t count = min(count0 + total.x, int64_t(a.num_pages));
  const int64_t upto = from.y + c.take();
  const bool granted = c.fits && (c.take() == 0 || upto <= count);
  if (live) {
    give_from[b] = from.x, take_from[b] = from.y;
    old[b] = c.held, now[b] = granted ? c.need : c.held;
    if (a.granted) a.granted[b] = granted;
    a.held[b] = now[b];
  }
  __syncthreads();  // (all have read the count)
  const bool crosses = live && upto > count && from.y <= count;  // the first request that is refused
  if (crosses || (b == a.B - 1 && upto <= count)) *a.free_count = int(count - (crosses ? from.y : upto));
  give_back(a, 0, a.B, give_from, now, total.x, count0 + total.x - 1, 0, 1);
  __syncthreads();
  for (int64_t k = b; k < min(total.y, count); k += kPagesThreads) {
    const int r = last_upto(take_from, a.B, k);
    const int i = int(k - take_from[r]);
    if (i < now[r] - old[r]) a.table[r * a.table_stride + old[r] + i] = a.free_pages[count - 1 - k];
  }
  if (!a.query_start) return;
  const int first = max(start[0], 0), end = min(start[a.B], a.T);
  for (int t = first + b; t < end; t += kPagesThreads) {
    const int r = last_upto(start, a.B, t);
    if (t < start[r] || t >= start[r + 1]) continue;
    put_row(a, t, r, int64_t(length[r]) - (int64_t(start[r + 1]) - t), now[r], old[r], take_from[r], count);
  }
}

// What the first launch leaves for the second: the pages on the stack after what
// is given back, [B] pairs of exclusive sums, [B] pages held before.
__device__ __forceinline__ longlong2* sums_of(const PagesArgs& a) { return static_cast<longlong2*>(a.scratch) + 1; }
__device__ __forceinline__ int32_t* held_of(const PagesArgs& a) { return reinterpret_cast<int32_t*>(sums_of(a) + a.B); }

// The sums of requests blockIdx.x * tile .. + tile - 1 (at most 1024 of them),
// and the pages that these give back, by gridDim.y workgroups.
__global__ __launch_bounds__(kPagesThreads) void pages_give_kernel(PagesArgs a, int tile) {
  __shared__ SumsLds lds;
  __shared__ int64_t give_from[kPagesThreads];
  __shared__ int need[kPagesThreads];
  const int b0 = blockIdx.x * tile, n = min(tile, a.B - b0);
  // what requests before ours give and take, and what all give
  int64_t more[3] = {0, 0, 0};
  for (int b = threadIdx.x; b < a.B; b += kPagesThreads) {
    const Change c = change_of(a, b, a.held[b]);
    more[2] += c.give();
    if (b < b0) more[0] += c.give(), more[1] += c.take();
  }
  const int b = b0 + threadIdx.x;
  Change c = {0, 0, true};
  if (int(threadIdx.x) < n) c = change_of(a, b, a.held[b]);
  const Sums s = sum_up<3>({c.give(), c.take()}, more, lds);
  if (int(threadIdx.x) < n) {
    if (blockIdx.y == 0) {
      sums_of(a)[b] = {s.more[0] + s.before.x, s.more[1] + s.before.y};
      held_of(a)[b] = c.held;
    }
    give_from[threadIdx.x] = s.before.x;
    need[threadIdx.x] = c.need;
  }
  __syncthreads();
  const int64_t count = pages_on_stack(a) + s.more[2];
  if (b == 0 && blockIdx.y == 0) *static_cast<longlong2*>(a.scratch) = {0, min(count, int64_t(a.num_pages))};
  give_back(a, b0, n, give_from, need, s.total.x, count - 1 - s.more[0], blockIdx.y, gridDim.y);
}

// Request blockIdx.x's pages that it takes, and its rows.
__global__ __launch_bounds__(kMoveThreads) void pages_take_kernel(PagesArgs a) {
  const int b = blockIdx.x, tid = blockIdx.y * kMoveThreads + threadIdx.x, all = gridDim.y * kMoveThreads;
  const Change c = change_of(a, b, held_of(a)[b]);
  const int64_t count = static_cast<longlong2*>(a.scratch)->y, from = sums_of(a)[b].y, upto = from + c.take();
  const bool granted = c.fits && (c.take() == 0 || upto <= count);
  const int now = granted ? c.need : c.held;
  if (tid == 0) {
    if (a.granted) a.granted[b] = granted;
    a.held[b] = now;
    const bool crosses = upto > count && from <= count;  // the first request that is refused
    if (crosses || (b == a.B - 1 && upto <= count)) *a.free_count = int(count - (crosses ? from : upto));
  }
  for (int i = tid; i < now - c.held; i += all)
    a.table[b * a.table_stride + c.held + i] = a.free_pages[count - 1 - (from + i)];
  if (!a.query_start) return;
  const int64_t start = a.query_start[b], end = a.query_start[b + 1], len = max(a.kv_len[b], 0);
  for (int64_t t = max(start, int64_t(0)) + tid; t < min(end, int64_t(a.T)); t += all)
    put_row(a, int(t), b, len - (end - t), now, c.held, from, count);
}

// Rows that one workgroup takes along (a step taken and given back, one launch
// and two: 256 requests of 1280 rows 15.6 and 20.1 us, a prompt of 4000 14.4 and
// 17.8; 1000 requests of 5000 rows 24.5 and 22.0, 256 of 10394 34.7 and 20.3).
constexpr int kSmallRows = 4096;

bool small(int B, int T) { return B <= kPagesThreads && T <= kSmallRows; }

}  // namespace

size_t pages_scratch(int B, int T) {
  return small(B, T) ? 0 : sizeof(longlong2) * (size_t(B) + 1) + sizeof(int32_t) * size_t(B);
}

hipError_t launch_pages(const PagesArgs& a, hipStream_t stream) {
  if (small(a.B, a.T)) {
    hipLaunchKernelGGL(pages_small_kernel, dim3(1), dim3(kPagesThreads), 0, stream, a);
    return hipGetLastError();
  }
  // workgroups for few requests of many rows: four for a compute unit
  int per = (1024 + a.B - 1) / a.B;
  const int rows = (a.T + a.B - 1) / a.B, most = (rows + kMoveThreads - 1) / kMoveThreads;
  per = per < most ? per : most;
  const dim3 grid(a.B, per < 1 ? 1 : per);
  // (64 requests a workgroup keep those that give back much apart)
  const int even = (a.B + 255) / 256, tile = even < 64 ? 64 : even;
  const int tiles = (a.B + tile - 1) / tile, slices = tiles >= 128 ? 1 : tiles > 8 ? 128 / tiles : 16;
  hipLaunchKernelGGL(pages_give_kernel, dim3(tiles, slices), dim3(kPagesThreads), 0, stream, a, tile);
  hipLaunchKernelGGL(pages_take_kernel, grid, dim3(kMoveThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace sv
