// Room in a paged cache for the next tokens of S requests.
//
// Everything is prefix sums over the requests: of the pages that ended ones give
// back (the free pages are a stack, these go on top), of the pages the others
// need (i-th of them: the i-th from the top), of their new tokens. One workgroup
// does that, 1024 requests at a time; pages are then dealt flat over its threads,
// each finding its request in the prefix sums by bisection in LDS, so that one
// long prompt is as fast as many short ones. What the stack gives a request is
// known from the counts alone, so table entries are written once and positions and
// slots need no second pass over them but a load.
//
// Few tokens (a decode step) are done by the same workgroup; many by a second
// kernel over all CUs. Bound by latency: about four dependent trips to memory.
#pragma once
#include "common.h"

namespace carve {

struct AssignArgs {
  const int *kv_lens, *new_lens, *done, *free_count;
  int *table, *free_pages, *kv_out, *cu, *positions, *count_out;
  int64_t* slots;
  int64_t table_row, capacity;
  int S, N, width, page_shift;
};

constexpr int kAssignThreads = 1024;
constexpr int kAssignTokens = 4096;                 // up to here the first kernel does the tokens too
constexpr int64_t kMostInt = 0x7fffffff;

// Exclusive prefix sums over the workgroup of two numbers; their totals in `all`.
struct Two { int64_t a, b; };
__device__ __forceinline__ Two scan_two(Two x, Two& all) {
  __shared__ int64_t sum[kAssignThreads / 64][2];
  const int lane = lane_id(), wave = wave_id();
  Two y = x;
#pragma unroll
  for (int w = 1; w < 64; w <<= 1) {
    const int64_t a = __shfl_up(y.a, w), b = __shfl_up(y.b, w);
    if (lane >= w) { y.a += a; y.b += b; }
  }
  __syncthreads();                                  // the last call's readers are done
  if (lane == 63) { sum[wave][0] = y.a; sum[wave][1] = y.b; }
  __syncthreads();
  all = Two{0, 0};
  Two before{0, 0};
#pragma unroll
  for (int w = 0; w < kAssignThreads / 64; ++w) {
    if (w == wave) before = all;
    all.a += sum[w][0];
    all.b += sum[w][1];
  }
  return Two{before.a + y.a - x.a, before.b + y.b - x.b};
}

// Last i in [0, n) with first[i] <= at (first ascends, first[0] <= at).
template <typename T>
__device__ __forceinline__ int last_at(const T* first, int n, int64_t at) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (first[lo + half] <= at) { lo += half; n -= half; } else n = half;
  }
  return lo;
}

__device__ __forceinline__ int64_t pages_of(const AssignArgs& a, int64_t tokens) {
  const int64_t n = (tokens + (1 << a.page_shift) - 1) >> a.page_shift;
  return n < a.width ? n : a.width;
}

__device__ __forceinline__ int64_t at_least_0(int x) { return x > 0 ? x : 0; }

// Position and slot of token t, `s` its request, `c0` and `c1` the request's offsets.
__device__ __forceinline__ void put_token(const AssignArgs& a, int64_t t, int s, int64_t c0, int64_t c1, int64_t kv) {
  int64_t pos = 0, slot = -1;
  if (t < c1) {
    pos = kv - c1 + t;
    if (pos < 0) pos = 0;                           // lengths that stopped at 2^31 - 1
    const int64_t i = pos >> a.page_shift;
    if (a.slots && i < a.width) {
      const int64_t page = a.table[s * a.table_row + i];
      if (page >= 0) slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
  }
  if (a.positions) a.positions[t] = (int)pos;
  if (a.slots) a.slots[t] = slot;
}

__global__ __launch_bounds__(kAssignThreads) void paged_assign_kernel(AssignArgs a) {
  __shared__ int64_t first[kAssignThreads];         // a request's first page among the chunk's
  __shared__ int64_t offset[kAssignThreads + 1];    // and its first token
  __shared__ int have[kAssignThreads];              // pages it holds already
  const int tid = threadIdx.x;
  int64_t top = a.free_count[0];
  int64_t lacking = a.free_count[1];
  top = top < 0 ? 0 : top < a.capacity ? top : a.capacity;
  Two all;
  // what ended requests give back
  if (a.done)
    for (int s0 = 0; s0 < a.S; s0 += kAssignThreads) {
      const int s = s0 + tid, n = a.S - s0 < kAssignThreads ? a.S - s0 : kAssignThreads;
      const int64_t held = s < a.S && a.done[s] != 0 ? pages_of(a, at_least_0(a.kv_lens[s])) : 0;
      first[tid] = scan_two(Two{held, 0}, all).a;
      __syncthreads();
      const int64_t entries = all.a;
      for (int64_t i0 = 0; i0 < entries; i0 += kAssignThreads) {
        const int64_t i = i0 + tid;
        int page = -1;
        if (i < entries) {
          const int r = last_at(first, n, i);
          page = a.table[(s0 + r) * a.table_row + (i - first[r])];
        }
        const int64_t at = top + scan_two(Two{page >= 0, 0}, all).a;
        if (page >= 0 && at < a.capacity) a.free_pages[at] = page;
        top = top + all.a < a.capacity ? top + all.a : a.capacity;
      }
      __syncthreads();
    }
  // what the others take
  int64_t used = 0, tokens = 0;
  for (int s0 = 0; s0 < a.S; s0 += kAssignThreads) {
    const int s = s0 + tid, n = a.S - s0 < kAssignThreads ? a.S - s0 : kAssignThreads;
    int64_t fresh = 0, need = 0;
    if (s < a.S) {
      const int64_t old = a.done && a.done[s] != 0 ? 0 : at_least_0(a.kv_lens[s]);
      fresh = at_least_0(a.new_lens[s]);
      const int64_t len = old + fresh < kMostInt ? old + fresh : kMostInt, holds = pages_of(a, old);
      need = pages_of(a, len) - holds;
      have[tid] = (int)holds;
      a.kv_out[s] = (int)len;
    }
    const Two at = scan_two(Two{need, fresh}, all);
    first[tid] = at.a;
    auto offset_of = [&](int64_t x) { return tokens + x < kMostInt ? tokens + x : kMostInt; };
    offset[tid] = offset_of(at.b);
    if (s < a.S) a.cu[s] = (int)offset[tid];
    __syncthreads();
    for (int64_t i = tid; i < all.a; i += kAssignThreads) {
      const int r = last_at(first, n, i);
      const int64_t from = top - 1 - used - i;
      a.table[(s0 + r) * a.table_row + have[r] + (i - first[r])] = from >= 0 ? a.free_pages[from] : -1;
    }
    used += all.a;
    tokens += all.b;
    __syncthreads();
  }
  const int64_t total = tokens < kMostInt ? tokens : kMostInt;
  if (tid == 0) {
    a.cu[a.S] = (int)total;
    const int64_t lack = lacking + (used > top ? used - top : 0);
    a.count_out[0] = (int)(used < top ? top - used : 0);
    a.count_out[1] = (int)(lack < kMostInt ? lack : kMostInt);
  }
  if (a.N > kAssignTokens || a.S > kAssignThreads || (!a.positions && !a.slots)) return;
  // the tokens of one chunk of requests, whose offsets are still here
  const int s = tid < a.S ? tid : 0;
  if (tid < a.S) first[tid] = a.kv_out[s];
  if (tid == 0) offset[a.S] = total;
  __syncthreads();
  for (int64_t t = tid; t < a.N; t += kAssignThreads) {
    if (a.S == 0 || t >= total) { put_token(a, t, 0, 0, 0, 0); continue; }
    const int r = last_at(offset, a.S, t);
    put_token(a, t, r, offset[r], offset[r + 1], first[r]);
  }
}

// The tokens of a large call, 1024 to a workgroup.
__global__ __launch_bounds__(256) void paged_assign_tokens_kernel(AssignArgs a) {
  const int64_t total = a.cu[a.S];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t t = (int64_t)blockIdx.x * 1024 + u * 256 + threadIdx.x;
    if (t >= a.N) return;
    if (a.S == 0 || t >= total) { put_token(a, t, 0, 0, 0, 0); continue; }
    const int s = last_at(a.cu, a.S, t);
    put_token(a, t, s, a.cu[s], a.cu[s + 1], a.kv_out[s]);
  }
}

}  // namespace carve
