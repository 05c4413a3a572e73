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
// kernel over all CUs. Bound by latency (a step of 64 requests: lengths, page, entry and
// token wait for each other, 3.8 us) and by the scattered loads that one CU can make:
// 333 requests of which 57 end with 7,700 pages, 8,800 given out and 141,000 tokens 14.3
// and 4.4 us. Pages given back pass LDS, so that they are stored as they lie and taken
// again from there (18.7 us before that).
#pragma once
#include <type_traits>

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
constexpr int kAssignLds = 4096;                    // requests whose offsets the second one keeps in LDS
constexpr unsigned kMostInt = 0x7fffffff;

// Lengths and offsets stop at 2^31 - 1 (and pages in between cannot pass it: there are
// at most that many table entries).
__device__ __forceinline__ unsigned sum_to_most(unsigned a, unsigned b) { return a + b < kMostInt ? a + b : kMostInt; }

// Inclusive prefix sums over a wave: in rows of 16 lanes, then the last lane of a row to the next
// one and of the first half to the second.
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned plus_dpp(unsigned x) {
  return sum_to_most(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ unsigned scan_wave(unsigned x) {
  x = plus_dpp<0x111, 0xf>(x);
  x = plus_dpp<0x112, 0xf>(x);
  x = plus_dpp<0x114, 0xf>(x);
  x = plus_dpp<0x118, 0xf>(x);
  x = plus_dpp<0x142, 0xa>(x);
  return plus_dpp<0x143, 0xc>(x);
}

// Exclusive prefix sums over the workgroup of two numbers below 2^31; their totals in `all`.
struct Two { unsigned a, b; };
__device__ __forceinline__ Two scan_two(Two x, Two& all) {
  constexpr int W = kAssignThreads / 64;
  __shared__ unsigned sum[W][2];
  const int lane = lane_id(), wave = wave_id();
  const Two y{scan_wave(x.a), scan_wave(x.b)};
  __syncthreads();                                  // the last call's readers are done
  if (lane == 63) { sum[wave][0] = y.a; sum[wave][1] = y.b; }
  __syncthreads();
  all = Two{0, 0};
  Two before{0, 0};
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == wave) before = all;
    all.a = sum_to_most(all.a, sum[w][0]);
    all.b = sum_to_most(all.b, sum[w][1]);
  }
  const unsigned ua = __shfl_up(y.a, 1), ub = __shfl_up(y.b, 1);
  return Two{sum_to_most(before.a, lane ? ua : 0), sum_to_most(before.b, lane ? ub : 0)};
}

// Last i in [0, n) with first[i] <= at, for U numbers at a time (first ascends, first[0] <= at).
template <int U, typename T>
__device__ __forceinline__ void last_at(const T* first, int n, const unsigned (&at)[U], int (&lo)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) lo[u] = 0;
  while (n > 1) {
    const int half = n >> 1;
#pragma unroll
    for (int u = 0; u < U; ++u) lo[u] = (unsigned)first[lo[u] + half] <= at[u] ? lo[u] + half : lo[u];
    n -= half;
  }
}
template <typename T>
__device__ __forceinline__ int last_at(const T* first, int n, unsigned at) {
  int lo[1];
  last_at<1>(first, n, {at}, lo);
  return lo[0];
}

__device__ __forceinline__ unsigned pages_of(const AssignArgs& a, unsigned tokens) {
  const unsigned n = (tokens + ((1u << a.page_shift) - 1)) >> a.page_shift;
  return n < (unsigned)a.width ? n : a.width;
}

__device__ __forceinline__ unsigned at_least_0(int x) { return x > 0 ? x : 0; }

// Position of token t of a request whose tokens end before c1 at length kv.
__device__ __forceinline__ int position(int t, int c1, int kv) {
  const int pos = kv - c1 + t;
  return pos > 0 ? pos : 0;                         // lengths that stopped at 2^31 - 1
}
// Its page, -1 if there is none. No branch: the loads of several tokens go out together.
__device__ __forceinline__ int page_of(const AssignArgs& a, bool real, int s, int pos) {
  const int i = pos >> a.page_shift;
  const bool in = real && a.slots && i < a.width;
  const int page = *(in ? a.table + (s * a.table_row + i) : a.cu);
  return in ? page : -1;
}
__device__ __forceinline__ void put_token(const AssignArgs& a, int t, int pos, int page) {
  if (a.positions) a.positions[t] = pos;
  if (a.slots) a.slots[t] = page < 0 ? -1 : ((int64_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// Where few requests have many pages each, a thread takes this many of them: their loads
// overlap, and one prefix sum does for all.
constexpr int kAssignRun = 8;

__global__ __launch_bounds__(kAssignThreads) void paged_assign_kernel(AssignArgs a) {
  __shared__ unsigned first[kAssignThreads];        // a request's first page among the chunk's
  __shared__ unsigned offset[kAssignThreads + 1];   // and its first token
  __shared__ unsigned have[kAssignThreads];         // pages it holds already
  // pages given back last, those from moved_from on; a word in 32 is left out against bank conflicts
  __shared__ int moved[kAssignThreads * kAssignRun * 33 / 32];
  auto pad = [](unsigned i) { return i + i / 32; };
  const int tid = threadIdx.x;
  const unsigned capacity = (unsigned)a.capacity, lacking = a.free_count[1];
  unsigned top = at_least_0(a.free_count[0]);
  top = top < capacity ? top : capacity;
  unsigned moved_from = kMostInt;
  // the first chunk of requests, on its way while nothing waits for it
  const bool there = tid < a.S;
  const int kv0 = there ? a.kv_lens[tid] : 0, new0 = there ? a.new_lens[tid] : 0, done0 = there && a.done ? a.done[tid] : 0;
  Two all;
  // what ended requests give back
  if (a.done)
    for (int s0 = 0; s0 < a.S; s0 += kAssignThreads) {
      const int s = s0 + tid, n = a.S - s0 < kAssignThreads ? a.S - s0 : kAssignThreads;
      const int over = s0 == 0 ? done0 : s < a.S ? a.done[s] : 0;
      const unsigned held = over ? pages_of(a, at_least_0(s0 == 0 ? kv0 : a.kv_lens[s])) : 0;
      const unsigned mine = scan_two(Two{held, 0}, all).a;
      first[tid] = mine;
      __syncthreads();
      const unsigned entries = all.a;
      for (unsigned i0 = 0; i0 < entries; i0 += kAssignThreads * kAssignRun) {
        const unsigned i = i0 + tid * kAssignRun;
        int page[kAssignRun];
        unsigned good = 0;
        int r = i < entries ? last_at(first, n, i) : 0;
#pragma unroll
        for (int u = 0; u < kAssignRun; ++u) {
          page[u] = -1;
          if (i + u < entries) {
            while (r + 1 < n && first[r + 1] <= i + u) ++r;
            page[u] = a.table[(s0 + r) * a.table_row + (i + u - first[r])];
          }
        }
#pragma unroll
        for (int u = 0; u < kAssignRun; ++u) good += page[u] >= 0;
        unsigned at = scan_two(Two{good, 0}, all).a;
#pragma unroll
        for (int u = 0; u < kAssignRun; ++u)
          if (page[u] >= 0) moved[pad(at++)] = page[u];
        __syncthreads();
        const unsigned fit = all.a < capacity - top ? all.a : capacity - top;
        for (unsigned k = tid; k < fit; k += kAssignThreads) a.free_pages[top + k] = moved[pad(k)];
        moved_from = top;
        top += fit;
      }
      __syncthreads();
    }
  // what the others take
  unsigned used = 0, tokens = 0;
  for (int s0 = 0; s0 < a.S; s0 += kAssignThreads) {
    const int s = s0 + tid, n = a.S - s0 < kAssignThreads ? a.S - s0 : kAssignThreads;
    unsigned fresh = 0, need = 0;
    if (s < a.S) {
      const int over = s0 == 0 ? done0 : a.done ? a.done[s] : 0;
      const unsigned old = over ? 0 : at_least_0(s0 == 0 ? kv0 : a.kv_lens[s]);
      fresh = at_least_0(s0 == 0 ? new0 : a.new_lens[s]);
      const unsigned len = sum_to_most(old, fresh), holds = pages_of(a, old);
      need = pages_of(a, len) - holds;
      have[tid] = holds;
      a.kv_out[s] = (int)len;
    }
    const Two at = scan_two(Two{need, fresh}, all);
    first[tid] = at.a;
    offset[tid] = sum_to_most(tokens, at.b);
    if (s < a.S) a.cu[s] = (int)offset[tid];
    __syncthreads();
    auto deal = [&](auto run, unsigned i0) {        // entries i0 .. i0 + run kAssignThreads - 1
      constexpr int U = decltype(run)::value;
      unsigned i[U];
      int r[U], page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        i[u] = i0 + u * kAssignThreads + tid;
        i[u] = i[u] < all.a ? i[u] : all.a - 1;     // past the end, the last one again: the same entry and page
      }
      last_at<U>(first, n, i, r);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned from = sum_to_most(used, i[u]), at = top - 1 - from;
        page[u] = from >= top ? -1 : at >= moved_from ? moved[pad(at - moved_from)] : a.free_pages[at];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) a.table[(s0 + r[u]) * a.table_row + have[r[u]] + (i[u] - first[r[u]])] = page[u];
    };
    for (unsigned i0 = 0; i0 < all.a;) {
      if (all.a - i0 > kAssignThreads) {
        deal(std::integral_constant<int, kAssignRun>{}, i0);
        i0 += kAssignThreads * kAssignRun;
      } else {
        deal(std::integral_constant<int, 1>{}, i0);
        i0 += kAssignThreads;
      }
    }
    used = sum_to_most(used, all.a);
    tokens = sum_to_most(tokens, all.b);
    __syncthreads();
  }
  if (tid == 0) {
    a.cu[a.S] = (int)tokens;
    a.count_out[0] = (int)(used < top ? top - used : 0);
    a.count_out[1] = (int)sum_to_most(lacking, used > top ? used - top : 0);
  }
  if (a.N > kAssignTokens || a.S > kAssignThreads || (!a.positions && !a.slots)) return;
  // the tokens of one chunk of requests, whose offsets are still here
  if (tid < a.S) first[tid] = a.kv_out[tid];
  if (tid == 0) offset[a.S] = tokens;
  __syncthreads();
  for (int t = tid; t < a.N; t += kAssignThreads) {
    const bool real = (unsigned)t < tokens;
    const int r = real ? last_at(offset, a.S, t) : 0, pos = real ? position(t, offset[r + 1], first[r]) : 0;
    put_token(a, t, pos, page_of(a, real, r, pos));
  }
}

// The tokens of a large call, 1024 to a workgroup.
__global__ __launch_bounds__(256) void paged_assign_tokens_kernel(AssignArgs a) {
  __shared__ int offset[kAssignLds + 1];
  const bool here = a.S <= kAssignLds;
  if (here) {
    for (int s = threadIdx.x; s <= a.S; s += 256) offset[s] = a.cu[s];
    __syncthreads();
  }
  const int tokens = here ? offset[a.S] : a.cu[a.S];
  // four tokens of a thread at a time, their loads side by side
  constexpr int U = 4;
  unsigned t[U];
  int s[U], pos[U], page[U];
  bool real[U];
#pragma unroll
  for (int u = 0; u < U; ++u) t[u] = blockIdx.x * (256 * U) + u * 256 + threadIdx.x;
  if (here) last_at<U>(offset, a.S, t, s);
  else last_at<U>(a.cu, a.S, t, s);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    real[u] = t[u] < (unsigned)tokens;              // (then there is a request)
    const int after = real[u] ? s[u] + 1 : 0, c1 = here ? offset[after] : a.cu[after];
    const int kv = *(real[u] ? a.kv_out + s[u] : a.cu);
    pos[u] = real[u] ? position(t[u], c1, kv) : 0;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) page[u] = page_of(a, real[u], s[u], pos[u]);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (t[u] < (unsigned)a.N) put_token(a, t[u], pos[u], page[u]);
}

}  // namespace carve
