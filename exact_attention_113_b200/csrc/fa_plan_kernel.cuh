// fa_plan_kernel.cuh -- one serving step's page tables from the request
// lengths: cumulative lengths, the block table grown from a free list, and
// every new token's position and cache slot.
//
// With ctx_b tokens of request b in the cache, q_b new ones and pages of P:
//   have = ceil(ctx / P), need = ceil((ctx + q) / P), first_b = sum of
//   (need - have) over the requests before b;
//   table[b, have + i] = free[first_b + i],  i < need - have;
//   token t = cu_q[b] + i: position ctx_b + i, slot = page * P + position % P.
//
// One launch, bounded by its latency: every block scans all lengths, 256
// requests at a time (two prefix sums), and then serves its own 1024 tokens
// and its share of the new pages, so no block waits for another.  A token or
// page finds its request by a search in the tile's prefix sums.  A new token's
// page is taken from the free list directly, not from the table that another
// block may be writing.
#pragma once

#include <cuda_runtime.h>

namespace fa {

constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 1024;   // tokens of a block

struct PlanParams {
  const int *q_lens, *ctx_lens;
  int *table;
  long long table_stride;
  const int *free_pages;
  int n_free, B, max_pages, page_size, num_tokens;
  int *cu_q, *kv_lens, *positions;
  long long *slots;
  int *counts;   // tokens, pages taken, tokens without a slot
};

__device__ __forceinline__ int plan_sat(long long v) {
  return static_cast<int>(v > 0x7fffffffll ? 0x7fffffffll : v);
}

__global__ void __launch_bounds__(kPlanThreads) fa_plan_kernel(const PlanParams p) {
  __shared__ long long tok_s[kPlanThreads];       // first token of each request of the tile
  __shared__ long long page_s[kPlanThreads];      // first free-list entry
  __shared__ int ctx_s[kPlanThreads];
  __shared__ long long warp_t[kPlanThreads / 32], warp_p[kPlanThreads / 32];
  __shared__ long long short_s[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.page_size;
  const long long t0 = static_cast<long long>(blockIdx.x) * kPlanTokens;
  const long long t1 = min(t0 + kPlanTokens, static_cast<long long>(p.num_tokens));
  // the last request of the tile whose prefix sum is at most v
  auto find = [](const long long *pre, long long v) {
    int lo = 0, hi = kPlanThreads;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (pre[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
  };
  long long tokens = 0, pages = 0;   // before the tile
  long long missing = 0;             // this thread's requests'
  for (int base = 0, tile = 0; base < p.B; base += kPlanThreads, ++tile) {
    const int b = base + tid;
    int q = 0, ctx = 0;
    if (b < p.B) {
      q = max(p.q_lens[b], 0);
      ctx = max(p.ctx_lens[b], 0);
    }
    const long long kv = static_cast<long long>(ctx) + q;
    const int have = static_cast<int>((static_cast<long long>(ctx) + P - 1) / P);
    const int need = static_cast<int>(min((kv + P - 1) / P, static_cast<long long>(p.max_pages)));
    const int grown = max(need - have, 0);
    long long it = q, ip = grown;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, it, d), c = __shfl_up_sync(0xffffffffu, ip, d);
      if (lane >= d) {
        it += a;
        ip += c;
      }
    }
    __syncthreads();   // the tile before has been read
    if (lane == 31) {
      warp_t[warp] = it;
      warp_p[warp] = ip;
    }
    __syncthreads();
    const long long pages0 = pages;
    long long at = tokens + it - q, first = pages + ip - grown;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) {
        at += warp_t[w];
        first += warp_p[w];
      }
      tokens += warp_t[w];
      pages += warp_p[w];
    }
    tok_s[tid] = at;
    page_s[tid] = first;
    ctx_s[tid] = ctx;
    if (b < p.B && tile % gridDim.x == blockIdx.x) {
      p.cu_q[b] = plan_sat(at);
      if (b == p.B - 1) p.cu_q[p.B] = plan_sat(at + q);
      p.kv_lens[b] = plan_sat(kv);
    }
    if (blockIdx.x == 0) {
      // new tokens behind the last page the request could get
      const long long got = min(static_cast<long long>(grown), max(p.n_free - first, 0ll));
      const long long room = (static_cast<long long>(min(have, p.max_pages)) + got) * P - ctx;
      missing += q - min(static_cast<long long>(q), max(room, 0ll));
    }
    __syncthreads();
    for (long long k = pages0 + static_cast<long long>(blockIdx.x) * kPlanThreads + tid; k < pages;
         k += static_cast<long long>(gridDim.x) * kPlanThreads) {
      const int lo = find(page_s, k);
      const long long old = (static_cast<long long>(ctx_s[lo]) + P - 1) / P;
      p.table[(base + lo) * p.table_stride + old + k - page_s[lo]] =
          k < p.n_free ? p.free_pages[k] : -1;
    }
    for (long long t = max(t0, tok_s[0]) + tid; t < min(t1, tokens); t += kPlanThreads) {
      const int lo = find(tok_s, t);
      const long long pos = ctx_s[lo] + (t - tok_s[lo]);
      const long long pg = pos / P;
      const long long old = (static_cast<long long>(ctx_s[lo]) + P - 1) / P;
      int page = -1;
      if (pg < p.max_pages) {
        if (pg < old) {
          page = p.table[(base + lo) * p.table_stride + pg];
        } else {
          const long long f = page_s[lo] + pg - old;
          if (f < p.n_free) page = p.free_pages[f];
        }
      }
      p.positions[t] = plan_sat(pos);
      p.slots[t] = page < 0 ? -1 : static_cast<long long>(page) * P + pos % P;
    }
  }
  for (long long t = max(t0, tokens) + tid; t < t1; t += kPlanThreads) {   // padding
    p.positions[t] = -1;
    p.slots[t] = -1;
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) missing += __shfl_xor_sync(0xffffffffu, missing, d);
    if (lane == 0) short_s[warp] = missing;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kPlanThreads / 32; ++w) missing += short_s[w];
      p.counts[0] = plan_sat(tokens);
      p.counts[1] = plan_sat(min(pages, static_cast<long long>(p.n_free)));
      p.counts[2] = plan_sat(missing);
    }
  }
}

}  // namespace fa
