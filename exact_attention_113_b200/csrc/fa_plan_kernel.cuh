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
// One launch, bounded by its latency: every block scans all lengths, 1024
// requests at a time (two prefix sums, four requests a thread), and then serves
// its own 1024 tokens and its share of the new pages, so no block waits for
// another (5 to 6 us for 8 requests, as long as the host's call; 8.2 us for 1024
// requests of 197k tokens, of which the bytes are 0.4: the scan, then the new
// pages and four tokens a thread, one search, load and store after the other).
// A token or page finds its request by a search in the tile's prefix sums.  A new
// token's page is taken from the free list directly, not from the table that
// another block may be writing.
#pragma once

#include <cuda_runtime.h>

namespace fa {

constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 1024;   // tokens of a block
constexpr int kPlanTile = 1024;     // requests scanned at a time

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
  constexpr int kWarps = kPlanThreads / 32, kEach = kPlanTile / kPlanThreads;
  __shared__ long long tok_s[kPlanTile];    // first token of each request of the tile
  __shared__ long long page_s[kPlanTile];   // first free-list entry
  __shared__ int ctx_s[kPlanTile];
  __shared__ long long warp_t[kWarps], warp_p[kWarps], short_s[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.page_size;
  const long long t0 = static_cast<long long>(blockIdx.x) * kPlanTokens;
  const long long t1 = min(t0 + kPlanTokens, static_cast<long long>(p.num_tokens));
  // pages of n tokens (n < 2^32: contexts and new tokens are ints)
  auto pages_of = [&](long long n) {
    return static_cast<int>(static_cast<unsigned>(n) / static_cast<unsigned>(P)) +
           (static_cast<unsigned>(n) % static_cast<unsigned>(P) != 0);
  };
  // the last request of the tile (of n) whose prefix sum is at most v
  auto find = [](const long long *pre, int n, long long v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (pre[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
  };
  long long tokens = 0, pages = 0;   // before the tile
  long long missing = 0;             // this thread's requests'
  const bool counts = blockIdx.x == gridDim.x - 1;   // (the block with the fewest tokens)
  for (int base = 0, tile = 0; base < p.B; base += kPlanTile, ++tile) {
    const int n = min(kPlanTile, p.B - base);
    int q[kEach], ctx[kEach], grown[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid * kEach + e;
      q[e] = i < n ? max(p.q_lens[base + i], 0) : 0;
      ctx[e] = i < n ? max(p.ctx_lens[base + i], 0) : 0;
    }
    long long it = 0, ip = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      grown[e] = max(min(pages_of(static_cast<long long>(ctx[e]) + q[e]), p.max_pages) -
                         pages_of(ctx[e]), 0);
      it += q[e];
      ip += grown[e];
    }
    const long long mine_t = it, mine_p = ip;
    // New tokens that continue a partly filled page have no slot where an earlier
    // step got none.  (Its entry is old: no block writes it; it arrives meanwhile.)
    int filled[kEach], entry[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      filled[e] = entry[e] = 0;
      const int have = pages_of(ctx[e]);
      const unsigned left = static_cast<unsigned>(have) * P - static_cast<unsigned>(ctx[e]);
      if (counts && left != 0 && have <= p.max_pages) {
        filled[e] = min(q[e], static_cast<int>(left));
        entry[e] = p.table[(base + tid * kEach + e) * p.table_stride + have - 1];
      }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, it, d), c = __shfl_up_sync(0xffffffffu, ip, d);
      if (lane >= d) {
        it += a;
        ip += c;
      }
    }
    if (base > 0) __syncthreads();   // the tile before has been read
    if (lane == 31) {
      warp_t[warp] = it;
      warp_p[warp] = ip;
    }
    __syncthreads();
    const long long pages0 = pages;
    long long at = tokens + it - mine_t, first = pages + ip - mine_p;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        at += warp_t[w];
        first += warp_p[w];
      }
      tokens += warp_t[w];
      pages += warp_p[w];
    }
    const bool writes = tile % gridDim.x == blockIdx.x;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid * kEach + e;
      tok_s[i] = at;
      page_s[i] = first;
      ctx_s[i] = ctx[e];
      if (i < n && writes) {
        p.cu_q[base + i] = plan_sat(at);
        if (base + i == p.B - 1) p.cu_q[p.B] = plan_sat(at + q[e]);
        p.kv_lens[base + i] = plan_sat(static_cast<long long>(ctx[e]) + q[e]);
      }
      if (counts) {
        // new tokens behind the last page the request could get
        const long long got = min(static_cast<long long>(grown[e]), max(p.n_free - first, 0ll));
        const long long room =
            (static_cast<long long>(min(pages_of(ctx[e]), p.max_pages)) + got) * P - ctx[e];
        missing += q[e] - min(static_cast<long long>(q[e]), max(room, 0ll));
        if (entry[e] < 0) missing += filled[e];
      }
      at += q[e];
      first += grown[e];
    }
    __syncthreads();
    for (long long k = pages0 + static_cast<long long>(blockIdx.x) * kPlanThreads + tid; k < pages;
         k += static_cast<long long>(gridDim.x) * kPlanThreads) {
      const int lo = find(page_s, n, k);
      p.table[(base + lo) * p.table_stride + pages_of(ctx_s[lo]) + k - page_s[lo]] =
          k < p.n_free ? p.free_pages[k] : -1;
    }
    for (long long t = max(t0, tok_s[0]) + tid; t < min(t1, tokens); t += kPlanThreads) {
      const int lo = find(tok_s, n, t);
      const unsigned pos = static_cast<unsigned>(ctx_s[lo] + (t - tok_s[lo]));
      const unsigned pg = pos / static_cast<unsigned>(P);
      const int old = pages_of(ctx_s[lo]);
      int page = -1;
      if (pg < static_cast<unsigned>(p.max_pages)) {
        if (static_cast<int>(pg) < old) {
          page = p.table[(base + lo) * p.table_stride + pg];
        } else {
          const long long f = page_s[lo] + pg - old;
          if (f < p.n_free) page = p.free_pages[f];
        }
      }
      p.positions[t] = plan_sat(pos);
      p.slots[t] = page < 0 ? -1
                            : static_cast<long long>(page) * P + (pos - pg * static_cast<unsigned>(P));
    }
  }
  for (long long t = max(t0, tokens) + tid; t < t1; t += kPlanThreads) {   // padding
    p.positions[t] = -1;
    p.slots[t] = -1;
  }
  if (counts) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) missing += __shfl_xor_sync(0xffffffffu, missing, d);
    if (lane == 0) short_s[warp] = missing;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) missing += short_s[w];
      p.counts[0] = plan_sat(tokens);
      p.counts[1] = plan_sat(min(pages, static_cast<long long>(p.n_free)));
      p.counts[2] = plan_sat(missing);
    }
  }
}

}  // namespace fa
