// fa_paged_kernel.cuh -- attention of each request's new tokens over its
// paged key/value cache (sm_100a).
//
// Request b has q_len new tokens (packed rows cu_q[b] .. cu_q[b+1]) and
// kv_len tokens in the cache, the new ones last; its token p lies in row
// p % P of page table[b, p / P].  For new token i, at position
// x = kv_len - q_len + i, and query head h (K/V head h / G):
//   O = sum_j softmax_j(scale * q . k_j | j visible) v_j,  lse = ln sum_j e^..,
//   j visible iff j < kv_len, j >= x - window_left, j <= x + window_right.
//
// Query rows: the G heads that share a K/V head read the same keys, so a
// 128-row tile holds TQ = floor(128 / G) tokens of all G heads (row r is
// token r / G, head r % G): a key block is read once for the whole group.
// Work: a (request, K/V head, pair of tiles) reads `blocks` key blocks of
// 128 and costs that many and the item's own.  The costs form one line, cut in
// equal pieces, one per CTA (one CTA per SM), so that one long request, many
// short ones and causal triangles all fill the device.  A CTA walks its
// piece, whole items and, at the ends, parts of two items; parts leave an
// unnormalised fp32 O and (m, l) in the workspace, and the CTA that finishes an
// item's last part joins them (nothing waits).  Each CTA finds its piece from
// the lengths by itself (a scan over the requests during set-up), so a call
// needs no schedule from the host, which does not know the lengths.
//
// A pair of two tiles runs as the forward kernel's ping-pong: per key block
// S0, PV1(previous), S1, PV0, two softmax warpgroups in turns.  A single tile
// (decoding, short chunks) gives even key blocks to one warpgroup and odd ones
// to the other, each with its own (m, l, O), joined at the end; that keeps two
// blocks in flight where one tile's S -> softmax -> PV chain would be exposed.
//
// Warps (384 threads): 0-3, 4-7 softmax; 8 MMA and TMEM; 9 K; 10 V; 11 walks
// the piece, announces each item to the others and loads its Q (a lone warp
// takes over a microsecond for a step of the walk, so it runs ahead).
// TMEM: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D); P_t over
// the first 64 columns of S_t, or, for D <= 64, in [384+64t, 448+64t), so that
// the next S_t is computed while the softmax works on this one.
//
// Measured, back to back (of the copy rate, of the bf16 burst): decoding 64
// requests over 4k to 12k tokens, H32/8 D128, 319 us (2.0 GB, 0.97; 352 us on the
// slowest card); two chunks of up to 4096 tokens over up to 12k, H32/8 D128,
// 1350 us (0.61; the board's power limit, with pauses between the calls 1205 us
// and 0.68); 14 decoding requests beside 6 chunks of 250 to 475 tokens, window
// 4096, H16 D64, 133 us (0.37; the exponentials of the chunks and the latency of
// an item's ends); one request over 800 tokens, H32/8 D128, 16.6 us (launch,
// set-up 3, one block's chain 4, joining 5); 64 requests over 1000 tokens with 1,
// 2 and 4 new ones (4, 8 and 16 rows a tile), H32/8 D128, 57, 60 and 68 us (bytes
// 40): from 9 rows on a lane does all 128 exponentials of its row.
//
// The weights P enter the product with V in 16 bits, as the tensor cores take
// them beside a 16-bit V and as in the dense forward; the normaliser sums them
// unrounded.  Each is off by at most half a step (2^-8 of a bf16 weight, 2^-11 of
// an fp16 one), which moves O by no more than that share of sum_j p_j |v_j| / l;
// a second product for what the rounding took off would cost a prefill half as
// much again.  Up to 8 rows (decoding) have that second product for nothing, see
// kFewRows (64 requests over 8k: 317 us without, 319 with it).
//
// V rows no query of the item sees (behind the request's end, in a page's
// unwritten tail, or before every window) are cleared in shared memory: their
// weight is an exact 0, but 0 times an unwritten NaN would not be.
#pragma once

#include "fa_fwd_kernel.cuh"

namespace fa {

constexpr int kSchedWarp = 11;       // walks the work, loads Q
constexpr int kPagedMinUnits = 3;    // cost a CTA gets at least (4: single tokens 2 us slower)
constexpr int kPagedRows = 2 * kBM;  // rows of a work item
constexpr int kItemRing = 3;         // items announced ahead
constexpr uint32_t kCountedBar = 1;  // named barrier: warp 0 has left its role
// A single tile of at most this many rows (decoding) takes TMEM in the layout of a
// matrix fragment: four lanes share a row, 32 of a block's 128 exponentials each.
// One warp's 128 of a lane had set the pace (128 requests over 500 tokens, H32/8
// D128: 76 us so, 57 shared; 8 over 1000: 24.5 and 22).
// The fragment's other 8 rows, idle then, hold what the rounding of the weights
// to 16 bits took off, so the same products sum it, and the epilogue adds row
// g + 8 to row g: weights of 16 bits (bf16) or 22 (fp16) of precision.
constexpr int kFewRows = 8;

#ifdef FA_TEST_HOOKS
constexpr int kWithholdV = 1 << 16;   // g_fa_test_withhold_block: this + n is V's n-th fill
#endif

struct PagedParams {
  CUtensorMap tm_q;   // (D, H, total_q), box (cols, G, TQ)
  CUtensorMap tm_q1;  // the same, box (cols, G, 1)
  CUtensorMap tm_k;   // (D, P, H_kv, pages), box (cols, box_rows, 1, 1)
  CUtensorMap tm_v;
  const int *table;
  long long table_stride;
  const int *cu_q;
  const int *kv_lens;
  void *out;
  long long out_st, out_sh;   // element strides of a token and a head
  int out_wide;               // every row 32-byte aligned
  float *lse;                 // [total_q, H] or nullptr
  int B, H, H_kv, group, total_q;
  int tile_q;                 // tokens per tile
  int n_pages, page_shift, max_kv;  // page size 2^page_shift; max_kv: table columns * page size
  int box_rows;               // rows of one K/V copy: min(page size, 128)
  int wl, wr;                 // -1 = unbounded
  float scale_log2;
  float *ws_o;                // [2 * grid][D / 4][kPagedRows][4]
  float2 *ws_ml;              // [2 * grid][kPagedRows]
  unsigned long long *ticket; // [grid]
  unsigned long long call;    // this call's number, 48 bits, not 0
};

// ------------------------------------------------------------------ the work line
struct PagedReq {
  int q_start, q_len, kv_len;
  int first;   // position of the first new token
};

// Lengths of request b, cut to the tensors: no access lies outside them, and
// the tokens that have a row keep their positions.  cu_q and kv_lens may hold
// anything: with a row (q_start < e) `first` is above -2^31 before its bound and
// the last position below 2^30, so these and their sums with a window are ints;
// without one it is not used.
__device__ __forceinline__ PagedReq paged_req(const PagedParams &p, int b) {
  PagedReq r;
  const int a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1);
  r.q_start = min(max(a, 0), p.total_q);
  r.q_len = max(min(e, p.total_q) - r.q_start, 0);
  const int kv = min(max(__ldg(p.kv_lens + b), 0), 1 << 30);
  r.kv_len = min(kv, p.max_kv);
  r.first = r.q_len > 0 ? max(kv - (e - r.q_start), -(1 << 30)) : 0;
  return r;
}

__device__ __forceinline__ int paged_pairs(const PagedParams &p, int q_len) {
  return (q_len + 2 * p.tile_q - 1) / (2 * p.tile_q);
}

// Keys [klo, khi] that tokens [i0, i0 + n) of the request see; khi < klo: none.
__device__ __forceinline__ void paged_keys(const PagedParams &p, const PagedReq &r, int i0, int n,
                                           int &klo, int &khi) {
  const int first = r.first + i0, last = first + n - 1;
  klo = p.wl < 0 ? 0 : max(0, first - p.wl);
  khi = p.wr < 0 ? r.kv_len - 1 : min(r.kv_len - 1, last + p.wr);
  if (n <= 0 || khi < klo) {
    klo = 0;
    khi = -1;
  }
}

// Key blocks of pair `pair`.
__device__ __forceinline__ int paged_blocks(const PagedParams &p, const PagedReq &r, int pair) {
  const int i0 = pair * 2 * p.tile_q;
  int klo, khi;
  paged_keys(p, r, i0, min(2 * p.tile_q, r.q_len - i0), klo, khi);
  return khi < klo ? 0 : khi / kBN - klo / kBN + 1;
}

// Cost of an item on the work line.  Measured: a block of a pair takes 1.8 us at
// D 64 and 2.4 at D 128, one of a single tile 0.7 to 0.85 and 1.4; an item's
// beginning and end (first softmax, last PV, epilogue) 2 to 4 us, of few rows 1
// to 2.4.  (Against one block for an item: 8 chunks of up to 512 67 -> 62 us, 4
// decoding over 4k 24 -> 21.)  before(off): the item's blocks that lie before a
// cut at off.
struct PagedCost {
  int blocks, per, cost;   // cost = per * blocks + item()
  __device__ __forceinline__ int item() const { return cost - per * blocks; }
  __device__ __forceinline__ int before(int off) const {
    return off >= cost ? blocks : max(off - item(), 0) >> (per - 1);
  }
  // the largest off before which no block lies
  __device__ __forceinline__ int snap() const { return item() + per - 1; }
};
__device__ __forceinline__ PagedCost paged_cost(const PagedParams &p, const PagedReq &r, int pair) {
  PagedCost c;
  c.blocks = paged_blocks(p, r, pair);
  const int n = r.q_len - pair * 2 * p.tile_q;
  c.per = n > p.tile_q ? 2 : 1;
  c.cost = c.per * c.blocks + (n * p.group <= kFewRows ? 2 : 4);
  return c;
}

// Cost of one K/V head of a request; the whole warp calls it, each lane with
// its own request (q_len 0: none).  Long requests are summed by all lanes.
__device__ __forceinline__ long long paged_head_cost(const PagedParams &p, const PagedReq &r) {
  constexpr int kAlone = 4;
  const int lane = threadIdx.x & 31;
  const int np = paged_pairs(p, r.q_len);
  long long sum = 0;
  if (np <= kAlone)
    for (int i = 0; i < np; ++i) sum += paged_cost(p, r, i).cost;
  unsigned todo = __ballot_sync(0xffffffffu, np > kAlone);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    PagedReq o;
    o.q_start = 0;
    o.q_len = __shfl_sync(0xffffffffu, r.q_len, src);
    o.kv_len = __shfl_sync(0xffffffffu, r.kv_len, src);
    o.first = __shfl_sync(0xffffffffu, r.first, src);
    const int n = paged_pairs(p, o.q_len);
    long long all = 0;
    for (int i = lane; i < n; i += 32) all += paged_cost(p, o, i).cost;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    if (lane == src) sum = all;
  }
  return sum;
}

// Set-up state in shared memory.
struct PagedSetup {
  long long warp_sum[kThreads / 32];
  long long warp_rest[kThreads / 32];
  long long rest[2];      // units of the piece's ends within their request
  long long per_head[2];  // cost of one K/V head of that request
  int b[2];               // that request (B: the end of the line)
  long long end;          // the piece's end, moved to a border where it has to
};

// a / b of non-negative numbers: in 32 bits where they fit (a quarter of the
// instructions).
__device__ __forceinline__ long long paged_div(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// The work line cut in n pieces: piece c begins at cut(c).
struct PagedCuts {
  long long total, q;
  int n, r;
  __device__ __forceinline__ void set(long long total_, int ctas) {
    total = total_;
    n = static_cast<int>(max(1ll, min(static_cast<long long>(ctas), total / kPagedMinUnits)));
    q = paged_div(total, n);
    r = static_cast<int>(total - q * n);
  }
  __device__ __forceinline__ long long at(int c) const {
    return c >= n ? total : q * c + static_cast<unsigned>(r * c) / static_cast<unsigned>(n);
  }
  // the last piece that begins at or before u
  __device__ __forceinline__ int last(long long u) const {
    int c = static_cast<int>(min(static_cast<long long>(n - 1), paged_div(u * n, total)));
    while (c > 0 && at(c) > u) --c;
    while (c + 1 < n && at(c + 1) <= u) ++c;
    return c;
  }
};

// All threads: the line's length and the requests that the ends of this CTA's
// piece lie in.  The caller's barrier makes them visible.
__device__ __forceinline__ void paged_find_piece(const PagedParams &p, PagedSetup &st,
                                                 PagedCuts &cuts) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kThreads / 32;
  auto cost_of = [&](int b) {
    PagedReq r;
    r.q_start = r.q_len = r.kv_len = r.first = 0;
    if (b < p.B) r = paged_req(p, b);
    return paged_head_cost(p, r);
  };
  auto scan = [&](long long v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += o;
    }
    return v;
  };
  if (tid < 2) st.b[tid] = p.B;
  long long head = cost_of(tid), s = head * p.H_kv, incl = scan(s), rest = 0;
  for (int base = kThreads; base < p.B; base += kThreads) rest += cost_of(base + tid) * p.H_kv;
  if (p.B > kThreads) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, d);
  }
  if (lane == 31) {
    st.warp_sum[warp] = incl;
    st.warp_rest[warp] = rest;
  }
  __syncthreads();
  long long total = 0, pre = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) pre += st.warp_sum[w];
    total += st.warp_sum[w];
  }
  long long before = total;   // of the requests so far
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += st.warp_rest[w];
  cuts.set(total, gridDim.x);
  const int c = blockIdx.x;
  const long long want[2] = {cuts.at(c), cuts.at(c + 1)};
  auto look = [&](int b, long long lo) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (s > 0 && want[e] >= lo && want[e] < lo + s) {
        st.b[e] = b;
        st.rest[e] = want[e] - lo;
        st.per_head[e] = head;
      }
  };
  look(tid, pre + incl - s);
  for (int base = kThreads; base < p.B; base += kThreads) {
    head = cost_of(base + tid);
    s = head * p.H_kv;
    incl = scan(s);
    __syncthreads();
    if (lane == 31) st.warp_sum[warp] = incl;
    __syncthreads();
    pre = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += st.warp_sum[w];
      before += st.warp_sum[w];
    }
    look(base + tid, pre + incl - s);
  }
}

// One part of an item, as the roles see it.
struct PagedItem {
  int h, tok0, nt0, nt1;     // K/V head (-1: no more items); first tile's first packed row; tokens
  int first, kv_len, lo, hi; // position of the first token; key blocks of the part
  int lo0, hi0, lo1, hi1;    // ... of each tile
  int klo, khi, slot, b;     // keys some token of the item sees; -1: the whole item, else the part's slot
  int once, pad[3];          // no other item reads these keys
};
// A cut item of this CTA (slot 0, slot 1): the CTA where it began, its parts.
struct PagedCut {
  int cta0, parts;
};

// Walks a CTA's piece (one warp).
struct PagedWalk {
  int b, h, pair, off;
  long long u, end;          // on the work line: here, and the piece's end
  PagedReq r;
  long long began;           // of the item given last: its start, its cost
  PagedCost cost;

  // The place of end e of the piece; `at` moved back to the item's start where
  // no block of it lies before the cut.  All lanes.
  __device__ __forceinline__ void locate(const PagedParams &p, const PagedSetup &st, int e,
                                         long long &at) {
    const int lane = threadIdx.x & 31;
    b = st.b[e];
    h = pair = off = 0;
    if (b >= p.B) return;
    r = paged_req(p, b);
    const int np = paged_pairs(p, r.q_len);
    h = static_cast<int>(paged_div(st.rest[e], st.per_head[e]));
    long long in = st.rest[e] - h * st.per_head[e];
    if (np > 1) {
      for (int base = 0; base < np; base += 32) {
        const int i = base + lane;
        const long long cst = i < np ? paged_cost(p, r, i).cost : 0;
        long long incl = cst;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, incl > in);
        if (hit) {
          const int src = __ffs(hit) - 1;
          pair = base + src;
          in -= __shfl_sync(0xffffffffu, incl - cst, src);
          break;
        }
        in -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    off = static_cast<int>(in);
    if (paged_cost(p, r, pair).before(off) == 0) {
      at -= off;
      off = 0;
    }
  }
  __device__ __forceinline__ void start(const PagedParams &p, const PagedSetup &st,
                                        const PagedCuts &cuts) {
    end = st.end;
    u = cuts.at(blockIdx.x);
    locate(p, st, 0, u);
  }
  // To the next item, if the piece has one.  Requests without new tokens (most of
  // a batch captured for more) are passed over 128 at a time, all lanes looking:
  // 2^24 of them in some 100 ms, well within the limit of the others' waits.
  __device__ __forceinline__ void advance(const PagedParams &p) {
    off = 0;
    if (u >= end) return;
    if (++pair < paged_pairs(p, r.q_len)) return;
    pair = 0;
    if (++h < p.H_kv) return;
    h = 0;
    if (++b >= p.B) return;
    r = paged_req(p, b);
    if (__builtin_expect(r.q_len > 0, 1)) return;
    constexpr int kLook = 4;
    const int lane = threadIdx.x & 31;
    for (++b; b < p.B; b += 32 * kLook) {
      bool some[kLook];
#pragma unroll
      for (int v = 0; v < kLook; ++v) {
        const int i = b + 32 * v + lane;
        some[v] = i < p.B && paged_req(p, i).q_len > 0;
      }
#pragma unroll
      for (int v = 0; v < kLook; ++v) {
        const unsigned hit = __ballot_sync(0xffffffffu, some[v]);
        if (hit) {
          b += 32 * v + __ffs(hit) - 1;
          r = paged_req(p, b);
          return;
        }
      }
    }
    b = p.B;
  }
  __device__ __forceinline__ bool next(const PagedParams &p, PagedItem &t) {
    if (u >= end || b >= p.B) {
      t.h = -1;
      return false;
    }
    t.b = b;
    t.h = h;
    const int i0 = pair * 2 * p.tile_q;
    t.tok0 = r.q_start + i0;
    t.nt0 = min(p.tile_q, r.q_len - i0);
    t.nt1 = min(p.tile_q, r.q_len - i0 - t.nt0);
    t.first = r.first + i0;
    t.kv_len = r.kv_len;
    t.once = r.q_len <= 2 * p.tile_q;
    int klo0, khi0, klo1 = 0, khi1 = -1;
    paged_keys(p, r, i0, t.nt0, klo0, khi0);
    t.klo = klo0;
    t.khi = khi0;
    if (t.nt1 > 0) {
      paged_keys(p, r, i0 + p.tile_q, t.nt1, klo1, khi1);
      paged_keys(p, r, i0, t.nt0 + t.nt1, t.klo, t.khi);
    }
    const PagedCost c = paged_cost(p, r, pair);
    const int lo = t.klo / kBN;
    const int to = static_cast<int>(min(static_cast<long long>(c.cost), off + (end - u)));
    t.lo = lo + c.before(off);
    t.hi = lo + c.before(to);
    t.slot = off > 0 ? 0 : (to < c.cost ? 1 : -1);
    t.lo0 = max(t.lo, klo0 / kBN);
    t.hi0 = khi0 < klo0 ? t.lo0 : max(t.lo0, min(t.hi, khi0 / kBN + 1));
    t.lo1 = max(t.lo, klo1 / kBN);
    t.hi1 = khi1 < klo1 ? t.lo1 : max(t.lo1, min(t.hi, khi1 / kBN + 1));
    began = u - off;
    cost = c;
    u += to - off;
    if (to >= c.cost)
      advance(p);
    else
      off = to;
    return true;
  }
  // Of the item that next() gave last, by the cuts before they move to borders
  // (a 64-bit division or two: its readers need it only when they are done).
  __device__ __forceinline__ PagedCut cut_of(const PagedCuts &cuts) const {
    PagedCut k;
    k.cta0 = cuts.last(began + cost.snap());
    k.parts = cuts.last(began + cost.cost - 1) - k.cta0 + 1;
    return k;
  }
};

// ------------------------------------------------------------------ shared memory
template <int kSlots>
struct PagedBars {
  uint64_t item_full[kItemRing];
  uint64_t item_empty[kItemRing];
  uint64_t q_full[2];    // Q slot filled
  uint64_t q_empty[2];   // every S that reads it is done
  uint64_t full[kSlots];
  uint64_t empty[kSlots];
  uint64_t v_ragged;     // the copy of a V block whose hidden rows are cleared
  uint64_t s_full[2];
  uint64_t s_free[2];    // the softmax holds S_t in registers (D <= 64)
  uint64_t p_full[2];
  uint64_t pv_done[2];
  uint64_t o_free[2];    // O_t has been read by the epilogue
  uint64_t ml_full[2];   // single tile: warpgroup's (m, l) written
  uint64_t ml_free[2];   // ... and read
  uint64_t cut_full[2];  // cut[slot] written
  uint64_t part_done;    // a part's rows are in the workspace
  uint64_t part_last;    // whether they were the item's last is known
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int is_last;
  int ticketed[2];       // the CTA's parts whose arrival has been counted
  PagedCut cut[2];
  PagedItem item[kItemRing];
  PagedSetup setup;
};

template <int D>
struct PagedGeo : Geo<D, 2> {
  using G = Geo<D, 2>;
  static constexpr int kBarBytesPaged = 1024;
  static constexpr int kOffXch = G::kOffBar + kBarBytesPaged;   // (m, l) of 128 rows, twice
  static constexpr int kUsedPaged = kOffXch + 2 * kBM * 8;
  // (one CTA per SM, as the forward: at least 118 KB.  The base is 1024-byte
  // aligned by its declaration, as there is no other shared memory.)
  static constexpr int kSmemPaged = kUsedPaged > 118 * 1024 ? kUsedPaged : 118 * 1024;
  static_assert(kSmemPaged <= 232448, "shared memory budget");
  static_assert(sizeof(PagedBars<G::kSlots>) <= kBarBytesPaged, "barrier block");
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int c0, int c1, int c2, int c3, uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(cache_hint)
      : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// 16 lanes of TMEM in the layout of a matrix fragment.  Load, 64 columns: r[4j],
// r[4j + 1] are columns 8j + 2c, 8j + 2c + 1 of TMEM lane g, r[4j + 2], r[4j + 3]
// of lane g + 8, with g = lane / 4, c = lane % 4.  Store, 64 columns: r[2j] is
// column 4j + c of lane g, r[2j + 1] of lane g + 8.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// 16 columns.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_rows16(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// What the rounding of two values to 16 bits took off, itself so rounded.
template <int DT>
__device__ __forceinline__ uint32_t pack2_rest(const float2 &x, uint32_t rounded) {
  float2 r;
  if constexpr (DT == 0)
    r = __half22float2(*reinterpret_cast<const __half2 *>(&rounded));
  else
    r = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&rounded));
  r = __ffma2_rn(r, make_float2(-1.0f, -1.0f), x);
  return pack2<DT>(r.x, r.y);
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// Counts a part's arrival; true for the item's last.  The word holds the
// call's number and the parts so far; with another number in it (a new
// workspace, whatever it held) the count is 0, and the last arrival leaves 0.
__device__ __forceinline__ bool paged_ticket(const PagedParams &p, PagedCut cut) {
  unsigned long long *at = p.ticket + cut.cta0;
  // tried first: that this is the last part, which the joining waits for
  unsigned long long old = (p.call << 16) | static_cast<unsigned>(cut.parts - 1);
  while (true) {
    const unsigned long long n = ((old >> 16) == p.call ? (old & 0xffffull) : 0ull) + 1;
    const bool last = n == static_cast<unsigned long long>(cut.parts);
    const unsigned long long now = atomicCAS(at, old, last ? 0ull : (p.call << 16) | n);
    if (now == old) return last;
    old = now;
  }
}

// A slot of the workspace: [D / 4][kPagedRows] float4, so that the threads of a
// warp, which hold a row each, write and read neighbours.
__device__ __forceinline__ float4 *paged_slot(const PagedParams &p, int D, int slot) {
  return reinterpret_cast<float4 *>(p.ws_o) + static_cast<size_t>(slot) * kPagedRows * (D / 4);
}

// 16 results of one row, `c` its first column; 32-byte stores where every row
// of the output is aligned for them.
template <int DT>
__device__ __forceinline__ void paged_store16(const PagedParams &p, uint8_t *orow, int c,
                                              const float (&o)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) w[v] = pack2<DT>(o[2 * v], o[2 * v + 1]);
  if (p.out_wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(orow + 2 * c),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                 "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(orow + 2 * c) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(orow + 2 * c + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The results of up to kFewRows rows: a lane takes row g = lane / 4 of TMEM and
// row g + 8, the same columns of what the weights' rounding took off, so that
// their sum needs no exchange (64 requests over 1000, H32/8 D128: 59 us with rows
// in lanes and shuffles, so 57, as without rests to add).  As in the general
// epilogue a warpgroup joins every other 16 columns of the two O; sa, sb: their
// factors, of row `lane`.
template <int D, int DT>
__device__ __forceinline__ void paged_few_rows(const PagedParams &p, const PagedItem &t,
                                               uint32_t from, int u, int tok_of_g, bool none,
                                               bool two, float sa, float sb, int slot) {
  constexpr int kChunks = (D + 31) / 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const float ga = __shfl_sync(0xffffffffu, sa, g), gb = __shfl_sync(0xffffffffu, sb, g);
  float2 o[kChunks][2];   // columns c + 2q, c + 2q + 1 and c + 8 + 2q, c + 9 + 2q
#pragma unroll
  for (int i = 0; i < kChunks; ++i) o[i][0] = o[i][1] = make_float2(0.0f, 0.0f);
  auto held = [&](int i) { return 32 * i + 16 < D || u == 0; };
  // (beside an infinite value the rests, which may be 0 or of the other sign, are none)
  auto with_rest = [](float x, float rest) { return fabsf(x) < INFINITY ? x + rest : x; };
  auto add = [&](uint32_t at, float w) {
    uint32_t x[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (held(i)) tmem_ld_rows16(at + 32 * i, x[i]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      reg_dep(x[i]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t *v = x[i] + 4 * e;
        o[i][e].x += w * with_rest(__uint_as_float(v[0]), __uint_as_float(v[2]));
        o[i][e].y += w * with_rest(__uint_as_float(v[1]), __uint_as_float(v[3]));
      }
    }
  };
  if (!none) add(from + 16 * u, ga);
  if (two) add(from + D + 16 * u, gb);
  if (tok_of_g >= t.nt0) return;
  if (t.slot >= 0) {
    float2 *at = reinterpret_cast<float2 *>(paged_slot(p, D, slot) + g) + (q & 1);
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (held(i))
#pragma unroll
        for (int e = 0; e < 2; ++e)
          at[2 * (4 * (2 * i + u) + 2 * e + (q >> 1)) * kPagedRows] = o[i][e];
  } else {
    const int head = t.h * p.group + g - tok_of_g * p.group;
    uint8_t *at = static_cast<uint8_t *>(p.out) +
                  2 * (static_cast<long long>(t.tok0 + tok_of_g) * p.out_st +
                       static_cast<long long>(head) * p.out_sh + 16 * u + 2 * q);
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (held(i))
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint32_t *>(at + 64 * i + 16 * e) = pack2<DT>(o[i][e].x, o[i][e].y);
  }
}

// Joins the parts of a cut item: m = max_i m_i, w_i = 2^(m_i - m),
// O = sum_i w_i O_i / sum_i w_i l_i, lse = (m + log2 l) ln 2, in a fixed order
// of the parts, so that the result does not depend on which came last.  Part
// i lies in slot 1 of CTA cta0 (i = 0) or slot 0 of CTA cta0 + i.  A warp takes
// 32 rows and 16 columns at a time; fewer rows leave lanes that share a row's
// parts among them (a decoding item cut over many CTAs).
template <int D, int DT>
__device__ __forceinline__ void paged_merge(const PagedParams &p, const PagedItem &t, PagedCut cut,
                                            int warp, int warps) {
  const int lane = threadIdx.x & 31;
  const int rows0 = t.nt0 * p.group, rows1 = max(t.nt1, 0) * p.group;
  const int n0 = (rows0 + 31) / 32, nb = n0 + (rows1 + 31) / 32;   // blocks of 32 rows
  int R = 32;                                     // rows of a block, lanes / R share a row
  if (nb == 1)
    while (R / 2 >= rows0) R /= 2;
  const int share = 32 / R, mine = lane / R;
  auto slot_of = [&](int i) { return 2 * (cut.cta0 + i) + (i == 0 ? 1 : 0); };
  for (int unit = warp; unit < nb * (D / 16); unit += warps) {
    const int rb = unit % nb, c = unit / nb * 16;
    const int tile = rb >= n0 ? 1 : 0;
    const int rr = (rb - tile * n0) * 32 + lane % R;   // row within the tile
    const bool valid = rr < (tile ? rows1 : rows0);    // (other rows were not written)
    const size_t row = static_cast<size_t>(tile * kBM + rr);
    // one pass, (m, l, O) raised as it goes, so that all loads are under way at once
    float m = -INFINITY, acc[16], l = 0.0f;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    // both sides of a join relative to m_new (no visible key: weight 0)
    auto weight = [](float m_old, float m_new) { return ex2(m_old - (m_new == -INFINITY ? 0.0f : m_new)); };
    if (valid) {
#pragma unroll 2
      for (int i = mine; i < cut.parts; i += share) {
        const float2 ml = __ldcg(&p.ws_ml[static_cast<size_t>(slot_of(i)) * kPagedRows + row]);
        const float4 *o = paged_slot(p, D, slot_of(i)) + static_cast<size_t>(c / 4) * kPagedRows + row;
        float4 x[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = __ldcg(o + v * kPagedRows);
        const float m_new = fmaxf(m, ml.x), a = weight(m, m_new), w = weight(ml.x, m_new);
        m = m_new;
        l = l * a + w * ml.y;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          acc[4 * v] = acc[4 * v] * a + w * x[v].x;
          acc[4 * v + 1] = acc[4 * v + 1] * a + w * x[v].y;
          acc[4 * v + 2] = acc[4 * v + 2] * a + w * x[v].z;
          acc[4 * v + 3] = acc[4 * v + 3] * a + w * x[v].w;
        }
      }
    }
    __syncwarp();
    if (R < 32) {
      float top = m;
      for (int d = R; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float w = weight(m, top);
      m = top;
      l *= w;
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[v] *= w;
      for (int d = R; d < 32; d <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[v] += __shfl_xor_sync(0xffffffffu, acc[v], d);
      }
    }
    if (valid && mine == 0) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int tok = t.tok0 + tile * p.tile_q + rr / p.group, head = t.h * p.group + rr % p.group;
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[v] *= inv;
      paged_store16<DT>(p,
                        static_cast<uint8_t *>(p.out) +
                            2 * (static_cast<long long>(tok) * p.out_st +
                                 static_cast<long long>(head) * p.out_sh),
                        c, acc);
      if (c == 0 && p.lse != nullptr)
        p.lse[static_cast<size_t>(tok) * p.H + head] =
            l > 0.0f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------ the kernel
template <int D, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_kernel(const __grid_constant__ PagedParams p) {
  using G = Geo<D, 2>;
  using PG = PagedGeo<D>;
  constexpr int kSlots = G::kSlots;
  constexpr int kKStep = 16;
  constexpr bool kSplitP = G::kSplitP;   // P in columns of its own (D <= 64)
  extern __shared__ __align__(1024) uint8_t smem[];
  PagedBars<kSlots> *bars = reinterpret_cast<PagedBars<kSlots> *>(smem + G::kOffBar);
  volatile int *abort_flag = &bars->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sQ = smem_u32(smem + G::kOffQ);
  const uint32_t sRing = smem_u32(smem + G::kOffRing);

  // ---- setup
  if (sQ & 1023u) {   // (never: see PagedGeo)
    if (tid == 0) atomicOr(&g_fa_status, 1u);
    return;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (tid == kLoadWarp * 32) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bars->q_full[t]), 1);
      mbar_init(smem_u32(&bars->q_empty[t]), 1);
      mbar_init(smem_u32(&bars->s_full[t]), 1);
      mbar_init(smem_u32(&bars->s_free[t]), 4);
      mbar_init(smem_u32(&bars->p_full[t]), 4);
      mbar_init(smem_u32(&bars->pv_done[t]), 1);
      mbar_init(smem_u32(&bars->o_free[t]), 8);
      mbar_init(smem_u32(&bars->ml_full[t]), 4);
      mbar_init(smem_u32(&bars->ml_free[t]), 4);
    }
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(smem_u32(&bars->item_full[s]), 1);
      mbar_init(smem_u32(&bars->item_empty[s]), 11);   // MMA, K, V, eight softmax warps
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->v_ragged), 1);
    for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&bars->cut_full[s]), 1);
    mbar_init(smem_u32(&bars->part_done), 8);
    mbar_init(smem_u32(&bars->part_last), 1);
    mbar_init(smem_u32(&bars->mma_done), 1);
    bars->abort_flag = 0;
    bars->ticketed[0] = bars->ticketed[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm_q);
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  // Rows that no copy writes are zero: behind tiles of fewer than 128 rows (a
  // group that does not divide 128), and behind a single token's, whose other
  // 124 or so rows of products then switch next to nothing: with other
  // requests' rows in them a decoding batch ran into the board's power limit
  // (64 requests over 8k, for seconds: 370 us at 1.37 GHz, with zeros 327).
  const int q_rows = p.tile_q * p.group;
  for (int i = tid; i < 2 * G::kTileBytes / 16; i += kThreads)
    reinterpret_cast<uint4 *>(smem + G::kOffQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  PagedCuts cuts;
  paged_find_piece(p, bars->setup, cuts);
  __syncthreads();
  PagedWalk walk;                     // (of the scheduling warp)
  if (warp == kLoadWarpV) {           // its end, while that warp finds the start
    long long end = cuts.at(blockIdx.x + 1);
    walk.locate(p, bars->setup, 1, end);
    if (lane == 0) bars->setup.end = end;
  } else if (warp == kSchedWarp) {
    walk.u = cuts.at(blockIdx.x);
    walk.locate(p, bars->setup, 0, walk.u);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;

  // Takes item k from the ring; the warp's fields are in registers when it
  // returns.  False: no more, or given up.
  bool ok = true;
  auto take = [&](int k, PagedItem &t) -> bool {
    const int s = k % kItemRing;
    ok = mbar_wait_warp(smem_u32(&bars->item_full[s]), (k / kItemRing) & 1, abort_flag);
    if (!ok) return false;
    t = bars->item[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[s]));
    return t.h >= 0;
  };

  if (warp >= 8) {
  regs_dec<RegSplit::kSmall>();
  if (warp == kSchedWarp) {
    // =================================================== schedule and Q
    // Items are announced up to kItemRing ahead of their last reader, from the
    // second on one ahead of their Q: a tile with key blocks takes the next of two Q slots.
    walk.end = bars->setup.end;
    PagedItem t, ahead;
    int nq = 0, k = 0;
    const uint64_t pol = policy_evict_first();
    auto announce = [&](PagedItem &it) -> bool {
      const bool more = walk.next(p, it);
      const int s = k % kItemRing;
      if (k >= kItemRing)
        ok = mbar_wait_warp(smem_u32(&bars->item_empty[s]), (k / kItemRing - 1) & 1, abort_flag);
      if (!ok) return false;
      if (lane == 0) {
        bars->item[s] = it;
        mbar_arrive(smem_u32(&bars->item_full[s]));
      }
      __syncwarp();
      ++k;
      return more;
    };
    int dirty = 0;   // slots whose rows behind the first token may not be zero
    auto load = [&](int h, int tok, int n) {
      const int s = nq & 1;
      if (nq >= 2) ok = mbar_wait_warp(smem_u32(&bars->q_empty[s]), ((nq >> 1) - 1) & 1, abort_flag);
      if (!ok) return;
      const bool one = n == 1;
      if (!one) {
        dirty |= 1 << s;
      } else if (dirty & (1 << s)) {
        dirty &= ~(1 << s);
        constexpr int kUnits = G::kUnitsPerBoxRow;
#pragma unroll 1
        for (int bx = 0; bx < G::kNumBox; ++bx)
#pragma unroll 4
          for (int i = p.group * kUnits + lane; i < kBM * kUnits; i += 32)
            reinterpret_cast<uint4 *>(smem + G::kOffQ + s * G::kTileBytes + bx * G::kBoxBytes)[i] =
                make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t bar = smem_u32(&bars->q_full[s]);
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, (one ? p.group : q_rows) * G::kRowBytes);
#pragma unroll
        for (int bx = 0; bx < G::kNumBox; ++bx)
          tma_load_3d(sQ + s * G::kTileBytes + bx * G::kBoxBytes, one ? &p.tm_q1 : &p.tm_q, bar,
                      bx * G::kBoxCols, h * p.group, tok, pol);
      }
      __syncwarp();
      ++nq;
    };
    // the first item's Q goes before the second item is looked for (with the
    // order of the others its product began 1.5 us later)
    for (int i = 0; ok; ++i) {
      const bool more = announce(ahead);
      if (i == 0) t = ahead;
      if (ok && i != 1 && t.h >= 0) {
        if (t.hi0 > t.lo0) load(t.h, t.tok0, t.nt0);
        if (ok && t.hi1 > t.lo1) load(t.h, t.tok0 + p.tile_q, t.nt1);
      }
      if (!ok || !more) break;
      if (ahead.slot >= 0 && lane == 0) {   // (read when the part is finished)
        bars->cut[ahead.slot] = walk.cut_of(cuts);
        mbar_arrive(smem_u32(&bars->cut_full[ahead.slot]));
      }
      __syncwarp();
      t = ahead;
    }
    if (!ok || *abort_flag)   // let the copies in flight land before the CTA exits
      for (int n = max(0, nq - 2); n < nq; ++n)
        mbar_wait_slow(smem_u32(&bars->q_full[n & 1]), (n >> 1) & 1, abort_flag, false);
    named_barrier_sync(kCountedBar, 64);   // thread 0 counts no more parts
    if (__builtin_expect(*abort_flag != 0, 0)) {
      // the others are counted here, so that the tickets end at 0 for a captured
      // call's next run (in this role: its registers are what the walk needs)
      walk.start(p, bars->setup, cuts);
      while (walk.next(p, t))
        if (t.slot >= 0 && lane == 0 && !bars->ticketed[t.slot]) paged_ticket(p, walk.cut_of(cuts));
    }
  } else if (warp == kLoadWarp || warp == kLoadWarpV) {
    // =================================================== K and V producers
    // Lane i copies the i-th run of box_rows rows of a key block (one page, or
    // 128 rows of a larger one), one copy per swizzle span of columns.  A page
    // that holds no visible key, or is not one (-1 in the table), is replaced
    // by the first page behind the cache, which the copy fills with zeros.
    const bool is_k = warp == kLoadWarp;
    const int nslot = is_k ? G::kSlotsK : G::kSlotsV;
    const int base = is_k ? 0 : G::kSlotsK;
    const CUtensorMap *map = is_k ? &p.tm_k : &p.tm_v;
    const int per_block = kBN / p.box_rows;          // copies of rows per block
    const int in_mask = (1 << p.page_shift) - 1;
    const uint64_t pol_keep = policy_evict_last(), pol_stream = policy_evict_first();
#ifdef FA_TEST_HOOKS
    const int withheld = blockIdx.x != 0 || g_fa_test_withhold_block < 0 ? -1
                         : is_k ? g_fa_test_withhold_block
                                : g_fa_test_withhold_block - kWithholdV;
#else
    constexpr int withheld = -1;
#endif
    PagedItem t;
    int q = 0;             // fills so far
    int ragged = 0;        // V: ragged blocks so far
    int pend_slot = -1, pend_lo = 0, pend_hi = 0;   // V: the one not yet cleared

    // rows [0, lo) and [hi, 128) of the ragged block := 0, then release it
    auto clear = [&]() {
      uint8_t *tile = smem + G::kOffRing + pend_slot * G::kTileBytes;
      constexpr int kUnits = G::kUnitsPerBoxRow;
#pragma unroll 1
      for (int bx = 0; bx < G::kNumBox; ++bx) {
        uint4 *box = reinterpret_cast<uint4 *>(tile + bx * G::kBoxBytes);
#pragma unroll 1
        for (int i = lane; i < pend_lo * kUnits; i += 32) box[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 4
        for (int i = pend_hi * kUnits + lane; i < kBN * kUnits; i += 32)
          box[i] = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->full[pend_slot]));
      __syncwarp();
      pend_slot = -1;
    };
    auto finish_ragged = [&]() {
      ok = mbar_wait_warp(smem_u32(&bars->v_ragged), (ragged - 1) & 1, abort_flag);
      if (ok) clear();
    };
    // Wait for a barrier; a ragged block that lands meanwhile is released (the
    // barrier may be one that only what waits for the block completes).
    auto wait_clearing = [&](uint32_t bar, uint32_t parity) {
      const unsigned long long t0 = pend_slot >= 0 ? globaltimer_ns() : 0;
      while (pend_slot >= 0) {
        if (__all_sync(0xffffffffu, mbar_test(smem_u32(&bars->v_ragged), (ragged - 1) & 1))) {
          clear();
          break;
        }
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return;
        const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
        if (__any_sync(0xffffffffu, late)) {
          *abort_flag = 1;
          atomicOr(&g_fa_status, 1u);
        }
        if (__any_sync(0xffffffffu, late || *abort_flag != 0)) {
          ok = false;
          return;
        }
      }
      ok = mbar_wait_warp(bar, parity, abort_flag);
    };

    for (int k = 0; ok; ++k) {
      if (pend_slot >= 0)
        wait_clearing(smem_u32(&bars->item_full[k % kItemRing]), (k / kItemRing) & 1);
      if (!ok || !take(k, t)) break;
      const int *row = p.table + t.b * p.table_stride;
      const uint64_t pol = t.once ? pol_stream : pol_keep;
      // page of this lane's rows of block j (-1: none), read one block ahead
      auto page_of = [&](int j) {
        const int pos = j * kBN + lane * p.box_rows;
        if (lane >= per_block || j >= t.hi || pos > t.khi || pos + p.box_rows <= t.klo) return -1;
        return __ldg(row + (pos >> p.page_shift));
      };
      int page = page_of(t.lo);
      for (int j = t.lo; j < t.hi; ++j, ++q) {
        const int next_page = page_of(j + 1);
        const int slot = base + q % nslot;
        if (q >= nslot) {
          wait_clearing(smem_u32(&bars->empty[slot]), ((q / nslot) - 1) & 1);
          if (!ok) break;
        }
        const int k0 = j * kBN;
        const bool rag = !is_k && (k0 < t.klo || k0 + kBN - 1 > t.khi);
        if (rag && pend_slot >= 0) {
          finish_ragged();
          if (!ok) break;
        }
        const uint32_t bar = smem_u32(rag ? &bars->v_ragged : &bars->full[slot]);
        const bool given = withheld < 0 || q != withheld;   // (always, but in the watchdog test library)
        if (lane == 0 && given) mbar_arrive_expect_tx(bar, G::kTileBytes);
        __syncwarp();
        if (lane < per_block && given) {
          const int in_page = (k0 + lane * p.box_rows) & in_mask;
          if (page < 0 || page >= p.n_pages) page = p.n_pages;
          const uint32_t dst = sRing + slot * G::kTileBytes + lane * p.box_rows * G::kSwBytes;
#pragma unroll
          for (int bx = 0; bx < G::kNumBox; ++bx)
            tma_load_4d(dst + bx * G::kBoxBytes, map, bar, bx * G::kBoxCols, in_page, t.h, page,
                        pol);
        }
        __syncwarp();
        if (rag) {
          ++ragged;
          pend_slot = slot;
          pend_lo = max(t.klo - k0, 0);
          pend_hi = min(t.khi - k0 + 1, kBN);
        }
        page = next_page;
      }
    }
    if (ok && pend_slot >= 0) finish_ragged();
    if (!ok || *abort_flag) {
      // let the copies in flight land before the CTA exits; a ragged block's
      // copy lands on v_ragged
      if (pend_slot >= 0)
        mbar_wait_slow(smem_u32(&bars->v_ragged), (ragged - 1) & 1, abort_flag, false);
      for (int n = max(0, q - nslot); n < q; ++n)
        if (base + n % nslot != pend_slot)
          mbar_wait_slow(smem_u32(&bars->full[base + n % nslot]), (n / nslot) & 1, abort_flag,
                         false);
    }
  } else {
    // =================================================== MMA issuer
    constexpr uint32_t kIdescS = make_idesc_f16(kBM, kBN, DT, 0, 0);
    constexpr uint32_t kIdescPV = make_idesc_f16(kBM, D, DT, 0, 1);
    constexpr uint32_t kHi = desc_hi(8 * G::kSwBytes, G::kLayout);
    PagedItem t;
    int nq = 0;                   // Q slots used so far
    int q = 0;                    // key blocks so far (K and V fills)
    int ns0 = 0, ns1 = 0;         // S tiles issued so far
    int np0 = 0, np1 = 0;         // P tiles taken so far
    int no0 = 0, no1 = 0;         // O tiles begun so far
    auto kslot = [&](int n) { return n % G::kSlotsK; };
    auto vslot = [&](int n) { return G::kSlotsK + n % G::kSlotsV; };
    auto wait = [&](uint64_t *bar, int n) {
      ok = ok && mbar_wait_warp(smem_u32(bar), n & 1, abort_flag);
    };
    auto commit = [&](uint64_t *bar) {
      if (elect_one()) tc_commit(smem_u32(bar));
      __syncwarp();
    };
    // S_u = Q K^T; with P beside S it waits until the softmax holds the last
    // S_u, otherwise the PV before it (which reads P over S) was issued first
    auto issue_s = [&](int u, int qs, int slot) {
      const int n = u ? ns1 : ns0;
      if (kSplitP && n > 0) wait(&bars->s_free[u], n - 1);
      if (!ok) return;
      tc_fence_after_sync();
      const uint32_t qlo = desc_lo(sQ + qs * G::kTileBytes, 16);
      const uint32_t klo = desc_lo(sRing + slot * G::kTileBytes, 16);
      const uint32_t d_tmem = tmem + (u ? 128u : 0u);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / kKStep; ++kk) {
          const int byte = kk * 32;
          const uint32_t off = ((byte / G::kSwBytes) * G::kBoxBytes + (byte % G::kSwBytes)) >> 4;
          mma_ss(d_tmem, desc_join(qlo + off, kHi), desc_join(klo + off, kHi), kIdescS,
                 kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars->s_full[u]));
      }
      __syncwarp();
      if (u) ++ns1; else ++ns0;
    };
    // O_u (+)= P_u V; the item's first product of a tile waits until the
    // epilogue has read the last item's O
    auto issue_pv = [&](int u, int slot, bool first) {
      wait(&bars->p_full[u], u ? np1 : np0);
      if (first && (u ? no1 : no0) > 0) wait(&bars->o_free[u], (u ? no1 : no0) - 1);
      if (!ok) return;
      tc_fence_after_sync();
      const uint32_t vlo = desc_lo(sRing + slot * G::kTileBytes, G::kBoxBytes);
      const uint32_t a_tmem = tmem + (kSplitP ? 384u + (u ? 64u : 0u) : (u ? 128u : 0u));
      const uint32_t d_tmem = tmem + 256u + (u ? D : 0u);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kBN / kKStep; ++kk)
          mma_ts(d_tmem, a_tmem + kk * 8, desc_join(vlo + ((kk * kKStep * G::kSwBytes) >> 4), kHi),
                 kIdescPV, (!first || kk > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bars->pv_done[u]));
      }
      __syncwarp();
      if (u) ++np1; else ++np0;
      if (first) { if (u) ++no1; else ++no0; }
    };

    for (int k = 0; ok && take(k, t); ++k) {
      if (t.hi <= t.lo) continue;
      const int q0 = q;                       // fill index of block lo
      if (t.nt1 <= 0) {
        // one tile: even blocks to warpgroup 0, odd ones to warpgroup 1
        const int qs = nq & 1;
        wait(&bars->q_full[qs], nq >> 1);
        ++nq;
        const int nb = t.hi - t.lo;
        auto step_s = [&](int n) {
          wait(&bars->full[kslot(q0 + n)], (q0 + n) / G::kSlotsK);
          if (ok) issue_s(n & 1, qs, kslot(q0 + n));
          if (!ok) return;
          commit(&bars->empty[kslot(q0 + n)]);
          if (n == nb - 1) commit(&bars->q_empty[qs]);
        };
        auto step_pv = [&](int n) {
          wait(&bars->full[vslot(q0 + n)], (q0 + n) / G::kSlotsV);
          if (ok) issue_pv(n & 1, vslot(q0 + n), n < 2);
          if (ok) commit(&bars->empty[vslot(q0 + n)]);
        };
        for (int n = 0; n < nb + 2 && ok; ++n) {
          if (kSplitP) {
            if (n < nb) step_s(n);
            if (ok && n >= 2) step_pv(n - 2);
          } else {
            if (n >= 2) step_pv(n - 2);
            if (ok && n < nb) step_s(n);
          }
        }
      } else {
        const bool act0 = t.hi0 > t.lo0, act1 = t.hi1 > t.lo1;
        const int qs0 = nq & 1;
        if (act0) {
          wait(&bars->q_full[qs0], nq >> 1);
          ++nq;
        }
        const int qs1 = nq & 1;
        if (act1) {
          wait(&bars->q_full[qs1], nq >> 1);
          ++nq;
        }
        auto in0 = [&](int j) { return j >= t.lo0 && j < t.hi0; };
        auto in1 = [&](int j) { return j >= t.lo1 && j < t.hi1; };
        auto last_s = [&](int j) {   // after the S of block j
          commit(&bars->empty[kslot(q0 + j - t.lo)]);
          if (j == t.hi - 1) {
            if (act0) commit(&bars->q_empty[qs0]);
            if (act1) commit(&bars->q_empty[qs1]);
          }
        };
        if constexpr (kSplitP) {
          // S0(j), S1(j), PV0(j-1), PV1(j-1)
          for (int j = t.lo; j <= t.hi && ok; ++j) {
            const int n = q0 + j - t.lo;
            if (j < t.hi) {
              wait(&bars->full[kslot(n)], n / G::kSlotsK);
              if (ok && in0(j)) issue_s(0, qs0, kslot(n));
              if (ok && in1(j)) issue_s(1, qs1, kslot(n));
              if (!ok) break;
              last_s(j);
            }
            if (j > t.lo) {
              wait(&bars->full[vslot(n - 1)], (n - 1) / G::kSlotsV);
              if (ok && in0(j - 1)) issue_pv(0, vslot(n - 1), j - 1 == t.lo0);
              if (ok && in1(j - 1)) issue_pv(1, vslot(n - 1), j - 1 == t.lo1);
              if (ok) commit(&bars->empty[vslot(n - 1)]);
            }
          }
        } else {
          // ping-pong: S0(j), PV1(j-1), S1(j), PV0(j); the fills of V(j) and
          // K(j+1) are waited for before P0(j), the wait that lasts
          wait(&bars->full[kslot(q0)], q0 / G::kSlotsK);
          for (int j = t.lo; j < t.hi && ok; ++j) {
            const int n = q0 + j - t.lo;
            if (in0(j)) issue_s(0, qs0, kslot(n));
            if (j > t.lo) {
              if (in1(j - 1)) issue_pv(1, vslot(n - 1), j - 1 == t.lo1);
              if (!ok) break;
              commit(&bars->empty[vslot(n - 1)]);
            }
            if (in1(j)) issue_s(1, qs1, kslot(n));
            if (!ok) break;
            last_s(j);
            wait(&bars->full[vslot(n)], n / G::kSlotsV);
            if (j + 1 < t.hi) wait(&bars->full[kslot(n + 1)], (n + 1) / G::kSlotsK);
            if (!ok) break;
            if (in0(j)) issue_pv(0, vslot(n), j == t.lo0);
          }
          if (ok) {
            const int n = q0 + t.hi - 1 - t.lo;
            if (in1(t.hi - 1)) issue_pv(1, vslot(n), t.hi - 1 == t.lo1);
            if (ok) commit(&bars->empty[vslot(n)]);
          }
        }
      }
      q = q0 + t.hi - t.lo;
    }
    if (elect_one()) tc_commit(smem_u32(&bars->mma_done));
    __syncwarp();
  }
  } else {
    // =================================================== softmax / epilogue
    regs_inc<RegSplit::kBig>();
    const int u = warp >> 2;                 // warpgroup
    const int r = tid & 127;                 // tile row = TMEM lane
    const int r_tok = r / p.group, r_head = r - (r / p.group) * p.group;
    const int few_tok = (lane >> 2) / p.group;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + u * 128u;
    const uint32_t tP = kSplitP ? tmem + lane_base + 384u + u * 64u : tS;
    const uint32_t tO = tmem + lane_base + 256u + u * D;
    const uint32_t tO0 = tmem + lane_base + 256u;
    float2 *xch = reinterpret_cast<float2 *>(smem + PG::kOffXch);
    const float sl2 = p.scale_log2;
    const float2 sl2v = make_float2(sl2, sl2);
    PagedItem t;
    int ns = 0;                              // S tiles taken so far
    int nx = 0;                              // (m, l) exchanges so far
    int n_part = 0;                          // parts written so far
    // one arrival for the warp, after its lanes' work
    auto arrive = [&](uint64_t *bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(bar));
    };

    for (int k = 0; ok && take(k, t); ++k) {
      const bool single = t.nt1 <= 0;
      const int tile = single ? 0 : u;       // query tile of this warpgroup
      const int nt = tile ? t.nt1 : t.nt0;
      const int first = t.first + tile * p.tile_q, last = first + nt - 1;
      const bool valid = r_tok < nt;         // (r_tok >= tile_q: rows behind the tile)
      const bool busy = __any_sync(0xffffffffu, valid);
      const bool few = single && nt * p.group <= kFewRows;
      const int x = first + (few ? few_tok : r_tok);   // this lane's row of the softmax
      const int row_lo = p.wl < 0 ? 0 : max(0, x - p.wl);
      const int row_hi = p.wr < 0 ? t.kv_len - 1 : min(t.kv_len - 1, x + p.wr);
      const int full_lo = p.wl < 0 ? 0 : max(0, last - p.wl);
      const int full_hi = p.wr < 0 ? t.kv_len - 1 : min(t.kv_len - 1, first + p.wr);
      const int j0 = single ? t.lo + u : (tile ? t.lo1 : t.lo0);
      const int jstep = single ? 2 : 1;
      const int n_blocks = single ? (t.hi - t.lo + 1 - u) / 2
                                  : (tile ? t.hi1 - t.lo1 : t.hi0 - t.lo0);

      float m_use = -INFINITY;   // reference max, log2 units of the scaled scores
      float l = 0.0f;            // normaliser relative to m_use
      if (few && busy) {
        const bool real = few_tok < nt;
        for (int n = 0; n < n_blocks; ++n, ++ns) {
          const int k0 = (j0 + n * jstep) * kBN;
          ok = mbar_wait_warp(smem_u32(&bars->s_full[u]), ns & 1, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
          float2 s[16];
          {
            uint32_t sr[2][32];
            tmem_ld_rows16(tS, sr[0]);
            tmem_ld_rows16(tS + 64, sr[1]);
            tmem_wait_ld();
            reg_dep(sr[0]);
            reg_dep(sr[1]);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              s[j] = make_float2(__uint_as_float(sr[j >> 3][(j & 7) * 4]),
                                 __uint_as_float(sr[j >> 3][(j & 7) * 4 + 1]));
          }
          if (kSplitP) {   // S may be overwritten from here on
            tc_fence_before_sync();
            arrive(&bars->s_free[u]);
          }
          if (k0 < full_lo || k0 + kBN - 1 > full_hi) {
            const int at = k0 + 2 * (lane & 3), lo_c = row_lo - at, hi_c = row_hi - at;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (8 * j < lo_c || 8 * j > hi_c) s[j].x = -INFINITY;
              if (8 * j + 1 < lo_c || 8 * j + 1 > hi_c) s[j].y = -INFINITY;
            }
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 16; ++j) mx[j & 1] = fmax3(mx[j & 1], s[j].x, s[j].y);
          float m = fmaxf(mx[0], mx[1]);
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          m = m == -INFINITY ? -INFINITY : m * sl2;
          float alpha = 1.0f;
          const bool rescale = __any_sync(0xffffffffu, m > m_use + kRescaleThreshold);
          if (rescale) {
            const float m_upd = fmaxf(m_use, m);
            alpha = (m_upd == -INFINITY) ? 1.0f : ex2(m_use - m_upd);
            m_use = m_upd;
            l *= alpha;
          }
          const float nm = !real ? -INFINITY : (m_use == -INFINITY ? 0.0f : -m_use);
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 e = __ffma2_rn(s[j], sl2v, make_float2(nm, nm));
            const float2 pp = make_float2(ex2(e.x), ex2(e.y));
            ls[j & 1] = __fadd2_rn(ls[j & 1], pp);
            pk[2 * j] = pack2<DT>(pp.x, pp.y);
            pk[2 * j + 1] = pack2_rest<DT>(pp, pk[2 * j]);   // row g + 8
          }
          if (kSplitP && ns > 0) {
            ok = mbar_wait_warp(smem_u32(&bars->pv_done[u]), (ns - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
          }
          tmem_st_rows16(tP, pk);
          if (kSplitP && n == 0) {   // zeros behind, for the power
#pragma unroll
            for (int j = 0; j < 32; ++j) pk[j] = 0u;
            tmem_st_rows16(tP + (16u << 16), pk);
          }
          if (rescale && n > 0)
            scale_o_row<D>(tO, __shfl_sync(0xffffffffu, alpha, (4 * lane) & 31));
          l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
          tmem_wait_st();
          tc_fence_before_sync();
          arrive(&bars->p_full[u]);
        }
        // a lane holds the row of its TMEM lane again (the first 8, and in the
        // next 8 the same rows, whose O is the weights' rests')
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        l = __shfl_sync(0xffffffffu, l, (4 * lane) & 31);
        m_use = __shfl_sync(0xffffffffu, m_use, (4 * lane) & 31);
      } else {
      for (int n = 0; n < n_blocks; ++n, ++ns) {
        const int k0 = (j0 + n * jstep) * kBN;
        ok = mbar_wait_warp(smem_u32(&bars->s_full[u]), ns & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        if (!busy) {
          // nothing of this warp's rows is read or kept.  It must not arrive for
          // this P while the others have not for the last one.
          if (kSplitP) {
            tc_fence_before_sync();
            arrive(&bars->s_free[u]);
            if (ns > 0) ok = mbar_wait_warp(smem_u32(&bars->pv_done[u]), (ns - 1) & 1, abort_flag);
            if (!ok) break;
            if (n == 0) {   // zeros, for the power (beside S, P is what an earlier item left)
              tc_fence_after_sync();
              uint32_t z[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = 0u;
              store_p_half<DT>(tP, 0, z);
              store_p_half<DT>(tP, 1, z);
              tmem_wait_st();
            }
          }
        } else {
          auto load_s = [&](float (&sv)[kBN], auto masked) {
            uint32_t sr[4][32];
            tmem_ld_x32(tS + 0, sr[0]);
            tmem_ld_x32(tS + 32, sr[1]);
            tmem_ld_x32(tS + 64, sr[2]);
            tmem_ld_x32(tS + 96, sr[3]);
            tmem_wait_ld();
            reg_dep(sr[0]);
            reg_dep(sr[1]);
            reg_dep(sr[2]);
            reg_dep(sr[3]);
#pragma unroll
            for (int c = 0; c < kBN; ++c) sv[c] = __uint_as_float(sr[c >> 5][c & 31]);
            if constexpr (!decltype(masked)::value) return;
            if (k0 + kBN - 1 > full_hi) {   // some row's last key is in the block
              const int hi_c = row_hi - k0;
#pragma unroll
              for (int c = 0; c < kBN; ++c)
                if (c > hi_c) sv[c] = -INFINITY;
            }
            if (k0 < full_lo) {             // some row's window begins in it
              const int lo_c = row_lo - k0;
#pragma unroll
              for (int c = 0; c < kBN; ++c)
                if (c < lo_c) sv[c] = -INFINITY;
            }
          };
          float alpha = 1.0f;
          bool rescale = false;
          float2 ls[2];
          // the row's reference raised to m_new where some row of the warp
          // grew by more than 2^8
          auto raise = [&](float m_new) {
            rescale = __any_sync(0xffffffffu, m_new > m_use + kRescaleThreshold);
            if (rescale) {
              const float m_upd = fmaxf(m_use, m_new);
              alpha = (m_upd == -INFINITY) ? 1.0f : ex2(m_use - m_upd);
              m_use = m_upd;
              l *= alpha;
            }
          };
          auto row_max = [&](const float (&sv)[kBN]) {
            float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
            for (int c = 4; c < kBN - 4; c += 8)
#pragma unroll
              for (int v = 0; v < 4; ++v) mx[v] = fmax3(mx[v], sv[c + 2 * v], sv[c + 2 * v + 1]);
            const float m = fmax3(fmax3(mx[0], mx[1], sv[kBN - 4]), fmax3(mx[2], mx[3], sv[kBN - 3]),
                                  fmaxf(sv[kBN - 2], sv[kBN - 1]));
            return m == -INFINITY ? -INFINITY : m * sl2;
          };
          // minus the reference; rows that are none get zero weights
          auto neg_ref = [&]() {
            return !valid ? -INFINITY : (m_use == -INFINITY ? 0.0f : -m_use);
          };
          // P of one half against the reference; the weights summed unrounded
          auto exp_half = [&](const float (&sv)[kBN], int half, uint32_t (&pk)[32]) {
            const float nm = neg_ref();
            const float2 negm = make_float2(nm, nm);
#pragma unroll
            for (int c = 0; c < kBN / 2; c += 2) {
              const float2 e =
                  __ffma2_rn(make_float2(sv[half * 64 + c], sv[half * 64 + c + 1]), sl2v, negm);
              const float2 pp = make_float2(ex2(e.x), ex2(e.y));
              ls[(c >> 1) & 1] = __fadd2_rn(ls[(c >> 1) & 1], pp);
              put_p<DT>(pk, c >> 1, pp.x, pp.y);
            }
          };
          ls[0] = ls[1] = make_float2(0.f, 0.f);
          if constexpr (kSplitP) {
            float s[kBN];
            load_s(s, std::true_type{});
            // S may be overwritten from here on; P and O wait for the PV before
            tc_fence_before_sync();
            arrive(&bars->s_free[u]);
            raise(row_max(s));
            uint32_t pk[2][32];
            exp_half(s, 0, pk[0]);
            exp_half(s, 1, pk[1]);
            if (ns > 0) {
              ok = mbar_wait_warp(smem_u32(&bars->pv_done[u]), (ns - 1) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after_sync();
            }
            store_p_half<DT>(tP, 0, pk[0]);
            store_p_half<DT>(tP, 1, pk[1]);
            if (rescale && n > 0) scale_o_row<D>(tO, alpha);
          } else {
            auto exact_pass = [&](const float (&sv)[kBN]) {
              raise(row_max(sv));
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t pk[32];
                exp_half(sv, half, pk);
                store_p_half<DT>(tP, half, pk);
              }
              // O is complete up to the block before: S was issued after its PV
              if (rescale && n > 0) scale_o_row<D>(tO, alpha);
            };
            // every row has a reference: exponentials and maximum side by
            // side; redone if some row grew by more than 2^8
            bool done = false;
            auto guess = [&](auto masked) {
              float s[kBN];
              load_s(s, masked);
              const float nm = neg_ref();
              const float2 negm = make_float2(nm, nm);
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
              float2 lf[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              uint32_t pk[2][32];
#pragma unroll
              for (int c = 0; c < kBN; c += 2) {
                const int pair = c >> 1;
                mx[pair & 3] = fmax3(mx[pair & 3], s[c], s[c + 1]);
                const float2 e = __ffma2_rn(make_float2(s[c], s[c + 1]), sl2v, negm);
                const float2 pp = make_float2(ex2(e.x), ex2(e.y));
                lf[pair & 1] = __fadd2_rn(lf[pair & 1], pp);
                put_p<DT>(pk[c >> 6], pair & 31, pp.x, pp.y);
              }
              const float m_new = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
              done = !__any_sync(0xffffffffu, m_new > m_use + kRescaleThreshold);
              if (done) {
                store_p_half<DT>(tP, 0, pk[0]);
                store_p_half<DT>(tP, 1, pk[1]);
                ls[0] = lf[0];
                ls[1] = lf[1];
              }
            };
            if (__all_sync(0xffffffffu, m_use != -INFINITY)) {
              if (k0 >= full_lo && k0 + kBN - 1 <= full_hi)   // (a copy without masks: 5 % of a long prefill)
                guess(std::false_type{});
              else
                guess(std::true_type{});
            }
            if (!done) {
              float s[kBN];
              load_s(s, std::true_type{});
              exact_pass(s);
            }
          }
          l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
          tmem_wait_st();
        }
        tc_fence_before_sync();
        arrive(&bars->p_full[u]);
      }
      }
      if (ok && n_blocks > 0) {
        ok = mbar_wait_warp(smem_u32(&bars->pv_done[u]), (ns - 1) & 1, abort_flag);
        tc_fence_after_sync();
      }
      if (!ok) break;

      // ---- epilogue.  A single tile: the warpgroups exchange their (m, l) and
      // each joins every other 16 columns of the two O.
      float wa = 1.0f, wb = 0.0f;
      const bool two = single && t.hi - t.lo > 1;   // both O hold something
      if (single) {
        if (nx > 0) ok = mbar_wait_warp(smem_u32(&bars->ml_free[u]), (nx - 1) & 1, abort_flag);
        if (!ok) break;
        xch[u * kBM + r] = make_float2(m_use, l);
        tc_fence_before_sync();
        arrive(&bars->ml_full[u]);
        ok = mbar_wait_warp(smem_u32(&bars->ml_full[1 - u]), nx & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        const float2 o = xch[(1 - u) * kBM + r];
        arrive(&bars->ml_free[1 - u]);
        ++nx;
        const float m = fmaxf(m_use, o.x);
        const float w_mine = (m_use == -INFINITY) ? 0.0f : ex2(m_use - m);
        const float w_other = (o.x == -INFINITY) ? 0.0f : ex2(o.x - m);
        wa = u ? w_other : w_mine;
        wb = u ? w_mine : w_other;
        const float la = u ? o.y : l, lb = u ? l : o.y;
        l = wa * la + wb * lb;       // the same sum in both warpgroups
        m_use = m;
      }
      const bool none = t.hi <= t.lo || (!single && n_blocks <= 0);   // no O at all
      if (busy) {
        const float inv = t.slot >= 0 ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f);
        const int tok = t.tok0 + tile * p.tile_q + r_tok, head = t.h * p.group + r_head;
        uint8_t *orow = static_cast<uint8_t *>(p.out) +
                        2 * (static_cast<long long>(tok) * p.out_st +
                             static_cast<long long>(head) * p.out_sh);
        const int slot = 2 * blockIdx.x + max(t.slot, 0), srow = tile * kBM + r;
        float4 *wo = paged_slot(p, D, slot) + srow;
        const uint32_t from = single ? tO0 : tO;
        const float sa = wa * inv, sb = wb * inv;
        if (few)
          paged_few_rows<D, DT>(p, t, tO0, u, few_tok, none, two, sa, sb, slot);
#pragma unroll 1
        for (int c = few ? D : (single ? 16 * u : 0); c < D; c += single ? 32 : 16) {
          float o[16];
          if (none) {
#pragma unroll
            for (int v = 0; v < 16; ++v) o[v] = 0.0f;
          } else {
            uint32_t x0[16];
            tmem_ld_x16(from + c, x0);
            if (two) {
              uint32_t x1[16];
              tmem_ld_x16(from + D + c, x1);
              tmem_wait_ld();
              reg_dep(x0);
              reg_dep(x1);
#pragma unroll
              for (int v = 0; v < 16; ++v)
                o[v] = sa * __uint_as_float(x0[v]) + sb * __uint_as_float(x1[v]);
            } else {
              tmem_wait_ld();
              reg_dep(x0);
#pragma unroll
              for (int v = 0; v < 16; ++v) o[v] = sa * __uint_as_float(x0[v]);
            }
          }
          if (valid && t.slot >= 0) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              wo[(c / 4 + v) * kPagedRows] =
                  make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          } else if (valid) {
            paged_store16<DT>(p, orow, c, o);
          }
          __syncwarp();   // the next chunk's load is warp-collective
        }
        if (valid && !(single && u == 1)) {
          if (t.slot >= 0)
            p.ws_ml[static_cast<size_t>(slot) * kPagedRows + srow] =
                make_float2(l > 0.0f ? m_use : -INFINITY, l);
          else if (p.lse != nullptr)
            p.lse[static_cast<size_t>(tok) * p.H + head] =
                l > 0.0f ? (m_use + __log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
      }
      // O has been read: the next item's first PV may overwrite it.  (Eight
      // arrivals: a pair's tile has one warpgroup, whose warps count twice.)
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (single) {
          if (t.hi > t.lo) mbar_arrive(smem_u32(&bars->o_free[0]));
          if (two) mbar_arrive(smem_u32(&bars->o_free[1]));
        } else if (n_blocks > 0) {
          mbar_arrive_n(smem_u32(&bars->o_free[u]), 2);
        }
      }
      if (t.slot >= 0) {
        // a part: whoever finishes the item's last one joins them all
        // (one thread's fences order the CTA's rows, which it has seen arrive)
        arrive(&bars->part_done);
        if (tid == 0) {
          ok = mbar_wait(smem_u32(&bars->part_done), n_part & 1, abort_flag) &&
               mbar_wait(smem_u32(&bars->cut_full[t.slot]), 0, abort_flag);
          if (ok) {
            __threadfence();
            bars->is_last = paged_ticket(p, bars->cut[t.slot]);
            bars->ticketed[t.slot] = 1;
            __threadfence();
            mbar_arrive(smem_u32(&bars->part_last));
          }
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
        if (ok) ok = mbar_wait_warp(smem_u32(&bars->part_last), n_part & 1, abort_flag);
        if (!ok) break;
        ++n_part;
        if (bars->is_last) {
          paged_merge<D, DT>(p, t, bars->cut[t.slot], warp, 8);
        }
        // (is_last is written again only after all eight warps have arrived
        // for the next part)
      }
    }
    if (warp == 0) named_barrier_arrive(kCountedBar, 64);
  }

  // ---- teardown
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    mbar_wait_slow(smem_u32(&bars->mma_done), 0, abort_flag, false);
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace fa
