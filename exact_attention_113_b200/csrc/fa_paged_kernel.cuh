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
// 128 and costs blocks + 1.  The costs of all of them form one line, cut in
// equal pieces, one per CTA (one CTA per SM), so that one long request, many
// short ones and causal triangles all fill the device.  A CTA walks its
// piece, whole items and, at the ends, parts of two items; parts leave an
// unnormalised fp32 O and (m, l) in the workspace and fa_paged_merge_kernel
// joins them.  Each CTA finds its piece from the lengths by itself (a scan
// over the requests during set-up), so a call needs no schedule from the
// host, which does not know the lengths.
//
// A pair of two tiles runs as the forward kernel's ping-pong: per key block
// S0, PV1(previous), S1, PV0, two softmax warpgroups in turns.  A single tile
// (decoding, short chunks) gives even key blocks to one warpgroup and odd ones
// to the other, each with its own (m, l, O), joined at the end; that keeps two
// blocks in flight where one tile's S -> softmax -> PV chain would be exposed.
//
// Warps (384 threads): 0-3, 4-7 softmax; 8 MMA and TMEM; 9 K; 10 V; 11 Q.
// TMEM: S0 [0,128), S1 [128,256) (P over the first 64 columns of each),
// O0 [256,256+D), O1 [256+D,256+2D).
//
// V rows no query of the item sees (behind the request's end, in a page's
// unwritten tail, or before every window) are cleared in shared memory: their
// weight is an exact 0, but 0 times an unwritten NaN would not be.
#pragma once

#include "fa_fwd_kernel.cuh"

namespace fa {

constexpr int kLoadWarpQ = 11;
constexpr int kPagedMinUnits = 3;   // cost a CTA gets at least
constexpr int kPagedRows = 2 * kBM; // rows of a work item

struct PagedRec {   // what CTA c leaves for the merge (workspace)
  int cont;         // its first item began in an earlier CTA
  int ends;         // ... and ends here: this CTA's index names the merge
  int b, h, pair;   // that item
  int pad[3];
};

struct PagedParams {
  CUtensorMap tm_q;   // (D, H, total_q), box (cols, G, TQ)
  CUtensorMap tm_k;   // (D, P, H_kv, pages), box (cols, box_rows, 1, 1)
  CUtensorMap tm_v;
  const int *table;
  long long table_stride;
  const int *cu_q;
  const int *kv_lens;
  void *out;
  long long out_st, out_sh;   // element strides of a token and a head
  float *lse;                 // [total_q, H] or nullptr
  int B, H, H_kv, group, total_q;
  int tile_q;                 // tokens per tile
  int n_pages, page_size, max_kv;   // max_kv: table columns * page size
  int box_rows;               // rows of one K/V copy: min(page size, 128)
  int wl, wr;                 // -1 = unbounded
  float scale_log2;
  float *ws_o;                // [2 * grid][kPagedRows][D]
  float2 *ws_ml;              // [2 * grid][kPagedRows]
  PagedRec *rec;              // [grid]
};

// ------------------------------------------------------------------ the work line
struct PagedReq {
  int q_start, q_len, kv_len;
};

// Lengths of request b, clamped to the tensors: bad lengths give wrong rows,
// never an access outside them.
__device__ __forceinline__ PagedReq paged_req(const PagedParams &p, int b) {
  PagedReq r;
  const int a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1);
  r.q_start = min(max(a, 0), p.total_q);
  r.q_len = max(min(e, p.total_q) - r.q_start, 0);
  r.kv_len = min(max(__ldg(p.kv_lens + b), 0), p.max_kv);
  return r;
}

__device__ __forceinline__ int paged_pairs(const PagedParams &p, int q_len) {
  return (q_len + 2 * p.tile_q - 1) / (2 * p.tile_q);
}

// Keys [klo, khi] that tokens [i0, i0 + n) of the request see; khi < klo: none.
__device__ __forceinline__ void paged_keys(const PagedParams &p, const PagedReq &r, int i0, int n,
                                           int &klo, int &khi) {
  const int first = r.kv_len - r.q_len + i0, last = first + n - 1;
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

// Cost of one K/V head of a request; the whole warp calls it, each lane with
// its own request (q_len 0: none).  Long requests are summed by all lanes.
__device__ __forceinline__ long long paged_head_cost(const PagedParams &p, const PagedReq &r) {
  constexpr int kAlone = 4;
  const int lane = threadIdx.x & 31;
  const int np = paged_pairs(p, r.q_len);
  long long sum = 0;
  if (np <= kAlone)
    for (int i = 0; i < np; ++i) sum += paged_blocks(p, r, i) + 1;
  unsigned todo = __ballot_sync(0xffffffffu, np > kAlone);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    PagedReq o;
    o.q_start = 0;
    o.q_len = __shfl_sync(0xffffffffu, r.q_len, src);
    o.kv_len = __shfl_sync(0xffffffffu, r.kv_len, src);
    const int n = paged_pairs(p, o.q_len);
    long long all = 0;
    for (int i = lane; i < n; i += 32) all += paged_blocks(p, o, i) + 1;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    if (lane == src) sum = all;
  }
  return sum;
}

// A place on the work line: request, K/V head, pair and the offset in its cost.
struct PagedPos {
  int b, h, pair, off;
};

// Set-up state in shared memory.
struct PagedSetup {
  long long warp_sum[kThreads / 32];
  long long u[2];       // first and last unit of this CTA's piece
  PagedPos at[2];       // the same as places
  int cost[2];          // the cost of the item at them
};

// Finds this CTA's piece of the work line: st.u, st.at[0].  Called by all
// threads of the block; ends with a barrier.
__device__ __forceinline__ void paged_find_piece(const PagedParams &p, PagedSetup &st) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kThreads / 32;
  auto cost_of = [&](int b) {
    PagedReq r;
    r.q_start = r.q_len = r.kv_len = 0;
    if (b < p.B) r = paged_req(p, b);
    return paged_head_cost(p, r) * p.H_kv;
  };
  const long long first = cost_of(tid);
  long long mine = first;
  for (int base = kThreads; base < p.B; base += kThreads) mine += cost_of(base + tid);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  if (lane == 0) st.warp_sum[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += st.warp_sum[w];
  // pieces: as many as there are CTAs, none below kPagedMinUnits
  const long long n = max(1ll, min(static_cast<long long>(gridDim.x), total / kPagedMinUnits));
  const long long c = blockIdx.x;
  const long long want[2] = {c >= n ? total : total / n * c + total % n * c / n,
                             c + 1 >= n ? total : total / n * (c + 1) + total % n * (c + 1) / n};
  if (tid < 2) {
    st.at[tid] = {p.B, 0, 0, 0};
    st.u[tid] = want[tid];
    st.cost[tid] = 0;
  }
  long long before = 0;
  for (int base = 0; base < p.B; base += kThreads) {
    __syncthreads();
    const long long s = base == 0 ? first : cost_of(base + tid);
    long long incl = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) st.warp_sum[warp] = incl;
    __syncthreads();
    long long pre = before;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += st.warp_sum[w];
      before += st.warp_sum[w];
    }
    const long long lo = pre + incl - s;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (s > 0 && want[e] >= lo && want[e] < lo + s) {
        st.at[e].b = base + tid;
        st.u[e] = want[e] - lo;   // rest within the request, for the next step
      }
  }
  __syncthreads();
  // head, pair and offset: warp e searches for end e
  if (warp < 2 && st.at[warp].b < p.B) {
    const int e = warp;
    const PagedReq r = paged_req(p, st.at[e].b);
    const int np = paged_pairs(p, r.q_len);
    PagedReq alone = r;
    if (lane != 0) alone.q_len = 0;
    const long long per_head = __shfl_sync(0xffffffffu, paged_head_cost(p, alone), 0);
    const long long rest = st.u[e];
    const int h = static_cast<int>(rest / per_head);
    long long in = rest - h * per_head;
    int pair = 0, off = 0, cost = 0;
    for (int base = 0; base < np; base += 32) {
      const int i = base + lane;
      const int cst = i < np ? paged_blocks(p, r, i) + 1 : 0;
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
        cost = __shfl_sync(0xffffffffu, cst, src);
        off = static_cast<int>(in - (__shfl_sync(0xffffffffu, incl, src) - cost));
        break;
      }
      in -= __shfl_sync(0xffffffffu, incl, 31);
    }
    // A cut one unit behind an item's start would leave a part without a key
    // block, one unit before its end a part of one: move both to the border.
    long long u = want[e];
    if (off == 1) {
      off = 0;
      u -= 1;
    } else if (off == cost - 1 && off > 0) {
      off = cost;
      u += 1;
    }
    if (lane == 0) {
      st.at[e].h = h;
      st.at[e].pair = pair;
      st.at[e].off = off;
      st.u[e] = u;
      st.cost[e] = cost;
    }
  }
  __syncthreads();
}

// One part of an item, as a CTA's roles see it (warp-uniform).
struct PagedPart {
  int b, h, pair;
  int tok0;            // packed row of the first tile's first token
  int nt0, nt1;        // tokens of the tiles
  int first;           // position of the first token
  int kv_len;
  int lo, hi;          // key blocks of the part (both tiles)
  int lo0, hi0, lo1, hi1;   // ... of each tile
  int klo, khi;        // keys some token of the item sees
  int slot;            // -1: the whole item; 0 / 1: workspace slot of the part
};

// Walks a CTA's piece.  Every role walks it by itself.
struct PagedWalk {
  int b, h, pair, off;
  long long left;
  PagedReq r;

  __device__ __forceinline__ void start(const PagedParams &p, const PagedSetup &st) {
    b = st.at[0].b;
    h = st.at[0].h;
    pair = st.at[0].pair;
    off = st.at[0].off;
    left = st.u[1] - st.u[0];
    if (b < p.B) {
      r = paged_req(p, b);
      if (off >= st.cost[0]) advance(p);   // the cut moved to the item's end
    }
  }
  __device__ __forceinline__ void advance(const PagedParams &p) {
    off = 0;
    if (++pair < paged_pairs(p, r.q_len)) return;
    pair = 0;
    if (++h < p.H_kv) return;
    h = 0;
    while (++b < p.B) {
      r = paged_req(p, b);
      if (r.q_len > 0) return;
    }
  }
  __device__ __forceinline__ bool next(const PagedParams &p, PagedPart &t) {
    if (left <= 0 || b >= p.B) return false;
    t.b = b;
    t.h = h;
    t.pair = pair;
    const int i0 = pair * 2 * p.tile_q;
    t.tok0 = r.q_start + i0;
    t.nt0 = min(p.tile_q, r.q_len - i0);
    t.nt1 = min(p.tile_q, r.q_len - i0 - t.nt0);
    t.first = r.kv_len - r.q_len + i0;
    t.kv_len = r.kv_len;
    int klo0, khi0, klo1, khi1;
    paged_keys(p, r, i0, t.nt0, klo0, khi0);
    paged_keys(p, r, i0 + p.tile_q, t.nt1, klo1, khi1);
    paged_keys(p, r, i0, t.nt0 + t.nt1, t.klo, t.khi);
    const int blocks = t.khi < t.klo ? 0 : t.khi / kBN - t.klo / kBN + 1;
    const int lo = t.klo / kBN;
    const int cost = blocks + 1;
    const int end = static_cast<int>(min(static_cast<long long>(cost), off + left));
    t.lo = lo + max(off - 1, 0);
    t.hi = end >= cost ? lo + blocks : lo + end - 1;
    t.slot = off > 0 ? 0 : (end < cost ? 1 : -1);
    t.lo0 = max(t.lo, klo0 / kBN);
    t.hi0 = khi0 < klo0 ? t.lo0 : max(t.lo0, min(t.hi, khi0 / kBN + 1));
    t.lo1 = max(t.lo, klo1 / kBN);
    t.hi1 = khi1 < klo1 ? t.lo1 : max(t.lo1, min(t.hi, khi1 / kBN + 1));
    left -= end - off;
    if (end >= cost)
      advance(p);
    else
      off = end;
    return true;
  }
};

// ------------------------------------------------------------------ shared memory
template <int kSlots>
struct PagedBars {
  uint64_t q_full[2];    // Q slot filled
  uint64_t q_empty[2];   // every S that reads it is done
  uint64_t full[kSlots];
  uint64_t empty[kSlots];
  uint64_t v_ragged;     // the copy of a V block whose hidden rows are cleared
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t pv_done[2];
  uint64_t o_free[2];    // O_t has been read by the epilogue
  uint64_t ml_full;      // single tile: warpgroup 1's (m, l) written
  uint64_t ml_free;      // ... and read
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  PagedSetup setup;
};

template <int D>
struct PagedGeo : Geo<D, 2> {
  using G = Geo<D, 2>;
  static constexpr int kOffXch = G::kOffBar + 1024;       // (m, l) of 128 rows
  static constexpr int kUsedPaged = kOffXch + kBM * 8;
  // (one CTA per SM, as the forward: at least 118 KB)
  static constexpr int kSmemPaged =
      (kUsedPaged + 1024 > 118 * 1024) ? kUsedPaged + 1024 : 118 * 1024;
  static_assert(kSmemPaged <= 232448, "shared memory budget");
  static_assert(sizeof(PagedBars<G::kSlots>) <= 1024, "barrier block");
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

// ------------------------------------------------------------------ the kernel
template <int D, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_kernel(const __grid_constant__ PagedParams p) {
  using G = Geo<D, 2>;
  using PG = PagedGeo<D>;
  constexpr int kSlots = G::kSlots;
  constexpr int kKStep = 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  PagedBars<kSlots> *bars = reinterpret_cast<PagedBars<kSlots> *>(smem + G::kOffBar);
  volatile int *abort_flag = &bars->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sQ = smem_u32(smem + G::kOffQ);
  const uint32_t sRing = smem_u32(smem + G::kOffRing);

  // ---- setup
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bars->q_full[t]), 1);
      mbar_init(smem_u32(&bars->q_empty[t]), 1);
      mbar_init(smem_u32(&bars->s_full[t]), 1);
      mbar_init(smem_u32(&bars->p_full[t]), kBM);
      mbar_init(smem_u32(&bars->pv_done[t]), 1);
      mbar_init(smem_u32(&bars->o_free[t]), kBM);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->v_ragged), 1);
    mbar_init(smem_u32(&bars->ml_full), kBM);
    mbar_init(smem_u32(&bars->ml_free), kBM);
    mbar_init(smem_u32(&bars->mma_done), 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (tid == kLoadWarpQ * 32) {
    prefetch_tensormap(&p.tm_q);
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  // tiles of fewer than 128 rows (a group that does not divide 128): the rows
  // behind them are never copied, so they are set once
  const int q_rows = p.tile_q * p.group;
  if (q_rows < kBM) {
    for (int i = tid; i < 2 * G::kTileBytes / 16; i += kThreads)
      reinterpret_cast<uint4 *>(smem + G::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  paged_find_piece(p, bars->setup);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  PagedWalk walk;
  walk.start(p, bars->setup);
  if (tid == 0) {
    PagedRec rec = {};
    PagedWalk w = walk;
    PagedPart part;
    if (w.next(p, part) && part.slot == 0) {
      rec.cont = 1;
      rec.ends = w.off == 0;
      rec.b = part.b;
      rec.h = part.h;
      rec.pair = part.pair;
    }
    p.rec[blockIdx.x] = rec;
  }

  if (warp >= 8) {
  regs_dec<RegSplit::kSmall>();
  if (warp == kLoadWarpQ) {
    // =================================================== Q producer
    // A tile with key blocks takes the next of the two Q slots.
    PagedPart t;
    int nq = 0;
    bool ok = true;
    const uint64_t pol = policy_evict_first();
    auto load = [&](int tok) {
      const int s = nq & 1;
      if (nq >= 2) ok = mbar_wait_warp(smem_u32(&bars->q_empty[s]), ((nq >> 1) - 1) & 1, abort_flag);
      if (!ok) return;
      const uint32_t bar = smem_u32(&bars->q_full[s]);
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, q_rows * G::kRowBytes);
#pragma unroll
        for (int bx = 0; bx < G::kNumBox; ++bx)
          tma_load_3d(sQ + s * G::kTileBytes + bx * G::kBoxBytes, &p.tm_q, bar, bx * G::kBoxCols,
                      t.h * p.group, tok, pol);
      }
      __syncwarp();
      ++nq;
    };
    while (ok && walk.next(p, t)) {
      if (t.hi0 > t.lo0) load(t.tok0);
      if (ok && t.hi1 > t.lo1) load(t.tok0 + p.tile_q);
    }
    if (!ok)   // let the copies in flight land before the CTA exits
      for (int k = max(0, nq - 2); k < nq; ++k)
        mbar_wait_slow(smem_u32(&bars->q_full[k & 1]), (k >> 1) & 1, abort_flag, false);
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
    const uint64_t pol = policy_evict_last();
    PagedPart t;
    int q = 0;             // fills so far
    int ragged = 0;        // V: ragged blocks so far
    int pend_slot = -1, pend_lo = 0, pend_hi = 0;   // V: the one not yet cleared
    bool ok = true;

    // rows [0, lo) and [hi, 128) of the ragged block := 0, then release it
    auto clear = [&]() {
      uint8_t *tile = smem + G::kOffRing + pend_slot * G::kTileBytes;
      constexpr int kUnits = G::kUnitsPerBoxRow;
#pragma unroll
      for (int bx = 0; bx < G::kNumBox; ++bx) {
        uint4 *box = reinterpret_cast<uint4 *>(tile + bx * G::kBoxBytes);
        for (int i = lane; i < pend_lo * kUnits; i += 32) box[i] = make_uint4(0, 0, 0, 0);
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
    // Wait for a free slot; a ragged block that lands meanwhile is released
    // (the slot may be freed only by what waits for it).
    auto wait_slot = [&](uint32_t bar, uint32_t parity) {
      const unsigned long long t0 = pend_slot >= 0 ? globaltimer_ns() : 0;
      while (pend_slot >= 0) {
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return;
        if (__all_sync(0xffffffffu, mbar_test(smem_u32(&bars->v_ragged), (ragged - 1) & 1))) {
          clear();
          break;
        }
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

    while (ok && walk.next(p, t)) {
      const int *row = p.table + t.b * p.table_stride;
      // page of this lane's rows of block j (-1: none), read one block ahead
      auto page_of = [&](int j) {
        const int pos = j * kBN + lane * p.box_rows;
        if (lane >= per_block || j >= t.hi || pos > t.khi || pos + p.box_rows <= t.klo) return -1;
        return __ldg(row + pos / p.page_size);
      };
      int page = page_of(t.lo);
      for (int j = t.lo; j < t.hi; ++j, ++q) {
        const int next_page = page_of(j + 1);
        const int slot = base + q % nslot;
        if (q >= nslot) {
          wait_slot(smem_u32(&bars->empty[slot]), ((q / nslot) - 1) & 1);
          if (!ok) break;
        }
        const int k0 = j * kBN;
        const bool rag = !is_k && (k0 < t.klo || k0 + kBN - 1 > t.khi);
        if (rag && pend_slot >= 0) {
          finish_ragged();
          if (!ok) break;
        }
        const uint32_t bar = smem_u32(rag ? &bars->v_ragged : &bars->full[slot]);
        if (lane == 0) mbar_arrive_expect_tx(bar, G::kTileBytes);
        __syncwarp();
        if (lane < per_block) {
          const int in_page = (k0 + lane * p.box_rows) % p.page_size;
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
    if (!ok) {
      // let the copies in flight land before the CTA exits; a ragged block's
      // copy lands on v_ragged
      if (pend_slot >= 0)
        mbar_wait_slow(smem_u32(&bars->v_ragged), (ragged - 1) & 1, abort_flag, false);
      for (int k = max(0, q - nslot); k < q; ++k)
        if (base + k % nslot != pend_slot)
          mbar_wait_slow(smem_u32(&bars->full[base + k % nslot]), (k / nslot) & 1, abort_flag,
                         false);
    }
  } else {
    // =================================================== MMA issuer
    constexpr uint32_t kIdescS = make_idesc_f16(kBM, kBN, DT, 0, 0);
    constexpr uint32_t kIdescPV = make_idesc_f16(kBM, D, DT, 0, 1);
    constexpr uint32_t kHi = desc_hi(8 * G::kSwBytes, G::kLayout);
    PagedPart t;
    bool ok = true;
    int nq = 0;                   // Q slots used so far
    int q = 0;                    // key blocks so far (K and V fills)
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
    auto issue_s = [&](int u, int qs, int slot) {
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
    };
    // O_u (+)= P_u V; the item's first product of a tile waits until the
    // epilogue has read the last item's O
    auto issue_pv = [&](int u, int slot, bool first) {
      wait(&bars->p_full[u], u ? np1 : np0);
      if (first && (u ? no1 : no0) > 0) wait(&bars->o_free[u], (u ? no1 : no0) - 1);
      if (!ok) return;
      tc_fence_after_sync();
      const uint32_t vlo = desc_lo(sRing + slot * G::kTileBytes, G::kBoxBytes);
      const uint32_t a_tmem = tmem + (u ? 128u : 0u);
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

    while (ok && walk.next(p, t)) {
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
          if (!ok) return;
          tc_fence_after_sync();
          issue_s(n & 1, qs, kslot(q0 + n));
          commit(&bars->empty[kslot(q0 + n)]);
          if (n == nb - 1) commit(&bars->q_empty[qs]);
        };
        if (ok) step_s(0);
        if (ok && nb > 1) step_s(1);
        for (int n = 0; n < nb && ok; ++n) {
          wait(&bars->full[vslot(q0 + n)], (q0 + n) / G::kSlotsV);
          if (!ok) break;
          issue_pv(n & 1, vslot(q0 + n), n < 2);
          if (!ok) break;
          commit(&bars->empty[vslot(q0 + n)]);
          if (n + 2 < nb) step_s(n + 2);
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
        wait(&bars->full[kslot(q0)], q0 / G::kSlotsK);
        for (int j = t.lo; j < t.hi && ok; ++j) {
          const int n = q0 + j - t.lo;
          tc_fence_after_sync();
          if (in0(j)) issue_s(0, qs0, kslot(n));
          if (j > t.lo) {
            if (in1(j - 1)) issue_pv(1, vslot(n - 1), j - 1 == t.lo1);
            if (!ok) break;
            commit(&bars->empty[vslot(n - 1)]);
          }
          if (in1(j)) issue_s(1, qs1, kslot(n));
          commit(&bars->empty[kslot(n)]);
          if (j == t.hi - 1) {
            if (act0) commit(&bars->q_empty[qs0]);
            if (act1) commit(&bars->q_empty[qs1]);
          }
          wait(&bars->full[vslot(n)], n / G::kSlotsV);
          if (j + 1 < t.hi) wait(&bars->full[kslot(n + 1)], (n + 1) / G::kSlotsK);
          if (!ok) break;
          if (in0(j)) issue_pv(0, vslot(n), j == t.lo0);
        }
        if (ok) {
          const int n = q0 + t.hi - 1 - t.lo;
          tc_fence_after_sync();
          if (in1(t.hi - 1)) issue_pv(1, vslot(n), t.hi - 1 == t.lo1);
          if (ok) commit(&bars->empty[vslot(n)]);
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
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + u * 128u;
    const uint32_t tO = tmem + lane_base + 256u + u * D;
    const uint32_t tO0 = tmem + lane_base + 256u;
    float2 *xch = reinterpret_cast<float2 *>(smem + PG::kOffXch);
    const float sl2 = p.scale_log2;
    const float2 sl2v = make_float2(sl2, sl2);
    PagedPart t;
    bool ok = true;
    int ns = 0;                              // S tiles taken so far
    int nx = 0;                              // (m, l) hand-overs so far

    while (ok && walk.next(p, t)) {
      const bool single = t.nt1 <= 0;
      const int tile = single ? 0 : u;       // query tile of this warpgroup
      const int nt = tile ? t.nt1 : t.nt0;
      const int first = t.first + tile * p.tile_q, last = first + nt - 1;
      const bool valid = r_tok < nt;         // (r_tok >= tile_q: rows behind the tile)
      const bool busy = __any_sync(0xffffffffu, valid);
      const int x = first + r_tok;
      const int row_lo = p.wl < 0 ? 0 : x - p.wl;
      const int row_hi = p.wr < 0 ? t.kv_len - 1 : min(t.kv_len - 1, x + p.wr);
      const int full_lo = p.wl < 0 ? 0 : last - p.wl;
      const int full_hi = p.wr < 0 ? t.kv_len - 1 : min(t.kv_len - 1, first + p.wr);
      const int j0 = single ? t.lo + u : (tile ? t.lo1 : t.lo0);
      const int jstep = single ? 2 : 1;
      const int n_blocks = single ? (t.hi - t.lo + 1 - u) / 2
                                  : (tile ? t.hi1 - t.lo1 : t.hi0 - t.lo0);

      float m_use = -INFINITY;   // reference max, log2 units of the scaled scores
      float l = 0.0f;            // normaliser relative to m_use
      for (int n = 0; n < n_blocks; ++n, ++ns) {
        const int k0 = (j0 + n * jstep) * kBN;
        ok = mbar_wait_warp(smem_u32(&bars->s_full[u]), ns & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        if (busy) {
        const bool full = k0 >= full_lo && k0 + kBN - 1 <= full_hi;
        auto load_s = [&](float (&sv)[kBN]) {
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
          if (!full) {
            const int lo_c = row_lo - k0, hi_c = row_hi - k0;
#pragma unroll
            for (int c = 0; c < kBN; ++c)
              if (c < lo_c || c > hi_c) sv[c] = -INFINITY;
          }
        };
        // max first, the conditional rescale, then P
        auto exact_pass = [&](float (&sv)[kBN]) {
          float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int c = 4; c < kBN - 4; c += 8)
#pragma unroll
            for (int v = 0; v < 4; ++v) mx[v] = fmax3(mx[v], sv[c + 2 * v], sv[c + 2 * v + 1]);
          const float m_blk = fmax3(fmax3(mx[0], mx[1], sv[kBN - 4]),
                                    fmax3(mx[2], mx[3], sv[kBN - 3]),
                                    fmaxf(sv[kBN - 2], sv[kBN - 1]));
          const float m_new = (m_blk == -INFINITY) ? -INFINITY : m_blk * sl2;
          float alpha = 1.0f;
          const bool rescale = __any_sync(0xffffffffu, m_new > m_use + kRescaleThreshold);
          if (rescale) {
            const float m_upd = fmaxf(m_use, m_new);
            alpha = (m_upd == -INFINITY) ? 1.0f : ex2(m_use - m_upd);
            m_use = m_upd;
            l *= alpha;
          }
          const float m_sub = (m_use == -INFINITY) ? 0.0f : m_use;
          const float2 negm = make_float2(-m_sub, -m_sub);
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < kBN / 2; c += 2) {
              const float2 e =
                  __ffma2_rn(make_float2(sv[half * 64 + c], sv[half * 64 + c + 1]), sl2v, negm);
              const float2 pp = make_float2(ex2(e.x), ex2(e.y));
              ls[(c >> 1) & 1] = __fadd2_rn(ls[(c >> 1) & 1], pp);
              put_p<DT>(pk, c >> 1, pp.x, pp.y);
            }
            store_p_half<DT>(tS, half, pk);
          }
          l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
          // O is complete up to the block before: S was issued after its PV
          if (rescale && n > 0) scale_o_row<D>(tO, alpha);
        };
        // unmasked block, every row has a reference: exponentials and maximum
        // side by side; redone if some row's maximum grew by more than 2^8
        if (full && __all_sync(0xffffffffu, m_use != -INFINITY)) {
          float s[kBN];
          load_s(s);
          const float2 negm = make_float2(-m_use, -m_use);
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t pk[2][32];
#pragma unroll
          for (int c = 0; c < kBN; c += 2) {
            const int pair = c >> 1;
            mx[pair & 3] = fmax3(mx[pair & 3], s[c], s[c + 1]);
            const float2 e = __ffma2_rn(make_float2(s[c], s[c + 1]), sl2v, negm);
            const float2 pp = make_float2(ex2(e.x), ex2(e.y));
            ls[pair & 1] = __fadd2_rn(ls[pair & 1], pp);
            put_p<DT>(pk[c >> 6], pair & 31, pp.x, pp.y);
          }
          const float m_new = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
          if (__any_sync(0xffffffffu, m_new > m_use + kRescaleThreshold)) {
            float s2[kBN];
            load_s(s2);
            exact_pass(s2);
          } else {
            store_p_half<DT>(tS, 0, pk[0]);
            store_p_half<DT>(tS, 1, pk[1]);
            l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
          }
        } else {
          float s[kBN];
          load_s(s);
          exact_pass(s);
        }
        tmem_wait_st();
        }
        tc_fence_before_sync();
        mbar_arrive(smem_u32(&bars->p_full[u]));
      }
      if (ok && n_blocks > 0) {
        ok = mbar_wait_warp(smem_u32(&bars->pv_done[u]), (ns - 1) & 1, abort_flag);
        tc_fence_after_sync();
      }
      if (!ok) break;

      // ---- epilogue
      float wa = 1.0f, wb = 0.0f;
      bool both = false;
      if (single) {
        // warpgroup 1 hands its (m, l) over; warpgroup 0 joins and writes
        if (u == 1) {
          if (nx > 0) ok = mbar_wait_warp(smem_u32(&bars->ml_free), (nx - 1) & 1, abort_flag);
          if (!ok) break;
          xch[r] = make_float2(m_use, l);
          tc_fence_before_sync();
          mbar_arrive(smem_u32(&bars->ml_full));
          ++nx;
          continue;
        }
        ok = mbar_wait_warp(smem_u32(&bars->ml_full), nx & 1, abort_flag);
        if (!ok) break;
        tc_fence_after_sync();
        const float2 o = xch[r];
        mbar_arrive(smem_u32(&bars->ml_free));
        ++nx;
        both = t.hi - t.lo > 1;
        const float m = fmaxf(m_use, o.x);
        wa = (m_use == -INFINITY) ? 0.0f : ex2(m_use - m);
        wb = (o.x == -INFINITY) ? 0.0f : ex2(o.x - m);
        l = wa * l + wb * o.y;
        m_use = m;
      }
      if (busy) {
        const float inv = t.slot >= 0 ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f);
        const int tok = t.tok0 + tile * p.tile_q + r_tok, head = t.h * p.group + r_head;
        const size_t wrow =
            static_cast<size_t>(2 * blockIdx.x + max(t.slot, 0)) * kPagedRows + tile * kBM + r;
        uint8_t *orow = static_cast<uint8_t *>(p.out) +
                        2 * (static_cast<long long>(tok) * p.out_st +
                             static_cast<long long>(head) * p.out_sh);
        for_o_chunks<D>([&](int c, auto wd) {
          constexpr int W = decltype(wd)::value;
          uint32_t o[W];
          if (n_blocks > 0) {
            tmem_ld_cols<W>((single ? tO0 : tO) + c, o);
            uint32_t o1[W];
            if (both) tmem_ld_cols<W>(tO0 + D + c, o1);
            tmem_wait_ld();
            reg_dep(o);
            if (both) {
              reg_dep(o1);
#pragma unroll
              for (int v = 0; v < W; ++v)
                o[v] = __float_as_uint(wa * __uint_as_float(o[v]) + wb * __uint_as_float(o1[v]));
            }
          } else {
#pragma unroll
            for (int v = 0; v < W; ++v) o[v] = 0u;
          }
          if (valid && t.slot >= 0) {
            float4 *dst = reinterpret_cast<float4 *>(p.ws_o + wrow * D + c);
#pragma unroll
            for (int v = 0; v < W / 4; ++v)
              dst[v] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                   __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
          } else if (valid) {
#pragma unroll
            for (int v = 0; v < W / 8; ++v) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<DT>(__uint_as_float(o[8 * v + 2 * e]) * inv,
                                 __uint_as_float(o[8 * v + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4 *>(orow + 2 * c + 16 * v) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();   // the next chunk's load is warp-collective
        });
        if (valid) {
          if (t.slot >= 0)
            p.ws_ml[wrow] = make_float2(l > 0.0f ? m_use : -INFINITY, l);
          else if (p.lse != nullptr)
            p.lse[static_cast<size_t>(tok) * p.H + head] =
                l > 0.0f ? (m_use + __log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
      }
      // O has been read: the next item's first PV may overwrite it
      if (n_blocks > 0) {
        tc_fence_before_sync();
        mbar_arrive(smem_u32(&bars->o_free[u]));
        if (both) mbar_arrive(smem_u32(&bars->o_free[1]));
      }
    }
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

// ------------------------------------------------------------------ the merge
// Joins the parts of an item that was cut: m = max_i m_i, w_i = 2^(m_i - m),
// O = sum_i w_i O_i / sum_i w_i l_i, lse = (m + log2 l) ln 2.  blockIdx.x: the
// CTA in whose piece the item ended.  Its parts lie in that CTA's slot 0, in
// slot 0 of every earlier CTA wholly inside the item, and in slot 1 of the CTA
// where it began; they are joined in that order, so the result does not depend
// on timing.  Few parts: a warp per row; many (one long request): the warps
// of a block share a row's parts.
constexpr int kMergeThreads = 256;
constexpr int kMergeY = 8;        // blocks per item
constexpr int kMergeAlone = 8;    // parts a warp joins by itself

template <int D, int DT>
__global__ void __launch_bounds__(kMergeThreads)
    fa_paged_merge_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kWarps = kMergeThreads / 32;
  __shared__ float4 acc_s[kWarps][32];
  __shared__ float l_s[kWarps];
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedRec rec = p.rec[c];
  if (!rec.cont || !rec.ends) return;
  // parts: CTAs c, c-1, ..., c-n+1; the walk back ends at the first CTA that
  // does not lie wholly inside the item
  int n = 1;
  for (int back = 1; back <= c; back += 32) {
    const int o = c - back - lane;
    bool inside = false;
    if (o >= 0) inside = p.rec[o].cont && !p.rec[o].ends;
    const unsigned stop = ~__ballot_sync(0xffffffffu, inside);
    if (stop) {
      n = back + __ffs(stop);
      break;
    }
  }
  const PagedReq req = paged_req(p, rec.b);
  const int i0 = rec.pair * 2 * p.tile_q;
  const int nt0 = min(p.tile_q, req.q_len - i0);
  const int nt1 = min(p.tile_q, req.q_len - i0 - nt0);
  const int rows0 = nt0 * p.group, rows = rows0 + max(nt1, 0) * p.group;

  auto slot_of = [&](int i) {   // slot of part i (0: the last)
    return static_cast<size_t>(2 * (c - i) + (i == n - 1 ? 1 : 0)) * kPagedRows;
  };
  auto one_row = [&](int k, bool shared) {
    const int tile = k >= rows0 ? 1 : 0, rr = k - tile * rows0;
    const size_t in = static_cast<size_t>(tile) * kBM + rr;
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, p.ws_ml[slot_of(i) + in].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float m_sub = m == -INFINITY ? 0.0f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
    const int from = shared ? warp : 0, step = shared ? kWarps : 1;
#pragma unroll 4
    for (int i = from; i < n; i += step) {
      const float2 ml = p.ws_ml[slot_of(i) + in];
      const float w = exp2f(ml.x - m_sub);     // a part without a visible key: 0
      l += w * ml.y;
      if (lane * 4 < D) {
        const float4 o = *reinterpret_cast<const float4 *>(p.ws_o + (slot_of(i) + in) * D + 4 * lane);
        acc.x += w * o.x;
        acc.y += w * o.y;
        acc.z += w * o.z;
        acc.w += w * o.w;
      }
    }
    if (shared) {
      acc_s[warp][lane] = acc;
      if (lane == 0) l_s[warp] = l;
      __syncthreads();
      if (warp == 0) {
        acc = acc_s[0][lane];
        l = l_s[0];
        for (int w = 1; w < kWarps; ++w) {
          const float4 o = acc_s[w][lane];
          acc.x += o.x;
          acc.y += o.y;
          acc.z += o.z;
          acc.w += o.w;
          l += l_s[w];
        }
      }
    }
    if (!shared || warp == 0) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int tok = req.q_start + i0 + tile * p.tile_q + rr / p.group;
      const int head = rec.h * p.group + rr % p.group;
      if (lane * 4 < D) {
        uint2 *dst = reinterpret_cast<uint2 *>(
            static_cast<uint8_t *>(p.out) + 2 * (static_cast<long long>(tok) * p.out_st +
                                                 static_cast<long long>(head) * p.out_sh + 4 * lane));
        *dst = make_uint2(pack2<DT>(acc.x * inv, acc.y * inv), pack2<DT>(acc.z * inv, acc.w * inv));
      }
      if (lane == 0 && p.lse != nullptr)
        p.lse[static_cast<size_t>(tok) * p.H + head] =
            l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
    if (shared) __syncthreads();
  };
  if (n <= kMergeAlone) {
    for (int k = blockIdx.y * kWarps + warp; k < rows; k += kMergeY * kWarps) one_row(k, false);
  } else {
    for (int k = blockIdx.y; k < rows; k += kMergeY) one_row(k, true);
  }
}

}  // namespace fa
