// fa_serve_api.cu -- fa_paged_plan, fa_qk_norm_rope and fa_qk_norm_rope_bwd of
// the C ABI (include/fa.h): argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>

#include <cuda_runtime.h>

#include "fa.h"
#include "fa_plan_kernel.cuh"
#include "fa_rope_kernel.cuh"
#include "fa_serve_host.h"

namespace fa {
namespace {

// Query and key arguments that both directions of the norm share.
int rope_check(const fa_rope_args *a) {
  if (a->B < 1 || a->L < 0 || a->H < 1 || a->H_kv < 0) return FA_ERR_SHAPE;
  if (a->L > kMaxLen || a->H > (1 << 20) || a->H_kv > (1 << 20)) return FA_ERR_SHAPE;
  if (static_cast<long long>(a->B) * a->L > kMaxLen) return FA_ERR_SHAPE;
  if (!head_dim_ok(a->D)) return FA_ERR_HEADDIM;
  if (a->dtype != FA_F16 && a->dtype != FA_BF16) return FA_ERR_DTYPE;
  if (a->rot_dim < 0 || a->rot_dim > a->D || a->rot_dim % 16 != 0 || a->max_pos < 0)
    return FA_ERR_ARG;
  if (!std::isfinite(a->eps) || a->eps < 0.0f) return FA_ERR_ARG;
  if (a->positions_64 != 0 && a->positions_64 != 1) return FA_ERR_ARG;
  return FA_OK;
}

// A tensor of `heads` heads a token: pointer and strides.
int rope_tensor(const fa_rope_args *a, const fa_rows &t, int heads, bool needed) {
  if (heads == 0 || a->L == 0) return FA_OK;
  if (!t.ptr) return needed ? FA_ERR_NULL : FA_OK;
  if (!al(t.ptr, 16)) return FA_ERR_ALIGN;
  if (!stride_ok(a->B, t.stride_b) || !stride_ok(a->L, t.stride_l) || !stride_ok(heads, t.stride_h))
    return FA_ERR_ALIGN;
  return FA_OK;
}

// A tensor as the kernels walk it.  The stride of a one-element axis may be any
// number; lanes behind the last head form addresses with it, which a copy of no
// bytes wants aligned too, so it becomes 0.
RopeView view(const fa_rope_args *a, const fa_rows &t, int heads) {
  RopeView v;
  v.ptr = static_cast<const uint8_t *>(t.ptr);
  v.sb = a->B > 1 ? t.stride_b : 0;
  v.sl = a->L > 1 ? t.stride_l : 0;
  v.sh = heads > 1 ? t.stride_h : 0;
  return v;
}

RopeParams rope_params(const fa_rope_args *a) {
  RopeParams r;
  std::memset(&r, 0, sizeof(r));
  r.q = view(a, a->q, a->H);
  r.k = view(a, a->k, a->H_kv);
  r.wq = a->q_weight;
  r.wk = a->k_weight;
  r.cos_sin = a->cos_sin;
  r.pos = a->positions;
  r.pos64 = a->positions_64;
  r.pos_sb = a->positions_stride_b;
  r.pos_sl = a->positions_stride_l;
  r.B = a->B;
  r.L = a->L;
  r.H = a->H;
  r.H_kv = a->H_kv;
  r.D = a->D;
  r.rot = a->rot_dim;
  r.max_pos = a->max_pos;
  r.interleaved = a->interleaved != 0;
  // At least the smallest normal number: without it a row of zeros, and the lanes
  // of a step behind the last head, which hold zeros and are in the weights' sums,
  // would be 0 times infinity.  It is lost beside any mean square of 2^-102 or more.
  r.eps = std::max(a->eps, std::numeric_limits<float>::min());
  r.inv_d = 1.0f / a->D;
  return r;
}

int rope_seg(int D) { return D > 64 ? 8 : (D > 32 ? 4 : (D > 16 ? 2 : 1)); }

// Deals up to `blocks` blocks to three kinds of rows (query, key, value), of
// which a token has the given numbers of steps: at least one to a kind that has
// rows and no more than have a step for each warp.  A token's fixed work
// (addresses, angles, slot) is about that of a step, so a kind's share goes by
// its steps + 1 (the gradient at B2 L16384 H32/8 D128: 183 us, by its steps 200).
void rope_deal(long long tokens, int blocks, const int (&steps)[3], int (&out)[3]) {
  constexpr int kWarps = kRopeThreads / 32;
  long long all = 0;
  for (int i = 0; i < 3; ++i) all += steps[i] ? steps[i] + 1 : 0;
  for (int i = 2; i >= 0; --i) {
    const long long most = (tokens * steps[i] + kWarps - 1) / kWarps;
    const long long part = i == 0 ? blocks - out[1] - out[2] : blocks * (steps[i] + 1ll) / all;
    out[i] = static_cast<int>(std::min(std::max(part, 1ll), most));
  }
}

// Chunks of a token's steps: whole tokens where a warp gets 4 of them, else
// fewer steps, so that no warp has much more than its share.
void rope_cut(long long tokens, int steps, int blocks, int &chunks, int &per) {
  steps = std::max(steps, 1);
  const long long fit = tokens * steps / (4ll * (kRopeThreads / 32) * std::max(blocks, 1));
  const int most = static_cast<int>(std::min<long long>(std::max(fit, 1ll), steps));
  chunks = (steps + most - 1) / most;
  per = (steps + chunks - 1) / chunks;
  chunks = (steps + per - 1) / per;
}

// Bytes of an array, and whether two arrays share some.
struct Span {
  uintptr_t at, end;
};
Span span(const void *p, long long n, int size) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(n) * size};
}
bool meet(const Span &a, const Span &b) { return a.at < b.end && b.at < a.end; }

constexpr long long kRopeMostSteps = 0x7fffffffll;   // 32-bit indexes walk them

template <int kSeg, int DT>
int launch_rope_fwd(RopeParams &r, cudaStream_t stream) {
  constexpr int kRows = 32 / kSeg;
  const long long tokens = static_cast<long long>(r.B) * r.L;
  const int kv = (r.H_kv + kRows - 1) / kRows;
  const int steps[3] = {(r.H + kRows - 1) / kRows, kv, r.vc ? kv : 0};
  if (tokens * std::max(steps[0], kv) > kRopeMostSteps) return FA_ERR_SHAPE;
  int blocks[3];
  rope_deal(tokens, sms() * kRopeBlocks, steps, blocks);
  r.blocks_q = blocks[0];
  r.blocks_k = blocks[1];
  rope_cut(tokens, steps[0], blocks[0], r.chunks_q, r.per_q);
  rope_cut(tokens, steps[1], blocks[1], r.chunks_k, r.per_k);
  const unsigned grid = blocks[0] + blocks[1] + blocks[2];
  if (r.interleaved)
    fa_rope_fwd_kernel<kSeg, DT, true><<<grid, kRopeThreads, 0, stream>>>(r);
  else
    fa_rope_fwd_kernel<kSeg, DT, false><<<grid, kRopeThreads, 0, stream>>>(r);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int kSeg, int DT>
int launch_rope_bwd(RopeParams &r, cudaStream_t stream) {
  constexpr int kRows = 32 / kSeg;
  const long long tokens = static_cast<long long>(r.B) * r.L;
  const int steps[3] = {(r.H + kRows - 1) / kRows, (r.H_kv + kRows - 1) / kRows, 0};
  if (tokens * std::max(steps[0], steps[1]) > kRopeMostSteps) return FA_ERR_SHAPE;
  int blocks[3];
  rope_deal(tokens, sms() * kRopeBwdBlocks, steps, blocks);
  r.blocks_q = blocks[0];
  r.blocks_k = blocks[1];
  if (r.interleaved)
    fa_rope_bwd_kernel<kSeg, DT, true><<<blocks[0] + blocks[1], kRopeThreads, 0, stream>>>(r);
  else
    fa_rope_bwd_kernel<kSeg, DT, false><<<blocks[0] + blocks[1], kRopeThreads, 0, stream>>>(r);
  if (r.dwq || r.dwk) fa_rope_dw_kernel<<<dim3(2, (r.D + 31) / 32), 1024, 0, stream>>>(r);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" int fa_paged_plan(const int *q_lens, const int *ctx_lens, int *block_table,
                             long long table_stride, const int *free_pages, int n_free, int B,
                             int max_pages, int page_size, int num_tokens, int *cu_q, int *kv_lens,
                             int *positions, long long *slots, int *counts, cudaStream_t stream) {
  if (B < 1 || B > kMaxLen || n_free < 0 || max_pages < 0 || num_tokens < 0) return FA_ERR_SHAPE;
  if (page_size < 1 || page_size > kMaxLen || table_stride < max_pages) return FA_ERR_ARG;
  if (!q_lens || !ctx_lens || !cu_q || !kv_lens || !counts || (max_pages > 0 && !block_table) ||
      (n_free > 0 && !free_pages) || (num_tokens > 0 && (!positions || !slots)))
    return FA_ERR_NULL;
  if (!al(q_lens, 4) || !al(ctx_lens, 4) || !al(block_table, 4) || !al(free_pages, 4) ||
      !al(cu_q, 4) || !al(kv_lens, 4) || !al(positions, 4) || !al(slots, 8) || !al(counts, 4))
    return FA_ERR_ALIGN;
  {
    // every block reads all lengths while others write: what is written has
    // to lie apart (kv_lens on the next step's ctx_lens, for one, would not do)
    const long long rows = (B - 1) * table_stride + max_pages;
    const Span in[3] = {span(q_lens, B, 4), span(ctx_lens, B, 4), span(free_pages, n_free, 4)};
    const Span out[6] = {span(block_table, max_pages ? rows : 0, 4), span(cu_q, B + 1ll, 4),
                         span(kv_lens, B, 4), span(positions, num_tokens, 4),
                         span(slots, num_tokens, 8), span(counts, 3, 4)};
    for (int i = 0; i < 6; ++i) {
      for (const Span &x : in)
        if (meet(out[i], x)) return FA_ERR_ARG;
      for (int j = 0; j < i; ++j)
        if (meet(out[i], out[j])) return FA_ERR_ARG;
    }
  }
  PlanParams p;
  p.q_lens = q_lens;
  p.ctx_lens = ctx_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.B = B;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.num_tokens = num_tokens;
  p.cu_q = cu_q;
  p.kv_lens = kv_lens;
  p.positions = positions;
  p.slots = slots;
  p.counts = counts;
  const unsigned grid =
      static_cast<unsigned>(std::max<long long>(1, (num_tokens + kPlanTokens - 1ll) / kPlanTokens));
  fa_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_qk_norm_rope(const fa_rope_args *a, cudaStream_t stream) {
  if (!a) return FA_ERR_NULL;
  int st = rope_check(a);
  if (st != FA_OK) return st;
  const bool cache = a->k_cache != nullptr || a->v_cache != nullptr;
  if ((st = rope_tensor(a, a->q, a->H, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, a->q_out, a->H, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, a->k, a->H_kv, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, a->k_out, a->H_kv, !cache)) != FA_OK) return st;
  if (cache) {
    if (!a->k_cache || !a->v_cache) return FA_ERR_NULL;
    if ((st = rope_tensor(a, a->v, a->H_kv, true)) != FA_OK) return st;
    if (a->L > 0 && !a->slots) return FA_ERR_NULL;
    if (a->num_pages < 1 || a->page_size < 1) return FA_ERR_ARG;
    if (!al(a->k_cache, 16) || !al(a->v_cache, 16) || !al(a->slots, 8) ||
        !stride_ok(a->num_pages, a->cache_stride_page) ||
        !stride_ok(a->page_size, a->cache_stride_token) ||
        !stride_ok(a->H_kv, a->cache_stride_head))
      return FA_ERR_ALIGN;
  }
  if (a->L == 0) return FA_OK;
  if (!a->positions || (a->rot_dim > 0 && a->max_pos > 0 && !a->cos_sin)) return FA_ERR_NULL;
  if (!al(a->positions, a->positions_64 ? 8 : 4) || !al(a->cos_sin, 16) || !al(a->q_weight, 16) ||
      !al(a->k_weight, 16))
    return FA_ERR_ALIGN;
  RopeParams r = rope_params(a);
  r.qo = view(a, a->q_out, a->H);
  r.ko = view(a, a->k_out, a->H_kv);
  if (cache) {
    r.v = view(a, a->v, a->H_kv);
    r.kc = static_cast<uint8_t *>(a->k_cache);
    r.vc = static_cast<uint8_t *>(a->v_cache);
    r.c_sp = a->cache_stride_page;
    r.c_st = a->cache_stride_token;
    r.c_sh = a->cache_stride_head;
    r.slots = a->slots;
    r.page_size = a->page_size;
    r.n_slots = static_cast<long long>(a->num_pages) * a->page_size;
  }
  switch (rope_seg(r.D) * 2 + a->dtype) {
    case 2: return launch_rope_fwd<1, 0>(r, stream);
    case 3: return launch_rope_fwd<1, 1>(r, stream);
    case 4: return launch_rope_fwd<2, 0>(r, stream);
    case 5: return launch_rope_fwd<2, 1>(r, stream);
    case 8: return launch_rope_fwd<4, 0>(r, stream);
    case 9: return launch_rope_fwd<4, 1>(r, stream);
    case 16: return launch_rope_fwd<8, 0>(r, stream);
    case 17: return launch_rope_fwd<8, 1>(r, stream);
  }
  return FA_ERR_HEADDIM;
}

extern "C" size_t fa_qk_norm_rope_bwd_workspace_bytes(int D) {
  if (!head_dim_ok(D)) return 0;
  // (one block more than the grid's: each kind of rows gets at least one)
  return (static_cast<size_t>(sms()) * kRopeBwdBlocks + 1) * D * sizeof(float);
}

extern "C" int fa_qk_norm_rope_bwd(const fa_rope_args *a, fa_rows dq, fa_rows dk, float *dq_weight,
                                   float *dk_weight, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  if (!a) return FA_ERR_NULL;
  int st = rope_check(a);
  if (st != FA_OK) return st;
  if ((st = rope_tensor(a, a->q, a->H, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, a->q_out, a->H, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, dq, a->H, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, a->k, a->H_kv, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, a->k_out, a->H_kv, true)) != FA_OK) return st;
  if ((st = rope_tensor(a, dk, a->H_kv, true)) != FA_OK) return st;
  if (!al(dq_weight, 4) || !al(dk_weight, 4)) return FA_ERR_ALIGN;
  if ((a->q_weight != nullptr) != (dq_weight != nullptr) ||
      (a->k_weight != nullptr) != (dk_weight != nullptr))
    return FA_ERR_NULL;
  if (a->L == 0) {
    if (dq_weight && cudaMemsetAsync(dq_weight, 0, a->D * sizeof(float), stream) != cudaSuccess)
      return FA_ERR_CUDA;
    if (dk_weight && cudaMemsetAsync(dk_weight, 0, a->D * sizeof(float), stream) != cudaSuccess)
      return FA_ERR_CUDA;
    return FA_OK;
  }
  if (!a->positions || (a->rot_dim > 0 && a->max_pos > 0 && !a->cos_sin)) return FA_ERR_NULL;
  if (!al(a->positions, a->positions_64 ? 8 : 4) || !al(a->cos_sin, 16) || !al(a->q_weight, 16) ||
      !al(a->k_weight, 16))
    return FA_ERR_ALIGN;
  RopeParams r = rope_params(a);
  r.dyq = view(a, a->q_out, a->H);
  r.dyk = view(a, a->k_out, a->H_kv);
  r.dq = view(a, dq, a->H);
  r.dk = view(a, dk, a->H_kv);
  r.dwq = dq_weight;
  r.dwk = dk_weight;
  if (dq_weight || dk_weight) {
    if (!workspace) return FA_ERR_NULL;
    if (!al(workspace, 256)) return FA_ERR_ALIGN;
    if (workspace_bytes < fa_qk_norm_rope_bwd_workspace_bytes(a->D)) return FA_ERR_WORKSPACE;
    r.part = static_cast<float *>(workspace);
  }
  switch (rope_seg(r.D) * 2 + a->dtype) {
    case 2: return launch_rope_bwd<1, 0>(r, stream);
    case 3: return launch_rope_bwd<1, 1>(r, stream);
    case 4: return launch_rope_bwd<2, 0>(r, stream);
    case 5: return launch_rope_bwd<2, 1>(r, stream);
    case 8: return launch_rope_bwd<4, 0>(r, stream);
    case 9: return launch_rope_bwd<4, 1>(r, stream);
    case 16: return launch_rope_bwd<8, 0>(r, stream);
    case 17: return launch_rope_bwd<8, 1>(r, stream);
  }
  return FA_ERR_HEADDIM;
}
