// fa_paged_api.cu -- the C ABI's serving entries: fa_paged_plan,
// fa_qk_norm_rope, fa_qk_norm_rope_bwd and fa_fwd_paged (include/fa.h):
// argument checks, tensor maps, launches.  A translation unit of its own,
// with its own device status word, which fa_get_device_status() also reads.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_paged_kernel.cuh"
#include "fa_plan_kernel.cuh"
#include "fa_rope_kernel.cuh"

namespace fa {

// Reads and clears this unit's status word; negative: a CUDA call failed.
int paged_take_status() {
  unsigned int st = 0;
  if (cudaMemcpyFromSymbol(&st, g_fa_status, sizeof(st)) != cudaSuccess) return -1;
  if (st != 0) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_fa_status, &zero, sizeof(zero)) != cudaSuccess) return -1;
  }
  return st != 0 ? 1 : 0;
}

namespace {

constexpr int kMaxLen = 1 << 30;

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool al(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool head_dim_ok(int D) { return D >= 16 && D <= 128 && D % 16 == 0; }

// An axis' element stride: a multiple of 8 (16 bytes) and positive, unless
// the axis has one element, whose stride does not matter.
bool stride_ok(long long n, long long s) {
  return n <= 1 || (s > 0 && s % 8 == 0 && s < (1ll << 38));
}

// A map of 16-bit values with `rank` axes, the first contiguous; box in
// elements, the first one swizzle span wide.
bool encode(CUtensorMap *map, const void *base, int dtype, int rank, const long long *dims,
            const long long *strides, const int *box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], e[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    e[i] = 1;
    // (a one-element axis: any valid stride)
    if (i > 0) s[i - 1] = 2 * static_cast<cuuint64_t>(dims[i] > 1 ? strides[i] : dims[0]);
  }
  const int span = box[0] * 2;
  const CUtensorMapSwizzle sw = span == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                             : CU_TENSOR_MAP_SWIZZLE_32B;
  return enc(map, dtype == FA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             rank, const_cast<void *>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device (148 without one).
int sms() {
  static int count[64] = {};
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 148;
  }
  if (count[dev]) return count[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  count[dev] = n;
  return n;
}

struct PagedWs {
  size_t ml, rec, total;
};
PagedWs paged_ws(int D, int grid) {
  const size_t rows = static_cast<size_t>(2) * grid * kPagedRows;
  PagedWs w;
  w.ml = rows * D * sizeof(float);
  w.rec = w.ml + rows * sizeof(float2);
  w.total = w.rec + static_cast<size_t>(grid) * sizeof(PagedRec);
  return w;
}

template <int D, int DT>
int launch_paged(const PagedParams &prm, int grid, cudaStream_t stream) {
  auto kern = fa_paged_kernel<D, DT>;
  constexpr int smem = PagedGeo<D>::kSmemPaged;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  static bool configured[64] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64) return FA_ERR_CUDA;
    if (!configured[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess)
        return FA_ERR_CUDA;
      configured[dev] = true;
    }
  }
  kern<<<grid, kThreads, smem, stream>>>(prm);
  fa_paged_merge_kernel<D, DT><<<dim3(grid, kMergeY), kMergeThreads, 0, stream>>>(prm);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

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

RopeView view(const fa_rows &t) {
  RopeView v;
  v.ptr = static_cast<const uint8_t *>(t.ptr);
  v.sb = t.stride_b;
  v.sl = t.stride_l;
  v.sh = t.stride_h;
  return v;
}

RopeParams rope_params(const fa_rope_args *a) {
  RopeParams r;
  std::memset(&r, 0, sizeof(r));
  r.q = view(a->q);
  r.k = view(a->k);
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
  r.eps = a->eps;
  return r;
}

int rope_seg(int D) { return D > 64 ? 8 : (D > 32 ? 4 : (D > 16 ? 2 : 1)); }

template <int kSeg, int DT>
int launch_rope_fwd(const RopeParams &r, cudaStream_t stream) {
  const int rows = r.H + r.H_kv + (r.vc ? r.H_kv : 0);
  const int chunk = 32 / kSeg * kRopeUnroll;
  const long long items = static_cast<long long>(r.B) * r.L * ((rows + chunk - 1) / chunk);
  const long long blocks = (items + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 0x7fffffffll) return FA_ERR_SHAPE;
  fa_rope_fwd_kernel<kSeg, DT><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(r);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int kSeg, int DT>
int launch_rope_bwd(const RopeParams &r, cudaStream_t stream) {
  fa_rope_bwd_kernel<kSeg, DT><<<r.blocks_q + r.blocks_k, kRopeBwdThreads, 0, stream>>>(r);
  if (r.dwq || r.dwk) fa_rope_dw_kernel<<<2, 1024, 0, stream>>>(r);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

constexpr int kRopeBwdPerSm = 3;   // blocks per SM

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" int fa_paged_plan(const int *q_lens, const int *ctx_lens, int *block_table,
                             long long table_stride, const int *free_pages, int n_free, int B,
                             int max_pages, int page_size, int num_tokens, int *cu_q, int *kv_lens,
                             int *positions, long long *slots, int *counts, cudaStream_t stream) {
  if (B < 1 || n_free < 0 || max_pages < 0 || num_tokens < 0) return FA_ERR_SHAPE;
  if (page_size < 1 || page_size > kMaxLen || table_stride < max_pages) return FA_ERR_ARG;
  if (!q_lens || !ctx_lens || !cu_q || !kv_lens || !counts || (max_pages > 0 && !block_table) ||
      (n_free > 0 && !free_pages) || (num_tokens > 0 && (!positions || !slots)))
    return FA_ERR_NULL;
  if (!al(q_lens, 4) || !al(ctx_lens, 4) || !al(block_table, 4) || !al(free_pages, 4) ||
      !al(cu_q, 4) || !al(kv_lens, 4) || !al(positions, 4) || !al(slots, 8) || !al(counts, 4))
    return FA_ERR_ALIGN;
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
  r.qo = view(a->q_out);
  r.ko = view(a->k_out);
  if (cache) {
    r.v = view(a->v);
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
  return static_cast<size_t>(sms()) * kRopeBwdPerSm * D * sizeof(float);
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
  r.dyq = view(a->q_out);
  r.dyk = view(a->k_out);
  r.dq = view(dq);
  r.dk = view(dk);
  r.dwq = dq_weight;
  r.dwk = dk_weight;
  if (dq_weight || dk_weight) {
    if (!workspace) return FA_ERR_NULL;
    if (!al(workspace, 256)) return FA_ERR_ALIGN;
    if (workspace_bytes < fa_qk_norm_rope_bwd_workspace_bytes(a->D)) return FA_ERR_WORKSPACE;
    r.part = static_cast<float *>(workspace);
  }
  // blocks in proportion to the rows of each kind, at least one where there
  // are rows
  const int all = sms() * kRopeBwdPerSm;
  r.blocks_k = a->H_kv == 0 ? 0
                            : std::max(1, static_cast<int>(static_cast<long long>(all) * a->H_kv /
                                                           (a->H + a->H_kv)));
  r.blocks_q = all - r.blocks_k;
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

extern "C" size_t fa_paged_workspace_bytes(int D) {
  return head_dim_ok(D) ? paged_ws(D, sms()).total : 0;
}

extern "C" int fa_fwd_paged(const void *q, long long q_stride_t, long long q_stride_h,
                            const void *k_cache, const void *v_cache, long long cache_stride_page,
                            long long cache_stride_token, long long cache_stride_head,
                            const int *block_table, long long table_stride, const int *cu_q,
                            const int *kv_lens, void *out, long long out_stride_t,
                            long long out_stride_h, float *lse, int total_q, int B, int H, int H_kv,
                            int D, int num_pages, int page_size, int max_pages, float scale,
                            int causal, int window_left, int window_right, int dtype,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  // ---------------------------------------------------------------- checks
  if (total_q < 0 || B < 1 || H < 1 || H_kv < 1 || num_pages < 1 || max_pages < 1)
    return FA_ERR_SHAPE;
  if (H % H_kv != 0 || H / H_kv > kBM) return FA_ERR_SHAPE;
  if (total_q > kMaxLen || static_cast<long long>(B) * H_kv > kMaxLen) return FA_ERR_SHAPE;
  if (!head_dim_ok(D)) return FA_ERR_HEADDIM;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (page_size < 16 || page_size > kMaxLen ||
      (page_size < kBN ? kBN % page_size != 0 : page_size % kBN != 0))
    return FA_ERR_ARG;
  if (!std::isfinite(scale) || scale < 0.0f || table_stride < max_pages) return FA_ERR_ARG;
  if (total_q == 0) return FA_OK;
  if (!q || !k_cache || !v_cache || !block_table || !cu_q || !kv_lens || !out || !workspace)
    return FA_ERR_NULL;
  if (!al(q, 16) || !al(k_cache, 16) || !al(v_cache, 16) || !al(out, 16) || !al(lse, 4) ||
      !al(block_table, 4) || !al(cu_q, 4) || !al(kv_lens, 4) || !al(workspace, 256))
    return FA_ERR_ALIGN;
  if (!stride_ok(total_q, q_stride_t) || !stride_ok(H, q_stride_h) ||
      !stride_ok(total_q, out_stride_t) || !stride_ok(H, out_stride_h) ||
      !stride_ok(num_pages, cache_stride_page) || !stride_ok(page_size, cache_stride_token) ||
      !stride_ok(H_kv, cache_stride_head))
    return FA_ERR_ALIGN;
  const int grid = sms();
  const PagedWs ws = paged_ws(D, grid);
  if (workspace_bytes < ws.total) return FA_ERR_WORKSPACE;

  // ---------------------------------------------------------------- params
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  p.table = block_table;
  p.table_stride = table_stride;
  p.cu_q = cu_q;
  p.kv_lens = kv_lens;
  p.out = out;
  p.out_st = out_stride_t;
  p.out_sh = out_stride_h;
  p.lse = lse;
  p.B = B;
  p.H = H;
  p.H_kv = H_kv;
  p.group = H / H_kv;
  p.total_q = total_q;
  p.tile_q = kBM / p.group;
  p.n_pages = num_pages;
  p.page_size = page_size;
  p.max_kv = static_cast<int>(std::min<long long>(static_cast<long long>(max_pages) * page_size, kMaxLen));
  p.box_rows = std::min(page_size, kBN);
  // (a bound past the longest request is no bound)
  p.wl = window_left < 0 || window_left >= kMaxLen ? -1 : window_left;
  p.wr = window_right < 0 || window_right >= kMaxLen ? -1 : window_right;
  if (causal) p.wr = 0;
  const float sl2 = scale * 1.4426950408889634f;
  p.scale_log2 = sl2 < 1e-30f ? 1e-30f : sl2;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + ws.ml);
  p.rec = reinterpret_cast<PagedRec *>(static_cast<char *>(workspace) + ws.rec);
  const int row_bytes = D * 2;
  const int cols = (row_bytes % 128 == 0 ? 128 : (row_bytes % 64 == 0 ? 64 : 32)) / 2;
  const long long qd[3] = {D, H, total_q}, qs[3] = {1, q_stride_h, q_stride_t};
  const int qb[3] = {cols, p.group, p.tile_q};
  const long long cd[4] = {D, page_size, H_kv, num_pages};
  const long long cs[4] = {1, cache_stride_token, cache_stride_head, cache_stride_page};
  const int cb[4] = {cols, p.box_rows, 1, 1};
  if (!encode(&p.tm_q, q, dtype, 3, qd, qs, qb) || !encode(&p.tm_k, k_cache, dtype, 4, cd, cs, cb) ||
      !encode(&p.tm_v, v_cache, dtype, 4, cd, cs, cb))
    return FA_ERR_CUDA;
  switch (D * 2 + dtype) {
    case 32: return launch_paged<16, 0>(p, grid, stream);
    case 33: return launch_paged<16, 1>(p, grid, stream);
    case 64: return launch_paged<32, 0>(p, grid, stream);
    case 65: return launch_paged<32, 1>(p, grid, stream);
    case 96: return launch_paged<48, 0>(p, grid, stream);
    case 97: return launch_paged<48, 1>(p, grid, stream);
    case 128: return launch_paged<64, 0>(p, grid, stream);
    case 129: return launch_paged<64, 1>(p, grid, stream);
    case 160: return launch_paged<80, 0>(p, grid, stream);
    case 161: return launch_paged<80, 1>(p, grid, stream);
    case 192: return launch_paged<96, 0>(p, grid, stream);
    case 193: return launch_paged<96, 1>(p, grid, stream);
    case 224: return launch_paged<112, 0>(p, grid, stream);
    case 225: return launch_paged<112, 1>(p, grid, stream);
    case 256: return launch_paged<128, 0>(p, grid, stream);
    case 257: return launch_paged<128, 1>(p, grid, stream);
  }
  return FA_ERR_HEADDIM;
}
