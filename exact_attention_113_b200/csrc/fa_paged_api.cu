// fa_paged_api.cu -- fa_fwd_paged of the C ABI (include/fa.h): argument
// checks, tensor maps, launches.  A translation unit of its own, with its own
// device status word, which fa_get_device_status() also reads.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_paged_kernel.cuh"
#include "fa_serve_host.h"

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

#ifdef FA_TEST_HOOKS
bool paged_set_withhold(int block) {
  return cudaMemcpyToSymbol(g_fa_test_withhold_block, &block, sizeof(int)) == cudaSuccess;
}
#endif

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// So that a walk over requests without new tokens ends within the waits' limit.
constexpr int kMaxRequests = 1 << 24;

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
  // Fetches of 256 bytes where that many neighbours are read together: rows of
  // 256 bytes or adjacent ones.  A shorter row between other heads' rows would
  // bring their bytes too (decoding 32 requests over 4k, 16 K/V heads of D 64:
  // 88 us with 256, 77 with 128; 64 over 8k, D 128: 336 with 256, 350 with 128).
  const bool wide = 2 * dims[0] >= 256 || (rank > 1 && strides[1] == dims[0]);
  const CUtensorMapL2promotion promote =
      wide ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  return enc(map, dtype == FA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             rank, const_cast<void *>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct PagedWs {
  size_t ml, ticket, total;
};
PagedWs paged_ws(int D, int grid) {
  const size_t rows = static_cast<size_t>(2) * grid * kPagedRows;
  PagedWs w;
  w.ml = rows * D * sizeof(float);
  w.ticket = w.ml + rows * sizeof(float2);
  w.total = w.ticket + static_cast<size_t>(grid) * sizeof(unsigned long long);
  return w;
}

// A number for each call: 48 bits, not 0, from a start that differs between
// processes, so that what a workspace held before does not pass for it.
unsigned long long call_number() {
  static std::atomic<unsigned long long> next{
      static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) *
      0x9e3779b97f4a7c15ull};
  const unsigned long long n = next.fetch_add(1) & 0xffffffffffffull;
  return n ? n : next.fetch_add(1) & 0xffffffffffffull;
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
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

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
  if (total_q > kMaxLen || B > kMaxRequests || static_cast<long long>(B) * H_kv > kMaxLen)
    return FA_ERR_SHAPE;
  if (!head_dim_ok(D)) return FA_ERR_HEADDIM;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (page_size < 16 || page_size > kMaxLen || (page_size & (page_size - 1)) != 0)
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
  p.out_wide = al(out, 32) && (total_q <= 1 || out_stride_t % 16 == 0) &&
               (H <= 1 || out_stride_h % 16 == 0);
  p.lse = lse;
  p.B = B;
  p.H = H;
  p.H_kv = H_kv;
  p.group = H / H_kv;
  p.total_q = total_q;
  p.tile_q = kBM / p.group;
  p.n_pages = num_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
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
  p.ticket =
      reinterpret_cast<unsigned long long *>(static_cast<char *>(workspace) + ws.ticket);
  p.call = call_number();
  const int row_bytes = D * 2;
  const int cols = (row_bytes % 128 == 0 ? 128 : (row_bytes % 64 == 0 ? 64 : 32)) / 2;
  const long long qd[3] = {D, H, total_q}, qs[3] = {1, q_stride_h, q_stride_t};
  const int qb[3] = {cols, p.group, p.tile_q};
  const long long cd[4] = {D, page_size, H_kv, num_pages};
  const long long cs[4] = {1, cache_stride_token, cache_stride_head, cache_stride_page};
  const int cb[4] = {cols, p.box_rows, 1, 1};
  const int qb1[3] = {cols, p.group, 1};
  if (!encode(&p.tm_q, q, dtype, 3, qd, qs, qb) || !encode(&p.tm_q1, q, dtype, 3, qd, qs, qb1) ||
      !encode(&p.tm_k, k_cache, dtype, 4, cd, cs, cb) ||
      !encode(&p.tm_v, v_cache, dtype, 4, cd, cs, cb))
    return FA_ERR_CUDA;
  switch (D * 2 + dtype) {
#ifdef FA_TEST_HOOKS   // the watchdog test library: fp16 head dims 64 and 128 only
    case 128: return launch_paged<64, 0>(p, grid, stream);
    case 256: return launch_paged<128, 0>(p, grid, stream);
#else
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
#endif
  }
  return FA_ERR_HEADDIM;
}
