// fa_serve_host.h -- argument checks and device queries that the serving
// entries share (host code, one copy per translation unit).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fa {
namespace {

constexpr int kMaxLen = 1 << 30;

bool al(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool head_dim_ok(int D) { return D >= 16 && D <= 128 && D % 16 == 0; }

// An axis' element stride: a multiple of 8 (16 bytes) and positive, unless
// the axis has one element, whose stride does not matter.
bool stride_ok(long long n, long long s) {
  return n <= 1 || (s > 0 && s % 8 == 0 && s < (1ll << 38));
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

}  // namespace
}  // namespace fa
