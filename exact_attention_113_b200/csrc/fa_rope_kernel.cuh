// fa_rope_kernel.cuh -- RMS norm of every query and key head and the rotary
// position rotation in one pass, and its gradient.
//
//   y = R_pos(w .* x r),  r = (mean(x^2) + eps)^(-1/2)
// R turns the pairs (a, b) of a head's first `rot` values by its position's
// angles: (a cos - b sin, b cos + a sin); the pairs are (i, i + rot/2), or
// (2i, 2i + 1) when interleaved.  The gradient, with g = R^T dy:
//   dw = sum over rows of g .* x r,
//   dx = r (w .* g - x r mean(w .* g .* x r)).
//
// Both read and write every value once and do some ten operations on it: HBM
// bounds them.  A row (one head of one token) belongs to D / 16 lanes, each
// with two 16-byte vectors that hold whole pairs (8 values from each half, or
// 16 neighbours), so the rotation needs no exchange and only the norm's sum
// crosses lanes.  A warp takes one token's rows, kUnroll per lane with all
// their loads issued first, and reads its cosines and weights once for them.
// All arithmetic is fp32; the result is rounded once.
#pragma once

#include "sm100.cuh"

namespace fa {

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;
constexpr int kRopeBwdThreads = 256;

struct RopeView {
  const uint8_t *ptr;
  long long sb, sl, sh;   // strides in elements of batch, token, head
};

struct RopeParams {
  RopeView q, k, v;       // inputs
  RopeView qo, ko;        // outputs (ptr nullptr: not written)
  const void *wq, *wk;    // nullptr: no norm
  const float *cos_sin;   // [max_pos][rot]: rot/2 cosines, rot/2 sines
  const void *pos;        // int32 or int64
  int pos64;
  long long pos_sb, pos_sl;
  uint8_t *kc, *vc;       // paged caches or nullptr
  long long c_sp, c_st, c_sh;
  const long long *slots;
  long long n_slots;
  int page_size;
  int B, L, H, H_kv, D, rot, max_pos, interleaved;
  float eps;
  // backward
  RopeView dyq, dyk;      // gradients of the outputs
  RopeView dq, dk;        // written
  float *part;            // [blocks][D] partial weight gradients
  float *dwq, *dwk;       // [D]
  int blocks_q, blocks_k;
};

// This lane's place in a row of D values: two vectors of 8 and whether they
// are rotated; `i0` is the first of its 8 angles.
struct RopeLane {
  int a, b, i0;
  bool on, turn;
};
__device__ __forceinline__ RopeLane rope_lane(int s, int D, int rot, int interleaved) {
  RopeLane o;
  o.on = s < D / 16;
  o.turn = s < rot / 16;
  o.i0 = 8 * s;
  if (o.turn && !interleaved) {
    o.a = 8 * s;
    o.b = rot / 2 + 8 * s;
  } else {
    o.a = 16 * s;
    o.b = 16 * s + 8;
  }
  return o;
}

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (DT == 0)
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}

template <int DT>
__device__ __forceinline__ void unpack16(const uint4 &a, const uint4 &b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack2<DT>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <int DT>
__device__ __forceinline__ void pack16(const float (&x)[16], uint4 &a, uint4 &b) {
  a = make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]),
                 pack2<DT>(x[6], x[7]));
  b = make_uint4(pack2<DT>(x[8], x[9]), pack2<DT>(x[10], x[11]), pack2<DT>(x[12], x[13]),
                 pack2<DT>(x[14], x[15]));
}

// The lane's 8 pairs turned by +angle (kSign 1) or -angle (kSign -1).
template <int kSign>
__device__ __forceinline__ void turn16(float (&x)[16], const float (&c)[8], const float (&s)[8],
                                       int interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float si = kSign * s[i];
    if (interleaved) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * si;
      x[2 * i + 1] = b * c[i] + a * si;
    } else {
      const float a = x[i], b = x[8 + i];
      x[i] = a * c[i] - b * si;
      x[8 + i] = b * c[i] + a * si;
    }
  }
}

template <int kSeg>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int d = kSeg / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ long long rope_position(const RopeParams &p, int b, int l) {
  const long long at = b * p.pos_sb + l * p.pos_sl;
  return p.pos64 ? __ldg(static_cast<const long long *>(p.pos) + at)
                 : static_cast<long long>(__ldg(static_cast<const int *>(p.pos) + at));
}

__device__ __forceinline__ void rope_angles(const RopeParams &p, long long pos, const RopeLane &w,
                                            float (&c)[8], float (&s)[8]) {
  if (w.turn) {
    const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + pos * p.rot + w.i0);
    const float4 c0 = __ldg(row), c1 = __ldg(row + 1);
    const float4 *rs = reinterpret_cast<const float4 *>(p.cos_sin + pos * p.rot + p.rot / 2 + w.i0);
    const float4 s0 = __ldg(rs), s1 = __ldg(rs + 1);
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
    c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
    s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
  }
}

__device__ __forceinline__ uint4 ld16(const uint8_t *base, long long elem) {
  return *reinterpret_cast<const uint4 *>(base + 2 * elem);
}
__device__ __forceinline__ void st16(const uint8_t *base, long long elem, const uint4 &v) {
  *reinterpret_cast<uint4 *>(const_cast<uint8_t *>(base) + 2 * elem) = v;
}

// kSeg lanes a row: the smallest power of two >= D / 16.  Rows of a token:
// H query heads, H_kv key heads and, for the cache, H_kv value heads (copied).
template <int kSeg, int DT>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kRowsWarp = 32 / kSeg;
  constexpr int kChunk = kRowsWarp * kRopeUnroll;   // rows a warp takes
  const int lane = threadIdx.x & 31;
  const int rows = p.H + p.H_kv + (p.vc ? p.H_kv : 0);
  const int chunks = (rows + kChunk - 1) / kChunk;
  const long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.B) * p.L * chunks) return;
  const long long token = item / chunks;
  const int row0 = static_cast<int>(item - token * chunks) * kChunk + lane / kSeg;
  const int b = static_cast<int>(token / p.L), l = static_cast<int>(token - static_cast<long long>(b) * p.L);
  const RopeLane w = rope_lane(lane % kSeg, p.D, p.rot, p.interleaved);

  // all loads of the lane first
  uint4 xa[kRopeUnroll], xb[kRopeUnroll];
#pragma unroll
  for (int i = 0; i < kRopeUnroll; ++i) {
    const int row = row0 + i * kRowsWarp;
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (w.on && row < rows) {
      const RopeView &in = row < p.H ? p.q : (row < p.H + p.H_kv ? p.k : p.v);
      const int h = row < p.H ? row : (row < p.H + p.H_kv ? row - p.H : row - p.H - p.H_kv);
      const long long at = b * in.sb + l * in.sl + h * in.sh;
      // (value heads are copied: neighbouring vectors, whatever the pairs are)
      const bool copy = row >= p.H + p.H_kv;
      const int s = lane % kSeg;
      xa[i] = ld16(in.ptr, at + (copy ? 16 * s : w.a));
      xb[i] = ld16(in.ptr, at + (copy ? 16 * s + 8 : w.b));
    }
  }
  const long long pos = rope_position(p, b, l);
  if (pos < 0 || pos >= p.max_pos) return;   // padding: left as it was
  long long cache = -1;
  if (p.kc) {
    const long long slot = __ldg(p.slots + token);
    if (slot >= 0 && slot < p.n_slots)
      cache = slot / p.page_size * p.c_sp + slot % p.page_size * p.c_st;
  }
  float c[8], s[8];
  rope_angles(p, pos, w, c, s);
  uint4 wqa = make_uint4(0, 0, 0, 0), wqb = wqa, wka = wqa, wkb = wqa;
  if (w.on && p.wq) {
    wqa = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.wq) + 2 * w.a));
    wqb = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.wq) + 2 * w.b));
  }
  if (w.on && p.wk) {
    wka = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.wk) + 2 * w.a));
    wkb = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.wk) + 2 * w.b));
  }
#pragma unroll
  for (int i = 0; i < kRopeUnroll; ++i) {
    const int row = row0 + i * kRowsWarp;
    const bool is_q = row < p.H, copy = row >= p.H + p.H_kv;
    float x[16];
    unpack16<DT>(xa[i], xb[i], x);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss += x[e] * x[e];
    ss = seg_sum<kSeg>(ss);
    if (!w.on || row >= rows) continue;
    const int h = is_q ? row : (copy ? row - p.H - p.H_kv : row - p.H);
    if (copy) {
      if (cache >= 0) {
        const int s0 = 16 * (lane % kSeg);
        st16(p.vc, cache + h * p.c_sh + s0, xa[i]);
        st16(p.vc, cache + h * p.c_sh + s0 + 8, xb[i]);
      }
      continue;
    }
    if (is_q ? p.wq != nullptr : p.wk != nullptr) {
      const float r = 1.0f / sqrtf(ss / p.D + p.eps);
      float g[16];
      unpack16<DT>(is_q ? wqa : wka, is_q ? wqb : wkb, g);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * r * g[e];
    }
    if (w.turn) turn16<1>(x, c, s, p.interleaved);
    uint4 a, bb;
    pack16<DT>(x, a, bb);
    const RopeView &out = is_q ? p.qo : p.ko;
    if (out.ptr) {
      const long long at = b * out.sb + l * out.sl + h * out.sh;
      st16(out.ptr, at + w.a, a);
      st16(out.ptr, at + w.b, bb);
    }
    if (!is_q && cache >= 0) {
      st16(p.kc, cache + h * p.c_sh + w.a, a);
      st16(p.kc, cache + h * p.c_sh + w.b, bb);
    }
  }
}

// Blocks [0, blocks_q) take the query rows, the others the key rows, each
// block every blocks-th group of tokens: a lane meets the same columns in all
// its rows and sums its 16 weight gradients in registers; the block adds its
// lanes in a fixed order and leaves one partial row of D.
template <int kSeg, int DT>
__global__ void __launch_bounds__(kRopeBwdThreads) fa_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kRowsWarp = 32 / kSeg;
  constexpr int kWarps = kRopeBwdThreads / 32;
  constexpr int kUnroll = 2;
  constexpr int kChunk = kRowsWarp * kUnroll;
  __shared__ float red[kWarps][kRowsWarp][kSeg * 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_q = static_cast<int>(blockIdx.x) < p.blocks_q;
  const int block = is_q ? blockIdx.x : blockIdx.x - p.blocks_q;
  const int n_blocks = is_q ? p.blocks_q : p.blocks_k;
  const int H = is_q ? p.H : p.H_kv;
  const RopeView in = is_q ? p.q : p.k, dy = is_q ? p.dyq : p.dyk, dx = is_q ? p.dq : p.dk;
  const void *weight = is_q ? p.wq : p.wk;
  const int chunks = (H + kChunk - 1) / kChunk;
  const long long items = static_cast<long long>(p.B) * p.L * chunks;
  const RopeLane w = rope_lane(lane % kSeg, p.D, p.rot, p.interleaved);
  float g[16], acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f, g[e] = 1.0f;
  if (w.on && weight)
    unpack16<DT>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(weight) + 2 * w.a)),
                 __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(weight) + 2 * w.b)), g);
  const float inv_d = 1.0f / p.D;
  for (long long item = static_cast<long long>(block) * kWarps + warp; item < items;
       item += static_cast<long long>(n_blocks) * kWarps) {
    const long long token = item / chunks;
    const int row0 = static_cast<int>(item - token * chunks) * kChunk + lane / kSeg;
    const int b = static_cast<int>(token / p.L), l = static_cast<int>(token - static_cast<long long>(b) * p.L);
    uint4 xa[kUnroll], xb[kUnroll], ya[kUnroll], yb[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = row0 + i * kRowsWarp;
      xa[i] = xb[i] = ya[i] = yb[i] = make_uint4(0, 0, 0, 0);
      if (w.on && h < H) {
        const long long at = b * in.sb + l * in.sl + h * in.sh;
        const long long ay = b * dy.sb + l * dy.sl + h * dy.sh;
        xa[i] = ld16(in.ptr, at + w.a);
        xb[i] = ld16(in.ptr, at + w.b);
        ya[i] = ld16(dy.ptr, ay + w.a);
        yb[i] = ld16(dy.ptr, ay + w.b);
      }
    }
    const long long pos = rope_position(p, b, l);
    const bool real = pos >= 0 && pos < p.max_pos;
    float c[8], s[8];
    if (real) rope_angles(p, pos, w, c, s);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = row0 + i * kRowsWarp;
      float x[16], y[16];
      unpack16<DT>(xa[i], xb[i], x);
      unpack16<DT>(ya[i], yb[i], y);
      if (w.turn && real) turn16<-1>(y, c, s, p.interleaved);
      if (weight) {
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss += x[e] * x[e];
        const float r = 1.0f / sqrtf(seg_sum<kSeg>(ss) / p.D + p.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] *= r;
          if (real) acc[e] += y[e] * x[e];
          y[e] *= g[e];
          dot += y[e] * x[e];
        }
        dot = seg_sum<kSeg>(dot) * inv_d;
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = r * (y[e] - x[e] * dot);
      }
      if (w.on && h < H) {
        uint4 a, bb;
        pack16<DT>(y, a, bb);
        if (!real) a = bb = make_uint4(0, 0, 0, 0);   // a padding token has no output
        const long long at = b * dx.sb + l * dx.sl + h * dx.sh;
        st16(dx.ptr, at + w.a, a);
        st16(dx.ptr, at + w.b, bb);
      }
    }
  }
  if (weight) {
    float *mine = red[warp][lane / kSeg];
    if (w.on) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mine[w.a + e] = acc[e];
        mine[w.b + e] = acc[8 + e];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kRopeBwdThreads) {
      float sum = 0.0f;
      for (int i = 0; i < kWarps; ++i)
        for (int j = 0; j < kRowsWarp; ++j) sum += red[i][j][d];
      p.part[static_cast<long long>(blockIdx.x) * p.D + d] = sum;
    }
  }
}

// dw[d] = the sum of the blocks' partials, in a fixed order: one block per
// weight vector, 8 partial rows at a time.
__global__ void __launch_bounds__(1024) fa_rope_dw_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float red[8][128];
  const bool is_q = blockIdx.x == 0;
  float *out = is_q ? p.dwq : p.dwk;
  if (!out) return;
  const int d = threadIdx.x & 127, y = threadIdx.x >> 7;
  const float *part = p.part + (is_q ? 0 : static_cast<long long>(p.blocks_q) * p.D);
  const int n = is_q ? p.blocks_q : p.blocks_k;
  float sum = 0.0f;
  if (d < p.D)
    for (int i = y; i < n; i += 8) sum += part[static_cast<long long>(i) * p.D + d];
  red[y][d] = sum;
  __syncthreads();
  if (y == 0 && d < p.D) {
    for (int i = 1; i < 8; ++i) sum += red[i][d];
    out[d] = sum;
  }
}

}  // namespace fa
