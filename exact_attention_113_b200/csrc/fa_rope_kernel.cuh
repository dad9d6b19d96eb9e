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
// bounds them, and close behind it the instructions (unpacking 16-bit values,
// addresses), which is why the arithmetic runs on fp32 pairs.  A row (one head
// of one token) belongs to D / 16 lanes, each with two 16-byte vectors that
// hold whole pairs (8 values from each half, or 16 neighbours), so the rotation
// needs no exchange and only the norm's sum crosses lanes.  Rows are copied to
// shared memory two steps ahead.  All arithmetic is fp32; the result is
// rounded once.  Measured: forward 0.87 of the HBM copy rate at B4 L8192 H48
// D64 (142 us), 0.78 with the cache at 8192 tokens (40 us); gradient 0.84 at B2
// L16384 H32/8 D128 (183 us); up to 4 % more on other cards.
#pragma once

#include "sm100.cuh"

namespace fa {

// Stages and blocks per SM, measured on one card on 8192 tokens (32 + 8 + 8 rows
// of D 128, to the cache) and on B4 L8192 H48 D64: 3 stages, 4 blocks 40 / 142 us;
// 2 stages 50 / 175; 4 stages 39 / 139, for a third more shared memory; 3 blocks
// 45 / 156, 5 blocks 41 / 148.  The gradient at B2 L16384 H32/8 D128: 3 stages,
// 4 blocks 183 us; 2 stages 206; 4 stages 182.
constexpr int kRopeThreads = 128;
constexpr int kRopeStages = 3;        // rows a lane has in shared memory
constexpr int kRopeBlocks = 4;        // resident per SM
constexpr int kRopeBwdStages = 3;
constexpr int kRopeBwdBlocks = 4;

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
  float eps, inv_d;
  // backward
  RopeView dyq, dyk;      // gradients of the outputs
  RopeView dq, dk;        // written
  float *part;            // [blocks][D] partial weight gradients
  float *dwq, *dwk;       // [D]
  int blocks_q, blocks_k;     // blocks of query rows, of key rows (the rest: value rows)
  int chunks_q, chunks_k;     // chunks of a token's rows, and their steps (forward)
  int per_q, per_k;
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

// A lane's 16 values as fp32 pairs: x[0..3] the first vector, x[4..7] the
// second.  The arithmetic runs on pairs (one instruction for two values).
struct Row16 {
  float2 x[8];
};
template <int DT>
__device__ __forceinline__ Row16 unpack16(const uint4 &a, const uint4 &b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  Row16 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.x[i] = unpack2<DT>(w[i]);
  return r;
}
template <int DT>
__device__ __forceinline__ void pack16(const Row16 &r, uint4 &a, uint4 &b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<DT>(r.x[i].x, r.x[i].y);
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// sum of x .* y over the lane's 16 values
__device__ __forceinline__ float dot16(const Row16 &x, const Row16 &y) {
  float2 s[2] = {both(0.0f), both(0.0f)};
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i & 1] = __ffma2_rn(x.x[i], y.x[i], s[i & 1]);
  return (s[0].x + s[1].x) + (s[0].y + s[1].y);
}

// The lane's 8 pairs turned by +angle (kSign 1) or -angle (kSign -1); c, s:
// its 8 cosines and sines.
template <int kSign, bool kInter>
__device__ __forceinline__ void turn16(Row16 &r, const float4 (&c)[2], const float4 (&s)[2]) {
  const float2 cc[4] = {make_float2(c[0].x, c[0].y), make_float2(c[0].z, c[0].w),
                        make_float2(c[1].x, c[1].y), make_float2(c[1].z, c[1].w)};
  const float2 ss[4] = {make_float2(s[0].x, s[0].y), make_float2(s[0].z, s[0].w),
                        make_float2(s[1].x, s[1].y), make_float2(s[1].z, s[1].w)};
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ci = i & 1 ? cc[i >> 1].y : cc[i >> 1].x;
      const float si = kSign * (i & 1 ? ss[i >> 1].y : ss[i >> 1].x);
      const float2 v = r.x[i];
      r.x[i] = __ffma2_rn(v, both(ci), __fmul2_rn(make_float2(v.y, v.x), make_float2(-si, si)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = r.x[i], b = r.x[4 + i];
      const float2 p = make_float2(kSign * ss[i].x, kSign * ss[i].y), n = make_float2(-p.x, -p.y);
      r.x[i] = __ffma2_rn(a, cc[i], __fmul2_rn(b, n));
      r.x[4 + i] = __ffma2_rn(b, cc[i], __fmul2_rn(a, p));
    }
  }
}

template <int kSeg>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int d = kSeg / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ const void *rope_position(const RopeParams &p, int b, int l) {
  return static_cast<const char *>(p.pos) + (b * p.pos_sb + l * p.pos_sl) * (p.pos64 ? 8 : 4);
}
// The position that copy8 brought.
__device__ __forceinline__ long long rope_position_of(const RopeParams &p, const long long *at) {
  return p.pos64 ? *at : static_cast<long long>(*reinterpret_cast<const int *>(at));
}

// The lane's cosines and sines (the first reading of a row of the table comes
// from L2, the warp's others from L1, so they are not kept in registers).
__device__ __forceinline__ void rope_angles(const RopeParams &p, long long pos, const RopeLane &w,
                                            float4 (&c)[2], float4 (&s)[2]) {
  const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + pos * p.rot + w.i0);
  const float4 *rs = reinterpret_cast<const float4 *>(p.cos_sin + pos * p.rot + p.rot / 2 + w.i0);
  c[0] = __ldg(row);
  c[1] = __ldg(row + 1);
  s[0] = __ldg(rs);
  s[1] = __ldg(rs + 1);
}
template <int DT>
__device__ __forceinline__ Row16 rope_weight(const void *weight, const RopeLane &w) {
  const uint8_t *at = static_cast<const uint8_t *>(weight);
  return unpack16<DT>(__ldg(reinterpret_cast<const uint4 *>(at + 2 * w.a)),
                      __ldg(reinterpret_cast<const uint4 *>(at + 2 * w.b)));
}

__device__ __forceinline__ void st16(uint8_t *p, const uint4 &v) { *reinterpret_cast<uint4 *>(p) = v; }

// 4 or 8 bytes, the same way.
__device__ __forceinline__ void copy8(long long *dst, const void *src, bool wide) {
  if (wide)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// 16 bytes into the lane's own place in shared memory, asynchronously; zeros
// where !ok (nothing is read then).
__device__ __forceinline__ void copy16(uint4 *dst, const uint8_t *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// A warp's walk over the rows of its kind.  A token's rows are `steps` steps
// of 32 / kSeg rows, one a lane segment.
struct RopeWalk {
  int b, l, r;        // batch, token, step within the token
  bool fresh;         // another token, or another run of its steps, has begun
  __device__ __forceinline__ uint8_t *row(const RopeView &v, int h) const {
    return const_cast<uint8_t *>(v.ptr) + 2 * (b * v.sb + l * v.sl + h * v.sh);
  }
};

// Every n-th chunk of at most `per` steps: the warps that run together work on
// neighbouring tokens, whose rows of one head are neighbours in a
// [B, H, L, D] output (the forward at B4 L8192 H48 D64: 141 us, in runs 162).
struct RopeChunks : RopeWalk {
  unsigned item, items, n;
  int steps, chunks, per, end;
  __device__ __forceinline__ void start(const RopeParams &p, unsigned me, unsigned warps, int steps_,
                                        int chunks_, int per_) {
    steps = steps_;
    chunks = chunks_;
    per = per_;
    item = me;
    items = p.B * p.L * chunks;
    n = warps;
    locate(p);
  }
  __device__ __forceinline__ void locate(const RopeParams &p) {
    const unsigned token = chunks == 1 ? item : item / chunks;
    r = chunks == 1 ? 0 : (item - token * chunks) * per;
    end = min(r + per, steps);
    b = p.B == 1 ? 0 : token / p.L;
    l = token - b * p.L;
    fresh = true;
  }
  __device__ __forceinline__ bool more() const { return item < items; }
  __device__ __forceinline__ void next(const RopeParams &p) {
    fresh = false;
    if (++r == end) {
      item += n;
      locate(p);
    }
  }
};

// An equal run of steps for each warp, tokens in order: the fewest
// instructions (the gradient at B2 L16384 H32/8 D128: in chunks 15 % slower).
struct RopeRun : RopeWalk {
  unsigned at, to;
  int steps;
  __device__ __forceinline__ void start(const RopeParams &p, unsigned me, unsigned warps,
                                        int steps_) {
    steps = steps_;
    const unsigned total = p.B * p.L * steps, q = total / warps, rest = total % warps;
    at = q * me + min(me, rest);
    to = at + q + (me < rest ? 1 : 0);
    const unsigned token = at / steps;
    r = at - token * steps;
    b = p.B == 1 ? 0 : token / p.L;
    l = token - b * p.L;
    fresh = true;
  }
  __device__ __forceinline__ bool more() const { return at < to; }
  __device__ __forceinline__ void next(const RopeParams &p) {
    ++at;
    fresh = ++r == steps;
    if (fresh) {
      r = 0;
      if (++l == p.L) {
        l = 0;
        ++b;
      }
    }
  }
};

// Where token (b, l) goes in a cache; false: nowhere.
__device__ __forceinline__ bool rope_slot(const RopeParams &p, long long slot, long long &at) {
  if (slot < 0 || slot >= p.n_slots) return false;
  long long page, in_page;
  if (p.n_slots <= 0x7fffffffll) {   // (a 32-bit division is a third of the cost)
    page = static_cast<unsigned>(slot) / static_cast<unsigned>(p.page_size);
    in_page = static_cast<unsigned>(slot) % static_cast<unsigned>(p.page_size);
  } else {
    page = slot / p.page_size;
    in_page = slot % p.page_size;
  }
  at = page * p.c_sp + in_page * p.c_st;
  return true;
}

// kSeg lanes a row: the smallest power of two >= D / 16.  Blocks are dealt to
// the kinds of rows (query, key, and value rows, which only move to the cache),
// and a kind's chunks to its warps.  A lane has its next kRopeStages - 1 rows
// under way in shared memory, where no registers wait for them and, as it
// reads only what it copied itself, no barrier either; a token's position and
// slot come the same way, with its first row.
template <int kSeg, int DT, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    fa_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kRowsWarp = 32 / kSeg, S = kRopeStages, kWarps = kRopeThreads / 32;
  __shared__ uint4 ring[kWarps][S][2][32];
  __shared__ long long meta[kWarps][S][2][32];   // position, slot
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = lane % kSeg, hl = lane / kSeg;
  const int bid = blockIdx.x, qk = p.blocks_q + p.blocks_k;
  const bool is_q = bid < p.blocks_q, is_v = bid >= qk;
  const int first = is_q ? 0 : (is_v ? qk : p.blocks_q);
  const int blocks = is_q ? p.blocks_q : (is_v ? gridDim.x - qk : p.blocks_k);
  const int H = is_q ? p.H : p.H_kv;
  const RopeView in = is_q ? p.q : (is_v ? p.v : p.k), out = is_q ? p.qo : p.ko;
  const bool cached = !is_q && p.kc, want = !is_v && out.ptr;
  RopeLane w = rope_lane(s, p.D, p.rot, kInter);
  if (is_v) {   // copied: neighbouring vectors, whatever the pairs are
    w.a = 16 * s;
    w.b = 16 * s + 8;
  }
  const int ab = 2 * (w.b - w.a);
  const void *weight = is_v ? nullptr : (is_q ? p.wq : p.wk);
  Row16 g;
  if (w.on && weight) g = rope_weight<DT>(weight, w);
  RopeChunks fw, cw;
  fw.start(p, (bid - first) * kWarps + warp, blocks * kWarps, (H + kRowsWarp - 1) / kRowsWarp,
           is_q ? p.chunks_q : p.chunks_k, is_q ? p.per_q : p.per_k);
  cw = fw;
  const uint8_t *src = nullptr;
  auto fetch = [&](int slot) {
    if (fw.more()) {
      const int h = fw.r * kRowsWarp + hl;
      if (fw.fresh) {
        src = fw.row(in, h) + 2 * w.a;
        copy8(&meta[warp][slot][0][lane], rope_position(p, fw.b, fw.l), p.pos64);
        if (cached)
          copy8(&meta[warp][slot][1][lane], p.slots + static_cast<long long>(fw.b) * p.L + fw.l, true);
      }
      const bool ok = w.on && h < H;
      copy16(&ring[warp][slot][0][lane], src, ok);
      copy16(&ring[warp][slot][1][lane], src + ab, ok);
      src += 2 * kRowsWarp * in.sh;
      fw.next(p);
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch(k);
  int slot = 0;
  bool real = false, stored = false, turn = false;
  uint8_t *d0 = nullptr, *d1 = nullptr;   // where a row goes: the output, the cache
  float4 co[2], si[2];
  for (; cw.more(); cw.next(p)) {
    copy_wait<S - 2>();
    uint4 a = ring[warp][slot][0][lane], bb = ring[warp][slot][1][lane];
    const int h = cw.r * kRowsWarp + hl;
    if (cw.fresh) {
      const long long pos = rope_position_of(p, &meta[warp][slot][0][lane]);
      real = pos >= 0 && pos < p.max_pos;   // else padding: left as it was
      if (want) d0 = cw.row(out, h) + 2 * w.a;
      long long at = 0;
      stored = cached && rope_slot(p, meta[warp][slot][1][lane], at);
      d1 = (is_v ? p.vc : p.kc) + 2 * (at + h * p.c_sh + w.a);
      turn = w.turn && real && !is_v;
      if (turn) rope_angles(p, pos, w, co, si);
    }
    slot = slot + 1 == S ? 0 : slot + 1;
    fetch(slot + S - 2 >= S ? slot - 2 : slot + S - 2);   // the slot read one row ago
    if (!real) continue;
    if (!is_v) {
      Row16 x = unpack16<DT>(a, bb);
      if (weight) {
        const float2 q = both(rsqrtf(seg_sum<kSeg>(dot16(x, x)) * p.inv_d + p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x.x[e] = __fmul2_rn(__fmul2_rn(x.x[e], q), g.x[e]);
      }
      if (turn) turn16<1, kInter>(x, co, si);
      pack16<DT>(x, a, bb);
    }
    if (w.on && h < H) {
      if (want) {
        st16(d0, a);
        st16(d0 + ab, bb);
        d0 += 2 * kRowsWarp * out.sh;
      }
      if (stored) {
        st16(d1, a);
        st16(d1 + ab, bb);
        d1 += 2 * kRowsWarp * p.c_sh;
      }
    }
  }
}

// The same walk with two rows to a step, x and dy.  A lane meets the same
// columns in all its rows and sums its 16 weight gradients in registers; the
// block adds its lanes in a fixed order and leaves one partial row of D.  With
// t = sum(w g x) the input's gradient is dx = r w g - x r^3 t / D, so the two
// sums over a row, of x x and of w g x, cross the lanes together.
template <int kSeg, int DT, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdBlocks)
    fa_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kRowsWarp = 32 / kSeg, S = kRopeBwdStages, kWarps = kRopeThreads / 32;
  __shared__ uint4 ring[kWarps][S][4][32];
  __shared__ long long meta[kWarps][S][32];   // position
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hl = lane / kSeg;
  const bool is_q = static_cast<int>(blockIdx.x) < p.blocks_q;
  const unsigned me = (is_q ? blockIdx.x : blockIdx.x - p.blocks_q) * kWarps + warp;
  const unsigned n = (is_q ? p.blocks_q : p.blocks_k) * kWarps;
  const int H = is_q ? p.H : p.H_kv;
  const int steps = (H + kRowsWarp - 1) / kRowsWarp;
  const RopeView in = is_q ? p.q : p.k, dy = is_q ? p.dyq : p.dyk, dx = is_q ? p.dq : p.dk;
  const void *weight = is_q ? p.wq : p.wk;
  const RopeLane w = rope_lane(lane % kSeg, p.D, p.rot, kInter);
  const int ab = 2 * (w.b - w.a);
  Row16 g;
  float2 acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = g.x[e] = both(0.0f);
  if (w.on && weight) g = rope_weight<DT>(weight, w);

  RopeRun fw, cw;
  fw.start(p, me, n, steps);
  cw = fw;
  const uint8_t *sx = nullptr, *sy = nullptr;
  auto fetch = [&](int slot) {
    if (fw.more()) {
      const int h = fw.r * kRowsWarp + hl;
      if (fw.fresh) {
        sx = fw.row(in, h) + 2 * w.a;
        sy = fw.row(dy, h) + 2 * w.a;
        copy8(&meta[warp][slot][lane], rope_position(p, fw.b, fw.l), p.pos64);
      }
      const bool ok = w.on && h < H;
      copy16(&ring[warp][slot][0][lane], sx, ok);
      copy16(&ring[warp][slot][1][lane], sx + ab, ok);
      copy16(&ring[warp][slot][2][lane], sy, ok);
      copy16(&ring[warp][slot][3][lane], sy + ab, ok);
      sx += 2 * kRowsWarp * in.sh;
      sy += 2 * kRowsWarp * dy.sh;
      fw.next(p);
    }
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch(k);
  int slot = 0;
  bool real = false;
  uint8_t *dst = nullptr;
  float4 co[2], si[2];
  for (; cw.more(); cw.next(p)) {
    copy_wait<S - 2>();
    if (cw.fresh) {
      const long long pos = rope_position_of(p, &meta[warp][slot][lane]);
      real = pos >= 0 && pos < p.max_pos;   // else padding, without an output
      dst = cw.row(dx, cw.r * kRowsWarp + hl) + 2 * w.a;
      if (w.turn && real) rope_angles(p, pos, w, co, si);
    }
    Row16 x = unpack16<DT>(ring[warp][slot][0][lane], ring[warp][slot][1][lane]);
    Row16 y = unpack16<DT>(ring[warp][slot][2][lane], ring[warp][slot][3][lane]);
    slot = slot + 1 == S ? 0 : slot + 1;
    fetch(slot + S - 2 >= S ? slot - 2 : slot + S - 2);   // the slot read one row ago
    uint4 a = make_uint4(0, 0, 0, 0), bb = a;
    if (real) {
      if (w.turn) turn16<-1, kInter>(y, co, si);
      if (weight) {
        Row16 wg;
#pragma unroll
        for (int e = 0; e < 8; ++e) wg.x[e] = __fmul2_rn(y.x[e], g.x[e]);
        float ss = dot16(x, x), t = dot16(x, wg);
#pragma unroll
        for (int d = kSeg / 2; d > 0; d >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, d);
          t += __shfl_xor_sync(0xffffffffu, t, d);
        }
        const float q = rsqrtf(ss * p.inv_d + p.eps);
        const float u = -(q * q * p.inv_d) * (q * t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[e] = __ffma2_rn(y.x[e], __fmul2_rn(x.x[e], both(q)), acc[e]);
          y.x[e] = __ffma2_rn(x.x[e], both(u), __fmul2_rn(wg.x[e], both(q)));
        }
      }
      pack16<DT>(y, a, bb);
    }
    if (w.on && cw.r * kRowsWarp + hl < H) {
      st16(dst, a);
      st16(dst + ab, bb);
      dst += 2 * kRowsWarp * dx.sh;
    }
  }
  if (weight) {
    // the ring is idle now and takes the lanes' sums
    copy_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(ring);   // [kWarps * kRowsWarp][kSeg * 16]
    float *mine = red + (warp * kRowsWarp + hl) * (kSeg * 16);
    if (w.on) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<float2 *>(mine + w.a + 2 * e) = acc[e];
        *reinterpret_cast<float2 *>(mine + w.b + 2 * e) = acc[4 + e];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kRopeThreads) {
      float sum = 0.0f;
      for (int i = 0; i < kWarps * kRowsWarp; ++i) sum += red[i * (kSeg * 16) + d];
      p.part[static_cast<long long>(blockIdx.x) * p.D + d] = sum;
    }
  }
}

// dw[d] = the sum of the blocks' partials, in a fixed order: a block takes 32
// columns of one weight, its 32 rows of threads every 32nd partial.
__global__ void __launch_bounds__(1024) fa_rope_dw_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float red[32][33];
  const bool is_q = blockIdx.x == 0;
  float *out = is_q ? p.dwq : p.dwk;
  if (!out) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, d = blockIdx.y * 32 + x;
  const float *part = p.part + (is_q ? 0 : static_cast<long long>(p.blocks_q) * p.D);
  const int n = is_q ? p.blocks_q : p.blocks_k;
  float sum = 0.0f;
  if (d < p.D)
#pragma unroll 8
    for (int i = y; i < n; i += 32) sum += part[i * p.D + d];
  red[y][x] = sum;
  __syncthreads();
  sum = red[x][y];
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  if (x == 0 && blockIdx.y * 32 + y < p.D) out[blockIdx.y * 32 + y] = sum;
}

}  // namespace fa
