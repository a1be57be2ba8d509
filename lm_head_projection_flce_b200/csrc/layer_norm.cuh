// layer_norm.cuh - layer norm over the last dimension, in front of the LM
// head: forward, and the backward with the reduction of the weight's and the
// bias's gradients over the rows.
//
//   mean_n = sum_h x[n,h] / H      var_n = sum_h (x[n,h] - mean_n)^2 / H
//   rstd_n = 1 / sqrt(var_n + eps)           xhat = (x - mean_n) rstd_n
//   y      = xhat w + b
//   g      = dy w
//   dx     = rstd_n (g - sum_h g / H - xhat sum_h (g xhat) / H)
//   dw[h]  = sum_n dy xhat         db[h] = sum_n dy
//
// x, y, dy and dx are BF16 or FP32; everything between is FP32.  Both passes
// are bound by HBM: the forward reads x and writes y, the backward reads x and
// dy and writes dx, so a row is loaded once and held in registers, where the
// variance takes its second look at it.
//
// A mean in FP32, m0, is off by roundings of the row's magnitude.  So the second look
// also sums what it leaves, r = sum_h (x[n,h] - m0) / H, and
//   xhat = ((x - m0) - r) rstd_n      var_n = sum_h (x - m0)^2 / H - r^2
// are off by roundings of the row's spread only, however large the mean: FP32 rows of
// unit spread around 1000 by about 2e-7, where x - m0 alone is off by 1e-4, and the
// xhat of a constant row is 0.  The backward is given the mean rounded to FP32; where
// that is large against the spread, r is summed and taken out once more.
//
// A thread owns the same columns of every row it sees: the weights stay in its
// registers, and so do its shares of dw and db, which leave the block once, as one row
// of FP32 partials per block; a second kernel adds the partials in a fixed order (no
// atomics: the same inputs give the same bits).
#pragma once

#include <cuda_bf16.h>

#include <initializer_list>

#include "epilogues.cuh"
#include "extents.cuh"

namespace flce {

constexpr int kLnShare = 16;            // columns per thread
constexpr int kLnMaxThreads = 512;      // threads per row: rows up to 8192 columns in registers
constexpr int kLnWarpRows = 4;          // rows (warps) per block when a warp holds a row
constexpr int kLnWarpCols = 32 * kLnShare;
constexpr int kLnSms = 148;             // SMs the partials' layout is sized for
constexpr int kLnReduceCols = 32;       // columns per block of the partials' sum
constexpr int kLnReduceWarps = 16;

// N consecutive elements at a time, as floats.  The address is aligned to the
// vector's size (16 bytes at most per access).
template <typename T, int N>
struct LnIo;  // N: 1, 4 or 8
template <int N>
struct LnIo<__nv_bfloat16, N> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[N]) {
    if constexpr (N == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else if constexpr (N == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      x[0] = __uint_as_float(w.x << 16);
      x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = __uint_as_float(w.y << 16);
      x[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      x[0] = __bfloat162float(*p);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[N]) {
    if constexpr (N == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else if constexpr (N == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    } else {
      *p = __float2bfloat16_rn(x[0]);
    }
  }
};
template <int N>
struct LnIo<float, N> {
  static __device__ __forceinline__ void load(const float* p, float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + i);
        x[i] = w.x;
        x[i + 1] = w.y;
        x[i + 2] = w.z;
        x[i + 3] = w.w;
      }
    } else {
      x[0] = *p;
    }
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
      *p = x[0];
    }
  }
};

// 16 bytes at `off` bytes (a multiple of the element, not 0) past an aligned
// address: cut out of the two aligned vectors around them (the second is the
// neighbouring thread's first: an L1 hit).
__device__ __forceinline__ uint4 load16_shifted(uintptr_t aligned_at, uint32_t off) {
  const uint4 lo = *reinterpret_cast<const uint4*>(aligned_at);
  const uint4 hi = *reinterpret_cast<const uint4*>(aligned_at + 16);
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (off & 8u) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4u) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t sh = (off & 3u) * 8u;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], sh);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 16 bytes of elements [c, c + N) of a row at any alignment; `fill` (a word of
// them) behind `end`.  In a row that does not start on 16 bytes they are shifted
// into place; its first and last vectors, where the aligned ones would reach out of
// the row, are read by elements.
template <typename T>
__device__ __forceinline__ uint4 load16_any(const T* row, int64_t c, int64_t end, uint32_t fill) {
  constexpr int N = 16 / int(sizeof(T));
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
  const uint32_t off = static_cast<uint32_t>(at) & 15u;  // the same for the whole row
  if (off == 0 && c + N <= end) return *reinterpret_cast<const uint4*>(at);
  if (off != 0 && c >= N && c + 2 * N <= end) return load16_shifted(at - off, off);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = c + i < end ? reinterpret_cast<const uint32_t*>(row)[c + i] : fill;
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
      w[i] = (c + 2 * i < end ? p[c + 2 * i] : fill & 0xffffu) |
             uint32_t(c + 2 * i + 1 < end ? p[c + 2 * i + 1] : fill >> 16) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Sums of two or four values over a row's threads: a warp, or the whole block (at most
// 16 warps) through shared memory.  The values are folded into one another on the
// way: after the first exchange half of the warp carries one half of them, so two
// values take 5 shuffles and four take 6.  `buf` alternates between calls, so one
// barrier per call is enough: a buffer is written again only after every thread
// passed the barrier of the call in between.
constexpr int kLnMaxWarps = kLnMaxThreads / 32;
template <bool kWarpRow>
__device__ __forceinline__ float2 ln_row_sum(float2 v, float (*red)[4 * kLnMaxWarps], int& buf) {
  static_assert(kLnMaxWarps == 16, "half a warp adds the warps' sums");
  const int lane = threadIdx.x & 31;
  const bool up = (lane & 16) != 0;  // these lanes carry v.y
  float s = (up ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, up ? v.x : v.y, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (!kWarpRow) {
    if ((lane & 15) == 0) red[buf][(lane & 16) + (threadIdx.x >> 5)] = s;
    __syncthreads();
    s = (lane & 15) < int(blockDim.x >> 5) ? red[buf][lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    buf ^= 1;
  }
  const float other = __shfl_xor_sync(0xffffffffu, s, 16);
  return up ? make_float2(other, s) : make_float2(s, other);
}
template <bool kWarpRow>
__device__ __forceinline__ float4 ln_row_sum(float4 v, float (*red)[4 * kLnMaxWarps], int& buf) {
  const int lane = threadIdx.x & 31;
  const bool up = (lane & 16) != 0, mid = (lane & 8) != 0;  // lane / 8: the value carried
  const float a = (up ? v.z : v.x) + __shfl_xor_sync(0xffffffffu, up ? v.x : v.z, 16);
  const float b = (up ? v.w : v.y) + __shfl_xor_sync(0xffffffffu, up ? v.y : v.w, 16);
  float s = (mid ? b : a) + __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (!kWarpRow) {
    const int warps = int(blockDim.x >> 5), i = lane & 7;
    if (i == 0) red[buf][(lane >> 3) * kLnMaxWarps + (threadIdx.x >> 5)] = s;
    __syncthreads();
    const float* of = red[buf] + (lane >> 3) * kLnMaxWarps;
    s = (i < warps ? of[i] : 0.0f) + (i + 8 < warps ? of[i + 8] : 0.0f);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    buf ^= 1;
  }
  return make_float4(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 8),
                     __shfl_sync(0xffffffffu, s, 16), __shfl_sync(0xffffffffu, s, 24));
}

// What a row's sums say: of x - m0 and of its squares.
struct LnStats {
  float mean, rest, rstd;  // rest: r
};
__device__ __forceinline__ LnStats ln_stats(float m0, float sum, float squares, float inv_h, float eps) {
  LnStats s;
  s.rest = sum * inv_h;
  const float var = fmaf(-s.rest, s.rest, squares * inv_h);
  s.rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);  // a NaN stays one
  s.mean = m0 + s.rest;
  return s;
}

struct LnArgs {
  const void* x;
  int64_t ldx;
  const void* w;  // nullptr: ones
  const void* b;  // nullptr: zeros
  int64_t n, h;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;  // either may be nullptr
  float* rstd;
};

// A thread's 16 columns as 8 pairs (packed FP32 arithmetic works on two at a time):
// vector i of VN columns starts at column (i * tpr + t) * VN for thread t of the
// tpr that share the row.
// kExact: the block's shares cover the row exactly; else columns behind its end
// read as `fill`.
template <typename T, int VN, bool kExact>
__device__ __forceinline__ void ln_share_load(const T* src, int t, int tpr, int h, float fill,
                                              float2 (&v)[8]) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16 / VN; ++i) {
    const int c = (i * tpr + t) * VN;
    float one[VN];
#pragma unroll
    for (int j = 0; j < VN; ++j) one[j] = fill;
    if (kExact || c < h) LnIo<T, VN>::load(src + c, one);
#pragma unroll
    for (int j = 0; j < VN; ++j) x[i * VN + j] = one[j];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
}
template <typename T, int VN, bool kExact>
__device__ __forceinline__ void ln_share_store(T* dst, int t, int tpr, int h,
                                               const float2 (&v)[8]) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = v[i].x;
    x[2 * i + 1] = v[i].y;
  }
#pragma unroll
  for (int i = 0; i < 16 / VN; ++i) {
    const int c = (i * tpr + t) * VN;
    float one[VN];
#pragma unroll
    for (int j = 0; j < VN; ++j) one[j] = x[i * VN + j];
    if (kExact || c < h) LnIo<T, VN>::store(dst + c, one);
  }
}
// Zeroes the columns behind the row's end.
template <int VN>
__device__ __forceinline__ void ln_share_clip(int t, int tpr, int h, float2 (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = e / VN;
    if ((i * tpr + t) * VN >= h) (e % 2 ? v[e / 2].y : v[e / 2].x) = 0.0f;
  }
}
__device__ __forceinline__ float2 ln_both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float ln_share_sum(const float2 (&v)[8]) {
  float2 s = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) s = __fadd2_rn(s, v[i]);
  return s.x + s.y;
}
// Subtracts m0; returns the share's sum and sum of squares.
template <int VN, bool kExact>
__device__ __forceinline__ float2 ln_share_centre(float m0, int t, int tpr, int h, float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fadd2_rn(v[i], ln_both(-m0));
  if constexpr (!kExact) ln_share_clip<VN>(t, tpr, h, v);
  float2 q = __fmul2_rn(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) q = __ffma2_rn(v[i], v[i], q);
  return make_float2(ln_share_sum(v), q.x + q.y);
}
// y in place of x - m0.
__device__ __forceinline__ void ln_share_y(const LnStats& s, const float2 (&w)[8], const float2 (&b)[8],
                                           float2 (&v)[8]) {
  const float2 k = ln_both(s.rstd), c = ln_both(-s.rest * s.rstd);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __ffma2_rn(__ffma2_rn(v[i], k, c), w[i], b[i]);
}
// xhat in place of x, the row's shares of dw and db, g = dy w in place of dy;
// returns the shares of sum g and sum g xhat.  Behind the row's end dy is 0.
__device__ __forceinline__ float2 ln_share_grads(float mean, float rstd, const float2 (&w)[8],
                                                 float2 (&xh)[8], float2 (&d)[8], float2 (&aw)[8],
                                                 float2 (&ab)[8]) {
  float2 s1 = ln_both(0.0f), s2 = ln_both(0.0f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    xh[k] = __fmul2_rn(__fadd2_rn(xh[k], ln_both(-mean)), ln_both(rstd));
    ab[k] = __fadd2_rn(ab[k], d[k]);
    aw[k] = __ffma2_rn(d[k], xh[k], aw[k]);
    d[k] = __fmul2_rn(d[k], w[k]);
    s1 = __fadd2_rn(s1, d[k]);
    s2 = __ffma2_rn(d[k], xh[k], s2);
  }
  return make_float2(s1.x + s1.y, s2.x + s2.y);
}
// dx in place of g, from the row's sums of g and g xhat over H.
__device__ __forceinline__ void ln_share_dx(float2 means, float rstd, const float2 (&xh)[8],
                                            float2 (&d)[8]) {
  const float2 m1 = ln_both(-means.x), m2 = ln_both(-means.y);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    d[k] = __fmul2_rn(__ffma2_rn(xh[k], m2, __fadd2_rn(d[k], m1)), ln_both(rstd));
}

// Rows straight from global memory: few rows, or rows that a warp holds (kWarpRow;
// no barriers).  Two rows at a time: both sums of a reduction travel together.
template <typename T, typename W, int VN, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kLnWarpRows : kLnMaxThreads)
    ln_forward_kernel(const LnArgs a) {
  __shared__ float red[2][4 * kLnMaxWarps];
  const int tpr = kWarpRow ? 32 : int(blockDim.x), h = int(a.h);
  const int t = kWarpRow ? int(threadIdx.x & 31) : int(threadIdx.x);
  const int rpb = kWarpRow ? int(blockDim.x >> 5) : 1;
  const int64_t step = int64_t(gridDim.x) * rpb;
  const float inv_h = 1.0f / float(h);
  int buf = 0;
  float2 w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = ln_both(1.0f);
    b[i] = ln_both(0.0f);
  }
  if (a.w) ln_share_load<W, VN, false>(static_cast<const W*>(a.w), t, tpr, h, 0.0f, w);
  if (a.b) ln_share_load<W, VN, false>(static_cast<const W*>(a.b), t, tpr, h, 0.0f, b);
  auto finish = [&](int64_t r, float2 (&v)[8], const LnStats& s) {
    if (t == 0) {
      if (a.mean) a.mean[r] = s.mean;
      if (a.rstd) a.rstd[r] = s.rstd;
    }
    ln_share_y(s, w, b, v);
    ln_share_store<T, VN, false>(static_cast<T*>(a.y) + r * a.ldy, t, tpr, h, v);
  };
  // The loop is uniform over the threads that share a row.
  for (int64_t r = int64_t(blockIdx.x) * rpb + (kWarpRow ? int(threadIdx.x >> 5) : 0); r < a.n;
       r += 2 * step) {
    const bool two = r + step < a.n;
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    float2 v0[8], v1[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v1[k] = ln_both(0.0f);
    ln_share_load<T, VN, false>(x, t, tpr, h, 0.0f, v0);
    if (two) ln_share_load<T, VN, false>(x + step * a.ldx, t, tpr, h, 0.0f, v1);
    const float2 s = ln_row_sum<kWarpRow>(make_float2(ln_share_sum(v0), ln_share_sum(v1)), red, buf);
    const float m0 = s.x * inv_h, m1 = s.y * inv_h;
    const float2 c0 = ln_share_centre<VN, false>(m0, t, tpr, h, v0);
    const float2 c1 = ln_share_centre<VN, false>(m1, t, tpr, h, v1);
    const float4 c = ln_row_sum<kWarpRow>(make_float4(c0.x, c0.y, c1.x, c1.y), red, buf);
    finish(r, v0, ln_stats(m0, c.x, c.y, inv_h, a.eps));
    if (two) finish(r + step, v1, ln_stats(m1, c.z, c.w, inv_h, a.eps));
  }
}

// ---------------------------------------------------------------- rows through a ring
// With more rows than blocks a block that loads a row, reduces it and stores it
// leaves HBM idle between its loads (195 + 280 us forward + backward of 16384
// rows of 8192 BF16, against 97 + 134 us this way: 5.5 and 6.0 TB/s, 86% and 93% of
// the copy bandwidth).  So one block (or 512 / tpr of them) per SM streams
// its rows through a ring of shared-memory slots with bulk copies, several rows
// ahead; a slot is refilled right after the first barrier of the row that used
// it.  A thread's columns, weights and gradient sums stay in registers.
//
// Rows that do not start or end on 16 bytes are copied with the bytes around them,
// up to the boundaries; these belong to neighbouring rows or the gaps between
// rows.  The tensor's first and last row, whose surroundings belong to somebody
// else, are loaded directly instead.
constexpr int kLnSlots = 8;                  // rows in flight per block, at most
constexpr int kLnRingBytes = 192 * 1024;     // per SM

struct LnRing {
  int slots;
  uint32_t slot_bytes;   // per tensor
  unsigned* err;
  uint64_t timeout_ns;
};

// Position in the ring of the next row to use or to load.
struct LnRingPos {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int slots) {
    if (++slot == slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

struct LnRingRow {
  const uint8_t* begin;  // 16-byte aligned start of the copy
  uint32_t bytes;
  uint32_t phase;        // offset of the row's first element in it
  bool direct;
};
template <typename T>
__device__ __forceinline__ LnRingRow ln_ring_row(const void* base, int64_t ld, int64_t n, int64_t h,
                                                 int64_t r) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(static_cast<const T*>(base) + r * ld);
  LnRingRow row;
  row.phase = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
  row.begin = p - row.phase;
  const uint32_t len = row.phase + static_cast<uint32_t>(h * int64_t(sizeof(T)));
  row.bytes = (len + 15u) & ~15u;
  row.direct = (r == 0 && row.phase != 0) || (r == n - 1 && row.bytes != len);
  return row;
}
template <typename T, int VN, bool kExact>
__device__ __forceinline__ void ln_ring_read(const uint8_t* slot, const void* base, int64_t ld,
                                             int64_t n, int h, int64_t r, float2 (&v)[8]) {
  if constexpr (VN == 1) {
    const LnRingRow row = ln_ring_row<T>(base, ld, n, h, r);
    if (row.direct)
      ln_share_load<T, VN, kExact>(reinterpret_cast<const T*>(row.begin + row.phase), threadIdx.x,
                                   blockDim.x, h, 0.0f, v);
    else
      ln_share_load<T, VN, kExact>(reinterpret_cast<const T*>(slot + row.phase), threadIdx.x,
                                   blockDim.x, h, 0.0f, v);
  } else {  // whole rows of 16-byte pieces: never direct
    ln_share_load<T, VN, kExact>(reinterpret_cast<const T*>(slot), threadIdx.x, blockDim.x, h, 0.0f,
                                 v);
  }
}
// After a wait that ran out, by the thread that issues the copies: those still in flight
// get time to land before the block can exit.
__device__ __forceinline__ void ln_ring_settle() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 200000ull) {
  }
}
// Two rows at a time: both sums of a reduction travel together.
template <typename T, typename W, int VN, bool kExact>
__global__ void __launch_bounds__(kLnMaxThreads, 1)
    ln_forward_ring_kernel(const LnArgs a, const LnRing g) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kLnSlots];
  __shared__ float red[2][4 * kLnMaxWarps];
  __shared__ PipeCtl ctl;
  const int t = threadIdx.x, tpr = blockDim.x, h = int(a.h);
  const int count = int((a.n - blockIdx.x + gridDim.x - 1) / gridDim.x);  // this block's rows
  int loaded = 0;  // thread 0: rows issued so far, and the slot of the next
  LnRingPos put, get;
  auto issue = [&]() {
    if (loaded >= count || put.slot < 0) return;
    const LnRingRow row =
        ln_ring_row<T>(a.x, a.ldx, a.n, a.h, int64_t(blockIdx.x) + int64_t(loaded++) * gridDim.x);
    const uint32_t bar = smem_u32(&full[put.slot]);
    if (row.direct) {
      mbar_arrive(bar);  // keeps the slot's phases in step
    } else {
      mbar_arrive_expect_tx(bar, row.bytes);
      bulk_load(smem_u32(ring) + uint32_t(put.slot) * g.slot_bytes, row.begin, row.bytes, bar);
    }
    put.advance(g.slots);
  };
  if (t == 0) {
    for (int s = 0; s < g.slots; ++s) mbar_init(smem_u32(&full[s]), 1);
    ctl.abort = 0;
    fence_barrier_init();
    for (int s = 0; s < g.slots; ++s) issue();
  }
  float2 w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = ln_both(1.0f);
    b[i] = ln_both(0.0f);
  }
  if (a.w) ln_share_load<W, VN, kExact>(static_cast<const W*>(a.w), t, tpr, h, 0.0f, w);
  if (a.b) ln_share_load<W, VN, kExact>(static_cast<const W*>(a.b), t, tpr, h, 0.0f, b);
  __syncthreads();
  const float inv_h = 1.0f / float(h);
  int buf = 0;
  auto fetch = [&](int64_t r, float2 (&v)[8]) {
    // A wait that ran out is recorded and the row's result lost; nothing more is loaded,
    // and the loop ends as usual.
    const uint32_t bar = smem_u32(&full[get.slot]);
    if (!mbar_try_wait(bar, get.parity) &&
        !wait_phase(bar, get.parity, &ctl, g.err, g.timeout_ns) && t == 0)
      put.slot = -1;  // tested where the slot is needed anyway: a flag of its own took 2% longer
    ln_ring_read<T, VN, kExact>(ring + uint32_t(get.slot) * g.slot_bytes, a.x, a.ldx, a.n, h, r, v);
    get.advance(g.slots);
  };
  auto finish = [&](int64_t r, float2 (&v)[8], const LnStats& s) {
    if (t == 0) {
      if (a.mean) a.mean[r] = s.mean;
      if (a.rstd) a.rstd[r] = s.rstd;
    }
    ln_share_y(s, w, b, v);
    ln_share_store<T, VN, kExact>(static_cast<T*>(a.y) + r * a.ldy, t, tpr, h, v);
  };
  int64_t r = blockIdx.x;
  for (int i = 0; i < count; i += 2, r += 2 * int64_t(gridDim.x)) {
    const bool two = i + 1 < count;
    float2 v0[8], v1[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v1[k] = ln_both(0.0f);
    fetch(r, v0);
    if (two) fetch(r + gridDim.x, v1);
    const float2 s = ln_row_sum<false>(make_float2(ln_share_sum(v0), ln_share_sum(v1)), red, buf);
    if (t == 0) {
      issue();
      if (two) issue();
    }
    const float m0 = s.x * inv_h, m1 = s.y * inv_h;
    const float2 c0 = ln_share_centre<VN, kExact>(m0, t, tpr, h, v0);
    const float2 c1 = ln_share_centre<VN, kExact>(m1, t, tpr, h, v1);
    const float4 c = ln_row_sum<false>(make_float4(c0.x, c0.y, c1.x, c1.y), red, buf);
    finish(r, v0, ln_stats(m0, c.x, c.y, inv_h, a.eps));
    if (two) finish(r + gridDim.x, v1, ln_stats(m1, c.z, c.w, inv_h, a.eps));
  }
  if (t == 0 && ctl.abort) ln_ring_settle();
}

// Rows too long for the registers of one block: three looks at the row, the
// later ones from L2.  A thread's share has no bound here: the mean is summed in
// FP64, 32 elements of the thread at a time, and its remainder as above.
constexpr int kLnLongThreads = 1024;
// Sum over a block of whole warps, in FP64.
__device__ __forceinline__ double ln_block_sum(double v) {
  __shared__ double red[32];
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the last call's values have been read
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < int(blockDim.x >> 5) ? red[lane] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <typename T, typename W>
__global__ void __launch_bounds__(kLnLongThreads) ln_forward_long_kernel(const LnArgs a) {
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.y) + r * a.ldy;
    float v[1], w[1], b[1];
    double sum = 0.0;
    for (int64_t c0 = threadIdx.x; c0 < a.h; c0 += 32 * kLnLongThreads) {
      const int64_t end = min(a.h, c0 + 32 * kLnLongThreads);
      float part = 0.0f;
      for (int64_t c = c0; c < end; c += kLnLongThreads) {
        LnIo<T, 1>::load(x + c, v);
        part += v[0];
      }
      sum += double(part);
    }
    const double inv_h = 1.0 / double(a.h);
    const float m0 = float(ln_block_sum(sum) * inv_h);
    float left = 0.0f, squares = 0.0f;
    for (int64_t c = threadIdx.x; c < a.h; c += kLnLongThreads) {
      LnIo<T, 1>::load(x + c, v);
      v[0] -= m0;
      left += v[0];
      squares += v[0] * v[0];
    }
    const double rest = ln_block_sum(double(left)) * inv_h;
    const double var = ln_block_sum(double(squares)) * inv_h - rest * rest;
    const float rstd = 1.0f / sqrtf(float(var < 0.0 ? 0.0 : var) + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = float(double(m0) + rest);
      if (a.rstd) a.rstd[r] = rstd;
    }
    const float shift = float(-rest * double(rstd));
    for (int64_t c = threadIdx.x; c < a.h; c += kLnLongThreads) {
      LnIo<T, 1>::load(x + c, v);
      v[0] = fmaf(v[0] - m0, rstd, shift);
      if (a.w) {
        LnIo<W, 1>::load(static_cast<const W*>(a.w) + c, w);
        v[0] *= w[0];
      }
      if (a.b) {
        LnIo<W, 1>::load(static_cast<const W*>(a.b) + c, b);
        v[0] += b[0];
      }
      LnIo<T, 1>::store(y + c, v);
    }
  }
}

struct LnBwdArgs {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* w;  // nullptr: ones
  const float* mean;
  const float* rstd;
  int64_t n, h;
  void* dx;       // nullptr: not wanted
  int64_t lddx;
  float* part_w;  // [gridDim.x][h] each; nullptr: not wanted
  float* part_b;
};

// The backward's mean is off by a rounding, 2^-24 |mean|, and with it xhat by that times
// rstd: for a mean within 16 standard deviations 1e-6 at most, no more than by the sums'
// roundings.  Rows beyond are rare, and a block does them once more behind its other
// rows (where all of them are, 16384 x 8192 BF16 takes 724 us against 135): what the
// means leave over, summed for every row within its loop, cost all backwards 2% at that
// size, 9% at 4096 x 8191, and 28% where dx is not wanted.
__device__ __forceinline__ bool ln_far(float mean, float rstd) { return fabsf(mean) * rstd > 16.0f; }
// Whether a thread sees such a row, when the block deals out the rows first, first + step, ...
__device__ __forceinline__ bool ln_sees_far(const LnBwdArgs& a, int64_t first, int64_t step) {
  bool any = false;
  for (int64_t r = first + threadIdx.x * step; r < a.n; r += blockDim.x * step)
    any |= ln_far(a.mean[r], a.rstd[r]);
  return any;
}
// Of the rows [r, r + kRun), r = first, first + step, ..., by a whole block: dx is written
// again, and `part_w`, the row of partials that holds these rows' shares of dw, put
// right; either may be nullptr.  any: whether this thread saw a row to do.
template <typename T, typename W, int VN, int kRun>
__device__ __forceinline__ void ln_backward_far(const LnBwdArgs& a, bool any, float* part_w,
                                                int64_t first, int64_t step) {
  if (!__syncthreads_or(any)) return;  // the block's partials and dx are written, too
  if (part_w == nullptr && a.dx == nullptr) return;
  const double inv_h = 1.0 / double(a.h);
  for (int64_t r = first, i = 0; r - i < a.n; i + 1 < kRun ? (++i, ++r) : (r += step - i, i = 0)) {
    if (r >= a.n) continue;
    const float mean = a.mean[r], rstd = a.rstd[r];
    if (!ln_far(mean, rstd)) continue;  // the same for every thread
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    float v[VN], g[VN], w[VN];
    auto xhat = [&](int64_t c) {
      LnIo<T, VN>::load(x + c, v);
#pragma unroll
      for (int j = 0; j < VN; ++j) v[j] = (v[j] - mean) * rstd;
    };
    auto weight = [&](int64_t c) {
#pragma unroll
      for (int j = 0; j < VN; ++j) w[j] = 1.0f;
      if (a.w) LnIo<W, VN>::load(static_cast<const W*>(a.w) + c, w);
    };
    const int64_t t = int64_t(threadIdx.x) * VN, next = int64_t(blockDim.x) * VN;
    float s = 0.0f;
    for (int64_t c = t; c < a.h; c += next) {
      xhat(c);
#pragma unroll
      for (int j = 0; j < VN; ++j) s += v[j];
    }
    const float rest = float(ln_block_sum(double(s)) * inv_h);
    float m1 = 0.0f, m2 = 0.0f;
    if (a.dx) {
      for (int64_t c = t; c < a.h; c += next) {
        xhat(c);
        LnIo<T, VN>::load(dy + c, g);
        weight(c);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          m1 += g[j] * w[j];
          m2 += g[j] * w[j] * (v[j] - rest);
        }
      }
      m1 = float(ln_block_sum(double(m1)) * inv_h);
      m2 = float(ln_block_sum(double(m2)) * inv_h);
    }
    for (int64_t c = t; c < a.h; c += next) {
      LnIo<T, VN>::load(dy + c, g);
      if (part_w) {
        LnIo<float, VN>::load(part_w + c, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) w[j] -= g[j] * rest;
        LnIo<float, VN>::store(part_w + c, w);
      }
      if (a.dx == nullptr) continue;
      xhat(c);
      weight(c);
#pragma unroll
      for (int j = 0; j < VN; ++j) g[j] = rstd * (g[j] * w[j] - m1 - (v[j] - rest) * m2);
      LnIo<T, VN>::store(static_cast<T*>(a.dx) + r * a.lddx + c, g);
    }
  }
}

template <typename T, typename W, int VN, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kLnWarpRows : kLnMaxThreads)
    ln_backward_kernel(const LnBwdArgs a) {
  __shared__ float red[2][4 * kLnMaxWarps];
  __shared__ __align__(16) float part[kWarpRow ? kLnWarpRows : 1][kWarpRow ? kLnWarpCols : 4];
  grid_launch_dependents();
  const int tpr = kWarpRow ? 32 : int(blockDim.x), h = int(a.h);
  const int t = kWarpRow ? int(threadIdx.x & 31) : int(threadIdx.x);
  const int warp = threadIdx.x >> 5;
  const int rpb = kWarpRow ? kLnWarpRows : 1;
  const int64_t step = int64_t(gridDim.x) * rpb;
  const float inv_h = 1.0f / float(h);
  int buf = 0;
  float2 w[8], aw[8], ab[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = ln_both(1.0f);
    aw[i] = ab[i] = ln_both(0.0f);
  }
  if (a.w) ln_share_load<W, VN, false>(static_cast<const W*>(a.w), t, tpr, h, 0.0f, w);
  bool far = false;
  for (int64_t r = int64_t(blockIdx.x) * rpb + (kWarpRow ? warp : 0); r < a.n; r += step) {
    const float mean = a.mean[r], rstd = a.rstd[r];
    far |= ln_far(mean, rstd);
    float2 xh[8], d[8];
    ln_share_load<T, VN, false>(static_cast<const T*>(a.x) + r * a.ldx, t, tpr, h, 0.0f, xh);
    ln_share_load<T, VN, false>(static_cast<const T*>(a.dy) + r * a.lddy, t, tpr, h, 0.0f, d);
    float2 s = ln_share_grads(mean, rstd, w, xh, d, aw, ab);
    if (a.dx == nullptr) continue;  // the same for every thread
    s = ln_row_sum<kWarpRow>(s, red, buf);
    ln_share_dx(make_float2(s.x * inv_h, s.y * inv_h), rstd, xh, d);
    ln_share_store<T, VN, false>(static_cast<T*>(a.dx) + r * a.lddx, t, tpr, h, d);
  }
  // The block's row of partials: its threads' sums, or the sum over its warps.
  float* out[2] = {a.part_w, a.part_b};
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (out[p] == nullptr) continue;
    float* to = out[p] + int64_t(blockIdx.x) * h;
    if constexpr (kWarpRow) {
      ln_share_store<float, VN, false>(part[warp], t, tpr, h, p == 0 ? aw : ab);
    } else {
      ln_share_store<float, VN, false>(to, t, tpr, h, p == 0 ? aw : ab);
    }
    if constexpr (kWarpRow) {
      __syncthreads();
      for (int c = threadIdx.x; c < h; c += 32 * kLnWarpRows) {
        float v = part[0][c];
#pragma unroll
        for (int k = 1; k < kLnWarpRows; ++k) v += part[k][c];
        to[c] = v;
      }
      __syncthreads();
    }
  }
  ln_backward_far<T, W, VN, kWarpRow ? kLnWarpRows : 1>(
      a, far, a.part_w ? a.part_w + int64_t(blockIdx.x) * h : nullptr, int64_t(blockIdx.x) * rpb, step);
}

// The backward through the ring: a slot holds the row of x and the row of dy.
template <typename T, typename W, int VN, bool kExact>
__global__ void __launch_bounds__(kLnMaxThreads, 1)
    ln_backward_ring_kernel(const LnBwdArgs a, const LnRing g) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kLnSlots];
  __shared__ float red[2][4 * kLnMaxWarps];
  __shared__ PipeCtl ctl;
  const int t = threadIdx.x, tpr = blockDim.x, h = int(a.h);
  const int count = int((a.n - blockIdx.x + gridDim.x - 1) / gridDim.x);
  int loaded = 0;  // thread 0: rows issued so far, and the slot of the next
  LnRingPos put, get;
  auto issue = [&]() {
    if (loaded >= count) return;
    const int64_t r = int64_t(blockIdx.x) + int64_t(loaded++) * gridDim.x;
    const LnRingRow rx = ln_ring_row<T>(a.x, a.ldx, a.n, a.h, r);
    const LnRingRow rd = ln_ring_row<T>(a.dy, a.lddy, a.n, a.h, r);
    const uint32_t bar = smem_u32(&full[put.slot]);
    const uint32_t at = smem_u32(ring) + uint32_t(put.slot) * 2u * g.slot_bytes;
    const uint32_t bytes = (rx.direct ? 0u : rx.bytes) + (rd.direct ? 0u : rd.bytes);
    put.advance(g.slots);
    if (bytes == 0) {
      mbar_arrive(bar);  // keeps the slot's phases in step
      return;
    }
    mbar_arrive_expect_tx(bar, bytes);
    if (!rx.direct) bulk_load(at, rx.begin, rx.bytes, bar);
    if (!rd.direct) bulk_load(at + g.slot_bytes, rd.begin, rd.bytes, bar);
  };
  if (t == 0) {
    for (int s = 0; s < g.slots; ++s) mbar_init(smem_u32(&full[s]), 1);
    ctl.abort = 0;
    fence_barrier_init();
    for (int s = 0; s < g.slots; ++s) issue();
  }
  float2 w[8], aw[8], ab[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = ln_both(1.0f);
    aw[i] = ab[i] = ln_both(0.0f);
  }
  if (a.w) ln_share_load<W, VN, kExact>(static_cast<const W*>(a.w), t, tpr, h, 0.0f, w);
  __syncthreads();
  const float inv_h = 1.0f / float(h);
  int buf = 0;
  int64_t r = blockIdx.x;
  float mean = a.mean[r], rstd = a.rstd[r];  // a block has two rows at least
  for (int i = 0; i < count; ++i, r += gridDim.x) {
    const int64_t next = i + 1 < count ? r + gridDim.x : r;
    const float next_mean = a.mean[next], next_rstd = a.rstd[next];
    const uint8_t* at = ring + uint32_t(get.slot) * 2u * g.slot_bytes;
    if (!wait_phase(smem_u32(&full[get.slot]), get.parity, &ctl, g.err, g.timeout_ns))
      loaded = count;  // as in the forward
    get.advance(g.slots);
    float2 xh[8], d[8];
    ln_ring_read<T, VN, kExact>(at, a.x, a.ldx, a.n, h, r, xh);
    ln_ring_read<T, VN, kExact>(at + g.slot_bytes, a.dy, a.lddy, a.n, h, r, d);
    float2 s = ln_share_grads(mean, rstd, w, xh, d, aw, ab);
    if (a.dx == nullptr) {  // the same for every thread
      __syncthreads();
      if (t == 0) issue();
    } else {
      s = ln_row_sum<false>(s, red, buf);
      if (t == 0) issue();
      ln_share_dx(make_float2(s.x * inv_h, s.y * inv_h), rstd, xh, d);
      ln_share_store<T, VN, kExact>(static_cast<T*>(a.dx) + r * a.lddx, t, tpr, h, d);
    }
    mean = next_mean;
    rstd = next_rstd;
  }
  if (t == 0 && ctl.abort) ln_ring_settle();
  if (a.part_w) ln_share_store<float, VN, kExact>(a.part_w + int64_t(blockIdx.x) * h, t, tpr, h, aw);
  if (a.part_b) ln_share_store<float, VN, kExact>(a.part_b + int64_t(blockIdx.x) * h, t, tpr, h, ab);
  ln_backward_far<T, W, VN, 1>(a, ln_sees_far(a, blockIdx.x, gridDim.x),
                               a.part_w ? a.part_w + int64_t(blockIdx.x) * h : nullptr, blockIdx.x,
                               gridDim.x);
}

// Long rows: dx row by row (two looks at x and dy) ...
template <typename T, typename W>
__global__ void __launch_bounds__(kLnLongThreads) ln_backward_long_dx_kernel(const LnBwdArgs a) {
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    T* dx = static_cast<T*>(a.dx) + r * a.lddx;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float v[1], g[1], w[1] = {1.0f};
    float2 s = make_float2(0.0f, 0.0f);
    for (int64_t c = threadIdx.x; c < a.h; c += kLnLongThreads) {
      LnIo<T, 1>::load(x + c, v);
      LnIo<T, 1>::load(dy + c, g);
      if (a.w) LnIo<W, 1>::load(static_cast<const W*>(a.w) + c, w);
      s.x += g[0] * w[0];
      s.y += g[0] * w[0] * ((v[0] - mean) * rstd);
    }
    const float m1 = float(ln_block_sum(double(s.x)) / double(a.h));
    const float m2 = float(ln_block_sum(double(s.y)) / double(a.h));
    for (int64_t c = threadIdx.x; c < a.h; c += blockDim.x) {
      LnIo<T, 1>::load(x + c, v);
      LnIo<T, 1>::load(dy + c, g);
      if (a.w) LnIo<W, 1>::load(static_cast<const W*>(a.w) + c, w);
      g[0] = rstd * (g[0] * w[0] - m1 - (v[0] - mean) * rstd * m2);
      LnIo<T, 1>::store(dx + c, g);
    }
  }
}
// ... and the weight partials column by column: block (cb, p) sums the rows
// p, p + gridDim.y, ... of its columns.
template <typename T>
__global__ void __launch_bounds__(256) ln_backward_long_dw_kernel(const LnBwdArgs a) {
  const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= a.h) return;
  float sw = 0.0f, sb = 0.0f, v[1], g[1];
  for (int64_t r = blockIdx.y; r < a.n; r += gridDim.y) {
    LnIo<T, 1>::load(static_cast<const T*>(a.x) + r * a.ldx + c, v);
    LnIo<T, 1>::load(static_cast<const T*>(a.dy) + r * a.lddy + c, g);
    sw += g[0] * ((v[0] - a.mean[r]) * a.rstd[r]);
    sb += g[0];
  }
  if (a.part_w) a.part_w[int64_t(blockIdx.y) * a.h + c] = sw;
  if (a.part_b) a.part_b[int64_t(blockIdx.y) * a.h + c] = sb;
}

// ... and the rows whose mean is large once more, a block per row of partials.
template <typename T, typename W>
__global__ void __launch_bounds__(kLnLongThreads) ln_backward_long_far_kernel(const LnBwdArgs a) {
  ln_backward_far<T, W, 1, 1>(a, ln_sees_far(a, blockIdx.x, gridDim.x),
                              a.part_w ? a.part_w + int64_t(blockIdx.x) * a.h : nullptr, blockIdx.x,
                              gridDim.x);
}

// dw and db (blockIdx.y = 0, 1) from the `parts` rows of partials, in a fixed
// order.  With no rows the sums are zero.
template <typename W>
__global__ void __launch_bounds__(32 * kLnReduceWarps)
    ln_reduce_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int parts,
                     int64_t h, W* __restrict__ dw, W* __restrict__ db) {
  __shared__ float sm[kLnReduceWarps][kLnReduceCols];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  W* out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * kLnReduceCols + lane;
  float s = 0.0f;
  if (c < h)
    for (int p = warp; p < parts; p += kLnReduceWarps) s += part[int64_t(p) * h + c];
  sm[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= h) return;
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kLnReduceWarps; ++w) t += sm[w][lane];
  float o[1] = {t};
  LnIo<W, 1>::store(out + c, o);
}

// How a row is laid over threads, 16 columns each: whole 16-byte vectors where every
// pointer, row stride and the row's length allow them, else single elements; a
// warp per row while that suffices, then one block per row.
struct LnShape {
  int vn;        // elements per vector (0: the row is too long for registers)
  int threads;   // per block
  bool warp_row;
  int rpb;       // rows per block
};

static LnShape ln_shape(int dtype, int64_t h, bool vec) {
  LnShape s{};
  s.vn = vec ? (dtype == FLCE_BF16 ? 8 : 4) : 1;
  s.warp_row = h <= kLnWarpCols;
  s.rpb = s.warp_row ? kLnWarpRows : 1;
  s.threads = s.warp_row ? 32 * kLnWarpRows : int(std::min<int64_t>(cdiv(h, 32 * kLnShare) * 32, 1024));
  if (h > kLnMaxThreads * kLnShare) s.vn = 0;
  return s;
}

// The ring's plan for rows that a block holds.
struct LnRingShape {
  int vn, threads, blocks_per_sm;
  LnRing ring;
  size_t smem;
};
static bool ln_ring_shape(int dtype, int64_t h, bool vec, int tensors, int64_t n, int sms,
                          LnRingShape* out) {
  const int esz = dtype == FLCE_F32 ? 4 : 2;
  LnRingShape s{};
  s.vn = vec ? 16 / esz : 1;
  if (h <= kLnWarpCols || h > kLnMaxThreads * kLnShare) return false;
  s.threads = int(cdiv(h, 32 * kLnShare) * 32);
  s.blocks_per_sm = std::max(1, kLnMaxThreads / s.threads);
  // fewer rows than two per block: nothing to stream
  if (n < 2 * int64_t(sms) * s.blocks_per_sm) return false;
  s.ring.slot_bytes = uint32_t((h * esz + 15) / 16 * 16 + (vec ? 0 : 16));
  const int64_t fit = int64_t(kLnRingBytes / s.blocks_per_sm) / (int64_t(s.ring.slot_bytes) * tensors);
  s.ring.slots = int(std::min<int64_t>(kLnSlots, fit));
  if (s.ring.slots < 2) return false;
  s.smem = size_t(s.ring.slots) * tensors * s.ring.slot_bytes;
  *out = s;
  return true;
}

// True when all rows of a tensor are whole, aligned 16-byte vectors.
static bool ln_vec(const void* p, int64_t ld, int64_t h, int esz) {
  return p == nullptr || (aligned(p, 16) && (ld * esz) % 16 == 0 && (h * esz) % 16 == 0);
}

// Rows of partials of the weight gradients: one per block of the backward.
static int64_t ln_parts(int64_t n, const LnShape& s) {
  const int64_t per_sm = std::max(1, kLnMaxThreads / s.threads);
  return std::min<int64_t>(cdiv(std::max<int64_t>(n, 1), s.rpb), kLnSms * per_sm);
}
// Before the pointers' alignment is known: the most any layout takes.
static int64_t ln_max_parts(int64_t n, int64_t h) {
  int64_t parts = std::min<int64_t>(std::max<int64_t>(n, 1), kLnSms);  // long rows
  for (int dtype = 0; dtype < 2; ++dtype)
    for (int vec = 0; vec < 2; ++vec) {
      parts = std::max(parts, ln_parts(n, ln_shape(dtype, h, vec != 0)));
      LnRingShape r;
      if (ln_ring_shape(dtype, h, vec != 0, 2, n, 1, &r))
        parts = std::max<int64_t>(parts, int64_t(kLnSms) * r.blocks_per_sm);
    }
  return parts;
}

static bool ln_sizes_ok(int64_t n, int64_t h) {
  return n >= 0 && h > 0 && n <= kMaxDim && h <= kMaxDim && n <= (int64_t(1) << 40) / h;
}
static bool ln_ld_ok(int64_t n, int64_t h, int64_t ld) {
  return ld >= h && ld <= (int64_t(1) << 40) / std::max<int64_t>(n, 1);
}
// n rows of `row` bytes, ld bytes apart (nothing where p is nullptr), read or written.
static Extent ln_extent(const void* p, int64_t n, int64_t row, int64_t ld, bool written) {
  return make_extent(p, {ld, 0, 0}, {p == nullptr ? 1 : n, 1, 1}, p == nullptr ? 0 : row, written);
}
// True where one of them is written over another one.
static bool ln_overlap(std::initializer_list<Extent> all) {
  for (const Extent* a = all.begin(); a != all.end(); ++a)
    for (const Extent* b = a + 1; b != all.end(); ++b)
      if ((a->written || b->written) && extents_overlap(*a, *b)) return true;
  return false;
}
static bool ln_dtype_ok(int d) { return d == FLCE_BF16 || d == FLCE_F32; }

template <typename T, typename W>
static void ln_dispatch_fwd(const LnArgs& a, const LnShape& s, int grid, cudaStream_t st) {
  constexpr int kFull = 16 / int(sizeof(T));
  if (s.vn == 0)
    ln_forward_long_kernel<T, W><<<grid, kLnLongThreads, 0, st>>>(a);
  else if (s.vn == 1 && s.warp_row)
    ln_forward_kernel<T, W, 1, true><<<grid, s.threads, 0, st>>>(a);
  else if (s.vn == 1)
    ln_forward_kernel<T, W, 1, false><<<grid, s.threads, 0, st>>>(a);
  else if (s.warp_row)
    ln_forward_kernel<T, W, kFull, true><<<grid, s.threads, 0, st>>>(a);
  else
    ln_forward_kernel<T, W, kFull, false><<<grid, s.threads, 0, st>>>(a);
}
template <typename Kern, typename Args>
static int ln_launch_ring(Kern kern, const Args& a, const LnRingShape& s, int grid, cudaStream_t st) {
  // The limit belongs to the kernel, not to the launch: always the same, so that a call
  // of another thread cannot lower it before this one launches.
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLnRingBytes) !=
      cudaSuccess)
    return FLCE_ERR_CUDA;
  kern<<<grid, s.threads, s.smem, st>>>(a, s.ring);
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
template <typename T, typename W>
static int ln_ring_fwd(const LnArgs& a, const LnRingShape& s, int grid, cudaStream_t st) {
  constexpr int kFull = 16 / int(sizeof(T));
  if (s.vn == 1) return ln_launch_ring(ln_forward_ring_kernel<T, W, 1, false>, a, s, grid, st);
  return a.h == int64_t(s.threads) * kLnShare
             ? ln_launch_ring(ln_forward_ring_kernel<T, W, kFull, true>, a, s, grid, st)
             : ln_launch_ring(ln_forward_ring_kernel<T, W, kFull, false>, a, s, grid, st);
}
template <typename T, typename W>
static int ln_ring_bwd(const LnBwdArgs& a, const LnRingShape& s, int grid, cudaStream_t st) {
  constexpr int kFull = 16 / int(sizeof(T));
  if (s.vn == 1) return ln_launch_ring(ln_backward_ring_kernel<T, W, 1, false>, a, s, grid, st);
  return a.h == int64_t(s.threads) * kLnShare
             ? ln_launch_ring(ln_backward_ring_kernel<T, W, kFull, true>, a, s, grid, st)
             : ln_launch_ring(ln_backward_ring_kernel<T, W, kFull, false>, a, s, grid, st);
}
template <typename T, typename W>
static void ln_dispatch_bwd(const LnBwdArgs& a, const LnShape& s, int grid, cudaStream_t st) {
  constexpr int kFull = 16 / int(sizeof(T));
  if (s.vn == 1 && s.warp_row)
    ln_backward_kernel<T, W, 1, true><<<grid, s.threads, 0, st>>>(a);
  else if (s.vn == 1)
    ln_backward_kernel<T, W, 1, false><<<grid, s.threads, 0, st>>>(a);
  else if (s.warp_row)
    ln_backward_kernel<T, W, kFull, true><<<grid, s.threads, 0, st>>>(a);
  else
    ln_backward_kernel<T, W, kFull, false><<<grid, s.threads, 0, st>>>(a);
}

}  // namespace flce

extern "C" size_t flce_layer_norm_workspace_size(int64_t n, int64_t h) {
  if (!ln_sizes_ok(n, h)) return 0;
  return 2 * align_up(size_t(ln_max_parts(n, h)) * size_t(h) * 4);
}

extern "C" int flce_layer_norm_forward(const void* x, int dtype, int64_t n, int64_t h, int64_t ldx,
                                       const void* weight, const void* bias, int w_dtype,
                                       float eps, void* y, int64_t ldy, float* mean, float* rstd,
                                       flce_stream_t stream) {
  NvtxRange range("flce_layer_norm_forward");
  if (!ln_sizes_ok(n, h) || !ln_ld_ok(n, h, ldx) || !ln_ld_ok(n, h, ldy) || !ln_dtype_ok(dtype) ||
      !ln_dtype_ok(w_dtype) || !(eps >= 0.0f) || !std::isfinite(eps))
    return FLCE_ERR_INVALID_ARG;
  const int esz = dtype == FLCE_F32 ? 4 : 2, wsz = w_dtype == FLCE_F32 ? 4 : 2;
  if (!aligned(weight, wsz) || !aligned(bias, wsz)) return FLCE_ERR_INVALID_ARG;
  if (n == 0) return FLCE_OK;
  if (x == nullptr || y == nullptr || !aligned(x, esz) || !aligned(y, esz) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return FLCE_ERR_INVALID_ARG;
  if (ln_overlap({ln_extent(x, n, h * esz, ldx * esz, false), ln_extent(weight, 1, h * wsz, 0, false),
                  ln_extent(bias, 1, h * wsz, 0, false), ln_extent(y, n, h * esz, ldy * esz, true),
                  ln_extent(mean, 1, n * 4, 0, true), ln_extent(rstd, 1, n * 4, 0, true)}))
    return FLCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const LnShape s = ln_shape(dtype, h, ln_vec(x, ldx, h, esz) && ln_vec(y, ldy, h, esz) &&
                                           aligned(weight, 16) && aligned(bias, 16));
  const LnArgs a{x, ldx, weight, bias, n, h, eps, y, ldy, mean, rstd};
  LnRingShape rs;
  if (ln_ring_shape(dtype, h, s.vn > 1, 1, n, dev->num_sms, &rs)) {
    rs.ring.err = dev->err;
    rs.ring.timeout_ns = kDefaultTimeoutNs;
    const int grid = dev->num_sms * rs.blocks_per_sm;
    LaunchScope scope(KF_LN_FWD, 0.0, double(n) * double(h) * 2.0 * esz + 8.0 * double(n), cs);
    if (dtype == FLCE_BF16)
      return w_dtype == FLCE_BF16 ? ln_ring_fwd<__nv_bfloat16, __nv_bfloat16>(a, rs, grid, cs)
                                  : ln_ring_fwd<__nv_bfloat16, float>(a, rs, grid, cs);
    return w_dtype == FLCE_BF16 ? ln_ring_fwd<float, __nv_bfloat16>(a, rs, grid, cs)
                                : ln_ring_fwd<float, float>(a, rs, grid, cs);
  }
  const int64_t per_sm = s.vn == 0 ? 2 : std::max(1, 2048 / s.threads);
  const int grid = int(std::min<int64_t>(cdiv(n, s.vn == 0 ? 1 : s.rpb), dev->num_sms * per_sm));
  LaunchScope scope(KF_LN_FWD, 0.0, double(n) * double(h) * 2.0 * esz + 8.0 * double(n), cs);
  if (dtype == FLCE_BF16 && w_dtype == FLCE_BF16)
    ln_dispatch_fwd<__nv_bfloat16, __nv_bfloat16>(a, s, grid, cs);
  else if (dtype == FLCE_BF16)
    ln_dispatch_fwd<__nv_bfloat16, float>(a, s, grid, cs);
  else if (w_dtype == FLCE_BF16)
    ln_dispatch_fwd<float, __nv_bfloat16>(a, s, grid, cs);
  else
    ln_dispatch_fwd<float, float>(a, s, grid, cs);
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

extern "C" int flce_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int dtype,
                                        int64_t n, int64_t h, int64_t ldx, const void* weight,
                                        int w_dtype, const float* mean, const float* rstd,
                                        void* dx, int64_t lddx, void* dweight, void* dbias,
                                        void* workspace, size_t ws_bytes, flce_stream_t stream) {
  NvtxRange range("flce_layer_norm_backward");
  if (!ln_sizes_ok(n, h) || !ln_ld_ok(n, h, ldx) || !ln_ld_ok(n, h, lddy) ||
      (dx != nullptr && !ln_ld_ok(n, h, lddx)) || !ln_dtype_ok(dtype) || !ln_dtype_ok(w_dtype))
    return FLCE_ERR_INVALID_ARG;
  const int esz = dtype == FLCE_F32 ? 4 : 2, wsz = w_dtype == FLCE_F32 ? 4 : 2;
  if (!aligned(weight, wsz) || !aligned(dweight, wsz) || !aligned(dbias, wsz) || !aligned(dx, esz))
    return FLCE_ERR_INVALID_ARG;
  if (n > 0 && (x == nullptr || dy == nullptr || mean == nullptr || rstd == nullptr ||
                !aligned(x, esz) || !aligned(dy, esz) || !aligned(mean, 4) || !aligned(rstd, 4)))
    return FLCE_ERR_INVALID_ARG;
  const bool params = dweight != nullptr || dbias != nullptr;
  const size_t half = align_up(size_t(ln_max_parts(n, h)) * size_t(h) * 4);
  if (params && (workspace == nullptr || !aligned(workspace, 16) || ws_bytes < 2 * half))
    return FLCE_ERR_WORKSPACE;
  if (!params && (dx == nullptr || n == 0)) return FLCE_OK;
  if (ln_overlap({ln_extent(dy, n, h * esz, lddy * esz, false), ln_extent(x, n, h * esz, ldx * esz, false),
                  ln_extent(weight, 1, h * wsz, 0, false), ln_extent(mean, 1, n * 4, 0, false),
                  ln_extent(rstd, 1, n * 4, 0, false), ln_extent(dx, n, h * esz, lddx * esz, true),
                  ln_extent(dweight, 1, h * wsz, 0, true), ln_extent(dbias, 1, h * wsz, 0, true),
                  ln_extent(params ? workspace : nullptr, 1, int64_t(2 * half), 0, true)}))
    return FLCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  float* part_w = dweight ? static_cast<float*>(workspace) : nullptr;
  float* part_b =
      dbias ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + half) : nullptr;
  int parts = 0;
  if (n > 0) {
    const LnShape s =
        ln_shape(dtype, h, ln_vec(x, ldx, h, esz) && ln_vec(dy, lddy, h, esz) &&
                               ln_vec(dx, lddx, h, esz) && aligned(weight, 16));
    const LnBwdArgs a{dy, lddy, x, ldx, weight, mean, rstd, n, h, dx, lddx, part_w, part_b};
    const double bytes = double(n) * double(h) * 3.0 * esz + 8.0 * double(n);
    LnRingShape rs;
    if (ln_ring_shape(dtype, h, s.vn > 1, 2, n, dev->num_sms, &rs) &&
        dev->num_sms <= kLnSms) {
      rs.ring.err = dev->err;
      rs.ring.timeout_ns = kDefaultTimeoutNs;
      parts = dev->num_sms * rs.blocks_per_sm;
      LaunchScope scope(KF_LN_BWD, 0.0, bytes, cs);
      int rc;
      if (dtype == FLCE_BF16)
        rc = w_dtype == FLCE_BF16 ? ln_ring_bwd<__nv_bfloat16, __nv_bfloat16>(a, rs, parts, cs)
                                  : ln_ring_bwd<__nv_bfloat16, float>(a, rs, parts, cs);
      else
        rc = w_dtype == FLCE_BF16 ? ln_ring_bwd<float, __nv_bfloat16>(a, rs, parts, cs)
                                  : ln_ring_bwd<float, float>(a, rs, parts, cs);
      if (rc != FLCE_OK) return rc;
    } else if (s.vn == 0) {
      if (dx != nullptr) {
        const int grid = int(std::min<int64_t>(n, int64_t(dev->num_sms) * 2));
        LaunchScope scope(KF_LN_BWD, 0.0, bytes, cs);
        if (dtype == FLCE_BF16 && w_dtype == FLCE_BF16)
          ln_backward_long_dx_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kLnLongThreads, 0, cs>>>(a);
        else if (dtype == FLCE_BF16)
          ln_backward_long_dx_kernel<__nv_bfloat16, float><<<grid, kLnLongThreads, 0, cs>>>(a);
        else if (w_dtype == FLCE_BF16)
          ln_backward_long_dx_kernel<float, __nv_bfloat16><<<grid, kLnLongThreads, 0, cs>>>(a);
        else
          ln_backward_long_dx_kernel<float, float><<<grid, kLnLongThreads, 0, cs>>>(a);
        if (cudaGetLastError() != cudaSuccess) return FLCE_ERR_CUDA;
      }
      if (params) {
        parts = int(std::min<int64_t>(n, kLnSms));
        const dim3 grid(unsigned(cdiv(h, 256)), unsigned(parts));
        LaunchScope scope(KF_LN_BWD, 0.0, bytes, cs);
        if (dtype == FLCE_BF16)
          ln_backward_long_dw_kernel<__nv_bfloat16><<<grid, 256, 0, cs>>>(a);
        else
          ln_backward_long_dw_kernel<float><<<grid, 256, 0, cs>>>(a);
        if (cudaGetLastError() != cudaSuccess) return FLCE_ERR_CUDA;
      }
      if (dx != nullptr || dweight != nullptr) {
        const int grid = int(std::min<int64_t>(n, kLnSms));  // as many as rows of partials
        LaunchScope scope(KF_LN_BWD, 0.0, 8.0 * double(n), cs);
        if (dtype == FLCE_BF16 && w_dtype == FLCE_BF16)
          ln_backward_long_far_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kLnLongThreads, 0, cs>>>(a);
        else if (dtype == FLCE_BF16)
          ln_backward_long_far_kernel<__nv_bfloat16, float><<<grid, kLnLongThreads, 0, cs>>>(a);
        else if (w_dtype == FLCE_BF16)
          ln_backward_long_far_kernel<float, __nv_bfloat16><<<grid, kLnLongThreads, 0, cs>>>(a);
        else
          ln_backward_long_far_kernel<float, float><<<grid, kLnLongThreads, 0, cs>>>(a);
      }
    } else {
      parts = int(ln_parts(n, s));
      LaunchScope scope(KF_LN_BWD, 0.0, bytes, cs);
      if (dtype == FLCE_BF16 && w_dtype == FLCE_BF16)
        ln_dispatch_bwd<__nv_bfloat16, __nv_bfloat16>(a, s, parts, cs);
      else if (dtype == FLCE_BF16)
        ln_dispatch_bwd<__nv_bfloat16, float>(a, s, parts, cs);
      else if (w_dtype == FLCE_BF16)
        ln_dispatch_bwd<float, __nv_bfloat16>(a, s, parts, cs);
      else
        ln_dispatch_bwd<float, float>(a, s, parts, cs);
    }
    if (cudaGetLastError() != cudaSuccess) return FLCE_ERR_CUDA;
  }
  if (params) {
    const dim3 grid(unsigned(cdiv(h, kLnReduceCols)), 2);
    LaunchScope scope(KF_LN_REDUCE, 0.0, 8.0 * double(parts) * double(h), cs);
    const dim3 block(32 * kLnReduceWarps);
    return w_dtype == FLCE_BF16
               ? launch_dependent(ln_reduce_kernel<__nv_bfloat16>, grid, block, 0, cs, part_w, part_b,
                                  parts, h, static_cast<__nv_bfloat16*>(dweight),
                                  static_cast<__nv_bfloat16*>(dbias))
               : launch_dependent(ln_reduce_kernel<float>, grid, block, 0, cs, part_w, part_b, parts, h,
                                  static_cast<float*>(dweight), static_cast<float*>(dbias));
  }
  return FLCE_OK;
}
