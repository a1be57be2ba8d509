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
// variance takes its second look at it (centred, so a large mean costs no
// digits).  A thread owns the same columns of every row it sees: the weights
// stay in its registers, and so do its shares of dw and db, which leave the
// block once, as one row of FP32 partials per block; a second kernel adds the
// partials in a fixed order (no atomics: the same inputs give the same bits).
#pragma once

#include <cuda_bf16.h>

#include "epilogues.cuh"

namespace flce {

constexpr int kLnMaxThreads = 512;      // threads per row with the short per-thread share
constexpr int kLnWarpRows = 4;          // rows (warps) per block when a warp holds a row
constexpr int kLnRowThreads = 1024;     // resident threads per SM the grid aims at
constexpr int kLnSms = 148;             // blocks per "one block per SM" of the partials' layout
constexpr int kLnReduceCols = 32;       // columns per block of the partials' sum
constexpr int kLnReduceWarps = 16;

// Threads of a block whose threads hold `share` columns each, at most: the
// backward keeps five values per column in registers.
__host__ __device__ constexpr int ln_block(int share, bool warp_row) {
  return warp_row ? 32 * kLnWarpRows : (share > 8 ? kLnMaxThreads : 2 * kLnMaxThreads);
}

// N consecutive elements at a time, as floats.  The address is aligned to the
// vector's size (16 bytes at most per access).
template <typename T, int N>
struct LnIo;
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
    } else if constexpr (N == 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      x[0] = __uint_as_float(w << 16);
      x[1] = __uint_as_float(w & 0xffff0000u);
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
    } else if constexpr (N == 2) {
      *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x[0], x[1]);
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
    } else if constexpr (N == 2) {
      const float2 w = *reinterpret_cast<const float2*>(p);
      x[0] = w.x;
      x[1] = w.y;
    } else {
      x[0] = *p;
    }
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else if constexpr (N == 2) {
      *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    } else {
      *p = x[0];
    }
  }
};

// Sum of a pair over a row's threads: a warp, or the whole block through
// shared memory.  `buf` alternates between calls, so one barrier per call is
// enough: a buffer is written again only after every thread passed the barrier
// of the call in between.
template <bool kWarpRow>
__device__ __forceinline__ float2 ln_row_sum(float2 v, float2 (*red)[32], int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (kWarpRow) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = v;
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int w = 0; w < warps; ++w) {
    s.x += red[buf][w].x;
    s.y += red[buf][w].y;
  }
  buf ^= 1;
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

// kWarpRow: a warp holds a row (no barrier); else the block does.  A thread's
// share is NV vectors of VN elements, `tpr` vectors apart.
template <typename T, typename W, int VN, int NV, bool kWarpRow>
__global__ void __launch_bounds__(ln_block(VN * NV, kWarpRow))
    ln_forward_kernel(const LnArgs a) {
  __shared__ float2 red[2][32];
  const int tpr = kWarpRow ? 32 : int(blockDim.x);
  const int t = kWarpRow ? int(threadIdx.x & 31) : int(threadIdx.x);
  const int rpb = kWarpRow ? int(blockDim.x >> 5) : 1;
  const int64_t r0 = int64_t(blockIdx.x) * rpb + (kWarpRow ? int(threadIdx.x >> 5) : 0);
  const int64_t step = int64_t(gridDim.x) * rpb;
  const float inv_h = 1.0f / float(a.h);
  int buf = 0;
  for (int64_t r = r0; r < a.n; r += step) {  // uniform over the threads that share a row
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    float v[NV][VN];
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t(i) * tpr + t) * VN;
      if (c < a.h) {
        LnIo<T, VN>::load(x + c, v[i]);
#pragma unroll
        for (int j = 0; j < VN; ++j) s.x += v[i][j];
      }
    }
    const float mean = ln_row_sum<kWarpRow>(s, red, buf).x * inv_h;
    s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t(i) * tpr + t) * VN;
      if (c < a.h) {
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          v[i][j] -= mean;
          s.x += v[i][j] * v[i][j];
        }
      }
    }
    const float rstd = 1.0f / sqrtf(ln_row_sum<kWarpRow>(s, red, buf).x * inv_h + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    T* y = static_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t(i) * tpr + t) * VN;
      if (c < a.h) {
        float w[VN], b[VN];
        if (a.w) LnIo<W, VN>::load(static_cast<const W*>(a.w) + c, w);
        if (a.b) LnIo<W, VN>::load(static_cast<const W*>(a.b) + c, b);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          float o = v[i][j] * rstd;
          if (a.w) o *= w[j];
          if (a.b) o += b[j];
          v[i][j] = o;
        }
        LnIo<T, VN>::store(y + c, v[i]);
      }
    }
  }
}

// Rows too long for the registers of one block: three looks at the row, the
// later ones from L2.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) ln_forward_long_kernel(const LnArgs a) {
  __shared__ float2 red[2][32];
  int buf = 0;
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.y) + r * a.ldy;
    float2 s = make_float2(0.0f, 0.0f);
    float v[1], w[1], b[1];
    for (int64_t c = threadIdx.x; c < a.h; c += blockDim.x) {
      LnIo<T, 1>::load(x + c, v);
      s.x += v[0];
    }
    const float mean = ln_row_sum<false>(s, red, buf).x / float(a.h);
    s = make_float2(0.0f, 0.0f);
    for (int64_t c = threadIdx.x; c < a.h; c += blockDim.x) {
      LnIo<T, 1>::load(x + c, v);
      s.x += (v[0] - mean) * (v[0] - mean);
    }
    const float rstd = 1.0f / sqrtf(ln_row_sum<false>(s, red, buf).x / float(a.h) + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    for (int64_t c = threadIdx.x; c < a.h; c += blockDim.x) {
      LnIo<T, 1>::load(x + c, v);
      v[0] = (v[0] - mean) * rstd;
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

template <typename T, typename W, int VN, int NV, bool kWarpRow>
__global__ void __launch_bounds__(ln_block(VN * NV, kWarpRow))
    ln_backward_kernel(const LnBwdArgs a) {
  __shared__ float2 red[2][32];
  const int tpr = kWarpRow ? 32 : int(blockDim.x);
  const int t = kWarpRow ? int(threadIdx.x & 31) : int(threadIdx.x);
  const int rpb = kWarpRow ? int(blockDim.x >> 5) : 1;
  const int64_t r0 = int64_t(blockIdx.x) * rpb + (kWarpRow ? int(threadIdx.x >> 5) : 0);
  const int64_t step = int64_t(gridDim.x) * rpb;
  const float inv_h = 1.0f / float(a.h);
  int buf = 0;
  float w[NV][VN], aw[NV][VN], ab[NV][VN];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t(i) * tpr + t) * VN;
#pragma unroll
    for (int j = 0; j < VN; ++j) {
      w[i][j] = 1.0f;
      aw[i][j] = 0.0f;
      ab[i][j] = 0.0f;
    }
    if (a.w && c < a.h) LnIo<W, VN>::load(static_cast<const W*>(a.w) + c, w[i]);
  }
  for (int64_t r = r0; r < a.n; r += step) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float xh[NV][VN], g[NV][VN];
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t(i) * tpr + t) * VN;
      if (c < a.h) {
        LnIo<T, VN>::load(x + c, xh[i]);
        LnIo<T, VN>::load(dy + c, g[i]);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          xh[i][j] = (xh[i][j] - mean) * rstd;
          ab[i][j] += g[i][j];
          aw[i][j] += g[i][j] * xh[i][j];
          g[i][j] *= w[i][j];
          s.x += g[i][j];
          s.y += g[i][j] * xh[i][j];
        }
      }
    }
    if (a.dx == nullptr) continue;  // the same for every thread
    s = ln_row_sum<kWarpRow>(s, red, buf);
    const float m1 = s.x * inv_h, m2 = s.y * inv_h;
    T* dx = static_cast<T*>(a.dx) + r * a.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t(i) * tpr + t) * VN;
      if (c < a.h) {
#pragma unroll
        for (int j = 0; j < VN; ++j) g[i][j] = rstd * (g[i][j] - m1 - xh[i][j] * m2);
        LnIo<T, VN>::store(dx + c, g[i]);
      }
    }
  }
  if (a.part_w == nullptr && a.part_b == nullptr) return;
  // The block's partial row: the block's only row group, or the sum over its
  // warps, one warp after the other (each column stays with one lane).
  for (int turn = 0; turn < rpb; ++turn) {
    if (kWarpRow) __syncthreads();
    if (kWarpRow && int(threadIdx.x >> 5) != turn) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t(i) * tpr + t) * VN;
      if (c >= a.h) continue;
#pragma unroll
      for (int j = 0; j < VN; ++j) {
        const int64_t at = int64_t(blockIdx.x) * a.h + c + j;
        if (a.part_w) a.part_w[at] = turn == 0 ? aw[i][j] : a.part_w[at] + aw[i][j];
        if (a.part_b) a.part_b[at] = turn == 0 ? ab[i][j] : a.part_b[at] + ab[i][j];
      }
    }
  }
}

// Long rows: dx row by row (two looks at x and dy) ...
template <typename T, typename W>
__global__ void __launch_bounds__(1024) ln_backward_long_dx_kernel(const LnBwdArgs a) {
  __shared__ float2 red[2][32];
  int buf = 0;
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    T* dx = static_cast<T*>(a.dx) + r * a.lddx;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float v[1], g[1], w[1] = {1.0f};
    float2 s = make_float2(0.0f, 0.0f);
    for (int64_t c = threadIdx.x; c < a.h; c += blockDim.x) {
      LnIo<T, 1>::load(x + c, v);
      LnIo<T, 1>::load(dy + c, g);
      if (a.w) LnIo<W, 1>::load(static_cast<const W*>(a.w) + c, w);
      s.x += g[0] * w[0];
      s.y += g[0] * w[0] * ((v[0] - mean) * rstd);
    }
    s = ln_row_sum<false>(s, red, buf);
    const float m1 = s.x / float(a.h), m2 = s.y / float(a.h);
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

// How a row is laid over threads: the widest vector that every pointer and row
// stride allows, then a warp per row while a lane's share is at most NV = 2
// vectors (8 narrow ones), then one block per row.
struct LnShape {
  int vn;        // elements per vector (0: the row is too long for registers)
  int nv;        // vectors per thread
  int threads;   // per block
  bool warp_row;
  int rpb;       // rows per block
};

static LnShape ln_shape(int dtype, int64_t h, int max_vec) {
  const int full = dtype == FLCE_BF16 ? 8 : 4;
  LnShape s{};
  s.vn = max_vec >= full ? full : (dtype == FLCE_BF16 && max_vec >= 2 ? 2 : 1);
  const int64_t vecs = (h + s.vn - 1) / s.vn;
  const bool wide = s.vn == full;
  s.nv = wide ? 2 : 8;
  if (vecs <= 32 * s.nv) {
    s.warp_row = true;
    s.threads = 32 * kLnWarpRows;
    s.rpb = kLnWarpRows;
    return s;
  }
  if (wide && vecs > int64_t(kLnMaxThreads) * s.nv) s.nv = 4;
  const int64_t t = (vecs + s.nv - 1) / s.nv;
  s.rpb = 1;
  s.threads = int((t + 31) / 32 * 32);
  if (t > ln_block(s.nv * s.vn, false)) s.vn = 0;
  return s;
}

// Largest vector (elements, a power of two) that all rows of a tensor allow.
static int ln_vec(const void* p, int64_t ld, int64_t h, int esz) {
  if (p == nullptr) return 8;
  int v = 16 / esz;
  while (v > 1 && ((reinterpret_cast<uintptr_t>(p) % (size_t(v) * esz)) != 0 || ld % v != 0 || h % v != 0))
    v >>= 1;
  return v;
}
static int ln_vec_w(const void* p, int esz) {  // the weights: one row, up to 8 elements as 16-byte loads
  if (p == nullptr) return 8;
  int v = 8;
  while (v > 1 && (reinterpret_cast<uintptr_t>(p) % size_t(std::min(16, v * esz))) != 0) v >>= 1;
  return v;
}

// Rows of partials of the weight gradients: one per block of the backward.
static int64_t ln_parts(int64_t n, const LnShape& s) {
  const int64_t per_sm = std::max<int64_t>(1, kLnRowThreads / std::max(s.threads, 1));
  return std::max<int64_t>(1, std::min<int64_t>(cdiv(std::max<int64_t>(n, 1), std::max(s.rpb, 1)),
                                                kLnSms * per_sm));
}
// Before the pointers' alignment is known: the most any layout takes.
static int64_t ln_max_parts(int64_t n, int64_t h) {
  int64_t parts = std::min<int64_t>(std::max<int64_t>(n, 1), kLnSms);  // long rows
  for (int dtype = 0; dtype < 2; ++dtype)
    for (int v = 1; v <= 8; v *= 2) parts = std::max(parts, ln_parts(n, ln_shape(dtype, h, v)));
  return parts;
}

static bool ln_sizes_ok(int64_t n, int64_t h) {
  return n >= 0 && h > 0 && n <= kMaxDim && h <= kMaxDim && n <= (int64_t(1) << 40) / h;
}
static bool ln_ld_ok(int64_t n, int64_t h, int64_t ld) {
  return ld >= h && ld <= (int64_t(1) << 40) / std::max<int64_t>(n, 1);
}
static bool ln_dtype_ok(int d) { return d == FLCE_BF16 || d == FLCE_F32; }

template <typename T, typename W, int VN, int NV>
static void ln_launch_fwd(const LnArgs& a, const LnShape& s, int grid, cudaStream_t st) {
  if constexpr (NV != 4) {  // the warp-per-row layouts
    if (s.warp_row) {
      ln_forward_kernel<T, W, VN, NV, true><<<grid, s.threads, 0, st>>>(a);
      return;
    }
  }
  ln_forward_kernel<T, W, VN, NV, false><<<grid, s.threads, 0, st>>>(a);
}
template <typename T, typename W>
static void ln_dispatch_fwd(const LnArgs& a, const LnShape& s, int grid, cudaStream_t st) {
  constexpr int kFull = 16 / int(sizeof(T));
  if (s.vn == 0)
    ln_forward_long_kernel<T, W><<<grid, 1024, 0, st>>>(a);
  else if (s.vn == kFull && s.nv == 2)
    ln_launch_fwd<T, W, kFull, 2>(a, s, grid, st);
  else if (s.vn == kFull)
    ln_launch_fwd<T, W, kFull, 4>(a, s, grid, st);
  else if (sizeof(T) == 2 && s.vn == 2)
    ln_launch_fwd<T, W, 2, 8>(a, s, grid, st);
  else
    ln_launch_fwd<T, W, 1, 8>(a, s, grid, st);
}
template <typename T, typename W, int VN, int NV>
static void ln_launch_bwd(const LnBwdArgs& a, const LnShape& s, int grid, cudaStream_t st) {
  if constexpr (NV != 4) {  // the warp-per-row layouts
    if (s.warp_row) {
      ln_backward_kernel<T, W, VN, NV, true><<<grid, s.threads, 0, st>>>(a);
      return;
    }
  }
  ln_backward_kernel<T, W, VN, NV, false><<<grid, s.threads, 0, st>>>(a);
}
template <typename T, typename W>
static void ln_dispatch_bwd(const LnBwdArgs& a, const LnShape& s, int grid, cudaStream_t st) {
  constexpr int kFull = 16 / int(sizeof(T));
  if (s.vn == kFull && s.nv == 2)
    ln_launch_bwd<T, W, kFull, 2>(a, s, grid, st);
  else if (s.vn == kFull)
    ln_launch_bwd<T, W, kFull, 4>(a, s, grid, st);
  else if (sizeof(T) == 2 && s.vn == 2)
    ln_launch_bwd<T, W, 2, 8>(a, s, grid, st);
  else
    ln_launch_bwd<T, W, 1, 8>(a, s, grid, st);
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
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const LnShape s = ln_shape(dtype, h, std::min({ln_vec(x, ldx, h, esz), ln_vec(y, ldy, h, esz),
                                                 ln_vec_w(weight, wsz), ln_vec_w(bias, wsz)}));
  const LnArgs a{x, ldx, weight, bias, n, h, eps, y, ldy, mean, rstd};
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
        ln_shape(dtype, h, std::min({ln_vec(x, ldx, h, esz), ln_vec(dy, lddy, h, esz),
                                     ln_vec(dx, lddx, h, esz), ln_vec_w(weight, wsz)}));
    const LnBwdArgs a{dy, lddy, x, ldx, weight, mean, rstd, n, h, dx, lddx, part_w, part_b};
    const double bytes = double(n) * double(h) * 3.0 * esz + 8.0 * double(n);
    if (s.vn == 0) {
      if (dx != nullptr) {
        const int grid = int(std::min<int64_t>(n, int64_t(dev->num_sms) * 2));
        LaunchScope scope(KF_LN_BWD, 0.0, bytes, cs);
        if (dtype == FLCE_BF16 && w_dtype == FLCE_BF16)
          ln_backward_long_dx_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 1024, 0, cs>>>(a);
        else if (dtype == FLCE_BF16)
          ln_backward_long_dx_kernel<__nv_bfloat16, float><<<grid, 1024, 0, cs>>>(a);
        else if (w_dtype == FLCE_BF16)
          ln_backward_long_dx_kernel<float, __nv_bfloat16><<<grid, 1024, 0, cs>>>(a);
        else
          ln_backward_long_dx_kernel<float, float><<<grid, 1024, 0, cs>>>(a);
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
    if (w_dtype == FLCE_BF16)
      ln_reduce_kernel<__nv_bfloat16><<<grid, 32 * kLnReduceWarps, 0, cs>>>(
          part_w, part_b, parts, h, static_cast<__nv_bfloat16*>(dweight),
          static_cast<__nv_bfloat16*>(dbias));
    else
      ln_reduce_kernel<float><<<grid, 32 * kLnReduceWarps, 0, cs>>>(
          part_w, part_b, parts, h, static_cast<float*>(dweight), static_cast<float*>(dbias));
    if (cudaGetLastError() != cudaSuccess) return FLCE_ERR_CUDA;
  }
  return FLCE_OK;
}
