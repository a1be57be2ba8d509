// mxfp4.cuh - microscaled 4-bit floating point (MXFP4): every 32 consecutive
// elements of a row share a power of two, and each element is an E2M1 number
// (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times it.
//
//   amax  = max |x| of the block
//   e     = floor(log2 amax) - 2, at least -127     (E2M1's largest exponent is 2)
//   code  = E2M1 nearest to x / 2^e, ties to the even code, saturating at 6
//   scale = e + 127 (E8M0); 255 = NaN when the block holds an Inf or a NaN
//
// Dividing by a power of two is exact and the nearest code is unique, so the
// codes are a function of the input alone, whatever computes them.
//
// Layout in memory, as the tensor core reads it, so that a stage of the product
// is a few contiguous copies (row-major codes, read in 128-byte pieces a row's
// pitch apart, took 79 us where these took 73 in the product's first form).
// Codes: tiles of 128 rows x 256 columns, 16 KB, the tiles of 128 rows one after
// the other along the columns.  Inside a tile a row is 128 bytes, element 2i in
// the low half of byte i, and the 16-byte piece q of row r sits at q ^ (r % 8)
// (the 128-byte swizzle).  Columns behind the last one are zeros.
// Scales: tiles of 128 rows x 4 blocks, 512 bytes, in the same order, two per
// tile of codes; the scale of row r, block k sits at (r % 32) * 16 + (r / 32) * 4
// + k, which tensor memory wants (32 lanes x 16 bytes).  Blocks behind a row's
// last one have scale 127 (up to a multiple of 8 blocks).
// Rows behind the last one are left as they were; nothing reads their products.
//
// Both kernels are bound by HBM (quantising BF16 reads 2 bytes and writes
// 17/32 of one per element).  Four threads share a block: each converts 8
// elements (16 bytes of BF16, 32 of FP32), the block's maximum takes two
// shuffles, and 4 bytes of codes per thread make whole sectors per warp.
// 128256 x 4096 BF16: 220 us to quantise, 214 us to dequantise (6.1 and 6.2 TB/s,
// 94% and 96% of the copy bandwidth).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>

#include "epilogues.cuh"
#include "layer_norm.cuh"  // LnIo: typed vector loads and stores

namespace flce {

constexpr int kMxBlock = 32;          // elements per scale
constexpr int kMxTileRows = 128;      // rows of a scale tile
constexpr int kMxTileBlocks = 4;      // column blocks of a scale tile
constexpr int kMxTileBytes = kMxTileRows * kMxTileBlocks;
constexpr int kMxTileCols = 256;      // columns of a tile of codes
constexpr int kMxCodeBytes = kMxTileRows * kMxTileCols / 2;
constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;          // vectors of 8 elements in flight per thread

__host__ __device__ __forceinline__ int64_t mx_blocks(int64_t cols) {
  return (cols + kMxBlock - 1) / kMxBlock;
}
// Tiles of codes (256 columns) along a row; twice as many tiles of scales.
__host__ __device__ __forceinline__ int64_t mx_ctiles(int64_t cols) {
  return (cols + kMxTileCols - 1) / kMxTileCols;
}
__host__ __device__ __forceinline__ int64_t mx_ktiles(int64_t cols) { return 2 * mx_ctiles(cols); }

struct MxQuantArgs {
  const void* x;
  int64_t rows, cols, ld;
  uint8_t* codes;
  uint8_t* scales;
  int64_t segs;  // pieces a row is cut into, a warp each (whole tiles of 256 columns)
};

// 8 elements as they were loaded, and what the conversion needs of them: the
// largest magnitude as bits (NaN and Inf order above every number), and the
// scaled values.
template <typename T>
struct MxVec;
template <>
struct MxVec<__nv_bfloat16> {
  uint32_t u[4];
  __device__ __forceinline__ void zero() { u[0] = u[1] = u[2] = u[3] = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    u[0] = w.x;
    u[1] = w.y;
    u[2] = w.z;
    u[3] = w.w;
  }
  // Over the four lanes of the block: two 16-bit magnitudes at a time.
  __device__ __forceinline__ int exponent() const {
    uint32_t m = u[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, u[i] & 0x7fff7fffu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return int(max(m >> 16, m & 0xffffu) >> 7);
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
};
template <>
struct MxVec<float> {
  float x[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  }
  __device__ __forceinline__ void load(const float* p) { LnIo<float, 8>::load(p, x); }
  __device__ __forceinline__ int exponent() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return int(m >> 23);
  }
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(x[2 * i], x[2 * i + 1]); }
};

// A warp takes a piece of a row, a tile's 256 columns (32 vectors of 8) per step:
// lane l holds columns 8 l.. of the tile, so its places in the tiles of codes
// and scales only move on by whole tiles.
// kVec: rows start on 16 bytes and hold whole vectors of 8.
// kU: tiles per step.
template <typename T, bool kVec, int kU>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const MxQuantArgs a) {
  constexpr bool kStage = !kVec;
  __shared__ __align__(16) T
      stage_s[kStage ? kMxThreads / 32 : 1][kStage ? kU : 1][kStage ? kMxTileCols : 8];
  grid_launch_dependents();  // the product's set-up; it waits for this grid's end itself
  const int lane = threadIdx.x & 31;
  const int64_t warps = int64_t(gridDim.x) * (kMxThreads / 32);
  const int64_t ctiles = mx_ctiles(a.cols);
  const int64_t per = (ctiles + a.segs - 1) / a.segs;
  for (int64_t unit = int64_t(blockIdx.x) * (kMxThreads / 32) + (threadIdx.x >> 5);
       unit < a.rows * a.segs; unit += warps) {
    const int64_t r = a.segs == 1 ? unit : unit / a.segs;
    const int64_t s0 = (unit - r * a.segs) * per, s1 = min(ctiles, s0 + per);
    const int tr = int(r % kMxTileRows);
    const T* src = static_cast<const T*>(a.x) + r * a.ld + s0 * kMxTileCols + lane * 8;
    const int64_t tile = (r / kMxTileRows) * ctiles + s0;
    uint8_t* code = a.codes + tile * kMxCodeBytes + tr * 128 + (((lane >> 2) ^ (tr & 7)) << 4) +
                    (lane & 3) * 4;
    uint8_t* scale = a.scales + tile * (2 * kMxTileBytes) + (lane >> 4) * kMxTileBytes +
                     (tr % 32) * 16 + (tr / 32) * 4;
    int64_t left = a.cols - s0 * kMxTileCols - lane * 8;  // columns from this lane's first on
    for (int64_t s = s0; s < s1; s += kU) {
      MxVec<T> v[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        v[i].zero();
        if constexpr (kStage) {
          // 256 neighbours coalesced, then 8 to each lane through shared memory (7335 x
          // 4930: 75 -> 40 us in FP32, 41 -> 36 us in BF16 against shifted 16-byte loads).
          // Predicates, no branches, so that all of the batch's loads go out at once.
          T* stage = stage_s[threadIdx.x >> 5][i];
          const int64_t rest = left + lane * 8 - i * kMxTileCols;  // columns from the tile's first on
          const T* from = src - lane * 8 + i * kMxTileCols;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            stage[j * 32 + lane] =
                s + i < s1 && j * 32 + lane < rest ? from[j * 32 + lane] : T(0.0f);
        } else if (s + i < s1 && left > i * kMxTileCols) {
          v[i].load(src + i * kMxTileCols);
        }
      }
      if constexpr (kStage) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kU; ++i) v[i].load(stage_s[threadIdx.x >> 5][i] + lane * 8);
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        if (s + i >= s1) break;  // the same for the whole warp
        const int ex = v[i].exponent();
        const int sc = ex == 255 ? 255 : max(ex - 2, 0);
        const float inv = __uint_as_float(static_cast<uint32_t>(ex == 255 ? 127 : 254 - sc) << 23);
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(
                   __fmul2_rn(v[i].pair(j), make_float2(inv, inv)), __NV_E2M1, cudaRoundNearest))
               << (8 * j);
        *reinterpret_cast<uint32_t*>(code + i * kMxCodeBytes) = w;
        // Four blocks' scales as one word, written by the first of 16 lanes.  A
        // block starts at the first of its four lanes.
        const bool in = left + (lane & 3) * 8 > i * kMxTileCols;
        uint32_t word = (in ? static_cast<uint32_t>(sc) : 127u) << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scale + i * (2 * kMxTileBytes)) = word;
      }
      src += kU * kMxTileCols;
      code += kU * kMxCodeBytes;
      scale += kU * 2 * kMxTileBytes;
      left -= kU * kMxTileCols;
    }
  }
}

struct MxDequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, ld;
  void* out;
  int64_t segs;
};

// 2^(sc - 127); 255 is NaN.  (2^-127 is subnormal in FP32.)
__device__ __forceinline__ float mx_scale(uint32_t sc) {
  return sc == 255u ? __uint_as_float(0x7fc00000u)
                    : __uint_as_float(sc == 0u ? 0x00400000u : sc << 23);
}

template <typename T, bool kVec, int kU>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(const MxDequantArgs a) {
  // Rows of any alignment: a tile's 256 values change hands through shared memory,
  // so that a warp stores 32 neighbours at a time.
  __shared__ __align__(16) T stage_s[kVec ? 1 : kMxThreads / 32][kVec ? 8 : kMxTileCols];
  const int lane = threadIdx.x & 31;
  const int64_t warps = int64_t(gridDim.x) * (kMxThreads / 32);
  const int64_t ctiles = mx_ctiles(a.cols);
  const int64_t per = (ctiles + a.segs - 1) / a.segs;
  for (int64_t unit = int64_t(blockIdx.x) * (kMxThreads / 32) + (threadIdx.x >> 5);
       unit < a.rows * a.segs; unit += warps) {
    const int64_t r = a.segs == 1 ? unit : unit / a.segs;
    const int64_t s0 = (unit - r * a.segs) * per, s1 = min(ctiles, s0 + per);
    const int tr = int(r % kMxTileRows);
    T* dst = static_cast<T*>(a.out) + r * a.ld + s0 * kMxTileCols + lane * 8;
    const int64_t tile = (r / kMxTileRows) * ctiles + s0;
    const uint8_t* code = a.codes + tile * kMxCodeBytes + tr * 128 +
                          (((lane >> 2) ^ (tr & 7)) << 4) + (lane & 3) * 4;
    const uint8_t* scale = a.scales + tile * (2 * kMxTileBytes) + (lane >> 4) * kMxTileBytes +
                           (tr % 32) * 16 + (tr / 32) * 4 + ((lane >> 2) & 3);
    int64_t left = a.cols - s0 * kMxTileCols - lane * 8;
    for (int64_t s = s0; s < s1; s += kU) {
      uint32_t w[kU], sc[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        w[i] = sc[i] = 0;
        if (s + i < s1 && left > i * kMxTileCols) {
          w[i] = *reinterpret_cast<const uint32_t*>(code + i * kMxCodeBytes);
          sc[i] = scale[i * (2 * kMxTileBytes)];
        }
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        if (s + i >= s1) break;  // the same for the whole warp
        if (kVec && left <= i * kMxTileCols) continue;
        const float k = mx_scale(sc[i]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
              static_cast<__nv_fp4x2_storage_t>((w[i] >> (8 * j)) & 0xffu), __NV_E2M1);
          const float2 f = __half22float2(__half2(h));
          v[2 * j] = f.x * k;
          v[2 * j + 1] = f.y * k;
        }
        if constexpr (kVec) {
          LnIo<T, 8>::store(dst + i * kMxTileCols, v);
        } else {
          T* stage = stage_s[threadIdx.x >> 5];
          LnIo<T, 8>::store(stage + lane * 8, v);
          __syncwarp();
          // first column of the tile, and how many there are from it on
          T* to = dst - lane * 8 + i * kMxTileCols;
          const int64_t n = left + lane * 8 - i * kMxTileCols;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j * 32 + lane < n) to[j * 32 + lane] = stage[j * 32 + lane];
          __syncwarp();
        }
      }
      dst += kU * kMxTileCols;
      code += kU * kMxCodeBytes;
      scale += kU * 2 * kMxTileBytes;
      left -= kU * kMxTileCols;
    }
  }
}

static bool mx_sizes_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols > 0 && rows <= kMaxDim && cols <= kMaxDim &&
         cols <= (int64_t(1) << 40) / std::max<int64_t>(rows, 1);
}
static size_t mx_codes_bytes(int64_t rows, int64_t cols) {
  return size_t(cdiv(rows, kMxTileRows)) * size_t(mx_ctiles(cols)) * kMxCodeBytes;
}
static size_t mx_scales_bytes(int64_t rows, int64_t cols) {
  return size_t(cdiv(rows, kMxTileRows)) * size_t(mx_ktiles(cols)) * kMxTileBytes;
}
// Pieces per row (a warp each) and blocks: enough warps for the GPU when rows are few.
static int64_t mx_segments(int64_t rows, int64_t cols, int sms, int64_t* grid) {
  const int64_t steps = mx_ctiles(cols);
  const int64_t want = cdiv(int64_t(sms) * 32, std::max<int64_t>(rows, 1));
  const int64_t segs = std::max<int64_t>(1, std::min(steps, want));
  *grid = std::max<int64_t>(1, std::min<int64_t>(cdiv(rows * segs, kMxThreads / 32), int64_t(sms) * 16));
  return segs;
}
static bool mx_vec_ok(const void* p, int64_t ld, int64_t cols, int esz) {
  return aligned(p, 16) && (ld * esz) % 16 == 0 && cols % 8 == 0;
}

static int mx_quantize(const DeviceInfo& dev, const void* x, int dtype, int64_t rows, int64_t cols,
                       int64_t ld, uint8_t* codes, uint8_t* scales, cudaStream_t cs) {
  const int esz = dtype == FLCE_F32 ? 4 : 2;
  int64_t grid = 0;
  MxQuantArgs a{x, rows, cols, rows > 1 ? ld : cols, codes, scales, 0};
  a.segs = mx_segments(rows, cols, dev.num_sms, &grid);
  const bool vec = mx_vec_ok(x, rows > 1 ? ld : 0, cols, esz);
  LaunchScope scope(KF_MX_QUANT, 0.0, double(rows) * double(cols) * (esz + 17.0 / 32.0), cs);
  // Pieces of fewer tiles than a step takes: one at a time (100000 x 65: 63 -> 45 us).
  const bool single = cdiv(mx_ctiles(cols), a.segs) < kMxUnroll;
  auto go = [&](auto kern) { kern<<<unsigned(grid), kMxThreads, 0, cs>>>(a); };
  if (dtype == FLCE_BF16 && vec)
    single ? go(mx_quantize_kernel<__nv_bfloat16, true, 1>)
           : go(mx_quantize_kernel<__nv_bfloat16, true, kMxUnroll>);
  else if (dtype == FLCE_BF16)
    single ? go(mx_quantize_kernel<__nv_bfloat16, false, 1>)
           : go(mx_quantize_kernel<__nv_bfloat16, false, kMxUnroll>);
  else if (vec)
    single ? go(mx_quantize_kernel<float, true, 1>) : go(mx_quantize_kernel<float, true, kMxUnroll>);
  else
    single ? go(mx_quantize_kernel<float, false, 1>) : go(mx_quantize_kernel<float, false, kMxUnroll>);
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // namespace flce

extern "C" size_t flce_mxfp4_codes_size(int64_t rows, int64_t cols) {
  return mx_sizes_ok(rows, cols) ? mx_codes_bytes(rows, cols) : 0;
}
extern "C" size_t flce_mxfp4_scales_size(int64_t rows, int64_t cols) {
  return mx_sizes_ok(rows, cols) ? mx_scales_bytes(rows, cols) : 0;
}

extern "C" int flce_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld,
                                   void* codes, void* scales, flce_stream_t stream) {
  NvtxRange range("flce_mxfp4_quantize");
  if (!mx_sizes_ok(rows, cols) || !ln_ld_ok(rows, cols, ld) || !ln_dtype_ok(dtype))
    return FLCE_ERR_INVALID_ARG;
  if (rows == 0) return FLCE_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr ||
      !aligned(x, dtype == FLCE_F32 ? 4 : 2) || !aligned(codes, 16) || !aligned(scales, 16))
    return FLCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  return mx_quantize(*dev, x, dtype, rows, cols, ld, static_cast<uint8_t*>(codes),
                     static_cast<uint8_t*>(scales), static_cast<cudaStream_t>(stream));
}

extern "C" int flce_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows,
                                     int64_t cols, void* out, int dtype, int64_t ld,
                                     flce_stream_t stream) {
  NvtxRange range("flce_mxfp4_dequantize");
  if (!mx_sizes_ok(rows, cols) || !ln_ld_ok(rows, cols, ld) || !ln_dtype_ok(dtype))
    return FLCE_ERR_INVALID_ARG;
  if (rows == 0) return FLCE_OK;
  const int esz = dtype == FLCE_F32 ? 4 : 2;
  if (out == nullptr || codes == nullptr || scales == nullptr || !aligned(out, esz) ||
      !aligned(codes, 16) || !aligned(scales, 16))
    return FLCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int64_t grid = 0;
  MxDequantArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows,
                  cols, rows > 1 ? ld : cols, out, 0};
  a.segs = mx_segments(rows, cols, dev->num_sms, &grid);
  const bool vec = mx_vec_ok(out, rows > 1 ? ld : 0, cols, esz);
  LaunchScope scope(KF_MX_DEQUANT, 0.0, double(rows) * double(cols) * (esz + 17.0 / 32.0), cs);
  const bool single = cdiv(mx_ctiles(cols), a.segs) < kMxUnroll;
  auto go = [&](auto kern) { kern<<<unsigned(grid), kMxThreads, 0, cs>>>(a); };
  if (dtype == FLCE_BF16 && vec)
    single ? go(mx_dequantize_kernel<__nv_bfloat16, true, 1>)
           : go(mx_dequantize_kernel<__nv_bfloat16, true, kMxUnroll>);
  else if (dtype == FLCE_BF16)
    single ? go(mx_dequantize_kernel<__nv_bfloat16, false, 1>)
           : go(mx_dequantize_kernel<__nv_bfloat16, false, kMxUnroll>);
  else  // a lane's 8 FP32 values are two sectors: staged, whatever the alignment (45 -> 33 us
        // for 7335 x 4928)
    single ? go(mx_dequantize_kernel<float, false, 1>)
           : go(mx_dequantize_kernel<float, false, kMxUnroll>);
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
