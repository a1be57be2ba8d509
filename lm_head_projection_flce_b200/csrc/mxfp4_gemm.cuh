// mxfp4_gemm.cuh - the LM head's product with both operands in MXFP4:
//   logits[n, v] = cap( sum_h A[n, h] W[v, h] ),   cap(z) = c tanh(z / c) or z
// A = the hidden states quantised on the fly, W = the head quantised once.
// The tensor core multiplies the 4-bit codes and applies both block scales
// itself (tcgen05.mma kind::mxf4, one E8M0 scale per 32 elements), with FP32
// accumulation in tensor memory.
//
// Two kernels.  Few tokens (up to 192): the head's rows are the M side of a tile
// (128), so its codes, which are nearly all of the traffic, fill whole tiles,
// and the tokens are the N side (16 to 192), which shrinks to those that exist;
// the head is read once and the kernel is bound by HBM.  Many tokens: CTA pairs
// and tiles of 256 tokens x 256 head rows (mx_gemm_pair_kernel, below), bound by
// the tensor core.  There a thread of the epilogue holds consecutive logits of
// one token and stores 32 bytes at a time; with the head on the M side its lanes
// hold consecutive logits and store 2 bytes each, which at 4096 tokens took
// longer than the product (1205 against 890 us, both on single CTAs).
//
// Warp 0 loads: per stage of 256 elements of K the head's tile of codes (16 KB),
// the tokens' rows of theirs, and both operands' scale tiles, each a contiguous
// bulk copy.  Warp 1 copies the stage's scales to tensor memory (tcgen05.cp, 32
// lanes x 16 bytes replicated to the four lane quarters) and issues the MMAs; both
// run in issue order, and each stage has scale columns of its own, rewritten only
// after the MMAs that read them completed (the stage's empty barrier).  Warps 2..9
// store the accumulator, of which there are two, every other 32 tokens each (with
// four warps 142 tokens x 512 x 69658 took 26 us against 20: a warp per scheduler
// waits for its own instructions).  Every wait is bounded.
//
// Measured on one B200: 8 tokens x 4096 x 128256 in 49 us with the quantisation of
// the tokens (5.8 TB/s, 89% of the copy bandwidth; without the product's
// MMAs or its scale copies the time is the same); 4096 tokens in 777 us for a
// burst and 850 us back to back under the power cap (5.5 and 5.1 PFLOP/s).  There no
// single part is the bound: without the stores 702 us, without the MMAs 701,
// without the scale copies 745, without both operands' loads 680.
#pragma once

#include "mxfp4.cuh"

namespace flce {

constexpr int kMxgKBytes = 128;        // bytes of codes per row and stage
constexpr int kMxgBlocks = 8;          // scale blocks (256 elements) per stage
constexpr int kMxgM = 128;             // rows on the M side of a tile
constexpr int kMxgMaxN = 192;          // on the N side: two accumulators and the scales fit
constexpr int kMxgEpiWarps = 8;
constexpr int kMxgThreads = 64 + 32 * kMxgEpiWarps;
constexpr int kMxgMaxStages = 12;
constexpr int kMxgSmem = 225 * 1024;   // shared memory for the stages

struct MxGemmArgs {
  int64_t rows_m, rows_n, h;  // rows of the operand on the M and on the N side
  const uint8_t* m_codes;
  const uint8_t* m_scales;
  const uint8_t* n_codes;
  const uint8_t* n_scales;
  int tile_n;         // N rows per tile: all there are, rounded up, or kMxpN
  int64_t m_tiles;    // of the pair kernel: tiles along its M side, the tokens
  int64_t tiles;
  int stages;
  float softcap, inv_softcap;
  void* out;
  int64_t ldo;
  int v8;             // all rows of logits start on 32 bytes
  unsigned* err;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void tmem_alloc_one(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_one() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_one(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// wait_phase by a whole warp, with one answer for all its lanes: a wait that ran
// out in one lane must not leave the others at a warp-wide instruction.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, PipeCtl* ctl,
                                          unsigned* err, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, wait_phase<kCluster>(bar, parity, ctl, err, timeout_ns)) != 0;
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_commit_one(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// 32 rows x 16 bytes of shared memory to 4 columns of all four lane quarters.
__device__ __forceinline__ void tc_copy_scales_one(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
      "p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::mxf4: E2M1 A and B (K-major), E8M0 scales,
// shape M x N; the scale words' first byte used (0 or 2) is added per MMA.
__host__ __device__ constexpr uint32_t mma_idesc_mxf4(int m, int n) {
  return (1u << 7)                                // A: E2M1
         | (1u << 10)                             // B: E2M1
         | (static_cast<uint32_t>(n >> 3) << 17)  // N / 8
         | (1u << 23)                             // scales: E8M0
         | (static_cast<uint32_t>(m >> 7) << 27); // M / 128
}
// A scale tile in shared memory: unswizzled, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t mx_scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// c tanh(z / c) of a thread's 32 values, to a few units in the last place of FP32.  With
// x = z / c and |x| <= 5/8 it is z + z t(x^2), t the odd series' tail as a polynomial
// of five terms (fitted here for a small largest relative error: 8.7e-9 with the
// coefficients rounded to FP32, at x = 0.604), and no special function; beyond, c -
// 2c / (exp(2 |x|) + 1) with z's sign.  The method, an odd polynomial near 0 and the
// exponential form beyond it, is that of Cody and Waite's "Software Manual for the
// Elementary Functions" (1980) and of Moshier's "Methods and Programs for
// Mathematical Functions" (1989).  A warp whose values are
// all small, as most logits of a cap are, skips the second: 1024 x 4096 x 65536 takes
// 109 us then, as without a cap, and 129 us with large values (tanhf for every
// value: 130 us either way).  One reciprocal for two values gained nothing.
__device__ __forceinline__ void mx_softcap(float (&z)[32], float c, float inv_c) {
  constexpr float kSmall = 0.625f;
  float top = 0.0f;  // a NaN passes through either branch
#pragma unroll
  for (int j = 0; j < 32; ++j) top = fmaxf(top, fabsf(z[j]));
  const bool small = __all_sync(0xffffffffu, top * inv_c <= kSmall) != 0;
  auto both = [](float v) { return make_float2(v, v); };
  auto series = [&](float2 v, float2 x) {
    const float2 u = __fmul2_rn(x, x);
    float2 t = __ffma2_rn(both(-0.00570497848f), u, both(0.0206390787f));
    t = __ffma2_rn(t, u, both(-0.0537397116f));
    t = __ffma2_rn(t, u, both(0.133314416f));
    t = __ffma2_rn(t, u, both(-0.333332807f));
    return __ffma2_rn(__fmul2_rn(t, u), v, v);
  };
  if (small) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 v = make_float2(z[j], z[j + 1]);
      const float2 y = series(v, __fmul2_rn(v, both(inv_c)));
      z[j] = y.x;
      z[j + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 v = make_float2(z[j], z[j + 1]), x = __fmul2_rn(v, both(inv_c));
      const float2 y = series(v, x);
      auto large = [&](float xi, float yi) {
        const float r = fast_rcp(fast_exp2(fabsf(xi) * (2.0f * kLog2e)) + 1.0f);
        return fabsf(xi) <= kSmall ? yi : copysignf(fmaf(-2.0f * c, r, c), xi);
      };
      z[j] = large(x.x, y.x);
      z[j + 1] = large(x.y, y.y);
    }
  }
}

__host__ __device__ __forceinline__ int mxg_scale_tiles(int tile_n) { return tile_n > 128 ? 2 : 1; }
// Bytes of a stage: codes of both operands, then 2 scale tiles (2 x 128 elements
// of K) per 128 rows of each.
__host__ __device__ __forceinline__ uint32_t mxg_stage_bytes(int tile_n) {
  return uint32_t((kMxgM + tile_n) * kMxgKBytes + (1 + mxg_scale_tiles(tile_n)) * 2 * kMxTileBytes);
}

// Tiles are 128 head rows x all tokens.
// kSft: scale tiles of 128 rows on the N side (2 above 128 tokens).
template <typename TO, int kSft>
__global__ void __launch_bounds__(kMxgThreads, 1)
    mx_gemm_kernel(const MxGemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMxgMaxStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ PipeCtl ctl_s;
  PipeCtl* ctl = &ctl_s;
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar_base = smem_u32(bars);
  const int stages = g.stages;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (kMxgMaxStages + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * kMxgMaxStages + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * kMxgMaxStages + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (2 * kMxgMaxStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = mxg_stage_bytes(g.tile_n);
  const uint32_t off_b = kMxgM * kMxgKBytes;
  const uint32_t off_sfa = off_b + uint32_t(g.tile_n) * kMxgKBytes;
  const uint32_t off_sfb = off_sfa + 2 * kMxTileBytes;
  const int64_t blocks = mx_blocks(g.h);
  const int num_kb = int(mx_ctiles(g.h));

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kMxgEpiWarps);
    }
    mbar_init(drain_bar, 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_one(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish_one();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  // Warps 0 and 1 run their loops with all lanes, so that addresses and
  // descriptors stay in uniform registers; one elected lane issues.  The loops
  // keep running values: with the multiplications in them, the two issuing
  // threads themselves were the bound (1690 -> 1205 us at 4096 tokens, 73 -> 64 us
  // at 8, when this kernel took both).
  if (warp == 0) {
    // -------------------------------------------------- loads
    const bool leader = elect_one();
    // The head, read once, is marked first to go, which spares the rest of L2 (64 -> 55 us
    // at 8 tokens x 4096 x 128256).
    const uint64_t pol_m = l2_policy_evict_first(), pol_n = l2_policy_evict_last();
    // The tokens' codes: up to 128 rows of one row tile, the rest from the next.
    constexpr bool two = kSft == 2;
    const uint32_t bytes0 = uint32_t(min(g.tile_n, kMxTileRows)) * kMxgKBytes;
    const uint32_t bytes1 = uint32_t(g.tile_n) * kMxgKBytes - bytes0;
    const uint32_t expect =
        kMxCodeBytes + 4 * kMxTileBytes + bytes0 + (two ? bytes1 + 2 * kMxTileBytes : 0u);
    int st = 0;
    uint32_t ph = 0, base = smem_base, full = full_bar(0);
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      const uint8_t* mc = g.m_codes + t * num_kb * kMxCodeBytes;
      const uint8_t* ms = g.m_scales + t * num_kb * (2 * kMxTileBytes);
      const uint8_t* nc = g.n_codes;
      const uint8_t* ns = g.n_scales;
      const uint8_t* nc1 = nc + num_kb * kMxCodeBytes;
      const uint8_t* ns1 = ns + num_kb * (2 * kMxTileBytes);
      int ahead = 0;
      if (t == blockIdx.x) {
        // The head does not depend on the kernel before this one, which puts the
        // tokens into 4 bits: its first stages are on their way before that ends.
        ahead = min(stages, num_kb);
        if (leader) {
          for (int s = 0; s < ahead; ++s) {
            const uint32_t to = smem_base + uint32_t(s) * stage_bytes;
            mbar_arrive_expect_tx(full_bar(s), expect);
            bulk_load_hint(to, mc + int64_t(s) * kMxCodeBytes, kMxCodeBytes, full_bar(s), pol_m);
            bulk_load_hint(to + off_sfa, ms + int64_t(s) * (2 * kMxTileBytes), 2 * kMxTileBytes,
                           full_bar(s), pol_m);
          }
        }
        __syncwarp();
        grid_dependency_wait();
      }
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!wait_warp(full + 8u * kMxgMaxStages, ph ^ 1u, ctl, g.err, g.timeout_ns)) {
          ok = false;
          break;
        }
        if (leader) {
          if (kb >= ahead) {
            mbar_arrive_expect_tx(full, expect);
            bulk_load_hint(base, mc, kMxCodeBytes, full, pol_m);
            bulk_load_hint(base + off_sfa, ms, 2 * kMxTileBytes, full, pol_m);
          }
          bulk_load_hint(base + off_b, nc, bytes0, full, pol_n);
          bulk_load_hint(base + off_sfb, ns, 2 * kMxTileBytes, full, pol_n);
          if (two) {
            bulk_load_hint(base + off_b + bytes0, nc1, bytes1, full, pol_n);
            bulk_load_hint(base + off_sfb + 2 * kMxTileBytes, ns1, 2 * kMxTileBytes, full, pol_n);
          }
        }
        mc += kMxCodeBytes;
        ms += 2 * kMxTileBytes;
        nc += kMxCodeBytes;
        ns += 2 * kMxTileBytes;
        nc1 += kMxCodeBytes;
        ns1 += 2 * kMxTileBytes;
        base += stage_bytes;
        full += 8u;
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
          base = smem_base;
          full = full_bar(0);
        }
      }
    }
    if (!ok) {
      // Give the copies in flight time to land before the block can exit.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------- scales to tensor memory, MMAs
    const bool leader = elect_one();
    const uint32_t idesc = mma_idesc_mxf4(kMxgM, g.tile_n);
    constexpr uint32_t kIdOdd = (2u << 4) | (2u << 29);  // bytes 2, 3 of the scale words
    constexpr uint64_t hi = desc_hi_sw128(16u, 1024u);
    const uint64_t da0 = hi | static_cast<uint64_t>((smem_base & 0x3FFFFu) >> 4);
    const uint64_t step = stage_bytes >> 4;
    const uint64_t db_off = off_b >> 4;
    const uint64_t dsa0 = mx_scale_desc(smem_base + off_sfa);
    // Scale columns of a stage: the M side's first and second half of K, 4 each;
    // then the N side's first half (4 per 128 rows) and second half.
    constexpr uint32_t kSfCols = 8 + 8 * kSft;
    const uint32_t sf0 = tmem + 2u * uint32_t(g.tile_n);
    int st = 0, acc = 0;
    uint32_t ph = 0, acc_ph = 0, full = full_bar(0), sfa = sf0;
    uint64_t da = da0, dsa = dsa0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      if (!wait_warp(tempty_bar(acc), acc_ph ^ 1u, ctl, g.err, g.timeout_ns)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t d = tmem + uint32_t(acc) * uint32_t(g.tile_n);
      int left = int(blocks);  // scale blocks still to multiply
      uint32_t more = 0;
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!wait_warp(full, ph, ctl, g.err, g.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (leader) {
          const uint32_t sfb = sfa + 8u;
          const uint64_t dsb = dsa + (2 * kMxTileBytes >> 4);
          constexpr uint64_t kTile = kMxTileBytes >> 4;
          tc_copy_scales_one(sfa, dsa);
          tc_copy_scales_one(sfa + 4u, dsa + kTile);
          tc_copy_scales_one(sfb, dsb);
          if (kSft == 2) tc_copy_scales_one(sfb + 4u, dsb + 2 * kTile);
          tc_copy_scales_one(sfb + 4u * kSft, dsb + kTile);
          if (kSft == 2) tc_copy_scales_one(sfb + 4u * kSft + 4u, dsb + 3 * kTile);
          const uint64_t db = da + db_off;
          tc_mma_mxf4_one(d, da, db, idesc, sfa, sfb, more);
          if (left > 2) tc_mma_mxf4_one(d, da + 2, db + 2, idesc | kIdOdd, sfa, sfb, 1u);
          if (left > 4) tc_mma_mxf4_one(d, da + 4, db + 4, idesc, sfa + 4u, sfb + 4u * kSft, 1u);
          if (left > 6)
            tc_mma_mxf4_one(d, da + 6, db + 6, idesc | kIdOdd, sfa + 4u, sfb + 4u * kSft, 1u);
          tc_commit_one(full + 8u * kMxgMaxStages);
        }
        __syncwarp();
        more = 1u;
        left -= kMxgBlocks;
        full += 8u;
        sfa += kSfCols;
        da += step;
        dsa += step;
        if (++st == stages) {
          st = 0;
          ph ^= 1u;
          full = full_bar(0);
          sfa = sf0;
          da = da0;
          dsa = dsa0;
        }
      }
      if (!ok) break;
      if (leader) tc_commit_one(tfull_bar(acc));
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1u;
    }
    if (leader) tc_commit_one(drain_bar);
    __syncwarp();
    drain_wait(drain_bar, 0, ok ? g.timeout_ns : 100000000ull);
  } else {
    // -------------------------------------------------- epilogue: lanes are M rows
    grid_dependency_wait();  // before anything is stored
    const int quarter = warp & 3, half = (warp - 2) >> 2;  // every other 32 columns
    int acc = 0;
    uint32_t acc_ph = 0;
    const bool capped = g.softcap > 0.0f;
    const int cols = int(g.rows_n);
    for (int64_t t = blockIdx.x; t < g.tiles; t += gridDim.x) {
      if (!wait_warp(tfull_bar(acc), acc_ph, ctl, g.err, g.timeout_ns)) break;
      __syncwarp();
      tc_fence_after_sync();
      const int64_t row = t * kMxgM + quarter * 32 + lane;
      const bool live = row < g.rows_m;
      const uint32_t taddr =
          tmem + (static_cast<uint32_t>(quarter * 32) << 16) + uint32_t(acc) * uint32_t(g.tile_n);
      for (int c0 = 32 * half; c0 < cols; c0 += 64) {
        float x[32];
        __syncwarp();  // lanes behind the last row store nothing and come here first
        tmem_load_32cols(taddr + c0, x);
        if (capped) mx_softcap(x, g.softcap, g.inv_softcap);
        if (!live) continue;  // what is above is for the whole warp
        TO* out = static_cast<TO*>(g.out) + int64_t(c0) * g.ldo + row;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float one[1] = {x[j]};
          if (c0 + j < cols) LnIo<TO, 1>::store(out + int64_t(j) * g.ldo, one);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1u;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_one(tmem, kTmemCols);
  }
}

template <typename TO, int kSft>
static int mx_launch_gemm(const MxGemmArgs& g, int grid, cudaStream_t cs) {
  auto kern = mx_gemm_kernel<TO, kSft>;
  const size_t smem = 1024 + size_t(g.stages) * mxg_stage_bytes(g.tile_n);
  // The limit belongs to the kernel, not to the launch: always the same, so that a call
  // of another thread cannot lower it before this one launches.
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kMxgSmem) !=
      cudaSuccess)
    return FLCE_ERR_CUDA;
  return launch_dependent(kern, dim3(unsigned(grid)), dim3(kMxgThreads), smem, cs, g);
}

// ---------------------------------------------------------------- CTA pairs
// A cluster of two CTAs on neighbouring SMs multiplies tiles of 256 tokens x 256
// head rows (tcgen05.mma.cta_group::2): CTA r holds token rows [128 r, 128 r +
// 128) and head rows [128 r, 128 r + 128) of a tile, one tile of codes each per
// stage, and the scales of its own tokens and of all 256 head rows.  Per MMA a
// single CTA's 128 x 192 tile moves 1.6 times the bytes through shared memory per
// product, more than the tensor core leaves time for.  256 accumulator
// columns and the scales (24 columns per stage, 6 stages) leave no room for a
// second accumulator, so eight epilogue warps empty it into registers at once
// (128 columns each) and store while the next tile is multiplied.
constexpr int kMxpStages = 6;
constexpr int kMxpN = 256;
constexpr int kMxpEpiWarps = 8;
constexpr int kMxpThreads = 64 + 32 * kMxpEpiWarps;
constexpr uint32_t kMxpOffB = kMxCodeBytes;
constexpr uint32_t kMxpOffSfa = 2 * kMxCodeBytes;
constexpr uint32_t kMxpOffSfb = kMxpOffSfa + 2 * kMxTileBytes;
constexpr uint32_t kMxpStageBytes = kMxpOffSfb + 4 * kMxTileBytes;  // 35 KB
constexpr size_t kMxpSmem = 1024 + size_t(kMxpStages) * kMxpStageBytes;
static_assert(kMxpN + kMxpStages * 24 <= kTmemCols, "accumulator and scales in tensor memory");

__device__ __forceinline__ void tc_copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                 uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
      "p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// `bytes` (< 32) of the words at `to`, 16-byte aligned, in pieces of 16, 8, 4 and 2.
__device__ __forceinline__ void store_pieces(uint8_t* to, const uint32_t (&w)[8], int bytes) {
  const bool b16 = (bytes & 16) != 0, b8 = (bytes & 8) != 0, b4 = (bytes & 4) != 0;
  if (b16) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  uint32_t v[4], u[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = b16 ? w[i + 4] : w[i];
  to += bytes & 16;
  if (b8) *reinterpret_cast<uint2*>(to) = make_uint2(v[0], v[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) u[i] = b8 ? v[i + 2] : v[i];
  to += bytes & 8;
  if (b4) *reinterpret_cast<uint32_t*>(to) = u[0];
  to += bytes & 4;
  if (bytes & 2) *reinterpret_cast<uint16_t*>(to) = uint16_t(b4 ? u[1] : u[0]);
}
// `count` (<= 128) consecutive logits of a row at any alignment, from one thread: up to
// the first 32-byte boundary in pieces of 1, 2, 4 and 8 elements, each aligned to its
// size, then 32 bytes at a time, cut out of the words around them by a shift of 4, 2
// and 1 words, and the end in pieces again.  (Blocks of 32 x 32 transposed by
// shuffles, so that the lanes' 2-byte stores were consecutive, took a 1561 x 104 x
// 25615 product 87 us against 41.)
template <typename TO>
__device__ __forceinline__ void store_run(TO* out, const float (&x)[4][32], int count) {
  constexpr int kWords = 32 * int(sizeof(TO)), kPer = 32 / int(sizeof(TO));  // elements in 32 bytes
  if (count < kPer) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float one[1] = {x[0][j]};
      if (j < count) LnIo<TO, 1>::store(out + j, one);
    }
    return;
  }
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (sizeof(TO) == 4)
      w[i] = __float_as_uint(x[i / 32][i % 32]);
    else
      w[i] = pack_bf16x2(x[i / 16][2 * i % 32], x[i / 16][2 * i % 32 + 1]);
  }
  uint8_t* at = reinterpret_cast<uint8_t*>(out);
  const uint32_t head = (32u - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out)) & 31u)) & 31u;
  const bool b4 = (head & 4u) != 0, b8 = (head & 8u) != 0, b16 = (head & 16u) != 0;
  if constexpr (sizeof(TO) == 2) {
    if (head & 2u) *reinterpret_cast<uint16_t*>(at) = uint16_t(w[0]);
    at += head & 2u;
    const uint32_t sh = (head & 2u) * 8u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], i + 1 < kWords ? w[i + 1] : 0u, sh);
  }
  {
    uint32_t v[6], u[4];
    if (b4) *reinterpret_cast<uint32_t*>(at) = w[0];
    at += head & 4u;
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = b4 ? w[i + 1] : w[i];
    if (b8) *reinterpret_cast<uint2*>(at) = make_uint2(v[0], v[1]);
    at += head & 8u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = b8 ? v[i + 2] : v[i];
    if (b16) *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
    at += head & 16u;
  }
  int left = count * int(sizeof(TO)) - int(head);  // bytes
#pragma unroll
  for (int k = 0; k < kWords; k += 8) {
    auto word = [&](int i) { return k + i < kWords ? w[(k + i) % kWords] : 0u; };
    uint32_t v[11], u[9], e[8];
#pragma unroll
    for (int i = 0; i < 11; ++i) v[i] = b16 ? word(i + 4) : word(i);
#pragma unroll
    for (int i = 0; i < 9; ++i) u[i] = b8 ? v[i + 2] : v[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = b4 ? u[i + 1] : u[i];
    if (left >= 32)
      st_global_v8(at, e[0], e[1], e[2], e[3], e[4], e[5], e[6], e[7]);
    else if (left > 0)
      store_pieces(at, e, left);
    at += 32;
    left -= 32;
  }
}

struct __align__(64) MxPairMaps {
  // Codes as rows of 128 bytes, 128 rows per tile; scales as rows of 128 bytes,
  // 8 rows per tile of codes.  No swizzle: the codes are stored swizzled.
  CUtensorMap m_codes, m_scales, n_codes, n_scales;
};

template <typename TO>
__global__ void __launch_bounds__(kMxpThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ MxPairMaps maps, const MxGemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMxpStages + 3];
  __shared__ uint32_t tmem_slot;
  __shared__ PipeCtl ctl_s;
  PipeCtl* ctl = &ctl_s;
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar_base = smem_u32(bars);
  const uint32_t rank = cluster_cta_rank();
  const uint32_t leader_bars = map_shared_to_rank(bar_base, 0);
  constexpr uint32_t kEmpty = 8u * kMxpStages;
  const uint32_t tfull = bar_base + 16u * kMxpStages, tempty = tfull + 8u, drain_bar = tfull + 16u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_kb = int(mx_ctiles(g.h));
  const int64_t m_row_tiles = (g.rows_m + kMxTileRows - 1) / kMxTileRows;
  const int64_t n_row_tiles = (g.rows_n + kMxTileRows - 1) / kMxTileRows;
  const int64_t pairs = gridDim.x >> 1, first = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMxpStages; ++s) {
      mbar_init(bar_base + 8u * s, 1);
      mbar_init(bar_base + kEmpty + 8u * s, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kMxpEpiWarps);
    mbar_init(drain_bar, 1);
    ctl->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.m_codes);
    tma_prefetch_desc(&maps.m_scales);
    tma_prefetch_desc(&maps.n_codes);
    tma_prefetch_desc(&maps.n_scales);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers exist before anyone signals them
  tc_fence_after_sync();
  grid_dependency_wait();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // -------------------------------------------------- loads (both CTAs)
    const bool leader = elect_one();
    // Both operands are read again by other pairs; the logits, written once, should
    // not displace them (923 -> 860 us at 4096 x 4096 x 128256, back to back).
    const uint64_t pol = l2_policy_evict_last();
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t t = first; ok && t < g.tiles; t += pairs) {
      // The token tiles of a head tile follow one another, and share it in L2.
      const int64_t nt = t / g.m_tiles, mt = t - nt * g.m_tiles;
      // Row tiles that exist: token tile 2 mt + 1 and head tile 2 nt + 1 may not.
      const int ma = 2 * mt + 1 < m_row_tiles ? 2 : 1, nb = 2 * nt + 1 < n_row_tiles ? 2 : 1;
      const bool have_a = int(rank) < ma, have_b = int(rank) < nb;
      const uint32_t expect = uint32_t(ma) * (kMxCodeBytes + 2 * kMxTileBytes) +
                              uint32_t(nb) * (kMxCodeBytes + 4 * kMxTileBytes);
      int am = int((2 * mt + rank) * num_kb), bn = int((2 * nt + rank) * num_kb);
      int b0 = int(2 * nt * num_kb);
      for (int kb = 0; kb < num_kb; ++kb, ++am, ++bn, ++b0) {
        if (!wait_warp(bar_base + kEmpty + 8u * st, ph ^ 1u, ctl, g.err, g.timeout_ns)) {
          ok = false;
          break;
        }
        const uint32_t base = smem_base + uint32_t(st) * kMxpStageBytes;
        const uint32_t full = leader_bars + 8u * st;  // counts both CTAs' bytes
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(bar_base + 8u * st, expect);
          if (have_a) {
            tma_load_2d_pair_hint(base, &maps.m_codes, full, 0, am * 128, pol);
            tma_load_2d_pair_hint(base + kMxpOffSfa, &maps.m_scales, full, 0, am * 8, pol);
          }
          if (have_b) tma_load_2d_pair_hint(base + kMxpOffB, &maps.n_codes, full, 0, bn * 128, pol);
          tma_load_2d_pair_hint(base + kMxpOffSfb, &maps.n_scales, full, 0, b0 * 8, pol);
          if (nb == 2)
            tma_load_2d_pair_hint(base + kMxpOffSfb + 2 * kMxTileBytes, &maps.n_scales, full, 0,
                                  (b0 + num_kb) * 8, pol);
        }
        __syncwarp();
        if (++st == kMxpStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok) {
      // Copies this warp started signal the leader's barriers; give them time to
      // land before the CTA can exit.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------ scales and MMAs of both CTAs
      const bool leader = elect_one();
      constexpr uint32_t idesc = mma_idesc_mxf4(2 * kMxgM, kMxpN);
      constexpr uint32_t kIdOdd = (2u << 4) | (2u << 29);  // bytes 2, 3 of the scale words
      constexpr uint64_t hi = desc_hi_sw128(16u, 1024u);
      constexpr uint64_t kTile = kMxTileBytes >> 4;
      const uint64_t da0 = hi | static_cast<uint64_t>((smem_base & 0x3FFFFu) >> 4);
      const uint64_t dsa0 = mx_scale_desc(smem_base + kMxpOffSfa);
      const uint32_t sf0 = tmem + kMxpN;
      int st = 0;
      uint32_t ph = 0, acc_ph = 0, sfa = sf0;
      uint64_t da = da0, dsa = dsa0;
      bool ok = true;
      const int blocks = int(mx_blocks(g.h));
      for (int64_t t = first; ok && t < g.tiles; t += pairs) {
        if (!wait_warp<true>(tempty, acc_ph ^ 1u, ctl, g.err, g.timeout_ns)) {
          ok = false;
          break;
        }
        acc_ph ^= 1u;
        tc_fence_after_sync();
        int left = blocks;
        uint32_t more = 0;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_warp(bar_base + 8u * st, ph, ctl, g.err, g.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (leader) {
            const uint32_t sfb = sfa + 8u;
            const uint64_t dsb = dsa + ((kMxpOffSfb - kMxpOffSfa) >> 4);
            tc_copy_scales_pair(sfa, dsa);
            tc_copy_scales_pair(sfa + 4u, dsa + kTile);
            tc_copy_scales_pair(sfb, dsb);
            tc_copy_scales_pair(sfb + 4u, dsb + 2 * kTile);
            tc_copy_scales_pair(sfb + 8u, dsb + kTile);
            tc_copy_scales_pair(sfb + 12u, dsb + 3 * kTile);
            const uint64_t db = da + (kMxpOffB >> 4);
            tc_mma_mxf4_pair(tmem, da, db, idesc, sfa, sfb, more);
            if (left > 2) tc_mma_mxf4_pair(tmem, da + 2, db + 2, idesc | kIdOdd, sfa, sfb, 1u);
            if (left > 4) tc_mma_mxf4_pair(tmem, da + 4, db + 4, idesc, sfa + 4u, sfb + 8u, 1u);
            if (left > 6)
              tc_mma_mxf4_pair(tmem, da + 6, db + 6, idesc | kIdOdd, sfa + 4u, sfb + 8u, 1u);
            tc_commit_pair_mc(bar_base + kEmpty + 8u * st, 0x3);
          }
          __syncwarp();
          more = 1u;
          left -= kMxgBlocks;
          sfa += 24u;
          da += kMxpStageBytes >> 4;
          dsa += kMxpStageBytes >> 4;
          if (++st == kMxpStages) {
            st = 0;
            ph ^= 1u;
            sfa = sf0;
            da = da0;
            dsa = dsa0;
          }
        }
        if (!ok) break;
        if (leader) tc_commit_pair_mc(tfull, 0x3);
        __syncwarp();
      }
      if (leader) tc_commit_pair_mc(drain_bar, 0x1);
      __syncwarp();
      drain_wait(drain_bar, 0, ok ? g.timeout_ns : 100000000ull);
    }
  } else {
    // -------------------------------------------------- epilogue: lanes are tokens
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + uint32_t(half) * 128u;
    const uint32_t leader_tempty = map_shared_to_rank(tempty, 0);
    const bool capped = g.softcap > 0.0f;
    uint32_t acc_ph = 0;
    for (int64_t t = first; t < g.tiles; t += pairs) {
      const int64_t nt = t / g.m_tiles, mt = t - nt * g.m_tiles;
      if (!wait_warp(tfull, acc_ph, ctl, g.err, g.timeout_ns)) break;
      acc_ph ^= 1u;
      __syncwarp();
      tc_fence_after_sync();
      float x[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_load_32cols(taddr + 32u * q, x[q]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_tempty);
      const int64_t row = (2 * mt + rank) * kMxgM + quarter * 32 + lane;
      const int64_t c0 = nt * kMxpN + half * 128;
      if (capped) {
#pragma unroll
        for (int q = 0; q < 4; ++q) mx_softcap(x[q], g.softcap, g.inv_softcap);
      }
      if (row >= g.rows_m || c0 >= g.rows_n) continue;
      // 128 consecutive logits of a token
      TO* out = static_cast<TO*>(g.out) + row * g.ldo + c0;
      if (!g.v8) {
        store_run(out, x, int(min(int64_t(128), g.rows_n - c0)));
        continue;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t left = g.rows_n - (c0 + 32 * q);
        if (left <= 0) break;
        if (left >= 32) {
          if constexpr (sizeof(TO) == 2) {
            store_bf16x32(reinterpret_cast<uint4*>(out + 32 * q), x[q], true);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              st_global_v8(out + 32 * q + j, __float_as_uint(x[q][j]), __float_as_uint(x[q][j + 1]),
                           __float_as_uint(x[q][j + 2]), __float_as_uint(x[q][j + 3]),
                           __float_as_uint(x[q][j + 4]), __float_as_uint(x[q][j + 5]),
                           __float_as_uint(x[q][j + 6]), __float_as_uint(x[q][j + 7]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float one[1] = {x[q][j]};
            if (j < left) LnIo<TO, 1>::store(out + 32 * q + j, one);
          }
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // the leader's MMAs into this CTA's tensor memory are done
  tc_fence_after_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// `tiles` tiles of box_rows rows of 128 bytes.
static bool mx_tmap(CUtensorMap* tm, const void* base, int64_t tiles, int box_rows) {
  cuuint64_t dims[2] = {128, cuuint64_t(tiles) * cuuint64_t(box_rows)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TO>
static int mx_launch_pair(const MxGemmArgs& g, DeviceInfo& dev, cudaStream_t cs) {
  auto kern = mx_gemm_pair_kernel<TO>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMxpSmem)) !=
      cudaSuccess)
    return FLCE_ERR_CUDA;
  const int64_t kb = mx_ctiles(g.h);
  const int64_t mt = cdiv(g.rows_m, kMxTileRows) * kb, nt = cdiv(g.rows_n, kMxTileRows) * kb;
  MxPairMaps maps;
  if (!mx_tmap(&maps.m_codes, g.m_codes, mt, 128) || !mx_tmap(&maps.m_scales, g.m_scales, mt, 8) ||
      !mx_tmap(&maps.n_codes, g.n_codes, nt, 128) || !mx_tmap(&maps.n_scales, g.n_scales, nt, 8))
    return FLCE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMxpThreads, 1, 1);
  cfg.dynamicSmemBytes = kMxpSmem;
  cfg.stream = cs;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = dev.mx_pairs;
  if (pairs == 0) {  // pairs that can be resident at once, queried once per device
    cfg.gridDim = dim3(2 * (dev.num_sms / 2), 1, 1);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) n = dev.num_sms / 2;
    pairs = std::min(n, dev.num_sms / 2);
    std::lock_guard<std::mutex> lock(g_mutex);
    dev.mx_pairs = pairs;
  }
  cfg.gridDim = dim3(unsigned(2 * std::min<int64_t>(pairs, g.tiles)), 1, 1);
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, maps, g) != cudaSuccess) return FLCE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

struct MxLogitsPlan {
  size_t off_scales, total;
};
static MxLogitsPlan plan_mx_logits(int64_t n, int64_t h) {
  MxLogitsPlan p{};
  p.off_scales = align_up(mx_codes_bytes(n, h));
  p.total = std::max(kAlign, align_up(p.off_scales + mx_scales_bytes(n, h)));
  return p;
}

}  // namespace flce

extern "C" size_t flce_mxfp4_logits_workspace_size(int64_t n, int64_t h) {
  return mx_sizes_ok(n, h) ? plan_mx_logits(n, h).total : 0;
}

extern "C" int flce_mxfp4_logits(const void* hidden, int dtype, int64_t n, int64_t h, int64_t ldh,
                                 const void* w_codes, const void* w_scales, int64_t vp,
                                 int64_t unpadded, float softcap, void* logits, int out_dtype,
                                 int64_t ldo, void* workspace, size_t ws_bytes,
                                 flce_stream_t stream) {
  NvtxRange range("flce_mxfp4_logits");
  const int64_t v = unpadded <= 0 ? vp : unpadded;
  if (!mx_sizes_ok(n, h) || !mx_sizes_ok(vp, h) || vp <= 0 || v > vp || !ln_ld_ok(n, h, ldh) ||
      !ln_ld_ok(n, v, ldo) || !ln_dtype_ok(dtype) || !ln_dtype_ok(out_dtype) ||
      !(softcap >= 0.0f) || !std::isfinite(softcap) ||
      (softcap > 0.0f && !std::isfinite(1.0f / softcap)))
    return FLCE_ERR_INVALID_ARG;
  if (w_codes == nullptr || w_scales == nullptr || !aligned(w_codes, 16) || !aligned(w_scales, 16))
    return FLCE_ERR_INVALID_ARG;
  if (n == 0) return FLCE_OK;
  if (hidden == nullptr || logits == nullptr || !aligned(hidden, dtype == FLCE_F32 ? 4 : 2) ||
      !aligned(logits, out_dtype == FLCE_F32 ? 4 : 2))
    return FLCE_ERR_INVALID_ARG;
  const MxLogitsPlan p = plan_mx_logits(n, h);
  if (workspace == nullptr || !aligned(workspace, 16) || ws_bytes < p.total)
    return FLCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* a_codes = static_cast<uint8_t*>(workspace);
  uint8_t* a_scales = a_codes + p.off_scales;
  st = mx_quantize(*dev, hidden, dtype, n, h, ldh, a_codes, a_scales, cs);
  if (st != FLCE_OK) return st;
  MxGemmArgs g{};
  const int esz = out_dtype == FLCE_F32 ? 4 : 2;
  const int64_t ld = n > 1 ? ldo : v;
  const bool tokens_m = n > kMxgMaxN;
  const uint8_t* wc = static_cast<const uint8_t*>(w_codes);
  const uint8_t* wsc = static_cast<const uint8_t*>(w_scales);
  g.rows_m = tokens_m ? n : v;
  g.rows_n = tokens_m ? v : n;
  g.h = h;
  g.m_codes = tokens_m ? a_codes : wc;
  g.m_scales = tokens_m ? a_scales : wsc;
  g.n_codes = tokens_m ? wc : a_codes;
  g.n_scales = tokens_m ? wsc : a_scales;
  g.tile_n = int(std::min<int64_t>(cdiv(g.rows_n, 16) * 16, kMxgMaxN));
  if (g.tile_n > 128) g.tile_n = kMxgMaxN;
  if (tokens_m) g.tile_n = kMxpN;
  g.m_tiles = cdiv(g.rows_m, tokens_m ? 2 * kMxgM : kMxgM);
  g.tiles = g.m_tiles * cdiv(g.rows_n, g.tile_n);  // one along the N side with few tokens
  const int sf_stages = (kTmemCols - 2 * g.tile_n) / (8 + 8 * mxg_scale_tiles(g.tile_n));
  g.stages = std::min({kMxgMaxStages, sf_stages, int(kMxgSmem / mxg_stage_bytes(g.tile_n))});
  g.softcap = softcap;
  g.inv_softcap = softcap > 0.0f ? 1.0f / softcap : 0.0f;
  g.out = logits;
  g.ldo = ld;
  g.v8 = aligned(logits, 32) && (ld * esz) % 32 == 0;
  g.err = dev->err;
  g.timeout_ns = kDefaultTimeoutNs;
  const int grid = int(std::min<int64_t>(g.tiles, dev->num_sms));
  const double osz = out_dtype == FLCE_F32 ? 4.0 : 2.0;
  LaunchScope scope(KF_MX_GEMM, 2.0 * double(n) * double(h) * double(v),
                    double(n + v) * double(h) * 17.0 / 32.0 + osz * double(n) * double(v), cs);
  const bool bf = out_dtype == FLCE_BF16;
  if (tokens_m) {
    // coordinates of the tensor maps are 32-bit
    if ((cdiv(std::max(n, v), kMxTileRows) + 2) * mx_ctiles(h) * 128 > kMaxDim)
      return FLCE_ERR_UNSUPPORTED;
    return bf ? mx_launch_pair<__nv_bfloat16>(g, *dev, cs) : mx_launch_pair<float>(g, *dev, cs);
  }
  if (g.tile_n > 128)
    return bf ? mx_launch_gemm<__nv_bfloat16, 2>(g, grid, cs)
              : mx_launch_gemm<float, 2>(g, grid, cs);
  return bf ? mx_launch_gemm<__nv_bfloat16, 1>(g, grid, cs)
            : mx_launch_gemm<float, 1>(g, grid, cs);
}
