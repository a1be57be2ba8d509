// beam.cuh - beam search behind the LM head: which continuations of the K beams
// of each batch item are kept, and the reordering of the beams' states.
//
// Selection.  For item b with logits z[k, v] and cumulative log-probabilities s_k:
//   score(k, v) = s_k + z[k, v] - lse_k,   lse_k = log sum_v exp z[k, v]
// the M best of the K V candidates, ties to the lowest k V + v.  A finished beam
// has one candidate, (k, eos) with score s_k.  A beam whose s_k is not finite,
// and a candidate whose score is NaN, count as -inf; where fewer than M
// candidates are above -inf, the lowest unused k V + v fill up with -inf.
//
// One pass over the logits finds both sums and candidates: a block streams a
// segment of a beam's row, each thread keeping its running maximum and sum of
// exponentials, and its largest element with the vector that held it.  A value
// that M of the 256 threads' maxima reach bounds the M-th largest element from
// below, so the M best elements of the segment all lie with the few more than M
// threads above the bound.  Each thread also leaves the maximum of every few
// batches in shared memory (16 bits of it, rounded down), so of those threads'
// vectors only the ones that can hold such an element are loaded again (all of
// them would be M / 256 of the segment, but in pieces of 16 bytes, which cost HBM a
// quarter of the pass), and the few elements above the bound are sorted by
// counting.  The pass costs one exponential per element and one
// comparison per vector, like a plain logsumexp, and is bound by HBM; what comes
// after it (bound, second look, ranks) is latency that nothing hides when all
// blocks fit at once.  32 x 8 beams x 200000 FP32: 43 us (4.8 TB/s), 34 us without
// that end; the merge takes 5 more.
// A second kernel merges an item's segments: lse_k, the candidates' scores in
// FP64 (scores of different beams lie next to one another; in FP32 their
// rounding would decide), and the M best, by the same bound.
//
// Elements are dealt to threads by their index in the row, never by address,
// so equal rows give equal sums bit for bit and their ties stay ties.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <vector>

#include "chunked_ce.cuh"
#include "extents.cuh"
#include "layer_norm.cuh"

namespace flce {

constexpr int kBeamThreads = 256;
constexpr int kBeamMaxBeams = 64;
constexpr int kBeamMaxSelect = 64;
constexpr int kBeamUnroll = 4;            // vectors in flight per thread
constexpr int kBeamResident = 4;          // blocks per SM the registers are limited for
constexpr int kBeamGroups = 32;           // recorded maxima per thread, at most
constexpr int kBeamList = 1024;           // elements above the bound that are sorted in one go
constexpr int64_t kBeamMinSegment = 4096; // elements
constexpr int kBeamEnough = 16;           // keys above a bound that are not worth thinning out
constexpr int kBeamFew = 128;             // candidates that are cheaper to rank than to bound
constexpr int kBeamCluster = 8;           // blocks per item when one launch does it all
constexpr int64_t kBeamClusterShare = 16384;  // elements such a block reads, at most
constexpr int kBeamMaxItems = 4096;       // candidates merged per batch item: K x segments x M

// Total order of (value, index): larger value first, then the lower index; a key
// of 0 is below every element.  -0 and +0 are equal values.
__device__ __forceinline__ uint32_t beam_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float beam_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t beam_key(float x, uint32_t index) {
  return (static_cast<uint64_t>(beam_order(x)) << 32) | (0xffffffffu - index);
}

// The largest element of a vector (NaN does not count).
template <typename T>
__device__ __forceinline__ float beam_max(const uint4& v) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    auto pair = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
    const float2 f = __bfloat1622float2(
        __hmax2(__hmax2(pair(v.x), pair(v.y)), __hmax2(pair(v.z), pair(v.w))));
    return fmaxf(f.x, f.y);
  }
}
// The elements of a vector, as pairs.
template <typename T>
__device__ __forceinline__ void beam_unpack(const uint4& v, float2 (&x)[8 / int(sizeof(T))]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}

// A bound from below on the select-th largest of the block's items, from one key
// per thread, the largest of its items (0: none); keys may be equal.  Any value
// that at least `select` keys reach is such a bound, the fewer reach it the
// better.  Every group of 256 / P threads (P groups, a power of two >= select) gives
// its maximum: at least `select` keys are no smaller than the least of those.  Where
// many are, the block bisects from there to the largest key, counting the keys
// at a barrier, until at most a quarter more than `select` are left, or 16.  (Ranking
// those keys against one another for the exact one cost more: the whole call at
// 18 x 16 x 2000 BF16, 32 wanted, took 21.3 us of device time against 13.3.)  Returns
// 0 where fewer than `select` threads hold a key.  Every thread of the block calls it.
struct BeamBound {
  uint64_t warp_min[kBeamThreads / 32];
  uint64_t warp_max[kBeamThreads / 32];
};
__device__ __forceinline__ uint64_t beam_bound(uint64_t mine, int select, BeamBound& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t top = mine;
  for (int o = 1; o < 32 && o * 2 * select <= kBeamThreads; o <<= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  uint64_t low = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (lane == 0) {
    sm.warp_min[warp] = low;
    sm.warp_max[warp] = top;
  }
  __syncthreads();
  low = sm.warp_min[0];
  top = sm.warp_max[0];
#pragma unroll
  for (int w = 1; w < kBeamThreads / 32; ++w) {
    low = min(low, sm.warp_min[w]);
    top = max(top, sm.warp_max[w]);
  }
  if (low == 0) low = 1;  // a group without a key
  const int enough = max(select + select / 4, kBeamEnough);
  const int held = __syncthreads_count(mine >= low);
  if (held < select) return 0;
  if (held > enough) {
    uint64_t high = top + 1;  // reached by none
    for (int i = 0; i < 24 && high - low > 1; ++i) {
      const uint64_t mid = low + (high - low) / 2;
      const int n = __syncthreads_count(mine >= mid);
      if (n >= select) {
        low = mid;
        if (n <= enough) break;
      } else {
        high = mid;
      }
    }
  }
  return low;
}

// Calls use(i, r) for every i < n with r = how many j have above(i, j): 1 to 8
// threads per i, as many as there are.  Every thread of the block calls it.
template <typename Above, typename Use>
__device__ __forceinline__ void beam_ranks(int n, Above&& above, Use&& use) {
  int team = 1;
  while (team < 8 && n * team * 2 <= kBeamThreads) team *= 2;
  const int part = int(threadIdx.x) & (team - 1);
  for (int i0 = 0; i0 < n; i0 += kBeamThreads / team) {
    const int i = i0 + int(threadIdx.x) / team;
    int r = 0;
    if (i < n) {
#pragma unroll 4
      for (int j = part; j < n; j += team) r += above(i, j) ? 1 : 0;
    }
    for (int o = team / 2; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (i < n && part == 0) use(i, r);
  }
}

struct BeamPartArgs {
  const void* logits;
  int64_t ld, vocab, segment;
  int splits, select;
  int group_shift;          // batches per recorded maximum, as a power of two
  const float* scores;      // [rows]
  const uint8_t* finished;  // [rows] or nullptr
  float* part_m;            // [rows][splits]: maximum, and sum of exp(z - maximum)
  double* part_s;
  float* cand_z;            // [rows][splits][select], best first; index -1: none
  int* cand_v;
};

__device__ __forceinline__ bool beam_is_live(float score) {
  return fabsf(score) <= 3.402823466e38f;  // finite
}

struct BeamUnitShared {
  BeamBound bound;
  uint64_t list[kBeamList];
  uint16_t owners[kBeamThreads];
  int n_owners, n_list;
  float red_m[kBeamThreads / 32];
  double red_s[kBeamThreads / 32];
};

// Segment `part` of a live beam's row, by a whole block.  `seen`: [groups][threads],
// the upper half of beam_order(maximum).
template <typename T>
__device__ __forceinline__ void beam_unit(const BeamPartArgs& a, int64_t row, int part,
                                          BeamUnitShared& sm, uint16_t* seen) {
  constexpr int VN = 16 / int(sizeof(T));
  constexpr uint32_t kNegInf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  const int64_t begin = int64_t(part) * a.segment, end = min(a.vocab, begin + a.segment);
  const int count = int(max(int64_t(0), (end - begin + VN - 1) / VN));  // vectors

  float m = -INFINITY, best = -INFINITY;
  float2 s2 = make_float2(0.0f, 0.0f);
  uint32_t best_at = 0;  // first element of the vector that holds `best`
  // The next batch is loaded before the current one is used: a block alone, or
  // with few neighbours, would otherwise leave HBM idle between its loads.
  uint4 raw[kBeamUnroll];
  // Batches of whole vectors need no look at their ends: vectors [first, whole).
  const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(z)) & 15u;
  const uintptr_t body = reinterpret_cast<uintptr_t>(z + begin) - off;
  const int first = off != 0 && begin == 0 ? 1 : 0;
  const int whole = int(min(int64_t(count), (a.vocab - begin) / VN - (off != 0 ? 1 : 0)));
  auto fetch = [&](int j0) {
    if (j0 >= first && j0 + (kBeamUnroll - 1) * kBeamThreads < whole) {
      const uintptr_t at = body + int64_t(j0) * 16;
      if (off == 0) {
#pragma unroll
        for (int u = 0; u < kBeamUnroll; ++u)
          raw[u] = *reinterpret_cast<const uint4*>(at + u * kBeamThreads * 16);
      } else {
#pragma unroll
        for (int u = 0; u < kBeamUnroll; ++u) raw[u] = load16_shifted(at + u * kBeamThreads * 16, off);
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < kBeamUnroll; ++u) {
      const int j = j0 + u * kBeamThreads;
      // vectors end at the row's end, not the segment's: a segment is whole vectors
      if (j < count) raw[u] = load16_any<T>(z, begin + int64_t(j) * VN, a.vocab, kNegInf);
      else raw[u] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
    }
  };
  fetch(tid);
  float gm = -INFINITY;  // maximum of the current group of batches
  int batch = 0;
  for (int j0 = tid; j0 < count; j0 += kBeamUnroll * kBeamThreads) {
    uint4 cur[kBeamUnroll];
#pragma unroll
    for (int u = 0; u < kBeamUnroll; ++u) cur[u] = raw[u];
    fetch(j0 + kBeamUnroll * kBeamThreads);
    float bm = -INFINITY;
#pragma unroll
    for (int u = 0; u < kBeamUnroll; ++u) {
      const float vm = beam_max<T>(cur[u]);
      if (vm > best) {
        best = vm;
        best_at = uint32_t(begin) + uint32_t(j0 + u * kBeamThreads) * VN;
      }
      bm = fmaxf(bm, vm);
    }
    // Written at every batch; the group's last one stays.
    gm = (batch & ((1 << a.group_shift) - 1)) == 0 ? bm : fmaxf(gm, bm);
    seen[(batch >> a.group_shift) * kBeamThreads + tid] = uint16_t(beam_order(gm) >> 16);
    ++batch;
    if (bm > m) {
      s2 = __fmul2_rn(s2, ln_both(fast_exp2((m - bm) * kLog2e)));
      m = bm;
    }
    // Before the first element above -inf the terms are taken against 0: -inf
    // adds nothing, and a NaN still reaches the sum.
    const float2 base = ln_both(m == -INFINITY ? 0.0f : -m);
#pragma unroll
    for (int u = 0; u < kBeamUnroll; ++u) {
      float2 x[VN / 2];
      beam_unpack<T>(cur[u], x);
#pragma unroll
      for (int j = 0; j < VN / 2; ++j) {
        const float2 t = __fmul2_rn(__fadd2_rn(x[j], base), ln_both(kLog2e));
        s2 = __fadd2_rn(s2, make_float2(fast_exp2(t.x), fast_exp2(t.y)));
      }
    }
  }
  const float s = s2.x + s2.y;

  // The segment's maximum and sum, added in a fixed order.
  float bm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
  if (lane == 0) sm.red_m[warp] = bm;
  const uint64_t mine = best > -INFINITY ? beam_key(best, best_at) : 0;
  if (tid == 0) sm.n_owners = sm.n_list = 0;
  __syncthreads();
  bm = sm.red_m[0];
#pragma unroll
  for (int w = 1; w < kBeamThreads / 32; ++w) bm = fmaxf(bm, sm.red_m[w]);
  double ds = m == -INFINITY ? double(s) : double(s) * double(fast_exp2((m - bm) * kLog2e));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
  if (lane == 0) sm.red_s[warp] = ds;
  // Threads' keys are distinct (no two hold the same vector): few more than `select`
  // of them reach the bound.
  const uint64_t bound = beam_bound(mine, a.select, sm.bound);
  if (mine != 0 && mine >= bound) sm.owners[atomicAdd(&sm.n_owners, 1)] = uint16_t(tid);
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < kBeamThreads / 32; ++w) t += sm.red_s[w];
    const int64_t at = row * a.splits + part;
    a.part_m[at] = bm;
    a.part_s[at] = t;
  }
  __syncthreads();

  // Elements of the owners' vectors whose (value, vector) is not below the bound.
  const int size = kBeamUnroll << a.group_shift;  // vectors per group
  const int per = (count + kBeamThreads - 1) / kBeamThreads;  // vectors per thread
  const int groups = (per + size - 1) / size;
  const int work = sm.n_owners * groups;
  const uint32_t least = uint32_t(bound >> 48);
  auto scan = [&](auto&& take) {
    for (int w = tid; w < work; w += kBeamThreads) {
      const int q = w / groups, g = w - q * groups, owner = sm.owners[q];
      // the owner's last group may have no batch, and no record
      if (owner + g * size * kBeamThreads >= count || seen[g * kBeamThreads + owner] < least) continue;
      for (int u0 = 0; u0 < size; u0 += kBeamUnroll) {
        const int j0 = owner + (g * size + u0) * kBeamThreads;
        uint4 raw[kBeamUnroll];  // a batch's loads before any of them is used
#pragma unroll
        for (int u = 0; u < kBeamUnroll; ++u) {
          const int j = j0 + u * kBeamThreads;
          raw[u] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
          if (j < count) raw[u] = load16_any<T>(z, begin + int64_t(j) * VN, a.vocab, kNegInf);
        }
#pragma unroll
        for (int u = 0; u < kBeamUnroll; ++u) {
          const uint32_t at = uint32_t(begin) + uint32_t(j0 + u * kBeamThreads) * VN;
          const float top = beam_max<T>(raw[u]);
          if (!(top > -INFINITY) || beam_key(top, at) < bound) continue;
          float2 x[VN / 2];
          beam_unpack<T>(raw[u], x);
          auto one = [&](float v, uint32_t i) {
            if (v > -INFINITY && beam_key(v, at) >= bound) take(beam_key(v, at + i));
          };
#pragma unroll
          for (int i = 0; i < VN / 2; ++i) {
            one(x[i].x, 2 * i);
            one(x[i].y, 2 * i + 1);
          }
        }
      }
    }
  };
  scan([&](uint64_t key) {
    const int at = atomicAdd(&sm.n_list, 1);
    if (at < kBeamList) sm.list[at] = key;
  });
  __syncthreads();
  const int n = sm.n_list;
  const int64_t out = (row * a.splits + part) * a.select;
  auto put = [&](int slot, uint64_t key) {
    a.cand_z[out + slot] = beam_value(uint32_t(key >> 32));
    a.cand_v[out + slot] = int(0xffffffffu - uint32_t(key));
  };
  if (n <= kBeamList) {
    // The list's order is that of the atomics; the keys are distinct, so their
    // ranks are not.
    beam_ranks(n, [&](int i, int j) { return sm.list[j] > sm.list[i]; },
               [&](int i, int r) {
                 if (r < a.select) put(r, sm.list[i]);
               });
    for (int i = n + tid; i < a.select; i += kBeamThreads) a.cand_v[out + i] = -1;
    return;
  }
  // More elements above the bound than the list holds (a few threads own nearly
  // all large elements): the largest one below the last, `select` times over.
  uint64_t last = ~uint64_t(0);
  for (int slot = 0; slot < a.select; ++slot) {
    uint64_t top = 0;
    scan([&](uint64_t key) {
      if (key < last && key > top) top = key;
    });
    __syncthreads();
    sm.list[tid] = top;
    __syncthreads();
    for (int h = kBeamThreads / 2; h > 0; h >>= 1) {
      if (tid < h) sm.list[tid] = max(sm.list[tid], sm.list[tid + h]);
      __syncthreads();
    }
    last = sm.list[0];  // never 0: more than kBeamList >= select elements qualify
    if (tid == 0) put(slot, last);
  }
}

template <typename T>
__global__ void __launch_bounds__(kBeamThreads, kBeamResident) beam_partials_kernel(const BeamPartArgs a) {
  extern __shared__ uint64_t dyn[];
  __shared__ BeamUnitShared sm;
  const int64_t row = blockIdx.x / a.splits;
  if (!beam_is_live(a.scores[row]) || (a.finished && a.finished[row])) return;
  grid_launch_dependents();
  beam_unit<T>(a, row, int(blockIdx.x - row * a.splits), sm, reinterpret_cast<uint16_t*>(dyn));
}

struct BeamMergeArgs {
  int beams, splits, select;
  int64_t vocab, eos;
  const float* scores;
  const uint8_t* finished;
  const float* part_m;
  const double* part_s;
  const float* cand_z;
  const int* cand_v;
  float* out_scores;  // [batch][select]
  int64_t* parents;
  int64_t* tokens;
};

// Totals in FP64 as ordered integers (NaN: 0, below -inf); flat candidate index.
__device__ __forceinline__ uint64_t beam_order64(double x) {
  if (x != x) return 0;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (uint64_t(1) << 63));
}
__device__ __forceinline__ double beam_value64(uint64_t o) {
  return __longlong_as_double(static_cast<long long>((o >> 63) ? (o & ~(uint64_t(1) << 63)) : ~o));
}

struct BeamMergeShared {
  BeamBound bound;
  double lse[kBeamMaxBeams];
  int n_list;
  uint32_t chosen[kBeamMaxSelect];
};

// Batch item b, by a whole block; dyn: 24 bytes per candidate.
__device__ __forceinline__ void beam_merge_item(const BeamMergeArgs& a, int64_t b,
                                                BeamMergeShared& sm, uint64_t* dyn) {
  constexpr int kAhead = 4;  // items per thread loaded before the sums are known
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Item i is candidate i / lists of list i % lists: the lists are sorted, and dealt
  // this way their best entries lie with different threads, which keeps the
  // bound tight (list by list, 64 candidates of 64 lists took 129 us to merge).
  const int lists = a.beams * a.splits, items = lists * a.select;
  const uint32_t vocab = uint32_t(a.vocab);
  uint64_t* tot = dyn;                                       // [items]
  uint32_t* idx = reinterpret_cast<uint32_t*>(tot + items);  // [items]
  uint32_t* sel_i = idx + items;                             // [items]: what is above the bound
  uint64_t* sel_t = reinterpret_cast<uint64_t*>(sel_i + items);  // 16 bytes per item behind tot
  const float* scores = a.scores + b * a.beams;
  const uint8_t* finished = a.finished ? a.finished + b * a.beams : nullptr;
  const int64_t at0 = b * items;
  auto place = [&](int i) { return (i % lists) * a.select + i / lists; };
  float az[kAhead];
  int av[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int i = tid + u * kBeamThreads;
    // dead and finished beams' entries were never written: loaded, not used
    az[u] = i < items ? a.cand_z[at0 + place(i)] : 0.0f;
    av[u] = i < items ? a.cand_v[at0 + place(i)] : -1;
  }
  if (tid == 0) sm.n_list = 0;
  const double ninf = -static_cast<double>(INFINITY);
  for (int k = warp; k < a.beams; k += kBeamThreads / 32) {
    const int64_t at = (b * a.beams + k) * a.splits;
    float pm = lane < a.splits ? a.part_m[at + lane] : -INFINITY;
    double ps = lane < a.splits ? a.part_s[at + lane] : 0.0;
    if (!beam_is_live(scores[k]) || (finished && finished[k])) continue;
    float m = pm;
    for (int p = lane + 32; p < a.splits; p += 32) m = fmaxf(m, a.part_m[at + p]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // an all -inf segment's sum is 0, or NaN where it holds one
    double s = 0.0;
    for (int p = lane; p < a.splits; p += 32) {
      if (p != lane) {
        pm = a.part_m[at + p];
        ps = a.part_s[at + p];
      }
      s += pm == m || pm == -INFINITY ? ps : ps * exp(double(pm) - double(m));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sm.lse[k] = double(m) + log(s);
  }
  __syncthreads();

  uint64_t top = 0;
  auto item = [&](int i, float z, int v) {
    const int k = (i % lists) / a.splits;
    double t = ninf;
    const float s = scores[k];
    if (beam_is_live(s)) {
      if (finished && finished[k]) {
        v = int(a.eos);
        if (i == k * a.splits) t = double(s);
      } else if (v >= 0) {
        t = double(s) + double(z) - sm.lse[k];
      }
    }
    const uint64_t o = t > ninf ? beam_order64(t) : 0;  // NaN and -inf: none
    tot[i] = o;
    idx[i] = uint32_t(k) * vocab + uint32_t(v);
    top = max(top, o);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (tid + u * kBeamThreads < items) item(tid + u * kBeamThreads, az[u], av[u]);
  for (int i = tid + kAhead * kBeamThreads; i < items; i += kBeamThreads)
    item(i, a.cand_z[at0 + place(i)], a.cand_v[at0 + place(i)]);
  // Up to kBeamFew candidates are ranked as they are.
  uint64_t bound = 0;
  if (items > kBeamFew)  // the same for the whole block
    bound = beam_bound(top, a.select, sm.bound);
  else
    __syncthreads();
  for (int i = tid; i < items; i += kBeamThreads)
    if (tot[i] != 0 && tot[i] >= bound) {
      const int at = atomicAdd(&sm.n_list, 1);
      sel_t[at] = tot[i];
      sel_i[at] = idx[i];
    }
  __syncthreads();
  const int n = sm.n_list;
  beam_ranks(n,
             [&](int i, int j) {
               return sel_t[j] > sel_t[i] || (sel_t[j] == sel_t[i] && sel_i[j] < sel_i[i]);
             },
             [&](int i, int r) {
               if (r >= a.select) return;
               const uint32_t f = sel_i[i];
               const int64_t at = b * a.select + r;
               a.out_scores[at] = float(beam_value64(sel_t[i]));
               a.parents[at] = int64_t(f / vocab);
               a.tokens[at] = int64_t(f % vocab);
               sm.chosen[r] = f;
             });
  __syncthreads();
  if (tid == 0 && n < a.select) {  // fewer candidates than wanted: the lowest unused indices
    uint32_t f = 0;
    for (int r = n; r < a.select; ++r, ++f) {
      for (int j = 0; j < n; ++j)
        if (sm.chosen[j] == f) {
          ++f;
          j = -1;
        }
      const int64_t at = b * a.select + r;
      a.out_scores[at] = -INFINITY;
      a.parents[at] = int64_t(f / vocab);
      a.tokens[at] = int64_t(f % vocab);
    }
  }
}

// One block per batch item.
__global__ void __launch_bounds__(kBeamThreads) beam_merge_kernel(const BeamMergeArgs a) {
  extern __shared__ uint64_t dyn[];
  __shared__ BeamMergeShared sm;
  grid_dependency_wait();
  beam_merge_item(a, blockIdx.x, sm, dyn);
}

// Few items with little to read: a cluster of blocks per item, a segment each, and the
// first block merges them once all have arrived at the cluster's barrier: one launch.
template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 1)
    beam_cluster_kernel(const BeamPartArgs a, const BeamMergeArgs g) {
  extern __shared__ uint64_t dyn[];
  __shared__ union {
    BeamUnitShared unit;
    BeamMergeShared merge;
  } sm;
  const int64_t b = blockIdx.x / kBeamCluster;
  const uint32_t rank = cluster_cta_rank();
  for (int u = int(rank); u < g.beams * a.splits; u += kBeamCluster) {
    const int k = u / a.splits;
    const int64_t row = b * g.beams + k;
    if (beam_is_live(a.scores[row]) && !(a.finished && a.finished[row]))
      beam_unit<T>(a, row, u - k * a.splits, sm.unit, reinterpret_cast<uint16_t*>(dyn));
    __syncthreads();  // the next segment uses the same shared memory
  }
  cluster_sync_all();  // the other blocks' partials are written
  if (rank == 0) beam_merge_item(g, b, sm.merge, dyn);
}

struct BeamPlan {
  bool cluster;
  int splits;
  int64_t segment;
  size_t off_s, off_m, off_z, off_v, total;
};

// Segments per row: as many as keep all blocks resident at once (a second, partly
// filled wave costs more than longer segments: 19.5 against 14.5 us for 64 rows of
// 50001), none shorter than kBeamMinSegment, and no more candidates per item than
// one block merges.
static BeamPlan plan_beam(int64_t batch, int64_t beams, int64_t vocab, int64_t select) {
  BeamPlan p{};
  const int64_t rows = std::max<int64_t>(1, batch * beams);
  int64_t s = std::max<int64_t>(1, int64_t(kBeamResident) * kLnSms / rows);
  s = std::min({s, std::max<int64_t>(1, vocab / kBeamMinSegment),
                std::max<int64_t>(1, kBeamMaxItems / (beams * select))});
  // A cluster per item while all of them fit at once and each of its blocks has at most
  // one segment to read, and a short one (14 x 1 beam x 31398 FP32: 16.8 us per call
  // and 9.9 on the device in one launch, 18.3 and 10.7 in two; with two segments per
  // block 22.5 against 18.1 us per call, with 65536 elements per block 14.2 against
  // 10.8 us on the device).
  p.cluster = batch * kBeamCluster <= kLnSms && beams <= kBeamCluster &&
              beams * vocab <= kBeamCluster * kBeamClusterShare;
  if (p.cluster)
    s = std::min<int64_t>({kBeamCluster / beams, std::max<int64_t>(1, vocab / kBeamMinSegment),
                           std::max<int64_t>(1, kBeamMaxItems / (beams * select))});
  p.segment = cdiv(cdiv(vocab, s), 8) * 8;
  p.splits = int(cdiv(vocab, p.segment));
  const size_t units = size_t(rows) * size_t(p.splits);
  size_t o = 0;
  p.off_s = o;  o = align_up(o + units * 8);
  p.off_m = o;  o = align_up(o + units * 4);
  p.off_z = o;  o = align_up(o + units * size_t(select) * 4);
  p.off_v = o;  o = align_up(o + units * size_t(select) * 4);
  p.total = o;
  return p;
}

template <typename T>
static int beam_launch_cluster(const BeamPartArgs& a, const BeamMergeArgs& g, int64_t batch,
                               size_t smem, cudaStream_t cs) {
  auto kern = beam_cluster_kernel<T>;
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBeamMaxItems * 24) !=
          cudaSuccess)
    return FLCE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(batch * kBeamCluster));
  cfg.blockDim = dim3(kBeamThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = cs;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBeamCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a, g) != cudaSuccess) return FLCE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

static bool beam_sizes_ok(int64_t batch, int64_t beams, int64_t vocab, int64_t select) {
  return batch >= 0 && beams >= 1 && beams <= kBeamMaxBeams && vocab >= 1 && select >= 1 &&
         select <= kBeamMaxSelect && batch <= kMaxDim / kBeamMaxItems &&
         vocab <= kMaxDim / beams && select <= beams * vocab;
}

// ---------------------------------------------------------------- reordering of states

constexpr int kReorderStates = 16;  // per launch
constexpr int kReorderThreads = 256;

struct ReorderState {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_batch, src_beam, dst_batch, dst_beam;  // strides in bytes
  int64_t outer, outer_stride, inner;                // pieces of `inner` bytes
};
struct ReorderArgs {
  ReorderState st[kReorderStates];
  const int64_t* parents;
  int64_t batch;
  int beams;
  unsigned* err;
};

// dst[b, k] = src[b, parents[b, k]].  A thread takes one vector position of all
// K beams: it loads the parents' values, then stores.  In place (kInPlace) that
// makes the permutation safe without scratch memory, as no other thread touches
// this position; beams that keep their own state are neither read nor written.
// Otherwise groups of KM beams at a time; a parent shared by several beams is
// read from HBM once, by whichever load comes first.  Bound by HBM: four states of
// 16 x 8 beams x 8 x 777 x 128 BF16 into second buffers in 214 us (6.2 TB/s, 96% of
// the copy bandwidth).
template <typename V, int KM, bool kInPlace>
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int parent[kBeamMaxBeams];
  const ReorderState& st = a.st[blockIdx.z];
  const int64_t per = st.inner / int64_t(sizeof(V)), total = st.outer * per;
  for (int64_t b = blockIdx.y; b < a.batch; b += gridDim.y) {
    __syncthreads();
    if (threadIdx.x < a.beams) {
      int64_t p = a.parents[b * a.beams + threadIdx.x];
      if (p < 0 || p >= a.beams) {
        if (blockIdx.x == 0) atomicOr(a.err, kDevErrBadIndex);
        p = threadIdx.x;
      }
      parent[threadIdx.x] = int(p);
    }
    __syncthreads();
    for (int64_t i = int64_t(blockIdx.x) * kReorderThreads + threadIdx.x; i < total;
         i += int64_t(gridDim.x) * kReorderThreads) {
      const int64_t o = i / per, c = i - o * per;
      const uint8_t* src = st.src + b * st.src_batch + o * st.outer_stride + c * int64_t(sizeof(V));
      uint8_t* dst = st.dst + b * st.dst_batch + o * st.outer_stride + c * int64_t(sizeof(V));
      for (int k0 = 0; k0 < a.beams; k0 += KM) {
        V v[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j)
          if (k0 + j < a.beams && !(kInPlace && parent[k0 + j] == k0 + j))
            v[j] = *reinterpret_cast<const V*>(src + parent[k0 + j] * st.src_beam);
#pragma unroll
        for (int j = 0; j < KM; ++j)
          if (k0 + j < a.beams && !(kInPlace && parent[k0 + j] == k0 + j))
            *reinterpret_cast<V*>(dst + (k0 + j) * st.dst_beam) = v[j];
      }
    }
  }
}

// Extents [first, last), in ascending order of their bases, that are slices of one buffer's
// entries (a cache's layers, keys and values behind [batch, beams]): the same strides,
// each slice behind the one before, all of them within the stride of the entries. Such
// slices share nothing, and need not be looked at in pairs (160 of them: 460 us).
static bool reorder_slices(const Extent* first, const Extent* last) {
  const int big = first->stride[0] >= first->stride[1] ? 0 : 1;
  const uint64_t large = uint64_t(first->stride[big]), small = uint64_t(first->stride[1 - big]);
  uint64_t end = first->base;
  for (const Extent* e = first; e != last; ++e) {
    if (e->base < end || e->stride[0] != first->stride[0] || e->stride[1] != first->stride[1]) return false;
    end = e->base + uint64_t(e->count[2] - 1) * uint64_t(e->stride[2]) + uint64_t(e->inner);
  }
  const uint64_t span = end - first->base;
  if (small != 0 && span > small) return false;
  return large == 0 || span + uint64_t(first->count[1 - big] - 1) * small <= large;
}
// FLCE_ERR_INVALID_ARG where a block could read or write what another one writes: a
// state written over another one, over one that is read or over the parents.
static int reorder_check(const flce_beam_state* states, int64_t count, const int64_t* parents,
                         int64_t batch, int64_t beams) try {
  std::vector<Extent> all;
  all.reserve(size_t(2 * count + 1));
  all.push_back(make_extent(parents, {0, 0, 0}, {1, 1, 1}, batch * beams * 8, false));
  for (int64_t i = 0; i < count; ++i) {
    const flce_beam_state& s = states[i];
    if (s.outer * s.inner == 0) continue;
    const int64_t counts[3] = {batch, beams, s.outer};
    all.push_back(make_extent(s.dst, {s.dst_batch_stride, s.dst_beam_stride, s.outer_stride}, counts,
                              s.inner, true));
    if (s.src != s.dst)
      all.push_back(make_extent(s.src, {s.src_batch_stride, s.src_beam_stride, s.outer_stride}, counts,
                                s.inner, false));
  }
  std::sort(all.begin(), all.end(),
            [](const Extent& a, const Extent& b) { return a.base < b.base; });
  for (size_t first = 0, last; first < all.size(); first = last) {
    uint64_t end = all[first].end;  // of those up to `last`, which lie among one another
    for (last = first + 1; last < all.size() && all[last].base < end; ++last)
      end = std::max(end, all[last].end);
    if (reorder_slices(all.data() + first, all.data() + last)) continue;
    for (size_t i = first; i < last; ++i)
      for (size_t j = i + 1; j < last && all[j].base < all[i].end; ++j)
        if ((all[i].written || all[j].written) && extents_overlap(all[i], all[j]))
          return FLCE_ERR_INVALID_ARG;
  }
  return FLCE_OK;
} catch (...) {  // no memory for the list
  return FLCE_ERR_UNSUPPORTED;
}

}  // namespace flce

extern "C" size_t flce_beam_select_workspace_size(int64_t batch, int64_t beams, int64_t vocab,
                                                  int64_t select) {
  return beam_sizes_ok(batch, beams, vocab, select) ? plan_beam(batch, beams, vocab, select).total
                                                    : 0;
}

extern "C" int flce_beam_select(const void* logits, int dtype, int64_t batch, int64_t beams,
                                int64_t vocab, int64_t ld, const float* scores,
                                const uint8_t* finished, int64_t eos_token, int64_t num_select,
                                float* out_scores, int64_t* parents, int64_t* tokens,
                                void* workspace, size_t ws_bytes, flce_stream_t stream) {
  NvtxRange range("flce_beam_select");
  if (!beam_sizes_ok(batch, beams, vocab, num_select) || !ln_dtype_ok(dtype) ||
      !ln_ld_ok(batch * beams, vocab, ld))
    return FLCE_ERR_INVALID_ARG;
  if (finished != nullptr && (eos_token < 0 || eos_token >= vocab)) return FLCE_ERR_INVALID_ARG;
  if (batch == 0) return FLCE_OK;
  if (logits == nullptr || scores == nullptr || out_scores == nullptr || parents == nullptr ||
      tokens == nullptr || !aligned(logits, dtype == FLCE_F32 ? 4 : 2) || !aligned(scores, 4) ||
      !aligned(out_scores, 4) || !aligned(parents, 8) || !aligned(tokens, 8))
    return FLCE_ERR_INVALID_ARG;
  const BeamPlan p = plan_beam(batch, beams, vocab, num_select);
  if (workspace == nullptr || !aligned(workspace, 16) || ws_bytes < p.total)
    return FLCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t rows = batch * beams;
  BeamPartArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.vocab = vocab;
  a.segment = p.segment;
  a.splits = p.splits;
  a.select = int(num_select);
  a.scores = scores;
  a.finished = finished;
  a.part_s = reinterpret_cast<double*>(ws + p.off_s);
  a.part_m = reinterpret_cast<float*>(ws + p.off_m);
  a.cand_z = reinterpret_cast<float*>(ws + p.off_z);
  a.cand_v = reinterpret_cast<int*>(ws + p.off_v);
  BeamMergeArgs g{};
  g.beams = int(beams);
  g.splits = p.splits;
  g.select = int(num_select);
  g.vocab = vocab;
  g.eos = eos_token;
  g.scores = scores;
  g.finished = finished;
  g.part_m = a.part_m;
  g.part_s = a.part_s;
  g.cand_z = a.cand_z;
  g.cand_v = a.cand_v;
  g.out_scores = out_scores;
  g.parents = parents;
  g.tokens = tokens;
  const size_t smem = size_t(beams) * size_t(p.splits) * size_t(num_select) * 24;
  const int64_t batches = cdiv(p.segment, int64_t(kBeamUnroll) * kBeamThreads * (dtype == FLCE_F32 ? 4 : 8));
  while (cdiv(batches, int64_t(1) << a.group_shift) > kBeamGroups) ++a.group_shift;
  const size_t seen =
      size_t(cdiv(batches, int64_t(1) << a.group_shift)) * kBeamThreads * sizeof(uint16_t);
  const double bytes = double(rows) * double(vocab) * (dtype == FLCE_F32 ? 4 : 2);
  if (p.cluster) {
    LaunchScope scope(KF_BEAM_PART, 0.0, bytes, cs);
    return dtype == FLCE_BF16 ? beam_launch_cluster<__nv_bfloat16>(a, g, batch, std::max(seen, smem), cs)
                              : beam_launch_cluster<float>(a, g, batch, std::max(seen, smem), cs);
  }
  {
    LaunchScope scope(KF_BEAM_PART, 0.0, bytes, cs);
    const unsigned grid = unsigned(rows * p.splits);
    if (dtype == FLCE_BF16)
      beam_partials_kernel<__nv_bfloat16><<<grid, kBeamThreads, seen, cs>>>(a);
    else
      beam_partials_kernel<float><<<grid, kBeamThreads, seen, cs>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FLCE_ERR_CUDA;
  }
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kBeamMaxItems * 24) != cudaSuccess)
    return FLCE_ERR_CUDA;
  LaunchScope scope(KF_BEAM_MERGE, 0.0, double(rows) * p.splits * (12.0 + 8.0 * double(num_select)), cs);
  // Launched while the first kernel still runs; its blocks wait for that kernel's
  // end (griddepcontrol.wait) before they read anything.
  return launch_dependent(beam_merge_kernel, dim3(unsigned(batch)), dim3(kBeamThreads), smem, cs, g);
}

extern "C" int flce_beam_reorder(const flce_beam_state* states, int64_t count,
                                 const int64_t* parents, int64_t batch, int64_t beams,
                                 flce_stream_t stream) {
  NvtxRange range("flce_beam_reorder");
  if (count < 0 || batch < 0 || batch > kMaxDim || beams < 1 || beams > kBeamMaxBeams ||
      (count > 0 && states == nullptr))
    return FLCE_ERR_INVALID_ARG;
  if (count == 0 || batch == 0) return FLCE_OK;
  if (parents == nullptr || !aligned(parents, 8)) return FLCE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    const flce_beam_state& s = states[i];
    if (s.src == nullptr || s.dst == nullptr || s.outer < 0 || s.inner < 0 || s.outer_stride < 0 ||
        s.src_batch_stride < 0 || s.src_beam_stride < 0 || s.dst_batch_stride < 0 ||
        s.dst_beam_stride < 0 || (s.outer > 1 && s.outer_stride < s.inner) ||
        (s.inner > 0 && s.outer > (int64_t(1) << 46) / s.inner))
      return FLCE_ERR_INVALID_ARG;
    // the same buffer: in place, so the same layout
    if (s.src == s.dst && (s.src_batch_stride != s.dst_batch_stride ||
                           s.src_beam_stride != s.dst_beam_stride))
      return FLCE_ERR_INVALID_ARG;
  }
  int st = reorder_check(states, count, parents, batch, beams);
  if (st != FLCE_OK) return st;
  DeviceInfo* dev = nullptr;
  st = device_info(&dev);
  if (st != FLCE_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // States of one kind (in place or not, the same widest vector) share launches.
  for (int in_place = 0; in_place < 2; ++in_place) {
    // In place a thread holds a position of all beams, so more beams mean narrower vectors.
    const int widest = !in_place || beams <= 16 ? 16 : (beams <= 32 ? 8 : 4);
    for (int vb = 16; vb >= 1; vb >>= 1) {
      ReorderArgs a{};
      a.parents = parents;
      a.batch = batch;
      a.beams = int(beams);
      a.err = dev->err;
      int n = 0;
      int64_t most = 0;
      double bytes = 0.0;
      for (int64_t i = 0; i <= count; ++i) {
        if (i < count) {
          const flce_beam_state& s = states[i];
          const uint64_t bits = reinterpret_cast<uint64_t>(s.src) | reinterpret_cast<uint64_t>(s.dst) |
                                uint64_t(s.src_batch_stride) | uint64_t(s.src_beam_stride) |
                                uint64_t(s.dst_batch_stride) | uint64_t(s.dst_beam_stride) |
                                uint64_t(s.outer > 1 ? s.outer_stride : 0) | uint64_t(s.inner);
          int v = widest;
          while (bits % uint64_t(v) != 0) v >>= 1;
          if ((s.src == s.dst) != (in_place == 1) || v != vb || s.outer * s.inner == 0) continue;
          a.st[n++] = ReorderState{static_cast<const uint8_t*>(s.src), static_cast<uint8_t*>(s.dst),
                                   s.src_batch_stride, s.src_beam_stride, s.dst_batch_stride,
                                   s.dst_beam_stride, s.outer, s.outer_stride, s.inner};
          most = std::max(most, s.outer * (s.inner / vb));
          bytes += 2.0 * double(batch) * double(beams) * double(s.outer) * double(s.inner);
          if (n < kReorderStates) continue;
        }
        if (n == 0) continue;
        const unsigned gy = unsigned(std::min<int64_t>(batch, 65535));
        const int64_t want = std::max<int64_t>(1, int64_t(dev->num_sms) * 16 / (int64_t(gy) * n));
        const dim3 grid(unsigned(std::min<int64_t>(cdiv(most, kReorderThreads), want)), gy, unsigned(n));
        LaunchScope scope(KF_BEAM_REORDER, 0.0, bytes, cs);
        auto go = [&](auto kern) { kern<<<grid, kReorderThreads, 0, cs>>>(a); };
        if (in_place) {
          if (vb == 16 && beams <= 4) go(beam_reorder_kernel<uint4, 4, true>);
          else if (vb == 16 && beams <= 8) go(beam_reorder_kernel<uint4, 8, true>);
          else if (vb == 16) go(beam_reorder_kernel<uint4, 16, true>);
          else if (vb == 8 && beams <= 32) go(beam_reorder_kernel<uint2, 32, true>);
          else if (vb == 4) go(beam_reorder_kernel<uint32_t, 64, true>);
          else if (vb == 2) go(beam_reorder_kernel<uint16_t, 64, true>);
          else go(beam_reorder_kernel<uint8_t, 64, true>);
        } else {
          if (vb == 16) go(beam_reorder_kernel<uint4, 8, false>);
          else if (vb == 8) go(beam_reorder_kernel<uint2, 8, false>);
          else if (vb == 4) go(beam_reorder_kernel<uint32_t, 8, false>);
          else if (vb == 2) go(beam_reorder_kernel<uint16_t, 8, false>);
          else go(beam_reorder_kernel<uint8_t, 8, false>);
        }
        if (cudaGetLastError() != cudaSuccess) return FLCE_ERR_CUDA;
        n = 0;
        most = 0;
        bytes = 0.0;
      }
    }
  }
  return FLCE_OK;
}
