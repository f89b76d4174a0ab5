// Beam selection: the best continuations over a request's beams and vocabulary.
//
//   score(i, v) = s_i + x[i][v] - lse_i,  lse_i = log sum_w e^{x[i][w]}
//
// One pass over the logits, in which nothing is sorted: a warp reads blocks of
// 512 consecutive bytes of a row, adds up e^(x - m) and keeps each block's
// maximum (a word for 512 bytes).  Blocks rank like their maxima, so the K best
// elements lie in the K best blocks: K blocks with larger maxima (or equal ones
// and lower indices) hold K better elements than any element of another block.
// The same holds for the units of up to 32 blocks that a warp takes.  A second
// kernel ranks a request's units, the blocks of the best K, then the elements of
// the best K of those: some thousand keys in place of a million logits.
//
// Ranks are over (score, index) with the score as an unevaluated sum of two fp32
// numbers (48 bits): what does not depend on v is computed in 64 bits, and x added
// to it without an error.  Sums are fp32 over at most 256 terms a lane, then 64 bits
// over the units; e^x is off by 2^-22 of itself.
//
// What bounds it: the first kernel reads each logit once.
#include <cuda_fp16.h>

#include <type_traits>

#include "cache_ptx.cuh"
#include "step.cuh"

namespace smla {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanBatch = 4;                     // blocks a warp has in flight

template <class T>
struct Vec {
  static constexpr int kLane = 16 / sizeof(T);    // elements of a lane's 16 bytes
  static constexpr int kBlock = 32 * kLane;
};

__device__ __forceinline__ float element(const float* x) { return *x; }
__device__ __forceinline__ float element(const __half* x) { return __half2float(*x); }
__device__ __forceinline__ float element(const __nv_bfloat16* x) { return __bfloat162float(*x); }

__device__ __forceinline__ void unpack(uint4 v, float (&x)[4], const float*) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(uint4 v, float (&x)[8], const __nv_bfloat16*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(uint4 v, float (&x)[8], const __half*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
    x[2 * k] = f.x, x[2 * k + 1] = f.y;
  }
}

// A row's logits from the 16-byte boundary at or before its first: element e of
// the row is element e + before of `base`.
template <class T>
struct Row {
  const T* base;
  int before;
};
template <class T>
__device__ __forceinline__ Row<T> logits_row(const BeamParams& p, int64_t row) {
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  const int before = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  return {x - before, before};
}

// The lane's 16 bytes of a block, from element `at` of the row's base on; -infinity
// in place of elements before its first and from `end` on.
template <class T>
__device__ __forceinline__ uint4 load_lane(const Row<T>& r, int64_t at, int64_t end) {
  if (at >= r.before && at + Vec<T>::kLane <= end) return __ldcs(reinterpret_cast<const uint4*>(r.base + at));
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      w[k] = at + k >= r.before && at + k < end ? reinterpret_cast<const uint32_t*>(r.base)[at + k] : 0xff800000u;
    } else {
      constexpr uint32_t none = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
      uint32_t v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t i = at + 2 * k + e;
        v[e] = i >= r.before && i < end ? reinterpret_cast<const uint16_t*>(r.base)[i] : none;
      }
      w[k] = v[0] | v[1] << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Is the beam of this row one whose logits count?
__device__ __forceinline__ bool live_beam(const BeamParams& p, int64_t row) {
  if (p.finished != nullptr && p.finished[row] != 0) return false;
  const float s = fetch(p.scores + row);
  return s > -INFINITY && s < INFINITY;
}

// One warp a unit: maxima of its blocks, and the sum of e^(x - m) with the
// largest of them as m.
template <class T>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamParams p) {
  constexpr int kLane = Vec<T>::kLane;
  const int lane = threadIdx.x & 31;
  const int64_t all = (int64_t)p.batch * p.beams * p.plan.units;
  const int64_t warps = (int64_t)gridDim.x * (kScanThreads / 32);
  await_prior_kernel();
  admit_next_kernel();
  for (int64_t u = (int64_t)blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5); u < all; u += warps) {
    const int64_t row = u / p.plan.units;
    const int j0 = (int)(u - row * p.plan.units) * p.plan.unit_blocks;
    const int j1 = min(j0 + p.plan.unit_blocks, p.plan.blocks);
    if (!live_beam(p, row)) continue;
    const Row<T> r = logits_row<T>(p, row);
    const int64_t end = (int64_t)r.before + p.vocab;
    auto load = [&](int j, uint4 (&v)[kScanBatch]) {
      const int64_t at = (int64_t)j * Vec<T>::kBlock + lane * kLane;
      if (j > 0 && j + kScanBatch <= j1 && (int64_t)(j + kScanBatch) * Vec<T>::kBlock <= end) {
#pragma unroll
        for (int k = 0; k < kScanBatch; ++k) v[k] = __ldcs(reinterpret_cast<const uint4*>(r.base + at + k * Vec<T>::kBlock));
      } else {
#pragma unroll 1
        for (int k = 0; k < kScanBatch; ++k) {
          const uint4 x = load_lane(r, at + k * Vec<T>::kBlock, j + k < j1 ? end : 0);
#pragma unroll
          for (int i = 0; i < kScanBatch; ++i)
            if (i == k) v[i] = x;
        }
      }
    };
    float m = -INFINITY, sum = 0.f, keep = -INFINITY;
    uint4 next[kScanBatch];                       // a batch ahead, so that loads are always in flight
    load(j0, next);
    for (int j = j0; j < j1; j += kScanBatch) {
      uint4 v[kScanBatch];
#pragma unroll
      for (int k = 0; k < kScanBatch; ++k) v[k] = next[k];
      if (j + kScanBatch < j1) load(j + kScanBatch, next);
      float top = m;
#pragma unroll
      for (int k = 0; k < kScanBatch; ++k) {
        float x[kLane];
        unpack(v[k], x, r.base);
        float t = x[0];
#pragma unroll
        for (int e = 1; e < kLane; ++e) t = fmaxf(t, x[e]);
        t = ptx::warp_max(t);
        if (lane == j + k - j0) keep = t;
        top = fmaxf(top, t);
      }
      const float ref = top == -INFINITY ? 0.f : top;
      if (top > m) {                              // (the same in all lanes)
        sum *= fast_exp2((m - ref) * kLog2e);
        m = top;
      }
#pragma unroll
      for (int k = 0; k < kScanBatch; ++k) {
        float x[kLane];
        unpack(v[k], x, r.base);
#pragma unroll
        for (int e = 0; e < kLane; ++e) x[e] = fast_exp2((x[e] - ref) * kLog2e);
#pragma unroll
        for (int d = 1; d < kLane; d *= 2)
#pragma unroll
          for (int e = 0; e < kLane; e += 2 * d) x[e] += x[e + d];
        sum += x[0];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (j0 + lane < j1) p.block_max[row * p.plan.blocks + j0 + lane] = keep;
    if (lane == 0) p.partial[u] = make_float2(m, sum);
  }
}

// ---------------------------------------------------------------- choice

// (score, index) in the order of the choice: larger keys are better, among equal
// ones lower indices.  Key 0 is none.
struct Rank {
  uint64_t key;
  uint32_t index;
};
__device__ __forceinline__ bool better(Rank a, Rank b) {
  return a.key > b.key || (a.key == b.key && a.index < b.index);
}

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);    // (-0 as 0)
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t b) {
  return __uint_as_float(b ^ ((uint32_t)((int32_t)~b >> 31) | 0x80000000u));
}

// A beam: x scores (x - top) + offset, top its largest logit and offset = s - log
// of the sum of e^(x - top), as two numbers (not s - lse: logits may all lie at their
// type's lowest value, beside which the sum is nothing).  hi = NaN: no continuations.
struct Beam {
  float hi, lo, top;
};
// The score's key: the sum of four numbers as two, the first one rounded.
__device__ __forceinline__ uint64_t score_key(const Beam& c, float x) {
  if (!(x > -INFINITY) || isnan(c.hi)) return 0;
  const float d = __fsub_rn(x, c.top), dx = __fadd_rn(d, c.top);
  const float s = __fadd_rn(c.hi, d), b = __fsub_rn(s, c.hi);
  if (!(fabsf(s) < INFINITY)) return 0;
  const float e = __fadd_rn(__fsub_rn(x, dx), __fsub_rn(__fsub_rn(dx, d), c.top));   // (x - top) - d
  const float f = __fadd_rn(__fsub_rn(c.hi, __fsub_rn(s, b)), __fsub_rn(d, b));      // (hi + d) - s
  const float t = __fadd_rn(__fadd_rn(f, e), c.lo);
  const float hi = __fadd_rn(s, t), lo = __fsub_rn(t, __fsub_rn(hi, s));
  return (uint64_t)ordered(hi) << 32 | ordered(lo);
}

constexpr int kPickThreads = 1024;
constexpr int kGroups = 128;                      // whose best ones bound the K-th best of all
constexpr int kTile = 8192;                       // keys ranked at a time
constexpr int kReach = SMLA_MAX_BEAM_OUT * (kTile / kGroups);   // of them that may reach the bound
constexpr int kGathered = kMaxUnitBlocks * SMLA_MAX_BEAM_OUT;   // keys gathered by a bound that is known
constexpr int kDirect = 256;                      // keys ranked without a bound of their own
static_assert(kGathered + SMLA_MAX_BEAM_OUT * (kGathered / kGroups) <= kReach, "both lists of settle()");

struct Pick {
  uint64_t key[kReach + SMLA_MAX_BEAM_OUT];
  uint32_t index[kReach + SMLA_MAX_BEAM_OUT];
  Rank group[kPickThreads];
  Rank best[SMLA_MAX_BEAM_OUT];
  Rank bound;
  uint32_t chosen[SMLA_MAX_BEAM_OUT];
  Beam beam[SMLA_MAX_BEAMS];
  bool single[SMLA_MAX_BEAMS];                    // finished: one continuation
  int count, found;
};

// The keys among n (any order) that reach a lower bound of their K-th best one, to
// the list from `to` on; sh.count of them.  Each of 128 groups of keys has a best
// one; the K-th best of those is the bound, and at most K groups have keys that
// reach it: K * n / 128, and for keys in no particular order hardly more than K.
// Whole CTA.
template <class F>
__device__ __forceinline__ void reach(Pick& sh, int keep, int n, int to, F key) {
  const Rank none = {0, 0xffffffffu};
  Rank mine = none;
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const Rank r = key(i);
    if (r.key != 0 && better(r, mine)) mine = r;
  }
  sh.group[threadIdx.x] = mine;
  if (threadIdx.x == 0) {
    sh.count = 0;
    sh.bound = none;
  }
  __syncthreads();
  // eight threads a group: its best one, and a share of the comparisons with the others
  constexpr int kEach = kPickThreads / kGroups;
  const int group = threadIdx.x / kEach, lane = threadIdx.x % kEach;
  mine = sh.group[lane * kGroups + group];
#pragma unroll
  for (int o = 1; o < kEach; o *= 2) {
    const Rank r = {__shfl_xor_sync(0xffffffffu, mine.key, o), __shfl_xor_sync(0xffffffffu, mine.index, o)};
    if (better(r, mine)) mine = r;
  }
  __syncthreads();
  if (lane == 0) sh.group[group] = mine;
  __syncthreads();
  int rank = 0;
#pragma unroll
  for (int k = lane; k < kGroups; k += kEach) rank += better(sh.group[k], mine);
#pragma unroll
  for (int o = 1; o < kEach; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (lane == 0 && rank == keep - 1 && mine.key != 0) sh.bound = mine;
  __syncthreads();
  const Rank bound = sh.bound;
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const Rank r = key(i);
    if (r.key != 0 && !better(bound, r)) {
      const int at = to + atomicAdd(&sh.count, 1);
      sh.key[at] = r.key;
      sh.index[at] = r.index;
    }
  }
  __syncthreads();
}

// The K best of the list's entries [from, from + count), in order, to sh.best: each
// entry's rank is the number of better ones, counted by eight threads.
__device__ __forceinline__ void rank_list(Pick& sh, int keep, int from, int count) {
  constexpr int kEach = 8;
  const int lane = threadIdx.x % kEach;
  for (int base = 0; base < count; base += kPickThreads / kEach) {
    const int i = base + (int)threadIdx.x / kEach;
    const Rank mine = {sh.key[from + min(i, count - 1)], sh.index[from + min(i, count - 1)]};
    int rank = 0;
    for (int k = lane; k < count; k += kEach) rank += better({sh.key[from + k], sh.index[from + k]}, mine);
#pragma unroll
    for (int o = 1; o < kEach; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (lane == 0 && i < count && rank < keep) sh.best[rank] = mine;
  }
  if (threadIdx.x == 0) sh.found = min(keep, count);
  __syncthreads();
}

// The K best of n keys, a tile at a time beside the best ones so far.
template <class F>
__device__ __forceinline__ void pick(Pick& sh, int keep, int64_t n, F key) {
  int found = 0;
  for (int64_t base = 0; base < n; base += kTile) {
    reach(sh, keep, (int)min((int64_t)kTile, n - base), 0, [&](int i) { return key(base + i); });
    const int count = sh.count;
    if (threadIdx.x < found) {
      sh.key[count + threadIdx.x] = sh.best[threadIdx.x].key;
      sh.index[count + threadIdx.x] = sh.best[threadIdx.x].index;
    }
    __syncthreads();
    rank_list(sh, keep, 0, count + found);
    found = sh.found;
  }
  if (threadIdx.x == 0) sh.found = found;
  __syncthreads();
}

// The K best of n keys of which at least K are `least` or more, if it is not 0: those
// are gathered, and what is left to rank is little more than K, but for ties.
template <class F>
__device__ __forceinline__ void pick_from(Pick& sh, int keep, int n, uint64_t least, F key) {
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const Rank r = key(i);
    if (r.key != 0 && r.key >= least) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kGathered) {
        sh.key[at] = r.key;
        sh.index[at] = r.index;
      }
    }
  }
  __syncthreads();
  const int count = sh.count;
  __syncthreads();
  if (count <= kDirect) {
    rank_list(sh, keep, 0, count);
  } else if (count <= kGathered) {
    reach(sh, keep, count, kGathered, [&](int i) -> Rank { return {sh.key[i], sh.index[i]}; });
    rank_list(sh, keep, kGathered, sh.count);
  } else {
    pick(sh, keep, n, [&](int64_t i) { return key((int)i); });
  }
}

// sh.best's indices in rising order to sh.chosen; so that positions in what they
// stand for compare like (beam, token).
__device__ __forceinline__ void sort_chosen(Pick& sh) {
  const int found = sh.found;
  if (threadIdx.x < found) {
    const uint32_t mine = sh.best[threadIdx.x].index;
    int at = 0;
    for (int k = 0; k < found; ++k) at += sh.best[k].index < mine;
    sh.chosen[at] = mine;
  }
  __syncthreads();
}

template <class T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Pick& sh = *reinterpret_cast<Pick*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * p.beams;
  await_prior_kernel();
  admit_next_kernel();

  // the beams, a warp each
  for (int i = warp; i < p.beams; i += kPickThreads / 32) {
    const float s = fetch(p.scores + row0 + i);
    const bool done = p.finished != nullptr && p.finished[row0 + i] != 0;
    bool bad = isnan(s) || s == INFINITY;
    double c = NAN;
    float m = 0.f;
    if (done) {
      if (!bad && s > -INFINITY) c = s;
    } else if (live_beam(p, row0 + i)) {
      const float2* part = p.partial + (row0 + i) * p.plan.units;
      m = -INFINITY;
      for (int k = lane; k < p.plan.units; k += 32) m = fmaxf(m, fetch(part + k).x);
      m = ptx::warp_max(m);
      double sum = 0;
      for (int k = lane; k < p.plan.units; k += 32) {
        const float2 v = fetch(part + k);
        if (!(v.x == -INFINITY && v.y == 0.f)) sum += (double)(v.y * fast_exp2((v.x - m) * kLog2e));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      bad = isnan(sum);
      if (!bad && m > -INFINITY) c = (double)s - log(sum);
    }
    if (lane == 0) {
      const float hi = (float)c;
      sh.beam[i] = {hi, (float)(c - (double)hi), m};
      sh.single[i] = done;
      if (bad && p.err != nullptr) atomicOr(p.err, SMLA_DEVERR_BAD_LOGITS);
    }
  }
  __syncthreads();

  // the best units, the best blocks of those, the best elements of those
  const int keep = p.num_out, per = p.plan.unit_blocks, units = p.plan.units;
  const float2* part = p.partial + row0 * units;
  pick(sh, keep, (int64_t)p.beams * units, [&](int64_t at) -> Rank {
    const uint32_t i = (uint32_t)at / (uint32_t)units;
    const Beam c = sh.beam[i];
    if (isnan(c.hi)) return {0, 0};
    if (sh.single[i]) return {at == (int64_t)i * units ? score_key(c, 0.f) : 0, (uint32_t)at};
    return {score_key(c, fetch(&part[at].x)), (uint32_t)at};
  });
  uint64_t least = sh.found == keep ? sh.best[keep - 1].key : 0;
  sort_chosen(sh);
  const float* top = p.block_max + row0 * p.plan.blocks;
  pick_from(sh, keep, sh.found * per, least, [&](int at) -> Rank {
    const uint32_t unit = sh.chosen[at / per], i = unit / (uint32_t)units;
    const int j = (int)(unit - i * units) * per + at % per;
    Rank r = {0, i * (uint32_t)p.plan.blocks + j};
    if (sh.single[i]) r.key = j == 0 ? score_key(sh.beam[i], 0.f) : 0;
    else if (j < p.plan.blocks) r.key = score_key(sh.beam[i], fetch(top + r.index));
    return r;
  });
  least = sh.found == keep ? sh.best[keep - 1].key : 0;
  sort_chosen(sh);
  constexpr int kBlock = Vec<T>::kBlock;
  pick_from(sh, keep, sh.found * kBlock, least, [&](int at) -> Rank {
    const uint32_t block = sh.chosen[at / kBlock], i = block / (uint32_t)p.plan.blocks;
    Rank r = {0, (uint32_t)at};
    if (sh.single[i]) {
      if (at % kBlock == 0) r.key = score_key(sh.beam[i], 0.f);
    } else {
      const Row<T> row = logits_row<T>(p, row0 + i);
      const int64_t j = (int64_t)(block - i * p.plan.blocks) * kBlock + at % kBlock;
      if (j >= row.before && j < (int64_t)row.before + p.vocab) r.key = score_key(sh.beam[i], element(row.base + j));
    }
    return r;
  });
  if (threadIdx.x < p.num_out) {
    float score = -INFINITY;
    int parent = -1, token = -1;
    if (threadIdx.x < sh.found) {
      const Rank r = sh.best[threadIdx.x];
      const uint32_t block = sh.chosen[r.index / kBlock];
      const int i = (int)(block / (uint32_t)p.plan.blocks);
      score = unordered((uint32_t)(r.key >> 32));
      parent = (int)(row0 + i);
      token = sh.single[i] ? p.end_token
                           : (int)((int64_t)(block % (uint32_t)p.plan.blocks) * kBlock + r.index % kBlock -
                                   logits_row<T>(p, row0 + i).before);
    }
    const int64_t at = (int64_t)blockIdx.x * p.num_out + threadIdx.x;
    p.out_scores[at] = score;
    p.out_parents[at] = parent;
    p.out_tokens[at] = token;
  }
}

template <class T>
cudaError_t launch(const BeamParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.batch * p.beams * p.plan.units, ctas = (units + kScanThreads / 32 - 1) / (kScanThreads / 32);
  cudaError_t e = launch_overlapped(beam_scan_kernel<T>, dim3((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20)), kScanThreads, 0,
                                    stream, p);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(beam_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Pick));
  if (e != cudaSuccess) return e;
  return launch_overlapped(beam_pick_kernel<T>, dim3((unsigned)p.batch), kPickThreads, sizeof(Pick), stream, p);
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t stream) {
  if (p.dtype == SMLA_LOGITS_BF16) return launch<__nv_bfloat16>(p, stream);
  if (p.dtype == SMLA_LOGITS_FP16) return launch<__half>(p, stream);
  return launch<float>(p, stream);
}

}  // namespace smla
