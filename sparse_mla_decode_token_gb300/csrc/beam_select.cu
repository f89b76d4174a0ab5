// Beam selection: the best continuations over a request's beams and vocabulary.
//
//   score(i, v) = s_i + x[i][v] - lse_i,  lse_i = log sum_w e^{x[i][w]}
//
// One pass over the logits, in which nothing is sorted: a warp reads blocks of
// 512 consecutive bytes of a row, adds up e^(x - m) and keeps each block's
// maximum (a word for 512 bytes).  Blocks rank like their maxima, so the K best
// elements lie in the K best blocks: K blocks with larger maxima (or equal ones
// and lower indices) hold K better elements than any element of another block.
// A second kernel ranks a request's blocks and looks at the elements of the best
// K of them only.
//
// Ranks are over (score, index) with the score as an unevaluated sum of two fp32
// numbers (48 bits): what does not depend on v is computed in 64 bits, and x added
// to it without an error.  Sums are fp32 over at most 256 terms a lane, then 64 bits over the
// units; e^x is off by 2^-22 of itself.
//
// What bounds it: the first kernel reads each logit once.
#include <cuda_fp16.h>

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

// The lane's elements of a block (-infinity where there are none).
template <class T>
__device__ __forceinline__ void load_lane(const Row<T>& r, int64_t at, int64_t end, float (&x)[Vec<T>::kLane]) {
  if (at >= r.before && at + Vec<T>::kLane <= end) {
    unpack(*reinterpret_cast<const uint4*>(r.base + at), x, r.base);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::kLane; ++e)
      x[e] = at + e >= r.before && at + e < end ? element(r.base + at + e) : -INFINITY;
  }
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
    float m = -INFINITY, sum = 0.f, keep = -INFINITY;
    for (int j = j0; j < j1; j += kScanBatch) {
      float x[kScanBatch][kLane];
      const int64_t at = (int64_t)j * Vec<T>::kBlock + lane * kLane;
      if (j > 0 && j + kScanBatch <= j1 && (int64_t)(j + kScanBatch) * Vec<T>::kBlock <= end) {
        uint4 v[kScanBatch];
#pragma unroll
        for (int k = 0; k < kScanBatch; ++k) v[k] = __ldcs(reinterpret_cast<const uint4*>(r.base + at + k * Vec<T>::kBlock));
#pragma unroll
        for (int k = 0; k < kScanBatch; ++k) unpack(v[k], x[k], r.base);
      } else {
#pragma unroll
        for (int k = 0; k < kScanBatch; ++k) load_lane(r, at + k * Vec<T>::kBlock, j + k < j1 ? end : 0, x[k]);
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kScanBatch; ++k) {
        float t = x[k][0];
#pragma unroll
        for (int e = 1; e < kLane; ++e) t = fmaxf(t, x[k][e]);
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
        float t[kLane];
#pragma unroll
        for (int e = 0; e < kLane; ++e) t[e] = fast_exp2((x[k][e] - ref) * kLog2e);
#pragma unroll
        for (int d = 1; d < kLane; d *= 2)
#pragma unroll
          for (int e = 0; e < kLane; e += 2 * d) t[e] += t[e + d];
        sum += t[0];
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
__device__ __forceinline__ bool better(const Rank& a, const Rank& b) {
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
constexpr int kGroups = 256;                      // whose best ones bound the K-th best of all
constexpr int kTile = 32768;                      // keys ranked at a time
constexpr int kList = SMLA_MAX_BEAM_OUT * (kTile / kGroups);   // that may reach the bound

struct Pick {
  Rank list[kList + SMLA_MAX_BEAM_OUT];
  Rank group[kPickThreads];
  Rank best[SMLA_MAX_BEAM_OUT], chosen[SMLA_MAX_BEAM_OUT];
  Rank bound;
  Beam beam[SMLA_MAX_BEAMS];
  bool single[SMLA_MAX_BEAMS];                    // finished: one continuation
  int count, found;
};

// The K best of n keys (any order) to sh.best, in order; sh.found of them.  Each
// of 256 groups of keys has a best one; the K-th best of those bounds the K-th
// best of all from below, and what reaches it is at most K groups' keys: K * n /
// 256, and for keys in no particular order hardly more than K.  Whole CTA.
template <class F>
__device__ __forceinline__ void pick_tile(Pick& sh, int keep, int n, Rank* list, F key) {
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
  if (threadIdx.x < kGroups) {
#pragma unroll
    for (int k = 1; k < kPickThreads / kGroups; ++k) {
      const Rank r = sh.group[threadIdx.x + k * kGroups];
      if (better(r, mine)) mine = r;
    }
  }
  __syncthreads();
  if (threadIdx.x < kGroups) sh.group[threadIdx.x] = mine;
  __syncthreads();
  if (threadIdx.x < kGroups && mine.key != 0) {
    int rank = 0;
    for (int k = 0; k < kGroups; ++k) rank += better(sh.group[k], mine);
    if (rank == keep - 1) sh.bound = mine;
  }
  __syncthreads();
  const Rank bound = sh.bound;
  for (int i = threadIdx.x; i < n; i += kPickThreads) {
    const Rank r = key(i);
    if (r.key != 0 && !better(bound, r)) list[atomicAdd(&sh.count, 1)] = r;
  }
  __syncthreads();
}

// Ranks the `count` keys of the list by counting the better ones of each.
__device__ __forceinline__ void rank_list(Pick& sh, int keep, const Rank* list, int count) {
  for (int i = threadIdx.x; i < count; i += kPickThreads) {
    const Rank mine = list[i];
    int rank = 0;
    for (int k = 0; k < count && rank < keep; ++k) rank += better(list[k], mine);
    if (rank < keep) sh.best[rank] = mine;
  }
  __syncthreads();
}

template <class F>
__device__ __forceinline__ void pick(Pick& sh, int keep, int64_t n, F key) {
  int found = 0;
  for (int64_t base = 0; base < n || base == 0; base += kTile) {
    const int tile = (int)min((int64_t)kTile, n - base);
    pick_tile(sh, keep, tile, sh.list, [&](int i) { return key(base + i); });
    int count = sh.count;
    if (threadIdx.x < found) sh.list[count + threadIdx.x] = sh.best[threadIdx.x];
    __syncthreads();
    count += found;
    rank_list(sh, keep, sh.list, count);
    found = min(keep, count);
  }
  if (threadIdx.x == 0) sh.found = found;
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

  // the best blocks
  const float* top = p.block_max + row0 * p.plan.blocks;
  pick(sh, p.num_out, (int64_t)p.beams * p.plan.blocks, [&](int64_t at) -> Rank {
    const int i = (int)(at / p.plan.blocks);
    const Beam c = sh.beam[i];
    if (isnan(c.hi)) return {0, 0xffffffffu};
    if (sh.single[i]) return {at % p.plan.blocks == 0 ? score_key(c, 0.f) : 0, (uint32_t)at};
    return {score_key(c, fetch(top + at)), (uint32_t)at};
  });
  const int blocks = sh.found;
  const Rank worst = blocks == p.num_out ? sh.best[blocks - 1] : Rank{0, 0xffffffffu};
  // in order of their indices, so that their elements' indices compare like (beam, token)
  if (threadIdx.x < blocks) {
    const Rank mine = sh.best[threadIdx.x];
    int at = 0;
    for (int k = 0; k < blocks; ++k) at += sh.best[k].index < mine.index;
    sh.chosen[at] = mine;
  }
  __syncthreads();

  // the best elements of those blocks
  constexpr int kBlock = Vec<T>::kBlock;
  pick(sh, p.num_out, (int64_t)blocks * kBlock, [&](int64_t at) -> Rank {
    const int k = (int)at / kBlock, e = (int)at % kBlock;
    const uint32_t block = sh.chosen[k].index;
    const int i = (int)(block / (uint32_t)p.plan.blocks);
    const Beam c = sh.beam[i];
    Rank r = {0, (uint32_t)at};
    if (sh.single[i]) {
      if (e == 0) r.key = score_key(c, 0.f);
    } else {
      const Row<T> row = logits_row<T>(p, row0 + i);
      const int64_t j = (int64_t)(block % (uint32_t)p.plan.blocks) * kBlock + e;
      if (j >= row.before && j < (int64_t)row.before + p.vocab) r.key = score_key(c, element(row.base + j));
    }
    return r.key >= worst.key ? r : Rank{0, (uint32_t)at};
  });
  if (threadIdx.x < p.num_out) {
    float score = -INFINITY;
    int parent = -1, token = -1;
    if (threadIdx.x < sh.found) {
      const Rank r = sh.best[threadIdx.x];
      const uint32_t block = sh.chosen[r.index / kBlock].index;
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
