// Beam selection: the best continuations over a request's beams and vocabulary.
//
//   score(i, v) = s_i + x[i][v] - lse_i,  lse_i = log sum_w e^{x[i][w]}
//
// One pass over the logits, in which nothing is sorted: a warp reads blocks of
// 512 consecutive bytes of a row, adds up e^(x - m) and keeps each block's
// maximum (a word for 512 bytes).  Blocks rank like their maxima, so the K best
// elements lie in the K best blocks: K blocks with larger maxima (or equal ones
// and lower indices) hold K better elements than any element of another block.
// The same holds for the units of up to 16 blocks that a warp takes.  A second
// kernel ranks a request's units, the blocks of the best K, then the elements of
// the best K of those: some thousand keys in place of a million logits.
//
// Ranks are over (score, index) with the score as an unevaluated sum of two fp32
// numbers (48 bits), to which x adds without an error: one beam's continuations rank
// like its logits.  Between beams ranks carry the error of their log sums, under 2^-17:
// five values of e^x, each off by 2^-22 of itself, and four products on a term's way to
// the sum, 24 additions (fp32 over at most 64 terms a lane, a warp's lanes, then such
// pairs over the units) and one logarithm are 49 times 2^-24; arguments of e^x, rounded
// three times, add 2.25 times 2^-24 of their mean size, at most log V by the weights
// that they have.  (In fp64, which has a fiftieth of fp32's rate, the second kernel takes
// 15 us for the 32 beams of a request alone.)
//
// What bounds it: the first kernel reads each logit once with two thirds of the issue
// slots taken (116 MB in 21.5 us, 5.4 TB/s, replayed behind itself, so that some of them
// are still in L2; a kernel that only reads them takes 20; 25.1 us with flushed caches
// under the profiler), the second is a dozen dependent phases of one CTA a request.
// Measured on a GB300, replayed from a graph: 64 requests of 8 beams over 128000 BF16
// logits, 16 kept: 32.7 us (the choice 11); 8 of 32 beams over 151001 FP32 logits, 64
// kept: 45.4 (19); one of 4 beams over 32000: 12.1 (9).  As calls on other logits each
// time: 34.5, 46.5 and 12.7.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "cache_ptx.cuh"
#include "step.cuh"

namespace smla {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanBatch = 4;                     // blocks that a warp takes at a time
static_assert((1 << kMinUnitShift) % kScanBatch == 0, "units are whole batches");

// Batches in a warp's ring: copies run one or two ahead.  (16-bit logits, which take more
// instructions a byte: 33.3 us with two, 34.1 with three; fp32: 53.6 and 51.5.)
template <class T>
constexpr int kScanStages = sizeof(T) == 4 ? 3 : 2;
// CTAs of an SM (16-bit logits: 32.6 us with five, 33.0 with four; fp32, whose ring is
// longer: 49.7 and 47.0).
template <class T>
constexpr int kScanCtas = sizeof(T) == 4 ? 4 : 5;
template <class T>
constexpr int kScanSmem = kScanThreads / 32 * kScanStages<T> * kScanBatch * kBeamBlockBytes;

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

// The largest of a lane's elements (16-bit ones in pairs); NaN are passed over.
__device__ __forceinline__ float largest(uint4 v, const float*) {
  return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
template <class T>
__device__ __forceinline__ float largest(uint4 v, const T*) {
  using Two = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  const auto two = [](const uint32_t& w) { return *reinterpret_cast<const Two*>(&w); };
  const Two t = __hmax2(__hmax2(two(v.x), two(v.y)), __hmax2(two(v.z), two(v.w)));
  return fmaxf(element(&t.x), element(&t.y));
}

// Four elements, at a multiple of four from a 16-byte boundary.
__device__ __forceinline__ void load_four(const float* at, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(at);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
template <class T>
__device__ __forceinline__ void load_four(const T* at, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(at);
  float y[8];
  unpack(make_uint4(v.x, v.y, 0, 0), y, at);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = y[e];
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

// The lane's 16 bytes from element `at` of the row's base on; -infinity in place of
// elements before its first and from `end` on.
template <class T>
__device__ __noinline__ uint4 load_edge(const T* base, int before, uint32_t at, uint32_t end) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      w[k] = at + k >= before && at + k < end ? reinterpret_cast<const uint32_t*>(base)[at + k] : 0xff800000u;
    } else {
      constexpr uint32_t none = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
      uint32_t v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t i = at + 2 * k + e;
        v[e] = i >= before && i < end ? reinterpret_cast<const uint16_t*>(base)[i] : none;
      }
      w[k] = v[0] | v[1] << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Is the beam of this row one whose logits count?
__device__ __forceinline__ bool live_beam(const BeamParams& p, int64_t row) {
  const float s = fetch(p.scores + row);
  const bool done = p.finished != nullptr && fetch(p.finished + row) != 0;
  return (s > -INFINITY) & (s < INFINITY) & !done;
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// Where a warp stands: a batch of blocks of one of its units.
template <class T>
struct Cursor {
  uint32_t unit, row;                             // unit >= all: no more
  int j0, j1, j;                                  // the unit's blocks, the batch's first

  // The unit, or the next one `step` away whose logits count.
  __device__ __forceinline__ void settle(const BeamParams& p, uint32_t all, uint32_t step) {
    for (; unit < all; unit += step) {
      row = unit / (uint32_t)p.plan.units;
      if (live_beam(p, row)) break;
    }
    j = j0 = (int)(unit - row * p.plan.units) << p.plan.unit_shift;
    j1 = min(j0 + (1 << p.plan.unit_shift), p.plan.blocks);
  }
  __device__ __forceinline__ bool next(const BeamParams& p, uint32_t all, uint32_t step) {
    j += kScanBatch;
    if (j < j1) return false;
    unit += step;
    settle(p, all, step);
    return true;
  }
};

// Maxima of a unit's blocks, and the sum of e^(x - m) with the largest of them as m.
// Each lane copies 16 bytes of every block into a ring of its warp's and reads them
// there itself, so nothing but its own copies is waited for; the copies run
// ahead through the ends of units.
template <class T>
__global__ void __launch_bounds__(kScanThreads, kScanCtas<T>) beam_scan_kernel(const BeamParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kLane = Vec<T>::kLane, kStage = kScanBatch * kBeamBlockBytes, kStages = kScanStages<T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* const mine = ring + warp * (kStages * kStage) + lane * 16;
  const uint32_t all = (uint32_t)(p.batch * p.beams) * p.plan.units;
  // (units that follow one another go to different CTAs)
  const uint32_t step = gridDim.x * (kScanThreads / 32);
  await_prior_kernel();
  admit_next_kernel();
  Cursor<T> ahead, at;
  ahead.unit = warp * gridDim.x + blockIdx.x;
  ahead.settle(p, all, step);
  at = ahead;
  Row<T> r = {};
  if (ahead.unit < all) r = logits_row<T>(p, ahead.row);
  auto load = [&](int stage) {
    if (ahead.unit < all) {
      const uint32_t end = (uint32_t)r.before + (uint32_t)p.vocab;
      uint8_t* const to = mine + stage * kStage;
      const uint32_t first = (uint32_t)ahead.j * Vec<T>::kBlock;
      if (first >= r.before && first + kScanBatch * Vec<T>::kBlock <= end) {   // (units are whole batches, but for a row's end)
        const T* const from = r.base + first + lane * kLane;
#pragma unroll
        for (int k = 0; k < kScanBatch; ++k) copy_async(ptx::smem_addr(to) + k * kBeamBlockBytes, from + k * Vec<T>::kBlock);
      } else {
#pragma unroll 1
        for (int k = 0; k < kScanBatch; ++k) {
          const uint32_t e = first + k * Vec<T>::kBlock + lane * kLane;
          if (e >= r.before && e + kLane <= end) copy_async(ptx::smem_addr(to) + k * kBeamBlockBytes, r.base + e);
          else *reinterpret_cast<uint4*>(to + k * kBeamBlockBytes) = load_edge(r.base, r.before, e, end);
        }
      }
      if (ahead.next(p, all, step) && ahead.unit < all) r = logits_row<T>(p, ahead.row);
    }
    copy_commit();
  };
#pragma unroll 1
  for (int k = 0; k < kStages - 1; ++k) load(k);
  float m = -INFINITY, keep = -INFINITY;
  uint64_t sum = 0;                               // two sums
  for (int stage = 0; at.unit < all;) {
    load(stage == 0 ? kStages - 1 : stage - 1);
    copy_wait<kStages - 1>();
    const uint8_t* const from = mine + stage * kStage;
    uint4 v[kScanBatch];
    float top = m;
#pragma unroll
    for (int k = 0; k < kScanBatch; ++k) {
      v[k] = *reinterpret_cast<const uint4*>(from + k * kBeamBlockBytes);
      const float t = ptx::warp_max(largest(v[k], r.base));
      if (lane == at.j + k - at.j0) keep = t;
      top = fmaxf(top, t);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    if (top > m) {                                // (the same in all lanes)
      const float by = fast_exp2((m - ref) * kLog2e);
      sum = ptx::f2_mul(sum, ptx::f2_pack(by, by));
      m = top;
    }
    const uint64_t ref2 = ptx::f2_pack(-ref, -ref), log2e2 = ptx::f2_pack(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < kScanBatch; ++k) {
      float x[kLane];
      unpack(v[k], x, r.base);
      uint64_t y[kLane / 2];
#pragma unroll
      for (int e = 0; e < kLane / 2; ++e) {
        float a, b;
        ptx::f2_unpack(ptx::f2_mul(ptx::f2_add(ptx::f2_pack(x[2 * e], x[2 * e + 1]), ref2), log2e2), a, b);
        y[e] = ptx::f2_pack(fast_exp2(a), fast_exp2(b));
      }
#pragma unroll
      for (int d = 1; d < kLane / 2; d *= 2)
#pragma unroll
        for (int e = 0; e < kLane / 2; e += 2 * d) y[e] = ptx::f2_add(y[e], y[e + d]);
      sum = ptx::f2_add(sum, y[0]);
    }
    if (at.j + kScanBatch >= at.j1) {             // the unit is done
      float total, other;
      ptx::f2_unpack(sum, total, other);
      total += other;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (at.j0 + lane < at.j1) p.block_max[(int64_t)at.row * p.plan.blocks + at.j0 + lane] = keep;
      if (lane == 0) p.partial[at.unit] = make_float2(m, total);
      m = keep = -INFINITY;
      sum = 0;
    }
    at.next(p, all, step);
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
}

// ---------------------------------------------------------------- choice

// Scores as whole numbers in the same order: the first of a score's two numbers, then
// the second; among equal ones lower indices are better.  hi = 0 is none.
struct Rank {
  uint32_t hi, lo, index;
};
__device__ __forceinline__ bool better(const Rank& a, const Rank& b) {
  return a.hi > b.hi || (a.hi == b.hi && (a.lo > b.lo || (a.lo == b.lo && a.index < b.index)));
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
// The score's rank: the sum of four numbers as two, the first one rounded.  (Each
// difference's rounding is found by Knuth's two-sum, as in add_exact.)
__device__ __noinline__ Rank score_rank(Beam c, float x, uint32_t index) {
  if (!(x > -INFINITY) || isnan(c.hi)) return {0, 0, index};
  const float d = __fsub_rn(x, c.top), dx = __fadd_rn(d, c.top);
  const float s = __fadd_rn(c.hi, d), b = __fsub_rn(s, c.hi);
  if (!(fabsf(s) < INFINITY)) return {0, 0, index};
  const float e = __fadd_rn(__fsub_rn(x, dx), __fsub_rn(__fsub_rn(dx, d), c.top));   // (x - top) - d
  const float f = __fadd_rn(__fsub_rn(c.hi, __fsub_rn(s, b)), __fsub_rn(d, b));      // (hi + d) - s
  const float t = __fadd_rn(__fadd_rn(f, e), c.lo);
  const float hi = __fadd_rn(s, t), lo = __fsub_rn(t, __fsub_rn(hi, s));
  return {ordered(hi), ordered(lo), index};
}

// hi + lo += x, the rounding of hi kept in lo (two-sum).
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
  lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
  hi = s;
}
// log 2: its first 16 bits, with which small whole numbers multiply exactly, and the rest.
constexpr float kLog2Hi = 45426.f / 65536.f, kLog2Lo = (float)(0.69314718055994531 - 45426.0 / 65536.0);

constexpr int kPickThreads = 1024;
constexpr int kGroups = kPickThreads / 8;         // of entries, whose best ones bound the K-th best of all
constexpr int kDirect = 64;                       // entries ranked without such a bound
constexpr int kMany = 512;                        // entries that are not ranked before equal ones are told apart
constexpr int kTile = 8192;                       // keys looked at at a time,
constexpr int kSureTile = 4096;                   // at a time that may all be enough (equal scores)
constexpr int kGathered = kSureTile + SMLA_MAX_BEAM_OUT;
static_assert(kGroups >= SMLA_MAX_BEAM_OUT, "a K-th best group");

struct List {
  uint32_t hi[kGathered], lo[kGathered], index[kGathered];

  __device__ __forceinline__ Rank get(int i) const { return {hi[i], lo[i], index[i]}; }
  __device__ __forceinline__ void set(int i, const Rank& r) { hi[i] = r.hi, lo[i] = r.lo, index[i] = r.index; }
  // Adds r where `add` holds (whole warp).
  __device__ __forceinline__ void append(int* count, bool add, const Rank& r) {
    const int lane = threadIdx.x & 31;
    const uint32_t all = __ballot_sync(0xffffffffu, add);
    if (all == 0) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(count, __popc(all));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(all & ((1u << lane) - 1u));
    if (add && at < kGathered) set(at, r);
  }
};

struct Pick {
  List list, reached;
  __align__(16) uint32_t group[kGroups];
  Rank exact[kPickThreads];
  Rank best[SMLA_MAX_BEAM_OUT], bound;
  int2 chosen[SMLA_MAX_BEAM_OUT];                 // beam, number within it
  Beam beam[SMLA_MAX_BEAMS];
  float cut[SMLA_MAX_BEAMS];                      // logits under it do not reach `least`
  bool single[SMLA_MAX_BEAMS];                    // finished: one continuation
  uint32_t least;                                 // hi of the K-th best of a step: a bound for the next one; 0: none
  int count, reaching, found;
};

// What a beam's logits have to be at least for a score of `least` or more: 2^-20 of
// what is added up below it, for fp32's roundings.
__device__ __forceinline__ float logit_cut(const Beam& c, uint32_t least) {
  const float score = unordered(least), cut = (score - c.hi) + c.top;
  return least == 0 ? -INFINITY : cut - 0x1p-20f * (fabsf(score) + fabsf(c.hi) + fabsf(c.top));
}

// The entries of sh.reached (n, more than kMany: equal scores) that reach the K-th best
// one of the groups' best ones by index, too, to sh.list: K * n / kPickThreads at most.
__device__ __noinline__ int narrow(Pick& sh, int keep, int n) {
  __syncthreads();                                // (n has been read)
  Rank mine = {0, 0, 0xffffffffu};
  for (int i = threadIdx.x; i < n; i += kPickThreads)
    if (better(sh.reached.get(i), mine)) mine = sh.reached.get(i);
  sh.exact[threadIdx.x] = mine;
  if (threadIdx.x == 0) sh.bound = {0, 0, 0xffffffffu}, sh.reaching = 0;
  __syncthreads();
  int rank = 0;
  for (int k = 0; k < kPickThreads && rank < keep; ++k) rank += better(sh.exact[k], mine);
  if (rank == keep - 1 && mine.hi != 0) sh.bound = mine;
  __syncthreads();
  const Rank bound = sh.bound;
  for (int base = 0; base < n; base += kPickThreads) {
    const int i = base + (int)threadIdx.x;
    const Rank r = sh.reached.get(min(i, n - 1));
    sh.list.append(&sh.reaching, i < n && !better(bound, r), r);
  }
  __syncthreads();
  return sh.reaching;
}

// What is left of sh.list's `count` entries: the K best, in order, in sh.best; or a few
// more, up to `room`, in no order.  sh.chosen
// are those in rising order of their indices (beam * per_beam + number), so that
// positions in what they stand for compare like (beam, token); sh.cut what the next
// step's logits have to be.  Each of 128 groups of entries has a best score; the K-th
// best of those is a lower bound of the K-th best of all, which for entries in no
// particular order hardly more than K reach; an entry's rank is then the number of
// better ones.  Whole CTA.  (Out of line, once for all steps: what this kernel costs is
// latency, of which instructions fetched for the first time are a part.)
__device__ __noinline__ void settle(Pick& sh, int keep, int count, int per_beam, int beams, int room, bool again) {
  uint32_t least = sh.least;
  List* list = &sh.list;
  if (count > kDirect) {
    const int group = threadIdx.x / 8, lane = threadIdx.x % 8;
    uint32_t top = 0;
    for (int i = lane * kGroups + group; i < count; i += kPickThreads) top = max(top, sh.list.hi[i]);
#pragma unroll
    for (int o = 1; o < 8; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.group[group] = top;
    if (threadIdx.x == 0) sh.reaching = 0;
    __syncthreads();
    int rank = 0;
#pragma unroll
    for (int k = 0; k < kGroups / 32; ++k) {
      const int at = 4 * (lane + 8 * k);
      const uint4 v = *reinterpret_cast<const uint4*>(sh.group + at);
      rank += (v.x > top) + (v.y > top) + (v.z > top) + (v.w > top);
      rank += (v.x == top && at < group) + (v.y == top && at + 1 < group) + (v.z == top && at + 2 < group) +
              (v.w == top && at + 3 < group);
    }
#pragma unroll
    for (int o = 1; o < 8; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (lane == 0 && rank == keep - 1) sh.bound.hi = top;
    __syncthreads();
    const uint32_t bound = max(sh.bound.hi, 1u);
    least = max(least, bound);
    for (int base = 0; base < count; base += kPickThreads) {
      const int i = base + (int)threadIdx.x;
      const Rank r = sh.list.get(min(i, count - 1));
      sh.reached.append(&sh.reaching, i < count && r.hi >= bound, r);
    }
    __syncthreads();
    count = sh.reaching;
    list = &sh.reached;
    if (count > kMany) {
      count = narrow(sh, keep, count);
      list = &sh.list;
    }
  }
  if (count > room) {
    const int lane = threadIdx.x % 8;
    for (int base = 0; base < count; base += kPickThreads / 8) {
      const int i = base + (int)threadIdx.x / 8;
      const Rank mine = list->get(min(i, count - 1));
      int rank = 0;
#pragma unroll 4
      for (int k = lane; k < count; k += 8) {
        const uint32_t hi = list->hi[k];
        if (hi > mine.hi) ++rank;
        else if (hi == mine.hi && k != i) rank += better(list->get(k), mine);
      }
#pragma unroll
      for (int o = 1; o < 8; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (lane == 0 && i < count && rank < keep) sh.best[rank] = mine;
    }
    __syncthreads();
    if (count >= keep) least = max(least, sh.best[keep - 1].hi);
    count = min(keep, count);
  } else {
    if (threadIdx.x < count) sh.best[threadIdx.x] = list->get(threadIdx.x);
    __syncthreads();
  }
  const int found = count;
  if (room > 0) {
    constexpr int kEach = kPickThreads / SMLA_MAX_BEAM_OUT;      // threads for each
    const int i = threadIdx.x / kEach, lane = threadIdx.x % kEach;
    const uint32_t mine = i < found ? sh.best[i].index : 0;
    int at = 0;
    for (int k = lane; k < found; k += kEach) at += sh.best[k].index < mine;
#pragma unroll
    for (int o = 1; o < kEach; o *= 2) at += __shfl_xor_sync(0xffffffffu, at, o);
    if (lane == 0 && i < found) {
      const uint32_t beam = mine / (uint32_t)per_beam;
      sh.chosen[at] = make_int2((int)beam, (int)(mine - beam * per_beam));
    }
  }
  if (room > 0 || again)
    for (int i = kPickThreads - 1 - (int)threadIdx.x; i < beams; i += kPickThreads) sh.cut[i] = logit_cut(sh.beam[i], least);
  if (threadIdx.x == 0) {
    sh.found = found;
    sh.least = least;
  }
  __syncthreads();
}

// The K best of n keys, of which at least K reach sh.least where that is not 0: a tile
// of keys at a time is gathered (those that are enough) and settled beside the best
// ones so far.  load(i, x) gives the numbers of keys i .. i + kEach - 1, always, so that
// all of a thread's are on their way at a time; enough(i, number) says whether key i may
// count, rank(i, number) is its rank.  Keys that reach the bound are little more than K,
// but for ties.  `room`: keys that the next step takes; 0: this is the last.
template <int kEach, class L, class E, class F>
__device__ __forceinline__ void pick(Pick& sh, int keep, int64_t n, int per_beam, int beams, int room, L load, E enough, F rank) {
  constexpr int kRounds = kTile / kPickThreads / kEach;
  int found = 0, most = kTile;
  for (int64_t tile = 0; tile < n || tile == 0;) {
    const int here = (int)min(n - tile, (int64_t)most);
    const uint32_t least = sh.least;
    if (threadIdx.x == 0) sh.count = found;
    if (threadIdx.x < found) sh.list.set(threadIdx.x, sh.best[threadIdx.x]);
    float x[kRounds][kEach];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int i = (k * kPickThreads + (int)threadIdx.x) * kEach;
      if (k * kPickThreads * kEach < here) load(tile + min(i, here - kEach), x[k]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int i = (k * kPickThreads + (int)threadIdx.x) * kEach;
      if (k * kPickThreads * kEach >= here) break;
      uint32_t maybe = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) maybe |= (uint32_t)(i < here && enough(tile + i + e, x[k][e])) << e;
      if (kEach > 1 && !__any_sync(0xffffffffu, maybe != 0)) continue;
#pragma unroll 1
      do {                                        // each lane's next one (where there are many, few get here)
        const int e = __ffs(maybe) - 1;
        float y = x[k][0];
#pragma unroll
        for (int c = 1; c < kEach; ++c) y = e == c ? x[k][c] : y;
        Rank r = {0, 0, 0};
        if (maybe != 0) r = rank(tile + i + e, y);
        sh.list.append(&sh.count, r.hi != 0 && r.hi >= least, r);
        maybe &= maybe - 1;
      } while (kEach > 1 && __any_sync(0xffffffffu, maybe != 0));
    }
    __syncthreads();
    const int count = sh.count;
    if (count > kGathered) {                      // once more, in tiles that are sure to fit
      most = kSureTile;
      __syncthreads();
      continue;
    }
    const bool more = tile + here < n;
    settle(sh, keep, count, per_beam, beams, more ? 0 : room, more);
    found = sh.found;
    tile += here > 0 ? here : 1;
  }
}

template <class T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Pick& sh = *reinterpret_cast<Pick*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * p.beams;
  await_prior_kernel();
  admit_next_kernel();

  if (threadIdx.x == 0) sh.least = 0;
  // the beams, a warp each
  for (int i = warp; i < p.beams; i += kPickThreads / 32) {
    const float s = fetch(p.scores + row0 + i);
    const bool done = p.finished != nullptr && p.finished[row0 + i] != 0;
    bool bad = isnan(s) || s == INFINITY;
    Beam c = {NAN, 0.f, 0.f};
    if (done) {
      if (!bad && s > -INFINITY) c.hi = s;
    } else if (live_beam(p, row0 + i)) {
      const float2* part = p.partial + (row0 + i) * p.plan.units;
      float m = -INFINITY;
      for (int k = lane; k < p.plan.units; k += 32) m = fmaxf(m, fetch(part + k).x);
      m = ptx::warp_max(m);
      float hi = 0.f, lo = 0.f;                   // the sum, as two numbers
      for (int k = lane; k < p.plan.units; k += 32) {
        const float2 v = fetch(part + k);
        if (!(v.x == -INFINITY && v.y == 0.f)) add_exact(hi, lo, v.y * fast_exp2((v.x - m) * kLog2e));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
        add_exact(hi, lo, h);
        lo += l;
      }
      bad = isnan(hi);
      if (!bad && m > -INFINITY) {
        // log of the sum: e log 2 + log f for 2^e f with f in [0.75, 1.5), so that the second term is small
        const int e = (__float_as_int(hi) - 0x3f400000) >> 23;
        const float down = __int_as_float((127 - e) << 23), f = hi * down;
        c.hi = s;
        add_exact(c.hi, c.lo, -(float)e * kLog2Hi);
        add_exact(c.hi, c.lo, -(logf(f) + (lo * down) / f));
        c.lo -= (float)e * kLog2Lo;
        c.top = m;
      }
    }
    if (lane == 0) {
      sh.beam[i] = c;
      sh.single[i] = done;
      if (bad && p.err != nullptr) atomicOr(p.err, SMLA_DEVERR_BAD_LOGITS);
    }
  }
  __syncthreads();

  // the best units, the best blocks of those, the best elements of those
  constexpr int kBlock = Vec<T>::kBlock;
  const int keep = p.num_out, shift = p.plan.unit_shift, units = p.plan.units, blocks = p.plan.blocks;
  const float2* part = p.partial + row0 * units;
  pick<1>(
      sh, keep, (int64_t)p.beams * units, units, p.beams, SMLA_MAX_BEAM_OUT,
      [&](int64_t at, float (&x)[1]) { x[0] = fetch(&part[at].x); },
      [&](int64_t, float) { return true; },
      [&](int64_t at, float x) -> Rank {
        const uint32_t i = (uint32_t)at / (uint32_t)units;
        if (sh.single[i] && at != (int64_t)i * units) return {0, 0, 0};
        return score_rank(sh.beam[i], sh.single[i] ? 0.f : x, (uint32_t)at);
      });
  const float* top = p.block_max + row0 * blocks;
  pick<1>(
      sh, keep, sh.found << shift, blocks, p.beams, kSureTile / kBlock,
      [&](int64_t at, float (&x)[1]) {
        const int2 unit = sh.chosen[(int)at >> shift];
        x[0] = fetch(top + unit.x * blocks + min((unit.y << shift) + ((int)at & ((1 << shift) - 1)), blocks - 1));
      },
      [&](int64_t at, float x) {
        const int2 unit = sh.chosen[(int)at >> shift];
        const int j = (unit.y << shift) + ((int)at & ((1 << shift) - 1));
        return sh.single[unit.x] ? j == 0 : j < blocks && !(x < sh.cut[unit.x]);
      },
      [&](int64_t at, float x) -> Rank {
        const int2 unit = sh.chosen[(int)at >> shift];
        return score_rank(sh.beam[unit.x], sh.single[unit.x] ? 0.f : x,
                          (uint32_t)(unit.x * blocks + (unit.y << shift) + ((int)at & ((1 << shift) - 1))));
      });
  // (the blocks' elements: where they lie, which of them are the row's)
  __shared__ const T* s_base[SMLA_MAX_BEAM_OUT];
  __shared__ float s_cut[SMLA_MAX_BEAM_OUT];
  __shared__ int s_beam[SMLA_MAX_BEAM_OUT], s_from[SMLA_MAX_BEAM_OUT], s_to[SMLA_MAX_BEAM_OUT], s_token[SMLA_MAX_BEAM_OUT];
  if (threadIdx.x < sh.found) {
    const int k = threadIdx.x;
    const int2 block = sh.chosen[k];
    const Row<T> row = logits_row<T>(p, row0 + block.x);
    const int64_t j = (int64_t)block.y * kBlock;
    s_base[k] = row.base + j;
    s_beam[k] = block.x;
    s_from[k] = (int)max(row.before - j, (int64_t)0);
    s_to[k] = (int)min(row.before + (int64_t)p.vocab - j, (int64_t)kBlock);
    s_token[k] = (int)(j - row.before);
    s_cut[k] = sh.cut[block.x];
    if (sh.single[block.x]) {                     // (one of a finished beam's stands for it)
      s_to[k] = s_from[k] + 1;
      s_cut[k] = -INFINITY;
    }
  }
  __syncthreads();
  pick<4>(
      sh, keep, sh.found * kBlock, 1, p.beams, 0,
      [&](int64_t at, float (&x)[4]) {
        const int k = (int)at / kBlock, e = (int)at % kBlock;
        const T* from = s_base[k] + e;
        if (e >= s_from[k] && e + 4 <= s_to[k]) {
          load_four(from, x);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = e + i >= s_from[k] && e + i < s_to[k] ? element(from + i) : 0.f;
        }
      },
      [&](int64_t at, float x) {
        const int k = (int)at / kBlock, e = (int)at % kBlock;
        return e >= s_from[k] && e < s_to[k] && !(x < s_cut[k]);
      },
      [&](int64_t at, float x) -> Rank {
        const int i = s_beam[(int)at / kBlock];
        return score_rank(sh.beam[i], sh.single[i] ? 0.f : x, (uint32_t)at);
      });
  if (threadIdx.x < p.num_out) {
    float score = -INFINITY;
    int parent = -1, token = -1;
    if (threadIdx.x < sh.found) {
      const Rank r = sh.best[threadIdx.x];
      const int k = r.index / kBlock;
      score = unordered(r.hi);
      parent = (int)(row0 + s_beam[k]);
      token = sh.single[s_beam[k]] ? p.end_token : s_token[k] + (int)(r.index % kBlock);
    }
    const int64_t at = (int64_t)blockIdx.x * p.num_out + threadIdx.x;
    p.out_scores[at] = score;
    p.out_parents[at] = parent;
    p.out_tokens[at] = token;
  }
}

template <class T>
cudaError_t launch(const BeamParams& p, int sms, cudaStream_t stream) {
  const int64_t units = (int64_t)p.batch * p.beams * p.plan.units, ctas = (units + kScanThreads / 32 - 1) / (kScanThreads / 32);
  cudaError_t e = cudaFuncSetAttribute(beam_scan_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScanSmem<T>);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(beam_scan_kernel<T>, dim3((unsigned)std::min<int64_t>(ctas, (int64_t)sms * kScanCtas<T>)), kScanThreads,
                        kScanSmem<T>, stream, p);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(beam_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Pick));
  if (e != cudaSuccess) return e;
  return launch_overlapped(beam_pick_kernel<T>, dim3((unsigned)p.batch), kPickThreads, sizeof(Pick), stream, p);
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams& p, int sms, cudaStream_t stream) {
  if (p.dtype == SMLA_LOGITS_BF16) return launch<__nv_bfloat16>(p, sms, stream);
  if (p.dtype == SMLA_LOGITS_FP16) return launch<__half>(p, sms, stream);
  return launch<float>(p, sms, stream);
}

}  // namespace smla
