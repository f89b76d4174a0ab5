// Attention over the paged latent cache with a sliding window and visible
// first tokens (tcgen05 / TMEM / TMA, sm_103a).
//
//   l_j = bmm1 s_j <q, c_j>,  O = bmm2 sum_j e^{l_j} s_j c_j / (sum_j e^{l_j} + e^{sink}),
//   LSE2 = log2 sum_j e^{l_j},  j over the visible rows, c_j E4M3 codes, s_j their block's scale.
//
// Both products take the codes as they lie in the cache, at the E4M3 rate, and
// still keep BF16's precision for the other operand: a BF16 number has eight
// significant bits, an E4M3 number four, so q 2^k = hi + 2^-5 lo with two E4M3
// numbers, hi the rounded value and lo the rest, which has sums of its own and
// so a scale of its own: exact down to 2^-14 of the head's largest element, an
// absolute error of at most 2^-22 of that element below.  P is hi in E4M3 + lo in
// E5M2 with one scale: BF16's rounding from 2^-6 up (split_weights).  Two such
// products cost what one BF16 product would, without widening the cache's rows in
// shared memory.
//
// Layout: one CTA takes 64 heads of one token and one split of its rows, and
// computes transposed products, rows by heads and dims by heads:
//
//   S^T[128 rows, 64 hi | 64 lo heads] = C Q^T      M = 128, N = 128, K = 512
//   O^T[512 dims, 64 heads] += C^T (P_hi + P_lo)    4 x M = 128, N = 64, K = 128
//
// An fp32 accumulator of 128 heads x 512 dims would fill tensor memory alone;
// 64 heads' O^T takes 256 columns and two S^T buffers the other 256, so no
// second CTA and no exchange is needed.  The row of a logit is its thread:
// masks and block scales are per thread, and the running maximum is needed per
// head only when the reference has to move (one barrier-vote a tile); then the
// maxima are taken over lanes and warps, and O is rescaled.
//
// With t_j = log2(e) l_j + log2 s_j and the reference m, P_j = 2^(t_j - m + 4)
// weighs the raw code c_j, and the denominator takes P_j / s_j: a block's scale is
// folded into P, never into the tile.  P has a floor (what lies under 2^-6 has
// fewer bits than BF16, under 2^-17 it is nothing), and one row may hold nearly
// all of the weight and little of the value, as first tokens do.  So
//   - m puts the largest weight of a tile between 2^-6 and 2^8.75 (P <= 431 < 448),
//     in both directions: O and the sums are fp32 and bear a smaller reference as
//     well as a larger one (up to 2^24 below its highest, and not for tiles that are
//     nothing beside what set it);
//   - where m moves up, a row of small codes (under 16 beside large ones; else under
//     a sixteenth of the tile's largest) is multiplied up in the tile by a power of
//     two, exactly, and its weights divided by it, so that m is set by what rows can
//     add to O (a row of zeros counts as 2^-40).
// A row's contribution to O is then off by at most 2^-8 of itself, BF16's rounding,
// or 2^-14 * 448 against the 2^4 * 16 or more of the one that m was set by.  (With a reference that only rises and a
// floor of 2^-14 of the largest weight, a first token with 95 % of the weight and
// small values took 14 % of the output of 2048 rows with it; now a head is off by 0.2 to
// 0.3 %, the roundings of P and of the output.  It costs 8 to 12 % of the time: the look at
// each tile's lightest head, tiles that move m down, a look at 16 codes a thread.)
//
// Rows come by TMA as chunks of 32 (16, 8) consecutive rows of one page, 5-D
// boxes {128 B, 8 rows, 4 column blocks, groups, page}, which land as 8-row
// atoms 4096 bytes apart: K-major for S^T, MN-major for O^T.  The visible rows
// [0, first) and [pos - window + 1, pos] are a list of such chunks; rows of a
// chunk that the token does not see (or that no page backs) are masked in S^T
// and set to zero in the tile before the second product, so that nothing they
// hold (NaN codes of memory never written) reaches O.
//
// Sums and maxima are fp32, O accumulates in fp32; split partials are fp32.
//
// CTAs are persistent, one an SM, and take units (64 heads of a token, a range
// of its tiles) in turn.  Sixteen warps do the softmax (all 128 rows, 16 heads
// a thread); four others issue the first products, issue the second ones, load
// rows, and look up scales.  Two tiles are in flight: while one is in the
// softmax, the other's products run, and each second product frees its tile by
// quarters, so that the next rows land behind it.
//
// What bounds it: a tile costs a CTA 2.5 us (4800 clocks, a fourth of the tiles moving
// the reference, which the others do not), of which its tensor
// instructions take 2670 (16 first products of 67 clocks; 32 second ones of 50,
// not 32: with N = 64 they wait for their A operand out of shared memory).  The
// rest is the chain second product -> free quarter -> rows -> first product ->
// softmax of a buffer, which two 64 KB tiles (Q takes 64 KB, P 32) cannot hide
// whole, and 7 us a unit for its query, sums and results.  Measured on a GB300:
// 128 requests of one token, 128 heads, 2052 rows: 98.3 us, 701 TFLOP/s of the
// plain products' count; 2049 tokens of four prompts, 128 heads, a window of 512:
// 624 us, 444 TFLOP/s; two requests of 64 heads and 2 tiles: 13.4 us.  Logits so wide
// that nearly every tile moves the reference (queries twice as long): decode 112 us;
// codes all under 16, which takes a look at whole rows where it moves: 111 us.
//
// Five kinds of warps share an instruction cache that a unit's code overflows, so
// code that need not be long is not: the products' loops are rolled to four and
// eight instructions, each look-up stands once (prompts 583 -> 548 us, before the same).
//
// Tried and slower (at these sizes, before the reference moved both ways): both products issued by one warp (decode
// 114 us against 98), warps of their own for the query (prefill 688 against
// 577), waits that poll (613 against 606), two or four times less headroom in
// the reference (prefill 552 to 564 against 576, at up to twice the error).
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "cache.cuh"
#include "cache_ptx.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace smla {
namespace {

using namespace ptx;
using namespace tc;

constexpr int kNH = kWindowHeads;                 // 64 heads
constexpr int kRows = kWindowTile;                // 128 cache rows a tile
constexpr int kSoftmaxWarps = 16;                 // four warpgroups: all 128 rows, 16 heads each
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kHW = kNH / 4;                      // heads of a softmax thread
static_assert(kHW == 16, "tmem_ld16, tmem_st16, tmem_ld_16x16");
constexpr int kScoreWarp = kSoftmaxWarps;         // issues the first products; allocates and frees TMEM
constexpr int kOutWarp = kSoftmaxWarps + 1;       // issues the second products
constexpr int kLoadWarp = kSoftmaxWarps + 2;      // looks up the units and loads the rows
constexpr int kScaleWarp = kSoftmaxWarps + 3;     // looks up the rows' masks and block scales
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
constexpr int kUnitReaders = kSoftmaxWarps + 3;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 0;                     // O^T: four blocks of 128 dims, 64 columns each
constexpr uint32_t kSCol = 256;                   // S^T: two buffers of 64 hi + 64 lo columns
constexpr float kHeadroom = 4.f;                  // log2 of P at the reference
constexpr float kMaxLog2 = 8.75f;                 // a weight may go this high before the reference moves: P <= 431 < 448
constexpr float kMinLog2 = -6.f;                  // a tile's largest may lie this low: below, P has fewer bits than BF16
constexpr float kMaxDrop = 24.f;                  // log2 that the reference may fall below its highest place
constexpr float kSumShift = 32.f;                 // log2 by which the sums of P / s are held down: blocks of 2^-64, rows of
                                                  // zeros (2^40) and a low reference (2^24) take them up to 2^104 a row
constexpr float kMinScaleLog2 = -64.f;
constexpr int kTileBytes = kRows * kHeadDim;      // 64 KB
constexpr int kGroupBytes = 8 * kHeadDim;         // 8 rows x four 128-byte column blocks
constexpr int kQBlock = 128 * 128;                // one column block of Q: 64 hi + 64 lo rows
constexpr int kPHalf = kRows * kNH;               // hi or lo of one tile's P: 8 KB
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 4 * kQBlock;
constexpr int kOffP = kOffK + 2 * kTileBytes;
constexpr int kOffSmall = kOffP + 4 * kPHalf;

// How the work is cut: each pair of a token and 64 heads by one CTA; some pairs in
// splits; by the plan of a batch whose groups share prefixes (prefix_attention.cu, which
// says what that measures).
// Pairs of a batch with groups have lists of two tables, as a plan's.
constexpr int kPairs = 0, kSplitPairs = 1, kPlanned = 2, kGroupedPairs = 3, kGroupedSplitPairs = 4;
constexpr bool has_parts(int mode) { return mode == kSplitPairs || mode == kPlanned || mode == kGroupedSplitPairs; }
constexpr bool two_tables(int mode) { return mode >= kPlanned; }

struct alignas(16) Small {
  float qscale[kNH];                              // bmm1 log2(e) 2^-k of each head
  float negref[kNH];                              // headroom - reference of each head
  float wmax[4][kNH];                             // maxima or sums of each lane quarter; a head's thread, having
                                                  // read its four, puts the change of negref in row 0, a factor in row 1
  float scale[2][kRows];                          // block scale of each row of a tile, negative: masked
  uint32_t light[2][kSoftmaxWarps];               // per lane quarter and warpgroup: its heads (bits) whose weights all lie
                                                  // under 2^kMinLog2; bit 16: no row of the quarter is seen, 17: none is small, 18: no wait has given up
  Unit unit[2];
  uint64_t k_full[2], k_free[2][4], s_full[2], s_empty[2], p_full[2], scale_full[2], unit_full[2], unit_empty[2];
  uint64_t q_full[2], drained[2];
  uint32_t tmem;
  int32_t abort_flag;
};
constexpr int kSmemBytes = kOffSmall + sizeof(Small);
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
static_assert(kNH * 128 * 2 == 2 * kPHalf, "a P buffer stages 128 dims of the output");

struct KernelParams {
  WindowParams p;
  CUtensorMap map, out_map;
  int32_t groups;                                 // head groups
  int32_t units;
  PrefixPlan plan;                                // kPlanned
};

__device__ __forceinline__ int chunk_at(const Unit& u, int k) {
  return k < u.first_chunks ? k : u.window_chunk + (k - u.first_chunks);
}

// Unit x: its heads, and (whole warp; the same result in every lane) its rows.
// Units 0 .. whole - 1 are (token, head group) pairs, the others splits of the pairs behind those.
template <bool kParts>
__device__ __forceinline__ void unit_heads(const KernelParams& kp, int x, Unit* u) {
  const WindowParams& p = kp.p;
  u->part = !kParts || x < p.whole ? -1 : x - p.whole;
  const int pair = !kParts || x < p.whole ? x : p.whole + u->part / p.num_splits;
  u->h0 = (pair % kp.groups) * kNH;
  u->t = pair / kp.groups;
  u->heads = min(kNH, p.H - u->h0);
}

// Unit x > 0 of the CTA's share of a plan (the first one stands in it).
template <int kShift>
__device__ __forceinline__ Unit planned_unit(const KernelParams& kp, int x, int lane) {
  const CacheView& c = kp.p.c;
  const PrefixPlan& plan = kp.plan;
  const int4 mine = __ldcg(plan.share + blockIdx.x);
  const int unit = mine.x + x;
  const int segment = mine.z + last_request(plan.groups + c.sum_q - mine.z, lane,
                                            [&](int s) { return __ldcg(plan.unit_of + mine.z + s) <= unit; });
  return plan_unit(c, plan, kp.p.H, kShift, blockIdx.x, __ldcg(plan.share_cost), unit, segment, x > 0, plan.cost_of,
                   plan.unit_of, plan.shared_of, plan.group, plan.token);
}

// Do the groups' starts fall, or lie outside the batch?  (Whole warp.)
__device__ __forceinline__ bool groups_out_of_order(const KernelParams& kp, int lane) {
  bool bad = false;
  for (int g = lane; g < kp.plan.groups; g += 32) {
    const int lo = fetch(kp.plan.group_starts + g), hi = fetch(kp.plan.group_starts + g + 1);
    bad |= lo < 0 || hi < lo || hi > kp.p.c.batch;
  }
  return __any_sync(0xffffffffu, bad);
}

// The prefix that request b's group shares (0: none), and the request that holds it:
// the first one of the group with new tokens.  (Whole warp; starts in order.)
__device__ __forceinline__ int group_prefix(const KernelParams& kp, int b, int lane, int* lead) {
  const CacheView& c = kp.p.c;
  *lead = b;
  if (kp.plan.groups == 0) return 0;
  const int g = last_request(kp.plan.groups, lane, [&](int x) { return fetch(kp.plan.group_starts + x) <= b; });
  const int lo = fetch(kp.plan.group_starts + g), hi = fetch(kp.plan.group_starts + g + 1);
  if (b < lo || b >= hi) return 0;
  int first = 0x7fffffff, limit = 0x7fffffff;
  for (int x = lo + lane; x < hi; x += 32) {
    int at, count;
    request_tokens(c, x, &at, &count);
    const int len = max(fetch(c.seq_lens + x), 0);
    if (count > 0 && at < c.sum_q && (int64_t)at + count > 0) {
      first = min(first, x);
      limit = min(limit, max(0, len - count + 1));
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  limit = __reduce_min_sync(0xffffffffu, limit);
  if (first == 0x7fffffff) return 0;
  *lead = first;
  return min(min(max(fetch(kp.plan.prefix_lens + g), 0), limit), c.max_pages * c.page_size);
}

template <int kShift, int kMode>
__device__ __forceinline__ Unit make_unit(const KernelParams& kp, int x, int lane, bool alone = false) {
  if constexpr (kMode == kPlanned) return planned_unit<kShift>(kp, x, lane);
  constexpr bool kParts = has_parts(kMode);
  const WindowParams& p = kp.p;
  const CacheView& c = p.c;
  Unit u;
  unit_heads<kParts>(kp, x, &u);
  int first, count;
  u.b = c.cum != nullptr ? last_request(c.batch, lane, [&](int b) { return fetch(c.cum + b) <= u.t; })
                         : u.t / (c.sum_q / c.batch);
  request_tokens(c, u.b, &first, &count);
  const bool owned = u.t >= first && u.t - first < count;   // else a token of no request: its outputs are left alone
  if (!owned) u.heads = 0;
  u.pos = owned ? max(fetch(c.seq_lens + u.b), 0) - count + (u.t - first) : -1;   // (negative lengths: none)
  u.lo = (int)max((int64_t)u.pos - p.window + 1, (int64_t)0);
  u.first_chunks = u.window_chunk = u.chunks = 0;
  const int cap = c.max_pages * c.page_size, last = min(u.pos, cap - 1);
  if (u.pos >= cap && lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
  if constexpr (two_tables(kMode)) {
    u.first = owned && u.pos >= 0 && !alone ? group_prefix(kp, u.b, lane, &u.b0) : 0;   // (the same in all lanes)
    if (u.first == 0) u.b0 = u.b;
    u.lo = u.first;
    u.first_chunks = (u.first + (1 << kShift) - 1) >> kShift;
    u.window_chunk = u.lo >> kShift;
    u.chunks = u.first_chunks + (last >= u.lo ? (last >> kShift) - u.window_chunk + 1 : 0);
  } else if (last >= 0) {
    u.first_chunks = (min(p.first_tokens, last + 1) + (1 << kShift) - 1) >> kShift;
    u.window_chunk = max(u.lo >> kShift, u.first_chunks);
    u.chunks = u.first_chunks + max(0, (last >> kShift) - u.window_chunk + 1);
  }
  const int tiles = (u.chunks + (kRows >> kShift) - 1) >> (7 - kShift);
  u.tile0 = 0;
  u.tiles = tiles;
  if (kParts && u.part >= 0) {
    const int per = (tiles + p.num_splits - 1) / p.num_splits;
    u.tile0 = min(tiles, u.part % p.num_splits * per);
    u.tiles = min(tiles, u.tile0 + per) - u.tile0;
  }
  return u;
}

// Page of list entry k, or -1 (past the list, or no page of the pool).  Tables are
// read past L1, of which the tiles leave a few KB (by L1: prompts 593 us against 581).
template <int kMode>
__device__ __forceinline__ const int32_t* chunk_table(const KernelParams& kp, const Unit& u, int k) {
  return kp.p.c.bt + (two_tables(kMode) && k < u.first_chunks ? u.b0 : u.b) * kp.p.c.bt_stride;
}
template <int kShift, int kMode>
__device__ __forceinline__ int chunk_page(const KernelParams& kp, const Unit& u, int k) {
  const CacheView& c = kp.p.c;
  if (k >= u.chunks) return -1;
  const int page = __ldcg(chunk_table<kMode>(kp, u, k) + (uint32_t)(chunk_at(u, k) << kShift) / (uint32_t)c.page_size);
  return page >= 0 && page < c.num_pages ? page : -1;
}

// Two weights of at most 431 to hi = RN(p) in E4M3 and lo = RN(p - hi) in E5M2,
// through fp16 (11 bits, its subnormals end at 2^-24).  The rest of a p in
// [2^e, 2^(e+1)) is at most 2^(e-4), three bits of it leave 2^(e-8): BF16's
// rounding, down to 2^-6 where E4M3's subnormals begin.  Below, p is off by 2^-14
// at most, under 2^-10 (where lo holds it alone) by an eighth of itself, under
// 2^-14 by 2^-17.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t* hi, uint32_t* lo) {
  const __half2 p = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(p), __NV_SATFINITE, __NV_E4M3);
  const __half2 back(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3));
  *hi = h;
  *lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(p, back)), __NV_SATFINITE, __NV_E5M2);
}

// The larger of m and the magnitude bits of the largest of 16 codes.
__device__ __forceinline__ uint32_t largest_code(uint32_t m, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m2 = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m2 = __vmaxu2(m2, __vmaxu2(w[k] & 0x7f007f00u, w[k] << 8 & 0x7f007f00u));
  return max(m, max(m2 >> 16, m2 & 0xffffu) >> 8);
}

// log2 by which a row with codes of magnitude bits up to `most` falls short of
// [128, 256), if they all lie under kLargeCode; 40 for a row of zeros.
constexpr uint32_t kLargeCode = 0x58;             // 16
__device__ __forceinline__ int shortfall(uint32_t most) {
  return most >= kLargeCode ? 0 : most == 0 ? 40 : 14 - (int)(most >> 3);
}
__device__ __forceinline__ uint32_t largest_byte(uint32_t w) {
  return max(max(w & 0xffu, w >> 8 & 0xffu), max(w >> 16 & 0xffu, w >> 24));
}

// Codes times 2^k, which the caller knows to be exact.
__device__ __forceinline__ uint32_t scale_codes(uint32_t w, __half2 by) {
  const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
  const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
  return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(lo, by)), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(hi, by)), __NV_SATFINITE, __NV_E4M3) << 16;
}

// Two query values, scaled to magnitudes under 2^8, to E4M3 pairs hi = RN(q) and
// lo = 2^5 (q - hi), at most 2^8: the rest of a value of 8 bits has four, so lo
// is exact where hi and lo end above their subnormals' step of 2^-9, that is down
// to q = 2^-7; below, q - hi is off by half of 2^-14 at most.
constexpr float kLowScale = 1.f / 32;
__device__ __forceinline__ void split_query_pair(float a, float b, uint32_t* hi, uint32_t* lo) {
  const __half2 q = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(q), __NV_SATFINITE, __NV_E4M3);
  const __half2 back(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3));
  const __half2 rest = __hmul2(__hsub2(q, back), __float2half2_rn(1.f / kLowScale));
  *hi = h;
  *lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
}

// Q of 64 heads as E4M3 pairs: rows 0-63 hi, 64-127 lo, K-major with 128-byte
// swizzle, column blocks of 128 dims.  A warp takes four heads, a lane 16 dims
// of each.
template <int kMode>
__device__ __forceinline__ void split_query(const KernelParams& kp, const Unit& u, uint8_t* sq, Small& sm, int warp,
                                            int lane) {
  const WindowParams& p = kp.p;
  constexpr int kHeads = kNH / kSoftmaxWarps;
  // (a plan's units often have a few rows only: those are every warp's, one by one)
  constexpr int kEach = kMode == kPlanned ? kSoftmaxWarps : 1;
  const int h = kMode == kPlanned ? warp : warp * kHeads;
  const __nv_bfloat16* q = p.q + (int64_t)u.t * p.q_stride_token + (int64_t)(u.h0 + h) * kHeadDim + lane * 16;
  auto at = [&](int i) {                          // the lane's dims of the warp's row i
    if constexpr (kMode != kPlanned) return q + i * kHeadDim;
    const int row = u.h0 + h + i * kEach, t = row / p.H;   // (a plan's rows may run through several tokens)
    return p.q + (int64_t)(u.t + t) * p.q_stride_token + (int64_t)(row - t * p.H) * kHeadDim + lane * 16;
  };
  const float scale = fetch_scale(p.bmm1, p.bmm1_dev) * kLog2e;
  auto load = [&](int i, uint4* v) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      v[k] = h + i * kEach < u.heads ? fetch(reinterpret_cast<const uint4*>(at(i)) + k) : make_uint4(0, 0, 0, 0);
  };
  uint4 next[2][2];                               // two heads ahead
  load(0, next[0]);
  load(1, next[1]);
  // (a loop, not unrolled: this runs once a unit, and what it costs is its instructions' way to the SM)
#pragma unroll 1
  for (int i = 0; i < kHeads; ++i) {
    const uint32_t w[8] = {next[0][0].x, next[0][0].y, next[0][0].z, next[0][0].w,
                           next[0][1].x, next[0][1].y, next[0][1].z, next[0][1].w};
    next[0][0] = next[1][0];
    next[0][1] = next[1][1];
    if (i + 2 < kHeads) load(i + 2, next[1]);
    uint32_t m2 = 0;                              // largest magnitudes as BF16 bits, even and odd dims
#pragma unroll
    for (int e = 0; e < 8; ++e) m2 = __vmaxu2(m2, w[e] & 0x7fff7fffu);
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    // 2^k that takes the largest element into [128, 256); BF16 exponent field e: magnitude in [2^(e-127), 2^(e-126))
    const int e = min(max((int)(m >> 7), 8), 254);
    const int k = 134 - e;
    const float up = __uint_as_float((uint32_t)(k + 127) << 23), down = __uint_as_float((uint32_t)(127 - k) << 23);
    if (lane == 0) sm.qscale[h + i * kEach] = scale * down;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      split_query_pair(__uint_as_float(w[x] << 16) * up, __uint_as_float(w[x] & 0xffff0000u) * up, hi + x, lo + x);
    uint4 h16 = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16, hi[6] | hi[7] << 16);
    uint4 l16 = make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, lo[4] | lo[5] << 16, lo[6] | lo[7] << 16);
    if (m >= 0x7f80u) {                           // a head with an infinity or NaN gets NaN everywhere
      h16 = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
      l16 = make_uint4(0, 0, 0, 0);
    }
    uint8_t* to = sq + (lane >> 3) * kQBlock;     // column block; 16-byte chunk lane % 8 of it
    *reinterpret_cast<uint4*>(to + sw128_offset(h + i * kEach, lane & 7)) = h16;
    *reinterpret_cast<uint4*>(to + sw128_offset(h + i * kEach + kNH, lane & 7)) = l16;
  }
}

// kShift: log2 of a TMA box's rows; kMode: without the code of splits the kernel is
// 3 % faster where units are many (what runs once a unit comes through the
// instruction cache every time)
template <int kShift, int kMode>
__global__ void __launch_bounds__(kThreads, 1) window_kernel(const __grid_constant__ KernelParams kp) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr bool kParts = has_parts(kMode);
  Small& sm = *reinterpret_cast<Small*>(smem + kOffSmall);
  const WindowParams& p = kp.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t k_addr = smem_addr(smem + kOffK), q_addr = smem_addr(smem + kOffQ), p_addr = smem_addr(smem + kOffP);
  auto bar = [](uint64_t& b) { return smem_addr(&b); };

  if (smem_addr(smem) & 1023u) {                  // the operands' swizzles count on the alignment asked for above
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_INTERNAL);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm.k_full[i]), 1);
      for (int k = 0; k < 4; ++k) mbar_init(bar(sm.k_free[i][k]), 1);
      mbar_init(bar(sm.s_full[i]), 1);
      mbar_init(bar(sm.s_empty[i]), kSoftmaxWarps);
      mbar_init(bar(sm.p_full[i]), kSoftmaxWarps);
      mbar_init(bar(sm.scale_full[i]), 1);
      mbar_init(bar(sm.unit_full[i]), 1);
      mbar_init(bar(sm.unit_empty[i]), kUnitReaders);
      mbar_init(bar(sm.q_full[i]), kSoftmaxWarps);
      mbar_init(bar(sm.drained[i]), 1);
    }
    sm.abort_flag = 0;
    fence_mbar_init_cluster();
    fence_proxy_async_smem();
  }
  if (warp == kScoreWarp) tmem_alloc(smem_addr(&sm.tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  await_prior_kernel();
  const uint32_t tmem = sm.tmem;
  Ctx cx{&sm.abort_flag, p.err};
  // Tiles are numbered through all units of the CTA: tile n uses buffers n & 1,
  // and completes phase n >> 1 of their barriers.  Its second product frees the
  // tile 32 rows at a time; k_free[b][3] is also its end.  Queries are numbered
  // too, and take q_full in turn: behind a first unit without tiles the second
  // unit's may be there before the first products' warp has waited for the first
  // one's, but no third is before it has waited for both.
  union {
    int4 words[4];
    Unit unit;
  } first;                                        // of a plan
  if (kMode == kPlanned && warp == kLoadWarp)
#pragma unroll
    for (int k = 0; k < 4; ++k) first.words[k] = __ldcg(kp.plan.first + blockIdx.x * 4 + k);
  const int mine = kMode == kPlanned ? __ldcg(kp.plan.share + blockIdx.x).y
                                     : (kp.units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  if (kMode == kPlanned && mine <= 0) {
    if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
    return;
  }

  if (warp == kLoadWarp) {
    // ------------------------------------------------------ units and rows
    constexpr int kBoxes = kRows >> kShift;       // of a tile
    int n = 0;
    bool ok = true;
    bool alone = false;                           // groups out of order share nothing
    if constexpr (kMode == kGroupedPairs || kMode == kGroupedSplitPairs) {
      alone = groups_out_of_order(kp, lane);
      if (alone && lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_STATE);
    }
    Unit ahead = kMode == kPlanned ? first.unit : make_unit<kShift, kMode>(kp, blockIdx.x, lane, alone);
    auto prefetch_query = [&](const Unit& u) {
      if constexpr (kMode == kPlanned) {          // rows of several tokens: one by one
        for (int i = lane; u.tiles > 0 && i < u.heads; i += 32) {
          const int t = (u.h0 + i) / p.H, head = u.h0 + i - t * p.H;
          bulk_prefetch_l2(p.q + (int64_t)(u.t + t) * p.q_stride_token + (int64_t)head * kHeadDim, kHeadDim * 2);
        }
        __syncwarp();
        return;
      }
      if (u.tiles > 0 && elect_one())
        bulk_prefetch_l2(p.q + (int64_t)u.t * p.q_stride_token + (int64_t)u.h0 * kHeadDim, u.heads * kHeadDim * 2);
      __syncwarp();
    };
    if constexpr (kMode != kPlanned) prefetch_query(ahead);   // (a plan's first unit: the softmax waits for it, and loads them then)
    for (int x = 0; ok && x < mine; ++x) {
      const Unit u = ahead;
      if (x >= 2) ok = warp_wait(cx, bar(sm.unit_empty[x & 1]), ((x >> 1) - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        sm.unit[x & 1] = u;
        mbar_arrive(bar(sm.unit_full[x & 1]));
      }
      __syncwarp();
      // Lane l looks up box l of the tile; one lane then holds all of them, so
      // that nothing but the wait and the copy stands between a quarter of the
      // buffer and its rows.
      auto look_up = [&](int i, int* page, int* group) {
        const int k = (u.tile0 + i) * kBoxes + lane;
        *page = lane < kBoxes && i < u.tiles ? chunk_page<kShift, kMode>(kp, u, k) : -1;
        *group = (uint32_t)(chunk_at(u, min(k, u.chunks - 1)) << kShift) % (uint32_t)p.c.page_size / 8;
      };
      int page = -1, group = 0;
      for (int i = -1; ok && i < u.tiles; ++i) {
        const int b = n & 1;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, page >= 0)) * kHeadDim << kShift;
        int pg[kBoxes], g[kBoxes];
#pragma unroll
        for (int k = 0; k < kBoxes; ++k) {
          pg[k] = __shfl_sync(0xffffffffu, page, k);
          g[k] = __shfl_sync(0xffffffffu, group, k);
        }
        if (i + 1 < u.tiles) look_up(i + 1, &page, &group);
        bool good = true;
        if (i >= 0 && elect_one()) {
          const uint32_t full = bar(sm.k_full[b]), dst = k_addr + b * kTileBytes;
#pragma unroll
          for (int k = 0; k < kBoxes; ++k) {
            constexpr int kPerQuarter = kBoxes / 4;
            if (k % kPerQuarter == 0 && n >= 2)
              good = good && wait_bar(cx, bar(sm.k_free[b][k / kPerQuarter]), ((n >> 1) - 1) & 1, false);
            if (!good) break;
            if (k == 0) mbar_arrive_expect_tx(full, bytes);
            if (pg[k] >= 0) tma_load_5d(dst + k * (kHeadDim << kShift), &kp.map, 0, 0, 0, g[k], pg[k], full);
          }
        }
        ok = __all_sync(0xffffffffu, good);
        n += i >= 0;
        if (i == min(1, u.tiles - 1) && x + 1 < mine) {       // the next unit and its queries' way to L2
          ahead = make_unit<kShift, kMode>(kp, kMode == kPlanned ? x + 1 : blockIdx.x + (x + 1) * gridDim.x, lane, alone);
          prefetch_query(ahead);
        }
      }
    }
    // after an abort the last copies may still be in flight
    for (int i = max(0, n - 2); i < n + (ok ? 0 : 1); ++i) drain_wait(bar(sm.k_full[i & 1]), (i >> 1) & 1);
  } else if (warp == kScaleWarp) {
    // -------------------------------------------------- the rows' scales
    // four rows a lane, looked up a tile before their buffer is free
    constexpr int per_tile = kRows >> kShift;
    int n = 0;
    bool ok = true;
    for (int x = 0; ok && x < mine; ++x) {
      ok = warp_wait(cx, bar(sm.unit_full[x & 1]), (x >> 1) & 1);
      const Unit u = sm.unit[x & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.unit_empty[x & 1]));
      float next[kRows / 32] = {};
      // (every load is unconditional, at a clamped place: the four are in flight together)
      auto look_up = [&](int i) {
        constexpr int kY = kRows / 32;
        int off[kY], page[kY];
        bool seen[kY], missing = false;
#pragma unroll
        for (int y = 0; y < kY; ++y) {
          const int r = y * 32 + lane, k = (u.tile0 + i) * per_tile + (r >> kShift);
          const uint32_t j = (uint32_t)((chunk_at(u, min(k, u.chunks - 1)) << kShift) + (r & ((1 << kShift) - 1)));
          if constexpr (two_tables(kMode))
            seen[y] = k < u.chunks && (k < u.first_chunks ? (int)j < u.first : (int)j >= u.lo && (int)j <= u.pos);
          else
            seen[y] = k < u.chunks && (int)j <= u.pos && ((int)j >= u.lo || (int)j < p.first_tokens);
          const uint32_t col = j / (uint32_t)p.c.page_size;
          page[y] = __ldcg(chunk_table<kMode>(kp, u, k) + col);
          off[y] = (int)((j - col * (uint32_t)p.c.page_size) / (uint32_t)p.c.block_rows);
        }
#pragma unroll
        for (int y = 0; y < kY; ++y) {
          const bool in = page[y] >= 0 && page[y] < p.c.num_pages;
          next[y] = fetch(p.c.scales + (int64_t)(in ? page[y] : 0) * p.c.scale_stride + off[y]);
          missing |= seen[y] && !in;
          seen[y] = seen[y] && in;
        }
        if (missing && p.err) atomicOr(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
#pragma unroll
        for (int y = 0; y < kY; ++y) next[y] = seen[y] ? fabsf(next[y]) : -1.f;
      };
      // A tile on its way to L2 long before it is loaded: DRAM's latency would
      // otherwise stand between a tile's last product and the next one in its buffer.
      auto prefetch = [&](int i) {
        const int k = (u.tile0 + i) * per_tile + lane;
        const int page = lane < per_tile && i < u.tiles ? chunk_page<kShift, kMode>(kp, u, k) : -1;
        const int group = (uint32_t)(chunk_at(u, min(k, u.chunks - 1)) << kShift) % (uint32_t)p.c.page_size / 8;
#pragma unroll 1
        for (int y = 0; y < per_tile; ++y) {
          const int pg = __shfl_sync(0xffffffffu, page, y), g = __shfl_sync(0xffffffffu, group, y);
          if (pg >= 0 && elect_one()) tma_prefetch_5d(&kp.map, 0, 0, 0, g, pg);
          __syncwarp();
        }
      };
      for (int i = -1; ok && i < u.tiles; ++i) {
        const int b = n & 1;
        float s[kRows / 32];
#pragma unroll
        for (int y = 0; y < kRows / 32; ++y) s[y] = next[y];
        if (i + 1 < u.tiles) {
          look_up(i + 1);
          prefetch(i + 3);
        }
        if (i < 0) continue;
        // (the softmax has read this buffer's last scales before it gave its P)
        if (n >= 2) ok = warp_wait(cx, bar(sm.p_full[b]), ((n >> 1) - 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int y = 0; y < kRows / 32; ++y) sm.scale[b][y * 32 + lane] = s[y];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.scale_full[b]));
        ++n;
      }
    }
  } else if (warp == kScoreWarp) {
    // ------------------------------------------------------ first products
    constexpr uint32_t idesc_s = idesc(true, 128, 128, false);
    int n = 0, q = 0;
    bool ok = true;
    for (int x = 0; ok && x < mine; ++x) {
      ok = warp_wait(cx, bar(sm.unit_full[x & 1]), (x >> 1) & 1);
      const int tiles = sm.unit[x & 1].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.unit_empty[x & 1]));
      // (the first unit's queries come in any case)
      if (ok && (tiles > 0 || x == 0)) {
        ok = warp_wait(cx, bar(sm.q_full[q & 1]), (q >> 1) & 1);
        ++q;
      }
      if (!ok || tiles == 0) continue;
      for (int i = 0; ok && i < tiles; ++i, ++n) {
        const int b = n & 1;
        ok = warp_wait(cx, bar(sm.k_full[b]), (n >> 1) & 1);
        if (ok && n >= 2) ok = warp_wait(cx, bar(sm.s_empty[b]), ((n >> 1) - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t tile = k_addr + b * kTileBytes;
#pragma unroll 4
          for (int k = 0; k < 16; ++k)
            mma<true>(tmem + kSCol + b * 128, desc_sw128(tile + (k >> 2) * 1024 + (k & 3) * 32, 16, kGroupBytes),
                      desc_sw128(q_addr + (k >> 2) * kQBlock + (k & 3) * 32, 16, 1024), idesc_s, k > 0);
          mma_commit(bar(sm.s_full[b]));
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(bar(sm.drained[0]));
    drain_wait(bar(sm.drained[0]), 0);
  } else if (warp == kOutWarp) {
    // ----------------------------------------------------- second products
    constexpr uint32_t idesc_o = idesc(true, 128, kNH, true) | kIdescAMnMajor;
    constexpr uint32_t idesc_half[2] = {idesc_o, idesc_o | kIdescBE5M2};
    int n = 0;
    bool ok = true;
    for (int x = 0; ok && x < mine; ++x) {
      ok = warp_wait(cx, bar(sm.unit_full[x & 1]), (x >> 1) & 1);
      const int tiles = sm.unit[x & 1].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.unit_empty[x & 1]));
      for (int i = 0; ok && i < tiles; ++i, ++n) {
        const int b = n & 1;
        ok = warp_wait(cx, bar(sm.p_full[b]), (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t tile = k_addr + b * kTileBytes, pb = p_addr + b * 2 * kPHalf;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int m = 0; m < 4; ++m)
                mma<true>(tmem + kOCol + m * kNH, desc_sw128(tile + m * 1024 + k * 4 * kGroupBytes, 1024, kGroupBytes),
                          desc_sw64(pb + half * kPHalf + k * 32 * kNH, 512, 512), idesc_half[half], i > 0 || k > 0 || half > 0);
            mma_commit(bar(sm.k_free[b][k]));
          }
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(bar(sm.drained[1]));
    drain_wait(bar(sm.drained[1]), 0);
  } else {
    // ------------------------------------------------------------- softmax
    const int r = threadIdx.x & (kRows - 1);      // row of the tile = TMEM lane
    const int hw = (threadIdx.x / kRows) * kHW;   // first of the thread's heads
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint64_t sum[kHW / 2];                        // of two heads each
    float drop = 0.f;                             // how far head threadIdx.x's reference lies below its highest place,
                                                  // counted for rows with a code of 16 or more
    int n = 0, q = 0;
    bool failed = false;
    {
      // the first unit's queries, while its rows are looked up (a unit without any leaves them unused)
      Unit u;
      if constexpr (kMode == kPlanned) {
        failed = !warp_wait(cx, bar(sm.unit_full[0]), 0);
        u = sm.unit[0];
        if (failed) u.heads = 0;
      } else {
        unit_heads<kParts>(kp, blockIdx.x, &u);
      }
      split_query<kMode>(kp, u, smem + kOffQ, sm, warp, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.q_full[0]));
      ++q;
    }
    if constexpr (kMode != kPlanned) failed = !warp_wait(cx, bar(sm.unit_full[0]), 0);
    if (threadIdx.x < kNH) sm.negref[threadIdx.x] = 0.f;
    for (int x = 0; x < mine; ++x) {
      if (named_bar_or(1, kSoftmaxThreads, failed)) break;   // also: qscale and negref are written
      const int tiles = sm.unit[x & 1].tiles;
#pragma unroll
      for (int e = 0; e < kHW / 2; ++e) sum[e] = 0;
      bool fresh = true;                          // no row seen, so no reference yet
      int i = 0;
      for (; i < tiles; ++i, ++n) {
        const int b = n & 1;
        failed |= !warp_wait(cx, bar(sm.scale_full[b]), (n >> 1) & 1);
        const float s = sm.scale[b][r];
        const bool seen = !(s < 0.f);             // (a NaN scale is seen, and makes the result NaN)
        const float ls = fmaxf(fast_log2(s), kMinScaleLog2);
        float inv = fast_exp2(-ls - kSumShift);
        // Is the row one of small codes?  (While its first product runs; of most, 16 codes of the thread's block say no.)
        failed |= !warp_wait(cx, bar(sm.k_full[b]), (n >> 1) & 1);
        uint8_t* const codes = smem + kOffK + b * kTileBytes + (r >> 3) * kGroupBytes + (r & 7) * 128 + (hw / kHW) * 1024;
        auto codes16 = [&](int y) { return reinterpret_cast<uint4*>(codes + ((y ^ (r & 7)) << 4)); };
        uint32_t most = largest_code(0, *codes16(0));
        failed |= !warp_wait(cx, bar(sm.s_full[b]), (n >> 1) & 1);
        tc_fence_after();
        uint64_t d[kHW / 2];                      // t - reference + headroom
        {
          uint32_t hi[kHW], lo[kHW];
          tmem_ld16(lane_base + kSCol + b * 128 + hw, hi);
          tmem_ld16(lane_base + kSCol + b * 128 + kNH + hw, lo);
          tmem_wait_ld();
          const uint64_t s2 = f2_pack(s, s), ls2 = f2_pack(ls, ls), low2 = f2_pack(kLowScale, kLowScale);
#pragma unroll
          for (int e = 0; e < kHW / 2; e += 2) {
            const ulonglong2 qs = *reinterpret_cast<const ulonglong2*>(sm.qscale + hw + 2 * e);
            const ulonglong2 ng = *reinterpret_cast<const ulonglong2*>(sm.negref + hw + 2 * e);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int h = 2 * (e + k);
              const uint64_t v = f2_fma(f2_pack(__uint_as_float(lo[h]), __uint_as_float(lo[h + 1])), low2,
                                        f2_pack(__uint_as_float(hi[h]), __uint_as_float(hi[h + 1])));
              d[e + k] = f2_add(f2_fma(f2_mul(v, k ? qs.y : qs.x), s2, ls2), k ? ng.y : ng.x);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.s_empty[b]));
        float top = -INFINITY;
        uint32_t light = most >= kLargeCode;      // then: signs of d - kMinLog2, first head highest (NaN is not light)
#pragma unroll
        for (int e = 0; e < kHW / 2; ++e) {
          float v, w;
          f2_unpack(d[e], v, w);
          top = fmaxf(top, fmaxf(v, w));
          f2_unpack(f2_add(d[e], f2_pack(-kMinLog2, -kMinLog2)), v, w);
          light = __funnelshift_l(__float_as_uint(v), light, 1);
          light = __funnelshift_l(__float_as_uint(w), light, 1);
        }
        light = __reduce_and_sync(0xffffffffu, (seen ? (light & 0xffffu) | (light >> 16) << 17 : 0x3ffffu) | (failed ? 0u : 0x40000u));
        if (lane == 0) sm.light[b][(warp & 3) * 4 + hw / kHW] = light;
        if (i == 0 && warp == 0 && elect_one()) bulk_store_wait_read<0>();   // the last unit's output has left the P buffers
        bool move = named_bar_or(1, kSoftmaxThreads, failed || fresh || (seen && top > kMaxLog2));
        uint4 all = reinterpret_cast<const uint4*>(sm.light[b])[0];
#pragma unroll
        for (int y = 1; y < 4; ++y) {
          const uint4 a = reinterpret_cast<const uint4*>(sm.light[b])[y];
          all.x &= a.x, all.y &= a.y, all.z &= a.z, all.w &= a.w;
        }
        const bool any = (all.x & 0x10000u) == 0;      // (the same in all threads)
        if (__builtin_expect(move || (any && ((all.x | all.y | all.z | all.w) & 0xffffu) != 0), 0)) {
          // ---- a new reference, by what the rows can add to O at most: their weights times their largest codes
          const uint32_t every = all.x & all.y & all.z & all.w;
          if (every < 0x40000u) break;
          // (a light tile's small rows are nothing beside what set the reference)
          int up = 0, low = 0;                    // by how much the row's codes are small beside the tile's, and the tile's
          if (move && (every & 0x20000u) == 0) {
            uint32_t* const rows = reinterpret_cast<uint32_t*>(smem + kOffP + b * 2 * kPHalf);      // (P comes behind barriers)
#pragma unroll 1
            for (int y = 1; y < 8; ++y) most = largest_code(most, *codes16(y));
            reinterpret_cast<uint8_t*>(rows + r)[hw / kHW] = (uint8_t)(seen ? most : 0u);
            named_bar_sync(1, kSoftmaxThreads);
            uint32_t largest = 0;
#pragma unroll
            for (int y = 0; y < kRows / 32; ++y) largest = max(largest, largest_byte(rows[y * 32 + lane]));
            low = shortfall(__reduce_max_sync(0xffffffffu, largest));
            up = seen ? shortfall(largest_byte(rows[r])) - low : 0;
            if (up < 4) up = 0;                   // (as 16 and 448 are both large)
          }
          const uint64_t down2 = f2_pack(-(float)up, -(float)up);
#pragma unroll
          for (int e = 0; e < kHW / 2; ++e) {
            float v, w;
            f2_unpack(f2_add(d[e], down2), v, w);
            v = warp_max(seen ? v : -INFINITY);
            w = warp_max(seen ? w : -INFINITY);
            if (lane == e) *reinterpret_cast<float2*>(&sm.wmax[warp & 3][hw + 2 * e]) = make_float2(v, w);
          }
          named_bar_sync(1, kSoftmaxThreads);
          float by = 0.f;                         // by how much the reference of head threadIdx.x moves
          if (threadIdx.x < kNH) {
            const int h = threadIdx.x;
            const float m = fmaxf(fmaxf(sm.wmax[0][h], sm.wmax[1][h]), fmaxf(sm.wmax[2][h], sm.wmax[3][h])) - kHeadroom;
            if (fresh) {
              if (m != -INFINITY) by = m;
              drop = -(float)low;
            } else if (m > 0.f) {
              by = m;
              drop = fmaxf(drop - by, -(float)low);
            } else if (m < kMinLog2 - kHeadroom &&
                       m > drop - kHeadroom - 10.f - fast_log2((float)(sm.unit[x & 1].chunks << kShift))) {
              // (as many rows as there are of less than that, with codes of 448, are under 2^-9 of one at the
              // highest reference with 16)
              by = fmaxf(m, drop - kMaxDrop);
              drop -= by;
            }
            // (by what it is rounded to, as the sums are: they would drift apart from it over many moves)
            const float now = sm.negref[h], then = now - by;
            by = now - then;
            sm.negref[h] = then;
            sm.wmax[0][h] = -by;
            sm.wmax[1][h] = fresh ? 0.f : fast_exp2(-by);
          }
          const bool moved = named_bar_or(1, kSoftmaxThreads, by != 0.f);
          // (by the rows, not by the maxima: a head of NaN has none, and the others keep theirs)
          fresh = fresh && !any;
          if (moved && i > 0) {
            // O^T by column, once the products into it are done
            failed |= !warp_wait(cx, bar(sm.k_free[b ^ 1][3]), ((n - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              uint32_t o[kHW];
              tmem_ld16(lane_base + kOCol + m * kNH + hw, o);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < kHW; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * sm.wmax[1][hw + h]);
              tmem_st16(lane_base + kOCol + m * kNH + hw, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          if (moved) {
#pragma unroll
            for (int e = 0; e < kHW / 2; ++e) {
              d[e] = f2_add(d[e], *reinterpret_cast<const uint64_t*>(sm.wmax[0] + hw + 2 * e));
              sum[e] = f2_mul(sum[e], *reinterpret_cast<const uint64_t*>(sm.wmax[1] + hw + 2 * e));
            }
          }
          if (up != 0) {
            // a row of small codes: the codes up, exactly, its weights down, which may be too large for P
#pragma unroll
            for (int e = 0; e < kHW / 2; ++e) d[e] = f2_add(d[e], down2);
            inv *= __uint_as_float((uint32_t)(127 + up) << 23);
            if (up <= 14) {                       // (more: a row of zeros)
              const __half2 factor = __half2half2(__ushort_as_half((unsigned short)((15 + up) << 10)));
#pragma unroll 1
              for (int y = 0; y < 8; ++y) {
                uint4* const at = codes16(y);
                const uint4 v = *at;
                *at = make_uint4(scale_codes(v.x, factor), scale_codes(v.y, factor), scale_codes(v.z, factor),
                                 scale_codes(v.w, factor));
              }
            }
          }
        }
        // P in pairs: row r of the MN-major operand is 64 bytes, heads along it
        uint8_t* pb = smem + kOffP + b * 2 * kPHalf + r * kNH;
        const uint64_t inv2 = f2_pack(inv, inv);
        {
          uint32_t hi[8] = {}, lo[8] = {};
          if (seen) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float v, w;
              f2_unpack(d[e], v, w);
              v = fast_exp2(v);
              w = fast_exp2(w);
              sum[e] = f2_fma(f2_pack(v, w), inv2, sum[e]);
              split_weights(v, w, hi + e, lo + e);
            }
          }
          const int at = ((hw >> 4) ^ ((r >> 1) & 3)) << 4;             // 64-byte swizzle
          *reinterpret_cast<uint4*>(pb + at) = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16,
                                                          hi[4] | hi[5] << 16, hi[6] | hi[7] << 16);
          *reinterpret_cast<uint4*>(pb + kPHalf + at) = make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16,
                                                                   lo[4] | lo[5] << 16, lo[6] | lo[7] << 16);
        }
        if (__builtin_expect(!seen, 0)) {
          // the first product has read the row (its commit is what s_full waited for); the second must find zeros
          uint8_t* row = smem + kOffK + b * kTileBytes + (r >> 3) * kGroupBytes + (r & 7) * 128 + (hw / kHW) * 1024;
#pragma unroll
          for (int y = 0; y < 8; ++y) *reinterpret_cast<uint4*>(row + ((y ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.p_full[b]));
      }
      if (i < tiles) break;                       // a wait gave up (all threads agreed)

      // the next unit's queries, while the last products of this one run (their
      // buffer is free: the last S of this unit has been read)
      float sink = -INFINITY;                     // of head threadIdx.x, in log2 units
      if (p.sinks != nullptr && (!kParts || sm.unit[x & 1].part < 0) && threadIdx.x < sm.unit[x & 1].heads)
        sink = fetch(p.sinks + sm.unit[x & 1].h0 + threadIdx.x) * kLog2e;
      const float out_scale = !kParts || sm.unit[x & 1].part < 0 ? fetch_scale(p.bmm2, p.bmm2_dev) : 1.f;
      const int t = sm.unit[x & 1].t, h0 = sm.unit[x & 1].h0, heads = sm.unit[x & 1].heads;
      const bool whole = !kParts || sm.unit[x & 1].part < 0;
      const int64_t part = (int64_t)sm.unit[x & 1].part * kNH;                // its first partial row
      if (x + 1 < mine) {
        failed |= !warp_wait(cx, bar(sm.unit_full[(x + 1) & 1]), ((x + 1) >> 1) & 1);
        if (!failed && sm.unit[(x + 1) & 1].tiles > 0) {
          split_query<kMode>(kp, sm.unit[(x + 1) & 1], smem + kOffQ, sm, warp, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm.q_full[q & 1]));
          ++q;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.unit_empty[x & 1]));

      // ---------------------------------------------------------- results
      const int64_t th = (int64_t)t * p.H + h0;                               // first (token, head) of the unit
      if (__builtin_expect(tiles == 0, 0)) {      // no visible row (of this split)
        if (!whole) {
          if (threadIdx.x < heads) p.part_lse[part + threadIdx.x] = -INFINITY;
        } else {
          uint4* o = reinterpret_cast<uint4*>(p.out + th * kHeadDim);
          for (int k = threadIdx.x; k < heads * (kHeadDim / 8); k += kSoftmaxThreads) o[k] = make_uint4(0, 0, 0, 0);
          if (p.out_lse && threadIdx.x < heads) p.out_lse[th + threadIdx.x] = -INFINITY;
        }
        continue;
      }
      // sums over the rows: the warp's lanes halve the heads they hold at each
      // step; lanes l and l + 16 end with head l's
      float total;
      {
        float v[kHW];
#pragma unroll
        for (int e = 0; e < kHW / 2; ++e) f2_unpack(sum[e], v[2 * e], v[2 * e + 1]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
          for (int h = 0; h < o; ++h) {
            const float give = (lane & o) ? v[h] : v[h + o], keep = (lane & o) ? v[h + o] : v[h];
            v[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        total = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
      }
      failed |= !warp_wait(cx, bar(sm.k_free[(n - 1) & 1][3]), ((n - 1) >> 1) & 1);
      tc_fence_after();
      if (named_bar_or(1, kSoftmaxThreads, failed)) break;
      if (lane < kHW) sm.wmax[warp & 3][hw + lane] = total;
      named_bar_sync(1, kSoftmaxThreads);
      if (threadIdx.x < kNH) {
        const int h = threadIdx.x;
        total = (sm.wmax[0][h] + sm.wmax[1][h]) + (sm.wmax[2][h] + sm.wmax[3][h]);
        float f = 0.f, lse = -INFINITY;
        if (!(total == 0.f)) {                    // NaN passes
          lse = fast_log2(total) + kSumShift - sm.negref[h];
          f = out_scale * (1.f / (1ull << (int)kSumShift)) / (total + total * fast_exp2(sink - lse));
        }
        sm.wmax[1][h] = f;
        sm.negref[h] = 0.f;                       // the next unit's
        if (h < heads) {
          if (!whole) p.part_lse[part + h] = lse;
          else if (p.out_lse) p.out_lse[th + h] = lse;
        }
      }
      named_bar_sync(1, kSoftmaxThreads);
      if (__builtin_expect(!whole, 0)) {
        // (a plan's units of up to 16 rows: 128 dims of all of them a warpgroup)
        const bool few = kMode == kPlanned && heads <= kHW;
        const int h0 = few ? 0 : hw;
#pragma unroll 1
        for (int m = few ? hw / kHW : 0; m < (few ? hw / kHW + 1 : 4); ++m) {   // dims 128 m .. + 127, one a thread
          uint32_t o[kHW];
          tmem_ld16(lane_base + kOCol + m * kNH + h0, o);
          tmem_wait_ld();
          float* dst = p.part_o + (part + h0) * kHeadDim + m * 128 + r;
#pragma unroll
          for (int h = 0; h < kHW; ++h)
            if (h0 + h < heads) dst[h * kHeadDim] = __uint_as_float(o[h]) * sm.wmax[1][h0 + h];
        }
      } else {
        // 8 x 8 fragments, transposed on their way into a P buffer: [64 heads][64 dims] BF16 twice, 128-byte
        // swizzle, stored by TMA while the next 128 dims are read
        float f[kHW / 4];                         // of this lane's heads: 8 j + 2 (lane % 4) and + 1
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f[2 * j] = sm.wmax[1][hw + 8 * j + 2 * (lane & 3)];
          f[2 * j + 1] = sm.wmax[1][hw + 8 * j + 2 * (lane & 3) + 1];
        }
#pragma unroll 1
        for (int m = 0; m < 4; m += 2) {
          if (m > 0) {                            // the buffers' first stores have read them
            if (warp == 0 && elect_one()) bulk_store_wait_read<0>();
            named_bar_sync(1, kSoftmaxThreads);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t o[2][8];
            tmem_ld_16x16(lane_base + kOCol + (m + k) * kNH + hw, o[0]);
            tmem_ld_16x16(lane_base + (16u << 16) + kOCol + (m + k) * kNH + hw, o[1]);
            tmem_wait_ld();
            const uint32_t stage = p_addr + k * 2 * kPHalf + ((warp & 3) >> 1) * (kNH * 128);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)         // dims 8 i .. + 7 of the warp's 32
                v[i] = pack_bf16x2(__uint_as_float(o[i >> 1][4 * j + 2 * (i & 1)]) * f[2 * j],
                                   __uint_as_float(o[i >> 1][4 * j + 2 * (i & 1) + 1]) * f[2 * j + 1]);
              const int head = hw + 8 * j + (lane & 7), ch = (warp & 1) * 4 + (lane >> 3);
              stmatrix4_trans(stage + head * 128 + ((ch ^ (head & 7)) << 4), v[0], v[1], v[2], v[3]);
            }
          }
          fence_proxy_async_smem();
          named_bar_sync(1, kSoftmaxThreads);
          if (warp == 0 && elect_one())
#pragma unroll
            for (int k = 0; k < 4; ++k) tma_store_3d(&kp.out_map, m * 128 + k * 64, h0, t, p_addr + k * (kNH * 128));
        }
      }
      tc_fence_before();
    }
    admit_next_kernel();
    if (warp == 0 && elect_one()) bulk_store_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
}

// Merges the S normalised fp32 partials of a split pair's heads: weights
// 2^(LSE_s - LSE), then the sink and bmm2.  The weights first, a split a thread;
// then no partial's load waits for another's.  Up to four teams of threads share
// many splits (64 heads over 32768 rows in 128 splits: 34.6 us of both kernels with
// one team, 24.2 with four; over 262144 rows 72.0 and 60.1).
constexpr int kMergeThreads = 128;                // of a team; one head: four dims a thread
constexpr int kMergeTeams = 4;

template <int kTeams>
__global__ void __launch_bounds__(kMergeThreads * kTeams) window_merge_kernel(const WindowParams p, int groups) {
  constexpr int kThreads = kMergeThreads * kTeams;
  __shared__ float weight[kMaxWindowSplits];
  __shared__ float warp_top[kThreads / 32], warp_sum[kThreads / 32];
  __shared__ float4 share[kTeams][kMergeThreads];
  const int pair = blockIdx.x / kNH, hl = blockIdx.x % kNH, warp = threadIdx.x / 32;
  const int team = threadIdx.x / kMergeThreads, lane4 = threadIdx.x % kMergeThreads, d = lane4 * 4;
  const int t = (p.whole + pair) / groups, h = (p.whole + pair) % groups * kNH + hl;
  if (h >= p.H) return;
  const int64_t th = (int64_t)t * p.H + h;
  await_prior_kernel();
  admit_next_kernel();
  if (p.c.cum != nullptr && (t < fetch(p.c.cum) || t >= fetch(p.c.cum + p.c.batch))) return;   // no request's
  const int64_t row = (int64_t)pair * p.num_splits * kNH + hl;
  float top = -INFINITY;
  bool nan = false;
  for (int s = threadIdx.x; s < p.num_splits; s += kThreads) {
    const float l = fetch(p.part_lse + row + s * kNH);
    weight[s] = l;
    nan |= isnan(l);
    top = fmaxf(top, l);
  }
  top = warp_max(top);
  if ((threadIdx.x & 31) == 0) warp_top[warp] = top;
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
  float sum = 0.f;
  for (int s = threadIdx.x; s < p.num_splits; s += kThreads) {
    const float w = weight[s] == -INFINITY ? 0.f : fast_exp2(weight[s] - top);
    weight[s] = w;
    sum += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) warp_sum[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) sum += warp_sum[w];
  const float* o_s = p.part_o + row * kHeadDim + d;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = team; s < p.num_splits; s += kTeams) {
    const float w = weight[s];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);   // an empty partial is not written
    if (w != 0.f) o = fetch(reinterpret_cast<const float4*>(o_s + (int64_t)s * kNH * kHeadDim));
    acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y), acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
  }
  if constexpr (kTeams > 1) {
    share[team][lane4] = acc;
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int w = 1; w < kTeams; ++w) {
      const float4 o = share[w][lane4];
      acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
    }
  }
  float lse = -INFINITY, f = 0.f;
  if (top != -INFINITY || nan) {
    lse = nan ? NAN : top + fast_log2(sum);
    f = fetch_scale(p.bmm2, p.bmm2_dev) / sum;
    if (p.sinks != nullptr) f *= 1.f / (1.f + fast_exp2(fetch(p.sinks + h) * kLog2e - lse));
  }
  uint2 v;
  v.x = pack_bf16x2(acc.x * f, acc.y * f);
  v.y = pack_bf16x2(acc.z * f, acc.w * f);
  *reinterpret_cast<uint2*>(p.out + th * kHeadDim + d) = v;
  if (threadIdx.x == 0 && p.out_lse) p.out_lse[th] = lse;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeTiledFn* out) {
  static std::atomic<EncodeTiledFn> cached{nullptr};   // looked up once; callers may be on several threads
  EncodeTiledFn fn = cached.load(std::memory_order_acquire);
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || ptr == nullptr) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeTiledFn>(ptr);
    cached.store(fn, std::memory_order_release);
  }
  *out = fn;
  return cudaSuccess;
}

// The pool as {128 bytes, 8 rows, 4 column blocks, row groups, pages}; box of
// `chunk` rows.  The call's checks make the base 16-byte aligned, every stride a
// multiple of 16 under 2^40 and page_size a multiple of 8.
cudaError_t encode_cache_map(CUtensorMap* map, const CacheView& c, int chunk) {
  EncodeTiledFn fn = nullptr;
  cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[5] = {128, 8, 4, (cuuint64_t)c.page_size / 8, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)c.row_stride, 128, (cuuint64_t)(8 * c.row_stride), (cuuint64_t)c.page_stride};
  const cuuint32_t box[5] = {128, 8, 4, (cuuint32_t)chunk / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, c.rows, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The output as [T, H, 512]; box of 64 dims x 64 heads of a token (heads past H are not written).
cudaError_t encode_out_map(CUtensorMap* map, const WindowParams& p) {
  EncodeTiledFn fn = nullptr;
  cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)p.H, (cuuint64_t)p.c.sum_q};
  const cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)p.H * kHeadDim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)kNH, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.out, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

namespace {

template <int kMode>
cudaError_t launch_window_kernel(const KernelParams& kp, unsigned grid, int shift, cudaStream_t stream) {
  auto launch = [&](auto kernel) -> cudaError_t {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (err != cudaSuccess) return err;
    return launch_overlapped(kernel, dim3(grid), kThreads, kSmemBytes, stream, kp);
  };
  if (shift == 5) return launch(window_kernel<5, kMode>);
  if (shift == 4) return launch(window_kernel<4, kMode>);
  return launch(window_kernel<3, kMode>);
}

}  // namespace

// plan: its groups, or nullptr for the window attention.
cudaError_t launch_pair_attention(const WindowParams& p, const PrefixPlan* plan, int sms, cudaStream_t stream) {
  KernelParams kp = {};
  kp.p = p;
  if (plan != nullptr) kp.plan = *plan;
  kp.groups = (p.H + kNH - 1) / kNH;
  const int pairs = (int)((int64_t)p.c.sum_q * kp.groups);
  kp.units = p.whole + (pairs - p.whole) * p.num_splits;
  const int shift = cache_box_shift(p.c.page_size);
  cudaError_t e = encode_cache_map(&kp.map, p.c, 1 << shift);
  if (e == cudaSuccess && p.whole > 0) e = encode_out_map(&kp.out_map, p);   // (partials are stored by threads)
  if (e != cudaSuccess) return e;
  const bool parts = pairs > p.whole;
  const unsigned grid = (unsigned)std::min(kp.units, sms);
  if (plan == nullptr)
    e = parts ? launch_window_kernel<kSplitPairs>(kp, grid, shift, stream) : launch_window_kernel<kPairs>(kp, grid, shift, stream);
  else
    e = parts ? launch_window_kernel<kGroupedSplitPairs>(kp, grid, shift, stream)
              : launch_window_kernel<kGroupedPairs>(kp, grid, shift, stream);
  if (e != cudaSuccess || !parts) return e;
  const dim3 heads((unsigned)((pairs - p.whole) * (int64_t)kNH));
  if (p.num_splits > 8)                           // what one team loads at a time
    return launch_overlapped(window_merge_kernel<kMergeTeams>, heads, kMergeThreads * kMergeTeams, 0, stream, p, kp.groups);
  return launch_overlapped(window_merge_kernel<1>, heads, kMergeThreads, 0, stream, p, kp.groups);
}

cudaError_t launch_planned_attention(const WindowParams& p, const PrefixPlan& plan, cudaStream_t stream) {
  KernelParams kp = {};
  kp.p = p;
  kp.plan = plan;
  kp.groups = (p.H + kNH - 1) / kNH;
  kp.units = 0;
  const int shift = cache_box_shift(p.c.page_size);
  cudaError_t e = encode_cache_map(&kp.map, p.c, 1 << shift);
  if (e == cudaSuccess) e = encode_out_map(&kp.out_map, p);
  if (e != cudaSuccess) return e;
  return launch_window_kernel<kPlanned>(kp, (unsigned)plan.shares, shift, stream);
}

}  // namespace smla
