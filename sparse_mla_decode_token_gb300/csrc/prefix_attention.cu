// Attention of a batch whose groups share long prefixes of the paged latent cache:
// the plan of its work, made on the device, and the merge of its partial results.
// What computes is the window attention's kernel (window_attention.cu, kPlanned).
//
// That kernel multiplies a tile of 128 cache rows with 64 queries.  A token of H
// heads fills H of them; the tokens of a group fill them together, wherever they
// stand, as every row of the prefix is seen by all.  So a group's prefix is worked
// through ceil(tokens * H / 64) times, not tokens * ceil(H / 64) times, and what
// each token has behind it by itself; softmax partials (normalised O, LSE) of both
// are merged per head.
//
// A group is split so where it saves tiles: with heads in multiples of 64, or one
// token, there is nothing to save, and its tokens go through one list of rows, the
// prefix through the table of the first request of the group that has new tokens.
// Where a call can save little in all, there is no plan: its tokens are the window
// attention's pairs, with such lists (kGroupedPairs; cache_api.cu chooses).
//
// The lengths are on the device, so the plan is made there, by one CTA.  Each block
// of 64 rows costs 2.25 tiles' time for its query, sums and results and one for each
// tile; all blocks laid end to end are cut into equal shares, one for each SM (a
// tile is the CTA's in whose share it begins).  A block that a cut goes through is
// given in pieces and merged.
//
// What bounds it: the tile's chain in the kernel (window_attention.cu; 2.4 us a tile, its
// tensor instructions 1.37), 8 us to a CTA's first scores and 4 of results, and before
// and behind it the plan (4.5 us: trips to L2 and barriers of one CTA; with 1024 threads
// 6) and the merge (3.5 us: four trips). Measured on a GB300, replayed from a graph: 64
// samples of 16 heads behind 8 prompts of 4 to 8 thousand 43.6 us, 305 TFLOP/s; 128 beams
// of 8 heads behind 4 documents of 16 thousand 66.4 us, 516 TFLOP/s (each token by itself:
// 81.6 and 274).  As calls on other inputs each time: 47.2 and 71.6.  Without a plan: 4
// samples of 16 heads behind 510 tokens 14.0 us (22.8 with one); 160 tokens of 128 heads
// over 1000 to 2560 rows 113.5 us, 659 TFLOP/s (117).  (Pieces of one
// size, the best of 32 by a cost model, in turns of the SMs: 54.6, 78.4 and 168 us where
// shares took 46.7, 69.8 and 126.)
#include <algorithm>

#include "cache.cuh"
#include "cache_ptx.cuh"
#include "tc_common.cuh"

namespace smla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kNearGroups = 256, kNearSegments = 1024;   // of which the plan's arrays lie in shared memory

__device__ __forceinline__ void flag(int32_t* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}
__device__ __forceinline__ int blocks_of(int rows) { return (rows + kWindowHeads - 1) / kWindowHeads; }

// Tiles of the list of `first` rows of one request, then the positions lo .. pos of another.
__device__ __forceinline__ int tiles_of(int first, int lo, int pos, int cap, int shift) {
  const int last = min(pos, cap - 1);
  const int chunks = ((first + (1 << shift) - 1) >> shift) + (last >= lo ? (last >> shift) - (lo >> shift) + 1 : 0);
  return (chunks + (kWindowTile >> shift) - 1) >> (7 - shift);
}

// The last s of 0 .. n - 1 with before(s); -1 if there is none.
template <class F>
__device__ __forceinline__ int last_of(int n, F before) {
  int lo = -1, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before(mid)) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Request {
  int first, count, len;                          // its tokens in the batch, all of them; its length
  int t0, t1;                                     // those that the batch holds
};
__device__ __forceinline__ Request request_of(const CacheView& c, int b) {
  Request r;
  request_tokens(c, b, &r.first, &r.count);
  r.len = max(fetch(c.seq_lens + b), 0);          // (negative: none; what is subtracted from it stays an int)
  r.t0 = min(max(r.first, 0), c.sum_q);
  r.t1 = r.count > 0 ? min(max(r.first + r.count, r.t0), c.sum_q) : r.t0;
  return r;
}

// a and b become the sums of those of the threads before; *all_a, *all_b of all.
struct Scan {
  int64_t a[kWarps], b[kWarps];
};
__device__ __forceinline__ void scan(Scan& sh, int64_t& a, int64_t& b, int64_t* all_a, int64_t* all_b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t a0 = a, b0 = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) a += x, b += y;
  }
  if (lane == 31) sh.a[warp] = a, sh.b[warp] = b;
  __syncthreads();
  int64_t wa = lane < kWarps ? sh.a[lane] : 0, wb = lane < kWarps ? sh.b[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, wa, d), y = __shfl_up_sync(0xffffffffu, wb, d);
    if (lane >= d) wa += x, wb += y;
  }
  *all_a = __shfl_sync(0xffffffffu, wa, 31);
  *all_b = __shfl_sync(0xffffffffu, wb, 31);
  const int64_t before_a = __shfl_sync(0xffffffffu, wa, max(warp - 1, 0)), before_b = __shfl_sync(0xffffffffu, wb, max(warp - 1, 0));
  a += (warp > 0 ? before_a : 0) - a0;
  b += (warp > 0 ? before_b : 0) - b0;
  __syncthreads();
}

// at / share_cost: exact by multiplication where at * share_cost < 2^64 (`by` is 0 where that is not sure)
__device__ __forceinline__ int share_of(int64_t at, int64_t share_cost, uint64_t by) {
  return by != 0 ? (int)__umul64hi((uint64_t)at, by) : (int)(at / share_cost);
}

__global__ void __launch_bounds__(kThreads) prefix_plan_kernel(const WindowParams p, const PrefixPlan plan, int shift) {
  __shared__ int s_starts[kNearGroups + 1], s_limit[kNearGroups], s_lead[kNearGroups];
  __shared__ int4 s_group[kNearGroups];
  __shared__ int64_t s_cost[kNearSegments + 1];
  __shared__ int s_unit[kNearSegments + 1];
  __shared__ int4 s_token[kNearSegments];
  __shared__ int s_shared[kNearSegments];
  __shared__ int s_first[kMaxShares + 1], s_end[kMaxShares + 1], s_segment[kMaxShares + 1];
  __shared__ Scan s_scan;
  __shared__ int s_most;                          // tiles of the longest list
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31;
  const int sms = plan.shares, heads = blocks_of(p.H), cap = c.max_pages * c.page_size, T = c.sum_q, segments = plan.groups + T;
  await_prior_kernel();
  admit_next_kernel();
  const bool near = plan.groups <= kNearGroups;
  const int* const starts = near ? s_starts : plan.group_starts;
  int* const limit = near ? s_limit : plan.limit;
  int* const lead = near ? s_lead : plan.lead;

  // what is out of order shares nothing
  const bool near_segments = segments <= kNearSegments;
  int4* const token = near_segments ? s_token : plan.token;
  const int b0 = threadIdx.x, g0 = threadIdx.x;   // the thread's first request and group: looked up at once
  Request mine = {0, 0, 0, 0, 0};
  if (b0 < c.batch) mine = request_of(c, b0);
  const int prefix0 = g0 < plan.groups ? fetch(plan.prefix_lens + g0) : 0;
  bool bad = false, unordered = mine.count < 0;
  for (int g = threadIdx.x; g < plan.groups; g += kThreads) {
    const int lo = fetch(plan.group_starts + g), hi = fetch(plan.group_starts + g + 1);
    bad |= lo < 0 || hi < lo || hi > c.batch;
    limit[g] = lead[g] = 0x7fffffff;
    if (near) {
      s_starts[g] = lo;
      s_starts[g + 1] = hi;                       // (both threads that write it write the same)
    }
  }
  if (c.cum != nullptr)
    for (int b = b0 + kThreads; b < c.batch; b += kThreads) unordered |= fetch(c.cum + b) > fetch(c.cum + b + 1);
  for (int t = threadIdx.x; t < T; t += kThreads) token[t] = make_int4(-1, 0, -1, 0);
  if (bad) flag(p.err, SMLA_DEVERR_PAGE_STATE);
  if (threadIdx.x == 0) s_most = 1;
  const int groups = __syncthreads_or(bad || unordered) ? 0 : plan.groups;
  auto group_of = [&](int b) {
    const int g = last_of(groups, [&](int x) { return starts[x] <= b; });
    return g >= 0 && b < starts[g + 1] ? g : -1;
  };

  // the positions that all of a group's tokens see, and the first request that has any
  const int group0 = mine.t1 > mine.t0 ? group_of(b0) : -1;
  if (group0 >= 0) {
    atomicMin(limit + group0, max(0, mine.len - mine.count + 1));
    atomicMin(lead + group0, b0);
  }
  for (int b = b0 + kThreads; b < c.batch && groups > 0; b += kThreads) {
    const Request r = request_of(c, b);
    const int g = r.t1 > r.t0 ? group_of(b) : -1;
    if (g < 0) continue;
    atomicMin(limit + g, max(0, r.len - r.count + 1));
    atomicMin(lead + g, b);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < plan.groups; g += kThreads) {
    int4 v = make_int4(0, 0, 0, 0);
    int prefix = 0;
    if (groups > 0 && limit[g] != 0x7fffffff) {
      const int lo = starts[g], hi = starts[g + 1];
      prefix = min(min(max(g == g0 ? prefix0 : fetch(plan.prefix_lens + g), 0), limit[g]), cap);
      int t0 = lo * (T / c.batch), t1 = hi * (T / c.batch);
      if (c.cum != nullptr) t0 = fetch(c.cum + lo), t1 = fetch(c.cum + hi);
      t0 = min(max(t0, 0), T), t1 = min(max(t1, t0), T);
      const int tiles = tiles_of(prefix, 0, -1, cap, shift), blocks = blocks_of((t1 - t0) * p.H);
      v = make_int4(lead[g], t0, (t1 - t0) * p.H, 0);
      if ((int64_t)((t1 - t0) * heads - blocks) * tiles > 3 * (int64_t)blocks) {
        v.w = prefix;
      }
    }
    plan.group[g] = v;
    if (near) s_group[g] = v;
    limit[g] = prefix;
  }
  __syncthreads();
  const int4* const group = near ? s_group : plan.group;

  // the requests' tokens
  for (int base = 0; base < c.batch; base += kThreads) {
    const int b = base + threadIdx.x;
    Request r = mine;
    int g = group0, prefix = 0, from = 0;
    if (base > 0) {
      r = {0, 0, 0, 0, 0};
      if (b < c.batch) r = request_of(c, b);
      g = r.t1 > r.t0 ? group_of(b) : -1;
    }
    if (r.t1 > r.t0) {
      prefix = g >= 0 ? limit[g] : 0;
      const int4 v = g >= 0 ? group[g] : make_int4(b, 0, 0, 0);
      from = v.w > 0 ? g | (int)0x80000000 : v.x;
    }
    const int pos0 = r.len - r.count - r.first;
    const bool many = r.t1 - r.t0 > 8;
    if (!many)
      for (int t = r.t0; t < r.t1; ++t) token[t] = make_int4(b, from, pos0 + t, prefix);
    for (uint32_t left = __ballot_sync(0xffffffffu, many); left != 0; left &= left - 1) {
      const int at = __ffs(left) - 1;
      const int t0 = __shfl_sync(0xffffffffu, r.t0, at), t1 = __shfl_sync(0xffffffffu, r.t1, at);
      const int4 v = make_int4(__shfl_sync(0xffffffffu, b, at), __shfl_sync(0xffffffffu, from, at),
                               __shfl_sync(0xffffffffu, pos0, at), __shfl_sync(0xffffffffu, prefix, at));
      for (int t = t0 + lane; t < t1; t += 32) token[t] = make_int4(v.x, v.y, v.z + t, v.w);
    }
  }
  __syncthreads();

  // where the segments begin: in cost, in units (blocks of 64 rows), in units whose results are partial in any case
  int64_t* const cost_of = near_segments ? s_cost : plan.cost_of;
  int* const unit_of = near_segments ? s_unit : plan.unit_of;
  int* const shared_of = near_segments ? s_shared : plan.shared_of;
  int64_t cost0 = 0;
  int unit0 = 0, shared0 = 0;
  for (int base = 0; base < segments; base += kThreads) {
    const int s = base + threadIdx.x;
    int tiles = 0, units = 0;
    bool shared = false;
    if (s < plan.groups) {
      const int4 v = group[s];
      shared = v.w > 0;
      if (shared) {
        tiles = tiles_of(v.w, 0, -1, cap, shift);
        units = blocks_of(v.z);
      }
    } else if (s < segments) {
      const int4 v = token[s - plan.groups];
      if (near_segments) plan.token[s - plan.groups] = v;
      if (v.x >= 0) {
        if (v.z >= cap) flag(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);   // (here, as such a token may have no unit)
        shared = v.y < 0;
        tiles = tiles_of(shared ? 0 : v.w, v.w, v.z, cap, shift);
        units = shared && tiles == 0 ? 0 : heads;
      }
    }
    // (units and shared units in one word: both are under 2^31)
    int64_t cost = (int64_t)units * plan_cost(tiles), counts = units | (int64_t)(shared ? units : 0) << 32;
    if (units > 0) atomicMax(&s_most, tiles);
    int64_t all_cost, all_counts;
    scan(s_scan, cost, counts, &all_cost, &all_counts);
    if (s < segments) {
      const int unit = unit0 + (int)(counts & 0xffffffff);
      plan.cost_of[s] = cost_of[s] = cost0 + cost;
      plan.unit_of[s] = unit_of[s] = unit;
      plan.shared_of[s] = shared_of[s] = shared0 + (int)(counts >> 32);
    }
    cost0 += all_cost;
    unit0 += (int)(all_counts & 0xffffffff);
    shared0 += (int)(all_counts >> 32);
  }
  if (threadIdx.x == 0) {
    plan.cost_of[segments] = cost_of[segments] = cost0;
    plan.unit_of[segments] = unit_of[segments] = unit0;
  }
  __syncthreads();

  // the shares: the first unit that has a tile in share c or behind it, and the units that have one before it
  const int64_t share = max((cost0 + sms - 1) / sms, (int64_t)kPlanTile);
  for (int i = threadIdx.x; i <= sms; i += kThreads) {
    const int64_t x = i * share;
    int first = unit0, end = unit0, s = 0;
    if (x < cost0) {
      s = last_of(segments, [&](int k) { return cost_of[k] <= x; });
      const int units = unit_of[s + 1] - unit_of[s];
      const int64_t all = cost_of[s + 1] - cost_of[s], in_segment = x - cost_of[s];
      const int64_t each = all >> 31 == 0 ? (uint32_t)all / (uint32_t)units : all / units;
      const int block = all >> 31 == 0 ? (uint32_t)in_segment / (uint32_t)each : (int)(in_segment / each);
      const int64_t in = in_segment - block * each;              // into the block
      first = unit_of[s] + block + (in > each - kPlanTile);      // its last tile begins there
      end = unit_of[s] + block + (in > kPlanUnit);
      while (first >= unit_of[s + 1] && s + 1 < segments) ++s;   // (behind a segment's last unit)
    }
    s_first[i] = first;
    s_end[i] = end;
    s_segment[i] = s;
  }
  // what the merge needs of its group's prefix, for each token
  for (int t = threadIdx.x; t < T && groups > 0; t += kThreads) {
    const int4 v = token[t];
    if (v.x < 0 || v.y >= 0) continue;
    const int g = v.y & 0x7fffffff;
    const int64_t cost = cost_of[g];
    plan.prefix_of[t] = make_int4((int)(cost & 0xffffffff), (int)(cost >> 32), shared_of[g], (t - group[g].y) * p.H);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < sms; i += kThreads) {
    const int units = max(0, s_end[i + 1] - s_first[i]);
    plan.share[i] = make_int4(s_first[i], units, s_segment[i], 0);
    if (units == 0) continue;
    union {
      int4 words[4];
      Unit unit;
    } first;
    first.unit = plan_unit(c, plan, p.H, shift, i, share, s_first[i], s_segment[i], false, cost_of, unit_of, shared_of, group,
                           token);
#pragma unroll
    for (int k = 0; k < 4; ++k) plan.first[i * 4 + k] = first.words[k];
  }
  if (threadIdx.x == 0) {
    *plan.share_cost = share;
    *plan.many = (int64_t)s_most * kPlanTile / share + 2 > kManyPieces;
    *plan.share_by = cost0 >> 34 == 0 && share >> 29 == 0 ? ~0ull / (uint64_t)share + 1 : 0;
  }
}

// ------------------------------------------------------------------- merge
// Weights 2^(LSE_s - LSE) of a head's partials, then the sink and bmm2.  A warp a head,
// 16 dims a lane; where blocks may be in many shares, a CTA a head, its eight warps
// sharing the partials.  (A CTA a head always, four teams of threads to share its
// partials: 60 us more, for starting CTAs that find nothing to do.)
constexpr int kMergeWarps = 8;

// A head's partials: of the prefix, then of the token's own list; one for each share
// that the block has tiles in.
struct Partials {
  int prefix, prefixes, own, owns;                // number of the first one, how many
  int own_first, own_step;                        // own list: shift of its first one, step between them
  int prefix_row, own_row;                        // the head's row of each
};

__device__ __forceinline__ int64_t partial_row(const Partials& q, int s) {
  if (s < q.prefixes) return (int64_t)(q.prefix + s) * kWindowHeads + q.prefix_row;
  s -= q.prefixes;
  return (int64_t)(q.own + s * q.own_step + (s == 0 ? q.own_first : 0)) * kWindowHeads + q.own_row;
}

// Items: `each` heads of each token; then, for shares 1 and up, 2 * each heads of a block
// that the share's beginning cuts (the second share of the block merges it).
constexpr int kMergeCtas = 3;

struct MergeItem {
  int t, h0, heads, tiles, own, owns, own_first, own_step;
  int row0, prefix_tiles, shared;                 // row0 < 0: no prefix
  int64_t prefix_at;
};

// What the plan says of an item; `loaded` between its trips to L2 and the rest.  heads = 0: nothing to do.
template <class F>
__device__ __forceinline__ MergeItem merge_item(const WindowParams& p, const PrefixPlan& plan, int64_t item, int each, F loaded) {
  const int per_token = (p.H + each - 1) / each;
  const int64_t token_items = (int64_t)p.c.sum_q * per_token;
  const int shift = cache_box_shift(p.c.page_size), cap = p.c.max_pages * p.c.page_size;
  MergeItem m = {};
  m.row0 = -1;
  m.own_step = 1;
  if (item >= token_items) {
    const int per_share = kWindowHeads / (2 * each);
    const int cut = (int)(item - token_items), i = 1 + cut / per_share;
    const int4 mine = __ldcg(plan.share + i);
    const int before = __ldcg(plan.share + i - 1).x;
    if (mine.y == 0 || mine.z < plan.groups) return m;
    m.t = mine.z - plan.groups;
    const int4 v = __ldcg(plan.token + m.t);
    const int block = mine.x - __ldcg(plan.unit_of + mine.z);
    const int64_t cost = __ldcg(plan.cost_of + mine.z);
    const auto [share, by] = loaded();
    m.tiles = tiles_of(v.w, v.w, v.z, cap, shift);
    const int64_t at = cost + block * plan_cost(m.tiles) + kPlanUnit;
    if (v.y < 0 || at >= i * share || at < (i - 1) * share) return m;   // shared, or not its second one
    m.h0 = block * kWindowHeads + cut % per_share * 2 * each;
    m.heads = 2 * each;
    m.own = 2 * (i - 1);
    m.own_step = 2;
    m.own_first = before != mine.x;
    m.owns = share_of(at + (int64_t)(m.tiles - 1) * kPlanTile, share, by) - (i - 1) + 1;
  } else {
    m.t = (int)(item / per_token);
    m.h0 = (int)(item - (int64_t)m.t * per_token) * each;
    const int4 v = __ldcg(plan.token + m.t), w = __ldcg(plan.prefix_of + m.t);
    const int64_t cost = __ldcg(plan.cost_of + plan.groups + m.t);
    const int units = __ldcg(plan.shared_of + plan.groups + m.t);
    if (v.x < 0 || v.y >= 0) return m;
    const auto [share, by] = loaded();
    m.heads = each;
    m.tiles = tiles_of(0, v.w, v.z, cap, shift);
    if (m.tiles > 0) {
      const int block = m.h0 / kWindowHeads;      // (eight heads from a multiple of eight lie in one)
      const int64_t at = cost + block * plan_cost(m.tiles) + kPlanUnit;
      const int c0 = share_of(at, share, by);
      m.own = 2 * plan.shares + units + block + c0;
      m.owns = share_of(at + (int64_t)(m.tiles - 1) * kPlanTile, share, by) - c0 + 1;
    }
    m.row0 = w.w;
    m.shared = w.z;
    m.prefix_at = ((int64_t)w.y << 32 | (uint32_t)w.x) + kPlanUnit;
    m.prefix_tiles = tiles_of(v.w, 0, -1, cap, shift);
  }
  return m;
}

struct ShareCost {
  int64_t cost;
  uint64_t by;
};

__global__ void __launch_bounds__(kMergeWarps * 32, kMergeCtas) prefix_merge_kernel(const WindowParams p, const PrefixPlan plan) {
  __shared__ float4 s_share[kMergeWarps][kHeadDim / 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shares = plan.shares;
  await_prior_kernel();
  admit_next_kernel();
  const ShareCost cost = {__ldcg(plan.share_cost), __ldcg(plan.share_by)};
  const bool many = __ldcg(plan.many) != 0;
  const int64_t share = cost.cost;
  const uint64_t by = cost.by;
  const auto loaded = [&] { return cost; };
  const int each = many ? 1 : kMergeWarps;
  const int64_t items = (int64_t)p.c.sum_q * ((p.H + each - 1) / each) + (shares - 1) * (kWindowHeads / (2 * each));
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const MergeItem m = many ? merge_item(p, plan, item, 1, loaded) : merge_item(p, plan, item, kMergeWarps, loaded);
    if (m.heads == 0) continue;
    const auto head = [&](int h) {                // the partials of head h
      Partials q = {0, 0, m.own, m.owns, m.own_first, m.own_step, 0, h % kWindowHeads};
      if (m.row0 >= 0) {
        const int row = m.row0 + h, block = row / kWindowHeads;
        const int64_t at = m.prefix_at + block * plan_cost(m.prefix_tiles);
        const int c0 = share_of(at, share, by);
        q.prefix = 2 * shares + m.shared + block + c0;
        q.prefixes = share_of(at + (int64_t)(m.prefix_tiles - 1) * kPlanTile, share, by) - c0 + 1;
        q.prefix_row = row % kWindowHeads;
      }
      return q;
    };
    for (int h = m.h0 + (many ? 0 : warp); h < min(m.h0 + m.heads, p.H); h += many ? 1 : kMergeWarps) {
      const Partials q = head(h);
      const int n = q.prefixes + q.owns;
      float top = -INFINITY, sum = 0.f;
      bool nan = false;
      for (int s = lane; s < n; s += 32) {
        const float l = fetch(p.part_lse + partial_row(q, s));
        nan |= isnan(l);
        top = fmaxf(top, l);
      }
      top = ptx::warp_max(top);
      nan = __any_sync(0xffffffffu, nan);
      float4 acc[4] = {};
      const int first = many ? warp : 0, step = many ? kMergeWarps : 1;
      for (int s0 = first; s0 < n; s0 += 32 * step) {
        // lane k's partial is s0 + k * step
        const int mine = s0 + lane * step;
        float w = 0.f;
        if (mine < n) {
          const float l = fetch(p.part_lse + partial_row(q, mine));
          w = l == -INFINITY ? 0.f : fast_exp2(l - top);
          sum += w;
        }
        const int here = min(32, (n - s0 + step - 1) / step);
#pragma unroll 1
        for (int k = 0; k < here; k += 2) {
          float weight[2];
          float4 o[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            weight[e] = __shfl_sync(0xffffffffu, w, (k + e) & 31);
            if (k + e >= here) weight[e] = 0.f;
            const float4* from = reinterpret_cast<const float4*>(p.part_o + partial_row(q, s0 + (k + e) * step) * kHeadDim) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {         // (an empty partial is not written)
              o[e][i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (weight[e] != 0.f) o[e][i] = __ldcg(from + 32 * i);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[i].x = fmaf(weight[e], o[e][i].x, acc[i].x), acc[i].y = fmaf(weight[e], o[e][i].y, acc[i].y);
              acc[i].z = fmaf(weight[e], o[e][i].z, acc[i].z), acc[i].w = fmaf(weight[e], o[e][i].w, acc[i].w);
            }
        }
      }
      if (many) {                                 // (each warp has the weights of its own partials)
        sum = 0.f;
        for (int s = lane; s < n; s += 32) {
          const float l = fetch(p.part_lse + partial_row(q, s));
          if (l != -INFINITY) sum += fast_exp2(l - top);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float lse = -INFINITY, f = 0.f;
      if (top != -INFINITY || nan) {
        lse = nan ? NAN : top + fast_log2(sum);
        f = fetch_scale(p.bmm2, p.bmm2_dev) / sum;
        if (p.sinks != nullptr) f *= 1.f / (1.f + fast_exp2(fetch(p.sinks + h) * kLog2e - lse));
      }
      const int64_t th = (int64_t)m.t * p.H + h;
      if (many) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s_share[warp][lane + 32 * i] = acc[i];
        __syncthreads();
        if (threadIdx.x < kHeadDim / 4) {
          float4 a = s_share[0][threadIdx.x];
#pragma unroll
          for (int w = 1; w < kMergeWarps; ++w) {
            const float4 x = s_share[w][threadIdx.x];
            a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
          }
          *reinterpret_cast<uint2*>(p.out + th * kHeadDim + threadIdx.x * 4) =
              make_uint2(tc::pack_bf16x2(a.x * f, a.y * f), tc::pack_bf16x2(a.z * f, a.w * f));
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint2*>(p.out + th * kHeadDim + (lane + 32 * i) * 4) =
              make_uint2(tc::pack_bf16x2(acc[i].x * f, acc[i].y * f), tc::pack_bf16x2(acc[i].z * f, acc[i].w * f));
      }
      if (lane == 0 && (!many || warp == 0) && p.out_lse) p.out_lse[th] = lse;
    }
  }
}

}  // namespace

cudaError_t launch_prefix_attention(const WindowParams& p, const PrefixPlan& plan, cudaStream_t stream) {
  cudaError_t e = launch_overlapped(prefix_plan_kernel, dim3(1), kThreads, 0, stream, p, plan, cache_box_shift(p.c.page_size));
  if (e == cudaSuccess) e = launch_planned_attention(p, plan, stream);
  if (e != cudaSuccess) return e;
  // (as many CTAs as the GPU holds at once, or as there may be heads)
  const int64_t items = (int64_t)p.c.sum_q * p.H + (int64_t)(plan.shares - 1) * (kWindowHeads / 2);
  return launch_overlapped(prefix_merge_kernel, dim3((unsigned)std::min<int64_t>(items, (int64_t)plan.shares * kMergeCtas)),
                           kMergeWarps * 32, 0, stream, p, plan);
}

}  // namespace smla
