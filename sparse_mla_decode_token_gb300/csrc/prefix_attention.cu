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
// prefix through the table of the group's first request.
//
// The lengths are on the device, so the plan is made there: one CTA finds each
// group's prefix, chooses the tiles of a piece out of 32 candidates (a warp each;
// a turn of the SMs costs its largest pieces and 2.8 tiles' time for each unit's
// query, sums and results) and numbers the units.
#include <algorithm>

#include "cache.cuh"
#include "cache_ptx.cuh"
#include "tc_common.cuh"

namespace smla {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr float kUnitTiles = 2.8f;                // what a unit costs beside its tiles, in tiles
constexpr int kMaxPieces = 480;                   // of one list

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

// The group of request b, or -1 (starts in order).
__device__ __forceinline__ int group_of(const PrefixPlan& plan, int b) {
  int lo = -1, hi = plan.groups - 1;              // the last group that begins at or before b
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (fetch(plan.group_starts + mid) <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo >= 0 && b < fetch(plan.group_starts + lo + 1) ? lo : -1;
}

struct Request {
  int first, count, len;                          // its tokens in the batch, all of them; its length
  int t0, t1;                                     // those that the batch holds
};
__device__ __forceinline__ Request request_of(const CacheView& c, int b) {
  Request r;
  request_tokens(c, b, &r.first, &r.count);
  r.len = fetch(c.seq_lens + b);
  r.t0 = min(max(r.first, 0), c.sum_q);
  r.t1 = r.count > 0 ? min(max(r.first + r.count, r.t0), c.sum_q) : r.t0;
  return r;
}

__global__ void __launch_bounds__(kThreads) prefix_plan_kernel(const WindowParams p, const PrefixPlan plan, int shift, int sms) {
  __shared__ float s_cost[kWarps];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int s_most, s_pieces;
  const CacheView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = blocks_of(p.H), cap = c.max_pages * c.page_size, T = c.sum_q;
  await_prior_kernel();
  admit_next_kernel();

  // what is out of order shares nothing
  bool bad = false, unordered = false;
  for (int g = threadIdx.x; g < plan.groups; g += kThreads) {
    const int lo = fetch(plan.group_starts + g), hi = fetch(plan.group_starts + g + 1);
    bad |= lo < 0 || hi < lo || hi > c.batch;
    plan.limit[g] = 0x7fffffff;
  }
  if (c.cum != nullptr)
    for (int b = threadIdx.x; b < c.batch; b += kThreads) unordered |= fetch(c.cum + b) > fetch(c.cum + b + 1);
  for (int t = threadIdx.x; t < T; t += kThreads) plan.token[t] = make_int4(-1, 0, -1, 0);
  if (threadIdx.x == 0) s_most = s_pieces = 0;
  if (bad) flag(p.err, SMLA_DEVERR_PAGE_STATE);
  bad = __syncthreads_or(bad);
  unordered = __syncthreads_or(unordered);
  const int groups = bad || unordered ? 0 : plan.groups;

  // the positions that all of a group's tokens see
  for (int b = threadIdx.x; b < c.batch && groups > 0; b += kThreads) {
    const Request r = request_of(c, b);
    const int g = r.t1 > r.t0 ? group_of(plan, b) : -1;
    if (g >= 0) atomicMin(plan.limit + g, max(0, r.len - r.count + 1));
  }
  __syncthreads();
  for (int g = threadIdx.x; g < plan.groups; g += kThreads) {
    int4 v = make_int4(0, 0, 0, 0);
    int prefix = 0;
    if (groups > 0) {
      const int lo = fetch(plan.group_starts + g), hi = fetch(plan.group_starts + g + 1);
      const int limit = __ldcg(plan.limit + g);
      if (limit != 0x7fffffff) {
        prefix = min(min(max(fetch(plan.prefix_lens + g), 0), limit), cap);
        int t0 = lo * (T / c.batch), t1 = hi * (T / c.batch);
        if (c.cum != nullptr) t0 = fetch(c.cum + lo), t1 = fetch(c.cum + hi);
        t0 = min(max(t0, 0), T), t1 = min(max(t1, t0), T);
        const int tiles = tiles_of(prefix, 0, -1, cap, shift), blocks = blocks_of((t1 - t0) * p.H);
        v = make_int4(lo, t0, (t1 - t0) * p.H, 0);
        if ((int64_t)((t1 - t0) * heads - blocks) * tiles > 3 * (int64_t)blocks) {
          v.w = prefix;
          atomicMax(&s_most, tiles);
        }
      }
    }
    plan.group[g] = v;
    plan.limit[g] = prefix;
  }
  __syncthreads();

  // the requests and their tokens
  for (int base = 0; base < c.batch; base += kThreads) {
    const int b = base + threadIdx.x;
    Request r = {0, 0, 0, 0, 0};
    int g = -1, prefix = 0, from = 0;
    if (b < c.batch) {
      r = request_of(c, b);
      if (r.t1 > r.t0) {
        g = groups > 0 ? group_of(plan, b) : -1;
        prefix = g >= 0 ? __ldcg(plan.limit + g) : 0;
        const int4 v = g >= 0 ? __ldcg(plan.group + g) : make_int4(b, 0, 0, 0);
        from = v.w > 0 ? v.x | (int)0x80000000 : v.x;
      }
      const int tiles = tiles_of(from < 0 ? 0 : prefix, prefix, r.len - r.count + (r.t1 - 1 - r.first), cap, shift);
      plan.request[b] = make_int4(r.t1 - r.t0, r.t1 > r.t0 ? tiles : 0, g, from);
      if (r.t1 > r.t0) atomicMax(&s_most, tiles);
    }
    const int pos0 = r.len - r.count - r.first;
    const bool many = r.t1 - r.t0 > 8;
    if (!many)
      for (int t = r.t0; t < r.t1; ++t) plan.token[t] = make_int4(b, from, pos0 + t, prefix);
    for (uint32_t left = __ballot_sync(0xffffffffu, many); left != 0; left &= left - 1) {
      const int from_lane = __ffs(left) - 1;
      const int t0 = __shfl_sync(0xffffffffu, r.t0, from_lane), t1 = __shfl_sync(0xffffffffu, r.t1, from_lane);
      const int4 v = make_int4(__shfl_sync(0xffffffffu, b, from_lane), __shfl_sync(0xffffffffu, from, from_lane),
                               __shfl_sync(0xffffffffu, pos0, from_lane), __shfl_sync(0xffffffffu, prefix, from_lane));
      for (int t = t0 + lane; t < t1; t += 32) plan.token[t] = make_int4(v.x, v.y, v.z + t, v.w);
    }
  }
  __syncthreads();

  // the tiles of a piece: candidate `warp`, from the fewest to all of the longest list
  const int most = max(s_most, 1), least = (most + kMaxPieces - 1) / kMaxPieces;
  auto candidate = [&](int i) {
    if (i == kWarps - 1) return most;
    const int v = (int)ceilf(exp2f(log2f((float)most) * ((float)i / (kWarps - 1))));
    return min(max(v, least), most);
  };
  {
    const int per = candidate(warp);
    float units1 = 0, tiles1 = 0, units2 = 0, tiles2 = 0, rows = 0;
    int64_t parts = 0;
    for (int g = lane; g < groups; g += 32) {
      const int4 v = __ldcg(plan.group + g);
      if (v.w == 0) continue;
      const int blocks = blocks_of(v.z), tiles = tiles_of(v.w, 0, -1, cap, shift), pieces = (tiles + per - 1) / per;
      units1 += (float)blocks * pieces;
      tiles1 += (float)blocks * tiles;
      rows += (float)v.z * pieces;
      parts += (int64_t)blocks * pieces;
    }
    for (int b = lane; b < c.batch; b += 32) {
      const int4 v = __ldcg(plan.request + b);
      const int pieces = (v.y + per - 1) / per;
      units2 += (float)v.x * heads * max(pieces, 1);
      tiles2 += (float)v.x * heads * v.y;
      if (pieces > 1 || v.w < 0) {
        rows += (float)v.x * p.H * pieces;
        parts += (int64_t)v.x * heads * pieces;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      units1 += __shfl_xor_sync(0xffffffffu, units1, o);
      tiles1 += __shfl_xor_sync(0xffffffffu, tiles1, o);
      units2 += __shfl_xor_sync(0xffffffffu, units2, o);
      tiles2 += __shfl_xor_sync(0xffffffffu, tiles2, o);
      rows += __shfl_xor_sync(0xffffffffu, rows, o);
      parts += __shfl_xor_sync(0xffffffffu, parts, o);
    }
    // turns of the prefixes' pieces, then those of the tokens' that do not fit beside the last of them
    const float turns = ceilf(units1 / sms), rest = fmaxf(0.f, units2 - (turns * sms - units1));
    float cost = turns * (tiles1 / fmaxf(units1, 1.f) + kUnitTiles) +
                 ceilf(rest / sms) * (tiles2 / fmaxf(units2, 1.f) + kUnitTiles) + rows / 7000.f + (rows > 0 ? 1.3f : 0.f);
    if (parts > plan.max_parts || (unordered && warp < kWarps - 1)) cost = INFINITY;
    if (lane == 0) s_cost[warp] = cost;
  }
  __syncthreads();
  int pick = kWarps - 1;
  for (int i = kWarps - 2; i >= 0; --i)
    if (s_cost[i] < s_cost[pick]) pick = i;
  const int per = candidate(pick);

  // the units' numbers: partial ones in the low word, whole ones in the high one
  int64_t before = 0;
  for (int base = 0; base < plan.groups + T; base += kThreads) {
    const int s = base + threadIdx.x;
    int64_t n = 0;
    int pieces = 0;
    if (s < plan.groups) {
      const int4 v = __ldcg(plan.group + s);
      if (v.w > 0) {
        pieces = (tiles_of(v.w, 0, -1, cap, shift) + per - 1) / per;
        n = (int64_t)blocks_of(v.z) * pieces;
      }
    } else if (s < plan.groups + T) {
      const int4 v = __ldcg(plan.token + (s - plan.groups));
      if (v.x >= 0) {
        const int tiles = tiles_of(v.y < 0 ? 0 : v.w, v.w, v.z, cap, shift);
        pieces = (tiles + per - 1) / per;
        if (v.y < 0 || pieces > 1) n = (int64_t)heads * pieces;
        else n = (int64_t)heads << 32;
      }
    }
    if (pieces > 0) atomicMax(&s_pieces, pieces);
    int64_t sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += x;
    }
    if (lane == 31) s_scan[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      int64_t all = s_scan[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, all, d);
        if (lane >= d) all += x;
      }
      s_scan[lane] = all;
    }
    __syncthreads();
    const int64_t at = before + sum - n + (warp > 0 ? s_scan[warp - 1] : 0);
    if (s < plan.groups + T) {
      plan.part_of[s] = (int)(at & 0xffffffff);
      if (s >= plan.groups) plan.whole_of[s - plan.groups] = (int)(at >> 32);
    }
    before += s_scan[kWarps - 1];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int parts = (int)(before & 0xffffffff), whole = (int)(before >> 32);
    plan.part_of[plan.groups + T] = parts;
    plan.whole_of[T] = whole;
    plan.header[kPlanPer] = per;
    plan.header[kPlanParts] = parts;
    plan.header[kPlanUnits] = parts + whole;
    plan.header[kPlanPieces] = s_pieces;
  }
}

// ------------------------------------------------------------------- merge
// Weights 2^(LSE_s - LSE) of a head's partials, then the sink and bmm2.  A warp a
// head, 16 dims a lane, where no list has more than kFew pieces; else the eight
// warps of a CTA share a head's partials.
constexpr int kMergeWarps = 8;
constexpr int kFew = 16;

struct Partials {
  int prefix, stride, prefixes;                   // first partial of the prefix, partials between its pieces, pieces
  int own, own_stride, owns;                      // the same of the token
  int prefix_row, own_row;                        // the head's row of each
};

__device__ __forceinline__ int64_t partial_row(const Partials& q, int s) {
  return s < q.prefixes ? (int64_t)(q.prefix + s * q.stride) * kWindowHeads + q.prefix_row
                        : (int64_t)(q.own + (s - q.prefixes) * q.own_stride) * kWindowHeads + q.own_row;
}

__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const WindowParams p, const PrefixPlan plan) {
  __shared__ float s_weight[kMergeWarps][2 * kFew];
  __shared__ float s_all[2 * kMaxPieces + 2];
  __shared__ float4 s_share[kMergeWarps][kHeadDim / 4];
  __shared__ float s_top[kMergeWarps], s_sum[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = blocks_of(p.H), T = p.c.sum_q;
  await_prior_kernel();
  admit_next_kernel();
  if (__ldcg(plan.header + kPlanParts) == 0) return;
  const bool few = __ldcg(plan.header + kPlanPieces) <= kFew;
  const int per = __ldcg(plan.header + kPlanPer), shift = cache_box_shift(p.c.page_size), cap = p.c.max_pages * p.c.page_size;
  const int each = few ? kMergeWarps : 1, items = (p.H + each - 1) / each;      // heads of a CTA, of a token
  for (int64_t i = blockIdx.x; i < (int64_t)T * items; i += gridDim.x) {
    const int t = (int)(i / items), h = (int)(i - (int64_t)t * items) * each + (few ? warp : 0);
    const int4 v = __ldcg(plan.token + t);
    if (v.x < 0) continue;
    Partials q;
    q.own = __ldcg(plan.part_of + plan.groups + t);
    q.own_stride = heads;
    q.owns = (__ldcg(plan.part_of + plan.groups + t + 1) - q.own) / heads;
    q.own_row = h % kWindowHeads;
    q.own += h / kWindowHeads;
    q.prefix = q.stride = q.prefixes = q.prefix_row = 0;
    if (v.y < 0) {
      const int g = __ldcg(plan.request + v.x).z;
      const int4 w = __ldcg(plan.group + g);
      const int row = (t - w.y) * p.H + h;
      q.prefix = __ldcg(plan.part_of + g) + row / kWindowHeads;
      q.stride = blocks_of(w.z);
      q.prefixes = (tiles_of(w.w, 0, -1, cap, shift) + per - 1) / per;
      q.prefix_row = row % kWindowHeads;
    }
    const int n = q.prefixes + q.owns;
    if (n == 0) continue;
    if (few && h >= p.H) continue;
    const int first = few ? lane : (int)threadIdx.x, step = few ? 32 : kMergeWarps * 32;
    float* const weight = few ? s_weight[warp] : s_all;
    float top = -INFINITY, sum = 0.f;
    bool nan = false;
    for (int s = first; s < n; s += step) {
      const float l = __ldcg(p.part_lse + partial_row(q, s));
      weight[s] = l;
      nan |= isnan(l);
      top = fmaxf(top, l);
    }
    top = ptx::warp_max(top);
    if (few) {
      nan = __any_sync(0xffffffffu, nan);
    } else {
      if (lane == 0) s_top[warp] = top;
      nan = __syncthreads_or(nan);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, s_top[w]);
    }
    for (int s = first; s < n; s += step) {
      const float w = weight[s] == -INFINITY ? 0.f : fast_exp2(weight[s] - top);
      weight[s] = w;
      sum += w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (few) {
      __syncwarp();
    } else {
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) sum += s_sum[w];
    }
    float4 acc[4] = {};
#pragma unroll 2
    for (int s = few ? 0 : warp; s < n; s += few ? 1 : kMergeWarps) {
      const float w = weight[s];
      if (w == 0.f) continue;                     // an empty partial is not written
      const float4* o = reinterpret_cast<const float4*>(p.part_o + partial_row(q, s) * kHeadDim) + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 x = __ldcg(o + 32 * k);
        acc[k].x = fmaf(w, x.x, acc[k].x), acc[k].y = fmaf(w, x.y, acc[k].y);
        acc[k].z = fmaf(w, x.z, acc[k].z), acc[k].w = fmaf(w, x.w, acc[k].w);
      }
    }
    float lse = -INFINITY, f = 0.f;
    if (top != -INFINITY || nan) {
      lse = nan ? NAN : top + fast_log2(sum);
      f = fetch_scale(p.bmm2, p.bmm2_dev) / sum;
      if (p.sinks != nullptr) f *= 1.f / (1.f + fast_exp2(fetch(p.sinks + h) * kLog2e - lse));
    }
    const int64_t th = (int64_t)t * p.H + h;
    if (!few) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s_share[warp][lane + 32 * k] = acc[k];
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
      if (threadIdx.x == 0 && p.out_lse) p.out_lse[th] = lse;
      __syncthreads();
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint2*>(p.out + th * kHeadDim + (lane + 32 * k) * 4) =
            make_uint2(tc::pack_bf16x2(acc[k].x * f, acc[k].y * f), tc::pack_bf16x2(acc[k].z * f, acc[k].w * f));
      if (lane == 0 && p.out_lse) p.out_lse[th] = lse;
      __syncwarp();
    }
  }
}

}  // namespace

cudaError_t launch_prefix_attention(const WindowParams& p, const PrefixPlan& plan, int sms, cudaStream_t stream) {
  cudaError_t e = launch_overlapped(prefix_plan_kernel, dim3(1), kThreads, 0, stream, p, plan, cache_box_shift(p.c.page_size), sms);
  if (e == cudaSuccess) e = launch_planned_attention(p, plan, sms, stream);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.c.sum_q * p.H;
  return launch_overlapped(prefix_merge_kernel, dim3((unsigned)std::min<int64_t>(rows, (int64_t)sms * 8)), kMergeWarps * 32, 0,
                           stream, p, plan);
}

}  // namespace smla
