// Shared definitions of the paged latent cache: kernel-side copies of the
// argument structs (strides already defaulted) and the launchers.
#pragma once

#include "common.cuh"

namespace smla {

struct CacheView {
  uint8_t* rows;
  int64_t row_stride, page_stride;     // bytes
  float* scales;
  int64_t scale_stride;                // elements
  int32_t num_pages, page_size, block_rows;
  const int32_t* bt;
  int64_t bt_stride;
  int32_t max_pages, batch;
  const int32_t* seq_lens;
  const int32_t* cum;                  // nullptr: uniform
  int32_t sum_q;
};

// The calls of a step follow one another on a stream, most of them short, so each
// kernel is launched while the one before it ends (programmatic dependent
// launch): it waits for all of that one's writes before it reads anything, and
// lets the next come as soon as it runs itself.
__device__ __forceinline__ void await_prior_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void admit_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A load of what a kernel before may have written.  Not by the read-only path,
// which holds its lines for a kernel's whole life: that began before those writes.
template <class T>
__device__ __forceinline__ T fetch(const T* p) {
  return *p;
}
__device__ __forceinline__ float fetch_scale(float value, const float* dev) { return dev != nullptr ? fetch(dev) : value; }

template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Request b's new tokens: [first, first + count) of the flattened batch.
__device__ __forceinline__ void request_tokens(const CacheView& c, int b, int* first, int* count) {
  if (c.cum != nullptr) {
    *first = fetch(c.cum + b);
    *count = fetch(c.cum + b + 1) - *first;
  } else {
    const int q = c.sum_q / c.batch;
    *first = b * q;
    *count = q;
  }
}

// The last request b of `batch` for which before(b) holds (before(0) is taken to;
// it holds up to some b and not behind it).  Whole warp, 32 requests looked at at
// a time, so that a batch of a thousand costs two trips to L2.
template <class F>
__device__ __forceinline__ int last_request(int batch, int lane, F before) {
  int lo = 0, n = batch - 1;                        // the answer is among lo .. lo + n
  while (n > 0) {
    const int step = (n + 31) / 32;
    const uint32_t miss = ~__ballot_sync(0xffffffffu, before(lo + min(n, (lane + 1) * step)));
    if (miss == 0) return lo + n;                   // (the last lanes look at lo + n)
    const int hits = __ffs(miss) - 1;               // the first miss, not a count: in range for offsets that fall, too
    lo += hits * step;
    n = min(n - hits * step, step - 1);             // lo + step is known to be behind it
  }
  return lo;
}

constexpr int kWindowHeads = 64;      // heads of one token that a CTA takes
constexpr int kWindowTile = 128;      // cache rows of one tile

struct WindowParams {
  CacheView c;
  int32_t H, window, first_tokens;
  int32_t whole, num_splits;   // (token, head group) pairs done whole, splits of each of the others
  const __nv_bfloat16* q;
  int64_t q_stride_token;
  const float* sinks;
  float bmm1, bmm2;
  const float* bmm1_dev;
  const float* bmm2_dev;
  __nv_bfloat16* out;
  float* out_lse;
  float* part_o;      // [pairs not whole, S, 64 heads, 512] fp32 normalised split partials
  float* part_lse;    // [pairs not whole, S, 64 heads] fp32 base-2 LSE of each
  int32_t* err;
};

constexpr int kMaxWindowSplits = 256;

// log2 of a TMA box's rows: the highest box that pages hold whole, up to a quarter
// of a tile (fewer copies to issue).
__host__ __device__ inline int cache_box_shift(int page_size) { return page_size % 32 == 0 ? 5 : page_size % 16 == 0 ? 4 : 3; }

// What a CTA works on at a time: 64 heads of a token, a range of tiles of its chunk list.
// In a plan, also 64 (token, head) rows of a group, and lists whose first chunks are
// another request's.
struct Unit {
  int t, h0, heads, part, b;                      // part: its partial's number, or -1 (it writes the output)
  int first_chunks, window_chunk, chunks;         // list: [0, first_chunks), then from window_chunk on
  int pos, lo;                                    // last and first visible position of the window
  int tile0, tiles;
  int b0, first;                                  // plan: the request of the list's first chunks, their rows
};

// Plan of a batch whose groups share prefixes, made on the device (prefix_attention.cu).
// Units are blocks of 64 (token, head) rows: those of the groups' shared prefixes,
// then those of the tokens, all laid end to end by cost and cut into a share for each
// SM.  Partials are numbered: two for each share (a block that its beginning, or
// only its end, cuts), then for shared prefixes and their tokens by unit and share.
constexpr int kPlanTile = 4, kPlanUnit = 9;       // cost of a tile; of a unit's query, sums and results
constexpr int kMaxShares = 256;
constexpr int kManyPieces = 16;
__host__ __device__ inline int64_t plan_cost(int tiles) { return kPlanUnit + (int64_t)(tiles > 0 ? tiles : 1) * kPlanTile; }
struct PrefixPlan {
  int32_t groups, shares;
  const int32_t* group_starts;          // [groups + 1] first request of each
  const int32_t* prefix_lens;           // [groups]
  int64_t* share_cost;                  // [1]
  uint64_t* share_by;                   // [1] 2^64 / share_cost, rounded up
  int32_t* many;                        // [1] a block may be in more than kManyPieces shares
  int64_t* cost_of;                     // [groups + T + 1] where a group's prefix, a token begins
  int32_t* unit_of;                     // [groups + T + 1] its first unit
  int32_t* shared_of;                   // [groups + T] the units of shared prefixes and their tokens before it
  int4* share;                          // [shares] first unit, units, the first one's segment
  int4* first;                          // [shares][4] the first unit
  int4* group;                          // [groups] first request with tokens, its first token, (token, head) rows, prefix (0: not shared)
  int4* token;                          // [T] request, the one that holds its prefix (or sign and group: shared), position, prefix
  int4* prefix_of;                      // [T] of a shared prefix: cost_of (two words), shared_of, the token's first row in it
  int32_t* limit;                       // [groups] positions that all the group's tokens see (where groups are many)
  int32_t* lead;                        // [groups] its first request with tokens
};

// Unit `unit`, of `segment`, as far as it is share `share`'s; later: not the share's
// first one.  (The arrays are given apart, as the plan's kernel has them in shared memory.)
__device__ __forceinline__ Unit plan_unit(const CacheView& c, const PrefixPlan& plan, int H, int shift, int share,
                                          int64_t share_cost, int unit, int segment, bool later, const int64_t* cost_of,
                                          const int* unit_of, const int* shared_of, const int4* group, const int4* token) {
  const int block = unit - fetch(unit_of + segment), shared = fetch(shared_of + segment);
  int64_t at = fetch(cost_of + segment);
  Unit u;
  u.h0 = block * kWindowHeads;
  bool partial = true;
  if (segment < plan.groups) {                    // a group's prefix
    const int4 g = fetch(group + segment);
    const int row = g.y * H + u.h0;
    u.heads = min(kWindowHeads, g.z - u.h0);
    u.t = row / H;
    u.h0 = row - u.t * H;
    u.b = u.b0 = g.x;
    u.first = g.w;
    u.pos = -1;
    u.lo = 0;
  } else {
    const int4 r = fetch(token + (segment - plan.groups));
    partial = r.y < 0;
    u.t = segment - plan.groups;
    u.heads = min(kWindowHeads, H - u.h0);
    u.b = r.x;
    u.b0 = partial ? r.x : r.y;
    u.first = partial ? 0 : r.w;                  // (a shared prefix is its group's)
    u.pos = r.z;
    u.lo = r.w;
  }
  const int last = min(u.pos, c.max_pages * c.page_size - 1);
  u.first_chunks = (u.first + (1 << shift) - 1) >> shift;
  u.window_chunk = u.lo >> shift;
  u.chunks = u.first_chunks + (last >= u.lo ? (last >> shift) - u.window_chunk + 1 : 0);
  const int tiles = (u.chunks + (kWindowTile >> shift) - 1) >> (7 - shift);
  at += block * plan_cost(tiles) + kPlanUnit;     // where its first tile begins
  auto from = [&](int s) {                        // its first tile that begins in share s or behind it
    return (int)min(max((s * share_cost - at + kPlanTile - 1) / kPlanTile, (int64_t)0), (int64_t)tiles);
  };
  u.tile0 = from(share);
  u.tiles = from(share + 1) - u.tile0;
  u.part = partial ? 2 * plan.shares + shared + block + share : u.tiles < tiles ? 2 * share + later : -1;
  return u;
}

cudaError_t launch_planned_attention(const WindowParams& p, const PrefixPlan& plan, cudaStream_t stream);
cudaError_t launch_prefix_attention(const WindowParams& p, const PrefixPlan& plan, cudaStream_t stream);

struct PrefixPlan;
cudaError_t launch_pair_attention(const WindowParams& p, const PrefixPlan* plan, int sms, cudaStream_t stream);

struct AppendParams {
  CacheView c;
  const __nv_bfloat16* latent;
  int64_t latent_stride;
  int32_t* err;
};

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);

struct PagesParams {
  int32_t* bt;
  int64_t bt_stride;
  int32_t rows, max_pages, page_size, num_pages;
  int32_t* refs;
  const int32_t* lens;
  const int32_t* new_lens;
  const int32_t* parents;
  int32_t* out_lens;
  int32_t* move_src;
  int32_t* move_dst;
  int32_t* move_count;
  int32_t* ws;
  int32_t* err;
};

// Workspace words of resize and compact: a header, per-row words (resize),
// per-page words, a count per 512 pages.
constexpr int kPagesHeader = 64;
inline int64_t pages_workspace_words(int64_t rows, int64_t num_pages) {
  return kPagesHeader + 2 * rows + num_pages + (num_pages + 511) / 512;
}

cudaError_t launch_pages_resize(const PagesParams& p, int sms, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_pages_reorder(const PagesParams& p, int sms, cudaStream_t stream);
cudaError_t launch_pages_shared_prefix(const PagesParams& p, const int32_t* group_starts, int num_groups, int32_t* prefix_lens,
                                       cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t stream);

constexpr int kCopyPools = 64;        // pools of one copy launch (kernel parameters)
struct CopyParams {
  struct Pool {
    uint8_t* base;
    int64_t stride;
    int32_t pieces;                   // pieces of `vec` bytes in a page
    int32_t vec;                      // 16, 4 or 1: what base, stride and page size share
  } pool[kCopyPools];
  int32_t num_pools, num_pages;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int32_t capacity;
  int32_t* err;
};
cudaError_t launch_pages_copy(const CopyParams& p, int sms, cudaStream_t stream);

}  // namespace smla
