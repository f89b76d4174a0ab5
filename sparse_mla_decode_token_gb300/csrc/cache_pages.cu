// Pages of the latent cache: growing, shrinking, forking and compacting the
// requests' page tables on the device, and copying pages.
//
// The state is a count per page (a page with count 0 is free) and a table row
// per request.  Ranking the free (or live) pages in order is a prefix sum over
// the counts, so every page's rank, hence who gets it, depends on nothing but
// the state.  Pages are counted in chunks of 512, a warp per chunk, the chunks
// dealt out to all warps in turn (those that hold the lowest free pages would
// otherwise be one CTA's); each CTA then sums the chunks' counts itself.
//
// A call is a few phases, each needing all of the one before.  Small calls run
// them in one launch, in one cluster of eight CTAs with cluster barriers between
// (resize of 128 requests x 128 pages in a pool of 16 thousand: 9.4 us; 10.9 with
// fences before the barriers, and with one CTA counting pages after summing the
// requests' needs); where tables and pool together pass kClusterEntries, eight
// SMs are too few and the phases are launches of their own over the whole GPU
// (resize, entries and pages together 34 thousand: 9.5 us in a cluster, 10.7 so; 67
// thousand 10.0 and 10.5; 132 thousand 12.3 and 11.3; 263 thousand 16.6 and 11.7; two
// million: 71 and 18.  Compaction crosses there too: 15.6 and 16.2, 19.9 and 16.4).
// What bounds both is latency: the counts (4 bytes a page) are read once, and
// again where pages are handed out; the rest is dependent trips to L2.
#include "cache.cuh"
#include "tc_ptx.cuh"

namespace smla {
namespace {

constexpr int kClusterCtas = 8;                       // portable cluster size
constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;
constexpr int64_t kClusterEntries = 1 << 17;           // table entries + pages that one cluster takes

__device__ __forceinline__ void flag(int32_t* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}

// Columns that `len` tokens hold; a length that cannot be is clamped, *bad set.
__device__ __forceinline__ int page_columns(const PagesParams& p, int len, bool* bad) {
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  if (len < 0 || len > cap) *bad = true;
  len = (int)min((int64_t)max(len, 0), cap);
  return len / p.page_size + (len % p.page_size != 0);
}
__device__ __forceinline__ int clamped_len(const PagesParams& p, int len) {
  return (int)min((int64_t)max(len, 0), (int64_t)p.max_pages * p.page_size);
}

__device__ __forceinline__ bool in_pool(const PagesParams& p, int page) { return page >= 0 && page < p.num_pages; }

// Drops one count of `page`; a count already at 0 stays there and is flagged.
__device__ __forceinline__ void drop_ref(const PagesParams& p, int page) {
  if (!in_pool(p, page)) {
    flag(p.err, SMLA_DEVERR_PAGE_STATE);
    return;
  }
  if (atomicSub(p.refs + page, 1) <= 0) {
    atomicAdd(p.refs + page, 1);
    flag(p.err, SMLA_DEVERR_PAGE_STATE);
  }
}

constexpr int kChunk = 512;                           // pages a warp counts at a time: 4 x 4 a lane

// Counts of pages [4 i, 4 i + 3] past `base` (pages past the pool: `pad`).
__device__ __forceinline__ int4 load_counts(const PagesParams& p, int64_t base, int i, int pad) {
  const int64_t at = base + 4 * (int64_t)i;
  const int32_t* r = p.refs + at;
  if (at + 3 < p.num_pages && (reinterpret_cast<uintptr_t>(r) & 15u) == 0)
    return __ldcg(reinterpret_cast<const int4*>(r));
  int4 v = make_int4(pad, pad, pad, pad);
  if (at < p.num_pages) v.x = __ldcg(r);
  if (at + 1 < p.num_pages) v.y = __ldcg(r + 1);
  if (at + 2 < p.num_pages) v.z = __ldcg(r + 2);
  if (at + 3 < p.num_pages) v.w = __ldcg(r + 3);
  return v;
}

// Pages of a chunk that are in use, before page `end` (whole warp; the same in every lane).
__device__ __forceinline__ int count_live(const PagesParams& p, int64_t base, int64_t end, int lane) {
  int4 v[kChunk / 128];
#pragma unroll
  for (int k = 0; k < kChunk / 128; ++k) v[k] = load_counts(p, base, k * 32 + lane, 0);
  int n = 0;
#pragma unroll
  for (int k = 0; k < kChunk / 128; ++k) {
    const int64_t at = base + 4 * (k * 32 + lane);
    n += (v[k].x > 0 && at < end) + (v[k].y > 0 && at + 1 < end) + (v[k].z > 0 && at + 2 < end) +
         (v[k].w > 0 && at + 3 < end);
  }
  return __reduce_add_sync(0xffffffffu, n);
}

// Calls f(page, count, pages in use before it in the chunk) for each page of a chunk.
template <class F>
__device__ __forceinline__ void walk(const PagesParams& p, int64_t base, int lane, F f) {
  int4 v[kChunk / 128];
#pragma unroll
  for (int k = 0; k < kChunk / 128; ++k) v[k] = load_counts(p, base, k * 32 + lane, 0);
  int before = 0;
#pragma unroll
  for (int k = 0; k < kChunk / 128; ++k) {
    const int r[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    int mine = 0, all = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t m = __ballot_sync(0xffffffffu, r[e] > 0);
      mine += __popc(m & ((1u << lane) - 1u));
      all += __popc(m);
    }
    mine += before;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t page = base + 4 * (k * 32 + lane) + e;
      if (page < p.num_pages) f((int)page, r[e], mine);
      mine += r[e] > 0;
    }
    before += all;
  }
}

// Who works: warp gw of `warps`, in CTA `cta` of `ctas`; neighbouring work goes
// to different SMs.
struct Team {
  int cta, ctas, gw, warps, lane;
};
__device__ __forceinline__ Team team(int cta, int ctas) {
  return {cta, ctas, cta + (int)(threadIdx.x >> 5) * ctas, ctas * kWarps, (int)(threadIdx.x & 31)};
}

constexpr int kRanked = 4;                            // chunks that a thread ranks
constexpr int kBatch = kPlanThreads * kRanked;        // of two million pages
struct Shared {
  int32_t scan[2][kWarps];
  int32_t prefix[kBatch];
};

// Counts the pages in use of each chunk (chunk c is warp c % warps's).
__device__ __forceinline__ void count_chunks(const PagesParams& p, int32_t* counts, int chunks, const Team& w) {
  const int lane = w.lane;
  for (int c = w.gw; c < chunks; c += w.warps) {
    const int n = count_live(p, (int64_t)c * kChunk, p.num_pages, lane);
    if (lane == 0) counts[c] = n;
  }
}

// Ranks a batch of up to kBatch chunks from c0 on, `before` pages being in use
// before them: sh.prefix holds those before each chunk, the result counts the
// batch in.  Whole CTA.
__device__ __forceinline__ int rank_batch(const int32_t* counts, int chunks, int c0, int before, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = c0 + (int)threadIdx.x * kRanked;
  int n[kRanked], sum = 0;
#pragma unroll
  for (int k = 0; k < kRanked; ++k) n[k] = c + k < chunks ? __ldcg(counts + c + k) : 0;
#pragma unroll
  for (int k = 0; k < kRanked; ++k) sum += n[k];
  const int own = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += x;
  }
  if (lane == 31) sh.scan[0][warp] = sum;
  __syncthreads();
  int at = before + sum - own + __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[0][lane] : 0);
#pragma unroll
  for (int k = 0; k < kRanked; ++k) {
    sh.prefix[threadIdx.x * kRanked + k] = at;
    at += n[k];
  }
  before += __reduce_add_sync(0xffffffffu, sh.scan[0][lane]);
  __syncthreads();
  return before;
}

// The CTA's share of the chunks of a ranked batch that `wanted(pages in use before
// the chunk, first page)` takes; f as for walk, with the pages in use before the
// page in the whole pool.
template <class W, class F>
__device__ __forceinline__ void walk_batch(const PagesParams& p, int chunks, int c0, const Team& w, const Shared& sh, W wanted,
                                           F f) {
  const int batch = min(kBatch, chunks - c0);
  for (int k = (w.gw - c0 % w.warps + w.warps) % w.warps; k < batch; k += w.warps) {
    const int live = sh.prefix[k];
    const int64_t base = (int64_t)(c0 + k) * kChunk;
    if (wanted(live, base)) walk(p, base, w.lane, [&](int page, int count, int in_chunk) { f(page, count, live + in_chunk); });
  }
}

template <class W, class F>
__device__ __forceinline__ void walk_chunks(const PagesParams& p, const int32_t* counts, int chunks, const Team& w,
                                            Shared& sh, W wanted, F f) {
  int before = 0;                                     // pages in use before this batch of chunks
  for (int c0 = 0; c0 < chunks; c0 += kBatch) {
    before = rank_batch(counts, chunks, c0, before, sh);
    walk_batch(p, chunks, c0, w, sh, wanted, f);
    __syncthreads();
  }
}

// Pages in use in the whole pool: every CTA sums the chunks' counts.
__device__ __forceinline__ int sum_counts(const int32_t* counts, int chunks, Shared& sh) {
  const int lane = threadIdx.x & 31;
  int32_t* s_warp = sh.scan[0];
  int n = 0;
  for (int c = threadIdx.x; c < chunks; c += kPlanThreads) n += __ldcg(counts + c);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) s_warp[threadIdx.x >> 5] = n;
  __syncthreads();
  n = __reduce_add_sync(0xffffffffu, s_warp[lane]);
  __syncthreads();
  return n;
}

// Calls f(row, first column, one past the last) for pieces of up to kPiece table
// entries of the rows' ranges [range(row).x, range(row).y), dealt out to the warps.
template <int kPiece = 128, class R, class F>
__device__ __forceinline__ void pieces(const PagesParams& p, const Team& w, R range, F f) {
  const int per_row = (p.max_pages + kPiece - 1) / kPiece;
  const int64_t all = (int64_t)p.rows * per_row;
  for (int64_t i = w.gw; i < all; i += w.warps) {
    const int b = (int)(i / per_row), c0 = (int)(i - (int64_t)b * per_row) * kPiece;
    const int2 r = range(b);
    const int from = max(r.x, c0), to = min(r.y, c0 + kPiece);
    if (from < to) f(b, from, to);
  }
}

// ---------------------------------------------------------------- resize
// ws: [0] pages needed in all; rows words at kPagesHeader: first needed entry
// of the row (x 2 + copy-on-write bit); rows words behind: copies before it;
// num_pages words behind: the free pages taken, in order; then the chunks' counts.
struct Resize {
  int32_t *off, *cows, *list, *counts;
  int chunks;
};
__device__ __forceinline__ Resize resize_state(const PagesParams& p) {
  Resize r;
  r.off = p.ws + kPagesHeader;
  r.cows = r.off + p.rows;
  r.list = r.cows + p.rows;
  r.counts = r.list + p.num_pages;
  r.chunks = (int)(((int64_t)p.num_pages + kChunk - 1) / kChunk);
  return r;
}

// 1. what shrinks
__device__ __forceinline__ void resize_drop(const PagesParams& p, const Team& w) {
  if (w.cta == 0 && threadIdx.x == 0) *p.move_count = 0;
  pieces(p, w,
         [&](int b) {
           bool bad = false;
           const int co = page_columns(p, fetch(p.lens + b), &bad), cn = page_columns(p, fetch(p.new_lens + b), &bad);
           if (bad) flag(p.err, SMLA_DEVERR_PAGE_STATE);
           return make_int2(cn, co);
         },
         [&](int b, int from, int to) {
           int32_t* row = p.bt + (int64_t)b * p.bt_stride;
           int page[4];
#pragma unroll
           for (int k = 0; k < 4; ++k) {
             const int c = from + k * 32 + w.lane;
             page[k] = c < to ? row[c] : 0;
           }
#pragma unroll
           for (int k = 0; k < 4; ++k) {
             const int c = from + k * 32 + w.lane;
             if (c < to) {
               drop_ref(p, page[k]);
               row[c] = -1;
             }
           }
         });
}

// 2. what the growing rows need, in order of the rows (one CTA)
__device__ __forceinline__ void resize_rows(const PagesParams& p, const Resize& r, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int need0 = 0, cow0 = 0;
  for (int base = 0; base < p.rows; base += kPlanThreads) {
    const int b = base + threadIdx.x;
    int need = 0, cow = 0;
    if (b < p.rows) {
      bool bad = false;
      const int old = clamped_len(p, fetch(p.lens + b)), now = clamped_len(p, fetch(p.new_lens + b));
      if (now > old) {
        need = page_columns(p, now, &bad) - page_columns(p, old, &bad);
        if (old % p.page_size != 0) {
          const int page = __ldcg(p.bt + (int64_t)b * p.bt_stride + old / p.page_size);
          if (in_pool(p, page)) cow = __ldcg(p.refs + page) > 1;
          else flag(p.err, SMLA_DEVERR_PAGE_STATE);
        }
        need += cow;
      }
    }
    int sn = need, sc = cow;                              // inclusive sums over the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sn, d), y = __shfl_up_sync(0xffffffffu, sc, d);
      if (lane >= d) sn += x, sc += y;
    }
    if (lane == 31) sh.scan[0][warp] = sn, sh.scan[1][warp] = sc;
    __syncthreads();
    const int wn = __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[0][lane] : 0);
    const int wc = __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[1][lane] : 0);
    if (b < p.rows) {
      r.off[b] = 2 * (need0 + wn + sn - need) + cow;
      r.cows[b] = cow0 + wc + sc - cow;
    }
    need0 += __reduce_add_sync(0xffffffffu, sh.scan[0][lane]);
    cow0 += __reduce_add_sync(0xffffffffu, sh.scan[1][lane]);
    __syncthreads();
  }
  if (threadIdx.x == 0) p.ws[0] = need0;
}

// The needs, and the pages in use beside them.
__device__ __forceinline__ void resize_needs(const PagesParams& p, const Resize& r, const Team& w, Shared& sh) {
  if (w.cta == 0) resize_rows(p, r, sh);
  if (w.ctas == 1) count_chunks(p, r.counts, r.chunks, w);
  else if (w.cta > 0) count_chunks(p, r.counts, r.chunks, team(w.cta - 1, w.ctas - 1));
}

// 3. the lowest free pages, in order: the smaller of what is needed and what is free
__device__ __forceinline__ int resize_list(const PagesParams& p, const Resize& r, const Team& w, Shared& sh) {
  const int need = __ldcg(p.ws);
  // (one batch is ranked and summed in one)
  const bool one = r.chunks <= kBatch;
  const int live_all = one ? rank_batch(r.counts, r.chunks, 0, 0, sh) : need > 0 ? sum_counts(r.counts, r.chunks, sh) : 0;
  const int take = min(need, p.num_pages - live_all);
  if (need > take && w.cta == 0 && threadIdx.x == 0) flag(p.err, SMLA_DEVERR_OUT_OF_PAGES);
  if (take == 0) return 0;
  const auto wanted = [&](int live, int64_t base) { return base - live < take; };   // free pages before the chunk
  const auto give = [&](int page, int count, int live) {
    const int k = page - live;
    if (count <= 0 && k < take) {
      r.list[k] = page;
      p.refs[page] = 1;
    }
  };
  if (one) walk_batch(p, r.chunks, 0, w, sh, wanted, give);
  else walk_chunks(p, r.counts, r.chunks, w, sh, wanted, give);
  return take;
}

// 4. handed out: the pages of growing rows, then the copies of shared pages
__device__ __forceinline__ void resize_assign(const PagesParams& p, const Resize& r, const Team& w, int take) {
  if (__ldcg(p.ws) == 0) return;
  pieces(p, w,
         [&](int b) {
           bool bad = false;
           const int old = clamped_len(p, fetch(p.lens + b)), now = clamped_len(p, fetch(p.new_lens + b));
           return now > old ? make_int2(page_columns(p, old, &bad), page_columns(p, now, &bad)) : make_int2(0, 0);
         },
         [&](int b, int from, int to) {
           bool bad = false;
           const int co = page_columns(p, clamped_len(p, fetch(p.lens + b)), &bad);
           const int o = __ldcg(r.off + b), k0 = (o >> 1) + (o & 1) - co;     // rank of column 0, as it were
           int32_t* row = p.bt + (int64_t)b * p.bt_stride;
           int page[4];
#pragma unroll
           for (int k = 0; k < 4; ++k) {
             const int c = from + k * 32 + w.lane;
             page[k] = c < to && k0 + c < take ? __ldcg(r.list + k0 + c) : -1;
           }
#pragma unroll
           for (int k = 0; k < 4; ++k) {
             const int c = from + k * 32 + w.lane;
             if (c < to) row[c] = page[k];
           }
         });
  // (from the CTA's last warp on, which the pieces reach last)
  for (int b = w.cta + (kPlanThreads - 1 - (int)threadIdx.x) * w.ctas; b < p.rows; b += w.ctas * kPlanThreads) {
    const int o = __ldcg(r.off + b), k = o >> 1;
    if ((o & 1) != 0 && k < take) {
      int32_t* at = p.bt + (int64_t)b * p.bt_stride + clamped_len(p, fetch(p.lens + b)) / p.page_size;
      const int from = __ldcg(at), to = __ldcg(r.list + k), m = __ldcg(r.cows + b);
      *at = to;
      atomicSub(p.refs + from, 1);
      p.move_src[m] = from;
      p.move_dst[m] = to;
      atomicMax(p.move_count, m + 1);                     // the rows that got a page are the first ones
    }
  }
}

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
pages_resize_kernel(const PagesParams p) {
  __shared__ Shared sh;
  const Team w = team((int)ptx::cluster_rank(), kClusterCtas);
  const Resize r = resize_state(p);
  await_prior_kernel();
  admit_next_kernel();
  resize_drop(p, w);
  ptx::cluster_sync();
  resize_needs(p, r, w, sh);
  ptx::cluster_sync();
  const int take = resize_list(p, r, w, sh);
  ptx::cluster_sync();
  resize_assign(p, r, w, take);
}

// The same phases as launches over the whole GPU (kPhase 0 .. 3).
template <int kPhase>
__global__ void __launch_bounds__(kPlanThreads, 1) pages_resize_phase_kernel(const PagesParams p) {
  __shared__ Shared sh;
  const Team w = team(blockIdx.x, gridDim.x);
  const Resize r = resize_state(p);
  await_prior_kernel();
  admit_next_kernel();
  if constexpr (kPhase == 0) {
    resize_drop(p, w);
  } else if constexpr (kPhase == 1) {
    resize_needs(p, r, w, sh);
  } else if constexpr (kPhase == 2) {
    const int take = resize_list(p, r, w, sh);
    if (w.cta == 0 && threadIdx.x == 0) p.ws[1] = take;
  } else {
    resize_assign(p, r, w, __ldcg(p.ws + 1));
  }
}

// ------------------------------------------------------------------ fork
__global__ void __launch_bounds__(256) pages_fork_kernel(const PagesParams p) {
  const int b = (int)((blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (b >= p.rows) return;
  await_prior_kernel();
  admit_next_kernel();
  const int parent = fetch(p.parents + b), own_len = fetch(p.lens + b);
  int len = own_len;
  if (parent >= 0) {
    if (parent >= p.rows || own_len != 0) {
      if (lane == 0) flag(p.err, SMLA_DEVERR_PAGE_STATE);
    } else {
      len = fetch(p.lens + parent);
      bool bad = false;
      const int n = page_columns(p, len, &bad);
      if (bad && lane == 0) flag(p.err, SMLA_DEVERR_PAGE_STATE);
      // a parent holds pages and a child none, so no row is both read and written
      const int32_t* from = p.bt + (int64_t)parent * p.bt_stride;
      int32_t* to = p.bt + (int64_t)b * p.bt_stride;
      for (int c = lane; c < n; c += 32) {
        const int page = from[c];
        to[c] = page;
        if (in_pool(p, page)) atomicAdd(p.refs + page, 1);
        else flag(p.err, SMLA_DEVERR_PAGE_STATE);
      }
    }
  }
  if (lane == 0) p.out_lens[b] = len;
}

// --------------------------------------------------------------- reorder
// Every row takes its parent's entries at once.  A beam keeps most of what it
// has (its prompt's pages are its parent's, too), so only entries that differ
// are counted and written.
//   1. the parents' entries into the workspace, the pages that a row did not
//      hold at that column counted once more;
//   2. rows overwritten from there, the pages given up counted once less (after
//      all of 1, so that no page that stays in use passes through 0).
// Both phases compare the same two entries: a row is changed by the thread that
// compared it only.  Latency again: 16 rows of 64 columns 6 us (one cluster), 1024 of
// 1024 in two launches of 5 and 9 (with pieces of 128 entries, two turns of the warps,
// 6 and 10).
constexpr int kReorderPer = 8;                        // columns a lane takes at a time

// Row b's parent, b itself for one that stays (one that is not a row is flagged), -1 for one that ends.
__device__ __forceinline__ int parent_of(const PagesParams& p, int b, bool* bad) {
  const int parent = fetch(p.parents + b);
  if (parent >= p.rows) {
    *bad = true;
    return b;
  }
  return max(parent, -1);
}

// Columns of row b's parent and of itself.
struct Reorder {
  int parent, theirs, mine;
};
__device__ __forceinline__ Reorder reorder_row(const PagesParams& p, int b) {
  bool bad = false;
  Reorder r;
  r.parent = parent_of(p, b, &bad);
  r.mine = page_columns(p, fetch(p.lens + b), &bad);
  r.theirs = r.parent >= 0 ? page_columns(p, fetch(p.lens + r.parent), &bad) : 0;
  if (bad) flag(p.err, SMLA_DEVERR_PAGE_STATE);
  return r;
}

template <bool kWrite>
__device__ __forceinline__ void reorder_phase(const PagesParams& p, const Team& w) {
  Reorder r;
  pieces<32 * kReorderPer>(
      p, w,
      [&](int b) {
        r = reorder_row(p, b);
        return make_int2(0, r.parent == b ? 0 : kWrite ? max(r.mine, r.theirs) : r.theirs);
      },
      [&](int b, int from, int to) {
        int32_t* const mine = p.bt + (int64_t)b * p.bt_stride;
        int32_t* const saved = p.ws + (int64_t)b * p.max_pages;
        const int32_t* const theirs = kWrite ? saved : p.bt + (int64_t)r.parent * p.bt_stride;
        int now[kReorderPer], old[kReorderPer];
#pragma unroll
        for (int k = 0; k < kReorderPer; ++k) {
          const int c = from + k * 32 + w.lane;
          now[k] = c < to && c < r.theirs ? __ldcg(theirs + c) : -1;
          old[k] = c < to && c < r.mine ? __ldcg(mine + c) : -1;
        }
#pragma unroll
        for (int k = 0; k < kReorderPer; ++k) {
          const int c = from + k * 32 + w.lane;
          if (c >= to) continue;
          const bool same = c < r.mine && c < r.theirs && old[k] == now[k];
          if constexpr (!kWrite) {
            saved[c] = now[k];
            if (same) continue;
            if (in_pool(p, now[k])) atomicAdd(p.refs + now[k], 1);
            else flag(p.err, SMLA_DEVERR_PAGE_STATE);
          } else if (!same) {
            mine[c] = now[k];
            if (c < r.mine) drop_ref(p, old[k]);
          }
        }
      });
}

__device__ __forceinline__ void reorder_save(const PagesParams& p, const Team& w) { reorder_phase<false>(p, w); }
__device__ __forceinline__ void reorder_write(const PagesParams& p, const Team& w) {
  reorder_phase<true>(p, w);
  // (from the CTA's last warp on, which the pieces reach last)
  for (int b = w.cta + (kPlanThreads - 1 - (int)threadIdx.x) * w.ctas; b < p.rows; b += w.ctas * kPlanThreads) {
    bool bad = false;
    const int parent = parent_of(p, b, &bad);
    p.out_lens[b] = parent >= 0 ? fetch(p.lens + parent) : 0;
  }
}

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
pages_reorder_kernel(const PagesParams p) {
  const Team w = team((int)ptx::cluster_rank(), kClusterCtas);
  await_prior_kernel();
  admit_next_kernel();
  reorder_save(p, w);
  ptx::cluster_sync();
  reorder_write(p, w);
}

template <int kPhase>
__global__ void __launch_bounds__(kPlanThreads, 1) pages_reorder_phase_kernel(const PagesParams p) {
  const Team w = team(blockIdx.x, gridDim.x);
  await_prior_kernel();
  admit_next_kernel();
  if constexpr (kPhase == 0) reorder_save(p, w);
  else reorder_write(p, w);
}

// --------------------------------------------------------- shared prefix
// Group g's rows with tokens hold `columns` whole pages each at least; the
// first column where one of them differs from the first ends the prefix.
// A CTA a group, its warps 256 columns of a row at a time, the front ones first,
// so that what lies behind an early difference is hardly read (64 groups of 16 rows of
// 600 columns: 6.5 us; 25 with a row a warp and its loads one behind another).
constexpr int kPrefixThreads = 1024;
constexpr int kPrefixPer = 8;                         // columns a lane takes at a time
__global__ void __launch_bounds__(kPrefixThreads)
pages_shared_prefix_kernel(const PagesParams p, const int32_t* group_starts, int32_t* prefix_lens) {
  __shared__ int s_columns, s_first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_columns = p.max_pages;
    s_first = p.rows;
  }
  __syncthreads();
  await_prior_kernel();
  admit_next_kernel();
  const int lo = min(max(fetch(group_starts + blockIdx.x), 0), p.rows);
  const int hi = min(fetch(group_starts + blockIdx.x + 1), p.rows);
  for (int b = lo + (int)threadIdx.x; b < hi; b += kPrefixThreads) {
    const int len = fetch(p.lens + b), n = clamped_len(p, len);
    if (n != len) flag(p.err, SMLA_DEVERR_PAGE_STATE);
    if (n > 0) {
      atomicMin(&s_columns, n / p.page_size);
      atomicMin(&s_first, b);
    }
  }
  __syncthreads();
  const int first = s_first, columns = s_columns;
  if (first < p.rows) {
    const int32_t* lead = p.bt + (int64_t)first * p.bt_stride;
    const int members = hi - first - 1;               // rows to compare with the first one
    const int64_t all = (int64_t)members * ((columns + 32 * kPrefixPer - 1) / (32 * kPrefixPer));
    for (int64_t i = warp; i < all; i += kPrefixThreads / 32) {
      const int c0 = (int)(i / members) * 32 * kPrefixPer, b = first + 1 + (int)(i % members);
      if (c0 >= __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_columns), 0)) break;
      if (clamped_len(p, fetch(p.lens + b)) == 0) continue;
      const int32_t* row = p.bt + (int64_t)b * p.bt_stride;
      int page[kPrefixPer], other[kPrefixPer];
#pragma unroll
      for (int k = 0; k < kPrefixPer; ++k) {
        const int c = c0 + k * 32 + lane;
        page[k] = c < columns ? __ldcg(lead + c) : 0;
        other[k] = c < columns ? __ldcg(row + c) : 0;
      }
      int miss = columns;
#pragma unroll
      for (int k = kPrefixPer - 1; k >= 0; --k)
        if (other[k] != page[k]) miss = c0 + k * 32 + lane;
      miss = __reduce_min_sync(0xffffffffu, miss);
      if (miss < columns && lane == 0) atomicMin(&s_columns, miss);
    }
    for (int c = threadIdx.x; c < columns; c += kPrefixThreads)
      if (__ldcg(lead + c) < 0) atomicMin(&s_columns, c);
  }
  __syncthreads();
  if (threadIdx.x == 0) prefix_lens[blockIdx.x] = first < p.rows ? s_columns * p.page_size : 0;
}

// --------------------------------------------------------------- compact
// ws: [0] pages in use n, [1] pages in use before page n; num_pages words at
// kPagesHeader: the move of each page in use at or past n; then the chunks' counts.
struct Compact {
  int32_t *move_of, *counts;
  int chunks;
};
__device__ __forceinline__ Compact compact_state(const PagesParams& p) {
  Compact c;
  c.move_of = p.ws + kPagesHeader;
  c.counts = c.move_of + p.num_pages;
  c.chunks = (int)(((int64_t)p.num_pages + kChunk - 1) / kChunk);
  return c;
}

// The moves, from the chunks' counts; returns how many.
__device__ __forceinline__ int compact_moves(const PagesParams& p, const Compact& c, const Team& w, Shared& sh) {
  const int n = sum_counts(c.counts, c.chunks, sh);
  // pages in use before page n: the chunks before its own, and those before it there
  const int own = n / kChunk;
  int low = sum_counts(c.counts, min(own, c.chunks), sh);
  if (own < c.chunks) low += count_live(p, (int64_t)own * kChunk, n, w.lane);
  if (w.cta == 0 && threadIdx.x == 0) {
    p.ws[0] = n;
    p.ws[1] = low;
    *p.move_count = n - low;
  }
  if (n > low)
    walk_chunks(p, c.counts, c.chunks, w, sh,
                [&](int live, int64_t base) { return base < n || live < n; },
                [&](int page, int count, int live) {      // live: pages in use before this one
                  if (count <= 0 && page < n) {
                    p.move_dst[page - live] = page;
                  } else if (count > 0 && page >= n) {
                    p.move_src[live - low] = page;
                    c.move_of[page] = live - low;
                  }
                });
  return n - low;
}

__device__ __forceinline__ void compact_counts(const PagesParams& p, const Team& w, int moves) {
  for (int k = w.cta * kPlanThreads + threadIdx.x; k < moves; k += w.ctas * kPlanThreads) {
    const int from = __ldcg(p.move_src + k), to = __ldcg(p.move_dst + k);
    p.refs[to] = __ldcg(p.refs + from);
    p.refs[from] = 0;
  }
}

// One table entry, once the moves are known.
__device__ __forceinline__ void renumber(const PagesParams& p, const int32_t* move_of, int live, int moves, int32_t* at) {
  const int page = *at;
  if (!in_pool(p, page)) {
    flag(p.err, SMLA_DEVERR_PAGE_STATE);
  } else if (page >= live) {
    // a page that was not in use has no move of its own
    const int k = __ldcg(move_of + page);
    if (k >= 0 && k < moves && __ldcg(p.move_src + k) == page) *at = __ldcg(p.move_dst + k);
    else flag(p.err, SMLA_DEVERR_PAGE_STATE);
  }
}

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
pages_compact_kernel(const PagesParams p) {
  __shared__ Shared sh;
  const Team w = team((int)ptx::cluster_rank(), kClusterCtas);
  const Compact c = compact_state(p);
  await_prior_kernel();
  admit_next_kernel();
  count_chunks(p, c.counts, c.chunks, w);
  ptx::cluster_sync();
  const int moves = compact_moves(p, c, w, sh);
  ptx::cluster_sync();
  compact_counts(p, w, moves);
  const int live = __ldcg(p.ws);
  pieces(p, w,
         [&](int b) {
           bool bad = false;
           const int n = page_columns(p, fetch(p.lens + b), &bad);
           if (bad) flag(p.err, SMLA_DEVERR_PAGE_STATE);
           return make_int2(0, n);
         },
         [&](int b, int from, int to) {
           for (int at = from + w.lane; at < to; at += 32) renumber(p, c.move_of, live, moves, p.bt + (int64_t)b * p.bt_stride + at);
         });
}

// The same phases as launches over the whole GPU (kPhase 0 .. 2; the counts may
// move only when nobody ranks them any more).
template <int kPhase>
__global__ void __launch_bounds__(kPlanThreads, 1) pages_compact_phase_kernel(const PagesParams p) {
  __shared__ Shared sh;
  const Team w = team(blockIdx.x, gridDim.x);
  const Compact c = compact_state(p);
  await_prior_kernel();
  admit_next_kernel();
  if constexpr (kPhase == 0) count_chunks(p, c.counts, c.chunks, w);
  else if constexpr (kPhase == 1) compact_moves(p, c, w, sh);
  else compact_counts(p, w, __ldcg(p.ws) - __ldcg(p.ws + 1));
}

// Then the tables, 256 columns of a row a CTA.
__global__ void __launch_bounds__(256) pages_renumber_kernel(const PagesParams p) {
  const int b = blockIdx.x;
  bool bad = false;
  await_prior_kernel();
  admit_next_kernel();
  const int n = page_columns(p, fetch(p.lens + b), &bad);
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) flag(p.err, SMLA_DEVERR_PAGE_STATE);
  const int live = __ldcg(p.ws), moves = live - __ldcg(p.ws + 1);
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < n; c += gridDim.y * blockDim.x)
    renumber(p, p.ws + kPagesHeader, live, moves, p.bt + (int64_t)b * p.bt_stride + c);
}

// ------------------------------------------------------------------ copy
// Bandwidth bound: every byte once in, once out (3417 moves of 33 KB pages in two
// pools: 73 us, 6.2 TB/s of 6.8 measured for a plain copy).  A unit is 512 consecutive
// pieces of one pool's moved pages, four per thread, all loaded before the
// first is stored.
constexpr int kCopyThreads = 128;
constexpr int kCopyPer = 4;
constexpr int kCopyUnit = kCopyThreads * kCopyPer;

template <class V>
__device__ __forceinline__ void copy_unit(const CopyParams& p, const CopyParams::Pool& pool, int64_t first, int64_t total) {
  const int64_t m0 = first / pool.pieces;
  const uint32_t r0 = (uint32_t)(first - m0 * pool.pieces);
  V v[kCopyPer];
  uint8_t* to[kCopyPer];
#pragma unroll
  for (int u = 0; u < kCopyPer; ++u) {
    const uint32_t i = u * kCopyThreads + threadIdx.x;
    to[u] = nullptr;
    if (first + i < total) {
      const uint32_t dm = (r0 + i) / (uint32_t)pool.pieces, r = r0 + i - dm * (uint32_t)pool.pieces;
      const int src = fetch(p.src + m0 + dm), dst = fetch(p.dst + m0 + dm);
      if (src >= 0 && src < p.num_pages && dst >= 0 && dst < p.num_pages) {
        v[u] = *reinterpret_cast<const V*>(pool.base + (int64_t)src * pool.stride + (int64_t)r * sizeof(V));
        to[u] = pool.base + (int64_t)dst * pool.stride + (int64_t)r * sizeof(V);
      } else {
        flag(p.err, SMLA_DEVERR_PAGE_STATE);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kCopyPer; ++u)
    if (to[u] != nullptr) *reinterpret_cast<V*>(to[u]) = v[u];
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyParams p) {
  await_prior_kernel();
  admit_next_kernel();
  const int64_t moves = min(max(fetch(p.count), 0), p.capacity);
  int64_t unit = blockIdx.x, done = 0;                    // units of the pools before this one
  for (int k = 0; k < p.num_pools; ++k) {
    const CopyParams::Pool& pool = p.pool[k];
    const int64_t total = moves * pool.pieces, units = (total + kCopyUnit - 1) / kCopyUnit;
    for (; unit < done + units; unit += gridDim.x) {
      const int64_t first = (unit - done) * kCopyUnit;
      if (pool.vec == 16) copy_unit<uint4>(p, pool, first, total);
      else if (pool.vec == 4) copy_unit<uint32_t>(p, pool, first, total);
      else copy_unit<uint8_t>(p, pool, first, total);
    }
    done += units;
  }
}

}  // namespace

namespace {

bool one_cluster(const PagesParams& p) { return (int64_t)p.rows * p.max_pages + p.num_pages <= kClusterEntries; }

// CTAs of a phase over the whole GPU: one an SM, no more than there is work for.
unsigned phase_ctas(int64_t warps, int sms) {
  const int64_t n = (warps + kWarps - 1) / kWarps;
  return (unsigned)(n < 1 ? 1 : n < sms ? n : sms);
}

}  // namespace

cudaError_t launch_pages_resize(const PagesParams& p, int sms, cudaStream_t stream) {
  if (one_cluster(p)) return launch_overlapped(pages_resize_kernel, dim3(kClusterCtas), kPlanThreads, 0, stream, p);
  const dim3 tables(phase_ctas((int64_t)p.rows * ((p.max_pages + 127) / 128), sms));
  const dim3 pages(phase_ctas(((int64_t)p.num_pages + kChunk - 1) / kChunk, sms));
  cudaError_t e = launch_overlapped(pages_resize_phase_kernel<0>, tables, kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_overlapped(pages_resize_phase_kernel<1>, pages, kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_overlapped(pages_resize_phase_kernel<2>, pages, kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_overlapped(pages_resize_phase_kernel<3>, tables, kPlanThreads, 0, stream, p);
  return e;
}

cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream) {
  return launch_overlapped(pages_fork_kernel, dim3((unsigned)((p.rows + 7) / 8)), 256, 0, stream, p);
}

cudaError_t launch_pages_reorder(const PagesParams& p, int sms, cudaStream_t stream) {
  if ((int64_t)p.rows * p.max_pages <= kClusterEntries)
    return launch_overlapped(pages_reorder_kernel, dim3(kClusterCtas), kPlanThreads, 0, stream, p);
  constexpr int kPiece = 32 * kReorderPer;
  const dim3 tables(phase_ctas((int64_t)p.rows * ((p.max_pages + kPiece - 1) / kPiece), sms));
  cudaError_t e = launch_overlapped(pages_reorder_phase_kernel<0>, tables, kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_overlapped(pages_reorder_phase_kernel<1>, tables, kPlanThreads, 0, stream, p);
  return e;
}

cudaError_t launch_pages_shared_prefix(const PagesParams& p, const int32_t* group_starts, int num_groups, int32_t* prefix_lens,
                                       cudaStream_t stream) {
  return launch_overlapped(pages_shared_prefix_kernel, dim3((unsigned)num_groups), kPrefixThreads, 0, stream, p, group_starts,
                           prefix_lens);
}

cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t stream) {
  if (one_cluster(p)) return launch_overlapped(pages_compact_kernel, dim3(kClusterCtas), kPlanThreads, 0, stream, p);
  const dim3 pages(phase_ctas(((int64_t)p.num_pages + kChunk - 1) / kChunk, sms));
  cudaError_t e = launch_overlapped(pages_compact_phase_kernel<0>, pages, kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_overlapped(pages_compact_phase_kernel<1>, pages, kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_overlapped(pages_compact_phase_kernel<2>, pages, kPlanThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  const int cols = (p.max_pages + 255) / 256;
  return launch_overlapped(pages_renumber_kernel, dim3((unsigned)p.rows, (unsigned)(cols < 64 ? cols : 64)), 256, 0, stream,
                           p);
}

cudaError_t launch_pages_copy(const CopyParams& p, int sms, cudaStream_t stream) {
  // the number of moves is on the device: the grid is what could be moved, at most what the GPU holds at once
  int64_t pieces = 0;
  for (int k = 0; k < p.num_pools; ++k) pieces += ((int64_t)p.capacity * p.pool[k].pieces + kCopyUnit - 1) / kCopyUnit;
  const int64_t grid = pieces < (int64_t)sms * 16 ? pieces : (int64_t)sms * 16;
  if (grid == 0) return cudaSuccess;
  return launch_overlapped(pages_copy_kernel, dim3((unsigned)grid), kCopyThreads, 0, stream, p);
}

}  // namespace smla
