// Pages of the latent cache: growing, shrinking, forking and compacting the
// requests' page tables on the device, and copying pages.
//
// The state is a count per page (a page with count 0 is free) and a table row
// per request.  Ranking the free (or live) pages in order is a prefix sum over
// the counts: resize and compact run it inside one cluster of CTAs, each warp
// owning one contiguous segment of the pool, so that the whole call is one
// launch with cluster barriers in between, and every page's rank (hence who
// gets it) depends on nothing but the state.  What bounds them is latency: the
// counts (4 bytes a page) are read once or twice, the rest is a few dependent
// L2 round trips.
#include "cache.cuh"
#include "tc_ptx.cuh"

namespace smla {
namespace {

constexpr int kClusterCtas = 8;                       // portable cluster size
constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;
constexpr int kClusterWarps = kClusterCtas * kWarps;

__device__ __forceinline__ void flag(int32_t* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}

// Columns that `len` tokens hold; a length that cannot be is clamped, *bad set.
__device__ __forceinline__ int page_columns(const PagesParams& p, int len, bool* bad) {
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  if (len < 0 || len > cap) *bad = true;
  len = (int)min((int64_t)max(len, 0), cap);
  return (len + p.page_size - 1) / p.page_size;
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

// Segment [begin, end) of the pool that warp w of the cluster ranks.
__device__ __forceinline__ void segment(int num_pages, int w, int* begin, int* end) {
  const int64_t per = (((int64_t)num_pages + kClusterWarps - 1) / kClusterWarps + 31) / 32 * 32;
  *begin = (int)min((int64_t)num_pages, per * w);
  *end = (int)min((int64_t)num_pages, per * (w + 1));
}

// Pages of [begin, end) with a count above 0 (whole warp; same result in every lane).
__device__ __forceinline__ int count_live(const int32_t* refs, int begin, int end, int lane) {
  constexpr int kUnroll = 8;                            // loads in flight per lane
  int n = 0;
  for (int base = begin; base < end; base += 32 * kUnroll) {
    int r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * 32 + lane;
      r[u] = i < end ? __ldcg(refs + i) : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) n += r[u] > 0;
  }
  return __reduce_add_sync(0xffffffffu, n);
}

// Calls f(page, live, live pages before it in the segment) for each page of
// [begin, end); f returns false (warp-uniformly) to stop early.
template <class F>
__device__ __forceinline__ void walk(const int32_t* refs, int begin, int end, int lane, F f) {
  constexpr int kUnroll = 4;
  int before = 0;
  for (int base = begin; base < end; base += 32 * kUnroll) {
    int r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * 32 + lane;
      r[u] = i < end ? __ldcg(refs + i) : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * 32 + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, r[u] > 0);
      if (i < end) f(i, r[u], before + __popc(m & ((1u << lane) - 1u)));
      before += __popc(m);
    }
  }
}

// Live pages before each warp's segment, for the whole cluster: returns this
// warp's, and the total.  One cluster barrier.
__device__ __forceinline__ int live_before(int live, int rank, int warp, int lane, int32_t* s_count, int* total) {
  if (lane == 0) s_count[warp] = live;
  ptx::cluster_sync();
  // the counts of all warps of all CTAs, read from their shared memory
  int before = 0, all = 0;
  for (int c = 0; c < kClusterCtas; ++c) {
    const uint32_t a = ptx::map_to_rank(ptx::smem_addr(s_count + lane), c);
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    all += v;
    if (c < rank || (c == rank && lane < warp)) before += v;
  }
  static_assert(kWarps == 32, "one lane per warp");
  *total = __reduce_add_sync(0xffffffffu, all);
  return __reduce_add_sync(0xffffffffu, before);
}

// ---------------------------------------------------------------- resize
// ws: [0] pages needed in all; rows words at kPagesHeader: first needed entry
// of the row (x 2 + copy-on-write bit); rows words behind: copies before it;
// num_pages words behind: the free pages taken, in order.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
pages_resize_kernel(const PagesParams p) {
  __shared__ int32_t s_count[kWarps];
  __shared__ int32_t s_scan[2][kWarps];
  const int rank = (int)ptx::cluster_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gw = rank * kWarps + warp;
  int32_t* off = p.ws + kPagesHeader;
  int32_t* cows = off + p.rows;
  int32_t* list = cows + p.rows;

  // 1. what shrinks
  if (rank == 0 && threadIdx.x == 0) *p.move_count = 0;
  for (int b = gw; b < p.rows; b += kClusterWarps) {
    bool bad = false;
    const int co = page_columns(p, __ldg(p.lens + b), &bad), cn = page_columns(p, __ldg(p.new_lens + b), &bad);
    if (bad) flag(p.err, SMLA_DEVERR_PAGE_STATE);
    int32_t* row = p.bt + (int64_t)b * p.bt_stride;
    for (int c = cn + lane; c < co; c += 32) {
      drop_ref(p, row[c]);
      row[c] = -1;
    }
  }
  __threadfence();
  ptx::cluster_sync();

  // 2. what the growing rows need, in order of the rows (the first CTA), and
  // how many pages of each segment are free
  if (rank == 0) {
    int need0 = 0, cow0 = 0;
    for (int base = 0; base < p.rows; base += kPlanThreads) {
      const int b = base + threadIdx.x;
      int need = 0, cow = 0;
      if (b < p.rows) {
        bool bad = false;
        const int old = clamped_len(p, __ldg(p.lens + b)), now = clamped_len(p, __ldg(p.new_lens + b));
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
      int sn = need, sc = cow;                            // inclusive sums over the block
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sn, d), y = __shfl_up_sync(0xffffffffu, sc, d);
        if (lane >= d) sn += x, sc += y;
      }
      if (lane == 31) s_scan[0][warp] = sn, s_scan[1][warp] = sc;
      __syncthreads();
      const int wn = __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[0][lane] : 0);
      const int wc = __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[1][lane] : 0);
      if (b < p.rows) {
        off[b] = 2 * (need0 + wn + sn - need) + cow;
        cows[b] = cow0 + wc + sc - cow;
      }
      need0 += __reduce_add_sync(0xffffffffu, s_scan[0][lane]);
      cow0 += __reduce_add_sync(0xffffffffu, s_scan[1][lane]);
      __syncthreads();
    }
    if (threadIdx.x == 0) p.ws[0] = need0;
    __threadfence();
  }
  int begin, end, live_all;
  segment(p.num_pages, gw, &begin, &end);
  const int live = live_before(count_live(p.refs, begin, end, lane), rank, warp, lane, s_count, &live_all);
  const int need_all = __ldcg(p.ws), free_all = p.num_pages - live_all;
  if (need_all > free_all && rank == 0 && threadIdx.x == 0) flag(p.err, SMLA_DEVERR_OUT_OF_PAGES);

  // 3. the lowest free pages, in order
  const int take = min(need_all, free_all);
  const int rank0 = begin - live;                         // free pages before the segment
  if (rank0 < take) {
    walk(p.refs, begin, end, lane, [&](int page, int count, int live_in_segment) {
      const int k = rank0 + (page - begin) - live_in_segment;
      if (count <= 0 && k < take) {
        list[k] = page;
        p.refs[page] = 1;
      }
    });
  }
  __threadfence();
  ptx::cluster_sync();

  // 4. handed out
  for (int b = gw; b < p.rows; b += kClusterWarps) {
    bool bad = false;
    const int old = clamped_len(p, __ldg(p.lens + b)), now = clamped_len(p, __ldg(p.new_lens + b));
    if (now <= old) continue;
    const int co = page_columns(p, old, &bad), cn = page_columns(p, now, &bad);
    const int o = __ldcg(off + b), cow = o & 1;
    int k = o >> 1;
    int32_t* row = p.bt + (int64_t)b * p.bt_stride;
    if (cow) {
      if (lane == 0 && k < take) {
        const int from = __ldcg(row + old / p.page_size), to = __ldcg(list + k);
        row[old / p.page_size] = to;
        atomicSub(p.refs + from, 1);
        const int m = __ldcg(cows + b);
        p.move_src[m] = from;
        p.move_dst[m] = to;
        atomicMax(p.move_count, m + 1);                   // the rows that got a page are the first ones
      }
      ++k;
    }
    for (int c = co + lane; c < cn; c += 32) {
      const int i = k + (c - co);
      row[c] = i < take ? __ldcg(list + i) : -1;
    }
  }
}

// ------------------------------------------------------------------ fork
__global__ void __launch_bounds__(256) pages_fork_kernel(const PagesParams p) {
  const int b = (int)((blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (b >= p.rows) return;
  const int parent = __ldg(p.parents + b), own_len = __ldg(p.lens + b);
  int len = own_len;
  if (parent >= 0) {
    if (parent >= p.rows || own_len != 0) {
      if (lane == 0) flag(p.err, SMLA_DEVERR_PAGE_STATE);
    } else {
      len = __ldg(p.lens + parent);
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

// --------------------------------------------------------------- compact
// ws: [0] pages in use n, [1] pages in use before page n; num_pages words at
// kPagesHeader: the move of each page in use at or past n.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
pages_compact_kernel(const PagesParams p) {
  __shared__ int32_t s_count[kWarps];
  const int rank = (int)ptx::cluster_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* move_of = p.ws + kPagesHeader;
  int begin, end, n;
  segment(p.num_pages, rank * kWarps + warp, &begin, &end);
  const int live = live_before(count_live(p.refs, begin, end, lane), rank, warp, lane, s_count, &n);
  // the pages in use before page n: counted by the warp whose segment n ends or lies in
  if ((n > begin && n <= end) || (n == 0 && rank == 0 && warp == 0)) {
    const int low = n == 0 ? 0 : live + count_live(p.refs, begin, n, lane);
    if (lane == 0) {
      p.ws[0] = n;
      p.ws[1] = low;
      *p.move_count = n - low;
    }
  }
  __threadfence();
  ptx::cluster_sync();
  const int low = __ldcg(p.ws + 1), moves = n - low;
  walk(p.refs, begin, end, lane, [&](int page, int count, int live_in_segment) {
    const int l = live + live_in_segment;                 // pages in use before this one
    if (count <= 0 && page < n) {
      p.move_dst[page - l] = page;
    } else if (count > 0 && page >= n) {
      p.move_src[l - low] = page;
      move_of[page] = l - low;
    }
  });
  __threadfence();
  ptx::cluster_sync();
  for (int k = (rank * kPlanThreads) + threadIdx.x; k < moves; k += kClusterCtas * kPlanThreads) {
    const int from = __ldcg(p.move_src + k), to = __ldcg(p.move_dst + k);
    p.refs[to] = __ldcg(p.refs + from);
    p.refs[from] = 0;
  }
}

// Renumbers the tables after the moves are known: one warp per 32 columns of a row.
__global__ void __launch_bounds__(256) pages_renumber_kernel(const PagesParams p) {
  const int b = blockIdx.x;
  bool bad = false;
  const int n = page_columns(p, __ldg(p.lens + b), &bad);
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) flag(p.err, SMLA_DEVERR_PAGE_STATE);
  const int live = __ldcg(p.ws), moves = live - __ldcg(p.ws + 1);
  const int32_t* move_of = p.ws + kPagesHeader;
  int32_t* row = p.bt + (int64_t)b * p.bt_stride;
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < n; c += gridDim.y * blockDim.x) {
    const int page = row[c];
    if (!in_pool(p, page)) {
      flag(p.err, SMLA_DEVERR_PAGE_STATE);
    } else if (page >= live) {
      // a page that was not in use has no move of its own
      const int k = __ldcg(move_of + page);
      if (k >= 0 && k < moves && __ldcg(p.move_src + k) == page) row[c] = __ldcg(p.move_dst + k);
      else flag(p.err, SMLA_DEVERR_PAGE_STATE);
    }
  }
}

// ------------------------------------------------------------------ copy
// Bandwidth bound: every byte once in, once out.  A unit is 512 consecutive
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
      const int src = __ldg(p.src + m0 + dm), dst = __ldg(p.dst + m0 + dm);
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
  const int64_t moves = min(max(__ldg(p.count), 0), p.capacity);
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

cudaError_t launch_pages_resize(const PagesParams& p, cudaStream_t stream) {
  pages_resize_kernel<<<kClusterCtas, kPlanThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PagesParams& p, cudaStream_t stream) {
  pages_fork_kernel<<<(unsigned)((p.rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesParams& p, cudaStream_t stream) {
  pages_compact_kernel<<<kClusterCtas, kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int cols = (p.max_pages + 255) / 256;
  pages_renumber_kernel<<<dim3((unsigned)p.rows, (unsigned)(cols < 64 ? cols : 64)), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(const CopyParams& p, int sms, cudaStream_t stream) {
  // the number of moves is on the device: the grid is what could be moved, at most what the GPU holds at once
  int64_t pieces = 0;
  for (int k = 0; k < p.num_pools; ++k) pieces += ((int64_t)p.capacity * p.pool[k].pieces + kCopyUnit - 1) / kCopyUnit;
  const int64_t grid = pieces < (int64_t)sms * 16 ? pieces : (int64_t)sms * 16;
  if (grid == 0) return cudaSuccess;
  pages_copy_kernel<<<(unsigned)grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace smla
