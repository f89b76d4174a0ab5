// Slot maps of a step: offsets, positions and physical slots of its new tokens
// from the requests' lengths, and the sparse decode's index table from page
// tables.  Integer arithmetic and look-ups, bound by their latency.  Measured on a
// GB300, both calls, replayed from a graph: 128 tokens with 2048 selected rows 6.2 us;
// 6704 tokens with 512 selected rows 12.8 us, 31 MB read and written.
#include "step.cuh"

namespace smla {
namespace {

__device__ __forceinline__ void flag(int32_t* err, int bit) {
  if (err != nullptr) atomicOr(err, bit);
}

// --------------------------------------------------------------- token slots
// Every CTA sums the requests' new tokens itself, a thousand requests at a time
// (a scan over the CTA; the lengths come out of L2), and looks its own tokens up
// in the offsets; the first one also writes them.
constexpr int kSlotThreads = 1024;

__global__ void __launch_bounds__(kSlotThreads) token_slots_kernel(const TokenSlotsParams p) {
  __shared__ int64_t s_cum[kSlotThreads + 1];
  __shared__ int64_t s_warp[kSlotThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kSlotThreads + threadIdx.x;
  const int64_t last = min((int64_t)(blockIdx.x + 1) * kSlotThreads, (int64_t)p.max_tokens);   // behind the CTA's tokens
  await_prior_kernel();
  admit_next_kernel();
  int request = -1, position = -1;
  int64_t before = 0;                             // new tokens of the requests before this batch of them
  for (int base = 0; base < p.batch && (blockIdx.x == 0 || before < last); base += kSlotThreads) {
    const int b = base + threadIdx.x;
    int64_t n = 0;
    if (b < p.batch) {
      const int32_t old = fetch(p.lens + b), now = fetch(p.new_lens + b);
      if (old < 0 || now < 0) flag(p.err, SMLA_DEVERR_PAGE_STATE);
      n = max(0, max(0, now) - max(0, old));         // (each at least 0: their difference is an int)
    }
    int64_t sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += x;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      int64_t all = s_warp[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, all, d);
        if (lane >= d) all += x;
      }
      s_warp[lane] = all;
    }
    __syncthreads();
    sum += before + (warp > 0 ? s_warp[warp - 1] : 0);
    s_cum[threadIdx.x + 1] = sum;
    if (threadIdx.x == 0) s_cum[0] = before;
    __syncthreads();
    if (blockIdx.x == 0 && b < p.batch) p.cum[b + 1] = (int32_t)min(sum, (int64_t)0x7fffffff);
    if (request < 0 && t < last && t >= s_cum[0] && t < s_cum[kSlotThreads]) {
      int lo = 0, hi = kSlotThreads - 1;          // the last request that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (s_cum[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      request = base + lo;
      position = max(0, fetch(p.lens + request)) + (int)(t - s_cum[lo]);
    }
    before = s_cum[kSlotThreads];
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.cum[0] = 0;
    if (before > p.max_tokens) flag(p.err, SMLA_DEVERR_TOO_MANY_TOKENS);
  }
  if (t >= p.max_tokens) return;
  if (p.requests != nullptr) p.requests[t] = request;
  if (p.positions != nullptr) p.positions[t] = position;
  if (p.slots != nullptr) {
    int64_t slot = -1;
    if (request >= 0) {
      const int column = position / p.page_size;
      const int page = column < p.max_pages ? fetch(p.bt + request * p.bt_stride + column) : -1;
      if (page >= 0) slot = (int64_t)page * p.page_size + (position - column * p.page_size);
      else flag(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
    }
    p.slots[t] = slot;
  }
}

// -------------------------------------------------------------- sparse slots
// kWarps warps a token: its columns, four a lane at a time (one 16-byte store where
// the table's rows allow it).  A CTA of 256 threads a token: 18 us for 6704 tokens of 640
// columns, 7 for 128 of 2176; a warp a token in the first case, sixteen in the second:
// 11.7 and 5.7.
constexpr int kSparseThreads = 512;

// Row of position j >= 0, or -1 (*bad set).
__device__ __forceinline__ int slot_row(const SlotTable& t, const int32_t* row, int j, bool* bad) {
  if (t.shift >= 0) {
    const int column = j >> t.shift;
    const int page = column < t.max_pages ? fetch(row + column) : -1;
    if ((uint32_t)page >> (31 - t.shift) == 0) return page << t.shift | (j & (t.page_size - 1));
  } else {
    const int column = j / t.page_size;
    const int page = column < t.max_pages ? fetch(row + column) : -1;
    const int64_t at = (int64_t)page * t.page_size + (j - column * t.page_size);
    if (page >= 0 && at <= 0x7fffffff) return (int)at;
  }
  *bad = true;
  return -1;
}

template <bool kVector, int kWarps>
__global__ void __launch_bounds__(kSparseThreads, 3) sparse_slots_kernel(const SparseSlotsParams p) {
  __shared__ int s_last[kSparseThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kSparseThreads / 32 / kWarps) + warp / kWarps;
  await_prior_kernel();
  admit_next_kernel();
  if (kWarps < kSparseThreads / 32 && t >= p.sum_q) {
    if constexpr (kWarps > 1) __syncthreads();
    return;
  }
  // the first selected positions, on their way while the request is looked up
  constexpr int kAhead = 2;
  const int columns = kSwaCols + p.num_selected, c0 = (warp % kWarps * 32 + lane) * 4;
  const int32_t* pick = p.selected + t * p.selected_stride - kSwaCols;
  auto select = [&](int c) {
    if (c < kSwaCols || c >= columns) return make_int4(-1, -1, -1, -1);
    if (p.selected == nullptr) return make_int4(c - kSwaCols, c - kSwaCols + 1, c - kSwaCols + 2, c - kSwaCols + 3);
    if (kVector) return *reinterpret_cast<const int4*>(pick + c);
    return make_int4(fetch(pick + c), c + 1 < columns ? fetch(pick + c + 1) : -1, c + 2 < columns ? fetch(pick + c + 2) : -1,
                     c + 3 < columns ? fetch(pick + c + 3) : -1);
  };
  int4 next[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) next[k] = select(c0 + k * kWarps * 128);
  int b, first, count;
  if (p.cum != nullptr) {
    b = last_request(p.batch, lane, [&](int x) { return fetch(p.cum + x) <= t; });
    first = fetch(p.cum + b);
    count = fetch(p.cum + b + 1) - first;
  } else {
    count = p.sum_q / p.batch;
    b = t / count;
    first = b * count;
  }
  const bool owned = t >= first && t - first < count;
  const int pos = owned ? max(0, fetch(p.seq_lens + b)) - count + (t - first) : -1;
  const int lo = max(0, pos - (kSwaCols - 1));
  const int limit = pos >= 0 ? (int)(((int64_t)pos + 1) / p.ratio) : 0;
  const int32_t* swa = p.swa.bt + b * p.swa.stride;
  const int32_t* comp = p.comp.bt + b * p.comp.stride;
  int32_t* out = p.out + t * p.out_stride;
  int last = 0;
  bool bad = false;
  auto rows = [&](int at, int4 q) {               // four columns from `at` on
    if (at >= columns) return;
    int v[4], c[4] = {q.x, q.y, q.z, q.w};
    const bool window = at < kSwaCols;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (window) c[e] = lo + at + e <= pos ? lo + at + e : -1;
      const bool seen = c[e] >= 0 && (window || (c[e] < limit && at + e < columns));
      v[e] = seen ? slot_row(window ? p.swa : p.comp, window ? swa : comp, c[e], &bad) : -1;
      if (!window && v[e] >= 0) last = max(last, at + e + 1 - kSwaCols);
    }
    if (kVector) {
      *reinterpret_cast<int4*>(out + at) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at + e < columns) out[at + e] = v[e];
    }
  };
  for (int base = c0; base < columns; base += kAhead * kWarps * 128) {
    int4 now[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) now[k] = next[k];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) next[k] = select(base + (kAhead + k) * kWarps * 128);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) rows(base + k * kWarps * 128, now[k]);
  }
  if (bad) flag(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
  last = __reduce_max_sync(0xffffffffu, last);
  if constexpr (kWarps > 1) {
    if (lane == 0) s_last[warp] = last;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) last = max(last, s_last[warp / kWarps * kWarps + w]);
  }
  if (warp % kWarps == 0 && lane == 0) p.topk[t] = pos >= 0 ? kSwaCols + last : 0;
}

}  // namespace

cudaError_t launch_token_slots(const TokenSlotsParams& p, cudaStream_t stream) {
  const unsigned ctas = (unsigned)(((int64_t)p.max_tokens + kSlotThreads - 1) / kSlotThreads);
  return launch_overlapped(token_slots_kernel, dim3(ctas > 0 ? ctas : 1), kSlotThreads, 0, stream, p);
}

cudaError_t launch_sparse_slots(const SparseSlotsParams& p, int sms, cudaStream_t stream) {
  auto whole = [](const void* at, int64_t stride) { return reinterpret_cast<uintptr_t>(at) % 16 == 0 && stride % 4 == 0; };
  const bool vector = p.num_selected % 4 == 0 && whole(p.out, p.out_stride) &&
                      (p.selected == nullptr || whole(p.selected, p.selected_stride));
  // as many warps a token as its columns feed and the GPU holds at once
  auto launch = [&](auto kernel, int warps) {
    const int each = kSparseThreads / 32 / warps;
    return launch_overlapped(kernel, dim3((unsigned)((p.sum_q + each - 1) / each)), kSparseThreads, 0, stream, p);
  };
  const int chunks = (kSwaCols + p.num_selected + 127) / 128;
  const int64_t room = (int64_t)sms * 64;
  if (chunks > 8 && p.sum_q * 16ll <= room)
    return vector ? launch(sparse_slots_kernel<true, 16>, 16) : launch(sparse_slots_kernel<false, 16>, 16);
  if (chunks > 2 && p.sum_q * 4ll <= room)
    return vector ? launch(sparse_slots_kernel<true, 4>, 4) : launch(sparse_slots_kernel<false, 4>, 4);
  return vector ? launch(sparse_slots_kernel<true, 1>, 1) : launch(sparse_slots_kernel<false, 1>, 1);
}

}  // namespace smla
