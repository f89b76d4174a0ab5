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

constexpr int kWindowHeads = 64;      // heads of one token that a CTA takes
constexpr int kWindowTile = 128;      // cache rows of one tile
constexpr int kMaxWindowSplits = 256;

cudaError_t launch_window_attention(const WindowParams& p, int sms, cudaStream_t stream);

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
