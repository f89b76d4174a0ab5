// Host side of the paged latent cache: argument checks, the split planner of
// the window attention, launches.  Shapes and pointers are checked before any
// CUDA call; no device memory is read, nothing is allocated, nothing
// synchronises.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "cache.cuh"
#include "kernels.h"

namespace smla {
namespace {

static_assert(SMLA_MAX_SPLITS <= kMaxWindowSplits, "forced splits");

smla_status fail(smla_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
smla_status fail(smla_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return record_error(st, buf);
}

#define SMLA_TRY(expr)                  \
  do {                                  \
    smla_status st_ = (expr);           \
    if (st_ != SMLA_OK) return st_;     \
  } while (0)

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

smla_status need_words(const char* name, const void* ptr, bool required) {
  if (ptr == nullptr) return required ? fail(SMLA_ERR_INVALID_ARG, "%s is required", name) : SMLA_OK;
  if (!aligned(ptr, 4)) return fail(SMLA_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return SMLA_OK;
}

smla_status need_rows(const char* name, const void* ptr) {
  if (ptr == nullptr) return fail(SMLA_ERR_INVALID_ARG, "%s is required", name);
  if (!aligned(ptr, 16)) return fail(SMLA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return SMLA_OK;
}

std::atomic<int> g_sms[64];   // per device; 0 = not queried yet

smla_status device_sms(int device, int* out) {
  if (device < 0 || device >= 64) return fail(SMLA_ERR_INVALID_ARG, "device %d out of range", device);
  int n = g_sms[device].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    g_sms[device].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return SMLA_OK;
}

smla_status current_sms(int* out) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  return device_sms(device, out);
}

smla_status launched(const char* what, cudaError_t e) {
  if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return SMLA_OK;
}

// ------------------------------------------------------------------ cache

smla_status check_cache(const smla_cache& c, int32_t sum_q) {
  if (sum_q < 0) return fail(SMLA_ERR_INVALID_ARG, "sum_q %d is negative", sum_q);
  if (c.batch < 1) return fail(SMLA_ERR_INVALID_ARG, "batch %d < 1", c.batch);
  if (c.cum_seq_lens_q == nullptr && sum_q % c.batch != 0)
    return fail(SMLA_ERR_INVALID_ARG, "sum_q %d is not a multiple of batch %d (pass cum_seq_lens_q)", sum_q, c.batch);
  if (c.num_pages < 1 || c.num_pages > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "num_pages %lld is outside 1 .. 2^31 - 1", (long long)c.num_pages);
  if (c.page_size < 8 || c.page_size % 8 != 0 || c.page_size > (1 << 20))
    return fail(SMLA_ERR_INVALID_ARG, "page_size %d is not a multiple of 8 of at most 2^20", c.page_size);
  if (c.block_rows < 1 || c.page_size % c.block_rows != 0)
    return fail(SMLA_ERR_INVALID_ARG, "block_rows %d does not divide page_size %d", c.block_rows, c.page_size);
  if (c.max_pages < 1 || (int64_t)c.max_pages * c.page_size > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "max_pages %d: a request holds 1 .. 2^31 - 1 tokens", c.max_pages);
  if (c.row_stride != 0 && (c.row_stride < kHeadDim || c.row_stride % 16 != 0))
    return fail(SMLA_ERR_INVALID_ARG, "row_stride %lld: at least %d bytes, a multiple of 16", (long long)c.row_stride,
                kHeadDim);
  const int64_t row = c.row_stride ? c.row_stride : kHeadDim;
  if (row > (1ll << 36)) return fail(SMLA_ERR_UNSUPPORTED, "row_stride %lld is too large", (long long)row);
  if (c.page_stride != 0 && (c.page_stride < (c.page_size - 1) * row + kHeadDim || c.page_stride % 16 != 0))
    return fail(SMLA_ERR_INVALID_ARG, "page_stride %lld: at least a page's bytes, a multiple of 16",
                (long long)c.page_stride);
  const int64_t page = c.page_stride ? c.page_stride : c.page_size * row;
  if (page >= (1ll << 40) || 8 * row >= (1ll << 40))
    return fail(SMLA_ERR_UNSUPPORTED, "page_stride %lld: pages are under 2^40 bytes apart", (long long)page);
  if (c.scale_stride != 0 && c.scale_stride < c.page_size / c.block_rows)
    return fail(SMLA_ERR_INVALID_ARG, "scale_stride %lld is less than a page's %d scales", (long long)c.scale_stride,
                c.page_size / c.block_rows);
  if (c.block_table_stride != 0 && c.block_table_stride < c.max_pages)
    return fail(SMLA_ERR_INVALID_ARG, "block_table_stride %lld < max_pages %d", (long long)c.block_table_stride,
                c.max_pages);
  return SMLA_OK;
}

smla_status check_cache_pointers(const smla_cache& c) {
  SMLA_TRY(need_rows("rows", c.rows));
  SMLA_TRY(need_words("scales", c.scales, true));
  SMLA_TRY(need_words("block_tables", c.block_tables, true));
  SMLA_TRY(need_words("seq_lens", c.seq_lens, true));
  return need_words("cum_seq_lens_q", c.cum_seq_lens_q, false);
}

CacheView view(const smla_cache& c, int32_t sum_q) {
  CacheView v;
  memset(&v, 0, sizeof(v));
  v.rows = static_cast<uint8_t*>(c.rows);
  v.row_stride = c.row_stride ? c.row_stride : kHeadDim;
  v.page_stride = c.page_stride ? c.page_stride : c.page_size * v.row_stride;
  v.scales = c.scales;
  v.scale_stride = c.scale_stride ? c.scale_stride : c.page_size / c.block_rows;
  v.num_pages = (int32_t)c.num_pages;
  v.page_size = c.page_size;
  v.block_rows = c.block_rows;
  v.bt = c.block_tables;
  v.bt_stride = c.block_table_stride ? c.block_table_stride : c.max_pages;
  v.max_pages = c.max_pages;
  v.batch = c.batch;
  v.seq_lens = c.seq_lens;
  v.cum = c.cum_seq_lens_q;
  v.sum_q = sum_q;
  return v;
}

// ----------------------------------------------------------------- window

smla_status check_window(const smla_window_args* a) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  SMLA_TRY(check_cache(a->cache, a->sum_q));
  if (a->num_heads < 1 || a->num_heads > 128)
    return fail(SMLA_ERR_UNSUPPORTED, "num_heads %d is outside 1 .. 128", a->num_heads);
  if (a->window < 1) return fail(SMLA_ERR_INVALID_ARG, "window %d < 1", a->window);
  if (a->first_tokens < 0) return fail(SMLA_ERR_INVALID_ARG, "first_tokens %d is negative", a->first_tokens);
  if (a->q_stride_token != 0 && (a->q_stride_token < (int64_t)a->num_heads * kHeadDim || a->q_stride_token % 8 != 0))
    return fail(SMLA_ERR_INVALID_ARG, "q_stride_token %lld: at least H * 512 elements, a multiple of 8",
                (long long)a->q_stride_token);
  if (a->num_splits < 0 || a->num_splits > SMLA_MAX_SPLITS)
    return fail(SMLA_ERR_INVALID_ARG, "num_splits %d is outside 0 .. %d", a->num_splits, SMLA_MAX_SPLITS);
  return SMLA_OK;
}

int head_groups(const smla_window_args* a) { return (a->num_heads + kWindowHeads - 1) / kWindowHeads; }

// How the (token, head group) pairs are worked through: the first `whole` each by
// one CTA, the others in `splits` ranges of their tiles that a second kernel
// merges.  Shapes only.
struct WindowPlan {
  int64_t whole, units;
  int splits;
  size_t lse, bytes;   // workspace: offset of the partials' LSEs, all of it
};

// Splits that cost `pairs` pairs of `tiles` tiles least on `sms` SMs, one CTA each
// at a time.  Measured on a GB300, a tile costs a CTA 2.5 us, and a second split
// the merge: 1.3 tiles' time and a 7000th of one for each partial row of 512 values
// (1 token x 64 heads, 2 tiles: 12.3 us whole, 12.9 in two; 3 tiles: 15.8 against
// 13.5 in three; 32 x 128, 5 tiles: 22.5 against 24.2 in two, 9: 33.2 against 30.0).
int cheapest_splits(int64_t pairs, int64_t tiles, int sms) {
  const int64_t most = std::min<int64_t>({sms / pairs, tiles, kMaxWindowSplits});
  int best = 1;
  double cost = (double)tiles;
  for (int64_t s = 2; s <= most; ++s) {
    const double c = (double)((tiles + s - 1) / s) + 1.3 + (double)pairs * kWindowHeads * s / 7000.0;
    if (c < cost) {
      cost = c;
      best = (int)s;
    }
  }
  return best;
}

WindowPlan window_plan(const smla_window_args* a, int sms) {
  WindowPlan w;
  const int64_t pairs = (int64_t)a->sum_q * head_groups(a);
  if (a->num_splits > 0) {
    w.splits = a->num_splits;
    w.whole = w.splits > 1 ? 0 : pairs;
  } else {
    const int64_t page = a->cache.page_size, chunk = page % 32 == 0 ? 32 : page % 16 == 0 ? 16 : 8;   // rows of a box
    const int64_t all = ((int64_t)a->cache.max_pages * page + chunk - 1) / chunk;
    const int64_t seen = ((int64_t)a->window + chunk - 2) / chunk + 1 + ((int64_t)a->first_tokens + chunk - 1) / chunk;
    const int64_t tiles = (std::min(all, seen) * chunk + kWindowTile - 1) / kWindowTile;
    // The pairs of the last, partly filled turn of the SMs are the ones worth splitting (160 pairs of 9 tiles: 61 us
    // whole, 49 so; 772: 182 and 171; 1232 of 5: 170.5 and 168.5).  Behind more turns they are a small part, and the
    // kernel with splits is 3 % slower (1864 of 5: 240 us whole, 243 so; 2448: 305 and 307; of 9: 382 and 372, 485 and 479).
    const int64_t rest = pairs % sms;
    w.splits = rest > 0 && pairs < 10 * (int64_t)sms ? cheapest_splits(rest, tiles, sms) : 1;
    w.whole = w.splits > 1 ? pairs - rest : pairs;
  }
  w.units = w.whole + (pairs - w.whole) * w.splits;
  const size_t rows = (size_t)(pairs - w.whole) * w.splits * kWindowHeads;
  w.lse = align_up(rows * kHeadDim * sizeof(float), 256);
  w.bytes = w.lse + align_up(rows * sizeof(float), 256);
  return w;
}

// ------------------------------------------------------------------ pages

smla_status check_pages(const smla_pages_args* a) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0) return fail(SMLA_ERR_INVALID_ARG, "rows %d is negative", a->rows);
  if (a->max_pages < 1) return fail(SMLA_ERR_INVALID_ARG, "max_pages %d < 1", a->max_pages);
  if (a->page_size < 1) return fail(SMLA_ERR_INVALID_ARG, "page_size %d < 1", a->page_size);
  if ((int64_t)a->max_pages * a->page_size > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "max_pages %d: a request holds 1 .. 2^31 - 1 tokens", a->max_pages);
  if ((int64_t)a->rows * ((int64_t)a->max_pages + 1) > 0x3fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "%d rows of %d pages: the tables hold under 2^30 entries", a->rows, a->max_pages);
  if (a->num_pages < 1 || a->num_pages > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "num_pages %lld is outside 1 .. 2^31 - 1", (long long)a->num_pages);
  if (a->block_table_stride != 0 && a->block_table_stride < a->max_pages)
    return fail(SMLA_ERR_INVALID_ARG, "block_table_stride %lld < max_pages %d", (long long)a->block_table_stride,
                a->max_pages);
  return SMLA_OK;
}

size_t pages_workspace(const smla_pages_args* a) {
  return align_up((size_t)pages_workspace_words(a->rows, a->num_pages) * sizeof(int32_t), 256);
}

smla_status check_page_pointers(const smla_pages_args* a) {
  SMLA_TRY(need_words("block_tables", a->block_tables, true));
  SMLA_TRY(need_words("ref_counts", a->ref_counts, true));
  SMLA_TRY(need_words("lens", a->lens, true));
  return need_words("error_word", a->error_word, false);
}

smla_status check_moves(const smla_pages_args* a, int64_t need) {
  if (a->move_capacity < need || a->move_capacity > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "move_capacity %lld: this call may write %lld moves", (long long)a->move_capacity,
                (long long)need);
  if (need > 0) {
    SMLA_TRY(need_words("move_src", a->move_src, true));
    SMLA_TRY(need_words("move_dst", a->move_dst, true));
  }
  SMLA_TRY(need_words("move_count", a->move_count, true));
  const size_t bytes = pages_workspace(a);
  if (a->workspace == nullptr || a->workspace_bytes < bytes)
    return fail(SMLA_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes given, %zu needed",
                a->workspace ? a->workspace_bytes : (size_t)0, bytes);
  if (!aligned(a->workspace, 256)) return fail(SMLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return SMLA_OK;
}

// A call without requests: what a copy of its moves would find.
smla_status no_moves(const smla_pages_args* a, void* stream) {
  SMLA_TRY(need_words("move_count", a->move_count, true));
  const cudaError_t e = cudaMemsetAsync(a->move_count, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "move_count: %s", cudaGetErrorString(e));
  return SMLA_OK;
}

PagesParams pages_params(const smla_pages_args* a) {
  PagesParams p;
  memset(&p, 0, sizeof(p));
  p.bt = a->block_tables;
  p.bt_stride = a->block_table_stride ? a->block_table_stride : a->max_pages;
  p.rows = a->rows;
  p.max_pages = a->max_pages;
  p.page_size = a->page_size;
  p.num_pages = (int32_t)a->num_pages;
  p.refs = a->ref_counts;
  p.lens = a->lens;
  p.new_lens = a->new_lens;
  p.parents = a->parents;
  p.out_lens = a->out_lens;
  p.move_src = a->move_src;
  p.move_dst = a->move_dst;
  p.move_count = a->move_count;
  p.ws = static_cast<int32_t*>(a->workspace);
  p.err = a->error_word;
  return p;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

smla_status smla_window_workspace_size(const smla_window_args* args, int device, size_t* bytes) {
  if (bytes == nullptr) return fail(SMLA_ERR_INVALID_ARG, "bytes is NULL");
  SMLA_TRY(check_window(args));
  int sms = 0;
  SMLA_TRY(device_sms(device, &sms));
  *bytes = window_plan(args, sms).bytes;
  return SMLA_OK;
}

smla_status smla_window_attention(const smla_window_args* a, void* stream) {
  SMLA_TRY(check_window(a));
  if (a->sum_q == 0) return SMLA_OK;
  SMLA_TRY(check_cache_pointers(a->cache));
  SMLA_TRY(need_rows("q", a->q));
  SMLA_TRY(need_rows("out", a->out));
  SMLA_TRY(need_words("out_lse", a->out_lse, false));
  SMLA_TRY(need_words("sinks", a->sinks, false));
  SMLA_TRY(need_words("bmm1_scale_dev", a->bmm1_scale_dev, false));
  SMLA_TRY(need_words("bmm2_scale_dev", a->bmm2_scale_dev, false));
  SMLA_TRY(need_words("error_word", a->error_word, false));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  const WindowPlan plan = window_plan(a, sms);
  if (plan.units > 0x7fffffff || (int64_t)a->sum_q * head_groups(a) > 0x7fffffff / kWindowHeads)
    return fail(SMLA_ERR_UNSUPPORTED, "%lld units are too many", (long long)plan.units);
  if (plan.bytes > 0) {
    if (a->workspace == nullptr || a->workspace_bytes < plan.bytes)
      return fail(SMLA_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes given, %zu needed",
                  a->workspace ? a->workspace_bytes : (size_t)0, plan.bytes);
    if (!aligned(a->workspace, 256)) return fail(SMLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  WindowParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(a->cache, a->sum_q);
  p.H = a->num_heads;
  p.window = a->window;
  p.first_tokens = a->first_tokens;
  p.whole = (int32_t)plan.whole;
  p.num_splits = plan.splits;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.q_stride_token = a->q_stride_token ? a->q_stride_token : (int64_t)a->num_heads * kHeadDim;
  p.sinks = a->sinks;
  p.bmm1 = a->bmm1_scale;
  p.bmm2 = a->bmm2_scale;
  p.bmm1_dev = a->bmm1_scale_dev;
  p.bmm2_dev = a->bmm2_scale_dev;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.out_lse = a->out_lse;
  p.err = a->error_word;
  if (plan.bytes > 0) {
    p.part_o = static_cast<float*>(a->workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + plan.lse);
  }
  return launched("window attention", launch_window_attention(p, sms, static_cast<cudaStream_t>(stream)));
}

smla_status smla_cache_append(const smla_append_args* a, void* stream) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  SMLA_TRY(check_cache(a->cache, a->sum_q));
  if (a->latent_stride != 0 && (a->latent_stride < kHeadDim || a->latent_stride % 8 != 0))
    return fail(SMLA_ERR_INVALID_ARG, "latent_stride %lld: at least %d elements, a multiple of 8",
                (long long)a->latent_stride, kHeadDim);
  if (a->sum_q == 0) return SMLA_OK;
  SMLA_TRY(check_cache_pointers(a->cache));
  SMLA_TRY(need_rows("latent", a->latent));
  SMLA_TRY(need_words("error_word", a->error_word, false));
  AppendParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(a->cache, a->sum_q);
  p.latent = static_cast<const __nv_bfloat16*>(a->latent);
  p.latent_stride = a->latent_stride ? a->latent_stride : kHeadDim;
  p.err = a->error_word;
  if ((int64_t)a->sum_q / p.c.block_rows + 2 * (int64_t)p.c.batch > 0x7fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "%d tokens of %d requests: the grid is too large", a->sum_q, p.c.batch);
  return launched("append", launch_cache_append(p, static_cast<cudaStream_t>(stream)));
}

smla_status smla_pages_workspace_size(const smla_pages_args* args, size_t* bytes) {
  if (bytes == nullptr) return fail(SMLA_ERR_INVALID_ARG, "bytes is NULL");
  SMLA_TRY(check_pages(args));
  *bytes = pages_workspace(args);
  return SMLA_OK;
}

smla_status smla_pages_resize(const smla_pages_args* a, void* stream) {
  SMLA_TRY(check_pages(a));
  if (a->rows == 0) return no_moves(a, stream);
  SMLA_TRY(check_page_pointers(a));
  SMLA_TRY(need_words("new_lens", a->new_lens, true));
  SMLA_TRY(check_moves(a, a->rows));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  return launched("pages resize", launch_pages_resize(pages_params(a), sms, static_cast<cudaStream_t>(stream)));
}

smla_status smla_pages_fork(const smla_pages_args* a, void* stream) {
  SMLA_TRY(check_pages(a));
  if (a->rows == 0) return SMLA_OK;
  SMLA_TRY(check_page_pointers(a));
  SMLA_TRY(need_words("parents", a->parents, true));
  SMLA_TRY(need_words("out_lens", a->out_lens, true));
  const uintptr_t out = reinterpret_cast<uintptr_t>(a->out_lens), in = reinterpret_cast<uintptr_t>(a->lens);
  if ((out > in ? out - in : in - out) < (uintptr_t)a->rows * sizeof(int32_t))
    return fail(SMLA_ERR_INVALID_ARG, "out_lens must not be lens or overlap it");
  return launched("pages fork", launch_pages_fork(pages_params(a), static_cast<cudaStream_t>(stream)));
}

smla_status smla_pages_compact(const smla_pages_args* a, void* stream) {
  SMLA_TRY(check_pages(a));
  if (a->rows == 0) return no_moves(a, stream);
  SMLA_TRY(check_page_pointers(a));
  SMLA_TRY(check_moves(a, a->num_pages / 2));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  return launched("pages compact", launch_pages_compact(pages_params(a), sms, static_cast<cudaStream_t>(stream)));
}

smla_status smla_pages_copy(const smla_pool* pools, int32_t num_pools, int64_t num_pages, const int32_t* move_src,
                            const int32_t* move_dst, const int32_t* move_count, int64_t move_capacity,
                            int32_t* error_word, void* stream) {
  if (num_pools < 0) return fail(SMLA_ERR_INVALID_ARG, "num_pools %d is negative", num_pools);
  if (num_pages < 1 || num_pages > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "num_pages %lld is outside 1 .. 2^31 - 1", (long long)num_pages);
  if (move_capacity < 0 || move_capacity > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "move_capacity %lld is outside 0 .. 2^31 - 1", (long long)move_capacity);
  if (num_pools == 0 || move_capacity == 0) return SMLA_OK;
  if (pools == nullptr) return fail(SMLA_ERR_INVALID_ARG, "pools is NULL");
  for (int i = 0; i < num_pools; ++i) {
    const smla_pool& q = pools[i];
    if (q.base == nullptr) return fail(SMLA_ERR_INVALID_ARG, "pool %d has no base", i);
    if (q.page_bytes < 1 || q.page_bytes > 0x7fffffff)
      return fail(SMLA_ERR_INVALID_ARG, "pool %d: page_bytes %lld is outside 1 .. 2^31 - 1", i, (long long)q.page_bytes);
    if (q.page_stride < q.page_bytes)
      return fail(SMLA_ERR_INVALID_ARG, "pool %d: page_stride %lld < page_bytes %lld", i, (long long)q.page_stride,
                  (long long)q.page_bytes);
  }
  SMLA_TRY(need_words("move_src", move_src, true));
  SMLA_TRY(need_words("move_dst", move_dst, true));
  SMLA_TRY(need_words("move_count", move_count, true));
  SMLA_TRY(need_words("error_word", error_word, false));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  for (int at = 0; at < num_pools; at += kCopyPools) {
    CopyParams p;
    memset(&p, 0, sizeof(p));
    p.num_pools = std::min(num_pools - at, kCopyPools);
    for (int i = 0; i < p.num_pools; ++i) {
      const smla_pool& q = pools[at + i];
      const uint64_t all = reinterpret_cast<uintptr_t>(q.base) | (uint64_t)q.page_bytes | (uint64_t)q.page_stride;
      p.pool[i].vec = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
      p.pool[i].base = static_cast<uint8_t*>(q.base);
      p.pool[i].stride = q.page_stride;
      p.pool[i].pieces = (int32_t)(q.page_bytes / p.pool[i].vec);
    }
    p.num_pages = (int32_t)num_pages;
    p.src = move_src;
    p.dst = move_dst;
    p.count = move_count;
    p.capacity = (int32_t)move_capacity;
    p.err = error_word;
    SMLA_TRY(launched("pages copy", launch_pages_copy(p, sms, static_cast<cudaStream_t>(stream))));
  }
  return SMLA_OK;
}

}  // extern "C"
