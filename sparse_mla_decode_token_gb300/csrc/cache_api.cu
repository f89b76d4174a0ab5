// Host side of the paged latent cache: argument checks, the split planner of
// the window attention, launches.  Shapes and pointers are checked before any
// CUDA call; no device memory is read, nothing is allocated, nothing
// synchronises.
#include <string.h>

#include <algorithm>

#include "api_checks.h"
#include "cache.cuh"

namespace smla {
namespace {

static_assert(SMLA_MAX_SPLITS <= kMaxWindowSplits, "forced splits");

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

// What the two attention calls have alike.
template <class Args>
smla_status check_attention(const Args* a) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  SMLA_TRY(check_cache(a->cache, a->sum_q));
  if (a->num_heads < 1 || a->num_heads > 128)
    return fail(SMLA_ERR_UNSUPPORTED, "num_heads %d is outside 1 .. 128", a->num_heads);
  if (a->q_stride_token != 0 && (a->q_stride_token < (int64_t)a->num_heads * kHeadDim || a->q_stride_token % 8 != 0))
    return fail(SMLA_ERR_INVALID_ARG, "q_stride_token %lld: at least H * 512 elements, a multiple of 8",
                (long long)a->q_stride_token);
  return SMLA_OK;
}

template <class Args>
smla_status check_attention_pointers(const Args* a) {
  SMLA_TRY(check_cache_pointers(a->cache));
  SMLA_TRY(need_rows("q", a->q));
  SMLA_TRY(need_rows("out", a->out));
  SMLA_TRY(need_words("out_lse", a->out_lse, false));
  SMLA_TRY(need_words("sinks", a->sinks, false));
  SMLA_TRY(need_words("bmm1_scale_dev", a->bmm1_scale_dev, false));
  SMLA_TRY(need_words("bmm2_scale_dev", a->bmm2_scale_dev, false));
  return need_words("error_word", a->error_word, false);
}

template <class Args>
WindowParams attention_params(const Args* a) {
  WindowParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(a->cache, a->sum_q);
  p.H = a->num_heads;
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
  return p;
}

smla_status check_window(const smla_window_args* a) {
  SMLA_TRY(check_attention(a));
  if (a->window < 1) return fail(SMLA_ERR_INVALID_ARG, "window %d < 1", a->window);
  if (a->first_tokens < 0) return fail(SMLA_ERR_INVALID_ARG, "first_tokens %d is negative", a->first_tokens);
  if (a->num_splits < 0 || a->num_splits > SMLA_MAX_SPLITS)
    return fail(SMLA_ERR_INVALID_ARG, "num_splits %d is outside 0 .. %d", a->num_splits, SMLA_MAX_SPLITS);
  return SMLA_OK;
}

template <class Args>
int head_groups(const Args* a) { return (a->num_heads + kWindowHeads - 1) / kWindowHeads; }

// How the (token, head group) pairs are worked through: the first `whole` each by
// one CTA, the others in `splits` ranges of their tiles that a second kernel
// merges.  Shapes only.
struct WindowPlan {
  int64_t whole, units;
  int splits;
  size_t lse, bytes;   // workspace: offset of the partials' LSEs, all of it
};

int64_t most_splits(int64_t pairs, int64_t tiles, int sms) {
  return std::min<int64_t>({sms / pairs, tiles, kMaxWindowSplits});
}
// Splits that cost `pairs` pairs of `tiles` tiles least on `sms` SMs, one CTA each
// at a time.  Measured on a GB300, a tile costs a CTA 2.5 us, and a second split
// the merge: 1.3 tiles' time and a 7000th of one for each partial row of 512 values
// (1 token x 64 heads, 2 tiles: 12.3 us whole, 12.9 in two; 3 tiles: 15.8 against
// 13.5 in three; 32 x 128, 5 tiles: 22.5 against 24.2 in two, 9: 33.2 against 30.0).
int cheapest_splits(int64_t pairs, int64_t tiles, int sms) {
  const int64_t most = most_splits(pairs, tiles, sms);
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

// fp32 values, `each` for every row of so many partials.
size_t parts_bytes(int64_t parts, int each) {
  return align_up((size_t)parts * kWindowHeads * each * sizeof(float), 256);
}

// Pairs of up to `tiles` tiles, in `splits` if that is not 0.
WindowPlan pair_plan(int64_t pairs, int64_t tiles, int splits, int sms) {
  WindowPlan w;
  if (splits > 0) {
    w.splits = splits;
    w.whole = w.splits > 1 ? 0 : pairs;
  } else {
    // The pairs of the last, partly filled turn of the SMs are the ones worth splitting (160 pairs of 9 tiles: 61 us
    // whole, 49 so; 772: 182 and 171; 1232 of 5: 170.5 and 168.5).  Behind more turns they are a small part, and the
    // kernel with splits is 3 % slower (1864 of 5: 240 us whole, 243 so; 2448: 305 and 307; of 9: 382 and 372, 485 and 479).
    const int64_t rest = pairs % sms;
    w.splits = rest > 0 && pairs < 10 * (int64_t)sms ? cheapest_splits(rest, tiles, sms) : 1;
    w.whole = w.splits > 1 ? pairs - rest : pairs;
  }
  w.units = w.whole + (pairs - w.whole) * w.splits;
  const int64_t parts = (pairs - w.whole) * w.splits;
  w.lse = parts_bytes(parts, kHeadDim);
  w.bytes = w.lse + parts_bytes(parts, 1);
  return w;
}

// Workspace of every such plan of at most so many pairs and tiles: one that is sized
// for a server's largest step serves the smaller ones, which may be split more.
size_t pair_workspace(int64_t pairs, int64_t tiles, int splits, int sms) {
  if (splits > 0) return pair_plan(pairs, tiles, splits, sms).bytes;
  int64_t parts = 0;
  for (int64_t rest = 1; rest <= std::min<int64_t>(pairs, sms - 1); ++rest) {
    const int64_t most = most_splits(rest, tiles, sms);
    if (most > 1) parts = std::max(parts, rest * most);
  }
  return parts_bytes(parts, kHeadDim) + parts_bytes(parts, 1);
}

// Rows of a page's boxes that a request may hold, and the tiles of `rows` of them.
int64_t box_rows(const smla_cache& c) { return 1ll << cache_box_shift(c.page_size); }
int64_t table_chunks(const smla_cache& c) { return ((int64_t)c.max_pages * c.page_size + box_rows(c) - 1) / box_rows(c); }
int64_t chunk_tiles(const smla_cache& c, int64_t chunks) { return (chunks * box_rows(c) + kWindowTile - 1) / kWindowTile; }

template <class Args>
int64_t pairs_of(const Args* a) { return (int64_t)a->sum_q * head_groups(a); }

int64_t window_tiles(const smla_window_args* a) {
  const int64_t chunk = box_rows(a->cache);
  const int64_t seen = ((int64_t)a->window + chunk - 2) / chunk + 1 + ((int64_t)a->first_tokens + chunk - 1) / chunk;
  return chunk_tiles(a->cache, std::min(table_chunks(a->cache), seen));
}

WindowPlan window_plan(const smla_window_args* a, int sms) {
  return pair_plan(pairs_of(a), window_tiles(a), a->num_splits, sms);
}

void set_parts(WindowParams* p, const WindowPlan& plan, void* workspace) {
  p->whole = (int32_t)plan.whole;
  p->num_splits = plan.splits;
  if (plan.bytes == 0) return;
  p->part_o = static_cast<float*>(workspace);
  p->part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.lse);
}

// ----------------------------------------------------------------- prefix

smla_status check_prefix(const smla_prefix_args* a) {
  SMLA_TRY(check_attention(a));
  if (a->num_groups < 0) return fail(SMLA_ERR_INVALID_ARG, "num_groups %d is negative", a->num_groups);
  if ((int64_t)a->num_groups + a->sum_q > 0x3fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "%d groups of %d tokens are too many", a->num_groups, a->sum_q);
  return SMLA_OK;
}

// Prefixes are computed once for a group's tokens where that can save more than the
// plan and the merge cost: 6 tiles an SM, by what the tables allow.  Measured on a GB300
// (shared, each by itself): 64 tokens of 8 heads over 1300 rows 29.1 us and 26.4 (4.1
// tiles an SM saved), over 2500 29.6 and 35.4 (7.4); of 32 heads over 2500 37.5 and 37.6
// (4.2), over 4900 51.0 and 57.9 (8.2); 16 of 32 heads over 16000 48.3 and 46.7 (6.6).
// Those tables were about as wide as the requests are long; the lengths are on the
// device, so short requests of wide tables are shared, too (4 samples of 16 heads behind
// 510 tokens: 14.0 us on tables of 10 pages, 22.8 on tables of 1024).
constexpr double kSavedTiles = 6;
bool shares_prefixes(const smla_prefix_args* a, int sms) {
  if (a->num_groups == 0) return false;
  const double empty = head_groups(a) - (double)a->num_heads / kWindowHeads;   // of a token's blocks of 64 rows
  return a->sum_q * empty * (double)chunk_tiles(a->cache, table_chunks(a->cache)) > kSavedTiles * sms;
}

// Else each token by itself: a list has a chunk more, where the prefix ends within one.
int64_t grouped_tiles(const smla_prefix_args* a) { return chunk_tiles(a->cache, table_chunks(a->cache) + 1); }
WindowPlan grouped_plan(const smla_prefix_args* a, int sms) { return pair_plan(pairs_of(a), grouped_tiles(a), 0, sms); }

// The workspace's parts: fp32 partials (two for each SM; where prefixes are shared, one
// more for each block of 64 rows and each cut through them), then the plan.
struct PrefixLayout {
  int64_t parts;
  int shares;
  size_t lse, header, cost_of, unit_of, shared_of, share, first, group, token, prefix_of, limit, lead, bytes;
};
PrefixLayout prefix_layout(const smla_prefix_args* a, int sms) {
  const int64_t T = a->sum_q, heads = (a->num_heads + kWindowHeads - 1) / kWindowHeads;
  PrefixLayout l;
  l.shares = std::min(sms, kMaxShares);
  l.parts = 3 * (int64_t)l.shares + T * heads + T * a->num_heads / kWindowHeads + a->num_groups;
  const size_t rows = (size_t)l.parts * kWindowHeads, segments = (size_t)a->num_groups + T;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t from = at;
    at = align_up(at + bytes, 256);
    return from;
  };
  take(rows * kHeadDim * sizeof(float));
  l.lse = take(rows * sizeof(float));
  l.header = take(2 * sizeof(int64_t) + sizeof(int32_t));
  l.cost_of = take((segments + 1) * sizeof(int64_t));
  l.unit_of = take((segments + 1) * sizeof(int32_t));
  l.shared_of = take(segments * sizeof(int32_t));
  l.share = take((size_t)l.shares * sizeof(int4));
  l.first = take((size_t)l.shares * 4 * sizeof(int4));
  l.group = take((size_t)a->num_groups * sizeof(int4));
  l.token = take((size_t)T * sizeof(int4));
  l.prefix_of = take((size_t)T * sizeof(int4));
  l.limit = take((size_t)a->num_groups * sizeof(int32_t));
  l.lead = take((size_t)a->num_groups * sizeof(int32_t));
  l.bytes = at;
  return l;
}

// ------------------------------------------------------------------ pages

smla_status check_tables(const smla_pages_args* a) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0) return fail(SMLA_ERR_INVALID_ARG, "rows %d is negative", a->rows);
  if (a->max_pages < 1) return fail(SMLA_ERR_INVALID_ARG, "max_pages %d < 1", a->max_pages);
  if (a->page_size < 1) return fail(SMLA_ERR_INVALID_ARG, "page_size %d < 1", a->page_size);
  if ((int64_t)a->max_pages * a->page_size > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "max_pages %d: a request holds 1 .. 2^31 - 1 tokens", a->max_pages);
  if ((int64_t)a->rows * ((int64_t)a->max_pages + 1) > 0x3fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "%d rows of %d pages: the tables hold under 2^30 entries", a->rows, a->max_pages);
  if (a->block_table_stride != 0 && a->block_table_stride < a->max_pages)
    return fail(SMLA_ERR_INVALID_ARG, "block_table_stride %lld < max_pages %d", (long long)a->block_table_stride,
                a->max_pages);
  return SMLA_OK;
}

smla_status check_pages(const smla_pages_args* a) {
  SMLA_TRY(check_tables(a));
  if (a->num_pages < 1 || a->num_pages > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "num_pages %lld is outside 1 .. 2^31 - 1", (long long)a->num_pages);
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

smla_status check_parents(const smla_pages_args* a) {
  SMLA_TRY(need_words("parents", a->parents, true));
  SMLA_TRY(need_words("out_lens", a->out_lens, true));
  const size_t bytes = (size_t)a->rows * sizeof(int32_t);
  if (overlap(a->out_lens, bytes, a->lens, bytes))
    return fail(SMLA_ERR_INVALID_ARG, "out_lens must not be lens or overlap it");
  return SMLA_OK;
}

Area tables_area(const smla_pages_args* a) {
  const int64_t stride = a->block_table_stride ? a->block_table_stride : a->max_pages;
  return area(a->block_tables, a->rows, (int64_t)a->max_pages * 4, stride * 4);
}

size_t reorder_workspace(const smla_pages_args* a) {
  return align_up((size_t)a->rows * a->max_pages * sizeof(int32_t), 256);
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
  return need_workspace(a->workspace, a->workspace_bytes, pages_workspace(a));
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
  *bytes = pair_workspace(pairs_of(args), window_tiles(args), args->num_splits, sms);
  return SMLA_OK;
}

smla_status smla_window_attention(const smla_window_args* a, void* stream) {
  SMLA_TRY(check_window(a));
  if (a->sum_q == 0) return SMLA_OK;
  SMLA_TRY(check_attention_pointers(a));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  const WindowPlan plan = window_plan(a, sms);
  if (plan.units > 0x7fffffff || pairs_of(a) > 0x7fffffff / kWindowHeads)
    return fail(SMLA_ERR_UNSUPPORTED, "%lld units are too many", (long long)plan.units);
  SMLA_TRY(need_workspace(a->workspace, a->workspace_bytes, plan.bytes));
  WindowParams p = attention_params(a);
  p.window = a->window;
  p.first_tokens = a->first_tokens;
  set_parts(&p, plan, a->workspace);
  return launched("window attention", launch_pair_attention(p, nullptr, sms, static_cast<cudaStream_t>(stream)));
}

smla_status smla_prefix_workspace_size(const smla_prefix_args* args, int device, size_t* bytes) {
  if (bytes == nullptr) return fail(SMLA_ERR_INVALID_ARG, "bytes is NULL");
  SMLA_TRY(check_prefix(args));
  int sms = 0;
  SMLA_TRY(device_sms(device, &sms));
  // (smaller calls may take each token by itself; where this one does, all of them do)
  *bytes = pair_workspace(pairs_of(args), grouped_tiles(args), 0, sms);
  if (shares_prefixes(args, sms)) *bytes = std::max(*bytes, prefix_layout(args, sms).bytes);
  return SMLA_OK;
}

smla_status smla_prefix_attention(const smla_prefix_args* a, void* stream) {
  SMLA_TRY(check_prefix(a));
  if (a->sum_q == 0) return SMLA_OK;
  SMLA_TRY(check_attention_pointers(a));
  SMLA_TRY(need_words("group_starts", a->group_starts, a->num_groups > 0));
  SMLA_TRY(need_words("prefix_lens", a->prefix_lens, a->num_groups > 0));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  WindowParams p = attention_params(a);
  PrefixPlan plan;
  memset(&plan, 0, sizeof(plan));
  plan.groups = a->num_groups;
  plan.group_starts = a->group_starts;
  plan.prefix_lens = a->prefix_lens;
  if (!shares_prefixes(a, sms)) {
    const WindowPlan w = grouped_plan(a, sms);
    if (w.units > 0x7fffffff || pairs_of(a) > 0x7fffffff / kWindowHeads)
      return fail(SMLA_ERR_UNSUPPORTED, "%lld units are too many", (long long)w.units);
    SMLA_TRY(need_workspace(a->workspace, a->workspace_bytes, w.bytes));
    set_parts(&p, w, a->workspace);
    return launched("prefix attention", launch_pair_attention(p, &plan, sms, static_cast<cudaStream_t>(stream)));
  }
  const PrefixLayout l = prefix_layout(a, sms);
  if (l.parts + 2 * (int64_t)a->sum_q > 0x7fffffff / kWindowHeads)
    return fail(SMLA_ERR_UNSUPPORTED, "%d tokens are too many", a->sum_q);
  SMLA_TRY(need_workspace(a->workspace, a->workspace_bytes, l.bytes));
  char* const ws = static_cast<char*>(a->workspace);
  p.part_o = static_cast<float*>(a->workspace);
  p.part_lse = reinterpret_cast<float*>(ws + l.lse);
  plan.shares = l.shares;
  plan.share_cost = reinterpret_cast<int64_t*>(ws + l.header);
  plan.share_by = reinterpret_cast<uint64_t*>(ws + l.header + sizeof(int64_t));
  plan.many = reinterpret_cast<int32_t*>(ws + l.header + 2 * sizeof(int64_t));
  plan.cost_of = reinterpret_cast<int64_t*>(ws + l.cost_of);
  plan.unit_of = reinterpret_cast<int32_t*>(ws + l.unit_of);
  plan.shared_of = reinterpret_cast<int32_t*>(ws + l.shared_of);
  plan.share = reinterpret_cast<int4*>(ws + l.share);
  plan.first = reinterpret_cast<int4*>(ws + l.first);
  plan.group = reinterpret_cast<int4*>(ws + l.group);
  plan.token = reinterpret_cast<int4*>(ws + l.token);
  plan.prefix_of = reinterpret_cast<int4*>(ws + l.prefix_of);
  plan.limit = reinterpret_cast<int32_t*>(ws + l.limit);
  plan.lead = reinterpret_cast<int32_t*>(ws + l.lead);
  return launched("prefix attention", launch_prefix_attention(p, plan, static_cast<cudaStream_t>(stream)));
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
  SMLA_TRY(check_parents(a));
  return launched("pages fork", launch_pages_fork(pages_params(a), static_cast<cudaStream_t>(stream)));
}

smla_status smla_pages_reorder_workspace_size(const smla_pages_args* args, size_t* bytes) {
  if (bytes == nullptr) return fail(SMLA_ERR_INVALID_ARG, "bytes is NULL");
  SMLA_TRY(check_tables(args));
  *bytes = reorder_workspace(args);
  return SMLA_OK;
}

smla_status smla_pages_reorder(const smla_pages_args* a, void* stream) {
  SMLA_TRY(check_pages(a));
  if (a->rows == 0) return SMLA_OK;
  SMLA_TRY(check_page_pointers(a));
  SMLA_TRY(check_parents(a));
  if (overlap(a->out_lens, (size_t)a->rows * sizeof(int32_t), a->parents, (size_t)a->rows * sizeof(int32_t)))
    return fail(SMLA_ERR_INVALID_ARG, "out_lens must not be parents or overlap them");
  if (overlap(area(a->out_lens, (int64_t)a->rows * 4), tables_area(a)) ||
      overlap(area(a->out_lens, (int64_t)a->rows * 4), area(a->ref_counts, a->num_pages * 4)))
    return fail(SMLA_ERR_INVALID_ARG, "out_lens must not overlap block_tables or ref_counts");
  SMLA_TRY(need_workspace(a->workspace, a->workspace_bytes, reorder_workspace(a)));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  return launched("pages reorder", launch_pages_reorder(pages_params(a), sms, static_cast<cudaStream_t>(stream)));
}

smla_status smla_pages_shared_prefix(const smla_pages_args* a, const int32_t* group_starts, int32_t num_groups,
                                     int32_t* prefix_lens, void* stream) {
  SMLA_TRY(check_tables(a));
  if (num_groups < 0) return fail(SMLA_ERR_INVALID_ARG, "num_groups %d is negative", num_groups);
  if (num_groups == 0) return SMLA_OK;
  SMLA_TRY(need_words("group_starts", group_starts, true));
  SMLA_TRY(need_words("prefix_lens", prefix_lens, true));
  SMLA_TRY(need_words("error_word", a->error_word, false));
  if (a->rows > 0) {
    SMLA_TRY(need_words("block_tables", a->block_tables, true));
    SMLA_TRY(need_words("lens", a->lens, true));
  }
  const size_t groups = (size_t)num_groups * sizeof(int32_t);
  if (overlap(prefix_lens, groups, group_starts, groups + sizeof(int32_t)) ||
      overlap(prefix_lens, groups, a->lens, (size_t)a->rows * sizeof(int32_t)) ||
      overlap(area(prefix_lens, (int64_t)groups), tables_area(a)))
    return fail(SMLA_ERR_INVALID_ARG, "prefix_lens must not overlap block_tables, lens or group_starts");
  return launched("pages shared prefix", launch_pages_shared_prefix(pages_params(a), group_starts, num_groups, prefix_lens,
                                                                    static_cast<cudaStream_t>(stream)));
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
