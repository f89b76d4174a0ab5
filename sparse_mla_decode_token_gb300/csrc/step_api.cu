// Host side of a step's calls beside the attention: argument checks and launches
// (shapes and pointers before any CUDA call; nothing read, allocated or waited for).
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "api_checks.h"
#include "step.cuh"

namespace smla {
namespace {

smla_status check_slot_table(const char* name, int64_t stride, int32_t max_pages, int32_t page_size) {
  if (max_pages < 1) return fail(SMLA_ERR_INVALID_ARG, "%s: max_pages %d < 1", name, max_pages);
  if (page_size < 1) return fail(SMLA_ERR_INVALID_ARG, "%s: page_size %d < 1", name, page_size);
  if ((int64_t)max_pages * page_size > 0x7fffffff)
    return fail(SMLA_ERR_INVALID_ARG, "%s: a request holds 1 .. 2^31 - 1 tokens", name);
  if (stride != 0 && stride < max_pages)
    return fail(SMLA_ERR_INVALID_ARG, "%s: row stride %lld < max_pages %d", name, (long long)stride, max_pages);
  return SMLA_OK;
}

SlotTable slot_table(const int32_t* bt, int64_t stride, int32_t max_pages, int32_t page_size) {
  SlotTable t;
  t.bt = bt;
  t.stride = stride ? stride : max_pages;
  t.max_pages = max_pages;
  t.page_size = page_size;
  t.shift = page_size > 0 && (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
  return t;
}

// Outputs that overlap an input, which other threads still read, or one another.
smla_status check_outputs(const char* what, std::initializer_list<Area> outputs, std::initializer_list<Area> inputs) {
  for (const Area* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Area& in : inputs)
      if (overlap(*o, in)) return fail(SMLA_ERR_INVALID_ARG, "%s must not overlap an input", what);
    for (const Area* other = outputs.begin(); other != o; ++other)
      if (overlap(*o, *other)) return fail(SMLA_ERR_INVALID_ARG, "%s must not overlap one another", what);
  }
  return SMLA_OK;
}

Area table_area(const SlotTable& t, int64_t rows) {
  return area(t.bt, rows, (int64_t)t.max_pages * 4, t.stride * 4);
}

smla_status check_beam(const smla_beam_args* a) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  if (a->batch < 0) return fail(SMLA_ERR_INVALID_ARG, "batch %d is negative", a->batch);
  if (a->beams < 1 || a->beams > SMLA_MAX_BEAMS)
    return fail(SMLA_ERR_UNSUPPORTED, "beams %d is outside 1 .. %d", a->beams, SMLA_MAX_BEAMS);
  if (a->vocab < 1) return fail(SMLA_ERR_INVALID_ARG, "vocab %d < 1", a->vocab);
  if (a->num_out < 1 || a->num_out > SMLA_MAX_BEAM_OUT)
    return fail(SMLA_ERR_UNSUPPORTED, "num_out %d is outside 1 .. %d", a->num_out, SMLA_MAX_BEAM_OUT);
  if (a->dtype < SMLA_LOGITS_BF16 || a->dtype > SMLA_LOGITS_FP32)
    return fail(SMLA_ERR_INVALID_ARG, "dtype %d is no SMLA_LOGITS_*", a->dtype);
  if (a->logits_stride != 0 && a->logits_stride < a->vocab)
    return fail(SMLA_ERR_INVALID_ARG, "logits_stride %lld < vocab %d", (long long)a->logits_stride, a->vocab);
  if ((int64_t)a->batch * a->beams > 0x7fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "%d requests of %d beams: rows are 32-bit numbers", a->batch, a->beams);
  return SMLA_OK;
}

int32_t units_of(int32_t blocks, int shift) { return (blocks + (1 << shift) - 1) >> shift; }

// Units of up to 16 blocks, shorter ones where there would not be 32 of them for
// each SM (as many as it holds warps).
BeamPlan beam_plan(const smla_beam_args* a, int sms) {
  const int size = a->dtype == SMLA_LOGITS_FP32 ? 4 : 2, block = kBeamBlockBytes / size;
  BeamPlan plan;
  plan.blocks = (int32_t)(((int64_t)a->vocab + 16 / size - 1 + block - 1) / block);   // (a row begins up to 15 bytes behind a boundary)
  const int64_t all = (int64_t)plan.blocks * a->batch * a->beams;
  plan.unit_shift = kMaxUnitShift;
  while (plan.unit_shift > kMinUnitShift && all >> plan.unit_shift < (int64_t)sms * 32) --plan.unit_shift;
  plan.units = units_of(plan.blocks, plan.unit_shift);
  return plan;
}

struct BeamLayout {
  size_t partial, bytes;
};
BeamLayout beam_layout(const smla_beam_args* a, const BeamPlan& plan) {
  const size_t rows = (size_t)a->batch * a->beams;
  BeamLayout l;
  l.partial = align_up(rows * plan.blocks * sizeof(float), 256);
  l.bytes = l.partial + align_up(rows * plan.units * sizeof(float2), 256);
  return l;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

smla_status smla_token_slots(const smla_token_slots_args* a, void* stream) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  if (a->batch < 0) return fail(SMLA_ERR_INVALID_ARG, "batch %d is negative", a->batch);
  if (a->max_tokens < 0) return fail(SMLA_ERR_INVALID_ARG, "max_tokens %d is negative", a->max_tokens);
  if (a->slots != nullptr) {
    SMLA_TRY(check_slot_table("block_tables", a->block_table_stride, a->max_pages, a->page_size));
    if (a->batch > 0) SMLA_TRY(need_words("block_tables", a->block_tables, true));
    if (!aligned(a->slots, 8)) return fail(SMLA_ERR_INVALID_ARG, "slots must be 8-byte aligned");
  }
  if (a->batch > 0) {
    SMLA_TRY(need_words("lens", a->lens, true));
    SMLA_TRY(need_words("new_lens", a->new_lens, true));
  }
  SMLA_TRY(need_words("cum_seq_lens_q", a->cum_seq_lens_q, true));
  SMLA_TRY(need_words("requests", a->requests, false));
  SMLA_TRY(need_words("positions", a->positions, false));
  SMLA_TRY(need_words("error_word", a->error_word, false));
  const int64_t lens = (int64_t)a->batch * 4, tokens = (int64_t)a->max_tokens * 4;
  const auto given = [](const void* at, int64_t bytes) { return area(at, at != nullptr ? bytes : 0); };
  const SlotTable tables = slot_table(a->block_tables, a->block_table_stride, a->max_pages, a->page_size);
  SMLA_TRY(check_outputs("cum_seq_lens_q, requests, positions and slots",
                         {area(a->cum_seq_lens_q, lens + 4), given(a->requests, tokens), given(a->positions, tokens),
                          given(a->slots, 2 * tokens)},
                         {given(a->lens, lens), given(a->new_lens, lens),
                          table_area(tables, a->slots != nullptr ? a->batch : 0)}));
  TokenSlotsParams p;
  memset(&p, 0, sizeof(p));
  p.lens = a->lens;
  p.new_lens = a->new_lens;
  p.batch = a->batch;
  p.max_tokens = a->max_tokens;
  p.bt = a->block_tables;
  p.bt_stride = a->block_table_stride ? a->block_table_stride : a->max_pages;
  p.max_pages = a->max_pages;
  p.page_size = a->page_size;
  p.cum = a->cum_seq_lens_q;
  p.requests = a->requests;
  p.positions = a->positions;
  p.slots = a->slots;
  p.err = a->error_word;
  return launched("token slots", launch_token_slots(p, static_cast<cudaStream_t>(stream)));
}

smla_status smla_sparse_slots(const smla_sparse_slots_args* a, void* stream) {
  if (a == nullptr) return fail(SMLA_ERR_INVALID_ARG, "args is NULL");
  if (a->sum_q < 0) return fail(SMLA_ERR_INVALID_ARG, "sum_q %d is negative", a->sum_q);
  if (a->batch < 1) return fail(SMLA_ERR_INVALID_ARG, "batch %d < 1", a->batch);
  if (a->cum_seq_lens_q == nullptr && a->sum_q % a->batch != 0)
    return fail(SMLA_ERR_INVALID_ARG, "sum_q %d is not a multiple of batch %d (pass cum_seq_lens_q)", a->sum_q, a->batch);
  SMLA_TRY(check_slot_table("swa_tables", a->swa_table_stride, a->swa_max_pages, a->swa_page_size));
  if (a->num_selected < 0 || a->num_selected > 1 << 30)                 // (the kernel counts columns past a row's end)
    return fail(SMLA_ERR_INVALID_ARG, "num_selected %d is outside 0 .. 2^30", a->num_selected);
  if (a->compress_ratio < 1) return fail(SMLA_ERR_INVALID_ARG, "compress_ratio %d < 1", a->compress_ratio);
  if (a->num_selected > 0)
    SMLA_TRY(check_slot_table("comp_tables", a->comp_table_stride, a->comp_max_pages, a->comp_page_size));
  if (a->selected_stride != 0 && a->selected_stride < a->num_selected)
    return fail(SMLA_ERR_INVALID_ARG, "selected_stride %lld < num_selected %d", (long long)a->selected_stride, a->num_selected);
  const int32_t columns = kSwaCols + a->num_selected;
  if (a->indices_row_stride != 0 && a->indices_row_stride < columns)
    return fail(SMLA_ERR_INVALID_ARG, "indices_row_stride %lld is less than a row's %d columns",
                (long long)a->indices_row_stride, columns);
  if (a->sum_q == 0) return SMLA_OK;
  SMLA_TRY(need_words("seq_lens", a->seq_lens, true));
  SMLA_TRY(need_words("cum_seq_lens_q", a->cum_seq_lens_q, false));
  SMLA_TRY(need_words("swa_tables", a->swa_tables, true));
  SMLA_TRY(need_words("comp_tables", a->comp_tables, a->num_selected > 0));
  SMLA_TRY(need_words("selected", a->selected, false));
  SMLA_TRY(need_words("sparse_indices", a->sparse_indices, true));
  SMLA_TRY(need_words("topk_lens", a->topk_lens, true));
  SMLA_TRY(need_words("error_word", a->error_word, false));
  SparseSlotsParams p;
  memset(&p, 0, sizeof(p));
  p.sum_q = a->sum_q;
  p.batch = a->batch;
  p.seq_lens = a->seq_lens;
  p.cum = a->cum_seq_lens_q;
  p.swa = slot_table(a->swa_tables, a->swa_table_stride, a->swa_max_pages, a->swa_page_size);
  p.comp = slot_table(a->comp_tables, a->comp_table_stride, a->comp_max_pages, a->comp_page_size);
  p.ratio = a->compress_ratio;
  p.num_selected = a->num_selected;
  p.selected = a->num_selected > 0 ? a->selected : nullptr;
  p.selected_stride = a->selected_stride ? a->selected_stride : a->num_selected;
  p.out = a->sparse_indices;
  p.out_stride = a->indices_row_stride ? a->indices_row_stride : columns;
  p.topk = a->topk_lens;
  p.err = a->error_word;
  // (a selection in place: each thread reads its own columns before it writes them)
  const bool in_place = p.selected == p.out + kSwaCols && (p.sum_q == 1 || p.selected_stride == p.out_stride);
  const Area out = area(p.out, p.sum_q, (int64_t)columns * 4, p.out_stride * 4), topk = area(p.topk, (int64_t)p.sum_q * 4),
             picks = area(p.selected, p.selected != nullptr ? p.sum_q : 0, (int64_t)p.num_selected * 4, p.selected_stride * 4);
  if (!in_place && overlap(out, picks))
    return fail(SMLA_ERR_INVALID_ARG, "selected must be the columns from %d on of sparse_indices or not overlap it", kSwaCols);
  if (overlap(topk, picks)) return fail(SMLA_ERR_INVALID_ARG, "topk_lens must not overlap an input");
  SMLA_TRY(check_outputs("sparse_indices and topk_lens", {out, topk},
                         {area(p.seq_lens, (int64_t)p.batch * 4), area(p.cum, p.cum != nullptr ? ((int64_t)p.batch + 1) * 4 : 0),
                          table_area(p.swa, p.batch), table_area(p.comp, p.num_selected > 0 ? p.batch : 0)}));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  return launched("sparse slots", launch_sparse_slots(p, sms, static_cast<cudaStream_t>(stream)));
}

smla_status smla_beam_workspace_size(const smla_beam_args* args, int device, size_t* bytes) {
  if (bytes == nullptr) return fail(SMLA_ERR_INVALID_ARG, "bytes is NULL");
  SMLA_TRY(check_beam(args));
  int sms = 0;
  SMLA_TRY(device_sms(device, &sms));
  // (smaller calls may have shorter units, so more of them a row: a size that serves those, too)
  BeamPlan plan = beam_plan(args, sms);
  plan.units = units_of(plan.blocks, kMinUnitShift);
  *bytes = beam_layout(args, plan).bytes;
  return SMLA_OK;
}

smla_status smla_beam_select(const smla_beam_args* a, void* stream) {
  SMLA_TRY(check_beam(a));
  if (a->batch == 0) return SMLA_OK;
  if (a->logits == nullptr) return fail(SMLA_ERR_INVALID_ARG, "logits is required");
  const int64_t size = a->dtype == SMLA_LOGITS_FP32 ? 4 : 2;
  if (!aligned(a->logits, size)) return fail(SMLA_ERR_INVALID_ARG, "logits must be %d-byte aligned", (int)size);
  SMLA_TRY(need_words("scores", a->scores, true));
  SMLA_TRY(need_words("out_scores", a->out_scores, true));
  SMLA_TRY(need_words("out_parents", a->out_parents, true));
  SMLA_TRY(need_words("out_tokens", a->out_tokens, true));
  SMLA_TRY(need_words("error_word", a->error_word, false));
  const int64_t rows = (int64_t)a->batch * a->beams, places = (int64_t)a->batch * a->num_out * 4;
  const Area out_scores = area(a->out_scores, places), scores = area(a->scores, rows * 4);
  // (in place: a request's scores are read by the CTA alone that writes them)
  if (!(a->out_scores == a->scores && a->num_out == a->beams) && overlap(out_scores, scores))
    return fail(SMLA_ERR_INVALID_ARG, "out_scores must be scores (num_out = beams) or not overlap it");
  const Area parents = area(a->out_parents, places), tokens = area(a->out_tokens, places);
  if (overlap(parents, scores) || overlap(tokens, scores))
    return fail(SMLA_ERR_INVALID_ARG, "out_parents and out_tokens must not overlap scores");
  SMLA_TRY(check_outputs("out_scores, out_parents and out_tokens", {out_scores, parents, tokens},
                         {area(a->logits, rows, a->vocab * size, (a->logits_stride ? a->logits_stride : a->vocab) * size),
                          area(a->finished, a->finished != nullptr ? rows : 0)}));
  int sms = 0;
  SMLA_TRY(current_sms(&sms));
  BeamParams p;
  memset(&p, 0, sizeof(p));
  p.plan = beam_plan(a, sms);
  if ((int64_t)p.plan.blocks * a->beams > kMaxBeamBlocks || (int64_t)p.plan.units * a->beams * a->batch > 0x7fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "%d requests of %d beams over a vocabulary of %d are too many blocks", a->batch,
                a->beams, a->vocab);
  const BeamLayout layout = beam_layout(a, p.plan);
  SMLA_TRY(need_workspace(a->workspace, a->workspace_bytes, layout.bytes));
  p.batch = a->batch;
  p.beams = a->beams;
  p.vocab = a->vocab;
  p.num_out = a->num_out;
  p.dtype = a->dtype;
  p.logits = a->logits;
  p.stride = a->logits_stride ? a->logits_stride : a->vocab;
  p.scores = a->scores;
  p.finished = a->finished;
  p.end_token = a->end_token;
  p.out_scores = a->out_scores;
  p.out_parents = a->out_parents;
  p.out_tokens = a->out_tokens;
  p.block_max = static_cast<float*>(a->workspace);
  p.partial = reinterpret_cast<float2*>(static_cast<char*>(a->workspace) + layout.partial);
  p.err = a->error_word;
  return launched("beam select", launch_beam_select(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
