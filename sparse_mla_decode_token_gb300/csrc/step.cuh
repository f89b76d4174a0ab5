// Kernel-side copies of the arguments of a step's calls beside the attention
// (strides already defaulted) and their launchers.
#pragma once

#include "cache.cuh"

namespace smla {

struct TokenSlotsParams {
  const int32_t* lens;
  const int32_t* new_lens;
  int32_t batch, max_tokens;
  const int32_t* bt;                 // nullptr: no slots
  int64_t bt_stride;
  int32_t max_pages, page_size;
  int32_t* cum;
  int32_t* requests;
  int32_t* positions;
  int64_t* slots;
  int32_t* err;
};
cudaError_t launch_token_slots(const TokenSlotsParams& p, cudaStream_t stream);

struct SlotTable {
  const int32_t* bt;
  int64_t stride;
  int32_t max_pages, page_size;
  int32_t shift;                     // log2 of page_size, or -1
};
struct SparseSlotsParams {
  int32_t sum_q, batch;
  const int32_t* seq_lens;
  const int32_t* cum;                // nullptr: uniform
  SlotTable swa, comp;
  int32_t ratio, num_selected;
  const int32_t* selected;
  int64_t selected_stride;
  int32_t* out;
  int64_t out_stride;
  int32_t* topk;
  int32_t* err;
};
cudaError_t launch_sparse_slots(const SparseSlotsParams& p, int sms, cudaStream_t stream);

// How a call's logits are cut: blocks of the 512 bytes that a warp loads at once,
// of which only the maxima are kept; units of 2^unit_shift consecutive blocks of
// a row, a warp each, which give the partial sums.
struct BeamPlan {
  int32_t blocks, unit_shift, units;
};
constexpr int kBeamBlockBytes = 512;
constexpr int kMinUnitShift = 2, kMaxUnitShift = 4;
constexpr int64_t kMaxBeamBlocks = 1ll << 30;   // of a request

struct BeamParams {
  int32_t batch, beams, vocab, num_out, dtype;
  BeamPlan plan;
  const void* logits;
  int64_t stride;
  const float* scores;
  const uint8_t* finished;
  int32_t end_token;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  float* block_max;                  // [rows, blocks]
  float2* partial;                   // [rows, units] maximum, sum of e^(x - maximum)
  int32_t* err;
};
cudaError_t launch_beam_select(const BeamParams& p, int sms, cudaStream_t stream);

}  // namespace smla
