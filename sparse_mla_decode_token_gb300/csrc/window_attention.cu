// Attention over the paged latent cache with a sliding window and visible
// first tokens.
//
//   l_j = bmm1 s_j <q, c_j>,  O = bmm2 sum_j e^{l_j} s_j c_j / (sum_j e^{l_j} + e^{sink}),
//   LSE2 = log2 sum_j e^{l_j},  j over the visible rows, c_j codes, s_j their block's scale.
//
// One warp per (token, head), one pass over the rows with the running maximum
// and sum; 16 dims per lane.
#include "cache.cuh"

namespace smla {
namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32) window_kernel(const WindowParams p) {
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31;
  const int64_t th = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (th >= (int64_t)c.sum_q * p.H) return;
  const int t = (int)(th / p.H), h = (int)(th % p.H);
  int lo = 0, hi = c.batch - 1, first, count;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    request_tokens(c, mid, &first, &count);
    if (first <= t) lo = mid; else hi = mid - 1;
  }
  request_tokens(c, lo, &first, &count);
  const int64_t pos = (int64_t)__ldg(c.seq_lens + lo) - count + (t - first);
  float q[16], acc[16];
  const __nv_bfloat16* qp = p.q + t * p.q_stride_token + h * kHeadDim + lane * 16;
  for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(qp[i]), acc[i] = 0.f;
  const float scale = load_scale(p.bmm1, p.bmm1_dev) * kLog2e;
  float m = -INFINITY, sum = 0.f;
  const int64_t begin = pos - p.window + 1 > p.first_tokens ? pos - p.window + 1 : p.first_tokens;
  for (int64_t j = 0; j <= pos; ++j) {
    if (j >= p.first_tokens && j < begin) j = begin;
    if (j > pos) break;
    const int64_t col = j / c.page_size;
    const int page = col < c.max_pages ? __ldg(c.bt + lo * c.bt_stride + col) : -1;
    if (page < 0 || page >= c.num_pages) {
      if (p.err) atomicOr(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
      if (col >= c.max_pages) break;
      continue;
    }
    const int r = (int)(j % c.page_size);
    const float s = __ldg(c.scales + page * c.scale_stride + r / c.block_rows);
    const uint4 v = *reinterpret_cast<const uint4*>(c.rows + page * c.page_stride + r * c.row_stride + lane * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float kv[16], dot = 0.f;
    for (int i = 0; i < 16; ++i) {
      kv[i] = e4m3_value(w[i / 4] >> (8 * (i % 4))) * s;
      dot = fmaf(q[i], kv[i], dot);
    }
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    const float l = dot * scale, mn = fmaxf(m, l);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(l - mn);
    sum = sum * a + e;
    for (int i = 0; i < 16; ++i) acc[i] = acc[i] * a + e * kv[i];
    m = mn;
  }
  float f = 0.f, lse = -INFINITY;
  if (m != -INFINITY) {
    lse = m + log2f(sum);
    const float sink = p.sinks ? exp2f(__ldg(p.sinks + h) * kLog2e - lse) : 0.f;
    f = load_scale(p.bmm2, p.bmm2_dev) / (sum * (1.f + sink));
  }
  for (int i = 0; i < 16; ++i) p.out[th * kHeadDim + lane * 16 + i] = __float2bfloat16(acc[i] * f);
  if (lane == 0 && p.out_lse) p.out_lse[th] = lse;
}

}  // namespace

cudaError_t launch_window_attention(const WindowParams& p, cudaStream_t stream) {
  const int64_t n = (int64_t)p.c.sum_q * p.H;
  window_kernel<<<(unsigned)((n + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace smla
