// Append to the paged latent cache: BF16 rows quantised to E4M3 with one
// power-of-two scale per block of tokens.
//
//   s = max(old, 2^k), 2^k the smallest power of two with amax <= 448 * 2^k;
//   new code = RN(x / s), older code of the block = RN(code * (old / s)).
//
// 448 = 1.75 * 2^8, so for amax = m * 2^e (1 <= m < 2) k is e - 8, or e - 7
// when m > 1.75.  A CTA takes one block of one request: its scale needs every
// new row of the block first, and no other block's.  The rows stay in
// registers between the maximum and the rounding (blocks of up to 16 new rows;
// longer ones are read again, from L2), so DRAM sees each row once: 1 KB in,
// 512 B out a token.  Its floor is that traffic; what it takes beyond is the chain
// offsets -> rows and page -> scale -> codes of a CTA, which many small CTAs an
// SM overlap, and the instructions.  Measured on a GB300, inputs from DRAM (four
// states in turn): 33.7 thousand tokens of 8 prompts 11.3 us (4.6 TB/s), 132 thousand
// of 32 33.1 us (6.1 TB/s): the shorter call does not reach the longer one's rate, and
// why is not known.  One state again and again, its 50 MB in L2: 8.2 us; so were
// measured: the maximum over packed BF16 magnitudes, two a lane (value by value 11.3 us
// against 9.2), and eight CTAs an SM (64 registers 8.8 us, 80 9.2, ten with spills
// 10.3).  128 requests of one token: 3.3 us behind another kernel.
#include <type_traits>

#include "cache.cuh"

namespace smla {
namespace {

constexpr int kThreads = 128;                    // two rows of 64 threads x 8 values at a time
constexpr int kGroups = kThreads / 64;
constexpr int kHeld = 8;                         // rows a thread holds in registers
constexpr int kMinExp = -64, kMaxExp = 64;

// Largest magnitude of 8 BF16 values and m's, as BF16 bits, of even and odd values.
__device__ __forceinline__ uint32_t amax8(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  return m;
}
// The same of the finite ones (infinities and NaN count as 0).
__device__ __forceinline__ uint32_t amax8_finite(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = w[i] & 0x7fff0000u;
    m = __vmaxu2(m, (lo < 0x7f80u ? lo : 0u) | (hi < 0x7f800000u ? hi : 0u));
  }
  return m;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// x / s and one rounding to E4M3.  For a power of two (kPow2; every scale that
// this call makes) s holds the exact reciprocal; a scale that the caller's own
// blocks came with takes a correctly rounded division.
template <bool kPow2>
__device__ __forceinline__ uint2 quantise8(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
    h[i] = kPow2 ? e4m3x2(a * s, b * s) : e4m3x2(__fdiv_rn(a, s), __fdiv_rn(b, s));
  }
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

__global__ void __launch_bounds__(kThreads, 8) cache_append_kernel(const AppendParams p) {
  const CacheView& c = p.c;
  __shared__ float s_max[kThreads / 32];
  // unit u -> (request, block): request b's units start at first(b) / block_rows + 2 b,
  // which leaves room for the blocks its tokens can touch, count / block_rows + 2
  const int64_t u = blockIdx.x;
  await_prior_kernel();
  admit_next_kernel();
  const int b = last_request(c.batch, threadIdx.x & 31, [&](int at) {
    int f, n;
    request_tokens(c, at, &f, &n);
    return (int64_t)(f / c.block_rows) + 2 * (int64_t)at <= u;
  });
  int first, count;
  request_tokens(c, b, &first, &count);
  if (first < 0 || count <= 0 || count > c.sum_q - first) return;       // (offsets that are none: nothing is written)
  const int start = fetch(c.seq_lens + b) - count;                      // position of the first new token
  const int end = start + count, from0 = max(start, 0);
  const int i = (int)(u - (first / c.block_rows + 2 * (int64_t)b));     // block of the request's touched ones
  if (i < 0) return;                                                    // (the units of a batch padded in front)
  if (i == 0 && start < 0 && threadIdx.x == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
  const int64_t block0 = ((int64_t)(from0 / c.block_rows) + i) * c.block_rows;   // first position of the block
  if (block0 >= end) return;
  const int pos0 = max((int)block0, from0);                             // first new position in the block
  const int pos1 = (int)min(block0 + c.block_rows, (int64_t)end);
  const int column = (int)block0 / c.page_size;
  const int row0 = (int)block0 - column * c.page_size;                  // the block's first row in its page
  // (the page is on its way while the rows are read)
  const int page = column < c.max_pages ? fetch(c.bt + (int64_t)b * c.bt_stride + column) : -1;
  const int older = pos0 - (int)block0, rows = pos1 - pos0;
  const __nv_bfloat16* src = p.latent + (first + (pos0 - start)) * p.latent_stride;
  const int group = threadIdx.x >> 6, lane8 = threadIdx.x & 63;         // row parity, 8 values

  uint4 held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int r = k * kGroups + group;
    if (r < rows) held[k] = fetch(reinterpret_cast<const uint4*>(src + r * p.latent_stride) + lane8);
  }
  if (page < 0 || page >= c.num_pages) {
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
    return;
  }
  uint8_t* dst = c.rows + (int64_t)page * c.page_stride + (int64_t)row0 * c.row_stride;
  float* scale = c.scales + (int64_t)page * c.scale_stride + row0 / c.block_rows;
  const float old = older > 0 ? *scale : 0.f;
  auto largest = [&](auto amax) {                         // of the warp's values, as BF16 bits
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (k * kGroups + group < rows) m2 = amax(held[k], m2);
    for (int r = kHeld * kGroups + group; r < rows; r += kGroups)
      m2 = amax(fetch(reinterpret_cast<const uint4*>(src + r * p.latent_stride) + lane8), m2);
    return __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
  };
  uint32_t bits16 = largest([](uint4 v, uint32_t m2) { return amax8(v, m2); });
  if (bits16 >= 0x7f80u) bits16 = largest([](uint4 v, uint32_t m2) { return amax8_finite(v, m2); });
  float m = __uint_as_float(bits16 << 16);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();                                        // also: every thread has read the old scale
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, s_max[w]);

  int k = kMinExp;
  if (m > 0.f) {
    int e;
    const float f = frexpf(m, &e);                        // m = f 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    k = min(max(f <= 0.875f ? e - 9 : e - 8, kMinExp), kMaxExp);
  }
  const float need = ldexpf(1.f, k);
  const float base = old > 0.f && old < INFINITY ? old : 0.f;
  const float s = fmaxf(base, need);
  if (threadIdx.x == 0) *scale = s;
  if (older > 0 && old != s) {
    const float ratio = __fdiv_rn(base, s);
    for (int r = group; r < older; r += kGroups) {
      uint2* at = reinterpret_cast<uint2*>(dst + r * c.row_stride) + lane8;
      const uint2 v = *at;
      const uint32_t w[2] = {v.x, v.y};
      uint32_t o[2];
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2)
        o[i2] = e4m3x2(e4m3_value(w[i2]) * ratio, e4m3_value(w[i2] >> 8) * ratio) |
                e4m3x2(e4m3_value(w[i2] >> 16) * ratio, e4m3_value(w[i2] >> 24) * ratio) << 16;
      *at = make_uint2(o[0], o[1]);
    }
  }
  dst += older * c.row_stride;
  auto store = [&](auto pow2, float by) {
    constexpr bool kPow2 = decltype(pow2)::value;
#pragma unroll
    for (int kk = 0; kk < kHeld; ++kk) {
      const int r = kk * kGroups + group;
      if (r < rows) reinterpret_cast<uint2*>(dst + r * c.row_stride)[lane8] = quantise8<kPow2>(held[kk], by);
    }
    for (int r = kHeld * kGroups + group; r < rows; r += kGroups)
      reinterpret_cast<uint2*>(dst + r * c.row_stride)[lane8] =
          quantise8<kPow2>(fetch(reinterpret_cast<const uint4*>(src + r * p.latent_stride) + lane8), by);
  };
  const uint32_t bits = __float_as_uint(s);
  // a normal power of two whose reciprocal is one too
  if ((bits & 0x7fffffu) == 0 && bits >= 0x00800000u && bits <= 0x7e800000u)
    store(std::true_type{}, __uint_as_float(0x7f000000u - bits));
  else
    store(std::false_type{}, s);
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.c.sum_q / p.c.block_rows + 2 * (int64_t)p.c.batch;
  return launch_overlapped(cache_append_kernel, dim3((unsigned)units), kThreads, 0, stream, p);
}

}  // namespace smla
