// Attention over the paged latent cache with a sliding window and visible
// first tokens (tcgen05 / TMEM / TMA, sm_103a).
//
//   l_j = bmm1 s_j <q, c_j>,  O = bmm2 sum_j e^{l_j} s_j c_j / (sum_j e^{l_j} + e^{sink}),
//   LSE2 = log2 sum_j e^{l_j},  j over the visible rows, c_j E4M3 codes, s_j their block's scale.
//
// Both products take the codes as they lie in the cache, at the E4M3 rate, and
// still keep BF16's precision for the other operand: a BF16 number has eight
// significant bits, an E4M3 number four, so q 2^k = hi + lo with two E4M3
// numbers, hi the rounded value and lo the rest (at most eight units in the
// last place, hence exact above 2^-18 of the head's largest element, where
// lo's subnormals end).  P is split the same way (its error is then below
// BF16's).  Two E4M3 products cost what one BF16 product would, without
// widening the cache's rows in shared memory.
//
// Layout: one CTA takes 64 heads of one token and one split of its rows, and
// computes transposed products, rows by heads and dims by heads:
//
//   S^T[128 rows, 64 hi | 64 lo heads] = C Q^T      M = 128, N = 128, K = 512
//   O^T[512 dims, 64 heads] += C^T (P_hi + P_lo)    4 x M = 128, N = 64, K = 128
//
// An fp32 accumulator of 128 heads x 512 dims would fill tensor memory alone;
// 64 heads' O^T takes 256 columns and two S^T buffers the other 256, so no
// second CTA and no exchange is needed.  The row of a logit is its thread:
// masks and block scales are per thread, and the running maximum is needed per
// head only when some logit passes the reference by more than 2^4 (one
// barrier-vote a tile); then the maxima are taken over lanes and warps, and O
// is rescaled.
//
// With t_j = log2(e) l_j + log2 s_j and the reference m (a running maximum of
// t to within 2^4), P_j = 2^(t_j - m + 4) <= 2^8 weighs the raw code c_j, and
// the denominator takes P_j / s_j: a block's scale is folded into P, never into
// the tile.
//
// Rows come by TMA as chunks of 16 (or 8) consecutive rows of one page, 5-D
// boxes {128 B, 8 rows, 4 column blocks, groups, page}, which land as 8-row
// atoms 4096 bytes apart: K-major for S^T, MN-major for O^T.  The visible rows
// [0, first) and [pos - window + 1, pos] are a list of such chunks; rows of a
// chunk that the token does not see (or that no page backs) are masked in S^T
// and set to zero in the tile before the second product, so that nothing they
// hold (NaN codes of memory never written) reaches O.
//
// Sums and maxima are fp32, O accumulates in fp32; split partials are fp32.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "cache.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace smla {
namespace {

using namespace ptx;
using namespace tc;

constexpr int kNH = kWindowHeads;                 // 64 heads
constexpr int kRows = kWindowTile;                // 128 cache rows a tile
constexpr int kSoftmaxWarps = 4;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kMmaWarp = kSoftmaxWarps;           // issues the products; allocates and frees TMEM
constexpr int kLoadWarp = kSoftmaxWarps + 1;
constexpr int kThreads = (kSoftmaxWarps + 2) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 0;                     // O^T: four blocks of 128 dims, 64 columns each
constexpr uint32_t kSCol = 256;                   // S^T: two buffers of 64 hi + 64 lo columns
constexpr float kHeadroom = 4.f;                  // log2: a logit may pass the reference by this
constexpr float kUnset = 3e38f;                   // minus the reference before the first row
constexpr float kMinScaleLog2 = -64.f;
constexpr int kTileBytes = kRows * kHeadDim;      // 64 KB
constexpr int kGroupBytes = 8 * kHeadDim;         // 8 rows x four 128-byte column blocks
constexpr int kQBlock = 128 * 128;                // one column block of Q: 64 hi + 64 lo rows
constexpr int kPHalf = kRows * kNH;               // hi or lo of one tile's P: 8 KB
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 4 * kQBlock;
constexpr int kOffP = kOffK + 2 * kTileBytes;
constexpr int kOffSmall = kOffP + 4 * kPHalf;

struct Small {
  float qscale[kNH];                              // bmm1 log2(e) 2^-k of each head
  float negref[kNH];                              // headroom - reference of each head
  float factor[kNH];
  float wmax[kSoftmaxWarps][kNH];
  uint64_t k_full[2], pv_done[2], s_full[2], s_empty[2], p_full[2], q_full;
  uint32_t tmem;
  int32_t abort_flag;
};
constexpr int kSmemBytes = kOffSmall + sizeof(Small) + 1024;     // 1024: the base is aligned by hand
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
static_assert(kNH * (kSoftmaxThreads + 1) * 4 <= kTileBytes, "the sums' transposition fits a tile buffer");
static_assert(kNH * kHeadDim * 2 <= kTileBytes, "the staged output fits a tile buffer");

struct KernelParams {
  WindowParams p;
  CUtensorMap map;
  int32_t chunk;                                  // rows of a TMA box: 16 or 8
  int32_t groups;                                 // head groups
};

// What one CTA works on: 64 heads of a token, a range of tiles of its chunk list.
struct Unit {
  int t, h0, heads, split, b;
  int first_chunks, window_chunk, chunks;         // list: [0, first_chunks), then from window_chunk on
  int64_t pos, lo;                                // last and first visible position of the window
  int tile0, tiles;
};

__device__ __forceinline__ int chunk_at(const Unit& u, int k) {
  return k < u.first_chunks ? k : u.window_chunk + (k - u.first_chunks);
}

__device__ __forceinline__ Unit make_unit(const KernelParams& kp) {
  const WindowParams& p = kp.p;
  const CacheView& c = p.c;
  Unit u;
  int x = blockIdx.x;
  u.h0 = (x % kp.groups) * kNH;
  x /= kp.groups;
  u.split = x % p.num_splits;
  u.t = x / p.num_splits;
  u.heads = min(kNH, p.H - u.h0);
  int first, count;
  if (c.cum != nullptr) {
    // requests that end at or before this token: all threads look at once
    int n = 0;
    for (int base = 0; base < c.batch; base += kThreads) {
      const int b = base + threadIdx.x;
      n += __syncthreads_count(b < c.batch && __ldg(c.cum + b + 1) <= u.t);
    }
    u.b = min(n, c.batch - 1);
  } else {
    u.b = u.t / (c.sum_q / c.batch);
  }
  request_tokens(c, u.b, &first, &count);
  u.pos = (int64_t)__ldg(c.seq_lens + u.b) - count + (u.t - first);
  u.lo = u.pos - p.window + 1 > 0 ? u.pos - p.window + 1 : 0;
  u.first_chunks = u.window_chunk = u.chunks = 0;
  const int64_t last = min(u.pos, (int64_t)c.max_pages * c.page_size - 1);
  if (last >= 0) {
    u.first_chunks = (int)((min((int64_t)p.first_tokens, last + 1) + kp.chunk - 1) / kp.chunk);
    u.window_chunk = max((int)(u.lo / kp.chunk), u.first_chunks);
    u.chunks = u.first_chunks + max(0, (int)(last / kp.chunk) - u.window_chunk + 1);
  }
  const int per_tile = kRows / kp.chunk;
  const int tiles = (u.chunks + per_tile - 1) / per_tile, per = (tiles + p.num_splits - 1) / p.num_splits;
  u.tile0 = min(tiles, u.split * per);
  u.tiles = min(tiles, u.tile0 + per) - u.tile0;
  return u;
}

// Page of list entry k, or -1 (past the list, or no page of the pool).
__device__ __forceinline__ int chunk_page(const KernelParams& kp, const Unit& u, int k) {
  const CacheView& c = kp.p.c;
  if (k >= u.chunks) return -1;
  const int page = __ldg(c.bt + u.b * c.bt_stride + (int64_t)chunk_at(u, k) * kp.chunk / c.page_size);
  return page >= 0 && page < c.num_pages ? page : -1;
}

// The block scale of tile row r (0 <= r < 128) of list tile `tile`; negative: masked.
__device__ __forceinline__ float row_scale(const KernelParams& kp, const Unit& u, int tile, int r) {
  const CacheView& c = kp.p.c;
  const int k = tile * (kRows / kp.chunk) + r / kp.chunk;
  const int page = chunk_page(kp, u, k);
  if (k >= u.chunks) return -1.f;
  const int64_t j = (int64_t)chunk_at(u, k) * kp.chunk + r % kp.chunk;
  if (j > u.pos || (j < u.lo && j >= kp.p.first_tokens)) return -1.f;
  if (page < 0) {
    if (kp.p.err) atomicOr(kp.p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
    return -1.f;
  }
  return fabsf(__ldg(c.scales + (int64_t)page * c.scale_stride + (int)(j % c.page_size) / c.block_rows));
}

// Q of 64 heads as E4M3 pairs: rows 0-63 hi, 64-127 lo, K-major with 128-byte
// swizzle, column blocks of 128 dims.  One warp per head at a time.
__device__ __forceinline__ void split_query(const KernelParams& kp, const Unit& u, uint8_t* sq, Small& sm, int warp,
                                            int lane) {
  const WindowParams& p = kp.p;
  const __nv_bfloat16* q = p.q + (int64_t)u.t * p.q_stride_token + (int64_t)u.h0 * kHeadDim;
  const float scale = load_scale(p.bmm1, p.bmm1_dev) * kLog2e;
  constexpr int kBatch = 4;
  for (int h = warp * (kNH / kSoftmaxWarps); h < (warp + 1) * (kNH / kSoftmaxWarps); h += kBatch) {
    uint4 v[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        v[i][k] = h + i < u.heads ? __ldg(reinterpret_cast<const uint4*>(q + (h + i) * kHeadDim) + k * 32 + lane)
                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      uint32_t m = 0;                             // largest magnitude as BF16 bits
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      const bool finite = m < 0x7f80u;
      // 2^k that takes the largest element into [128, 256); BF16 exponent field e: magnitude in [2^(e-127), 2^(e-126))
      const int e = min(max((int)(m >> 7), 8), 254);
      const int k2 = 134 - e;
      const float up = __uint_as_float((uint32_t)(k2 + 127) << 23), down = __uint_as_float((uint32_t)(127 - k2) << 23);
      if (lane == 0) sm.qscale[h + i] = scale * down;
      const int r = h + i;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float a = __uint_as_float(w[x] << 16) * up, b = __uint_as_float(w[x] & 0xffff0000u) * up;
          const uint32_t hv = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
          const float ra = a - e4m3_value(hv), rb = b - e4m3_value(hv >> 8);
          hi[x] = finite ? hv : 0x7f7fu;          // a head with an infinity or NaN gets NaN everywhere
          lo[x] = finite ? (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(ra, rb), __NV_SATFINITE, __NV_E4M3) : 0u;
        }
        const int idx = k * 32 + lane, block = idx >> 4, ch = (idx & 15) >> 1, half = (idx & 1) * 8;
        uint8_t* at = sq + block * kQBlock + half;
        *reinterpret_cast<uint2*>(at + sw128_offset(r, ch)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(at + sw128_offset(r + kNH, ch)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      }
    }
  }
}

// Two weights to E4M3 pairs: hi = RN(p), lo = RN(p - hi), through fp16 (11 bits
// of a weight of at most 2^8, its subnormals end at 2^-24).
__device__ __forceinline__ void split_pair(float a, float b, uint32_t* hi, uint32_t* lo) {
  const __half2 p = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(p), __NV_SATFINITE, __NV_E4M3);
  const __half2 back(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3));
  *hi = h;
  *lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(p, back)), __NV_SATFINITE, __NV_E4M3);
}

__global__ void __launch_bounds__(kThreads, 1) window_kernel(const __grid_constant__ KernelParams kp) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  Small& sm = *reinterpret_cast<Small*>(smem + kOffSmall);
  const WindowParams& p = kp.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t k_addr = smem_addr(smem + kOffK), q_addr = smem_addr(smem + kOffQ), p_addr = smem_addr(smem + kOffP);
  auto bar = [](uint64_t& b) { return smem_addr(&b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm.k_full[i]), 1);
      mbar_init(bar(sm.pv_done[i]), 1);
      mbar_init(bar(sm.s_full[i]), 1);
      mbar_init(bar(sm.s_empty[i]), kSoftmaxWarps);
      mbar_init(bar(sm.p_full[i]), kSoftmaxWarps);
    }
    mbar_init(bar(sm.q_full), kSoftmaxWarps);
    sm.abort_flag = 0;
    fence_mbar_init_cluster();
    fence_proxy_async_smem();
  }
  const Unit u = make_unit(kp);
  if (u.pos >= (int64_t)p.c.max_pages * p.c.page_size && threadIdx.x == 0 && p.err)
    atomicOr(p.err, SMLA_DEVERR_INDEX_OUT_OF_RANGE);
  const int64_t th = (int64_t)u.t * p.H + u.h0;                               // first (token, head) of the unit
  const int64_t part = ((int64_t)u.t * p.num_splits + u.split) * p.H + u.h0;  // first partial
  if (u.tiles == 0) {                             // no visible row (of this split)
    if (p.num_splits > 1) {
      if (threadIdx.x < u.heads) p.part_lse[part + threadIdx.x] = -INFINITY;
      return;
    }
    uint4* o = reinterpret_cast<uint4*>(p.out + th * kHeadDim);
    for (int i = threadIdx.x; i < u.heads * (kHeadDim / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (p.out_lse && threadIdx.x < u.heads) p.out_lse[th + threadIdx.x] = -INFINITY;
    return;
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  Ctx cx{&sm.abort_flag, p.err};
  const int per_tile = kRows / kp.chunk;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------- loads
    // a lane per list entry; the pages of 32 entries are looked up at once
    const int chunk_groups = kp.chunk / 8;
    int loaded = 0, pages = -1;
    for (; loaded < u.tiles; ++loaded) {
      const int entry = loaded * per_tile;                                    // of this split's list
      if (entry % 32 == 0) {
        const int mine = entry + lane;
        pages = mine < u.tiles * per_tile ? chunk_page(kp, u, u.tile0 * per_tile + mine) : -1;
      }
      const int b = loaded & 1;
      if (loaded >= 2 && !warp_wait(cx, bar(sm.pv_done[b]), ((loaded >> 1) - 1) & 1)) break;
      const bool here = lane >= entry % 32 && lane < entry % 32 + per_tile && pages >= 0;
      const uint32_t n = __popc(__ballot_sync(0xffffffffu, here));
      if (lane == 0) mbar_arrive_expect_tx(bar(sm.k_full[b]), n * kp.chunk * kHeadDim);
      __syncwarp();
      if (here) {
        const int slot = lane - entry % 32;
        const int64_t j = (int64_t)chunk_at(u, u.tile0 * per_tile + entry + slot) * kp.chunk;
        tma_load_5d(k_addr + b * kTileBytes + slot * chunk_groups * kGroupBytes, &kp.map, 0, 0, 0,
                    (int)(j % p.c.page_size) / 8, pages, bar(sm.k_full[b]));
      }
      __syncwarp();
    }
    // after an abort the last copies may still be in flight
    for (int i = max(0, loaded - 2); i < loaded; ++i) drain_wait(bar(sm.k_full[i & 1]), (i >> 1) & 1);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- products
    constexpr uint32_t idesc_s = idesc(true, 128, 128, false);
    constexpr uint32_t idesc_o = idesc(true, 128, kNH, true) | kIdescAMnMajor;
    auto scores = [&](int i) {
      const uint32_t tile = k_addr + (i & 1) * kTileBytes, d = tmem + kSCol + (i & 1) * 128;
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          mma<true>(d, desc_sw128(tile + (k >> 2) * 1024 + (k & 3) * 32, 16, kGroupBytes),
                    desc_sw128(q_addr + (k >> 2) * kQBlock + (k & 3) * 32, 16, 1024), idesc_s, k > 0);
        mma_commit(bar(sm.s_full[i & 1]));
      }
      __syncwarp();
    };
    bool ok = warp_wait(cx, bar(sm.q_full), 0) && warp_wait(cx, bar(sm.k_full[0]), 0);
    if (ok) {
      tc_fence_after();
      scores(0);
    }
    for (int i = 0; ok && i < u.tiles; ++i) {
      if (i + 1 < u.tiles) {
        const int n = i + 1, use = n >> 1;
        ok = warp_wait(cx, bar(sm.k_full[n & 1]), use & 1);
        if (ok && use > 0) ok = warp_wait(cx, bar(sm.s_empty[n & 1]), (use - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        scores(n);
      }
      ok = warp_wait(cx, bar(sm.p_full[i & 1]), (i >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t tile = k_addr + (i & 1) * kTileBytes, pb = p_addr + (i & 1) * 2 * kPHalf;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t a = desc_sw128(tile + m * 1024 + k * 4 * kGroupBytes, 1024, kGroupBytes);
            mma<true>(tmem + kOCol + m * kNH, a, desc_sw64(pb + k * 32 * kNH, 512, 512), idesc_o, i > 0 || k > 0);
            mma<true>(tmem + kOCol + m * kNH, a, desc_sw64(pb + kPHalf + k * 32 * kNH, 512, 512), idesc_o, 1u);
          }
        mma_commit(bar(sm.pv_done[i & 1]));
      }
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------- softmax
    split_query(kp, u, smem + kOffQ, sm, warp, lane);
    if (threadIdx.x < kNH) sm.negref[threadIdx.x] = kUnset;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(sm.q_full));
    const int r = threadIdx.x;                    // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    float sum[kNH];
#pragma unroll
    for (int h = 0; h < kNH; ++h) sum[h] = 0.f;
    named_bar_sync(1, kSoftmaxThreads);           // qscale and negref are written
    float scale = row_scale(kp, u, u.tile0, r);
    bool failed = false;
    for (int i = 0; i < u.tiles; ++i) {
      const int b = i & 1;
      const float s = scale;
      if (i + 1 < u.tiles) scale = row_scale(kp, u, u.tile0 + i + 1, r);      // in flight during this tile
      const bool seen = s >= 0.f;
      const float ls = seen ? fmaxf(fast_log2(s), kMinScaleLog2) : 0.f;
      const float inv = seen ? fast_exp2(-ls) : 0.f;
      failed |= !warp_wait(cx, bar(sm.s_full[b]), (i >> 1) & 1);
      tc_fence_after();
      float d[kNH];                               // t - reference + headroom
#pragma unroll
      for (int g = 0; g < kNH; g += 32) {
        uint32_t hi[32], lo[32];
        tmem_ld32(tmem + lane_base + kSCol + b * 128 + g, hi);
        tmem_ld32(tmem + lane_base + kSCol + b * 128 + kNH + g, lo);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 32; ++h) {
          const float x = (__uint_as_float(hi[h]) + __uint_as_float(lo[h])) * sm.qscale[g + h];
          d[g + h] = seen ? fmaf(x, s, ls) : -INFINITY;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.s_empty[b]));
      float top = -INFINITY;
#pragma unroll
      for (int h = 0; h < kNH; ++h) top = fmaxf(top, d[h] + sm.negref[h]);
      if (named_bar_or(1, kSoftmaxThreads, failed || top > 2.f * kHeadroom)) {
        // ---- a new reference: the heads' maxima over the tile
        if (named_bar_or(1, kSoftmaxThreads, failed)) break;
#pragma unroll
        for (int h = 0; h < kNH; ++h) {
          const float m = warp_max(d[h]);
          if (lane == (h & 31)) sm.wmax[warp][h] = m;
        }
        named_bar_sync(1, kSoftmaxThreads);
        float neg = 0.f, a = 1.f;
        if (r < kNH) {
          float m = fmaxf(fmaxf(sm.wmax[0][r], sm.wmax[1][r]), fmaxf(sm.wmax[2][r], sm.wmax[3][r]));
          const float old = sm.negref[r];
          neg = m > -INFINITY ? fminf(old, kHeadroom - m) : old;
          a = fast_exp2(neg - old);
        }
        named_bar_sync(1, kSoftmaxThreads);
        if (r < kNH) {
          sm.negref[r] = neg;
          sm.factor[r] = a;
        }
        named_bar_sync(1, kSoftmaxThreads);
#pragma unroll
        for (int h = 0; h < kNH; ++h) sum[h] *= sm.factor[h];
        if (i > 0) {
          // O^T by column, once the products into it are done
          failed |= !warp_wait(cx, bar(sm.pv_done[b ^ 1]), ((i - 1) >> 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + kOCol + g * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * sm.factor[(g & 1) * 32 + h]);
            tmem_st32(tmem + lane_base + kOCol + g * 32, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
      }
      // P in E4M3 pairs: row r of the MN-major operand is 64 bytes, heads along it
      uint8_t* pb = smem + kOffP + b * 2 * kPHalf + r * kNH;
#pragma unroll
      for (int g = 0; g < kNH; g += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int h = g + 2 * e;
          const float x = fast_exp2(d[h] + sm.negref[h]), y = fast_exp2(d[h + 1] + sm.negref[h + 1]);
          sum[h] = fmaf(x, inv, sum[h]);
          sum[h + 1] = fmaf(y, inv, sum[h + 1]);
          split_pair(x, y, hi + e, lo + e);
        }
        const int at = ((g >> 4) ^ ((r >> 1) & 3)) << 4;                      // 64-byte swizzle
        *reinterpret_cast<uint4*>(pb + at) = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16,
                                                        hi[6] | hi[7] << 16);
        *reinterpret_cast<uint4*>(pb + kPHalf + at) = make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16,
                                                                 lo[4] | lo[5] << 16, lo[6] | lo[7] << 16);
      }
      if (!seen) {
        // the first product has read the row (its commit is what s_full waited for); the second must find zeros
        uint8_t* row = smem + kOffK + b * kTileBytes + (r >> 3) * kGroupBytes + (r & 7) * 128;
        for (int cb = 0; cb < 4; ++cb)
          for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(row + cb * 1024 + x * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.p_full[b]));
    }

    // ------------------------------------------------------------ results
    const int n = u.tiles - 1;
    failed |= !warp_wait(cx, bar(sm.pv_done[n & 1]), (n >> 1) & 1);
    tc_fence_after();
    if (!named_bar_or(1, kSoftmaxThreads, failed)) {
      // sums over the rows: transposed through the second tile buffer
      float* ts = reinterpret_cast<float*>(smem + kOffK + kTileBytes);
#pragma unroll
      for (int h = 0; h < kNH; ++h) ts[h * (kSoftmaxThreads + 1) + r] = sum[h];
      named_bar_sync(1, kSoftmaxThreads);
      const int h2 = r >> 1;
      float total = 0.f;
      for (int k = 0; k < kSoftmaxThreads / 2; ++k)
        total += ts[h2 * (kSoftmaxThreads + 1) + (r & 1) * (kSoftmaxThreads / 2) + k];
      total += __shfl_xor_sync(0xffffffffu, total, 1);
      if ((r & 1) == 0) {
        float f = 0.f, lse = -INFINITY;
        if (!(total == 0.f)) {                    // NaN passes
          lse = fast_log2(total) - sm.negref[h2];
          f = 1.f / total;
          if (p.num_splits == 1) {
            f *= load_scale(p.bmm2, p.bmm2_dev);
            if (p.sinks != nullptr && h2 < u.heads) f *= 1.f / (1.f + fast_exp2(__ldg(p.sinks + u.h0 + h2) * kLog2e - lse));
          }
        }
        sm.factor[h2] = f;
        if (h2 < u.heads) {
          if (p.num_splits > 1) p.part_lse[part + h2] = lse;
          else if (p.out_lse) p.out_lse[th + h2] = lse;
        }
      }
      named_bar_sync(1, kSoftmaxThreads);
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {               // dims 128 (g / 2) .. + 127, heads 32 (g % 2) .. + 31
        uint32_t o[32];
        tmem_ld32(tmem + lane_base + kOCol + g * 32, o);
        tmem_wait_ld();
        const int dim = (g >> 1) * 128 + r, hb = (g & 1) * 32;
        if (p.num_splits > 1) {
          float* dst = p.part_o + (part + hb) * kHeadDim + dim;
#pragma unroll
          for (int h = 0; h < 32; ++h)
            if (hb + h < u.heads) dst[h * kHeadDim] = __uint_as_float(o[h]) * sm.factor[hb + h];
        } else {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(smem + kOffK) + hb * kHeadDim + dim;
#pragma unroll
          for (int h = 0; h < 32; ++h) dst[h * kHeadDim] = __float2bfloat16_rn(__uint_as_float(o[h]) * sm.factor[hb + h]);
        }
      }
      if (p.num_splits == 1) {
        fence_proxy_async_smem();
        named_bar_sync(1, kSoftmaxThreads);
        if (r == 0) {
          bulk_store(p.out + th * kHeadDim, k_addr, u.heads * kHeadDim * 2);
          bulk_store_wait();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    if (sm.abort_flag) {                          // products may still be in flight: their commit comes last
      if (lane == 0) mma_commit(bar(sm.q_full));  // (phase 1 needs kSoftmaxWarps arrivals: one commit each)
      if (lane == 0)
        for (int k = 1; k < kSoftmaxWarps; ++k) mma_commit(bar(sm.q_full));
      drain_wait(bar(sm.q_full), 1);
    }
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merges the S normalised fp32 partials of every (token, head): weights
// 2^(LSE_s - LSE), then the sink and bmm2.
constexpr int kMergeThreads = 128;                // one (token, head): four dims a thread

__global__ void __launch_bounds__(kMergeThreads) window_merge_kernel(const WindowParams p) {
  const int64_t th = blockIdx.x;
  const int t = (int)(th / p.H), h = (int)(th % p.H), d = threadIdx.x * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* lse_s = p.part_lse + (int64_t)t * p.num_splits * p.H + h;
  const float* o_s = p.part_o + ((int64_t)t * p.num_splits * p.H + h) * kHeadDim + d;
  float mx = -INFINITY;
  bool nan = false;
  for (int s = 0; s < p.num_splits; ++s) {
    const float l = __ldg(lse_s + (int64_t)s * p.H);
    nan |= isnan(l);
    mx = fmaxf(mx, l);
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float wsum = 0.f;
  for (int s = 0; s < p.num_splits; ++s) {
    const float l = __ldg(lse_s + (int64_t)s * p.H);
    if (l == -INFINITY) continue;                 // an empty partial is not written
    const float w = fast_exp2(l - mx);
    const float4 o = __ldg(reinterpret_cast<const float4*>(o_s + (int64_t)s * p.H * kHeadDim));
    acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y), acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
    wsum += w;
  }
  float lse = -INFINITY, f = 0.f;
  if (mx != -INFINITY || nan) {
    lse = nan ? NAN : mx + fast_log2(wsum);
    f = load_scale(p.bmm2, p.bmm2_dev) / wsum;
    if (p.sinks != nullptr) f *= 1.f / (1.f + fast_exp2(__ldg(p.sinks + h) * kLog2e - lse));
  }
  uint2 v;
  v.x = pack_bf16x2(acc.x * f, acc.y * f);
  v.y = pack_bf16x2(acc.z * f, acc.w * f);
  *reinterpret_cast<uint2*>(p.out + th * kHeadDim + d) = v;
  if (threadIdx.x == 0 && p.out_lse) p.out_lse[th] = lse;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The pool as {128 bytes, 8 rows, 4 column blocks, row groups, pages}; box of
// `chunk` rows.  The call's checks make the base 16-byte aligned, every stride a
// multiple of 16 under 2^40 and page_size a multiple of 8.
cudaError_t encode_cache_map(CUtensorMap* map, const CacheView& c, int chunk) {
  static std::atomic<EncodeTiledFn> cached{nullptr};
  EncodeTiledFn fn = cached.load(std::memory_order_acquire);
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || ptr == nullptr) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeTiledFn>(ptr);
    cached.store(fn, std::memory_order_release);
  }
  const cuuint64_t dims[5] = {128, 8, 4, (cuuint64_t)c.page_size / 8, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)c.row_stride, 128, (cuuint64_t)(8 * c.row_stride), (cuuint64_t)c.page_stride};
  const cuuint32_t box[5] = {128, 8, 4, (cuuint32_t)chunk / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, c.rows, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_window_attention(const WindowParams& p, cudaStream_t stream) {
  KernelParams kp;
  kp.p = p;
  kp.chunk = p.c.page_size % 16 == 0 ? 16 : 8;
  kp.groups = (p.H + kNH - 1) / kNH;
  cudaError_t e = encode_cache_map(&kp.map, p.c, kp.chunk);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(window_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.c.sum_q * kp.groups * p.num_splits;
  window_kernel<<<(unsigned)grid, kThreads, kSmemBytes, stream>>>(kp);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.num_splits == 1) return e;
  // programmatic dependent launch: scheduled while the split kernel drains
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.sum_q * (int64_t)p.H));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_merge_kernel, p);
}

}  // namespace smla
