// Merge of the split partials of the shared-prefix decode:
//   L = log(sum_s e^{lse_s} [+ e^{sink}]),  x = sum_s e^{lse_s - L} O_s.
// A split that saw nothing of a row has lse = -inf and O = 0 (every row of every
// split that the row's block uses is written); a NaN lse (a non-finite input the row sees) makes the row NaN.
//
// A row's lse values are reduced across a warp's lanes, which keep the splits' weights
// and hand them round. With many rows, one warp per row fills the GPU: each lane owns
// 16 columns and has its loads of four splits in flight. With few rows what counts is
// latency: eight warps take a row's four quarters and both halves of its splits, eight
// splits in flight, and the halves meet in shared memory.
#include "prefix.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

// kQuarters: parts of a row's columns, kShare: ranges of its splits, a warp each. kAsks:
// the blocks said how many splits they used.
template <typename T, int kQuarters, int kShare, bool kAsks>
__global__ void __launch_bounds__(kQuarters* kShare > 1 ? 32 * kQuarters * kShare : 128)
    prefix_combine(const PrefixParams p) {
  constexpr bool kRowPerCta = kQuarters * kShare > 1;
  constexpr int kCols = kCkv / 32 / kQuarters, kGroup = kRowPerCta ? 8 : 4;
  constexpr int kHeld = kPrefixMaxSplits / 32;   // weights a lane keeps
  __shared__ float4 sums[kShare > 1 ? kShare - 1 : 1][kCkv / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = kRowPerCta ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + warp;
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  if (r >= p.N) return;                          // whole warp; with a row per CTA never
  int S = p.num_splits;
  if constexpr (kAsks) S = min(S, p.ws_ranges[r >> p.block_shift]);
  const float sink = p.sinks ? p.sinks[(int)(r % p.HQ) / p.Q] : -INFINITY;
  float m = sink, w[kHeld];
  bool nan = false;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int s = lane + 32 * k;
    w[k] = -INFINITY;
    if (s < p.num_splits) w[k] = p.ws_lse[(int64_t)s * p.N + r];   // all, not behind the load of S
    if constexpr (kAsks) w[k] = s < S ? w[k] : -INFINITY;
    nan = nan || isnan(w[k]);
    m = fmaxf(m, w[k]);
  }
  if (kAsks && S == 1) return;                   // the row is final (the same for the row's warps)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  nan = __any_sync(0xffffffffu, nan);
  float den = 0.f;
  if (m != -INFINITY) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (32 * k < S) den += expf(w[k] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    den += expf(sink - m);
  }
  const float L = nan ? NAN : m == -INFINITY ? -INFINITY : m + logf(den);
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (32 * k < S) w[k] = w[k] == -INFINITY ? 0.f : expf(w[k] - L);

  const int quarter = kRowPerCta ? warp % kQuarters : 0, share = kRowPerCta ? warp / kQuarters : 0;
  const int c0 = quarter * (kCkv / kQuarters) + lane * kCols;
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
  // this warp's splits
  const int s_begin = (int)((int64_t)S * share / kShare), s_end = (int)((int64_t)S * (share + 1) / kShare);
#pragma unroll 1
  for (int s0 = s_begin; s0 < s_end; s0 += kGroup) {
    float4 v[kGroup][kCols / 4];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const float4* src =
          reinterpret_cast<const float4*>(p.ws_o + ((int64_t)min(s0 + g, s_end - 1) * p.N + r) * kCkv + c0);
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) v[g][i] = src[i];
    }
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int s = s0 + g;                      // the same for all lanes
      float held = w[0];
      if (S > 32) {
#pragma unroll
        for (int k = 1; k < kHeld; ++k)
          if (s >= 32 * k) held = w[k];
      }
      const float wt = s < s_end ? __shfl_sync(0xffffffffu, held, s & 31) : 0.f;
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        acc[4 * i] = fmaf(wt, v[g][i].x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(wt, v[g][i].y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(wt, v[g][i].z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(wt, v[g][i].w, acc[4 * i + 3]);
      }
    }
  }
  if constexpr (kShare > 1) {
    // in order of the ranges; column group i of lane l at [i][l], so lanes hit all banks
    float4* mine = &sums[0][quarter * (kCkv / 4 / kQuarters)];
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i)
      if (share > 0)
        mine[(share - 1) * (kCkv / 4) + 32 * i + lane] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    __syncthreads();
    if (share > 0) return;
#pragma unroll
    for (int k = 0; k < kShare - 1; ++k)
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 o = mine[k * (kCkv / 4) + 32 * i + lane];
        acc[4 * i] += o.x;
        acc[4 * i + 1] += o.y;
        acc[4 * i + 2] += o.z;
        acc[4 * i + 3] += o.w;
      }
  }
  T* xo = reinterpret_cast<T*>(p.x) + r * kCkv + c0;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < kCols; i += 4)
      *reinterpret_cast<uint2*>(xo + i) =
          make_uint2(sm100::pack_bf16(acc[i], acc[i + 1]), sm100::pack_bf16(acc[i + 2], acc[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < kCols; i += 4)
      *reinterpret_cast<float4*>(xo + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
  }
  if (p.lse && lane == 0 && quarter == 0) p.lse[r] = L;
}

template <typename T, int kQuarters, int kShare>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  constexpr int kWarps = kQuarters * kShare;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kWarps > 1 ? (unsigned)p.N : (unsigned)(((int64_t)p.N + 3) / 4));
  cfg.blockDim = dim3(kWarps > 1 ? 32 * kWarps : 128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.ws_ranges ? cudaLaunchKernelEx(&cfg, prefix_combine<T, kQuarters, kShare, true>, p)
                     : cudaLaunchKernelEx(&cfg, prefix_combine<T, kQuarters, kShare, false>, p);
}

}  // namespace

cudaError_t launch_prefix_combine(const PrefixParams& p, bool bf16, cudaStream_t st) {
  // few rows, and more splits than a warp loads at a time (whole calls of 1024 rows, one
  // warp a row against eight: 21.7 : 25 us with 4 splits, 25 : 20 with 9; of 2048 rows
  // 35 : 39 with 9)
  const bool few = p.N <= 1024 && p.num_splits > 4;
  cudaError_t e;
  if (bf16)
    e = few ? launch<__nv_bfloat16, 4, 2>(p, st) : launch<__nv_bfloat16, 1, 1>(p, st);
  else
    e = few ? launch<float, 4, 2>(p, st) : launch<float, 1, 1>(p, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
