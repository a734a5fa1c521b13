// Merge of the split partials of the shared-prefix decode:
//   L = log(sum_s e^{lse_s} [+ e^{sink}]),  x = sum_s e^{lse_s - L} O_s.
// A split that saw nothing of a row has lse = -inf and no O; a NaN lse (a
// non-finite input the row sees) makes the row NaN.
//
// A row's lse values are reduced across a warp's lanes; each lane owns 16 columns
// and issues its 16-byte loads of four splits before it uses them, so a row
// costs a few memory latencies. With few rows, four warps take a quarter of the
// row's splits each and meet in shared memory (latency: a quarter); with many,
// one warp per row fills the GPU.
#include "prefix.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

template <typename T, int kShare>
__global__ void __launch_bounds__(128) prefix_combine(const PrefixParams p) {
  constexpr int kCols = kCkv / 32, kGroup = 4;
  __shared__ float4 sums[kShare > 1 ? kShare - 1 : 1][kCkv / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = kShare > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + warp;
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  if (r >= p.N) return;                          // whole warp; with kShare > 1 never
  const int S = p.num_splits;
  const float sink = p.sinks ? p.sinks[(int)(r % p.HQ) / p.Q] : -INFINITY;
  float m = sink;
  bool nan = false;
  for (int s = lane; s < S; s += 32) {
    const float l = p.ws_lse[(int64_t)s * p.N + r];
    nan = nan || isnan(l);
    m = fmaxf(m, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  nan = __any_sync(0xffffffffu, nan);
  float den = 0.f;
  if (m != -INFINITY) {
    for (int s = lane; s < S; s += 32) den += expf(p.ws_lse[(int64_t)s * p.N + r] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    den += expf(sink - m);
  }
  const float L = nan ? NAN : m == -INFINITY ? -INFINITY : m + logf(den);

  const int c0 = lane * kCols;
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
  // this warp's splits
  const int s_begin = kShare > 1 ? (int)((int64_t)S * warp / kShare) : 0;
  const int s_end = kShare > 1 ? (int)((int64_t)S * (warp + 1) / kShare) : S;
  for (int s0 = s_begin; s0 < s_end; s0 += kGroup) {
    float4 v[kGroup][kCols / 4];
    float w[kGroup];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int64_t sr = (int64_t)min(s0 + g, s_end - 1) * p.N + r;
      const float l = p.ws_lse[sr];
      w[g] = (s0 + g >= s_end || l == -INFINITY) ? 0.f : expf(l - L);
      const float4* src = reinterpret_cast<const float4*>(p.ws_o + sr * kCkv + c0);
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) v[g][i] = src[i];
    }
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      if (w[g] == 0.f) continue;                 // an unwritten partial is not used
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        acc[4 * i] = fmaf(w[g], v[g][i].x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(w[g], v[g][i].y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(w[g], v[g][i].z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(w[g], v[g][i].w, acc[4 * i + 3]);
      }
    }
  }
  if constexpr (kShare > 1) {
    // in warp order; column group i of lane l at [i][l], so lanes hit all banks
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i)
      if (warp > 0) sums[warp - 1][32 * i + lane] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 0; k < kShare - 1; ++k)
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 o = sums[k][32 * i + lane];
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
  if (p.lse && lane == 0) p.lse[r] = L;
}

template <typename T, int kShare>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kShare > 1 ? (unsigned)p.N : (unsigned)(((int64_t)p.N + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_combine<T, kShare>, p);
}

}  // namespace

cudaError_t launch_prefix_combine(const PrefixParams& p, bool bf16, cudaStream_t st) {
  // few rows, and more splits than a warp loads at a time (whole calls of 1024 rows, one
  // warp a row against four: 22.3 : 25.4 us with 4 splits, 25.3 : 21.6 with 9; of 2048
  // rows 38.0 : 39.3 with 9)
  const bool few = p.N <= 1024 && p.num_splits > 4;
  cudaError_t e;
  if (bf16)
    e = few ? launch<__nv_bfloat16, 4>(p, st) : launch<__nv_bfloat16, 1>(p, st);
  else
    e = few ? launch<float, 4>(p, st) : launch<float, 1>(p, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
