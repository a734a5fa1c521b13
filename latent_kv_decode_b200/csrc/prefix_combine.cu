// Merge of the split partials of the shared-prefix decode:
//   L = log(sum_s e^{lse_s} [+ e^{sink}]),  x = sum_s e^{lse_s - L} O_s.
// A split that saw nothing of a row has lse = -inf and no O; a NaN lse (a
// non-finite input the row sees) makes the row NaN.
//
// kParts warps per row, each over 512 / kParts columns: every warp reduces the
// row's lse values across its lanes, and each lane issues its 16-byte loads of
// four splits before it uses them, so a row costs a few memory latencies.
#include "prefix.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

template <typename T, int kParts>
__global__ void __launch_bounds__(128) prefix_combine(const PrefixParams p) {
  constexpr int kCols = kCkv / (32 * kParts), kGroup = 4;
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t r = gw / kParts;
  const int part = (int)(gw % kParts);
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  if (r >= p.N) return;                          // whole warp
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

  const int c0 = part * (32 * kCols) + lane * kCols;
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < S; s0 += kGroup) {
    float4 v[kGroup][kCols / 4];
    float w[kGroup];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int64_t sr = (int64_t)min(s0 + g, S - 1) * p.N + r;
      const float l = p.ws_lse[sr];
      w[g] = (s0 + g >= S || l == -INFINITY) ? 0.f : expf(l - L);
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
  if (p.lse && lane == 0 && part == 0) p.lse[r] = L;
}

template <typename T, int kParts>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.N * kParts + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_combine<T, kParts>, p);
}

}  // namespace

cudaError_t launch_prefix_combine(const PrefixParams& p, bool bf16, cudaStream_t st) {
  // few rows: four warps each keep enough loads in flight
  const bool few = p.N < 1024;
  cudaError_t e;
  if (bf16)
    e = few ? launch<__nv_bfloat16, 4>(p, st) : launch<__nv_bfloat16, 1>(p, st);
  else
    e = few ? launch<float, 4>(p, st) : launch<float, 1>(p, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
