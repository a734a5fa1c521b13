// Products of few tokens with weights held as FP4 entries (mla_fp4_linear):
// one warp per output row and block of 8 tokens; lane i owns scale group i of
// every 512-channel entry (8 code bytes, one scale byte) and the row's dot
// products are summed across the lanes at the end, in float32.
#include "common.cuh"
#include "fp4_linear.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kTok = 8;

__global__ void __launch_bounds__(128) fp4_linear_simple(const mla_fp4_linear_args a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);   // g * N + n
  if (row >= (int64_t)a.G * a.N) return;
  const int g = (int)(row / a.N);
  const int T = a.B * a.Q;
  const int t0 = blockIdx.y * kTok, nt = min(kTok, T - t0);
  const int blocks = a.K / kCkv;
  const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w) + row * blocks * kFp4EntryBytes;
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x) + g * a.x_group_stride + 16 * lane;
  const __nv_bfloat16* xt[kTok];
  for (int t = 0; t < kTok; ++t) {
    const int tt = t0 + min(t, nt - 1);
    xt[t] = x + (int64_t)(tt / a.Q) * a.x_batch_stride + (int64_t)(tt % a.Q) * a.x_token_stride;
  }
  float acc[kTok] = {};
  for (int k = 0; k < blocks; ++k) {
    const uint8_t* e = w + (int64_t)k * kFp4EntryBytes;
    const uint2 c = *reinterpret_cast<const uint2*>(e + 8 * lane);
    const float s = e4m3_value(e[kCkv / 2 + lane]);
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = e2m1_value((c.x >> (4 * j)) & 15u) * s;
      v[8 + j] = e2m1_value((c.y >> (4 * j)) & 15u) * s;
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const __nv_bfloat16* xp = xt[t] + (int64_t)k * a.x_block_stride;
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[t] = fmaf(__bfloat162float(xp[j]), v[j], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if (lane == 0 && t < nt)
      reinterpret_cast<__nv_bfloat16*>(a.out)[(int64_t)(t0 + t) * a.G * a.N + row] =
          __float2bfloat16_rn(acc[t] * a.scale);
  }
}

}  // namespace

size_t fp4_linear_workspace_bytes(const mla_fp4_linear_args*, int) { return 0; }

cudaError_t launch_fp4_linear(const mla_fp4_linear_args* a, void*, int, cudaStream_t st) {
  const int64_t rows = (int64_t)a->G * a->N;
  const dim3 grid((unsigned)((rows + 3) / 4), (unsigned)((a->B * a->Q + kTok - 1) / kTok));
  fp4_linear_simple<<<grid, 128, 0, st>>>(*a);
  return cudaGetLastError();
}

}  // namespace mla
