// Products of few tokens, or small ones, with weights held as FP4 entries
// (mla_fp4_linear; fp4_linear.cu takes the others).
//
// Bound: the weights' bytes (0.5625 per element) and, at a few MB, the latency of
// one launch, one trip to memory and one sum across warps. So there is no first
// kernel, ring or tensor memory: a CTA owns 16 rows, each of its warps some of their
// entries (512 channels). A warp requests all codes and scales of an entry at once,
// decodes them in registers straight into the A fragments of mma.m16n8k16 (8 tokens
// are one instruction's columns, and bf16 activations its B fragments as they are),
// and the warps' sums meet in shared memory in warp order. Measured, calls back to
// back: 512 to 200, one token, 2.0 us; 8192 to 4096 8.7 us (2.2 TB/s; a copy without
// the decoding 6.7); 16384 to 7168 26 us, where instructions bound it (970 for a warp's
// 16 rows of an entry, the logic pipe 76% busy on the SMs with four CTAs). Entries
// through a shared-memory ring of cp.async: the same 26 to 27 us.
//
// A code's magnitude bits at the bottom of a bf16's exponent and the top of its
// mantissa are its value times 2^-126 (subnormals included); times scale * 2^119
// they are weight * 2^-7, which is exact: E2M1 x E4M3 products have 6 significant
// bits and lie between 2^-10 and 2688. bf16 has float32's exponents, so the
// activations need no scaling here. The epilogue multiplies the sums by 2^7.
//
// The four lanes of a row read 64 adjacent bytes of codes. An MMA's K positions
// are, for lane t of them, channels i, i+4, i+1, i+5 of one of its words: any order
// serves as long as both operands use it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "fp4_linear.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 16;                   // of an SM: 128 registers a thread
constexpr int kRows = 16;                    // of a CTA

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// volatile, as the codes' loads: each stays where the program has it
__device__ __forceinline__ uint4 ld_x(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t bits(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// The eight codes of a word times 2^-126 s: codes i and i + 4 in v[i]. A nibble n at
// the bottom of a half, or four bits up, becomes n << 12 + n << 6 by one multiply: its
// sign is then bit 15, its magnitude bits 6 .. 8.
__device__ __forceinline__ void decode8(uint32_t w, __nv_bfloat162 s, uint32_t (&v)[4]) {
  const uint32_t w8 = w >> 8;
  const uint32_t n[4] = {(w & 0x000f000fu) * 0x1040u, (w & 0x00f000f0u) * 0x104u, (w8 & 0x000f000fu) * 0x1040u,
                         (w8 & 0x00f000f0u) * 0x104u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = n[i] & 0x81c081c0u;
    v[i] = bits(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u), s));
  }
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kN: blocks of 8 tokens.
template <int kN>
__global__ void __launch_bounds__(32 * kWarps) fp4_few_kernel(const mla_fp4_linear_args a, int tiles) {
  extern __shared__ float part[];            // [warps][tokens][rows]
  constexpr int kToks = 8 * kN;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int g = blockIdx.x / tiles, n0 = (blockIdx.x - g * tiles) * kRows;
  const int T = a.B * a.Q, t0 = blockIdx.y * kToks, entries = a.K / kCkv;

  const uint8_t* row[2];                     // gid and gid + 8; rows past the last repeat it and are not stored
#pragma unroll
  for (int h = 0; h < 2; ++h)
    row[h] = reinterpret_cast<const uint8_t*>(a.w) +
             ((int64_t)g * a.N + min(n0 + 8 * h + gid, a.N - 1)) * entries * kFp4EntryBytes;
  const __nv_bfloat16* x[kN];                // likewise tokens past the last: a column of its own each
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int t = min(t0 + 8 * j + gid, T - 1);
    x[j] = reinterpret_cast<const __nv_bfloat16*>(a.x) + (int64_t)(t / a.Q) * a.x_batch_stride +
           (int64_t)(t % a.Q) * a.x_token_stride + (int64_t)g * a.x_group_stride + 32 * tig;
  }
  float acc[kN][4];
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;

  // a step's codes are requested an entry ahead, into the registers it just left
  uint4 q[2][4];
  uint2 sc[2];
  auto codes = [&](int h, int e, int s) { return ld_stream(row[h] + (int64_t)e * kFp4EntryBytes + 64 * s + 16 * tig); };
  auto scales = [&](int h, int e) {          // those of step s = tig
    return *reinterpret_cast<const uint2*>(row[h] + (int64_t)e * kFp4EntryBytes + 256 + 8 * tig);
  };
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h) q[h][s] = codes(h, warp, s);
#pragma unroll
  for (int h = 0; h < 2; ++h) sc[h] = scales(h, warp);

  // the activations too, where registers allow it, a step ahead (8192 to 4096, one
  // token: 10.1 -> 8.7 us)
  constexpr bool kAhead = kN == 1;
  auto act = [&](int j, int e, int s, int w) { return ld_x(x[j] + (int64_t)e * a.x_block_stride + 128 * s + 8 * w); };
  uint4 xn[kN][4];
  if constexpr (kAhead) {
#pragma unroll
    for (int j = 0; j < kN; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) xn[j][w] = act(j, warp, 0, w);
  }

#pragma unroll 1
  for (int e = warp; e < entries; e += warps) {
    const bool more = e + warps < entries;
    const uint2 sc_now[2] = {sc[0], sc[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (more) sc[h] = scales(h, e + warps);
#pragma unroll
    for (int s = 0; s < 4; ++s) {            // 128 channels, 32 per lane
      uint4 xv[kN][4];
#pragma unroll
      for (int j = 0; j < kN; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if constexpr (kAhead) {
            xv[j][w] = xn[j][w];
            if (s < 3 || more) xn[j][w] = act(j, s < 3 ? e : e + warps, (s + 1) & 3, w);
          } else {
            xv[j][w] = act(j, e, s, w);
          }
        }
      uint32_t now[2][4];
      __nv_bfloat162 m[2][2];                // 2^119 x the lane's two scales of a row
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        now[h][0] = q[h][s].x;
        now[h][1] = q[h][s].y;
        now[h][2] = q[h][s].z;
        now[h][3] = q[h][s].w;
        if (more) q[h][s] = codes(h, e + warps, s);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __shfl_sync(0xffffffffu, sc_now[h].x, s, 4), hi = __shfl_sync(0xffffffffu, sc_now[h].y, s, 4);
        const uint32_t two = ((tig & 2) ? hi : lo) >> (16 * (tig & 1));
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
        m[h][0] = __float2bfloat162_rn(f.x * 0x1p119f);
        m[h][1] = __float2bfloat162_rn(f.y * 0x1p119f);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {          // 8 channels
        uint32_t v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) decode8(now[h][w], m[h][w >> 1], v[h]);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const uint4 u = xv[j][w];          // as channels i and i + 4
          mma16816(acc[j], v[0][0], v[1][0], v[0][1], v[1][1], __byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632));
          mma16816(acc[j], v[0][2], v[1][2], v[0][3], v[1][3], __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
        }
      }
    }
  }

  float* mine = part + warp * kToks * kRows;
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) mine[(8 * j + 2 * tig + (k & 1)) * kRows + 8 * (k >> 1) + gid] = acc[j][k];
  __syncthreads();
  const double f = (double)a.scale * 128.0;
  for (int i = threadIdx.x; i < min(kToks, T - t0) * kRows; i += blockDim.x) {
    const int t = t0 + i / kRows, n = n0 + i % kRows;
    float sum = part[i];
    for (int k = 1; k < warps; ++k) sum += part[k * kToks * kRows + i];
    if (n < a.N)
      reinterpret_cast<__nv_bfloat16*>(a.out)[((int64_t)t * a.G + g) * a.N + n] = __float2bfloat16_rn((float)(sum * f));
  }
}

template <int kN>
cudaError_t launch(const mla_fp4_linear_args* a, int sms, cudaStream_t st) {
  const int tiles = (a->N + kRows - 1) / kRows;
  const int blocks = (a->B * a->Q + 8 * kN - 1) / (8 * kN);
  const int64_t ctas = (int64_t)a->G * tiles * blocks;
  // The 16 warps that an SM holds go to as many CTAs as it gets, up to four: 11.2,
  // 9.0 and 10.8 us with 16, 8 and 4 warps for 256 CTAs (8192 to 4096, one token),
  // 32.8, 28.1 and 28.0 for 448 (16384 to 7168), 5.5, 6.3 and 9.4 for 96.
  const int warps = std::min(ctas <= sms ? kWarps : ctas <= 2 * sms ? kWarps / 2 : kWarps / 4, a->K / kCkv);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(a->G * tiles), (unsigned)blocks);
  cfg.blockDim = dim3((unsigned)(32 * warps));
  cfg.dynamicSmemBytes = (size_t)warps * kRows * 8 * kN * sizeof(float);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_few_kernel<kN>, *a, tiles);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// This kernel against the other with its two launches, in us: 512 to 200 2.0 : 6.4
// (one token), 3.3 : 12.0 (64); 4096 to 1000 5.1 : 8.4 (16), 8.1 : 11.0 (64), 13.5 : 12.1
// (96); 7168 to 1536 5.8 : 9.1 (1), 8.0 : 10.2 (16), 12.1 : 10.3 (24); 8192 to 4096 8.9 :
// 13.2 (1), 10.5 : 13.4 (8), 14.4 : 13.6 (16); 16384 to 7168 26.2 : 28.3 (1), 30.9 : 28.2
// (8). Every 16 tokens read all weights again and every 16 rows all activations, so
// the limits are on tokens x weights, and on the weights where they are read twice.
bool fp4_few_tokens(const mla_fp4_linear_args* a) {
  // G*N is at most 2^30; K is at least 512, so a grid dimension holds the blocks of tokens
  const int64_t tokens = (int64_t)a->B * a->Q, weights = (int64_t)a->G * a->N * a->K;
  return weights <= ((int64_t)1 << 28) / tokens && (tokens <= 16 || weights <= 1 << 23);
}

cudaError_t launch_fp4_few(const mla_fp4_linear_args* a, int sms, cudaStream_t st) {
  return a->B * a->Q <= 8 ? launch<1>(a, sms, st) : launch<2>(a, sms, st);
}

}  // namespace mla
