// Products of few tokens with weights held as FP4 entries (mla_fp4_linear).
//
// The weights are the bytes: 0.5625 per element, read once per 64 tokens. What
// it takes to stream them is to turn 4-bit codes into tensor-core operands as
// fast as HBM delivers them (about 40 weights per clock and SM), so the operand
// type is float16: a code's magnitude bits moved to the bottom of the exponent
// and the top of the mantissa are its value times 2^-14 (subnormals included),
// so two shifts, two logic operations and one multiply by scale * 2^7 make two
// weights times 2^-7. That is exact: E2M1 x E4M3 products are multiples of 2^-10
// with 6 significant bits, at most 2688. (The conversion instruction runs on
// the pipe of the special functions, 16 lanes a clock: 50 us for the 66 MB of
// the 16384 x 7168 case, where that pipe was 71% busy.) The activations follow: a
// first kernel scales each token's row by a power of two that brings its
// largest finite magnitude to [2^14, 2^15) and stores it as float16. bf16 values keep their 8 bits down to 2^-29 of that
// magnitude, and below it the error is under 2^-40 of it, far below float32's
// accumulation. The epilogue takes the power of two out again.
//
//   x_to_f16      one CTA per (token, group): largest magnitude, then the row.
//   fp4_linear    one cluster of S CTAs per 128 output rows and 64 tokens, each a
//                 range of K in chunks of 128. 8 warps load codes and scales from
//                 global memory kAhead chunks ahead, convert, and write the K-major
//                 128-byte-swizzled A tile; TMA brings the tokens' B tile; one warp
//                 issues the MMAs (M = 128, N = tokens) into TMEM. The S partial
//                 sums meet through distributed shared memory in a fixed order.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "fp4_linear.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kRowsM = 128;                  // output rows per cluster
constexpr int kTokMax = 64;                  // tokens per cluster
constexpr int kChunkK = 128;                 // channels per stage: two 64-wide swizzled blocks
constexpr int kABytes = kRowsM * kChunkK * 2;
constexpr int kConv = 256;                   // converting threads
constexpr int kThreads = kConv + 64;         // + TMA warp + MMA warp
constexpr int kAhead = 3;                    // chunks a converting thread has in flight
constexpr int kMaxStages = 3;

enum : int { B_AF = 0, B_XF = kMaxStages, B_EMPTY = 2 * kMaxStages, B_DONE = 3 * kMaxStages, B_COUNT = B_DONE + 1 };

struct alignas(64) LinearParams {
  CUtensorMap tm_x;                          // scaled activations (K, T, G) float16, box 64 x tokens
  const uint8_t* w;
  const int* exps;                           // (G, T): token t's row holds x 2^-exps
  __nv_bfloat16* out;
  int T, G, N, K;
  int tok_pad;                               // tokens per cluster, a multiple of 16
  int tiles;                                 // 128-row tiles per group
  int stages;
  float scale;
  int32_t* err;
};

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) x_to_f16(const mla_fp4_linear_args a, __half* xs, int* exps) {
  __shared__ uint32_t top[8];
  pdl_wait();
  pdl_launch_dependents();                   // after the wait: what follows may read the weights at once
  const int t = blockIdx.x, g = blockIdx.y, T = a.B * a.Q;
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x) + (int64_t)(t / a.Q) * a.x_batch_stride +
                           (int64_t)(t % a.Q) * a.x_token_stride + (int64_t)g * a.x_group_stride;
  auto load = [&](int k) {
    return *reinterpret_cast<const uint4*>(x + (int64_t)(k >> 9) * a.x_block_stride + (k & 511));
  };
  // the largest finite magnitude, as bf16 bits
  constexpr int kHold = 4;                   // vectors kept between the two passes: K up to 8192
  uint4 v[kHold];
  uint32_t m = 0;
  auto fold = [&](const uint4& u) {
    const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = wd[i] & 0x7fffu, hi = (wd[i] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) m = max(m, lo);
      if (hi < 0x7f80u) m = max(m, hi);
    }
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = 8 * (threadIdx.x + 256 * i);
    if (k < a.K) v[i] = load(k);
  }
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (8 * (threadIdx.x + 256 * i) < a.K) fold(v[i]);
  for (int k = 8 * (threadIdx.x + 256 * kHold); k < a.K; k += 8 * 256) fold(load(k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, top[i]);
  int e = 0;
  if (m != 0) e = ilogbf(__uint_as_float(m << 16)) - 14;
  if (threadIdx.x == 0) exps[g * T + t] = e;
  // x 2^-e in two exact steps (either factor alone may pass float32's range)
  const float f1 = scalbnf(1.f, -e / 2), f2 = scalbnf(1.f, -e - (-e / 2));
  __half* dst = xs + ((int64_t)g * T + t) * a.K;
  auto store = [&](int k, const uint4& u) {
    // channels in the order 0 4 1 5 2 6 3 7 that the weights decode to
    const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(wd[i] << 16) * f1 * f2;
      f[2 * i + 1] = __uint_as_float(wd[i] & 0xffff0000u) * f1 * f2;
    }
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[i], f[i + 4]);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(dst + k) = make_uint4(r[0], r[1], r[2], r[3]);
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = 8 * (threadIdx.x + 256 * i);
    if (k < a.K) store(k, v[i]);
  }
  for (int k = 8 * (threadIdx.x + 256 * kHold); k < a.K; k += 8 * 256) store(k, load(k));
}

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
  return e;
}

// One MMA, or a commit, by the elected lane (e != 0) of a converged warp.
__device__ __forceinline__ void mma_one(uint32_t e, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t e, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(e)
      : "memory");
}

// kind::f16 with float16 A and B, float32 D
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// codes i and i + 4 of a word times 2^-14 s
template <int i>
__device__ __forceinline__ uint32_t decode2(uint32_t w, __half2 s) {
  const uint32_t mag = i < 3 ? w << (9 - 4 * (i < 3 ? i : 0)) : w >> 3;   // bits 4i .. 4i+2 to 9 .. 11
  const uint32_t sgn = w << (12 - 4 * i);                                  // bit 4i+3 to 15
  const uint32_t u = (mag & 0x0e000e00u) | (sgn & 0x80008000u);
  return half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&u), s));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads, 2) fp4_linear_kernel(const __grid_constant__ LinearParams P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[B_COUNT];
  __shared__ uint32_t tmem_ptr;
  __shared__ int failed;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb0 = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb0 - raw);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };
  const int stage_bytes = kABytes + P.tok_pad * kChunkK * 2;

  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
  const uint32_t rank = cluster_ctarank();
  const int tile = blockIdx.x / S;           // (group, 128 rows)
  const int g = tile / P.tiles, n0 = (tile - g * P.tiles) * kRowsM;
  const int t0 = blockIdx.y * kTokMax;
  const int chunks = P.K / kChunkK;
  const int c_begin = (int)((int64_t)chunks * rank / S), nc = (int)((int64_t)chunks * (rank + 1) / S) - c_begin;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(bar(B_AF + i), kConv / 32);
      mbar_init(bar(B_XF + i), 1);
      mbar_init(bar(B_EMPTY + i), 1);
    }
    mbar_init(bar(B_DONE), 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == kConv / 32) {
    tmem_alloc(smem_u32(&tmem_ptr), 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&tmem_ptr), 0);
  bool ok = true;

  if (warp < kConv / 32) {
    // ------------------------------------------------------------------ converting warps
    // lane: row 8 warp + lane / 4 (and 64 further on), channels 32 (lane % 4) .. + 31
    // of the chunk: 16 bytes of codes and two scales
    const int seg = lane & 3;
    const uint8_t* src[2];
    uint32_t dst[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 64 * h + 8 * warp + (lane >> 2);
      const int64_t row = (int64_t)g * P.N + min(n0 + r, P.N - 1);       // rows behind the last repeat it
      src[h] = P.w + row * (P.K / kCkv) * kFp4EntryBytes;
      dst[h] = (uint32_t)((seg >> 1) * (kRowsM * 128) + r * 128);
    }
    const int sw = (8 * warp + (lane >> 2)) & 7, c16 = 4 * (seg & 1), flip = (seg >> 1) << 1;
    uint4 q[kAhead][2];
    uint32_t sc[kAhead][2];
    auto fetch = [&](int c, uint4 (&qq)[2], uint32_t (&ss)[2]) {
      if (c >= nc) return;
      const int k = (c_begin + c) * kChunkK;
      const int64_t e = (int64_t)(k >> 9) * kFp4EntryBytes;
      const int in = k & 511;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* p = src[h] + e;
        qq[h] = __ldcs(reinterpret_cast<const uint4*>(p + in / 2 + 16 * seg));
        ss[h] = __ldcs(reinterpret_cast<const unsigned short*>(p + kCkv / 2 + in / 16 + 2 * seg));
      }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(u, q[u], sc[u]);
    int stage = 0, ph = 1;                   // the ring starts empty
    for (int c0 = 0; c0 < nc && ok; c0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (c0 + u >= nc || !ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_EMPTY + stage), ph));
        if (!ok) break;
        uint8_t* A = smem + stage * stage_bytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2 s2 = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)sc[u][h], __NV_E4M3)),
                                     __float2half2_rn(128.f));
          const uint32_t wd[4] = {q[u][h].x, q[u][h].y, q[u][h].z, q[u][h].w};
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            // the two 64-channel blocks in another order, so that eight lanes hit all banks
            const uint32_t x = flip ? wd[ii ^ 2] : wd[ii];
            const int i = flip ? ii ^ 2 : ii;
            const __half2 s = i < 2 ? __low2half2(s2) : __high2half2(s2);
            const uint4 v = make_uint4(decode2<0>(x, s), decode2<1>(x, s), decode2<2>(x, s), decode2<3>(x, s));
            *reinterpret_cast<uint4*>(A + dst[h] + 16 * ((c16 + i) ^ sw)) = v;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_AF + stage));
        fetch(c0 + u + kAhead, q[u], sc[u]);
        if (++stage == P.stages) {
          stage = 0;
          ph ^= 1;
        }
      }
    }
  } else if (warp == kConv / 32) {
    // ------------------------------------------------------------------ token loads
    pdl_wait();                              // the first kernel's rows
    if (lane == 0) {
      tma_prefetch_desc(&P.tm_x);
      int stage = 0, ph = 1;
      for (int c = 0; c < nc; ++c) {
        ok = mbar_wait(bar(B_EMPTY + stage), ph);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(B_XF + stage), (uint32_t)(P.tok_pad * kChunkK * 2));
        const uint32_t xb = sb0 + stage * stage_bytes + kABytes;
        const int k = (c_begin + c) * kChunkK;
        tma_load_3d(xb, &P.tm_x, bar(B_XF + stage), k, t0, g);
        tma_load_3d(xb + P.tok_pad * 128, &P.tm_x, bar(B_XF + stage), k + 64, t0, g);
        if (++stage == P.stages) {
          stage = 0;
          ph ^= 1;
        }
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  } else {
    // ------------------------------------------------------------------ MMA issue
    const uint32_t el = elect_one();
    const uint32_t idesc = idesc_f16_f32(kRowsM, P.tok_pad);
    int stage = 0, ph = 0;
    for (int c = 0; c < nc; ++c) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(B_XF + stage), ph) && mbar_wait(bar(B_AF + stage), ph));
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = sb0 + stage * stage_bytes;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint64_t ad = smem_desc(base + b * (kRowsM * 128), 16, 1024, kSwizzle128B);
        const uint64_t bd = smem_desc(base + kABytes + b * P.tok_pad * 128, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_one(el, tmem, desc_advance(ad, 32 * k), desc_advance(bd, 32 * k), idesc, c > 0 || b > 0 || k > 0);
      }
      commit_one(el, bar(B_EMPTY + stage));
      if (++stage == P.stages) {
        stage = 0;
        ph ^= 1;
      }
    }
    if (ok && nc > 0) commit_one(el, bar(B_DONE));
  }
  if (!ok) *reinterpret_cast<volatile int*>(&failed) = 1;
  __syncthreads();
  pdl_wait();                                // exps, for every thread

  // ---------------------------------------------------------------- epilogue
  // this CTA's sums as [token][row] in shared memory; then rank r sums the
  // cluster's partial results of tokens r, r + S, ... in rank order
  float* part = reinterpret_cast<float*>(smem);
  if (nc > 0 && !failed && !mbar_wait(bar(B_DONE), 0)) *reinterpret_cast<volatile int*>(&failed) = 1;
  tc_fence_after();
  if (warp < 4) {
    for (int c = 0; c < P.tok_pad; c += 16) {
      uint32_t v[16];
      if (nc > 0) {
        tmem_ld16(tmem + ((uint32_t)(32 * warp) << 16) + (uint32_t)c, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0u;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c + i) * kRowsM + 32 * warp + lane] = __uint_as_float(v[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && failed && P.err) atomicOr(P.err, MLA_DEVICE_ERR_TIMEOUT);
  cluster_sync();
  if (warp < kConv / 32) {
    const int r = threadIdx.x & 127;
    const uint32_t mine = smem_u32(part);
    const int nt = min(P.tok_pad, P.T - t0);
    for (int i = (int)(threadIdx.x >> 7) * (int)S + (int)rank; i < nt; i += 2 * (int)S) {
      float sum = 0.f;
      for (uint32_t k = 0; k < S; ++k) sum += ld_cluster_f32(map_to_rank(mine + 4u * (uint32_t)(i * kRowsM + r), k));
      if (n0 + r < P.N)
        P.out[(int64_t)(t0 + i) * P.G * P.N + (int64_t)g * P.N + n0 + r] = __float2bfloat16_rn(
            (float)ldexp((double)sum * (double)P.scale, P.exps[g * P.T + t0 + i] + 7));
    }
  }
  cluster_sync();                            // the peers have read this CTA's sums
  if (warp == kConv / 32) tmem_dealloc(tmem, 64);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

size_t xs_bytes(const mla_fp4_linear_args* a) {
  return ((size_t)a->B * a->Q * a->G * a->K * 2 + 255) & ~(size_t)255;
}

}  // namespace

size_t fp4_linear_workspace_bytes(const mla_fp4_linear_args* a) {
  return xs_bytes(a) + (size_t)a->B * a->Q * a->G * sizeof(int);
}

cudaError_t launch_fp4_linear(const mla_fp4_linear_args* a, void* ws, int sms, cudaStream_t st) {
  if (!encode_fn()) return cudaErrorNotSupported;
  LinearParams P;
  memset(static_cast<void*>(&P), 0, sizeof(P));
  const int T = a->B * a->Q;
  __half* xs = reinterpret_cast<__half*>(ws);
  int* exps = reinterpret_cast<int*>(reinterpret_cast<char*>(ws) + xs_bytes(a));
  P.w = reinterpret_cast<const uint8_t*>(a->w);
  P.exps = exps;
  P.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  P.T = T;
  P.G = a->G;
  P.N = a->N;
  P.K = a->K;
  P.scale = a->scale;
  P.err = a->err_flag;
  P.tok_pad = T >= kTokMax ? kTokMax : (T + 15) / 16 * 16;
  P.tiles = (a->N + kRowsM - 1) / kRowsM;
  P.stages = P.tok_pad <= 16 ? 3 : 2;        // two CTAs per SM
  {
    const cuuint64_t d[3] = {(cuuint64_t)a->K, (cuuint64_t)T, (cuuint64_t)a->G};
    const cuuint64_t s[2] = {(cuuint64_t)a->K * 2, (cuuint64_t)a->K * 2 * T};
    const cuuint32_t bx[3] = {64, (cuuint32_t)P.tok_pad, 1}, el[3] = {1, 1, 1};
    if (encode_fn()(&P.tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, xs, d, s, bx, el, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)T, (unsigned)a->G);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, x_to_f16, *a, xs, exps);
  if (e != cudaSuccess) return e;

  // K over as many CTAs as two per SM hold, each with at least one chunk
  const int64_t clusters = (int64_t)a->G * P.tiles * ((T + kTokMax - 1) / kTokMax);
  const int64_t fit = 2 * sms / clusters;
  const int S = (int)(fit < 1 ? 1 : fit > 8 ? 8 : fit);   // K holds 4 chunks or more; a rank may get none
  const size_t smem = (size_t)P.stages * (kABytes + P.tok_pad * kChunkK * 2) + 1024;
  e = cudaFuncSetAttribute(fp4_linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(a->G * P.tiles * S), (unsigned)((T + kTokMax - 1) / kTokMax));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, fp4_linear_kernel, P);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
