// Products of few tokens with weights held as FP4 entries (mla_fp4_linear); the
// fewest tokens, and small products, go to fp4_few.cu's kernel.
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
// largest finite magnitude to [2^14, 2^15) and stores it as float16. bf16 values
// keep their 8 bits down to 2^-29 of that magnitude, and below it the error is
// at most 2^-39 of it (half of float16's smallest step), far below float32's
// accumulation. The epilogue takes the power of two out again.
//
//   x_to_f16      one CTA per (token, group): largest magnitude, then the row.
//   fp4_linear    one cluster of S CTAs per 128 or 256 output rows and 64 tokens,
//                 each a range of K in entries of 512 channels. TMA brings the
//                 rows' entries into a ring (codes as two swizzled 128-byte
//                 blocks, so that the rows' reads hit all banks, and scales); 16
//                 warps decode them, 128 channels at a time, straight into the A
//                 operand in tensor memory (through a shared-memory A tile its
//                 writes and reads were the bound); TMA brings the tokens' B tile;
//                 one warp issues the MMAs (M = 128, N = tokens). The S partial
//                 sums meet through distributed shared memory in rank order.
//
// Measured per call (two launches): 8 groups of 4096 to 1024, 32 tokens, 12.5 us;
// 16384 to 7168, 64 tokens, 30.7 us. With few tokens an MMA takes 24 ns whatever
// its N (128 of them per CTA), behind 4 us for launch, activations and first entries
// and before 2 us of exchange. With 64, the tokens' tiles are as many bytes as the
// weights (130 MB come into 112 SMs together, 4.1 TB/s), and no pipe is full: issue slots
// 59%, logic 46%, tensor 34% of the active cycles on average, 83, 61 and 45 on the busiest SM.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <mutex>

#include "common.cuh"
#include "fp4_linear.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTokMax = 64;                  // tokens per cluster
constexpr int kChunkK = 128;                 // channels per A stage (64 columns a half) and token tile (two swizzled blocks)
constexpr int kPer = kCkv / kChunkK;         // chunks per entry
constexpr int kConv = 512;                   // converting threads
constexpr uint32_t kTmemCols = 512;

// A CTA's rows: kHalves MMAs of 128, which share the token tiles. 256 rows halve
// the tokens' traffic, 128 spread the weights over twice the CTAs.
template <int kHalves> struct Shape {
  static constexpr int kRows = 128 * kHalves;
  static constexpr int kGroups = 4 / kHalves;            // chunks decoded at a time: four warps per 128 rows
  static constexpr int kCode = kRows * 128;              // bytes of one of an entry's two code blocks
  static constexpr int kRawBytes = kRows * kFp4EntryBytes;
  // stages: entries, A chunks (64 columns a half, behind the halves' sums)
  static constexpr int kRaw = 4 / kHalves, kA = 8 / kHalves - 1;
  static constexpr uint32_t kColA = 64 * kHalves, kColStage = 64 * kHalves;
  // token tiles: as many as the 64 KB beside the entries hold. A tile arrives up to
  // a microsecond or more after its request, as it queues behind the entries.
  static constexpr int kXMax = 16;
  static constexpr int x_stages(int tok_pad) { return 65536 / (tok_pad * kChunkK * 2); }
  static constexpr size_t smem(int tok_pad) {
    return (size_t)kRaw * kRawBytes + (size_t)x_stages(tok_pad) * tok_pad * kChunkK * 2 + 1024;
  }
  enum : int {
    B_RF = 0,                // [kRaw] entries landed
    B_RE = B_RF + kRaw,      // [kRaw] entries converted (one arrival per converting warp)
    B_AF = B_RE + kRaw,      // [kA] A stage written (one arrival per warp of its group)
    B_AE = B_AF + kA,        // [kA] MMAs over the A stage done
    B_XF = B_AE + kA,        // [kXMax] token tile landed
    B_XE = B_XF + kXMax,     // [kXMax] MMAs over the token tile done
    B_DONE = B_XE + kXMax,
    B_COUNT
  };
};
constexpr int kThreads = kConv + 96;         // + entry loads, MMA issue, token loads

struct alignas(64) LinearParams {
  CUtensorMap tm_x;                          // scaled activations (K, T, G) float16, box 64 x tokens
  CUtensorMap tm_code, tm_scale;             // weights as (words of a row, N, G): boxes of 32 and 8 words x rows
  const int* exps;                           // (G, T): token t's row holds x 2^-exps
  __nv_bfloat16* out;
  int T, G, N, K;
  int tok_pad;                               // tokens per cluster, a multiple of 16
  int tiles;                                 // row tiles per group
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

// The MMAs of 64 channels (four of K = 16) with A in TMEM, or a commit, by the
// elected lane (e != 0) of a converged warp. One block of instructions: the issuing
// warp shares its scheduler with four decoding ones.
__device__ __forceinline__ void mma_four(uint32_t e, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
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

// Powers of two in registers the compiler cannot see through: a left shift
// written as a multiply by one of them runs on the multiplier's pipe, beside the
// logic operations, which keep the other integer pipe busy by themselves.
struct Shifts {
  uint32_t p1, p4, p5, p8, p9, p12;
  __device__ __forceinline__ Shifts() {
    asm volatile("mov.u32 %0, 2;" : "=r"(p1));
    asm volatile("mov.u32 %0, 16;" : "=r"(p4));
    asm volatile("mov.u32 %0, 32;" : "=r"(p5));
    asm volatile("mov.u32 %0, 256;" : "=r"(p8));
    asm volatile("mov.u32 %0, 512;" : "=r"(p9));
    asm volatile("mov.u32 %0, 4096;" : "=r"(p12));
  }
};

// The eight codes of a word times 2^-14 s: codes i and i + 4 in v[i]. Bits 4i ..
// 4i+2 (of each half) go to 9 .. 11, bit 4i+3 to 15.
__device__ __forceinline__ void decode8(uint32_t w, __half2 s, const Shifts& p, uint32_t* v) {
  const uint32_t mag[4] = {w * p.p9, w * p.p5, w * p.p1, w >> 3};
  const uint32_t sgn[4] = {w * p.p12, w * p.p8, w * p.p4, w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = (mag[i] & 0x0e000e00u) | (sgn[i] & 0x80008000u);
    v[i] = half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&u), s));
  }
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A ring position: the stage and the parity of its current pass.
struct Ring {
  int stages, stage = 0;
  uint32_t par = 0;
  __device__ __forceinline__ explicit Ring(int n) : stages(n) {}
  __device__ __forceinline__ void step() {
    if (++stage == stages) {
      stage = 0;
      par ^= 1;
    }
  }
};

template <int kHalves>
__global__ void __launch_bounds__(kThreads, 1) fp4_linear_kernel(const __grid_constant__ LinearParams P) {
  using F = Shape<kHalves>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[F::B_COUNT];
  __shared__ uint32_t tmem_ptr;
  __shared__ int failed;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb0 = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb0 - raw);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };
  const int x_bytes = P.tok_pad * kChunkK * 2;
  constexpr int off_x = F::kRaw * F::kRawBytes;

  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
  S = __shfl_sync(0xffffffffu, S, 0);          // warp-uniform, and so the loops below
  const uint32_t rank = __shfl_sync(0xffffffffu, cluster_ctarank(), 0);
  const int tile = blockIdx.x / S;           // (group, rows)
  const int g = tile / P.tiles, n0 = (tile - g * P.tiles) * F::kRows;
  const int t0 = blockIdx.y * kTokMax;
  const int entries = P.K / kCkv;
  const int e_begin = (int)((int64_t)entries * rank / S), ne = (int)((int64_t)entries * (rank + 1) / S) - e_begin;

  auto load_entry = [&](int i, int stage) {
    const uint32_t dst = sb0 + stage * F::kRawBytes, full = bar(F::B_RF + stage);
    const int word = (e_begin + i) * (kFp4EntryBytes / 4);
    mbar_arrive_expect_tx(full, F::kRawBytes);
    tma_load_3d(dst, &P.tm_code, full, word, n0, g);
    tma_load_3d(dst + F::kCode, &P.tm_code, full, word + 32, n0, g);
    tma_load_3d(dst + 2 * F::kCode, &P.tm_scale, full, word + 64, n0, g);
  };
  // Entries requested at once: what HBM delivers while the first kernel runs. The
  // others follow the tokens' first tiles, which come from L2 but queue behind
  // every entry requested before them (3 us with the whole ring ahead of them;
  // waiting for the tiles before asking for more left HBM idle, 12.5 -> 13.3 us).
  constexpr int kEarly = 2 / kHalves;
  if (threadIdx.x == kConv) {                // the entry warp's first lane
    for (int i = 0; i < F::B_COUNT; ++i)
      mbar_init(bar(i), i < F::B_RE ? 1 : i < F::B_AF ? kConv / 32 : i < F::B_AE ? 4 * kHalves : 1);
    failed = 0;
    fence_mbar_init();
    for (int i = 0; i < kEarly && i < ne; ++i) load_entry(i, i);   // weights do not wait for the first kernel
  }
  __syncwarp();
  if (warp == kConv / 32 + 1) {
    tmem_alloc(smem_u32(&tmem_ptr), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&tmem_ptr), 0);
  bool ok = true;

  if (warp < kConv / 32) {
    // ------------------------------------------------------------------ converting warps
    // Four warps decode 128 rows of a chunk; kGroups such groups per half take an
    // entry's chunks in turn. A thread decodes one row's chunk: 64 bytes of codes
    // and eight scales become 64 packed pairs, the 64 columns of an A stage in the
    // row's TMEM lane.
    const int half = (warp >> 2) / F::kGroups, grp = (warp >> 2) % F::kGroups;
    const int r = 128 * half + 32 * (warp & 3) + lane;
    const uint32_t a_tmem = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + F::kColA + 64u * (uint32_t)half;
    const Shifts pw;
    Ring rr(F::kRaw);
    Ring ra(F::kA);                          // of chunk 4e + c, c = grp, grp + kGroups, ...
    for (int i = 0; i < grp; ++i) ra.step();
    for (int e = 0; e < ne && ok; ++e) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(F::B_RF + rr.stage), rr.par));
      if (!ok) break;
      const uint8_t* src = smem + rr.stage * F::kRawBytes;
#pragma unroll 1
      for (int c = grp; c < kPer; c += F::kGroups) {
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = *reinterpret_cast<const uint4*>(src + (c >> 1) * F::kCode + r * 128 + 16 * ((4 * (c & 1) + i) ^ (r & 7)));
        const uint2 sc = *reinterpret_cast<const uint2*>(src + 2 * F::kCode + r * 32 + 8 * c);
        ok = __all_sync(0xffffffffu, mbar_wait(bar(F::B_AE + ra.stage), ra.par ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t col = a_tmem + (uint32_t)ra.stage * F::kColStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = (i < 2 ? sc.x : sc.y) >> (16 * (i & 1));
          const __half2 s2 = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)),
                                     __float2half2_rn(128.f));
          uint32_t v[16];
          decode8(q[i].x, __low2half2(s2), pw, v);
          decode8(q[i].y, __low2half2(s2), pw, v + 4);
          decode8(q[i].z, __high2half2(s2), pw, v + 8);
          decode8(q[i].w, __high2half2(s2), pw, v + 12);
          tmem_st16(col + 16u * i, v);
        }
        if (c + F::kGroups >= kPer) {        // the entry is read
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(F::B_RE + rr.stage));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(F::B_AF + ra.stage));
        for (int i = 0; i < F::kGroups; ++i) ra.step();
      }
      rr.step();
    }
  } else if (warp == kConv / 32) {
    // ------------------------------------------------------------------ entry loads
    pdl_wait();
    if (lane == 0) {
      Ring rr(F::kRaw);
      for (int i = 0; i < kEarly && i < ne; ++i) rr.step();
      for (int i = kEarly; i < ne && ok; ++i) {
        ok = i < F::kRaw || mbar_wait(bar(F::B_RE + rr.stage), rr.par ^ 1);
        if (!ok) break;
        load_entry(i, rr.stage);
        rr.step();
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  } else if (warp == kConv / 32 + 2) {
    // ------------------------------------------------------------------ token loads
    pdl_wait();                              // the first kernel's rows
    if (lane == 0) {
      Ring rx(F::x_stages(P.tok_pad));
      for (int c = 0; c < ne * kPer && ok; ++c) {
        ok = mbar_wait(bar(F::B_XE + rx.stage), rx.par ^ 1);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(F::B_XF + rx.stage), (uint32_t)x_bytes);
        const uint32_t xb = sb0 + off_x + rx.stage * x_bytes;
        const int k = e_begin * kCkv + c * kChunkK;
        tma_load_3d(xb, &P.tm_x, bar(F::B_XF + rx.stage), k, t0, g);
        tma_load_3d(xb + P.tok_pad * 128, &P.tm_x, bar(F::B_XF + rx.stage), k + 64, t0, g);
        rx.step();
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  } else {
    // ------------------------------------------------------------------ MMA issue
    const uint32_t el = elect_one();
    const uint32_t idesc = idesc_f16_f32(128, P.tok_pad);
    const uint64_t bd0 = smem_desc(sb0 + off_x, 16, 1024, kSwizzle128B);
    Ring rx(F::x_stages(P.tok_pad)), ra(F::kA);
    for (int c = 0; c < ne * kPer; ++c) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(F::B_XF + rx.stage), rx.par) && mbar_wait(bar(F::B_AF + ra.stage), ra.par));
      if (!ok) break;
      tc_fence_after();
      const uint64_t bd = desc_advance(bd0, rx.stage * x_bytes);
      const uint32_t at = tmem + F::kColA + (uint32_t)ra.stage * F::kColStage;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          mma_four(el, tmem + 64u * h, at + (uint32_t)(64 * h + b * 32), desc_advance(bd, b * P.tok_pad * 128), idesc,
                   c > 0 || b > 0);
      commit_one(el, bar(F::B_AE + ra.stage));
      commit_one(el, bar(F::B_XE + rx.stage));
      ra.step();
      rx.step();
    }
    if (ok && ne > 0) commit_one(el, bar(F::B_DONE));
  }
  if (!ok) *reinterpret_cast<volatile int*>(&failed) = 1;
  __syncthreads();
  pdl_wait();                                // exps, for every thread

  // ---------------------------------------------------------------- epilogue
  // this CTA's sums as [token][row] in shared memory (its tiles are used up);
  // rank r sums the cluster's partial results of tokens r, r + S, ... in rank order
  float* part = reinterpret_cast<float*>(smem);
  if (ne > 0 && !failed && !mbar_wait(bar(F::B_DONE), 0)) *reinterpret_cast<volatile int*>(&failed) = 1;
  tc_fence_after();
  const int half = (warp >> 2) / F::kGroups, within = warp % (4 * F::kGroups);   // a warp's half, its number there
  for (int c = 16 * (within >> 2); c < P.tok_pad && warp < kConv / 32; c += 16 * F::kGroups) {
    uint32_t v[16];
    if (ne > 0) {
      tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(64 * half + c), v);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) part[(c + i) * F::kRows + 128 * half + 32 * (warp & 3) + lane] = __uint_as_float(v[i]);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && failed && P.err) atomicOr(P.err, MLA_DEVICE_ERR_TIMEOUT);
  cluster_sync();
  const int nt = min(P.tok_pad, P.T - t0);
  for (int i = within * (int)S + (int)rank; i < nt && warp < kConv / 32; i += 4 * F::kGroups * (int)S) {
    const uint32_t mine = smem_u32(part + i * F::kRows + 128 * half + 4 * lane);
    float4 v[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
      if (k < S) v[k] = ld_cluster_f32x4(map_to_rank(mine, k));
    float4 sum = v[0];
#pragma unroll
    for (uint32_t k = 1; k < 8; ++k)
      if (k < S) sum = make_float4(sum.x + v[k].x, sum.y + v[k].y, sum.z + v[k].z, sum.w + v[k].w);
    const double f = ldexp((double)P.scale, P.exps[g * P.T + t0 + i] + 7);
    const float y[4] = {(float)(sum.x * f), (float)(sum.y * f), (float)(sum.z * f), (float)(sum.w * f)};
    const int n = n0 + 128 * half + 4 * lane;
    __nv_bfloat16* out = P.out + (int64_t)(t0 + i) * P.G * P.N + (int64_t)g * P.N + n;
    if (n + 3 < P.N && (reinterpret_cast<uintptr_t>(out) & 7u) == 0) {
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n + k < P.N) out[k] = __float2bfloat16_rn(y[k]);
    }
  }
  if (failed) {                              // a wait gave up: no copy or MMA may outlive the block
    const uint64_t begin = global_ns();
    while (global_ns() - begin < 50000ull) {
    }
  }
  cluster_sync();                            // the peers have read this CTA's sums
  if (warp == kConv / 32 + 1) tmem_dealloc(tmem, kTmemCols);
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

// CTAs per cluster (ranges of K). Clusters of S stay within a GPC, so how many
// of them run at once is the device's answer, asked once per device and shared
// memory size: 74, 33, 22, 15 clusters of 2, 4, 6, 8 on a B200. The count taken
// minimises waves x (entries per CTA + kFixed), kFixed being what a CTA spends
// besides its entries (launch, first load, exchange), in entries.
template <int kHalves>
cudaError_t pick_splits(int64_t clusters, int entries, int tok_pad, int* out) {
  constexpr int kMaxS = 8, kMaxDev = 64, kFixed = 4;
  static std::mutex mu;
  static int active[kMaxDev][kTokMax / 16][kMaxS];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  int* act = active[dev][tok_pad / 16 - 1];
  if (!act[0]) {
    // the largest size any call needs: the attribute is set once for all of them
    e = cudaFuncSetAttribute(fp4_linear_kernel<kHalves>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Shape<kHalves>::smem(kTokMax));
    if (e != cudaSuccess) return e;
    for (int S = kMaxS; S >= 1; --S) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)S;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3((unsigned)(S * 64));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = Shape<kHalves>::smem(tok_pad);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, fp4_linear_kernel<kHalves>, &cfg);
      if (e != cudaSuccess) return e;
      act[S - 1] = n;                        // [0] last: a filled table
    }
    if (act[0] < 1) return cudaErrorInvalidConfiguration;
  }
  int64_t best = 0;
  for (int S = 1; S <= kMaxS && S <= entries; ++S) {
    if (act[S - 1] < 1) continue;
    const int64_t cost = (clusters + act[S - 1] - 1) / act[S - 1] * ((entries + S - 1) / S + kFixed);
    if (S == 1 || cost < best) {
      best = cost;
      *out = S;
    }
  }
  return cudaSuccess;
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, const cuuint64_t* d, const cuuint64_t* s,
            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t el[3] = {1, 1, 1};
  return encode_fn()(m, type, 3, const_cast<void*>(base), d, s, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The products, with P's activations filled in.
template <int kHalves>
cudaError_t launch_products(const mla_fp4_linear_args* a, LinearParams& P, cudaStream_t st) {
  using F = Shape<kHalves>;
  const cuuint64_t pitch = (cuuint64_t)(a->K / kCkv) * kFp4EntryBytes;
  const cuuint64_t d[3] = {pitch / 4, (cuuint64_t)a->N, (cuuint64_t)a->G}, s[2] = {pitch, pitch * a->N};
  const cuuint32_t code[3] = {32, F::kRows, 1}, scale[3] = {8, F::kRows, 1};
  if (!encode(&P.tm_code, CU_TENSOR_MAP_DATA_TYPE_UINT32, a->w, d, s, code, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&P.tm_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, a->w, d, s, scale, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  P.tiles = (a->N + F::kRows - 1) / F::kRows;
  const int64_t blocks = (P.T + kTokMax - 1) / kTokMax;
  int S = 0;
  cudaError_t e = pick_splits<kHalves>((int64_t)a->G * P.tiles * blocks, a->K / kCkv, P.tok_pad, &S);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((int64_t)a->G * P.tiles * S), (unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = F::smem(P.tok_pad);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, fp4_linear_kernel<kHalves>, P);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t xs_bytes(const mla_fp4_linear_args* a) {
  return ((size_t)a->B * a->Q * a->G * a->K * 2 + 255) & ~(size_t)255;
}

}  // namespace

size_t fp4_linear_workspace_bytes(const mla_fp4_linear_args* a) {
  if (fp4_few_tokens(a)) return 0;
  return xs_bytes(a) + (size_t)a->B * a->Q * a->G * sizeof(int);
}

cudaError_t launch_fp4_linear(const mla_fp4_linear_args* a, void* ws, int sms, cudaStream_t st) {
  if (fp4_few_tokens(a)) return launch_fp4_few(a, sms, st);
  if (!encode_fn()) return cudaErrorNotSupported;
  LinearParams P;
  memset(static_cast<void*>(&P), 0, sizeof(P));
  const int T = a->B * a->Q;
  __half* xs = reinterpret_cast<__half*>(ws);
  int* exps = reinterpret_cast<int*>(reinterpret_cast<char*>(ws) + xs_bytes(a));
  P.exps = exps;
  P.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  P.T = T;
  P.G = a->G;
  P.N = a->N;
  P.K = a->K;
  P.scale = a->scale;
  P.err = a->err_flag;
  P.tok_pad = T >= kTokMax ? kTokMax : (T + 15) / 16 * 16;
  {
    const cuuint64_t d[3] = {(cuuint64_t)a->K, (cuuint64_t)T, (cuuint64_t)a->G};
    const cuuint64_t s[2] = {(cuuint64_t)a->K * 2, (cuuint64_t)a->K * 2 * T};
    const cuuint32_t bx[3] = {64, (cuuint32_t)P.tok_pad, 1};
    if (!encode(&P.tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xs, d, s, bx, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)T, (unsigned)a->G);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, x_to_f16, *a, xs, exps);
  if (e != cudaSuccess) return e;
  // A CTA brings in 288 bytes of weights a row and entry, and 1024 a token: 256
  // rows where the tokens' share of 128 would be the larger (64 tokens, 16384 to
  // 7168: 27 against 29 us), else 128, on twice the CTAs (one token, 8192 to 4096:
  // 12.5 against 10.7 us).
  return P.tok_pad > 32 ? launch_products<2>(a, P, st) : launch_products<1>(a, P, st);
}

}  // namespace mla
