// Cache append with the position rotation on the way (mla_rope_append). One warp
// per unit of a new token's work: unit 0 copies its latent row and rotates its
// rope row into the cache, the others rotate kIter vectors per lane of its
// heads' query position parts.
//
// A pair (2j, 2j+1) turns by a = (pos_offset + t) * theta^(-2j/Dr). The host
// passes theta^(-2j/Dr) / 2 pi in double; pos * that is the angle in turns,
// whose whole part is dropped in double (an error below 2^-24 turns up to
// position 2^28), so the remaining sine and cosine are float at full precision
// at any position. Lane j evaluates pair j; every lane takes those of its own
// vector, the same for all heads, by shuffles.
//
// The work is copies: 2 (512 + Dr + H Dr) elements of traffic per token and
// three float operations per rotated element, so what counts is bytes in flight.
// A unit issues all its 16-byte loads (4 KB a warp) before the chain of
// dependent lookups (token -> sequence -> length -> page) and the sine, and needs
// no block barrier. 12,241 tokens, 128 heads: 68 to 69 us, 6.2 TB/s; with one CTA per token
// and the loads behind the chain 85 us, with them before it in 70 registers 169 us.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "rope_append.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 32;

struct RopeParams {
  mla_rope_append_args a;
  double turns[kMaxPairs];   // theta^(-2j/Dr) / 2 pi
  int units;                 // per token: 1 + those of its heads
};

// One access of a lane: kW elements in 32-bit words, 16 bytes where every row is
// 16-byte aligned, else one pair by element accesses.
template <typename T, bool WIDE> struct Access {
  static constexpr int kW = WIDE ? 16 / (int)sizeof(T) : 2;
  static constexpr int kWords = kW * (int)sizeof(T) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (WIDE) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    } else if constexpr (sizeof(T) == 4) {
      w[0] = reinterpret_cast<const uint32_t*>(p)[0];
      w[1] = reinterpret_cast<const uint32_t*>(p)[1];
    } else {
      w[0] = (uint32_t)reinterpret_cast<const uint16_t*>(p)[0] | (uint32_t)reinterpret_cast<const uint16_t*>(p)[1] << 16;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (WIDE) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (sizeof(T) == 4) {
      reinterpret_cast<uint32_t*>(p)[0] = w[0];
      reinterpret_cast<uint32_t*>(p)[1] = w[1];
    } else {
      reinterpret_cast<uint16_t*>(p)[0] = (uint16_t)w[0];
      reinterpret_cast<uint16_t*>(p)[1] = (uint16_t)(w[0] >> 16);
    }
  }
  // pair k by (cs[k], sn[k]); the contraction is spelled out, so that every path
  // gives the same bits
  __device__ __forceinline__ void turn(const float (&cs)[kW / 2], const float (&sn)[kW / 2]) {
#pragma unroll
    for (int k = 0; k < kW / 2; ++k) {
      float e, o;
      if constexpr (sizeof(T) == 4) {
        e = __uint_as_float(w[2 * k]);
        o = __uint_as_float(w[2 * k + 1]);
      } else {
        e = __uint_as_float(w[k] << 16);
        o = __uint_as_float(w[k] & 0xffff0000u);
      }
      const float x = fmaf(e, cs[k], -__fmul_rn(o, sn[k])), y = fmaf(e, sn[k], __fmul_rn(o, cs[k]));
      if constexpr (sizeof(T) == 4) {
        w[2 * k] = __float_as_uint(x);
        w[2 * k + 1] = __float_as_uint(y);
      } else {
        w[k] = sm100::pack_bf16(x, y);
      }
    }
  }
};

// How many of the non-decreasing ends[1 .. B] are at or before n, by the whole
// warp: a 32-way search.
__device__ __forceinline__ int ends_before(const int32_t* ends, int B, int64_t n, int lane) {
  int lo = 0, len = B;
  while (len > 0) {
    const int step = (len + 31) / 32, k = lo + (lane + 1) * step;
    const uint32_t m = __ballot_sync(0xffffffffu, k <= lo + len && (int64_t)ends[k] <= n);
    const int skip = __popc(m) * step;
    lo += skip;
    len = min(step - 1, len - skip);
  }
  return lo;
}

constexpr int kIter = 8;       // vectors per lane and unit

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_kernel(const __grid_constant__ RopeParams P) {
  const mla_rope_append_args& a = P.a;
  using Vec = Access<T, WIDE>;
  constexpr int kW = Vec::kW;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int64_t n = unit / P.units;
  const int part = (int)(unit - n * P.units);
  if (n >= a.N) return;                            // whole warp

  const int per = a.Dr / kW;                       // vectors of a position part; divides 32
  const int my_c = (lane % per) * kW;              // this lane's elements of every part
  const int h0 = (part - 1) * kIter * (32 / per) + lane / per;   // its heads: h0, h0 + 32 / per, ...
  const T* k_src = reinterpret_cast<const T*>(a.k_pe) + n * a.k_pe_stride;
  const T* c_src = reinterpret_cast<const T*>(a.c_kv) + n * a.c_kv_stride;
  const T* q_src = reinterpret_cast<const T*>(a.q_pe) + n * a.q_token_stride + my_c;
  Vec v[kIter], kv;
  if (part == 0) {
#pragma unroll
    for (int u = 0; u < kIter; ++u)
      if ((lane + 32 * u) * kW < a.Ckv) v[u].load(c_src + (lane + 32 * u) * kW);
    if (lane < per) kv.load(k_src + my_c);
  } else {
#pragma unroll
    for (int u = 0; u < kIter; ++u)
      if (h0 + u * (32 / per) < a.H) v[u].load(q_src + (h0 + u * (32 / per)) * a.q_head_stride);
  }

  int b, i, cnt;
  if (a.cu_tokens) {
    b = ends_before(a.cu_tokens, a.B, n, lane);
    if (b >= a.B) return;                          // behind the last sequence
    const int c0 = a.cu_tokens[b], c1 = a.cu_tokens[b + 1];
    if (n < c0 || n >= c1) return;                 // before the first
    i = (int)(n - c0);
    cnt = c1 - c0;
  } else {
    b = (int)(n / a.Q);
    i = (int)(n - (int64_t)b * a.Q);
    cnt = a.Q;
  }
  const int64_t t = (int64_t)a.seq_lens[b] - cnt + i;
  float s = 0.f, c = 1.f;
  if (2 * lane < a.Dr) {
    const double turns = (double)(a.pos_offset + t) * P.turns[lane];
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
  }
  float sn[kW / 2], cs[kW / 2];
#pragma unroll
  for (int k = 0; k < kW / 2; ++k) {
    sn[k] = __shfl_sync(0xffffffffu, s, my_c / 2 + k);
    cs[k] = __shfl_sync(0xffffffffu, c, my_c / 2 + k);
  }
  if (part > 0) {
    T* q_dst = reinterpret_cast<T*>(a.q_out) + my_c +
               (a.cu_tokens ? n * a.o_token_stride : (int64_t)b * a.o_batch_stride + (int64_t)i * a.o_token_stride);
#pragma unroll
    for (int u = 0; u < kIter; ++u) {
      const int h = h0 + u * (32 / per);
      if (h < a.H) {
        v[u].turn(cs, sn);
        v[u].store(q_dst + h * a.o_head_stride);
      }
    }
    return;
  }
  int64_t row = -1, batch = 0;
  if (t >= 0 && t < a.Lk) {
    if (a.block_table) {
      const int page = a.block_table[(int64_t)b * a.max_pages + t / a.page_size];
      if (page >= 0 && page < a.num_pages) row = (int64_t)page * a.page_size + t % a.page_size;
    } else {
      row = t;
      batch = b;
    }
  }
  if (row < 0) {
    if (lane == 0 && a.err_flag) atomicOr(a.err_flag, MLA_DEVICE_ERR_BLOCK_TABLE);
    return;
  }
  T* c_dst = reinterpret_cast<T*>(a.kv_cache) + batch * a.kv_batch_stride + row * a.kv_row_stride;
  T* k_dst = reinterpret_cast<T*>(a.pe_cache) + batch * a.pe_batch_stride + row * a.pe_row_stride;
#pragma unroll
  for (int u = 0; u < kIter; ++u)
    if ((lane + 32 * u) * kW < a.Ckv) v[u].store(c_dst + (lane + 32 * u) * kW);
  if (lane < per) {
    kv.turn(cs, sn);
    kv.store(k_dst + my_c);
  }
}

bool wide_rows(const mla_rope_append_args* a, int64_t esz) {
  auto ok = [&](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  auto st = [&](int64_t s) { return (s * esz) % 16 == 0; };
  bool w = ok(a->c_kv) && ok(a->k_pe) && ok(a->kv_cache) && ok(a->pe_cache) && st(a->c_kv_stride) &&
           st(a->k_pe_stride) && st(a->kv_row_stride) && st(a->pe_row_stride);
  if (!a->block_table) w = w && st(a->kv_batch_stride) && st(a->pe_batch_stride);
  if (a->H > 0) {
    w = w && ok(a->q_pe) && ok(a->q_out) && st(a->q_token_stride) && st(a->q_head_stride) &&
        st(a->o_token_stride) && st(a->o_head_stride);
    if (!a->cu_tokens) w = w && st(a->o_batch_stride);
  }
  return w;
}

template <typename T>
cudaError_t launch(RopeParams& P, bool wide, cudaStream_t st) {
  const int per = P.a.Dr / (wide ? 16 / (int)sizeof(T) : 2);
  const int heads = kIter * (32 / per);          // of a unit
  P.units = 1 + (P.a.H + heads - 1) / heads;
  const int64_t blocks = ((int64_t)P.a.N * P.units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, rope_append_kernel<T, true>, P)
              : cudaLaunchKernelEx(&cfg, rope_append_kernel<T, false>, P);
}

}  // namespace

cudaError_t launch_rope_append(const mla_rope_append_args* a, cudaStream_t st) {
  if (a->N == 0) return cudaSuccess;
  RopeParams P;
  P.a = *a;
  for (int j = 0; j < kMaxPairs; ++j)
    P.turns[j] = j < a->Dr / 2 ? pow((double)a->rope_theta, -2.0 * j / a->Dr) * 0.15915494309189533577 : 0.0;
  const bool bf16 = a->dtype == MLA_BF16;
  const bool wide = wide_rows(a, bf16 ? 2 : 4);
  const cudaError_t e = bf16 ? launch<__nv_bfloat16>(P, wide, st) : launch<float>(P, wide, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
