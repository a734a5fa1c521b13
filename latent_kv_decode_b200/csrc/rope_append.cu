// Cache append with the position rotation on the way (mla_rope_append): one
// CTA per new token copies its latent row, rotates its rope row and its heads'
// query position parts by the angle of its position, and stores them where the
// decode reads them.
//
// A pair (2j, 2j+1) turns by a = (pos_offset + t) * theta^(-2j/Dr). The host
// passes theta^(-2j/Dr) / 2 pi in double; pos * that is the angle in turns,
// whose whole part is dropped in double (an error below 2^-24 turns up to position
// 2^28), so the remaining sine and cosine are float at full precision at any
// position. The first Dr/2 threads evaluate each pair once for the whole token.
//
// The work is copies: 2 (512 + Dr + H Dr) elements of traffic per token and
// three float operations per rotated element. A token's vectors are 16 bytes
// wide, loaded before the chain of dependent lookups (token -> sequence ->
// length -> page) and the sine, which they hide.
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
};

template <typename T> struct Vec16 { T v[16 / sizeof(T)]; };

template <typename T>
__device__ __forceinline__ void rotate(float c, float s, T& x, T& y) {
  const float e = to_f32<T>(x), o = to_f32<T>(y);
  x = from_f32<T>(e * c - o * s);
  y = from_f32<T>(e * s + o * c);
}

// kVec elements per access: 16 bytes where every row is 16-byte aligned, else
// one pair (two element accesses).
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams P) {
  const mla_rope_append_args& a = P.a;
  constexpr int kW = WIDE ? 16 / (int)sizeof(T) : 2;
  struct alignas(WIDE ? 16 : sizeof(T)) Vec { T v[kW]; };
  __shared__ float cs[kMaxPairs], sn[kMaxPairs];
  __shared__ int64_t slot_s[2];   // element offset of the token's kv and pe rows, -1 = not stored
  const int tid = threadIdx.x;
  const int64_t n = blockIdx.x;
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();

  // which sequence owns row n: the number of ends at or before it
  int b, i, cnt;
  if (a.cu_tokens) {
    int ends = 0;
    for (int k0 = 0; k0 < a.B; k0 += kRopeThreads) {
      const int k = k0 + tid;
      ends += __syncthreads_count(k < a.B && (int64_t)a.cu_tokens[k + 1] <= n);
    }
    b = ends;
    if (b >= a.B) return;                                    // behind the last sequence
    const int c0 = a.cu_tokens[b], c1 = a.cu_tokens[b + 1];
    if (n < c0 || n >= c1) return;                           // before the first
    i = (int)(n - c0);
    cnt = c1 - c0;
  } else {
    b = (int)(n / a.Q);
    i = (int)(n - (int64_t)b * a.Q);
    cnt = a.Q;
  }
  const int64_t t = (int64_t)a.seq_lens[b] - cnt + i;
  const int pairs = a.Dr / 2;
  if (tid < pairs) {
    const double turns = (double)(a.pos_offset + t) * P.turns[tid];
    const float frac = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * frac, &s, &c);
    cs[tid] = c;
    sn[tid] = s;
  } else if (tid == kRopeThreads - 1) {
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
    if (row < 0 && a.err_flag) atomicOr(a.err_flag, MLA_DEVICE_ERR_BLOCK_TABLE);
    slot_s[0] = row < 0 ? -1 : batch * a.kv_batch_stride + row * a.kv_row_stride;
    slot_s[1] = row < 0 ? -1 : batch * a.pe_batch_stride + row * a.pe_row_stride;
  }
  __syncthreads();

  if (slot_s[0] >= 0) {
    const T* src = reinterpret_cast<const T*>(a.c_kv) + n * a.c_kv_stride;
    T* dst = reinterpret_cast<T*>(a.kv_cache) + slot_s[0];
    for (int c = tid * kW; c < a.Ckv; c += kRopeThreads * kW)
      *reinterpret_cast<Vec*>(dst + c) = *reinterpret_cast<const Vec*>(src + c);
    src = reinterpret_cast<const T*>(a.k_pe) + n * a.k_pe_stride;
    dst = reinterpret_cast<T*>(a.pe_cache) + slot_s[1];
    for (int c = tid * kW; c < a.Dr; c += kRopeThreads * kW) {
      Vec v = *reinterpret_cast<const Vec*>(src + c);
#pragma unroll
      for (int k = 0; k < kW; k += 2) rotate<T>(cs[(c + k) >> 1], sn[(c + k) >> 1], v.v[k], v.v[k + 1]);
      *reinterpret_cast<Vec*>(dst + c) = v;
    }
  }
  if (a.H > 0) {
    const T* src = reinterpret_cast<const T*>(a.q_pe) + n * a.q_token_stride;
    T* dst = reinterpret_cast<T*>(a.q_out) +
             (a.cu_tokens ? n * a.o_token_stride : (int64_t)b * a.o_batch_stride + (int64_t)i * a.o_token_stride);
    const int per = a.Dr / kW;
    for (int k0 = tid; k0 < a.H * per; k0 += kRopeThreads) {
      const int h = k0 / per, c = (k0 - h * per) * kW;
      Vec v = *reinterpret_cast<const Vec*>(src + h * a.q_head_stride + c);
#pragma unroll
      for (int k = 0; k < kW; k += 2) rotate<T>(cs[(c + k) >> 1], sn[(c + k) >> 1], v.v[k], v.v[k + 1]);
      *reinterpret_cast<Vec*>(dst + h * a.o_head_stride + c) = v;
    }
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
cudaError_t launch(const RopeParams& P, bool wide, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)P.a.N);
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
