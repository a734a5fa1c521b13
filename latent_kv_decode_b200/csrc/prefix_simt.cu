// Shared-prefix decode on the CUDA cores, in float32: the path of float32
// inputs (which need full precision) and of page sizes that the tensor-core
// kernel does not take.
//
// A CTA owns 32 stacked rows and a range of their 16-token tiles, two of which
// are in flight: the next tile's rows arrive (cp.async) while this one computes.
//   S = Q . K^T    sixteen groups of 16 threads take a sixteenth of the 576-wide
//                  dot each, 8 x 4 scores per thread; the parts are summed by the
//                  softmax.
//   softmax        warp w keeps the online statistics of rows 4w .. 4w+3, two at
//                  a time, a lane per token.
//   O += P . V     thread = 8 rows x 8 columns of the 32 x 512 accumulator.
// Both products are packed float32 FMAs. What bounds them is what shared memory
// returns to registers, 32 floats a clock and SM: S reads 24 floats for 64 FMA,
// O 16 (tiles of 4 x 2 and 8 x 4 took 2.5 + 2.1 us a tile instead of 2.4 + 1.5).
//
// Tokens that no row may see are zeros in the tile, so whatever their cache
// rows hold stays out of the sums; where a tile that some rows do not see holds
// an infinity or NaN (its scores show it), the rows whose weight is 0 skip it.
#include <algorithm>

#include "once_per_device.h"
#include "prefix.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kRows = 32, kToks = 16;
constexpr int kThr = 256, kWarps = kThr / 32, kParts = kThr / 16;   // kParts slices of the dot product
constexpr int kPad = 4;             // floats of row padding: 16-byte rows, 8 rows over all banks
constexpr int kPart = kToks + 1;

__host__ __device__ constexpr int pitch_of(int D) { return D + kPad; }

using f32x2 = unsigned long long;                // two floats, the first in the low half
struct alignas(16) f32x4 { f32x2 lo, hi; };

__device__ __forceinline__ void fma2(f32x2& acc, f32x2 a, f32x2 b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void copy16(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// Rows of D = Ckv + Dr elements into shared memory as float32; row r comes from
// lat(r) and pe(r), zeros where lat(r) is null. Asynchronous for float32.
template <typename T, int kN, typename Lat, typename Pe>
__device__ __forceinline__ void load_rows(float* dst, int D, Lat lat, Pe pe) {
  const int d4 = D / 4, pitch = pitch_of(D), lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < kN; r += kWarps) {
    const T* l = lat(r);
    const T* e = l ? pe(r) - kCkv : nullptr;
    float* d = dst + r * pitch;
    if constexpr (sizeof(T) == 4) {
      const T* any = lat(-1);
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const int k = 4 * (lane + 32 * u);
        if (k < D) copy16(d + k, !l ? any : k < kCkv ? l + k : e + k, l != nullptr);
      }
    } else {
      float4 v[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const int k = 4 * (lane + 32 * u);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (l && k < D) v[u] = load4(k < kCkv ? l + k : e + k);
      }
#pragma unroll
      for (int u = 0; u < 5; ++u)
        if (lane + 32 * u < d4) *reinterpret_cast<float4*>(d + 4 * (lane + 32 * u)) = v[u];
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThr) prefix_simt(const PrefixParams p) {
  extern __shared__ float smem[];
  __shared__ const T* row_lat[2][kToks];         // the tile's cache rows, null where no row may see the token
  __shared__ const T* row_pe[2][kToks];
  const int D = p.D, pitch = pitch_of(D);
  float* qs = smem;                              // [kRows][pitch]
  float* ks = qs + kRows * pitch;                // [2][kToks][pitch]
  float* part = ks + 2 * kToks * pitch;          // [kParts][kRows][kPart] parts of the scores
  float* ps = part + kParts * kRows * kPart;     // [kToks][kRows] weights
  float* alpha = ps + kToks * kRows;             // [kRows]
  float* stat = alpha + kRows;                   // [kRows] 1 / denominator

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int r0 = blockIdx.x * kRows, z = blockIdx.y;
  const int nr = min(kRows, p.N - r0);
  const int b0 = r0 / p.HQ, b1 = (r0 + nr - 1) / p.HQ;
  __shared__ int lens[kRows / 8 + 1];            // H*Q >= 8: the sequences a block can hold rows of
  if (tid <= b1 - b0) lens[tid] = prefix_len_of(p, b0 + tid);
  __syncthreads();
  const int tiles = TileWalk<kToks>::count(p, lens, b0, b1);
  const int per = (tiles + p.num_splits - 1) / p.num_splits;
  const int j0 = min(tiles, z * per), j1 = min(tiles, j0 + per);

  const T* q_lat = reinterpret_cast<const T*>(p.q_lat) + (int64_t)r0 * p.Ckv;
  const T* q_pe = reinterpret_cast<const T*>(p.q_pe) + (int64_t)r0 * p.Dr;
  load_rows<T, kRows>(qs, D, [&](int r) { return r < nr ? q_lat + (int64_t)max(r, 0) * p.Ckv : nullptr; },
                      [&](int r) { return q_pe + (int64_t)r * p.Dr; });

  // the rows of tile `w` into buffer s (after a barrier that follows its last use)
  auto locate = [&](const TileWalk<kToks>& w, int s) {
    if (tid >= kToks) return;
    const bool pre = w.b < 0;
    const int t = w.t + tid;
    const int32_t* table = pre ? p.ptable : p.table ? p.table + (int64_t)w.b * p.max_pages : nullptr;
    bool ok = t < w.end && (!p.mask || p.mask[(pre ? 0 : p.Lp) + t] != 0);
    int64_t row = t;
    if (ok && table) {
      const int page = table[t / p.page_size];
      ok = page >= 0 && page < (pre ? p.p_pages : p.num_pages);
      row = (int64_t)page * p.page_size + t % p.page_size;
      if (!ok) prefix_flag(p, MLA_DEVICE_ERR_BLOCK_TABLE);
    }
    const T* kv = reinterpret_cast<const T*>(pre ? p.pkv : p.kv);
    const T* pe = reinterpret_cast<const T*>(pre ? p.ppe : p.pe);
    if (!pre && !table) {
      kv += w.b * p.kv_batch;
      pe += w.b * p.pe_batch;
    }
    row_lat[s][tid] = ok ? kv + row * (pre ? p.pkv_row : p.kv_row) : nullptr;
    row_pe[s][tid] = pe + row * (pre ? p.ppe_row : p.pe_row);
  };
  auto fetch = [&](int s) {
    load_rows<T, kToks>(ks + s * kToks * pitch, D, [&](int r) { return r < 0 ? q_lat : row_lat[s][r]; },
                        [&](int r) { return row_pe[s][r]; });
  };
  TileWalk<kToks> w, wn;                         // this tile and the next
  w.seek(p, lens, b0, b1, j0);
  wn = w;
  if (j0 < j1) {
    locate(w, 0);
    __syncthreads();
    fetch(0);
    wn.next(lens, b0);
  }
  copy_commit();

  // S: thread (ty, tx) of part kq holds rows ty + 4i, tokens tx + 4n
  const int kq = tid >> 4, ty = (tid >> 2) & 3, tx = tid & 3;
  const int kn = D / kParts;                     // channels per part, even (D is a multiple of 32)
  // softmax: rows 4 warp + 2i + lane / 16, token lane % 16
  const int sub = lane >> 4, tok = lane & 15;
  float m_run[2], l_run[2];
  int row_b[2], row_lim[2];                      // sequence and last visible own token of the row
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
    const int r = r0 + 4 * warp + 2 * i + sub;
    row_b[i] = r < p.N ? r / p.HQ : -2;
    row_lim[i] = 0x7fffffff;
    if (r < p.N && p.causal) row_lim[i] = lens[row_b[i] - b0] - p.Q + r % p.Q;
  }
  // O: rows 8 rg + i, columns 4 cg + k and 256 + 4 cg + k
  const int rg = tid >> 6, cg = tid & 63;
  f32x2 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0ull;

  for (int j = j0; j < j1; ++j) {
    const int buf = (j - j0) & 1;
    const bool more = j + 1 < j1;
    if (more) locate(wn, buf ^ 1);
    copy_wait<0>();
    __syncthreads();                             // this tile is in, the next one's rows are known, the other buffer is free
    if (more) fetch(buf ^ 1);
    copy_commit();
    const float* kt = ks + buf * kToks * pitch;
    const bool pre = w.b < 0;
    bool odd = false;                            // a non-finite score: a non-finite key
    {
      f32x2 s[8][4] = {};                          // sums over even and odd channels
      const float* qp = qs + ty * pitch + kq * kn;
      const float* kp = kt + tx * pitch + kq * kn;
#pragma unroll 2
      for (int k = 0; k < kn; k += 2) {
        f32x2 qv[8], kv[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) qv[i] = *reinterpret_cast<const f32x2*>(qp + 4 * i * pitch + k);
#pragma unroll
        for (int n = 0; n < 4; ++n) kv[n] = *reinterpret_cast<const f32x2*>(kp + 4 * n * pitch + k);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) fma2(s[i][n], qv[i], kv[n]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float2 v = unpack2(s[i][n]);
          part[(kq * kRows + ty + 4 * i) * kPart + tx + 4 * n] = v.x + v.y;
          odd = odd || !isfinite(v.x + v.y);
        }
    }
    const bool any_odd = __syncthreads_or(odd);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int srow = 4 * warp + 2 * i + sub;
      const int t = w.t + tok;
      // own tokens are seen by their sequence's rows; a causal row sees own
      // tokens up to row_lim (a negative one reaches back into the prefix)
      bool vis = row_lat[buf][tok] != nullptr && row_b[i] >= 0 && (pre || row_b[i] == w.b);
      vis = vis && (!p.causal || (pre ? t - p.Lp : t) <= row_lim[i]);
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kParts; ++k) s += part[(k * kRows + srow) * kPart + tok];
      s = vis ? s * p.scale : -INFINITY;
      float mx = s;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m_run[i], mx);
      const float al = m_run[i] == -INFINITY ? 0.f : expf(m_run[i] - m_new);
      const float e = vis ? expf(s - m_new) : 0.f;
      float sum = e;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l_run[i] = l_run[i] * al + sum;
      m_run[i] = m_new;
      ps[tok * kRows + srow] = e;
      if (tok == 0) alpha[srow] = al;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float al = alpha[8 * rg + i];
      const f32x2 al2 = pack2(al, al);
#pragma unroll
      for (int k = 0; k < 4; ++k) asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(acc[i][k]) : "l"(al2));
    }
    const int nt = min(kToks, w.end - w.t);      // tokens past it have no weight
    if (!any_odd) {
#pragma unroll 1
      for (int t4 = 0; t4 < nt; t4 += 4) {
#pragma unroll
        for (int tt = t4; tt < t4 + 4; ++tt) {
          const f32x4 v0 = *reinterpret_cast<const f32x4*>(kt + tt * pitch + 4 * cg);
          const f32x4 v1 = *reinterpret_cast<const f32x4*>(kt + tt * pitch + 256 + 4 * cg);
          const float4 pa = *reinterpret_cast<const float4*>(ps + tt * kRows + 8 * rg);
          const float4 pb = *reinterpret_cast<const float4*>(ps + tt * kRows + 8 * rg + 4);
          const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const f32x2 p2 = pack2(pr[i], pr[i]);
            fma2(acc[i][0], p2, v0.lo);
            fma2(acc[i][1], p2, v0.hi);
            fma2(acc[i][2], p2, v1.lo);
            fma2(acc[i][3], p2, v1.hi);
          }
        }
      }
    } else {
#pragma unroll 1
      for (int tt = 0; tt < nt; ++tt) {
        const f32x4 v0 = *reinterpret_cast<const f32x4*>(kt + tt * pitch + 4 * cg);
        const f32x4 v1 = *reinterpret_cast<const f32x4*>(kt + tt * pitch + 256 + 4 * cg);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float pr = ps[tt * kRows + 8 * rg + i];
          if (pr != 0.f) {
            const f32x2 p2 = pack2(pr, pr);
            fma2(acc[i][0], p2, v0.lo);
            fma2(acc[i][1], p2, v0.hi);
            fma2(acc[i][2], p2, v1.lo);
            fma2(acc[i][3], p2, v1.hi);
          }
        }
      }
    }
    w = wn;
    if (more) wn.next(lens, b0);
  }

  // the rows' denominators to the accumulator's threads
  const bool split = p.num_splits > 1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float m = m_run[i], l = l_run[i];
    const int r = r0 + 4 * warp + 2 * i + sub;
    float inv = 0.f;
    if (r < p.N) {
      float wt = 1.f;
      if (!split && p.sinks) {
        const float sk = p.sinks[(r % p.HQ) / p.Q], m2 = fmaxf(m, sk);
        wt = m == -INFINITY ? 0.f : expf(m - m2);
        l = l * wt + expf(sk - m2);
        m = m2;
      }
      const bool seen = !(m == -INFINITY && l == 0.f);   // a NaN denominator stays one
      inv = seen ? wt / l : 0.f;
      const float lse = seen ? m + logf(l) : -INFINITY;
      if (tok == 0) {
        if (split)
          p.ws_lse[(int64_t)z * p.N + r] = lse;
        else if (p.lse)
          p.lse[r] = lse;
      }
    }
    if (tok == 0) stat[r - r0] = inv;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 8 * rg + i;
    if (r >= p.N) continue;
    const float inv = stat[8 * rg + i];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = 256 * k + 4 * cg;
      const float2 lo = unpack2(acc[i][2 * k]), hi = unpack2(acc[i][2 * k + 1]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (inv != 0.f) v = make_float4(lo.x * inv, lo.y * inv, hi.x * inv, hi.y * inv);
      if (split)
        *reinterpret_cast<float4*>(p.ws_o + ((int64_t)z * p.N + r) * p.Ckv + c) = v;
      else if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(reinterpret_cast<T*>(p.x) + (int64_t)r * p.Ckv + c) = v;
      else
        *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.x) + (int64_t)r * p.Ckv + c) =
            make_uint2(sm100::pack_bf16(v.x, v.y), sm100::pack_bf16(v.z, v.w));
    }
  }
}

template <typename T>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  const size_t smem = prefix_simt_smem(p.D);
  static OncePerDevice smem_set;
  cudaError_t e = smem_set([] {
    return cudaFuncSetAttribute(prefix_simt<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prefix_simt_smem(kCkv + 64));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.N + kRows - 1) / kRows), (unsigned)p.num_splits);
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefix_simt<T>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t prefix_simt_smem(int D) {
  return sizeof(float) * ((size_t)(kRows + 2 * kToks) * pitch_of(D) + kParts * kRows * kPart + kToks * kRows + 2 * kRows);
}

// About one CTA per SM (its shared memory fills one), no split shorter than a
// tile: a tile takes 5.4 us, the merge of a few splits 3.
int prefix_simt_auto_splits(const mla_prefix_args* a, int sms) {
  const int HQ = a->H * a->Q;
  const int64_t rows = (int64_t)a->B * HQ;
  const int64_t blocks = (rows + kRows - 1) / kRows;
  const int64_t seqs = std::min<int64_t>(a->B, (kRows + HQ - 1) / HQ);   // of a block
  const int64_t tiles = ((int64_t)a->prefix_len + kToks - 1) / kToks + seqs * ((a->Lk + kToks - 1) / kToks);
  return even_splits(tiles, std::min({sms / blocks, tiles, (int64_t)64}));
}

cudaError_t launch_prefix_simt(const PrefixParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace mla
