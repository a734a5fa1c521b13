// Shared-prefix decode on the CUDA cores, in float32: the path of float32
// inputs (which need full precision) and of page sizes that the tensor-core
// kernel does not take.
//
// A CTA owns 32 stacked rows and a range of their 32-token tiles. Per tile:
//   S = Q . K^T    four groups of 64 threads take a quarter of the 576-wide dot
//                  each, 4 x 4 scores per thread; the quarters are summed by
//                  the softmax.
//   softmax        warp w keeps the online statistics of rows 4w .. 4w+3, lane
//                  = token.
//   O += P . V     thread = 8 rows x 8 columns of the 32 x 512 accumulator.
// Both products read 16-byte vectors of shared memory, 8 (S) and 16 (O) FMA per
// vector.
//
// Tokens that no row may see are zeros in the tile, so whatever their cache
// rows hold stays out of the sums; where a tile that some rows do not see holds
// an infinity or NaN, the rows whose weight is 0 skip it.
#include "prefix.h"

namespace mla {
namespace {

constexpr int kRows = 32, kToks = 32;
constexpr int kPad = 4;             // floats of row padding: 16-byte rows, 8 rows over all banks
constexpr int kPart = kToks + 1;

__host__ __device__ constexpr int pitch_of(int D) { return D + kPad; }

template <typename T> __device__ __forceinline__ float4 load4(const T* p);
template <> __device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

template <typename T>
__global__ void __launch_bounds__(256) prefix_simt(const PrefixParams p) {
  extern __shared__ float smem[];
  const int D = p.D, pitch = pitch_of(D);
  float* qs = smem;                              // [kRows][pitch]
  float* ks = qs + kRows * pitch;                // [kToks][pitch]
  float* part = ks + kToks * pitch;              // [4][kRows][kPart] quarter scores
  float* ps = part + 4 * kRows * kPart;          // [kToks][kRows] probabilities
  float* alpha = ps + kToks * kRows;             // [kRows]
  float* stat = alpha + kRows;                   // [kRows] 1 / denominator
  int* tok_ok = reinterpret_cast<int*>(stat + kRows);   // [kToks] some row may see the token

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * kRows, z = blockIdx.y;
  const int nr = min(kRows, p.N - r0);
  const int b0 = r0 / p.HQ, b1 = (r0 + nr - 1) / p.HQ;
  const int tiles = TileWalk<kToks>::count(p, b0, b1);
  const int per = (tiles + p.num_splits - 1) / p.num_splits;
  const int j0 = min(tiles, z * per), j1 = min(tiles, j0 + per);

  const int d4 = D / 4;
  for (int i = tid; i < kRows * d4; i += 256) {
    const int r = i / d4, k = 4 * (i - r * d4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nr)
      v = k < p.Ckv ? load4(reinterpret_cast<const T*>(p.q_lat) + (int64_t)(r0 + r) * p.Ckv + k)
                    : load4(reinterpret_cast<const T*>(p.q_pe) + (int64_t)(r0 + r) * p.Dr + (k - p.Ckv));
    *reinterpret_cast<float4*>(qs + r * pitch + k) = v;
  }

  // S: thread (ty, tx) of quarter kq holds rows ty + 8i, tokens tx + 8j
  const int kq = tid >> 6, ty = (tid >> 3) & 7, tx = tid & 7;
  const int kq4 = d4 / 4;                        // float4 steps per quarter (D is a multiple of 16)
  // softmax: rows 4 warp + i, lane = token
  float m_run[4], l_run[4];
  int row_b[4], row_lim[4];                      // sequence and last visible own token of the row
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
    const int r = r0 + 4 * warp + i;
    row_b[i] = r < p.N ? r / p.HQ : -2;
    row_lim[i] = 0x7fffffff;
    if (r < p.N && p.causal) row_lim[i] = prefix_len_of(p, row_b[i]) - p.Q + r % p.Q;
  }
  // O: rows 8 rg + i, columns 4 cg + k and 256 + 4 cg + k
  const int rg = tid >> 6, cg = tid & 63;
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;

  TileWalk<kToks> w;
  w.seek(p, b0, b1, j0);
  for (int j = j0; j < j1; ++j) {
    // a token's cache row; the base pointers are those of the tile's source
    const bool pre = w.b < 0;
    const T* kvp = reinterpret_cast<const T*>(pre ? p.pkv : p.kv);
    const T* pep = reinterpret_cast<const T*>(pre ? p.ppe : p.pe);
    const int64_t kvs = pre ? p.pkv_row : p.kv_row, pes = pre ? p.ppe_row : p.pe_row;
    const int32_t* table = pre ? p.ptable : p.table ? p.table + (int64_t)w.b * p.max_pages : nullptr;
    const int pages = pre ? p.p_pages : p.num_pages;
    if (!pre && !table) {
      kvp += w.b * p.kv_batch;
      pep += w.b * p.pe_batch;
    }
    const int pos0 = (pre ? 0 : p.Lp) + w.t;     // position of the tile's first token
    __syncthreads();                             // the last tile's readers are done
    bool odd = false;                            // this thread loaded an infinity or NaN
    for (int i = tid; i < kToks * d4; i += 256) {
      const int tt = i / d4, k = 4 * (i - tt * d4);
      const int t = w.t + tt;
      bool ok = t < w.end && (!p.mask || p.mask[pos0 + tt] != 0);
      int64_t row = t;
      if (ok && table) {
        const int page = table[t / p.page_size];
        ok = page >= 0 && page < pages;
        row = (int64_t)page * p.page_size + t % p.page_size;
        if (!ok) prefix_flag(p, MLA_DEVICE_ERR_BLOCK_TABLE);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ok) v = k < p.Ckv ? load4(kvp + row * kvs + k) : load4(pep + row * pes + (k - p.Ckv));
      odd = odd || !isfinite(v.x) || !isfinite(v.y) || !isfinite(v.z) || !isfinite(v.w);
      *reinterpret_cast<float4*>(ks + tt * pitch + k) = v;
      if (k == 0) tok_ok[tt] = ok;
    }
    const bool any_odd = __syncthreads_or(odd);
    {
      float s[4][4] = {};
      const float* qp = qs + ty * pitch + 4 * kq * kq4;
      const float* kp = ks + tx * pitch + 4 * kq * kq4;
#pragma unroll 2
      for (int k = 0; k < kq4; ++k) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qv[i] = *reinterpret_cast<const float4*>(qp + 8 * i * pitch + 4 * k);
          kv[i] = *reinterpret_cast<const float4*>(kp + 8 * i * pitch + 4 * k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            s[i][n] = fmaf(qv[i].x, kv[n].x, s[i][n]);
            s[i][n] = fmaf(qv[i].y, kv[n].y, s[i][n]);
            s[i][n] = fmaf(qv[i].z, kv[n].z, s[i][n]);
            s[i][n] = fmaf(qv[i].w, kv[n].w, s[i][n]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) part[(kq * kRows + ty + 8 * i) * kPart + tx + 8 * n] = s[i][n];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * warp + i;
      const int t = w.t + lane;
      // own tokens are seen by their sequence's rows; a causal row sees own
      // tokens up to row_lim (a negative one reaches back into the prefix)
      bool vis = tok_ok[lane] != 0 && row_b[i] >= 0 && (pre || row_b[i] == w.b);
      vis = vis && (!p.causal || (pre ? t - p.Lp : t) <= row_lim[i]);
      float s = -INFINITY;
      if (vis)
        s = ((part[r * kPart + lane] + part[(kRows + r) * kPart + lane]) +
             (part[(2 * kRows + r) * kPart + lane] + part[(3 * kRows + r) * kPart + lane])) * p.scale;
      float mx = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m_run[i], mx);
      const float al = m_run[i] == -INFINITY ? 0.f : expf(m_run[i] - m_new);
      const float e = vis ? expf(s - m_new) : 0.f;
      float sum = e;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l_run[i] = l_run[i] * al + sum;
      m_run[i] = m_new;
      ps[lane * kRows + r] = e;
      if (lane == 0) alpha[r] = al;
    }
    __syncthreads();
    float al[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) al[i] = alpha[8 * rg + i];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] *= al[i];
#pragma unroll 2
    for (int tt = 0; tt < kToks; ++tt) {
      const float4 p0 = *reinterpret_cast<const float4*>(ps + tt * kRows + 8 * rg);
      const float4 p1 = *reinterpret_cast<const float4*>(ps + tt * kRows + 8 * rg + 4);
      const float4 v0 = *reinterpret_cast<const float4*>(ks + tt * pitch + 4 * cg);
      const float4 v1 = *reinterpret_cast<const float4*>(ks + tt * pitch + 256 + 4 * cg);
      const float pr[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
      const float vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      if (!any_odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[i][k] = fmaf(pr[i], vv[k], acc[i][k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[i][k] = pr[i] != 0.f ? fmaf(pr[i], vv[k], acc[i][k]) : acc[i][k];
      }
    }
    w.next(p, b0);
  }

  // the rows' denominators to the accumulator's threads
  const bool split = p.num_splits > 1;
  __syncthreads();
  if (lane < 4) {
    float m = m_run[0], l = l_run[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (lane == i) {
        m = m_run[i];
        l = l_run[i];
      }
    const int r = r0 + 4 * warp + lane;
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
      if (split)
        p.ws_lse[(int64_t)z * p.N + r] = lse;
      else if (p.lse)
        p.lse[r] = lse;
    }
    stat[4 * warp + lane] = inv;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 8 * rg + i;
    if (r >= p.N) continue;
    const float inv = stat[8 * rg + i];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = (k < 4 ? 0 : 256) + 4 * cg + (k & 3);
      const float v = inv == 0.f ? 0.f : acc[i][k] * inv;
      if (split)
        p.ws_o[((int64_t)z * p.N + r) * p.Ckv + c] = v;
      else
        reinterpret_cast<T*>(p.x)[(int64_t)r * p.Ckv + c] = from_f32<T>(v);
    }
  }
}

template <typename T>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  const size_t smem = prefix_simt_smem(p.D);
  cudaError_t e = cudaFuncSetAttribute(prefix_simt<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  prefix_simt<T><<<dim3((p.N + kRows - 1) / kRows, p.num_splits), 256, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t prefix_simt_smem(int D) {
  return sizeof(float) * ((size_t)(kRows + kToks) * pitch_of(D) + 4 * kRows * kPart + kToks * kRows + 2 * kRows) +
         sizeof(int) * kToks;
}

// about one CTA per SM (its shared memory fills one), no split shorter than a tile
int prefix_simt_auto_splits(const mla_prefix_args* a, int sms) {
  const int64_t rows = (int64_t)a->B * a->H * a->Q;
  const int64_t blocks = (rows + kRows - 1) / kRows;
  const int64_t tiles = ((int64_t)a->prefix_len + kToks - 1) / kToks + (a->Lk + kToks - 1) / kToks;
  int64_t s = sms / blocks;
  if (s > tiles) s = tiles;
  if (s > 64) s = 64;
  return s < 1 ? 1 : (int)s;
}

cudaError_t launch_prefix_simt(const PrefixParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace mla
