// Shared-prefix decode in float32, without tensor memory: the path of float32 inputs
// and of page sizes that the other kernel does not take.
//
// A CTA owns 32 stacked rows and a range of their 16-token tiles, two of which
// are in flight: the next tile's rows arrive (cp.async) while this one computes.
//   S = Q . K^T    a warp sums every eighth 16 channels for all rows and tokens; the
//                  parts are summed by the softmax.
//   softmax        warp w keeps the online statistics of rows 4w .. 4w+3, two at
//                  a time, a lane per token.
//   O += P . V     a warp owns 64 of the 512 columns.
// The products are mma.m16n8k16 on bf16 parts: a float32 value is the sum of three
// bf16, exactly (down to their smallest, 2^-133), and of the nine products of two such
// sums the six largest count (the others are below 2^-25 of the first). With bf16 inputs
// a score is one product, and a weight, a float32, two parts (to 2^-16 of it). The
// instruction adds in float32 and truncates, so what it adds up is kept short: a warp's
// part of a score is at most 30 such additions, a tile's share of O six; parts and
// tiles are added by rounding instructions. Behind 131072 tokens in one range x is
// then within 7e-6 where O in the instruction's accumulator had lost 1e-3 of it. Q is
// split once per CTA, K and V as their fragments are read, the weights by the softmax.
// Measured: 4.2 us a tile (S 1.5, softmax 0.8, O 1.2), where packed float32 FMAs, which
// shared memory feeds with 32 floats a clock, took 5.4; 128 rows behind 2049 tokens 39
// -> 31 us. (The warp-level instruction, as its operands come from registers, split
// there; for tcgen05 the parts would have to be written to shared memory in its layout.)
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

constexpr int kRows = 1 << kPrefixLeastShift, kToks = 16;
constexpr int kThr = 256, kWarps = kThr / 32, kParts = kWarps;   // kParts slices of the dot product
constexpr int kPad = 8;             // floats of row padding: four rows x eight floats cover the banks
constexpr int kPart = kToks + 1;
constexpr float kTop = 3.3895313892515355e38f;   // bf16's largest
constexpr int kProw = kToks / 2 + 4;             // 32-bit words of a row of weights

__host__ __device__ constexpr int pitch_of(int D) { return D + kPad; }
__host__ __device__ constexpr int qpitch_of(int D) { return D / 2 + 4; }     // words of a query row's piece

// bf16 pieces of a float32 operand: x = piece 0 + piece 1 + piece 2 exactly (a bf16
// operand is its own piece). Two weights in [0, 1] of bf16 values need two.
template <typename T> constexpr int kPieces = sizeof(T) == 4 ? 3 : 1;
template <typename T> constexpr int kWPieces = sizeof(T) == 4 ? 3 : 2;

// The pieces of a pair, the first value in the low halves. Each is the rest's nearest
// bf16, so a piece is at most 2^-9 of the one before it.
template <int kP> __device__ __forceinline__ void split(float x, float y, uint32_t (&p)[kP]) {
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    p[i] = sm100::pack_bf16(x, y);
    x -= __uint_as_float(p[i] << 16);
    y -= __uint_as_float(p[i] & 0xffff0000u);
  }
}

// The pieces of a query value that is not below bf16's largest: that first, then the
// rest; a non-finite value is its own first piece.
template <int kP> __device__ __forceinline__ void split_large(float x, uint16_t (&p)[kP]) {
  const bool finite = isfinite(x);
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const float h = i > 0 ? (finite ? x : 0.f) : finite ? fminf(fmaxf(x, -kTop), kTop) : x;
    p[i] = (uint16_t)sm100::pack_bf16(h, h);
    x -= __uint_as_float((uint32_t)p[i] << 16);
  }
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void copy16(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
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

template <typename T> __device__ __forceinline__ void decode_range(const PrefixParams& p) {
  extern __shared__ float smem[];
  __shared__ const T* row_lat[2][kToks];         // the tile's cache rows, null where no row may see the token
  __shared__ const T* row_pe[2][kToks];
  const int D = p.D, pitch = pitch_of(D);
  constexpr int kP = kPieces<T>, kWP = kWPieces<T>;
  const int qpitch = qpitch_of(D);
  uint32_t* qs = reinterpret_cast<uint32_t*>(smem);             // [kP][kRows][qpitch] pairs of channels
  float* ks = smem + kP * kRows * qpitch;        // [2][kToks][pitch]
  float* part = ks + 2 * kToks * pitch;          // [kParts][kRows][kPart] parts of the scores
  uint32_t* ps = reinterpret_cast<uint32_t*>(part + kParts * kRows * kPart);   // [kWP][kRows][kProw] weights
  float* alpha = reinterpret_cast<float*>(ps + kWP * kRows * kProw);           // [kRows]
  float* stat = alpha + kRows;                   // [kRows] 1 / denominator

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int r0 = blockIdx.x * kRows, z = blockIdx.y;
  const int nr = min(kRows, p.N - r0);
  const T* q_lat = reinterpret_cast<const T*>(p.q_lat) + (int64_t)r0 * p.Ckv;
  const T* q_pe = reinterpret_cast<const T*>(p.q_pe) + (int64_t)r0 * p.Dr;
  float4 q[kRows / kWarps][5];                   // the query rows, before anything waits
#pragma unroll
  for (int h = 0; h < kRows / kWarps; ++h)
#pragma unroll
    for (int u = 0; u < 5; ++u) {
      const int r = warp + h * kWarps, k = 4 * (lane + 32 * u);
      q[h][u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nr && k < D) q[h][u] = load4(k < kCkv ? q_lat + (int64_t)r * kCkv + k : q_pe + (int64_t)r * p.Dr + (k - kCkv));
    }
  const int b0 = r0 / p.HQ, b1 = (r0 + nr - 1) / p.HQ;
  __shared__ int lens[kRows / 8 + 1];            // H*Q >= 8: the sequences a block can hold rows of
  if (tid <= b1 - b0) lens[tid] = prefix_len_of(p, b0 + tid);
  __syncthreads();
  const int tiles = TileWalk<kToks>::count(p, lens, b0, b1);
  const Cut cut = prefix_cut(p, tiles, 0x7fffffff, z);
  if (tid == 0 && z == 0) prefix_tell(p, blockIdx.x, tiles, cut);
  if (cut.idle) return;
  const int per = cut.per;
  const int j0 = min(tiles, z * per), j1 = min(tiles, j0 + per);

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

  // the query rows as pieces, while the first tile arrives
  bool large = false;
#pragma unroll
  for (int h = 0; h < kRows / kWarps; ++h)
#pragma unroll
    for (int u = 0; u < 5; ++u) {
      const int r = warp + h * kWarps, k = 4 * (lane + 32 * u);
      if (k >= D) continue;
      const float4 v = q[h][u];
      large = large || !(fabsf(v.x) < kTop && fabsf(v.y) < kTop && fabsf(v.z) < kTop && fabsf(v.w) < kTop);
      uint32_t lo[kP], hi[kP];
      split<kP>(v.x, v.y, lo);
      split<kP>(v.z, v.w, hi);
#pragma unroll
      for (int c = 0; c < kP; ++c)
        *reinterpret_cast<uint2*>(qs + (c * kRows + r) * qpitch + k / 2) = make_uint2(lo[c], hi[c]);
    }
  if (large) {
    for (int r = warp; r < nr; r += kWarps)
      for (int k = 4 * lane; k < D; k += 128)
        for (int e = 0; e < 4; ++e) {            // this thread's values once more
          const float v = load1(k < kCkv ? q_lat + (int64_t)r * kCkv + k + e : q_pe + (int64_t)r * p.Dr + (k - kCkv) + e);
          if (fabsf(v) < kTop) continue;
          uint16_t x[kP];
          split_large<kP>(v, x);
          for (int c = 0; c < kP; ++c) reinterpret_cast<uint16_t*>(qs + (c * kRows + r) * qpitch)[k + e] = x[c];
        }
  }

  // S: a warp sums every eighth 16 channels
  const int gid = lane >> 2, tig = lane & 3;
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
  // O: rows 16 m + 8 (k / 2) + gid, columns 64 warp + 8 n + 2 tig + k % 2
  float acc[2][8][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < 8; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;

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
      float c[2][2][4] = {};                     // [16 rows][8 tokens]
      for (int k = 16 * warp; k < D; k += 16 * kParts) {
        uint32_t qa[2][kP][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < kP; ++i) {
            const uint32_t* a = qs + (i * kRows + 16 * m + gid) * qpitch + k / 2 + tig;
            qa[m][i][0] = a[0];
            qa[m][i][1] = a[8 * qpitch];
            qa[m][i][2] = a[4];
            qa[m][i][3] = a[8 * qpitch + 4];
          }
        uint32_t kb[2][2][kP];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 v = *reinterpret_cast<const float2*>(kt + (8 * n + gid) * pitch + k + 8 * h + 2 * tig);
            split<kP>(v.x, v.y, kb[n][h]);
          }
        // products of pieces down to 2^-18 of the first; the others are below 2^-25
#pragma unroll
        for (int sum = kP - 1; sum >= 0; --sum)
#pragma unroll
          for (int i = 0; i <= sum; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < 2; ++n) mma16816(c[m][n], qa[m][i], kb[n][0][sum - i], kb[n][1][sum - i]);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            part[(warp * kRows + 16 * m + 8 * (k >> 1) + gid) * kPart + 8 * n + 2 * tig + (k & 1)] = c[m][n][k];
            odd = odd || !isfinite(c[m][n][k]);
          }
    }
    const bool any_odd = __syncthreads_or(odd);
    if (any_odd) {
      // an infinity's pieces are no sum: the tile's scores once more, channel by channel
      for (int i = tid; i < kRows * kToks; i += kThr) {
        const int r = i / kToks, t = i % kToks;
        float v = 0.f;
        for (int k = 0; k < D; ++k) {
          float q = 0.f;
#pragma unroll
          for (int c = kP - 1; c >= 0; --c) {
            const uint32_t u = qs[(c * kRows + r) * qpitch + k / 2];
            q += __uint_as_float(k & 1 ? u & 0xffff0000u : u << 16);
          }
          v = fmaf(q, kt[t * pitch + k], v);
        }
#pragma unroll
        for (int c = 0; c < kParts; ++c) part[(c * kRows + r) * kPart + t] = c ? 0.f : v;
      }
      __syncthreads();
    }
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
      const float e = s != -INFINITY ? expf(s - m_new) : 0.f;   // also a visible score of -inf, whatever m_new
      float sum = e;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l_run[i] = l_run[i] * al + sum;
      m_run[i] = m_new;
      // tokens t, t + 4, t + 8, t + 12 are an MMA's K positions 2t, 2t + 1, 2t + 8, 2t + 9
      const int pos = ((tok >> 3) << 3) + 2 * (tok & 3) + ((tok >> 2) & 1);
      float rest = e;
#pragma unroll
      for (int c = 0; c < kWP; ++c) {
        const __nv_bfloat16 h = __float2bfloat16_rn(rest);
        reinterpret_cast<__nv_bfloat16*>(ps + (c * kRows + srow) * kProw)[pos] = h;
        rest -= __bfloat162float(h);
      }
      if (tok == 0) alpha[srow] = al;
    }
    __syncthreads();
    float al[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      al[m][0] = alpha[16 * m + gid];
      al[m][1] = alpha[16 * m + 8 + gid];
    }
    const float* vt = kt + 64 * warp;
    if (!any_odd) {
      uint32_t pa[2][kWP][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < kWP; ++c) {
          const uint32_t* q = ps + (c * kRows + 16 * m + gid) * kProw + tig;
          pa[m][c][0] = q[0];
          pa[m][c][1] = q[8 * kProw];
          pa[m][c][2] = q[4];
          pa[m][c][3] = q[8 * kProw + 4];
        }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float* v = vt + tig * pitch + 8 * n + gid;
        uint32_t v0[kP], v1[kP];
        split<kP>(v[0], v[4 * pitch], v0);
        split<kP>(v[8 * pitch], v[12 * pitch], v1);
        float c[2][4] = {};                      // the tile's own sum
#pragma unroll
        for (int sum = kWP - 1; sum >= 0; --sum)
#pragma unroll
          for (int i = 0; i < kP; ++i)
            if (sum - i >= 0)
#pragma unroll
              for (int m = 0; m < 2; ++m) mma16816(c[m], pa[m][sum - i], v0[i], v1[i]);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][n][k] = fmaf(acc[m][n][k], al[m][k >> 1], c[m][k]);
      }
    } else {
      // rows whose weight is 0 skip the token
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][n][k] *= al[m][k >> 1];
#pragma unroll 1
      for (int t = 0; t < kToks; ++t) {
        const int pos = ((t >> 3) << 3) + 2 * (t & 3) + ((t >> 2) & 1);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float pr = 0.f;
#pragma unroll
            for (int c = kWP - 1; c >= 0; --c)
              pr += __bfloat162float(
                  reinterpret_cast<const __nv_bfloat16*>(ps + (c * kRows + 16 * m + 8 * h + gid) * kProw)[pos]);
            if (pr != 0.f) {
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const float2 v = *reinterpret_cast<const float2*>(vt + t * pitch + 8 * n + 2 * tig);
                acc[m][n][2 * h] = fmaf(pr, v.x, acc[m][n][2 * h]);
                acc[m][n][2 * h + 1] = fmaf(pr, v.y, acc[m][n][2 * h + 1]);
              }
            }
          }
      }
    }
    w = wn;
    if (more) wn.next(lens, b0);
  }

  // the rows' denominators to the accumulator's threads
  const bool parts = cut.several;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float m = m_run[i], l = l_run[i];
    const int r = r0 + 4 * warp + 2 * i + sub;
    float inv = 0.f;
    if (r < p.N) {
      float wt = 1.f;
      if (!parts && p.sinks) {
        const float sk = p.sinks[(r % p.HQ) / p.Q], m2 = fmaxf(m, sk);
        if (m2 != -INFINITY) {                   // else nothing was seen and the sink adds nothing
          wt = m == -INFINITY ? 0.f : expf(m - m2);
          l = l * wt + expf(sk - m2);
        }
        m = m2;
      }
      const bool seen = !(m == -INFINITY && l == 0.f);   // a NaN denominator stays one
      inv = seen ? wt / l : 0.f;
      const float lse = seen ? m + logf(l) : -INFINITY;
      if (tok == 0) {
        if (parts)
          p.ws_lse[(int64_t)z * p.N + r] = lse;
        else if (p.lse)
          p.lse[r] = lse;
      }
    }
    if (tok == 0) stat[r - r0] = inv;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 16 * m + 8 * h + gid;
      if (r >= p.N) continue;
      const float inv = stat[r - r0];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int c = 64 * warp + 8 * n + 2 * tig;
        float2 v = make_float2(0.f, 0.f);
        if (inv != 0.f) v = make_float2(acc[m][n][2 * h] * inv, acc[m][n][2 * h + 1] * inv);
        if (parts)
          *reinterpret_cast<float2*>(p.ws_o + ((int64_t)z * p.N + r) * p.Ckv + c) = v;
        else if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float2*>(reinterpret_cast<T*>(p.x) + (int64_t)r * p.Ckv + c) = v;
        else
          *reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(p.x) + (int64_t)r * p.Ckv + c) = sm100::pack_bf16(v.x, v.y);
      }
    }
}

// One CTA fills an SM. The compiler's own choice of registers is 168 for float32, which leaves
// room for the merge to start early (8 x 16 heads behind 2049 tokens 31.2 us, with 241 registers
// 32.0, where 64 x 16 behind 4096 take 305 and 291); for bf16 it is 128 and spills (245 : 209 us).
template <typename T> __global__ void prefix_simt(const __grid_constant__ PrefixParams p);
template <> __global__ void __launch_bounds__(kThr) prefix_simt<float>(const __grid_constant__ PrefixParams p) {
  decode_range<float>(p);
}
template <> __global__ void __launch_bounds__(kThr, 1) prefix_simt<__nv_bfloat16>(const __grid_constant__ PrefixParams p) {
  decode_range<__nv_bfloat16>(p);
}

template <typename T>
constexpr size_t smem_bytes(int D) {
  return 4 * ((size_t)kPieces<T> * kRows * qpitch_of(D) + 2 * kToks * pitch_of(D) + kParts * kRows * kPart +
              kWPieces<T> * kRows * kProw + 2 * kRows);
}

template <typename T>
cudaError_t launch(const PrefixParams& p, cudaStream_t st) {
  const size_t smem = smem_bytes<T>(p.D);
  static OncePerDevice smem_set;
  cudaError_t e = smem_set([] {
    return cudaFuncSetAttribute(prefix_simt<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<T>(kCkv + 64));
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

// About one CTA per SM (its shared memory fills one), no split shorter than a
// tile: a tile takes 4.2 us, the merge of a few splits 3.
int prefix_simt_auto_splits(const mla_prefix_args* a, int sms, int* wanted) {
  const int HQ = a->H * a->Q;
  const int64_t rows = (int64_t)a->B * HQ;
  const int64_t blocks = (rows + kRows - 1) / kRows;
  const int64_t seqs = std::min<int64_t>(a->B, (kRows + HQ - 1) / HQ);   // of a block
  const int64_t own = seqs * ((a->Lk + kToks - 1) / kToks);
  const int64_t tiles = ((int64_t)a->prefix_len + kToks - 1) / kToks + own;
  const int64_t fill = std::max<int64_t>(std::min({sms / blocks, tiles, (int64_t)64}), 1);
  *wanted = prefix_cut_by_lengths(a, own, tiles) ? (int)fill : 0;
  return even_splits(tiles, fill);
}

cudaError_t launch_prefix_simt(const PrefixParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace mla
