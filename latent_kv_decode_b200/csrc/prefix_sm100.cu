// Shared-prefix decode on the tensor cores (mla_prefix_decode; bf16, Ckv = 512,
// Dr in {0, 32, 64}, contiguous storage or pages of a multiple of 64 rows).
//
// The rows (b, h, q) of all sequences are stacked. One 2-CTA cluster owns 128
// of them and a range of their 128-token tiles: the prefix's tiles, which all
// rows see, then the own tiles of each sequence it holds rows of, which only
// that sequence's rows see (the others' weights are 0). One accumulator takes
// both, so nothing is merged unless the tiles are cut over several clusters.
// Per pair, S and O cost 2 * 128 * 1088 flops a token whatever H is, and a token
// is read once per 128 rows: at H*Q >= 128 the tensor pipe is the bound, not
// the cache.
//
//   S  = Q . K^T       pair MMA, M = 128 (CTA r: rows [64r, 64r + 64)), N = the
//                      tile's 128 tokens (each CTA supplies its 64), K = 512 + 64.
//   softmax            online, base 2. A row's reference is the maximum of the
//                      first tile it sees and moves only when a score exceeds it
//                      by 2^60: weights, their sums and O are floating point, so
//                      a reference that is too low costs no precision until it
//                      overflows. The common tile therefore needs no row maximum
//                      across threads and no exchange of factors: each warp
//                      only tells the other CTA that none of its rows moved.
//                      (2^60 of weight, 2^17 tokens: values beyond 2^50 may overflow.)
//                      The weights go on as bf16, V's type, as both operands of an MMA
//                      have one; a second part of them would be half as many MMAs again.
//                      A row's sum adds them unrounded, so lse is float32's, and x errs
//                      by roundings of either sign, at most 2^-8 sum p |v|: 0.0017 to
//                      0.0019 of x in the measured cases, 0.0017 of that x's own rounding.
//   O^T += V^T . P^T   pair MMA, M = 256 latent dims (CTA r: dims 256n + 128r ..
//                      + 127 for n = 0, 1), N = the 128 rows, K = the tokens.
//
// Each CTA loads its own 64 tokens of a tile once (four 16 KB boxes: latent
// chunks 0-1, 4-5, 2-3, 6-7 into slots 0-1, 2-3, 4-5, 6-7 of the tile's set; and
// the rope chunk), and, once S has used them, the other CTA's tokens of its
// own dims over the four slots it does not aggregate. Tokens of CTA 0 are then
// in slots 0-3 and tokens of CTA 1 in slots 4-7 of both CTAs.
//
// A weight of 0 does not silence an infinity or NaN in V. Tiles that may hold
// rows which some query must not see ("guarded": own tokens, a tile's ragged
// end, the prefix's end behind a causal row's last token, a mask, a bad page) are
// cleaned before the aggregation: warp 2 zeroes the rows no query may see, and if S
// shows a non-finite key, the softmax warps zero the non-finite values (the rows that
// see that key are NaN by their S). A tile of own tokens therefore takes a third longer
// than one of the prefix (64 x 128 heads, 4096 tokens: 79 us as own ones, 63 as a prefix).
//
// A tile's 17 + 16 MMA steps of K = 64 take about 2870 SM cycles in the tensor
// pipe (1.46 us); a tile takes 1.53 us in a small GPC and 1.65 to 1.74 with all 74
// clusters busy, 1.5 to 1.6 PFLOP/s by the device, where the power limit (1.42 for a long
// library product) comes into sight. Not loading the other CTA's tokens at all (32 of
// 104 KB a tile) gains 2%. Measured (whole call, merge included): 128 sequences of 16
// heads x 2 queries behind 16384 tokens 157 us, 64 of 128 heads behind 4096 tokens 77 us,
// 4 of 128 heads behind 131072 tokens 145 us: 0.94, 1.00 and 1.01 PFLOP/s, with 64, 64
// and 72 clusters.
//
// Warps (384 threads): 0 own-token producer, 1 QK issuer (CTA 0) and TMEM
// owner, 2 peer-token producer and cleaner, 3 PV issuer (CTA 0), 4-11 softmax +
// epilogue (TMEM lane = 32 (warp % 4) + lane; the two sets of four split a lane's
// 64 scores). Every wait is bounded; a timeout sets MLA_DEVICE_ERR_TIMEOUT
// and the kernel unwinds.
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "once_per_device.h"
#include "prefix.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kSets = 2;                    // softmax warp sets; each reads 64 / kSets tokens of a lane
constexpr int kSoft = 128 * kSets;          // softmax threads (warps 4 and up)
constexpr int kSoftWarps = kSoft / 32;
constexpr int kThreads = 128 + kSoft;
constexpr int kTileT = 128;                 // tokens per tile (both CTAs)
constexpr int kRowsT = 1 << kPrefixMostShift;     // stacked rows per cluster
constexpr int kChunk = 8192;                // 64 rows (tokens or query rows) x 128 B

constexpr int kOffQ = 0;                    // 9 chunks: q_lat 0-7, q_pe
constexpr int kOffL = kOffQ + 9 * kChunk;   // 2 sets x 8 latent chunk slots
constexpr int kOffR = kOffL + 16 * kChunk;  // rope chunk slot
constexpr int kOffP = kOffR + kChunk;       // P: 2 blocks (tokens 0-63, 64-127) of 64 rows x 128 B
constexpr int kBigBytes = kOffP + 2 * kChunk;   // the 1024-aligned operand region
enum : int {
  B_QFULL = 0,
  B_KF = 1,               // [2][4] slots 2i, 2i+1 of both CTAs landed
  B_PV = 9,               // [2][4] PV(j) over slots 2i, 2i+1 (and before) done (both CTAs, multicast)
  B_XF = 17,              // [2] peer-token boxes landed (of both CTAs; a guarded tile: of CTA 0)
  B_SFULL = 19,           // [2] S(j) computed (both CTAs, multicast commit)
  B_PFULL = 21,           // [2] P(j) written, O^T rescaled, V clean in both CTAs (count 2)
  B_QH0 = 23,             // [2] QK(j) over slots 0-3 done (both CTAs, multicast)
  B_AX = 25,              // [2] the flags of the peer's softmax warps for tile j arrived
  B_RF = 27,              // the rope chunk of tile j of both CTAs landed (phase j)
  B_RFREE = 28,           // QK(j) over the rope chunk done: the rope slot is free (multicast)
  B_AL = 29,              // the peer's 64 rescale factors arrived (phase: moves so far)
  B_EPX = 30,             // the peer's output scales arrived
  B_XL = 31,              // CTA 1: its peer-token box of a guarded tile landed
  B_ZD = 32,              // [2] this CTA's rows of a guarded tile are clean (phase: guarded tiles so far)
  B_COUNT = 34
};
// Control block: barriers, TMEM address, abort flag, the peer's flags, lengths. In the
// alignment gap below the operand region when it fits there, else after the
// exchange block (row statistics, rescale factors, output scales).
constexpr int kOffTmemPtr = 8 * B_COUNT;
constexpr int kOffAbort = kOffTmemPtr + 4;
constexpr int kOffFlags = (kOffAbort + 4 + 15) & ~15;     // int [2 tiles][16 warps of the peer]
constexpr int kMaxSeqs = kRowsT / 8 + 1;                  // H*Q >= 8: the sequences a block can hold rows of
constexpr int kOffLens = kOffFlags + 2 * kSoftWarps * 4;  // int [kMaxSeqs]: their own lengths
constexpr int kOffCut = kOffLens + kMaxSeqs * 4;         // int: bit 0 several ranges, bit 1 idle
constexpr int kCtrlBytes = (kOffCut + 4 + 15) & ~15;
constexpr int kOffXmax = kBigBytes;                       // float [sets][128 lanes]
constexpr int kOffAlpha = kOffXmax + 512 * kSets;                // float [128]
constexpr int kOffScl = kOffAlpha + 512;                  // float [128]
constexpr int kXchgEnd = kOffScl + 512;
constexpr int kSmemAlloc = 232448;                        // the per-block limit
static_assert(kXchgEnd + kCtrlBytes + (kCtrlBytes - 16) <= kSmemAlloc, "shared memory over the per-block limit");
static_assert(kXchgEnd + 1008 <= kSmemAlloc, "shared memory over the per-block limit");

constexpr uint32_t kColS = 0;               // S buffers at columns 0 and 64 (pair M = 128 layout)
constexpr uint32_t kColO = 128;             // O^T halves n = 0, 1 at columns 128 and 256
constexpr uint32_t kTmemCols = 512;

constexpr int kTok = 64 / kSets;            // scores of a tile per softmax thread
constexpr uint32_t kAll = 0xffffffffu >> (32 - kTok);
constexpr int kMostTiles = 2048;            // of a range, 2^18 tokens (prefix_sm100_auto_splits)
constexpr float kMove = 60.0f;              // log2: how far a score may exceed its row's reference
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

struct alignas(64) TcParams {
  CUtensorMap tm_q;        // q_lat (N, 512), box 64 x 64
  CUtensorMap tm_qpe;      // q_pe (N, Dr), box 64 x 64 (columns beyond Dr read as 0)
  CUtensorMap tm_kv[2];    // prefix, own: (64 dims, rows, 8 chunks, seq | page), box 64 rows x 2 chunks
  CUtensorMap tm_kx[2];    // the same as (64 dims, rows, 4 chunks, 2 groups of 4, seq | page), box
                           // 64 rows x 2 chunks x 2 groups = chunks c, c+1, c+4, c+5
  CUtensorMap tm_pe[2];    // prefix, own: (Dr, rows, seq | page), box 64 x 64 rows
  PrefixParams p;
  float scale_log2;
  int blocks;              // 128-row blocks
};

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
  return e;
}

// The pair MMA and its commit for a converged warp whose elected lane (e != 0)
// issues them. The surrounding loop stays uniform, so descriptors live in
// uniform registers: issued from a single-lane branch, an MMA took 50-60 ns of
// register moves, twice what the tensor pipe needs for it.
__device__ __forceinline__ void mma_pair(uint32_t e, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 z;\n\t"
      "mov.b32 z, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {z, z, z, z, z, z, z, z}, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}

__device__ __forceinline__ void commit_pair(uint32_t e, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "mov.b16 m, 3;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar),
      "r"(e)
      : "memory");
}

// 2^x on the SFU; subnormal results flush to zero (a weight below 2^-126 of the
// row's reference, and so of its maximum).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void named_bar_sync(int id, int count) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

__device__ __forceinline__ bool bar_or(int id, int count, bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "barrier.red.or.pred po, %2, %3, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(out)
      : "r"((uint32_t)pred), "r"(id), "r"(count)
      : "memory");
  return out != 0;
}

// The 64 tokens of one CTA in a tile: the pool page and row of its first
// token, and whether they may be read (a bad table entry: page 0, not visible).
struct Block64 {
  int y, zc;
  bool ok;
};

__device__ __forceinline__ Block64 block64(const PrefixParams& p, const TileWalk<kTileT>& w, int half) {
  const int t = w.t + 64 * half;
  const bool pre = w.b < 0;
  const int32_t* table = pre ? p.ptable : p.table ? p.table + (int64_t)w.b * p.max_pages : nullptr;
  Block64 k;
  k.ok = true;
  if (!table) {
    k.y = t;
    k.zc = pre ? 0 : w.b;
    return k;
  }
  k.y = 0;
  k.zc = 0;
  if (t >= w.end) return k;
  const int pg = table[t / p.page_size];
  k.ok = pg >= 0 && pg < (pre ? p.p_pages : p.num_pages);
  if (k.ok) {
    k.zc = pg;
    k.y = t % p.page_size;
  }
  return k;
}

// Does a page that tiles [j0, j0 + nt) of the block may touch have a bad table
// entry? Shared by n threads. Looked up once, the common answer spares every
// softmax thread two table lookups a tile (182 -> 168 us for 128 sequences, 16
// heads, a 16384-token paged prefix).
__device__ __forceinline__ bool bad_pages(const PrefixParams& p, const int* lens, int b0, int b1, int j0, int nt, int tid,
                                          int n) {
  bool bad = false;
  const int64_t ps = p.page_size;
  if (p.ptable) {
    // 64 bits: a block's tiles, up to 17 sequences', may hold more than 2^31 tokens
    const int64_t first = (int64_t)j0 * kTileT, end = min((int64_t)p.Lp, first + (int64_t)nt * kTileT);
    for (int64_t i = first / ps + tid; i * ps < end; i += n) bad = bad || p.ptable[i] < 0 || p.ptable[i] >= p.p_pages;
  }
  if (p.table)
    for (int b = b0; b <= b1; ++b) {
      const int32_t* t = p.table + (int64_t)b * p.max_pages;
      const int len = lens[b - b0];
      for (int64_t i = tid; i * ps < len; i += n) bad = bad || t[i] < 0 || t[i] >= p.num_pages;
    }
  return bad;
}

// The prefix tokens that every row of the block is sure to see. With fewer own tokens
// than queries, a causal row ends before the prefix does. For a whole warp.
__device__ __forceinline__ int seen_by_all(const PrefixParams& p, const int* lens, int b0, int b1, int lane) {
  const int least = __reduce_min_sync(0xffffffffu, lane <= b1 - b0 ? lens[lane] : 0x7fffffff);
  return p.mask ? 0 : p.causal ? p.Lp + min(0, least - p.Q + 1) : p.Lp;
}

// May the tile hold rows that some query must not see?
__device__ __forceinline__ bool guarded(const TileWalk<kTileT>& w, int to_all, bool ok0, bool ok1) {
  return w.b >= 0 || w.t + kTileT > to_all || !ok0 || !ok1;
}

// 96 registers: the compiler's own schedule with 121 is slower (64 sequences of 128 heads
// behind 4096 tokens 70 us, with 104 68, with 88 to 96 64 to 66, with 80, which spills, 70;
// which of its choices costs it is not known).
__global__ void __maxnreg__(96) prefix_sm100_kernel(const __grid_constant__ TcParams P) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb0 = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb0 - raw);
  const uint32_t ctrl = (sb0 - raw >= (uint32_t)kCtrlBytes) ? raw : sb0 + kXchgEnd;
  uint8_t* ctrl_p = smem_raw + (ctrl - raw);
  const PrefixParams& p = P.p;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp-uniform
  const uint32_t rank = cluster_ctarank();
  const int item = blockIdx.x >> 1;
  const int rb = item % P.blocks, z = item / P.blocks;   // clusters of one range run together
  pdl_launch_dependents();
  auto bar = [&](int i) -> uint32_t { return ctrl + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl_p + kOffAbort);

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) mbar_init(bar(i), i == B_PFULL || i == B_PFULL + 1 ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_2sm(ctrl + kOffTmemPtr, kTmemCols);
    tmem_relinquish_2sm();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(ctrl_p + kOffTmemPtr), 0);
  // everything above overlaps the previous kernel; inputs are read from here on
  pdl_wait();
  const int r0 = rb * kRowsT;
  const int b0 = r0 / p.HQ, b1 = (min(p.N, r0 + kRowsT) - 1) / p.HQ;
  const bool rope = p.Dr > 0;
  int* lens = reinterpret_cast<int*>(ctrl_p + kOffLens);
  if (threadIdx.x == 0) {
    // the query rows do not wait for the lengths (with the lengths kept in shared
    // memory: 177 -> 169 us and 88 -> 83 us, the first two sizes above)
    const int qrow = r0 + (int)rank * 64;
    const uint32_t qbar = map_to_rank(bar(B_QFULL), 0);
    if (rank == 0) mbar_arrive_expect_tx(bar(B_QFULL), 2 * (rope ? 9 : 8) * kChunk);
    if (rope) tma_load_2d_2sm(sb0 + kOffQ + 8 * kChunk, &P.tm_qpe, qbar, 0, qrow);
    for (int c = 0; c < 8; ++c) tma_load_2d_2sm(sb0 + kOffQ + c * kChunk, &P.tm_q, qbar, 64 * c, qrow);
  } else if (threadIdx.x >= 32 && threadIdx.x - 32 <= b1 - b0) {
    lens[threadIdx.x - 32] = prefix_len_of(p, b0 + (int)threadIdx.x - 32);
  }
  __syncthreads();
  const int tiles = TileWalk<kTileT>::count(p, lens, b0, b1);
  const Cut cut = prefix_cut(p, tiles, kMostTiles, z);
  if (z == 0 && rank == 0 && threadIdx.x == 0) prefix_tell(p, rb, tiles, cut);
  const int j_begin = min(tiles, z * cut.per);
  const int ntiles = __shfl_sync(0xffffffffu, min(tiles, j_begin + cut.per) - j_begin, 0);
  TileWalk<kTileT> w;
  w.seek(p, lens, b0, b1, j_begin);

  auto fail = [&]() {
    *abort_flag = 1;
    prefix_flag(p, MLA_DEVICE_ERR_TIMEOUT);
  };
  // after a timeout: let copies and MMAs already issued end before this CTA's shared
  // memory and tensor memory go away
  auto settle = []() {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 50000ull) {
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ own-token producer
    if (lane == 0 && ntiles > 0) {
      bool ok = true;
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j & 1;
        const Block64 k = block64(p, w, (int)rank);
        if (!k.ok) prefix_flag(p, MLA_DEVICE_ERR_BLOCK_TABLE);
        const CUtensorMap* kv = &P.tm_kv[w.b < 0 ? 0 : 1];
        if (rope) {
          // the single rope slot, once QK(j-1) has read it
          if (j >= 1 && !mbar_wait_cluster(bar(B_RFREE), (j - 1) & 1)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(bar(B_RF), 2 * kChunk);
          tma_load_3d_2sm(sb0 + kOffR, &P.tm_pe[w.b < 0 ? 0 : 1], map_to_rank(bar(B_RF), 0), 0, k.y, k.zc);
        }
        // slots 2i, 2i+1 of set s held tile j-2 until its aggregation passed them
        for (int i = 0; i < 4; ++i) {
          if (j >= 2 && !mbar_wait_cluster(bar(B_PV + 4 * s + i), ((j - 2) >> 1) & 1)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(bar(B_KF + 4 * s + i), 2 * 2 * kChunk);
          tma_load_4d_2sm(sb0 + kOffL + (s * 8 + 2 * i) * kChunk, kv, map_to_rank(bar(B_KF + 4 * s + i), 0), 0, k.y,
                          ((i & 1) << 2) | (i & 2), k.zc);
        }
        if (*abort_flag) ok = false;
        w.next(lens, b0);
      }
      if (!ok) fail();
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ peer-token producer, cleaner
    // The peer tokens' chunks of this CTA's dims (CTA 0: chunks 0, 1, 4, 5; CTA
    // 1: 2, 3, 6, 7) go, as one box, over the four slots of the chunks this CTA
    // does not aggregate (CTA 0: slots 4-7, free once S(j) is computed; CTA 1:
    // slots 0-3, free once QK(j) has passed them). The box counts on CTA 0's
    // barrier, whose PV issuer waits for it; in a guarded tile CTA 1 waits for
    // its own box itself, cleans it, and vouches for it through P's barrier.
    bool ok = true;
    int ng = 0;
    const bool look = __any_sync(0xffffffffu, bad_pages(p, lens, b0, b1, j_begin, ntiles, lane, 32));
    const int to_all = seen_by_all(p, lens, b0, b1, lane);
    for (int j = 0; j < ntiles && ok; ++j) {
      const int s = j & 1;
      const Block64 peer = block64(p, w, 1 - (int)rank);
      const bool own_ok = !look || block64(p, w, (int)rank).ok;
      const bool g = guarded(w, to_all, own_ok, peer.ok);
      if (lane == 0) {
        ok = mbar_wait_cluster(bar((rank == 0 ? B_SFULL : B_QH0) + s), (j >> 1) & 1);
        if (ok) {
          const bool local = g && rank == 1;
          if (rank == 0) mbar_arrive_expect_tx(bar(B_XF + s), (g ? 4 : 8) * kChunk);
          if (local) mbar_arrive_expect_tx(bar(B_XL), 4 * kChunk);
          tma_load_5d_2sm(sb0 + kOffL + (s * 8 + 4 * (1 - (int)rank)) * kChunk, &P.tm_kx[w.b < 0 ? 0 : 1],
                          local ? map_to_rank(bar(B_XL), 1) : map_to_rank(bar(B_XF + s), 0), 0, peer.y,
                          2 * (int)rank, 0, peer.zc);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (g && ok) {
        // slots 4h .. 4h+3 hold the tokens of CTA h; a token's row is 128 bytes
        // of each slot, whatever the swizzle
        const int pos0 = (w.b < 0 ? 0 : p.Lp) + w.t;
        auto clean = [&](int h, bool page_ok) {
          for (int i0 = 0; i0 < 64; i0 += 32) {
            const int i = 64 * h + i0 + lane;
            const bool bad = !page_ok || w.t + i >= w.end || (p.mask && p.mask[pos0 + i] == 0);
            const uint32_t m = __ballot_sync(0xffffffffu, bad);
            uint8_t* rows = smem + kOffL + (s * 8 + 4 * h + (lane >> 3)) * kChunk + i0 * 128 + 16 * (lane & 7);
            if (m == 0) continue;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if ((m >> k) & 1u) *reinterpret_cast<uint4*>(rows + 128 * k) = make_uint4(0u, 0u, 0u, 0u);
          }
        };
        if (rank == 1) ok = mbar_wait_cluster(bar(B_SFULL + s), (j >> 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) clean((int)rank, own_ok);
        if (ok) ok = rank == 0 ? mbar_wait_cluster(bar(B_XF + s), (j >> 1) & 1) : mbar_wait_cluster(bar(B_XL), ng & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) clean(1 - (int)rank, peer.ok);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_ZD + (ng & 1)));
        ++ng;
      }
      if (*abort_flag) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      w.next(lens, b0);
    }
    if (!ok && lane == 0) fail();
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ QK issuer (CTA 0)
    // S(j) = Q . K^T in five groups as their data lands: the rope chunk (then a
    // commit that frees its slot for tile j+1), then two slots at a time (after
    // slots 0-3 a commit that frees them for CTA 1's peer-token box). The S buffer was read by
    // softmax(j-2) once P(j-2) is complete.
    if (rank == 0 && ntiles > 0) {
      const uint32_t el = elect_one();
      const uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
      const uint64_t qd0 = smem_desc(sb0 + kOffQ, 16, 1024, kSwizzle128B);
      const uint64_t kd0 = smem_desc(sb0 + kOffL, 16, 1024, kSwizzle128B);
      const uint64_t rd0 = smem_desc(sb0 + kOffR, 16, 1024, kSwizzle128B);
      bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar(B_QFULL), 0));
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j & 1;
        const uint32_t d = tmem + kColS + 64u * s;
        if (j >= 2) ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar(B_PFULL + s), ((j - 2) >> 1) & 1));
        if (rope && ok) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar(B_RF), j & 1));
          tc_fence_after();
          const uint64_t qd = desc_advance(qd0, 8 * kChunk);
          if (ok) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_pair(el, d, desc_advance(qd, 32 * k), desc_advance(rd0, 32 * k), idesc_qk, k != 0);
            commit_pair(el, bar(B_RFREE));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar(B_KF + 4 * s + i), (j >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            // slot 2i + cc holds latent chunk (0, 1, 4, 5, 2, 3, 6, 7)[slot]
            const uint64_t qd = desc_advance(qd0, (((i & 1) << 2) | (i & 2) | cc) * kChunk);
            const uint64_t kd = desc_advance(kd0, (s * 8 + 2 * i + cc) * kChunk);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_pair(el, d, desc_advance(qd, 32 * k), desc_advance(kd, 32 * k), idesc_qk,
                       rope || i > 0 || cc > 0 || k > 0);
          }
          if (i == 1) commit_pair(el, bar(B_QH0 + s));
        }
        if (ok) commit_pair(el, bar(B_SFULL + s));
        if (__any_sync(0xffffffffu, *abort_flag != 0)) ok = false;
      }
      if (!ok && lane == 0) fail();
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------------ PV issuer (CTA 0)
    // O^T += V^T . P^T: first the tokens of CTA 0 (slots 2n, 2n+1 for half n), then
    // those of CTA 1 (slots 4+2n, 5+2n), each pair of slots freed by its commit.
    if (rank == 0) {
      const uint32_t el = elect_one();
      const uint32_t idesc_pv = idesc_bf16_f32(256, 128, true, false);
      const uint64_t vd0 = smem_desc(sb0 + kOffL, kChunk, 1024, kSwizzle128B);
      const uint64_t pd0 = smem_desc(sb0 + kOffP, 16, 1024, kSwizzle128B);
      bool ok = true;
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar(B_XF + s), (j >> 1) & 1) &&
                                         mbar_wait_cluster(bar(B_PFULL + s), (j >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {        // token half i / 2, dims half n = i % 2
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_pair(el, tmem + kColO + 128u * (i & 1), desc_advance(vd0, (s * 8 + 2 * i) * kChunk + kk * 2048),
                     desc_advance(pd0, (i >> 1) * kChunk + kk * 32), idesc_pv, j > 0 || i > 1 || kk > 0);
          commit_pair(el, bar(B_PV + 4 * s + i));
        }
        if (__any_sync(0xffffffffu, *abort_flag != 0)) ok = false;
      }
      if (!ok && lane == 0) fail();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    // Two warp sets read each TMEM lane quarter, 32 of the lane's 64 tokens each,
    // so a row's scores sit with four threads (two token halves x two sets).
    const int g = warp & 3;
    const int sset = (warp >> 2) - 1;
    const int L = 32 * g + lane;                // TMEM lane
    const int half = L >> 6, row = L & 63;      // S: this CTA's row, token half
    const int xi = 128 * sset + L;
    const bool owner = half == 0 && sset == 0;  // one thread per row sends its factors
    const bool leader = xi == 0;                // arrives for this CTA
    const int r = r0 + (int)rank * 64 + row;
    const bool live = r < p.N;
    const int my_b = live ? r / p.HQ : -2;
    const uint32_t lane_base = (uint32_t)(32 * g) << 16;
    float* xmax = reinterpret_cast<float*>(smem + kOffXmax);
    float* alpha_s = reinterpret_cast<float*>(smem + kOffAlpha);
    float* scl = reinterpret_cast<float*>(smem + kOffScl);
    const int* flags = reinterpret_cast<const int*>(ctrl_p + kOffFlags);
    const uint32_t peer = rank ^ 1u;
    const uint32_t peer_flag = map_to_rank(ctrl + kOffFlags + 4u * (uint32_t)(4 * sset + g), peer);
    // a row's values (two token halves x the sets) reduced to all of its threads
    auto across = [&](float v, auto op) {
      xmax[xi] = v;
      named_bar_sync(2, kSoft);
      float t = op(xmax[row], xmax[64 + row]);
#pragma unroll
      for (int k = 1; k < kSets; ++k) t = op(t, op(xmax[128 * k + row], xmax[128 * k + 64 + row]));
      return t;
    };
    const int col = (int)rank * 64 + row;       // this row's column of O^T
    float m_run = -INFINITY, l_part = 0.f;
    bool ab = false;
    int ng = 0, moves = 0;
    const float sl2 = P.scale_log2;
    const uint8_t* mask = p.mask;
    // the last token a causal row sees, as a position (own token 0 is at Lp)
    const int last_pos = !live ? -1 : p.causal ? p.Lp + lens[my_b - b0] - p.Q + r % p.Q : 0x3fffffff;

    // kept in shared memory over the loop, whose registers are counted
    volatile int* cut_s = reinterpret_cast<volatile int*>(ctrl_p + kOffCut);
    if (leader) *cut_s = (cut.several ? 1 : 0) | (cut.idle ? 2 : 0);
    const bool look = bar_or(1, kSoft, bad_pages(p, lens, b0, b1, j_begin, ntiles, xi, kSoft));
    const int to_all = seen_by_all(p, lens, b0, b1, lane);

    for (int j = 0; j < ntiles; ++j) {
      const int sb = j & 1;
      const int ts = w.t + 64 * half + kTok * sset;            // this thread's first token
      const int base = w.b < 0 ? 0 : p.Lp;
      bool ok0 = true, ok1 = true;
      if (look) {
        ok0 = block64(p, w, 0).ok;
        ok1 = block64(p, w, 1).ok;
      }
      const bool gd = guarded(w, to_all, ok0, ok1);
      int lim = min(w.end, last_pos - base + 1) - ts;          // tokens [ts, ts + lim) pass all but the mask
      if (!live || (w.b >= 0 && w.b != my_b) || !(half ? ok1 : ok0)) lim = 0;
      uint32_t vis = kAll;                                     // the mask over [ts, ts + kTok), the same across the warp
      if (mask) vis = kAll & __ballot_sync(0xffffffffu, ts + lane < w.end && mask[base + ts + lane] != 0);
      if (leader) mbar_arrive_expect_tx(bar(B_AX + sb), kSoftWarps * 4);
      if (!ab) ab = !mbar_wait_cluster(bar(B_SFULL + sb), (j >> 1) & 1);
      ab = __any_sync(0xffffffffu, ab);
      const uint32_t s_addr = tmem + lane_base + kColS + 64u * sb + (uint32_t)(kTok * sset);
      const float m_sub = m_run == -INFINITY ? 0.f : m_run;
      float e[kTok];
      auto load_scores = [&]() {
        uint32_t v[kTok / 16][16];
#pragma unroll
        for (int c = 0; c < kTok / 16; ++c) tmem_ld16(s_addr + 16u * c, v[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kTok; ++c) e[c] = __uint_as_float(v[c / 16][c % 16]);
      };
      if (!ab) {
        tc_fence_after();
        load_scores();
      } else {
        lim = 0;
#pragma unroll
        for (int c = 0; c < kTok; ++c) e[c] = 0.f;
      }
      tc_fence_before();
      // a non-finite score among the tile's tokens: a non-finite key (guarded tiles)
      bool odd = false;
      if (gd) {
        float acc = 0.f;
#pragma unroll
        for (int c = 0; c < kTok; ++c) acc += c < w.end - ts ? e[c] * 0.f : 0.f;
        odd = !(acc == 0.f);
      }
      // log2 units relative to the row's reference, masked
      const bool whole = __all_sync(0xffffffffu, lim >= kTok) && vis == kAll;
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto scale_scores = [&](float sub) {
        if (whole) {
#pragma unroll
          for (int c = 0; c < kTok; ++c) e[c] = fmaf(e[c], sl2, -sub);
        } else {
#pragma unroll
          for (int c = 0; c < kTok; ++c)
            e[c] = (c < lim && ((vis >> c) & 1u)) ? fmaf(e[c], sl2, -sub) : -INFINITY;
        }
      };
      scale_scores(m_sub);
#pragma unroll
      for (int c = 0; c < kTok; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], e[c]);
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      // the row's first visible score sets its reference (its O is 0 so far); one
      // far above the reference moves it, and O^T of both CTAs with it
      const bool first = m_run == -INFINITY && mx > -INFINITY;
      const bool need = m_run != -INFINITY && mx > kMove;
      const bool warp_need = __any_sync(0xffffffffu, need);
      if (lane == 0) st_async_b32(peer_flag + 4u * kSoftWarps * (uint32_t)sb, warp_need ? 1u : 0u, map_to_rank(bar(B_AX + sb), peer));

      float psum;
      uint32_t pk[kTok / 2];
      auto weights = [&]() {
        float ps4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kTok / 2; ++c) {
          const float p0 = fast_exp2(e[2 * c]), p1 = fast_exp2(e[2 * c + 1]);
          ps4[c & 3] += p0 + p1;
          pk[c] = pack_bf16(p0, p1);
        }
        psum = (ps4[0] + ps4[1]) + (ps4[2] + ps4[3]);
      };
      uint8_t* prow = smem + kOffP + half * kChunk + row * 128;
      auto store_weights = [&]() {
#pragma unroll
        for (int c = 0; c < kTok / 8; ++c)
          *reinterpret_cast<uint4*>(prow + 16 * ((kTok / 8 * sset + c) ^ (row & 7))) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
      };
      weights();
      // the P buffer (and O^T) are free once PV(j-1) is done
      if (j >= 1 && !ab) ab = !mbar_wait_cluster(bar(B_PV + 4 * (sb ^ 1) + 3), ((j - 1) >> 1) & 1);
      store_weights();
      if (!ab) ab = !mbar_wait_cluster(bar(B_AX + sb), (j >> 1) & 1);
      bool peer_need = false;
#pragma unroll
      for (int k = 0; k < kSoftWarps; ++k) peer_need = peer_need || flags[kSoftWarps * sb + k] != 0;
      if (bar_or(1, kSoft, first || need || odd || peer_need || ab)) {
        // the rare tile: a reference is set, or moves in one of the CTAs, or a
        // non-finite key has to be silenced
        if (bar_or(1, kSoft, ab)) {
          ab = true;
          break;
        }
        const bool set = bar_or(1, kSoft, first || need || peer_need);
        const bool move = bar_or(1, kSoft, need || peer_need);   // both CTAs agree
        const bool dirty = bar_or(1, kSoft, odd);
        float alpha = 1.f;
        if (set) {
          if (leader && move) mbar_arrive_expect_tx(bar(B_AL), 64 * 4);
          const float m_all = across(mx + m_sub, [](float a, float b) { return fmaxf(a, b); });
          const bool mv = m_run == -INFINITY ? m_all > -INFINITY : m_all > m_run + kMove;
          alpha = mv && m_run != -INFINITY ? exp2f(m_run - m_all) : 1.f;
          if (mv) m_run = m_all;
          l_part *= alpha;
          load_scores();
          scale_scores(m_run == -INFINITY ? 0.f : m_run);
          weights();
          store_weights();
        }
        if (move) {
          // O^T's columns are rows of both CTAs: both rescale their dims of all 128
          if (owner) {
            alpha_s[col] = alpha;
            st_async_b32(map_to_rank(smem_u32(alpha_s + col), peer), __float_as_uint(alpha), map_to_rank(bar(B_AL), peer));
          }
          if (!ab) ab = !mbar_wait_cluster(bar(B_AL), moves & 1);
          ++moves;
          ab = __any_sync(0xffffffffu, ab);
          named_bar_sync(2, kSoft);
          if (j > 0 && !ab) {
            tc_fence_after();
            // set n rescales half n
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              uint32_t v[16];
              const uint32_t ta = tmem + lane_base + kColO + 128u * sset + (uint32_t)c;
              tmem_ld16(ta, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha_s[c + i]);
              tmem_st16(ta, v);
            }
            tmem_wait_st();
          }
        }
        if (dirty) {
          if (!ab) ab = !mbar_wait_cluster(bar(B_ZD + (ng & 1)), (ng >> 1) & 1);   // both token blocks are in and cleaned
          uint4* v = reinterpret_cast<uint4*>(smem + kOffL + sb * 8 * kChunk);
          auto keep = [](uint32_t u) {
            if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
            if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
            return u;
          };
          for (int i = xi; i < 8 * kChunk / 16; i += kSoft) {
            const uint4 u = v[i];
            v[i] = make_uint4(keep(u.x), keep(u.y), keep(u.z), keep(u.w));
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        named_bar_sync(2, kSoft);
      }
      l_part += psum;
      if (gd) {
        if (leader && !ab) ab = !mbar_wait_cluster(bar(B_ZD + (ng & 1)), (ng >> 1) & 1);
        ++ng;
      }
      if (leader) mbar_arrive_remote_cta(map_to_rank(bar(B_PFULL + sb), 0));
      w.next(lens, b0);
    }

    // ---------------------------------------------------------------- epilogue
    // the rows' denominators, then each row's output scale to both CTAs
    ab = bar_or(1, kSoft, ab);
    const float l_tot = across(l_part, [](float a, float b) { return a + b; });
    const int cut_bits = *cut_s;
    const bool split = cut_bits & 1, idle = cut_bits & 2;
    const bool seen = !(m_run == -INFINITY && l_tot == 0.f);   // a NaN denominator stays one
    float scale_o = seen ? 1.f / l_tot : 0.f;
    float lse = seen ? (m_run + log2f(l_tot)) * kLn2 : -INFINITY;
    if (!split && p.sinks && live) {
      const float sk = p.sinks[(r % p.HQ) / p.Q] * kLog2e;
      const float m2 = fmaxf(m_run, sk);
      if (m2 != -INFINITY) {
        const float wt = seen ? exp2f(m_run - m2) : 0.f;
        const float l2 = (seen ? l_tot * wt : 0.f) + exp2f(sk - m2);
        scale_o = wt / l2;
        lse = (m2 + log2f(l2)) * kLn2;
      }
    }
    if (leader) mbar_arrive_expect_tx(bar(B_EPX), 64 * 4);
    if (owner) {
      scl[col] = scale_o;
      st_async_b32(map_to_rank(smem_u32(scl + col), peer), __float_as_uint(scale_o), map_to_rank(bar(B_EPX), peer));
      if (live && !idle) {
        if (split)
          p.ws_lse[(int64_t)z * p.N + r] = lse;
        else if (p.lse)
          p.lse[r] = lse;
      }
    }
    if (ntiles > 0 && !ab) ab = !mbar_wait_cluster(bar(B_PV + 4 * ((ntiles - 1) & 1) + 3), ((ntiles - 1) >> 1) & 1);
    if (!ab) ab = !mbar_wait_cluster(bar(B_EPX), 0);
    ab = __any_sync(0xffffffffu, ab);
    ab = bar_or(1, kSoft, ab);
    if (ab) fail();
    tc_fence_after();
    const bool have_o = ntiles > 0 && !ab;
    // this thread's O^T lane is latent dim d0 + lane of half n; its columns are
    // the block's rows. Each warp (32 dims) moves 16 rows at a time through
    // shared memory (the free tile slots), so the output goes out as 16-byte
    // stores of whole 64- or 128-byte row pieces.
    uint8_t* stage = smem + kOffL + (4 * sset + g) * 2048;   // 16 rows x 32 dims x 4 B per warp
    const int n = sset;                                      // set n stores half n
    const int d0 = 256 * n + 128 * (int)rank + 32 * g;       // this warp's first dim
#pragma unroll 1
    for (int c0 = 0; c0 < kRowsT && r0 + c0 < p.N && !idle; c0 += 16) {
      uint32_t v[16];
      if (have_o) {
        tmem_ld16(tmem + lane_base + kColO + 128u * n + (uint32_t)c0, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0u;
      }
      float f[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = scl[c0 + i] == 0.f ? 0.f : __uint_as_float(v[i]) * scl[c0 + i];
      if (split) {
        float* st = reinterpret_cast<float*>(stage);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i * 32 + lane] = f[i];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = (lane >> 3) + 4 * k, ch = lane & 7;
          if (r0 + c0 + rr < p.N)
            *reinterpret_cast<uint4*>(p.ws_o + ((int64_t)z * p.N + r0 + c0 + rr) * kCkv + d0 + 4 * ch) =
                *reinterpret_cast<const uint4*>(st + rr * 32 + 4 * ch);
        }
      } else {
        __nv_bfloat16* st = reinterpret_cast<__nv_bfloat16*>(stage);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i * 32 + lane] = __float2bfloat16_rn(f[i]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int rr = (lane >> 2) + 8 * k, ch = lane & 3;
          if (r0 + c0 + rr < p.N)
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.x) + (int64_t)(r0 + c0 + rr) * kCkv + d0 +
                                      8 * ch) = *reinterpret_cast<const uint4*>(st + rr * 32 + 8 * ch);
        }
      }
      __syncwarp();
    }
  }

  // ------------------------------------------------------------------ teardown
  // an empty range still has its query rows in flight (both CTAs' on CTA 0's barrier)
  if (ntiles == 0 && rank == 0 && threadIdx.x == 0 && !mbar_wait_cluster(bar(B_QFULL), 0)) fail();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) settle();                  // whichever wait gave up: no copy or MMA outlives the block
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_2sm(tmem, kTmemCols);
  }
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

bool encode(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
            const uint32_t* box) {
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base),
                     reinterpret_cast<const cuuint64_t*>(dims), reinterpret_cast<const cuuint64_t*>(strides),
                     reinterpret_cast<const cuuint32_t*>(box), elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of one source: `outer` sequences or pages of `rows` rows
bool encode_source(CUtensorMap* kv, CUtensorMap* kx, CUtensorMap* pe, const void* kvp, const void* pep, int64_t kv_row, int64_t pe_row,
                   uint64_t kv_outer, uint64_t pe_outer, uint64_t rows, uint64_t outer, int Dr) {
  const uint64_t d4[4] = {64, rows, 8, outer};
  const uint64_t s4[3] = {(uint64_t)kv_row * 2, 128, kv_outer * 2};
  const uint32_t b4[4] = {64, 64, 2, 1};
  if (!encode(kv, kvp, 4, d4, s4, b4)) return false;
  const uint64_t d[5] = {64, rows, 4, 2, outer};
  const uint64_t s[4] = {(uint64_t)kv_row * 2, 128, 512, kv_outer * 2};
  const uint32_t bx[5] = {64, 64, 2, 2, 1};
  if (!encode(kx, kvp, 5, d, s, bx)) return false;
  if (Dr == 0) return true;
  const uint64_t dp[3] = {(uint64_t)Dr, rows, outer};
  const uint64_t sp[2] = {(uint64_t)pe_row * 2, pe_outer * 2};
  const uint32_t bp[3] = {64, 64, 1};
  return encode(pe, pep, 3, dp, sp, bp);
}

}  // namespace

bool prefix_sm100_supported(const mla_prefix_args* a) {
  if (a->dtype != MLA_BF16) return false;
  if ((a->prefix_table || a->block_table) && a->page_size % 64 != 0) return false;
  static OncePerDevice sm100;
  return encode_fn() != nullptr && sm100([] {
           int dev = 0, major = 0;
           const cudaError_t e = cudaGetDevice(&dev);
           if (e != cudaSuccess) return e;
           return cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess && major == 10
                      ? cudaSuccess
                      : cudaErrorNotSupported;
         }) == cudaSuccess;
}

// As many clusters as run at once, but no range shorter than a tile of the blocks' most
// (own tokens counted as the storage allows, their lengths being on the device, where
// a block then takes the ranges that it needs): down to one tile a range the merge costs less than the tiles it spares (16 sequences of 8
// heads, 500 + 100 tokens: 43, 22, 16 us with 1, 5, 20 ranges). And no range much above
// 2^18 tokens: the tensor pipe adds to O once per 16 tokens and truncates, which takes
// more of x the longer the range (behind 2^17, 2^20, 2^22 tokens of equal weight 0.0008,
// 0.006 and 0.024 of it, where a rounding to bf16 takes at most 0.0039).
int prefix_sm100_auto_splits(const mla_prefix_args* a, int sms, int* wanted) {
  const int pairs = sms / 2, HQ = a->H * a->Q;
  const int64_t blocks = ((int64_t)a->B * HQ + kRowsT - 1) / kRowsT;
  const int64_t seqs = std::min<int64_t>(a->B, (kRowsT + HQ - 1) / HQ);   // of a block
  const int64_t own = seqs * ((a->Lk + kTileT - 1) / kTileT);
  const int64_t tiles = ((int64_t)a->prefix_len + kTileT - 1) / kTileT + own;
  const int64_t least = std::min<int64_t>(((int64_t)a->prefix_len + a->Lk + (1 << 18) - 1) >> 18, kPrefixMaxSplits);
  const int64_t fill = std::max<int64_t>(std::min(pairs / blocks, tiles), 1);
  *wanted = prefix_cut_by_lengths(a, own, tiles) ? (int)fill : 0;
  return even_splits(tiles, std::max(fill, least));
}

cudaError_t launch_prefix_sm100(const PrefixParams& p, cudaStream_t st) {
  TcParams P;
  memset(static_cast<void*>(&P), 0, sizeof(P));
  P.p = p;
  P.scale_log2 = p.scale * kLog2e;
  P.blocks = (p.N + kRowsT - 1) / kRowsT;
  const uint32_t box[2] = {64, 64};
  {
    const uint64_t d[2] = {512, (uint64_t)p.N}, s[1] = {1024};
    if (!encode(&P.tm_q, p.q_lat, 2, d, s, box)) return cudaErrorInvalidValue;
  }
  if (p.Dr > 0) {
    const uint64_t d[2] = {(uint64_t)p.Dr, (uint64_t)p.N}, s[1] = {(uint64_t)p.Dr * 2};
    if (!encode(&P.tm_qpe, p.q_pe, 2, d, s, box)) return cudaErrorInvalidValue;
  }
  if (p.Lp > 0) {
    const uint64_t rows = p.ptable ? p.page_size : p.Lp;
    if (!encode_source(&P.tm_kv[0], &P.tm_kx[0], &P.tm_pe[0], p.pkv, p.ppe, p.pkv_row, p.ppe_row, rows * p.pkv_row,
                       rows * p.ppe_row, rows, p.ptable ? p.p_pages : 1, p.Dr))
      return cudaErrorInvalidValue;
  }
  if (p.Lk > 0) {
    const uint64_t rows = p.table ? p.page_size : p.Lk;
    const bool dense = p.table || p.B == 1;      // the batch stride is unused
    if (!encode_source(&P.tm_kv[1], &P.tm_kx[1], &P.tm_pe[1], p.kv, p.pe, p.kv_row, p.pe_row,
                       dense ? rows * p.kv_row : (uint64_t)p.kv_batch, dense ? rows * p.pe_row : (uint64_t)p.pe_batch,
                       rows, p.table ? p.num_pages : p.B, p.Dr))
      return cudaErrorInvalidValue;
  }
  static OncePerDevice smem_set;
  cudaError_t e = smem_set([] {
    return cudaFuncSetAttribute(prefix_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * P.blocks * p.num_splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, prefix_sm100_kernel, P);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
