// Shared-prefix decode: parameters and host-side launchers (internal; the
// public call is mla_prefix_decode in include/mla.h).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {

// Rows r = (b, h, q) of all sequences are stacked: r / HQ is the sequence,
// r % Q its query. A block of stacked rows walks the prefix's tokens, then the
// own tokens of each sequence it holds rows of.
struct PrefixParams {
  int B, H, Q, HQ, Ckv, Dr, D, N;   // N = B * HQ rows
  const void* q_lat;
  const void* q_pe;
  const void* pkv;
  const void* ppe;
  int64_t pkv_row, ppe_row;
  int Lp;
  const int32_t* ptable;
  int p_pages;
  const void* kv;
  const void* pe;
  int64_t kv_row, pe_row, kv_batch, pe_batch;
  int Lk;
  const int32_t* seq_lens;
  const int32_t* table;
  int max_pages, page_size, num_pages;
  const uint8_t* mask;
  int causal;
  float scale;
  const float* sinks;
  int num_splits;                   // ranges of a block at the most: those of the launch
  int wanted;                       // ranges that fill the GPU (with ws_ranges)
  int block_shift;                  // log2 of a block's rows
  void* x;
  float* lse;
  int32_t* err;
  float* ws_o;                      // (S, N, Ckv) normalised partial outputs
  float* ws_lse;                    // (S, N)
  int32_t* ws_ranges;               // (blocks) ranges that a block used, or null: num_splits
};

__device__ __forceinline__ void prefix_flag(const PrefixParams& p, int bit) {
  if (p.err) atomicOr(p.err, bit);
}

// Own length of sequence b, clamped to [0, Lk] (outside it: flagged).
__device__ __forceinline__ int prefix_len_of(const PrefixParams& p, int b) {
  if (!p.seq_lens) return p.Lk;
  const int L = p.seq_lens[b];
  if (L < 0 || L > p.Lk) {
    prefix_flag(p, MLA_DEVICE_ERR_BLOCK_TABLE);
    return L < 0 ? 0 : p.Lk;
  }
  return L;
}

// The tiles of TILE tokens that a block of rows walks: the prefix's, then each
// of its sequences' own. `b` is -1 in the prefix; tokens [t, end) of that
// source are in the tile. `lens` holds the own lengths of the block's sequences
// b0 .. b1, read once into shared memory.
template <int TILE>
struct TileWalk {
  int b, last, t, end;

  __device__ __forceinline__ static int tiles_of(int len) { return (len + TILE - 1) / TILE; }

  // all tiles of the block
  __device__ __forceinline__ static int count(const PrefixParams& p, const int* lens, int b0, int b1) {
    int n = tiles_of(p.Lp);
    for (int b = b0; b <= b1; ++b) n += tiles_of(lens[b - b0]);
    return n;
  }
  // position at tile `skip` of the block
  __device__ __forceinline__ void seek(const PrefixParams& p, const int* lens, int b0, int b1, int skip) {
    b = -1;
    last = b1;
    end = p.Lp;
    while (skip >= tiles_of(end)) {
      skip -= tiles_of(end);
      b = b < 0 ? b0 : b + 1;
      if (b > last) {
        t = end = 0;
        return;
      }
      end = lens[b - b0];
    }
    t = skip * TILE;
  }
  __device__ __forceinline__ void next(const int* lens, int b0) {
    t += TILE;
    while (t >= end) {
      b = b < 0 ? b0 : b + 1;
      if (b > last) return;
      t = 0;
      end = lens[b - b0];
    }
  }
};

// How a block cuts its tiles. The launch counts own tokens as the storage allows, the
// block as they are: with the launch's count, 4 sequences of 8 heads, 256 + up to 500
// tokens took 23 us with a table for 131072 tokens, 15 now, and 13 with one for 512.
struct Cut {
  int per;                          // tiles of a range
  bool several;                     // the outputs are partial ones
  bool idle;                        // this range is not used: nothing to write, nothing reads it
};

// Range z of a block of `tiles`, none of more than `most` if the launch has that many.
__device__ __forceinline__ Cut prefix_cut(const PrefixParams& p, int tiles, int most, int z) {
  const int n = max(tiles, 1);
  int s = p.num_splits;
  if (p.ws_ranges) s = min(max(min(p.wanted, n), (n - 1) / most + 1), s);
  Cut c;
  c.per = (n + s - 1) / s;
  c.several = p.ws_ranges ? c.per < n : s > 1;
  c.idle = p.ws_ranges && z * c.per >= n;
  return c;
}

// The ranges that a block uses, for the merge.
__device__ __forceinline__ void prefix_tell(const PrefixParams& p, int block, int tiles, const Cut& c) {
  if (p.ws_ranges) p.ws_ranges[block] = (max(tiles, 1) + c.per - 1) / c.per;
}

constexpr int kPrefixLeastShift = 5, kPrefixMostShift = 7;   // log2 of a block's rows: prefix_simt, prefix_sm100
constexpr int kPrefixMaxSplits = 256;   // ranges of a block that the merge holds the weights of

// At most s ranges (1 if less), as few as keep the longest as short: ranges that
// would be empty or shorter only lengthen the merge.
inline int even_splits(int64_t tiles, int64_t s) {
  if (s <= 1 || tiles <= 1) return 1;
  const int64_t per = (tiles + s - 1) / s;
  return (int)((tiles + per - 1) / per);
}

cudaError_t launch_prefix_simt(const PrefixParams& p, bool bf16, cudaStream_t st);
// Should the blocks cut their tiles by the lengths that they have? Not where these are
// the storage's, nor where own tokens, as the storage allows them, are few of the tiles:
// the merge then waits for one load less (13.0 : 13.3 us, 31.2 : 31.8 for small calls).
inline bool prefix_cut_by_lengths(const mla_prefix_args* a, int64_t own, int64_t tiles) {
  return a->seq_lens && own > 8 && own > tiles / 8;
}

// Ranges of a launch; `wanted`: how many fill the GPU, where the blocks cut by their
// lengths, else 0.
int prefix_simt_auto_splits(const mla_prefix_args* a, int sms, int* wanted);

bool prefix_sm100_supported(const mla_prefix_args* a);
int prefix_sm100_auto_splits(const mla_prefix_args* a, int sms, int* wanted);
cudaError_t launch_prefix_sm100(const PrefixParams& p, cudaStream_t st);

// merges the split partials in p.ws_o / p.ws_lse into p.x / p.lse
cudaError_t launch_prefix_combine(const PrefixParams& p, bool bf16, cudaStream_t st);

}  // namespace mla
