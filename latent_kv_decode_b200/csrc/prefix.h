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
  int num_splits;
  void* x;
  float* lse;
  int32_t* err;
  float* ws_o;                      // (S, N, Ckv) normalised partial outputs
  float* ws_lse;                    // (S, N)
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

constexpr int kPrefixMaxSplits = 256;   // ranges of a block that the merge holds the weights of

// At most s ranges (1 if less), as few as keep the longest as short: ranges that
// would be empty or shorter only lengthen the merge.
inline int even_splits(int64_t tiles, int64_t s) {
  if (s <= 1 || tiles <= 1) return 1;
  const int64_t per = (tiles + s - 1) / s;
  return (int)((tiles + per - 1) / per);
}

cudaError_t launch_prefix_simt(const PrefixParams& p, bool bf16, cudaStream_t st);
int prefix_simt_auto_splits(const mla_prefix_args* a, int sms);

bool prefix_sm100_supported(const mla_prefix_args* a);
int prefix_sm100_auto_splits(const mla_prefix_args* a, int sms);
cudaError_t launch_prefix_sm100(const PrefixParams& p, cudaStream_t st);

// merges the split partials in p.ws_o / p.ws_lse into p.x / p.lse
cudaError_t launch_prefix_combine(const PrefixParams& p, bool bf16, cudaStream_t st);

}  // namespace mla
