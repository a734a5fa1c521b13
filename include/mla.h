/*
 * mla.h - C ABI of libmla.so: single-step Multi-Head Latent Attention decode
 * with weight absorption, on NVIDIA B200 (sm_100a).
 *
 * The operation is mla_decode_step of the 6547.cn exam question "MLA 单步解码":
 *
 *   q_lat  = q_nope . W_UK[h]                      (blank [1])   mla_absorb_q
 *   logit  = (q_lat . kv[t] + q_pe . pe[t]) * scale (blanks [2],[3])
 *   logit  = -inf where t is not visible           (blank [4])
 *   x      = softmax(logit) . kv                   (step 5)      mla_decode
 *                                                                 (+ mla_combine)
 *   out    = x . W_UV[h]^T                         (blank [5])   mla_up_proj
 *
 * with wkv_b (H, Dn+Vd, Ckv) split as W_UK = rows [0,Dn), W_UV = the last Vd
 * rows (the question's weight-split lines). The absorbed score
 * q_absorbed . c_kv + q_rope . k_rope is the associativity step written in
 * the comments of MultiHeadLatentAttention.forward_inference on the neuronix
 * page "DeepSeek-V3/R1 架构深度全景解析". The shared-latent variant (K = V =
 * one 512-dim latent stored as FP4 E2M1 with an E4M3 scale per 16 channels,
 * a sink logit per head, inverse RoPE on the output's last 64 dims) is the
 * openarchlab DeepSeek-V4.1-Flash page "4A · Multi-head Latent Attention"
 * (§1 Định nghĩa, §2 Luồng, §4 Profiling); the grouped output projection that
 * follows it there (§2 Luồng, §3 W_O nhóm) is mla_group_wo. The step before
 * the decode, writing a new token into its cache slot, is mla_cache_append;
 * mla_rope_append is that step on raw projection outputs, mla_prefix_decode the
 * decode of a batch that shares a prefix, mla_fp4_linear a projection whose
 * weights are FP4 entries.
 *
 * Conventions for every call:
 *  - Tensor pointers are DEVICE pointers owned by the caller. The library
 *    allocates no device memory and keeps no per-call state; calls are
 *    re-entrant. The one piece of library-global device state is the scratch
 *    array of mla_decode_static_scratch (a static device array, with its
 *    address looked up once per device); no other call touches it. Arrays
 *    are row-major (C order) and densely packed unless a stride argument says
 *    otherwise.
 *  - Every call only enqueues work on `stream` (a cudaStream_t; NULL = the
 *    legacy default stream) and returns without synchronising.
 *  - Arguments are validated on the host before anything is enqueued; a call
 *    that returns anything but MLA_OK has enqueued nothing, except
 *    MLA_ERR_CUDA, which reports a failed launch (see mla_last_cuda_error).
 *  - Device pointers must be 16-byte aligned.
 *  - Supported shapes (decode, projections, combine, append): Ckv = 512; Dr
 *    in {0 (shared-latent variant), 32, 64}; Dn in {64, 128}; Vd = 128; H a
 *    multiple of 8, at most 128; Q in [1, 4]. mla_group_wo, mla_rope_append,
 *    mla_prefix_decode and mla_fp4_linear state their own.
 *    Anything else returns MLA_ERR_UNSUPPORTED.
 */
#ifndef LATENT_KV_DECODE_MLA_H
#define LATENT_KV_DECODE_MLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mla_status {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,  /* null/shape/stride/alignment/range error */
  MLA_ERR_UNSUPPORTED = 2,  /* dims or dtype combination not built */
  MLA_ERR_WORKSPACE = 3,    /* workspace missing or too small */
  MLA_ERR_CUDA = 4          /* a launch failed; mla_last_cuda_error() has the code */
} mla_status_t;

typedef enum mla_dtype {
  MLA_F32 = 0,              /* IEEE float32 */
  MLA_BF16 = 1,             /* bfloat16 storage, float32 arithmetic */
  MLA_FP4_E2M1_E4M3x16 = 2  /* cache only: 288-byte entries, see mla_decode_args */
} mla_dtype_t;

/* Human-readable name of a status code (static string, never NULL). */
const char* mla_status_string(mla_status_t s);

/* cudaError_t of the last MLA_ERR_CUDA returned on the calling host thread (0 if none). */
int mla_last_cuda_error(void);

/* Library version, e.g. "0.1.0". */
const char* mla_version(void);

/*
 * mla_absorb_q - blank [1] of mla_decode_step: q_lat[b,h,q,:] = q_nope[b,h,q,:] . W_UK[h].
 *
 *   q_nope (B,H,Q,Dn)      dtype dt
 *   wkv_b  (H,Dn+Vd,Ckv)   dtype dt; rows [0,Dn) of each head are W_UK[h]
 *   q_lat  (B,H,Q,Ckv)     dtype dt, written
 * dt is MLA_F32 or MLA_BF16; accumulation is float32.
 */
mla_status_t mla_absorb_q(const void* q_nope, const void* wkv_b, void* q_lat, int B, int H,
                          int Q, int Dn, int Vd, int Ckv, mla_dtype_t dt, void* stream);

/*
 * mla_up_proj - blank [5] of mla_decode_step: out[b,h,q,:] = W_UV[h] . x[b,h,q,:].
 *
 *   x      (B,H,Q,Ckv)     dtype dt
 *   wkv_b  (H,Dn+Vd,Ckv)   dtype dt; the last Vd rows of each head are W_UV[h]
 *   out    (B,H,Q,Vd)      dtype dt, written
 */
mla_status_t mla_up_proj(const void* x, const void* wkv_b, void* out, int B, int H, int Q,
                         int Dn, int Vd, int Ckv, mla_dtype_t dt, void* stream);

/*
 * Arguments of mla_decode / mla_combine: blanks [2]-[4] and step 5 of
 * mla_decode_step over a compressed cache, with optional ragged lengths,
 * paging, causal speculative queries, sinks and split-KV.
 *
 * Query (rows r = (b, h, q)):
 *   q_lat   (B,H,Q,Ckv) dtype q_dtype. For the shared-latent variant this is the
 *           query itself (already RoPE-rotated on its tail).
 *   q_pe    (B,H,Q,Dr)  dtype q_dtype, or NULL when Dr == 0.
 *
 * Cache (cache_dtype = q_dtype, or MLA_FP4_E2M1_E4M3x16 with Dr == 0):
 *   Contiguous (block_table == NULL): token t of sequence b is row
 *     kv_cache + b*kv_batch_stride + t*kv_row_stride (in elements), and the
 *     same with pe_* for pe_cache; the question's kv_cache (B,Lk,Ckv) and
 *     pe_cache (B,Lk,Dr) have row strides Ckv and Dr. A combined 576-wide
 *     row (latent then rope) is kv_cache = base, pe_cache = base + 512, both
 *     row strides 576.
 *   Paged (block_table != NULL): kv_cache/pe_cache point at pools of
 *     num_pages pages of page_size rows; token t of sequence b is row
 *     (block_table[b*max_pages + t/page_size]*page_size + t%page_size) of the
 *     pool, with the given row strides (batch strides unused).
 *   FP4: each row is one 288-byte entry (strides in BYTES): bytes 0..255 hold
 *     512 E2M1 codes, channel 2i in the low nibble of byte i and 2i+1 in the
 *     high nibble; bytes 256..287 hold the E4M3 scale of channels 16g..16g+15.
 *     K = V = the dequantised latent (openarchlab 4A §1, 288 B per entry).
 *
 * Visibility of token t to row (b,h,q): t < len_b (len_b = seq_lens[b], or Lk
 *   when seq_lens is NULL) and causal_mask[t] != 0 (when causal_mask is given;
 *   the question's (1,1,1,Lk) mask, 1 = visible) and, when `causal` is
 *   non-zero, t <= len_b - Q + q (the Q new tokens are the last Q rows).
 *   A row that sees nothing gets x = 0 and lse = -inf.
 *
 * Softmax: logit = score * softmax_scale. With `sinks` (H floats) the
 *   denominator also holds exp(sinks[h]) (a raw logit, not scaled), which
 *   carries no value (openarchlab 4A §2 attn_sink column).
 * Epilogue: rope_tail in {0, 64}: x's last rope_tail dims are rotated back by
 *   the query position len_b - Q + q, pairs (D-tail+2j, D-tail+2j+1) by angle
 *   -pos * rope_theta^(-2j/tail) (openarchlab 4A §2 inverse RoPE).
 *
 * Outputs: x (B,H,Q,Ckv) in q_dtype; lse (B,H,Q) float32 natural-log softmax
 *   denominator (tokens and sink), or NULL.
 *
 * Split-KV: num_splits = 0 picks a count from the SM count and the shape
 *   (mla_decode_num_splits reports it). With 1 split, mla_decode writes x and
 *   lse itself. With S > 1 splits, sequence b's tokens are cut into S ranges
 *   of whole 64-token tiles; mla_decode writes each range's normalised
 *   partial output and log-sum-exp into the workspace, and mla_combine must
 *   then be called with the same arguments and workspace to write x and lse.
 *
 * err_flag: optional device int32; the kernels OR in MLA_DEVICE_ERR_* bits
 *   when they meet bad data (a block_table entry outside [0,num_pages)) and
 *   skip that data instead of reading out of bounds. The caller clears it.
 */
typedef struct mla_decode_args {
  int B, H, Q;
  int Ckv;                 /* 512 */
  int Dr;                  /* 0, 32 or 64 */
  mla_dtype_t q_dtype;     /* MLA_F32 or MLA_BF16 (q_lat, q_pe, x) */
  mla_dtype_t cache_dtype; /* q_dtype, or MLA_FP4_E2M1_E4M3x16 */
  const void* q_lat;
  const void* q_pe;
  const void* kv_cache;
  const void* pe_cache;
  int64_t kv_row_stride, pe_row_stride;      /* elements (bytes for FP4) */
  int64_t kv_batch_stride, pe_batch_stride;  /* contiguous layout only */
  int Lk;                  /* contiguous: rows per sequence; paged: max_pages*page_size */
  const int32_t* seq_lens; /* (B) or NULL */
  const int32_t* block_table; /* (B,max_pages) or NULL */
  int max_pages, page_size, num_pages;
  const uint8_t* causal_mask; /* (Lk) or NULL */
  int causal;
  float softmax_scale;
  const float* sinks;      /* (H) or NULL */
  int rope_tail;           /* 0 or 64 */
  float rope_theta;
  int num_splits;          /* 0 = auto */
  void* x;                 /* out (B,H,Q,Ckv) */
  float* lse;              /* out (B,H,Q) or NULL */
  int32_t* err_flag;       /* optional device status word */
} mla_decode_args;

#define MLA_DEVICE_ERR_BLOCK_TABLE 1  /* a page id outside [0,num_pages) or a seq_lens entry outside [0,Lk] */
#define MLA_DEVICE_ERR_TIMEOUT 2      /* a bounded wait inside a kernel gave up */

/* Resolved split count for these arguments (>= 1), or -1 if they are invalid. */
int mla_decode_num_splits(const mla_decode_args* a);

/* Workspace bytes mla_decode needs for these arguments (0 when 1 split). */
size_t mla_decode_workspace_size(const mla_decode_args* a);

/*
 * mla_decode - scores against the compressed cache, mask, softmax and latent
 * aggregation (blanks [2]-[4] and step 5). `workspace` is a device buffer of
 * at least mla_decode_workspace_size(a) bytes (may be NULL when that is 0).
 */
mla_status_t mla_decode(const mla_decode_args* a, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * mla_combine - merge the split partials that mla_decode left in `workspace`:
 * L = log(sum_s e^{lse_s} [+ e^{sink_h}]), x = sum_s e^{lse_s - L} O_s, then
 * the inverse-RoPE epilogue; writes a->x and a->lse. A no-op returning MLA_OK
 * when the resolved split count is 1.
 */
mla_status_t mla_combine(const mla_decode_args* a, const void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * mla_decode_static_scratch - mla_decode followed by mla_combine, for callers
 * that may not allocate device memory. The source pages have no counterpart: this is
 * a deployment variant of the two calls above.
 *
 * Some callers cannot call cudaMalloc or take memory from an allocator: a
 * serving engine that reserved nearly all of HBM for its KV cache at start-up
 * (an allocation at decode time would fail), or a plugin hook of a host
 * runtime that forbids allocation inside the hook. This entry point needs no
 * workspace argument: the split-KV partials go to one array of
 * MLA_STATIC_SCRATCH_BYTES bytes of device memory that the library owns,
 * which every GPU that loads the library holds until the process exits.
 *
 *   - Takes the same arguments as mla_decode and writes a->x and a->lse; they
 *     are final when the work it enqueued on `stream` completes.
 *   - Returns MLA_ERR_WORKSPACE, enqueuing nothing, when the resolved split
 *     count needs more than MLA_STATIC_SCRATCH_BYTES (see
 *     mla_decode_workspace_size); one split needs no scratch at all.
 *   - The first call on each device looks up the array's device address with
 *     that device current; make that first call before any stream capture.
 *     The address is kept for the life of the process, so this entry point
 *     does not support cudaDeviceReset (which reloads the module and moves
 *     the array) between its calls on a device.
 *   - All calls share the one array, whatever the stream. Calls whose GPU
 *     work overlaps in time race on it and give wrong results: serialise them
 *     (one stream, or events). The array keeps the last call's contents;
 *     nothing in it needs to start at zero, because mla_decode writes every
 *     partial that mla_combine reads in the same call.
 *   - Calls no cudaMalloc, cudaFree or allocating library routine.
 */
#define MLA_STATIC_SCRATCH_BYTES (32u << 20)
mla_status_t mla_decode_static_scratch(const mla_decode_args* a, void* stream);

/*
 * mla_cache_append - the step before the decode: write each sequence's Q new
 * tokens into the cache rows mla_decode reads. The neuronix DeepSeek-V3/R1
 * page's LatentKVCachePool gives a token's latent and rope parts a slot at its
 * position before attention runs; the openarchlab 4A page (§1, §4) stores the
 * shared latent, its tail rotated at the token's position, as a 288-byte FP4
 * entry.
 *
 *   c_kv  (B,Q,Ckv) new latent rows, src_dtype, contiguous.
 *   k_pe  (B,Q,Dr)  new rope rows (already rotated), src_dtype, contiguous;
 *         NULL when Dr == 0.
 *   seq_lens (B) int32, required: the lengths AFTER the append. New token i
 *     of sequence b is token t = seq_lens[b] - Q + i and goes to the row that
 *     mla_decode reads for t: the same kv_cache / pe_cache, row and batch
 *     strides, Lk, block_table, max_pages, page_size and num_pages rules.
 *   cache_dtype == src_dtype (MLA_F32 or MLA_BF16): the rows are copied.
 *   cache_dtype == MLA_FP4_E2M1_E4M3x16 (Ckv = 512, Dr = 0, src MLA_F32 or
 *     MLA_BF16, row stride in BYTES, >= 288 and a multiple of 16): the
 *     latent's last rope_tail (0 or 64) dims are rotated by +t, pairs
 *     (448+2j, 449+2j) by angle t * rope_theta^(-2j/64) (angles in double,
 *     results rounded to float); then each group of 16 channels gets
 *     scale = E4M3(amax / 6) and codes E2M1(x / scale), both rounded to
 *     nearest-even from float32 quotients with saturation (x's sign kept; a
 *     zero scale gives zero codes), in the entry layout mla_decode reads.
 *   err_flag: optional device int32; a token with t outside [0, Lk) or a page
 *     id outside [0, num_pages) sets MLA_DEVICE_ERR_BLOCK_TABLE and is not
 *     written.
 */
typedef struct mla_append_args {
  int B, Q;
  int Ckv, Dr;
  mla_dtype_t src_dtype;   /* MLA_F32 or MLA_BF16 (c_kv, k_pe) */
  mla_dtype_t cache_dtype; /* src_dtype, or MLA_FP4_E2M1_E4M3x16 */
  const void* c_kv;
  const void* k_pe;
  void* kv_cache;
  void* pe_cache;
  int64_t kv_row_stride, pe_row_stride;      /* elements (bytes for FP4) */
  int64_t kv_batch_stride, pe_batch_stride;  /* contiguous layout only */
  int Lk;                  /* contiguous: rows per sequence; paged: max_pages*page_size */
  const int32_t* seq_lens; /* (B), lengths after the append */
  const int32_t* block_table; /* (B,max_pages) or NULL */
  int max_pages, page_size, num_pages;
  int rope_tail;           /* FP4 only: 0 or 64 */
  float rope_theta;
  int32_t* err_flag;       /* optional device status word */
} mla_append_args;

mla_status_t mla_cache_append(const mla_append_args* a, void* stream);

/*
 * mla_group_wo - the step after the shared-latent decode's inverse RoPE: the
 * grouped low-rank output projection (openarchlab DeepSeek-V4.1-Flash 4A,
 * §2 Luồng "Group-LoRA W_O (8 nhóm × 1024)" back to [B, T, D_model]; §3 W_O
 * nhóm: each group of heads has its own small projection, the groups'
 * results side by side).
 *
 * For every token t = b*Q + q and group g of the G groups of H/G
 * consecutive heads:
 *   u_g[t]          = x[b, g*H/G .. (g+1)*H/G - 1, q, :] laid head-major ((H/G)*Ckv values)
 *   z[t, g*R + r]   = sum_k wo_a[g, r, k] * u_g[t, k]           (group g's own factor)
 *   out[t, n]       = sum_k wo_b[n, k] * z[t, k]                 (shared factor; omitted
 *                                                                 when wo_b is NULL: out = z)
 * D_model is not given by the page; D is the caller's.
 *
 * Layouts (row-major, bf16, device pointers owned by the caller, 16-byte
 * aligned): x (B,H,Q,Ckv); wo_a (G,R,(H/G)*Ckv); wo_b (D,G*R) or NULL;
 * out (B,Q,D), or (B,Q,G*R) without wo_b.
 * Supported: q/weight dtype MLA_BF16, Ckv a multiple of 64, H a multiple of
 *   G, R and D multiples of 128, Q in 1..16; fp32 accumulation, z rounded
 *   to bf16 between the two factors. Anything else: MLA_ERR_UNSUPPORTED.
 * workspace: at least mla_group_wo_workspace_size(a) bytes of device memory
 *   (z and the split-K partial sums), or NULL when that is 0; smaller gives
 *   MLA_ERR_WORKSPACE with nothing enqueued.
 * err_flag: optional device int32; MLA_DEVICE_ERR_TIMEOUT when a bounded
 *   wait inside the kernel gave up (the output is then not written).
 */
typedef struct mla_group_wo_args {
  int B, H, Q, Ckv;
  int G, R, D;             /* groups, rank per group, output width (ignored without wo_b) */
  mla_dtype_t dtype;       /* MLA_BF16 */
  const void* x;
  const void* wo_a;
  const void* wo_b;        /* or NULL */
  void* out;
  int32_t* err_flag;       /* optional device status word */
} mla_group_wo_args;

size_t mla_group_wo_workspace_size(const mla_group_wo_args* a);
mla_status_t mla_group_wo(const mla_group_wo_args* a, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * mla_rope_append - the append of a whole step or prompt with the position
 * rotation on the way: new latent rows are copied into the cache, the new
 * rope rows are rotated at their positions and stored, and the queries'
 * position parts are rotated by the same angles. mla_cache_append copies rope
 * rows that arrive rotated; this call takes the projections' raw outputs.
 *
 *   Tokens: N new tokens in rows of c_kv, k_pe and q_pe, in sequence order.
 *     cu_tokens == NULL: sequence b owns rows [b*Q, (b+1)*Q), N = B*Q.
 *     cu_tokens (B+1) int32, non-decreasing: sequence b owns rows
 *     [cu_tokens[b], cu_tokens[b+1]) (none is allowed); rows outside
 *     [cu_tokens[0], cu_tokens[B]) belong to no sequence: nothing is
 *     written for them. Q is then ignored.
 *   seq_lens (B) int32, required: the lengths AFTER the append. The i-th of a
 *     sequence's n new tokens is token t = seq_lens[b] - n + i and goes to the
 *     row mla_decode reads for t (kv_cache / pe_cache, strides, Lk,
 *     block_table, page_size as there).
 *   Rotation: position pos_offset + t (pos_offset = the length of a shared
 *     prefix stored elsewhere, else 0); pair (2j, 2j+1) of the Dr dims turns by
 *     pos * rope_theta^(-2j/Dr).
 *   c_kv row n at c_kv + n*c_kv_stride, k_pe row n at k_pe + n*k_pe_stride.
 *   q_pe (or NULL with H = 0): head h of row n at q_pe + n*q_token_stride +
 *     h*q_head_stride; its rotation goes to q_out + n*o_token_stride +
 *     h*o_head_stride with cu_tokens, and to q_out + (n/Q)*o_batch_stride +
 *     (n%Q)*o_token_stride + h*o_head_stride without (mla_decode's (B,H,Q,Dr)
 *     has strides H*Q*Dr, Dr, Q*Dr). q_out may be q_pe with the same strides;
 *     other overlaps of inputs and outputs are not allowed. Strides are in
 *     elements; pointers need the alignment of an element, and 16-byte
 *     aligned rows take the wide path.
 *   dtype: MLA_F32 or MLA_BF16, of every tensor. Ckv = 512; Dr 32 or 64; any H
 *     up to 1024.
 *   err_flag: optional device int32; a token with t outside [0, Lk) or a page
 *     id outside [0, num_pages) sets MLA_DEVICE_ERR_BLOCK_TABLE and is not
 *     written to the cache (its queries are still rotated).
 */
typedef struct mla_rope_append_args {
  int B, Q, N;
  int Ckv, Dr, H;
  mla_dtype_t dtype;       /* MLA_F32 or MLA_BF16 */
  const void* c_kv;
  const void* k_pe;
  const void* q_pe;        /* or NULL (H = 0) */
  void* q_out;             /* or NULL (H = 0) */
  int64_t c_kv_stride, k_pe_stride;
  int64_t q_token_stride, q_head_stride;
  int64_t o_batch_stride, o_token_stride, o_head_stride;
  void* kv_cache;
  void* pe_cache;
  int64_t kv_row_stride, pe_row_stride;
  int64_t kv_batch_stride, pe_batch_stride;  /* contiguous layout only */
  int Lk;                  /* contiguous: rows per sequence; paged: max_pages*page_size */
  const int32_t* seq_lens; /* (B), lengths after the append */
  const int32_t* block_table; /* (B,max_pages) or NULL */
  int max_pages, page_size, num_pages;
  const int32_t* cu_tokens; /* (B+1) or NULL */
  int pos_offset;
  float rope_theta;
  int32_t* err_flag;       /* optional device status word */
} mla_rope_append_args;

mla_status_t mla_rope_append(const mla_rope_append_args* a, void* stream);

/*
 * mla_prefix_decode - mla_decode for a batch whose sequences all begin with
 * the same prefix, stored once:
 *
 *   logit = (q_lat . c[t] + q_pe . r[t]) * softmax_scale over the prefix's
 *           tokens, then over the sequence's own
 *   x     = softmax(logit) . c,  lse = log sum exp(logit)
 *
 * The rows of all sequences are stacked, so the prefix is read once per 128
 * of them, whatever the number of heads per sequence.
 *
 *   q_lat (B,H,Q,Ckv), q_pe (B,H,Q,Dr), x (B,H,Q,Ckv), lse (B,H,Q) as for
 *     mla_decode, in dtype (lse float32).
 *   Prefix: prefix_len tokens (0 allowed). prefix_table == NULL: token t is row
 *     t of prefix_kv / prefix_pe (row strides in elements). Else token t is row
 *     prefix_table[t/page_size]*page_size + t%page_size of pools of
 *     prefix_num_pages pages; the table holds ceil(prefix_len/page_size) ids.
 *   Own tokens: kv_cache / pe_cache, strides, Lk, seq_lens, block_table,
 *     max_pages, num_pages as for mla_decode; they count the tokens behind the
 *     prefix, so token t of a sequence is at position prefix_len + t. Lk = 0
 *     (no own tokens; kv_cache may be NULL) and lengths of 0 are allowed.
 *     page_size is that of both tables. The two storages may share a pool.
 *   Visibility: t < length; causal_mask[position] != 0 when causal_mask
 *     (prefix_len + Lk) is given; when causal is non-zero, position <=
 *     prefix_len + len_b - Q + q. A row that sees nothing gets x = 0 and
 *     lse = -inf (+ the sink). Cache rows that no query may see (behind a
 *     sequence's end, masked by causal_mask, on a bad page) may hold
 *     anything, NaN included.
 *   sinks: as for mla_decode.
 *   Supported: MLA_F32 or MLA_BF16; Ckv = 512; Dr 0, 32 or 64; H a multiple of 8
 *     up to 128, Q 1..4; B*H*Q up to 2^24, prefix_len + Lk up to 2^30.
 *   Precision: MLA_F32 in float32's (a product is six of bf16 parts). MLA_BF16:
 *     exact products, float32 sums and statistics; for x the softmax weights
 *     are rounded to bf16 (at most 2^-8 of a weight, of either sign; lse uses
 *     them unrounded), with pages of other than a multiple of 64 rows to
 *     2^-16. bf16 with contiguous storage or pages of a multiple of 64 rows runs
 *     at the tensor cores' full rate; there x of a range loses about 2^-23 of
 *     itself per 16 tokens to truncation, 0.0008 behind 2^17 tokens.
 *   num_splits: 0 = auto (as many as fill the GPU, and for bf16 at least one per
 *     2^18 tokens; num_splits reports the most that the storage can ask for, a
 *     block uses what its lengths ask for). Each block of stacked rows cuts its
 *     tokens into this many ranges, and the call then merges the partial results itself (no
 *     mla_combine): x and lse are final when the enqueued work completes.
 *   workspace: mla_prefix_decode_workspace_size(a) bytes, 256-byte aligned
 *     (may be NULL when that is 0). It is written before it is read in every call;
 *     calls whose GPU work overlaps in time need one each.
 *   err_flag: as for mla_decode.
 */
typedef struct mla_prefix_args {
  int B, H, Q;
  int Ckv, Dr;
  mla_dtype_t dtype;
  const void* q_lat;
  const void* q_pe;
  const void* prefix_kv;
  const void* prefix_pe;
  int64_t prefix_kv_stride, prefix_pe_stride;
  int prefix_len;
  const int32_t* prefix_table; /* (ceil(prefix_len/page_size)) or NULL */
  int prefix_num_pages;
  const void* kv_cache;
  const void* pe_cache;
  int64_t kv_row_stride, pe_row_stride;
  int64_t kv_batch_stride, pe_batch_stride;  /* contiguous layout only */
  int Lk;
  const int32_t* seq_lens;    /* (B) or NULL */
  const int32_t* block_table; /* (B,max_pages) or NULL */
  int max_pages, page_size, num_pages;
  const uint8_t* causal_mask; /* (prefix_len + Lk) or NULL */
  int causal;
  float softmax_scale;
  const float* sinks;         /* (H) or NULL */
  int num_splits;             /* 0 = auto */
  void* x;
  float* lse;                 /* or NULL */
  int32_t* err_flag;          /* optional device status word */
} mla_prefix_args;

int mla_prefix_decode_num_splits(const mla_prefix_args* a);
size_t mla_prefix_decode_workspace_size(const mla_prefix_args* a);
mla_status_t mla_prefix_decode(const mla_prefix_args* a, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * mla_fp4_linear - products of few tokens with weights held in the cache's FP4
 * entries (E2M1 codes, an E4M3 scale per 16 channels):
 *
 *   out[t, g*N + n] = scale * sum_k x_g[t, k] * W[g, n, k],   t = b*Q + q
 *
 *   w   (G, N, K/512) entries of 288 bytes, packed: entry i of a row holds
 *       channels 512 i .. 512 i + 511 in the layout mla_decode reads.
 *       mla_cache_append with rope_tail = 0 writes such rows.
 *   x   bf16; channel k of group g of token (b, q) at x + b*x_batch_stride +
 *       q*x_token_stride + g*x_group_stride + (k/512)*x_block_stride + k%512,
 *       strides in elements, multiples of 8 (x (B,H,Q,512) with H/G heads per
 *       group: strides H*Q*512, 512, (H/G)*Q*512, Q*512).
 *   out (B*Q, G*N) bf16, packed. Products and sums are float32, rounded once.
 *   K a multiple of 512; B*Q up to 2^20, G up to 65535, G*N up to 2^30. x and w
 *       16-byte aligned.
 *   workspace: mla_fp4_linear_workspace_size(a) bytes, 256-byte aligned (may
 *       be NULL when that is 0). It is written before it is read in every call;
 *       calls whose GPU work overlaps in time need one each.
 *   err_flag: optional device int32; MLA_DEVICE_ERR_TIMEOUT when a bounded wait
 *       inside the kernel gave up (the output is then not valid).
 */
typedef struct mla_fp4_linear_args {
  int B, Q, G, N, K;
  const void* x;
  int64_t x_batch_stride, x_token_stride, x_group_stride, x_block_stride;
  const void* w;
  float scale;
  void* out;
  int32_t* err_flag;       /* optional device status word */
} mla_fp4_linear_args;

size_t mla_fp4_linear_workspace_size(const mla_fp4_linear_args* a);
mla_status_t mla_fp4_linear(const mla_fp4_linear_args* a, void* workspace, size_t workspace_bytes,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LATENT_KV_DECODE_MLA_H */
