// Python module _step: argument marshalling of mla_rope_append, mla_prefix_decode
// and mla_fp4_linear in C++. At a decode step's sizes these calls take the GPU a
// few microseconds, less than Python needs to read the sizes and strides of a
// dozen tensors (measured on B200's host: 20, 22 and 13 us a call through ctypes
// structs, 6, 9 and 5 here, 8 where the product takes two launches). It checks,
// allocates, fills the argument structs of
// include/mla.h and calls libmla.so on the caller's stream; ops.py holds the
// signatures and their documentation.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/Event.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <limits>
#include <memory>
#include <string>
#include <tuple>

#include "../../include/mla.h"

namespace py = pybind11;
using at::Tensor;
using c10::cuda::CUDAStream;
using OptTensor = std::optional<Tensor>;
using OptInt = std::optional<int64_t>;

namespace {

struct StepError : std::runtime_error {
  using std::runtime_error::runtime_error;
};

void need(bool ok, const char* what) {
  if (!ok) throw StepError(what);
}

void check_status(mla_status_t s, const char* what) {
  if (s == MLA_OK) return;
  std::string m = std::string(what) + " failed: " + mla_status_string(s);
  if (s == MLA_ERR_CUDA) m += " (cudaError " + std::to_string(mla_last_cuda_error()) + ")";
  throw StepError(m);
}

int to_int(int64_t v) {
  if (v < std::numeric_limits<int>::min() || v > std::numeric_limits<int>::max())
    throw StepError(std::to_string(v) + " is beyond 32 bits");
  return (int)v;
}

void same_device(const Tensor& first, std::initializer_list<const OptTensor*> others) {
  need(first.is_cuda(), "libmla takes CUDA tensors only");
  for (const OptTensor* t : others)
    if (*t) {
      need((*t)->is_cuda(), "libmla takes CUDA tensors only");
      need((*t)->get_device() == first.get_device(), "libmla takes CUDA tensors of one device");
    }
}

mla_dtype_t dtype_of(const Tensor& t) {
  const auto s = t.scalar_type();
  need(s == at::kFloat || s == at::kBFloat16, "libmla takes float32 and bfloat16 tensors");
  return s == at::kFloat ? MLA_F32 : MLA_BF16;
}

void* ptr(const OptTensor& t) { return t ? t->data_ptr() : nullptr; }

// Pointer of a contiguous int32 tensor, of n elements unless n < 0.
const int32_t* int32_ptr(const OptTensor& t, const char* name, int64_t n = -1) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || !t->is_contiguous()) throw StepError(std::string(name) + " must be contiguous int32");
  if (n >= 0 && t->numel() != n) throw StepError(std::string(name) + " must have " + std::to_string(n) + " elements");
  return static_cast<const int32_t*>(t->data_ptr());
}

// The device and stream of a call. Both are current while it lives, so that memory
// for the call comes from its stream's pool: a block of the caller's current stream
// may still be in use by work queued there, which the call's stream does not wait for.
struct Call {
  c10::cuda::CUDAGuard guard;
  CUDAStream current, stream;                    // the caller's, the call's
  std::optional<c10::cuda::CUDAStreamGuard> on;

  Call(const Tensor& t, OptInt handle)
      : guard(t.device()), current(c10::cuda::getCurrentCUDAStream(t.get_device())), stream(current) {
    if (handle && reinterpret_cast<cudaStream_t>(*handle) != current.stream()) {
      stream = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*handle), t.get_device());
      on.emplace(stream.unwrap());
    }
  }
  Call(const Call&) = delete;
  Call& operator=(const Call&) = delete;
  void* handle() const { return stream.stream(); }
  // The caller's tensors, which the call reads or writes on its stream.
  void used(std::initializer_list<const OptTensor*> ts) const {
    if (stream == current) return;
    for (const OptTensor* t : ts)
      if (*t) (*t)->record_stream(stream.unwrap());
  }
  // Tensors made here and handed out, which the caller goes on to use on its own stream.
  void made(std::initializer_list<const OptTensor*> ts) const {
    if (stream == current) return;
    for (const OptTensor* t : ts)
      if (*t) (*t)->record_stream(current.unwrap());
  }
};

// ---------------------------------------------------------------------------
// caches: (B, Lk, C) views, or (num_pages, page_size, C) pools with a table
// ---------------------------------------------------------------------------
template <typename Args>
void cache_fields(Args& a, const Tensor& kv, const OptTensor& pe, const OptTensor& table, int64_t page_size, OptInt Lk) {
  need(kv.dim() == 3 && kv.size(2) >= a.Ckv && kv.stride(2) == 1, "kv_cache must be 3-D with rows at least 512 wide, last dim packed");
  a.kv_cache = kv.data_ptr();
  a.kv_row_stride = kv.stride(1);
  a.kv_batch_stride = kv.stride(0);
  if (a.Dr > 0) {
    need(pe && pe->dim() == 3 && pe->size(0) == kv.size(0) && pe->size(1) == kv.size(1) && pe->size(2) >= a.Dr &&
             pe->stride(2) == 1,
         "pe_cache must hold kv_cache's rows, at least Dr wide, last dim packed");
    a.pe_cache = pe->data_ptr();
    a.pe_row_stride = pe->stride(1);
    a.pe_batch_stride = pe->stride(0);
  }
  if (!table) {
    need(kv.size(0) == a.B, "a contiguous cache must be (B, Lk, C)");
    need(!Lk || *Lk <= kv.size(1), "Lk is beyond the cache's rows");
    a.Lk = to_int(Lk ? *Lk : kv.size(1));
    return;
  }
  a.block_table = int32_ptr(table, "block_table");
  need(table->dim() == 2 && table->size(0) == a.B, "block_table must be (B, max_pages)");
  need(kv.size(1) == page_size, "the pool's pages must have page_size rows");
  need(kv.size(0) <= 1 || (kv.stride(0) == page_size * kv.stride(1) &&
                           (a.Dr == 0 || pe->stride(0) == page_size * pe->stride(1))),
       "a pool's pages must follow each other");
  a.max_pages = to_int(table->size(1));
  a.page_size = to_int(page_size);
  a.num_pages = to_int(kv.size(0));
  a.kv_batch_stride = a.pe_batch_stride = 0;
  a.Lk = to_int(Lk ? *Lk : table->size(1) * page_size);
}

// ---------------------------------------------------------------------------
// mla_rope_append
// ---------------------------------------------------------------------------
// Stride from token to token of (N, ...) or (B, Q, ...) rows with a packed last dim.
int64_t token_step(const Tensor& t, bool uniform) {
  need(t.stride(-1) == 1, "mla_rope_append: the last dim must be packed");
  if (!uniform || t.size(1) <= 1) return t.stride(0);
  need(t.size(0) <= 1 || t.stride(0) == t.size(1) * t.stride(1), "mla_rope_append: tokens must step evenly");
  return t.stride(1);
}

OptTensor rope_append(const Tensor& c_kv, const Tensor& k_pe, const Tensor& kv_cache, const Tensor& pe_cache,
                      const Tensor& seq_lens, const OptTensor& q_pe, const OptTensor& q_out_given,
                      const OptTensor& cu_tokens, const OptTensor& block_table, int64_t page_size, int64_t pos_offset,
                      double rope_theta, const OptTensor& err_flag, OptInt Lk, OptInt stream) {
  const OptTensor k_pe_o(k_pe), kv_o(kv_cache), pe_o(pe_cache), lens_o(seq_lens);
  same_device(c_kv, {&k_pe_o, &kv_o, &pe_o, &lens_o, &q_pe, &q_out_given, &cu_tokens, &block_table, &err_flag});
  const auto type = c_kv.scalar_type();
  need(k_pe.scalar_type() == type && kv_cache.scalar_type() == type && pe_cache.scalar_type() == type &&
           (!q_pe || q_pe->scalar_type() == type) && (!q_out_given || q_out_given->scalar_type() == type),
       "mla_rope_append: tensors must share one dtype");
  mla_rope_append_args a{};
  const bool uniform = !cu_tokens;
  const int lead = uniform ? 2 : 1;
  a.dtype = dtype_of(c_kv);
  a.B = to_int(seq_lens.numel());
  a.seq_lens = int32_ptr(lens_o, "seq_lens");
  a.cu_tokens = int32_ptr(cu_tokens, "cu_tokens", (int64_t)a.B + 1);
  need(c_kv.dim() == lead + 1 && k_pe.dim() == lead + 1 &&
           c_kv.sizes().slice(0, lead) == k_pe.sizes().slice(0, lead) && (!uniform || c_kv.size(0) == a.B),
       "mla_rope_append: c_kv and k_pe must be (B, Q, C), or (N, C) with cu_tokens");
  a.Ckv = to_int(c_kv.size(-1));
  a.Dr = to_int(k_pe.size(-1));
  a.Q = uniform ? to_int(c_kv.size(1)) : 0;
  a.N = to_int(uniform ? c_kv.size(0) * c_kv.size(1) : c_kv.size(0));
  a.c_kv = c_kv.data_ptr();
  a.k_pe = k_pe.data_ptr();
  a.c_kv_stride = token_step(c_kv, uniform);
  a.k_pe_stride = token_step(k_pe, uniform);
  OptTensor q_out = q_out_given;
  Call call(c_kv, stream);
  if (q_pe) {
    need(q_pe->dim() == lead + 2 && q_pe->sizes().slice(0, lead) == c_kv.sizes().slice(0, lead) &&
             q_pe->size(-1) == a.Dr,
         "mla_rope_append: q_pe must hold the tokens' heads, Dr wide");
    const int64_t H = q_pe->size(-2);
    a.H = to_int(H);
    const int64_t shape4[4] = {a.B, H, a.Q, a.Dr}, shape3[3] = {a.N, H, a.Dr};
    const at::IntArrayRef shape = uniform ? at::IntArrayRef(shape4, 4) : at::IntArrayRef(shape3, 3);
    if (!q_out) q_out = at::empty(shape, q_pe->options());
    need(q_out->sizes() == shape && q_out->stride(-1) == 1,
         "mla_rope_append: q_out must be (B, H, Q, Dr), or (N, H, Dr) with cu_tokens, last dim packed");
    a.q_pe = q_pe->data_ptr();
    a.q_out = q_out->data_ptr();
    a.q_token_stride = token_step(*q_pe, uniform);
    a.q_head_stride = q_pe->stride(-2);
    if (uniform) {
      a.o_batch_stride = q_out->stride(0);
      a.o_head_stride = q_out->stride(1);
      a.o_token_stride = q_out->stride(2);
    } else {
      a.o_token_stride = q_out->stride(0);
      a.o_head_stride = q_out->stride(1);
    }
  } else {
    need(!q_out, "mla_rope_append: q_out without q_pe");
  }
  cache_fields(a, kv_cache, pe_o, block_table, page_size, Lk);
  a.pos_offset = to_int(pos_offset);
  a.rope_theta = (float)rope_theta;
  a.err_flag = const_cast<int32_t*>(int32_ptr(err_flag, "err_flag"));
  check_status(mla_rope_append(&a, call.handle()), "mla_rope_append");
  const OptTensor c_kv_o(c_kv);
  call.used({&c_kv_o, &k_pe_o, &kv_o, &pe_o, &lens_o, &q_pe, &q_out_given, &cu_tokens, &block_table, &err_flag});
  if (!q_out_given) call.made({&q_out});
  return q_out;
}

// ---------------------------------------------------------------------------
// mla_prefix_decode
// ---------------------------------------------------------------------------
// A prepared call: its arguments, workspace and outputs, and the tensors its
// pointers refer to.
struct PrefixCall {
  mla_prefix_args a{};
  int num_splits = 0;
  size_t workspace_bytes = 0;
  OptTensor workspace, lse;
  Tensor x;
  std::vector<OptTensor> keep;
  // The stream it was prepared on and its place there: what was made for the call may
  // lie where work queued before that place is still busy. Not set while capturing.
  std::optional<CUDAStream> home;
  std::unique_ptr<c10::Event> ready;
};

PrefixCall prefix_make(const Tensor& q_lat, const OptTensor& q_pe, const OptTensor& prefix_kv,
                       const OptTensor& prefix_pe, const OptTensor& kv_cache, const OptTensor& pe_cache,
                       double softmax_scale, OptInt prefix_len, const OptTensor& prefix_table, const OptTensor& seq_lens,
                       const OptTensor& block_table, int64_t page_size, const OptTensor& causal_mask, bool causal,
                       const OptTensor& sinks, int64_t num_splits, const OptTensor& x, const OptTensor& lse,
                       bool want_lse, const OptTensor& workspace, const OptTensor& err_flag, OptInt Lk) {
  same_device(q_lat, {&q_pe, &prefix_kv, &prefix_pe, &kv_cache, &pe_cache, &prefix_table, &seq_lens, &block_table,
                      &causal_mask, &sinks, &x, &lse, &workspace, &err_flag});
  for (const OptTensor* t : {&q_pe, &prefix_kv, &prefix_pe, &kv_cache, &pe_cache, &x})
    need(!*t || (*t)->scalar_type() == q_lat.scalar_type(), "mla_prefix_decode: tensors must share one dtype");
  PrefixCall c;
  mla_prefix_args& a = c.a;
  need(q_lat.dim() == 4 && q_lat.is_contiguous(), "q_lat must be contiguous (B, H, Q, 512)");
  a.B = to_int(q_lat.size(0));
  a.H = to_int(q_lat.size(1));
  a.Q = to_int(q_lat.size(2));
  a.Ckv = to_int(q_lat.size(3));
  a.dtype = dtype_of(q_lat);
  a.q_lat = q_lat.data_ptr();
  if (q_pe) {
    need(q_pe->dim() == 4 && q_pe->is_contiguous() && q_pe->sizes().slice(0, 3) == q_lat.sizes().slice(0, 3),
         "q_pe must be contiguous (B, H, Q, Dr)");
    a.Dr = to_int(q_pe->size(3));
    a.q_pe = q_pe->data_ptr();
  }

  if (!prefix_kv) {
    need(!prefix_len || *prefix_len == 0, "prefix_len without prefix_kv");
  } else {
    const int dim = prefix_table ? 3 : 2;
    const Tensor& kv = *prefix_kv;
    need(kv.dim() == dim && kv.size(-1) >= a.Ckv && kv.stride(-1) == 1,
         "prefix_kv must be (rows, C), or (pages, page_size, C) with prefix_table, last dim packed");
    a.prefix_kv = kv.data_ptr();
    a.prefix_kv_stride = kv.stride(-2);
    if (a.Dr > 0) {
      need(prefix_pe && prefix_pe->dim() == dim && prefix_pe->sizes().slice(0, dim - 1) == kv.sizes().slice(0, dim - 1) &&
               prefix_pe->size(-1) >= a.Dr && prefix_pe->stride(-1) == 1,
           "prefix_pe must hold prefix_kv's rows, at least Dr wide, last dim packed");
      a.prefix_pe = prefix_pe->data_ptr();
      a.prefix_pe_stride = prefix_pe->stride(-2);
    }
    if (prefix_table) {
      a.prefix_table = int32_ptr(prefix_table, "prefix_table");
      need(prefix_len && kv.size(1) == page_size && *prefix_len <= prefix_table->numel() * page_size,
           "a paged prefix needs prefix_len, pages of page_size rows, and a table that covers it");
      need(kv.size(0) <= 1 || (kv.stride(0) == page_size * kv.stride(1) &&
                               (a.Dr == 0 || prefix_pe->stride(0) == page_size * prefix_pe->stride(1))),
           "a pool's pages must follow each other");
      a.prefix_num_pages = to_int(kv.size(0));
    } else {
      need(!prefix_len || *prefix_len <= kv.size(0), "prefix_len is beyond prefix_kv's rows");
    }
    a.prefix_len = to_int(prefix_len ? *prefix_len : kv.size(0));
  }
  a.page_size = to_int(page_size);
  if (kv_cache)
    cache_fields(a, *kv_cache, pe_cache, block_table, page_size, Lk);
  else
    need(!Lk || *Lk == 0, "Lk without kv_cache");
  a.seq_lens = int32_ptr(seq_lens, "seq_lens", a.B);
  if (causal_mask) {
    need((causal_mask->scalar_type() == at::kByte || causal_mask->scalar_type() == at::kBool) && causal_mask->is_contiguous(),
         "causal_mask must be contiguous uint8 or bool");
    need(causal_mask->numel() >= (int64_t)a.prefix_len + a.Lk, "causal_mask must cover prefix_len + Lk positions");
    a.causal_mask = static_cast<const uint8_t*>(causal_mask->data_ptr());
  }
  a.causal = causal;
  a.softmax_scale = (float)softmax_scale;
  a.num_splits = to_int(num_splits);
  if (sinks) {
    need(sinks->scalar_type() == at::kFloat && sinks->is_contiguous() && sinks->numel() == a.H, "sinks must be (H) float32");
    a.sinks = static_cast<const float*>(sinks->data_ptr());
  }
  need(!x || (x->is_contiguous() && x->sizes() == q_lat.sizes()), "x must be contiguous (B, H, Q, 512)");
  need(!lse || (lse->scalar_type() == at::kFloat && lse->is_contiguous() && lse->numel() == (int64_t)a.B * a.H * a.Q),
       "lse must be contiguous float32 (B, H, Q)");
  a.err_flag = const_cast<int32_t*>(int32_ptr(err_flag, "err_flag"));

  const c10::cuda::CUDAGuard guard(q_lat.device());   // the split rule reads the current device
  c.x = x ? *x : at::empty_like(q_lat);
  c.lse = lse;
  if (!lse && want_lse) c.lse = at::empty({a.B, a.H, a.Q}, q_lat.options().dtype(at::kFloat));
  a.x = c.x.data_ptr();
  a.lse = static_cast<float*>(ptr(c.lse));
  c.num_splits = mla_prefix_decode_num_splits(&a);
  need(c.num_splits >= 1, "mla_prefix_decode arguments rejected (MLA_ERR_INVALID_ARG or MLA_ERR_UNSUPPORTED)");
  c.workspace_bytes = mla_prefix_decode_workspace_size(&a);
  if (c.workspace_bytes > 0) {
    if (workspace)
      need(workspace->is_contiguous() && workspace->nbytes() >= c.workspace_bytes,
           "mla_prefix_decode: the workspace must be contiguous and hold workspace_bytes");
    c.workspace = workspace ? *workspace : at::empty({(int64_t)c.workspace_bytes}, q_lat.options().dtype(at::kByte));
  }
  c.keep = {q_lat, q_pe, prefix_kv, prefix_pe, kv_cache, pe_cache, prefix_table, seq_lens, block_table, causal_mask, sinks, err_flag};
  return c;
}

bool capturing() { return c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None; }

PrefixCall prefix_prepare(const Tensor& q_lat, const OptTensor& q_pe, const OptTensor& prefix_kv,
                          const OptTensor& prefix_pe, const OptTensor& kv_cache, const OptTensor& pe_cache,
                          double softmax_scale, OptInt prefix_len, const OptTensor& prefix_table,
                          const OptTensor& seq_lens, const OptTensor& block_table, int64_t page_size,
                          const OptTensor& causal_mask, bool causal, const OptTensor& sinks, int64_t num_splits,
                          const OptTensor& x, const OptTensor& lse, bool want_lse, const OptTensor& workspace,
                          const OptTensor& err_flag, OptInt Lk) {
  PrefixCall c = prefix_make(q_lat, q_pe, prefix_kv, prefix_pe, kv_cache, pe_cache, softmax_scale, prefix_len,
                             prefix_table, seq_lens, block_table, page_size, causal_mask, causal, sinks, num_splits, x,
                             lse, want_lse, workspace, err_flag, Lk);
  const c10::cuda::CUDAGuard guard(q_lat.device());
  c.home = c10::cuda::getCurrentCUDAStream();
  if (!capturing()) {
    c.ready = std::make_unique<c10::Event>(c10::DeviceType::CUDA);
    c.ready->record(c.home->unwrap());
  }
  return c;
}

void prefix_enqueue(PrefixCall& c, const Call& call) {
  check_status(mla_prefix_decode(&c.a, ptr(c.workspace), c.workspace_bytes, call.handle()), "mla_prefix_decode");
  for (const OptTensor& t : c.keep) call.used({&t});
}

std::tuple<Tensor, OptTensor> prefix_launch(PrefixCall& c, OptInt stream) {
  const Call call(c.x, stream);
  // a capture must not wait for work outside it; its replays are in the caller's order
  if (c.ready && call.stream != *c.home && !capturing()) c.ready->block(call.stream.unwrap());
  prefix_enqueue(c, call);
  const OptTensor x(c.x);
  for (const OptTensor* t : {&x, static_cast<const OptTensor*>(&c.lse), static_cast<const OptTensor*>(&c.workspace)})
    if (*t && call.stream != *c.home) (*t)->record_stream(call.stream.unwrap());
  return {c.x, c.lse};
}

std::tuple<Tensor, OptTensor> prefix_decode(const Tensor& q_lat, const OptTensor& q_pe, const OptTensor& prefix_kv,
                                            const OptTensor& prefix_pe, const OptTensor& kv_cache,
                                            const OptTensor& pe_cache, double softmax_scale, OptInt prefix_len,
                                            const OptTensor& prefix_table, const OptTensor& seq_lens,
                                            const OptTensor& block_table, int64_t page_size,
                                            const OptTensor& causal_mask, bool causal, const OptTensor& sinks,
                                            int64_t num_splits, const OptTensor& x, const OptTensor& lse, bool want_lse,
                                            const OptTensor& workspace, const OptTensor& err_flag, OptInt Lk,
                                            OptInt stream) {
  need(q_lat.is_cuda(), "libmla takes CUDA tensors only");
  const Call call(q_lat, stream);
  OptTensor mask = causal_mask;
  if (mask && mask->is_cuda() && mask->get_device() == q_lat.get_device() &&
      ((mask->scalar_type() != at::kByte && mask->scalar_type() != at::kBool) || !mask->is_contiguous()))
    mask = mask->ne(0).contiguous();   // on the call's stream, whose earlier work may still write the mask
  if (mask && !mask->is_same(*causal_mask)) call.used({&causal_mask});
  PrefixCall c = prefix_make(q_lat, q_pe, prefix_kv, prefix_pe, kv_cache, pe_cache, softmax_scale, prefix_len,
                             prefix_table, seq_lens, block_table, page_size, mask, causal, sinks, num_splits, x, lse,
                             want_lse, workspace, err_flag, Lk);
  prefix_enqueue(c, call);
  const OptTensor made_x(c.x);
  call.used({&x, &lse, &workspace});
  if (!x) call.made({&made_x});
  if (!lse) call.made({&c.lse});
  return {c.x, c.lse};
}

// ---------------------------------------------------------------------------
// mla_fp4_linear
// ---------------------------------------------------------------------------
constexpr int64_t kBlock = 512, kEntry = 288;

void fp4_launch(mla_fp4_linear_args& a, const Tensor& x, const Tensor& w, double scale, const Tensor& out,
                const OptTensor& err_flag, const Call& call) {
  need(w.scalar_type() == at::kByte && w.is_contiguous() && w.size(-1) == kEntry,
       "mla_fp4_linear weights are contiguous uint8 entries of 288 bytes");
  need(out.scalar_type() == at::kBFloat16 && out.is_contiguous(), "mla_fp4_linear: out must be contiguous bf16");
  if ((int64_t)a.B * a.Q == 0) return;             // no tokens
  a.x = x.data_ptr();
  a.w = w.data_ptr();
  a.scale = (float)scale;
  a.out = out.data_ptr();
  a.err_flag = const_cast<int32_t*>(int32_ptr(err_flag, "err_flag"));
  const size_t bytes = mla_fp4_linear_workspace_size(&a);
  OptTensor ws;
  if (bytes > 0) ws = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte));
  check_status(mla_fp4_linear(&a, ptr(ws), bytes, call.handle()), "mla_fp4_linear");
  const OptTensor xo(x), wo(w);
  call.used({&xo, &wo, &err_flag});
}

bool off16(const Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0; }

// A packed copy, made on the call's stream, which reads t.
Tensor packed(const Tensor& t, const Call& call) {
  const OptTensor o(t);
  call.used({&o});
  return t.clone(at::MemoryFormat::Contiguous);
}

Tensor linear_on(const Call& call, const Tensor& x, const Tensor& w, double scale, const OptTensor& out_given,
                 const OptTensor& err_flag) {
  const OptTensor wo(w);
  same_device(x, {&wo, &out_given, &err_flag});
  need(x.scalar_type() == at::kBFloat16, "mla_fp4_linear takes bf16 activations");
  need(x.dim() >= 1 && w.dim() == 3 && w.size(1) > 0 && x.size(-1) == w.size(1) * kBlock,
       "mla_fp4_linear: w must be (N, K/512, 288) for x (..., K)");
  const int64_t K = x.size(-1), N = w.size(0);
  std::vector<int64_t> shape = x.sizes().vec();
  shape.back() = N;
  Tensor rows = x;
  if (x.dim() != 2 || x.stride(1) != 1 || x.stride(0) % 8 != 0 || off16(x))
    rows = (x.is_contiguous() && !off16(x) ? x : packed(x, call)).view({-1, K});
  need(!out_given || out_given->sizes() == at::IntArrayRef(shape), "mla_fp4_linear: out has another shape");
  const Tensor out = out_given ? *out_given : at::empty(shape, x.options());
  mla_fp4_linear_args a{};
  a.B = to_int(rows.size(0));
  a.Q = a.G = 1;
  a.N = to_int(N);
  a.K = to_int(K);
  a.x_batch_stride = rows.stride(0);
  a.x_block_stride = kBlock;
  fp4_launch(a, rows, w, scale, out, err_flag, call);
  const OptTensor oo(out);
  out_given ? call.used({&oo}) : call.made({&oo});
  return out;
}

Tensor fp4_linear(const Tensor& x, const Tensor& w, double scale, const OptTensor& out, const OptTensor& err_flag,
                  OptInt stream) {
  need(x.is_cuda(), "libmla takes CUDA tensors only");
  return linear_on(Call(x, stream), x, w, scale, out, err_flag);
}

Tensor fp4_group_wo(const Tensor& x_given, const Tensor& wo_a, const OptTensor& wo_b, double scale_a, double scale_b,
                    const OptTensor& out, const OptTensor& err_flag, OptInt stream) {
  const OptTensor wa(wo_a);
  same_device(x_given, {&wa, &wo_b, &out, &err_flag});
  need(x_given.scalar_type() == at::kBFloat16, "mla_fp4_group_wo takes bf16 activations");
  need(x_given.dim() == 4 && x_given.size(3) == kBlock && wo_a.dim() == 4 && wo_a.size(0) * wo_a.size(2) == x_given.size(1),
       "mla_fp4_group_wo: x must be (B, H, Q, 512) and wo_a (G, R, H/G, 288)");
  const Call call(x_given, stream);
  Tensor x = x_given;
  if (x.stride(3) != 1 || x.stride(0) % 8 || x.stride(1) % 8 || x.stride(2) % 8 || off16(x)) x = packed(x, call);
  const int64_t B = x.size(0), Q = x.size(2), G = wo_a.size(0), R = wo_a.size(1), per = wo_a.size(2);
  const bool last = !wo_b;
  need(!last || !out || out->sizes() == at::IntArrayRef({B, Q, G * R}), "mla_fp4_group_wo: out has another shape");
  const Tensor z = last && out ? *out : at::empty({B, Q, G * R}, x.options());
  mla_fp4_linear_args a{};
  a.B = to_int(B);
  a.Q = to_int(Q);
  a.G = to_int(G);
  a.N = to_int(R);
  a.K = to_int(per * kBlock);
  a.x_batch_stride = x.stride(0);
  a.x_token_stride = x.stride(2);
  a.x_group_stride = per * x.stride(1);
  a.x_block_stride = x.stride(1);
  fp4_launch(a, x, wo_a, scale_a, z, err_flag, call);
  if (!last) return linear_on(call, z, *wo_b, scale_b, out, err_flag);
  const OptTensor zo(z);
  out ? call.used({&zo}) : call.made({&zo});
  return z;
}

}  // namespace

PYBIND11_MODULE(_step, m) {
  m.attr("built_for") = STEP_BUILT_FOR;          // the torch and Python it was compiled against
  // the package's own error class, set by ops.py when it loads the module
  static py::object* error = nullptr;
  m.def("set_error", [](py::object cls) {
    delete error;
    error = new py::object(std::move(cls));
  });
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const StepError& e) {
      PyErr_SetString(error ? error->ptr() : PyExc_RuntimeError, e.what());
    }
  });
  py::class_<PrefixCall>(m, "PrefixCall")
      .def_readonly("num_splits", &PrefixCall::num_splits)
      .def_readonly("workspace_bytes", &PrefixCall::workspace_bytes)
      .def_readonly("workspace", &PrefixCall::workspace)
      .def_readonly("x", &PrefixCall::x)
      .def_readonly("lse", &PrefixCall::lse);
  m.def("rope_append", &rope_append);
  m.def("prefix_make", &prefix_prepare);
  m.def("prefix_launch", &prefix_launch);
  m.def("prefix_decode", &prefix_decode);
  m.def("fp4_linear", &fp4_linear);
  m.def("fp4_group_wo", &fp4_group_wo);
}
