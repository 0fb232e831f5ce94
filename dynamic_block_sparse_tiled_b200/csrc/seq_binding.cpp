// seq_binding.cpp - the torch side of the operators over sequences of
// different lengths: checks tensors, allocates outputs and workspaces, fills
// the argument structs of include/blasst.h and calls the C ABI.
//
// Native because these calls are short on the GPU (4 to 30 us): the same work
// in Python through ctypes took 15 to 35 us a call, here it takes about 2.
// sequences.py holds the documented functions that call in here.
#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <initializer_list>
#include <optional>
#include <string>
#include <tuple>
#include <utility>

#include "../../include/blasst.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;
using Stream = std::optional<long long>;

namespace {

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

// Raises the package's error for a status that is not BLASST_OK.
void check(int rc, const char* name) {
  if (rc == BLASST_OK) return;
  py::module_::import("dynamic_block_sparse_tiled_b200").attr("_check")(rc, name);
}

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return BLASST_BF16;
    case at::kHalf: return BLASST_FP16;
    case at::kFloat: return BLASST_FP32;
    default: refuse(std::string("dtype ") + c10::toString(t.scalar_type()) + " is not supported");
  }
}

// The calls record nothing for autograd: a tensor whose gradient is asked for
// would lose it without a word. (Within an autograd function nothing is recorded.)
void no_gradient(const Tensor& t) {
  if (at::GradMode::is_enabled() && t.requires_grad())
    refuse(
        "a tensor requires a gradient, which this call does not record: call it under torch.no_grad() or in a "
        "torch.autograd.Function, with rotary_backward or attention_packed_backward for the gradients");
}

// The device of a call, its first tensor's (the rest is checked against it),
// and its stream, current while the call allocates.
class Call {
 public:
  Call(const Tensor& first, const Stream& given) {
    no_gradient(first);
    if (!first.is_cuda()) refuse("tensors passed to the CUDA library must live on a CUDA device");
    device_ = first.get_device();
    guard_.set_index(device_);
    const auto now = c10::cuda::getCurrentCUDAStream(device_);
    raw_ = now.stream();
    if (given && reinterpret_cast<cudaStream_t>(*given) != raw_) {
      raw_ = reinterpret_cast<cudaStream_t>(*given);
      caller_ = now.unwrap();
      given_ = c10::cuda::getStreamFromExternal(raw_, device_).unwrap();
      stream_guard_.reset_stream(*given_);
    }
  }
  // A float tensor of `dims` dimensions, contiguous in the last.
  const Tensor& rows(const Tensor& t, const char* name, int dims) const {
    here(t);
    if (t.dim() != dims) refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions");
    if (t.size(-1) > 1 && t.stride(-1) != 1)
      refuse(std::string(name) + " must be contiguous in its last dimension");
    return t;
  }
  // (on a stream of the caller's choice, a tensor that is freed behind the call
  // stays until the kernel has read it)
  void here(const Tensor& t) const {
    no_gradient(t);
    if (!t.is_cuda() || t.get_device() != device_) refuse("tensors must live on one CUDA device");
    if (given_) t.record_stream(*given_);
  }
  const int* index(const Tensor& t, const char* name, long long n) const {
    here(t);
    if (t.scalar_type() != at::kInt || t.dim() != 1 || !t.is_contiguous())
      refuse(std::string(name) + " must be a contiguous one-dimensional int32 tensor");
    if (t.size(0) != n) refuse(std::string(name) + " must have " + std::to_string(n) + " entries");
    return static_cast<const int*>(t.const_data_ptr());
  }
  // Sequences of a cu array.
  int sequences(const Tensor& cu, const char* name) const {
    if (cu.dim() != 1 || cu.size(0) < 1) refuse(std::string(name) + " must have one entry more than sequences");
    index(cu, name, cu.size(0));
    return static_cast<int>(cu.size(0) - 1);
  }
  const double* frequencies(const Tensor& f, int& rot) const {
    here(f);
    if (f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous())
      refuse("inv_freq must be a contiguous one-dimensional float64 tensor");
    rot = static_cast<int>(2 * f.size(0));
    return static_cast<const double*>(f.const_data_ptr());
  }
  void workspace(const Maybe& given, size_t bytes, const Tensor& like, void*& p, size_t& n) {
    Tensor w;
    if (given) {
      w = *given;
      here(w);
      if (!w.is_contiguous()) refuse("workspace must be contiguous");
    } else {
      w = made(at::empty({static_cast<long long>(bytes < 16 ? 16 : bytes)}, like.options().dtype(at::kByte)));
    }
    p = w.data_ptr();
    n = w.nbytes();
  }
  // A tensor allocated here, for the call's stream; the caller's own may use it too.
  Tensor made(Tensor t) {
    if (caller_) t.record_stream(*caller_);
    return t;
  }
  void* stream() const { return raw_; }

 private:
  c10::cuda::OptionalCUDAGuard guard_;
  c10::cuda::OptionalCUDAStreamGuard stream_guard_;
  std::optional<c10::Stream> caller_, given_;  // set if the call's stream is not the current one
  cudaStream_t raw_ = nullptr;
  c10::DeviceIndex device_ = 0;
};

int same_dtype(const Tensor& t, std::initializer_list<const Tensor*> others) {
  for (const Tensor* o : others)
    if (o->scalar_type() != t.scalar_type()) refuse("tensors must have one dtype");
  return dtype_of(t);
}

int narrow(int64_t n, const char* what) {
  if (n > 0x7fffffffll) refuse(std::string(what) + " is too large");
  return static_cast<int>(n);
}

// (token, head) strides; a dimension of one entry gets a stride that fits
// (torch allows any there).
void strides(const Tensor& t, long long& st, long long& sh) {
  sh = t.size(1) == 1 ? t.size(2) : t.stride(1);
  st = t.size(0) <= 1 ? std::max<long long>(sh * t.size(1), t.size(2)) : t.stride(0);
}

void page_strides(const Tensor& t, long long& sp, long long& st, long long& sh) {
  const long long d = t.size(3);
  sh = t.size(2) == 1 ? d : t.stride(2);
  st = t.size(1) == 1 ? d : t.stride(1);
  sp = t.size(0) == 1 ? t.size(1) * t.size(2) * d : t.stride(0);
}

template <typename Args>
void pages(const Call& c, Args& a, const Tensor& k, const Tensor& v, const Tensor& table,
           const Tensor& kv_lens, const Tensor& cu_q) {
  c.rows(k, "k_pages", 4);
  c.rows(v, "v_pages", 4);
  if (k.sizes() != v.sizes()) refuse("k_pages and v_pages must have one shape");
  c.here(table);
  if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("page_table must be a two-dimensional int32 tensor with contiguous rows");
  a.n_seq = c.sequences(cu_q, "cu_q");
  if (table.size(0) != a.n_seq) refuse("page_table must have " + std::to_string(a.n_seq) + " rows");
  a.cu_q = static_cast<const int*>(cu_q.const_data_ptr());
  a.kv_lens = c.index(kv_lens, "kv_lens", a.n_seq);
  a.page_table = static_cast<const int*>(table.const_data_ptr());
  a.table_width = narrow(table.size(1), "page_table");
  a.table_stride = table.size(0) > 1 ? table.stride(0) : table.size(1);
  a.n_pages = narrow(k.size(0), "k_pages");
  a.page_size = narrow(k.size(1), "k_pages");
  page_strides(k, a.kp_sp, a.kp_st, a.kp_sh);
  page_strides(v, a.vp_sp, a.vp_st, a.vp_sh);
}

Tensor rotary(const Tensor& x, const Tensor& inv_freq, const Maybe& positions, bool interleaved,
              double mscale, const Maybe& out, const Stream& stream, bool inverse) {
  Call c(x, stream);
  const bool packed = x.dim() == 3;
  c.rows(x, "x", packed ? 3 : 4);
  const Tensor y = out ? c.rows(*out, "out", static_cast<int>(x.dim()))
                       : c.made(at::empty(x.sizes(), x.options()));
  if (y.sizes() != x.sizes()) refuse("out must have the shape of x");
  blasst_rotary_args a{};
  a.dtype = same_dtype(x, {&y});
  a.x = x.const_data_ptr();
  a.y = y.data_ptr();
  a.B = packed ? 1 : narrow(x.size(0), "x");
  a.L = narrow(x.size(packed ? 0 : 2), "x");
  a.H = narrow(x.size(1), "x");
  a.d = narrow(x.size(-1), "x");
  a.x_sb = packed ? 0 : x.stride(0);
  a.y_sb = packed ? 0 : y.stride(0);
  a.x_sl = x.stride(packed ? 0 : 2);
  a.y_sl = y.stride(packed ? 0 : 2);
  a.x_sh = x.stride(1);
  a.y_sh = y.stride(1);
  if (positions) {
    const Tensor& p = *positions;
    c.here(p);
    if (p.scalar_type() != at::kInt && p.scalar_type() != at::kLong) refuse("positions must be int32 or int64");
    if (!(p.dim() == 1 && p.size(0) == a.L) && !(p.dim() == 2 && p.size(0) == a.B && p.size(1) == a.L))
      refuse("positions must be [tokens], or [batch, tokens]");
    if (a.L > 1 && p.stride(-1) != 1) refuse("positions must be contiguous in the last dimension");
    a.positions = p.const_data_ptr();
    a.pos64 = p.scalar_type() == at::kLong;
    a.pos_sb = p.dim() == 2 ? p.stride(0) : 0;
  }
  a.freq = c.frequencies(inv_freq, a.rot);
  a.interleaved = interleaved;
  a.inverse = inverse;
  a.scale = static_cast<float>(mscale);
  a.stream = c.stream();
  if (x.numel() > 0) check(blasst_rotary(&a), "blasst_rotary");
  return y;
}

Tensor paged_append(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& k_pages,
                    const Tensor& v_pages, const Tensor& table, const Tensor& kv_lens,
                    const Tensor& cu_q, const Maybe& inv_freq, bool interleaved, double mscale,
                    const Maybe& q_out, const Stream& stream) {
  Call c(q, stream);
  c.rows(q, "q", 3);
  c.rows(k, "k", 3);
  c.rows(v, "v", 3);
  blasst_append_args a{};
  pages(c, a, k_pages, v_pages, table, kv_lens, cu_q);
  a.T = narrow(q.size(0), "q");
  a.Hq = narrow(q.size(1), "q");
  a.d = narrow(q.size(2), "q");
  a.Hkv = narrow(k_pages.size(2), "k_pages");
  if (k.size(0) != a.T || k.size(1) != a.Hkv || k.size(2) != a.d || v.sizes() != k.sizes() ||
      k_pages.size(3) != a.d)
    refuse("k and v must be [T, Hkv, d], the pages [pages, page, Hkv, d]");
  const Tensor o = q_out ? c.rows(*q_out, "q_out", 3) : c.made(at::empty(q.sizes(), q.options()));
  if (o.sizes() != q.sizes() || o.scalar_type() != q.scalar_type()) refuse("q_out must have q's shape and dtype");
  a.dtype = same_dtype(q, {&k, &v, &k_pages, &v_pages});
  a.q = q.const_data_ptr();
  a.q_out = o.data_ptr();
  a.k = k.const_data_ptr();
  a.v = v.const_data_ptr();
  a.k_pages = k_pages.data_ptr();
  a.v_pages = v_pages.data_ptr();
  strides(q, a.q_st, a.q_sh);
  strides(o, a.qo_st, a.qo_sh);
  strides(k, a.k_st, a.k_sh);
  strides(v, a.v_st, a.v_sh);
  if (inv_freq) a.freq = c.frequencies(*inv_freq, a.rot);
  a.interleaved = interleaved;
  a.scale = static_cast<float>(mscale);
  a.stream = c.stream();
  if (a.T > 0) check(blasst_append(&a), "blasst_append");
  return o;
}

// What the packed calls share.
template <typename Args>
void packed(Call& c, Args& a, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_q,
            const Maybe& cu_k) {
  c.rows(q, "q", 3);
  c.rows(k, "k", 3);
  c.rows(v, "v", 3);
  a.Tq = narrow(q.size(0), "q");
  a.Hq = narrow(q.size(1), "q");
  a.d = narrow(q.size(2), "q");
  a.Tk = narrow(k.size(0), "k");
  a.Hkv = narrow(k.size(1), "k");
  if (k.size(2) != a.d || v.sizes() != k.sizes()) refuse("k and v must be [Tk, Hkv, d] with q's d");
  a.n_seq = c.sequences(cu_q, "cu_q");
  a.cu_q = static_cast<const int*>(cu_q.const_data_ptr());
  a.cu_k = cu_k ? c.index(*cu_k, "cu_k", a.n_seq + 1) : a.cu_q;
  a.q = q.const_data_ptr();
  a.k = k.const_data_ptr();
  a.v = v.const_data_ptr();
  strides(q, a.q_st, a.q_sh);
  strides(k, a.k_st, a.k_sh);
  strides(v, a.v_st, a.v_sh);
}

std::pair<Tensor, Tensor> attention_packed(const Tensor& q, const Tensor& k, const Tensor& v,
                                           const Tensor& cu_q, const Maybe& cu_k, bool causal,
                                           double scale, const Maybe& workspace, const Stream& stream) {
  Call c(q, stream);
  blasst_packed_args a{};
  packed(c, a, q, k, v, cu_q, cu_k);
  a.dtype = same_dtype(q, {&k, &v});
  Tensor o = c.made(at::empty({a.Tq, a.Hq, a.d}, q.options()));
  Tensor lse = c.made(at::empty({a.Tq, a.Hq}, q.options().dtype(at::kFloat)));
  a.o = o.data_ptr();
  a.lse = static_cast<float*>(lse.data_ptr());
  a.causal = causal;
  a.scale = static_cast<float>(scale);
  c.workspace(workspace, blasst_seq_workspace_bytes(a.d), q, a.workspace, a.workspace_bytes);
  a.stream = c.stream();
  if (a.Tq > 0) check(blasst_packed_fwd(&a), "blasst_packed_fwd");
  return {o, lse};
}

std::tuple<Tensor, Tensor, Tensor> attention_packed_backward(
    const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& lse,
    const Tensor& dout, const Tensor& cu_q, const Maybe& cu_k, bool causal, double scale,
    const Maybe& workspace, const Stream& stream) {
  Call c(q, stream);
  blasst_packed_bwd_args a{};
  packed(c, a, q, k, v, cu_q, cu_k);
  c.rows(o, "o", 3);
  c.rows(dout, "dout", 3);
  a.dtype = same_dtype(q, {&k, &v, &o, &dout});
  if (o.sizes() != q.sizes() || dout.sizes() != q.sizes()) refuse("o and dout must have q's shape");
  c.here(lse);
  if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != a.Tq || lse.size(1) != a.Hq ||
      !lse.is_contiguous())
    refuse("lse must be a contiguous float32 tensor [Tq, Hq]");
  Tensor dq = c.made(at::empty({a.Tq, a.Hq, a.d}, q.options()));
  Tensor dk = c.made(at::empty({a.Tk, a.Hkv, a.d}, q.options()));
  Tensor dv = c.made(at::empty({a.Tk, a.Hkv, a.d}, q.options()));
  a.o = o.const_data_ptr();
  a.dout = dout.const_data_ptr();
  a.lse = static_cast<const float*>(lse.const_data_ptr());
  a.dq = dq.data_ptr();
  a.dk = dk.data_ptr();
  a.dv = dv.data_ptr();
  strides(o, a.o_st, a.o_sh);
  strides(dout, a.do_st, a.do_sh);
  a.causal = causal;
  a.scale = static_cast<float>(scale);
  c.workspace(workspace, blasst_packed_bwd_workspace_bytes(a.Tq, a.Hq, a.Hkv), q, a.workspace,
              a.workspace_bytes);
  a.stream = c.stream();
  if (a.Tq > 0 || a.Tk > 0) check(blasst_packed_bwd(&a), "blasst_packed_bwd");
  return {dq, dk, dv};
}

std::pair<Tensor, Tensor> attention_paged(const Tensor& q, const Tensor& k_pages, const Tensor& v_pages,
                                          const Tensor& table, const Tensor& kv_lens,
                                          const Tensor& cu_q, bool causal, double scale,
                                          const Maybe& workspace, const Stream& stream) {
  Call c(q, stream);
  c.rows(q, "q", 3);
  blasst_paged_args a{};
  pages(c, a, k_pages, v_pages, table, kv_lens, cu_q);
  a.dtype = same_dtype(q, {&k_pages, &v_pages});
  a.Tq = narrow(q.size(0), "q");
  a.Hq = narrow(q.size(1), "q");
  a.d = narrow(q.size(2), "q");
  a.Hkv = narrow(k_pages.size(2), "k_pages");
  if (k_pages.size(3) != a.d) refuse("the pages must be [pages, page, Hkv, d] with q's d");
  Tensor o = c.made(at::empty({a.Tq, a.Hq, a.d}, q.options()));
  Tensor lse = c.made(at::empty({a.Tq, a.Hq}, q.options().dtype(at::kFloat)));
  a.q = q.const_data_ptr();
  a.k_pages = k_pages.const_data_ptr();
  a.v_pages = v_pages.const_data_ptr();
  a.o = o.data_ptr();
  a.lse = static_cast<float*>(lse.data_ptr());
  strides(q, a.q_st, a.q_sh);
  a.causal = causal;
  a.scale = static_cast<float>(scale);
  c.workspace(workspace, blasst_seq_workspace_bytes(a.d), q, a.workspace, a.workspace_bytes);
  a.stream = c.stream();
  if (a.Tq > 0) check(blasst_paged_fwd(&a), "blasst_paged_fwd");
  return {o, lse};
}

}  // namespace

PYBIND11_MODULE(_seq_binding, m) {
  m.def("rotary", &rotary);
  m.def("paged_append", &paged_append);
  m.def("attention_packed", &attention_packed);
  m.def("attention_packed_backward", &attention_packed_backward);
  m.def("attention_paged", &attention_paged);
}
