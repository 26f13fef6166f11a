// binding.cpp -- tensor binding of the masked-attention and training calls.
//
// Module _tensors: takes torch tensors, checks them, allocates outputs and calls
// the C ABI of include/h3.h.  The same in Python took 12 to 30 us per call, more
// than the shorter kernels themselves (the checks read some 60 tensor attributes);
// here it takes 1 to 2 us on top of the launches.  No arithmetic happens here.
// Arguments are positional; the Python functions of the package that call these
// carry the defaults and the documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/h3.h"

namespace {

PyObject* g_h3_error = nullptr;   // the package's H3Error(status, where)

struct Refused {                  // a wrong argument: ValueError or TypeError
  PyObject* type;
  std::string text;
};

[[noreturn]] void refuse(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

// One call's arguments, device and stream.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, const char* name) : args_(args), name_(name) {
    if (n != want) throw Refused{PyExc_TypeError, std::string(name) + ": wrong number of arguments"};
    dev_ = c10::cuda::current_device();
    PyObject* s = args[n - 1];    // a torch.cuda.Stream or None
    if (s == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream(dev_).stream();
    } else {
      auto attr = [&](const char* a) {
        PyObject* v = PyObject_GetAttrString(s, a);
        const long long x = v != nullptr ? PyLong_AsLongLong(v) : -1;
        Py_XDECREF(v);
        if (PyErr_Occurred()) {
          PyErr_Clear();
          throw Refused{PyExc_TypeError, "stream must be a torch.cuda.Stream"};
        }
        return x;
      };
      const auto st = c10::cuda::CUDAStream::unpack3(attr("stream_id"), static_cast<c10::DeviceIndex>(attr("device_index")),
                                                     static_cast<c10::DeviceType>(attr("device_type")));
      if (st.device_index() != dev_) refuse("stream must be one of the current CUDA device");
      guard_.emplace(st);         // outputs are allocated for that stream
      stream_ = st.stream();
    }
  }

  bool given(int i) const { return args_[i] != Py_None; }
  const at::Tensor& tensor(int i, const char* what) const {
    if (!THPVariable_Check(args_[i])) throw Refused{PyExc_TypeError, std::string(what) + " must be a tensor"};
    return THPVariable_Unpack(args_[i]);
  }
  int64_t integer(int i) const {
    const long long v = PyLong_AsLongLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) throw_pending();
    return v;
  }
  double number(int i) const {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw_pending();
    return v;
  }
  bool flag(int i) const {
    const int v = PyObject_IsTrue(args_[i]);
    if (v < 0) throw_pending();
    return v == 1;
  }

  int device() const { return dev_; }
  void* stream() const { return stream_; }

  void on_device(const at::Tensor& t, const char* what) const {
    if (!t.is_cuda() || t.get_device() != dev_) refuse(std::string(what) + " must be on the current CUDA device");
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    return at::Tensor(at::detail::empty_cuda(
        shape, dtype, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev_)), std::nullopt));
  }

  // Runs f (a call of the C ABI) without the interpreter lock and raises H3Error
  // unless it returns H3_OK.
  template <typename F>
  void run(F f) const {
    h3_status st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS if (st != H3_OK) {
      PyObject* e = PyObject_CallFunction(g_h3_error, "is", static_cast<int>(st), name_);
      if (e != nullptr) {
        PyErr_SetObject(g_h3_error, e);
        Py_DECREF(e);
      }
      throw_pending();
    }
  }

 private:
  [[noreturn]] static void throw_pending() {
    python_error e;
    e.persist();
    throw e;
  }
  PyObject* const* args_;
  const char* name_;
  int dev_;
  void* stream_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

// A [.., N, H, 128] bf16 view: rows of heads.
struct Heads {
  int64_t batch, rows, heads, stride;
  char* ptr;
  bool same(const Heads& o) const { return batch == o.batch && rows == o.rows && heads == o.heads; }
};

Heads heads_of(const Call& c, const at::Tensor& t, const char* what) {
  if (t.scalar_type() != at::kBFloat16) throw Refused{PyExc_TypeError, std::string(what) + " must be bf16"};
  if (!t.is_cuda()) throw Refused{PyExc_TypeError, std::string(what) + " must be a CUDA tensor"};
  c.on_device(t, what);
  const int64_t d = t.dim();
  if (d != 3 && d != 4) refuse(std::string(what) + " must be [N, H, 128] or [B, N, H, 128]");
  const auto size = t.sizes();
  const auto stride = t.strides();
  Heads h{d == 4 ? size[0] : 1, size[d - 3], size[d - 2], stride[d - 3], static_cast<char*>(t.data_ptr())};
  if (size[d - 1] != 128 || stride[d - 1] != 1 || (h.heads > 1 && stride[d - 2] != 128))
    refuse(std::string(what) + " must be [N, H, 128] or [B, N, H, 128] with heads contiguous");
  if (h.rows * h.batch <= 1) h.stride = 128 * h.heads;         // no second row
  else if (h.rows == 1) h.stride = stride[0];
  if (h.rows > 1 && h.batch > 1 && stride[0] != h.rows * h.stride)
    refuse(std::string(what) + ": the batch stride must be n_rows * row_stride");
  return h;
}

// Data pointer of a contiguous tensor of `numel` elements of `dtype`.
template <typename T = void>
T* plain(const Call& c, const at::Tensor& t, at::ScalarType dtype, int64_t numel, const char* what) {
  if (t.scalar_type() != dtype || t.numel() != numel || !t.is_contiguous())
    refuse(std::string(what) + " must be a contiguous " + c10::toString(dtype) + " tensor of " + std::to_string(numel) +
           " elements");
  c.on_device(t, what);
  return static_cast<T*>(t.data_ptr());
}

// Row stride of an [n, c] tensor with unit inner stride.
int64_t row_stride(const Call& call, const at::Tensor& t, int64_t n, int64_t c, at::ScalarType dtype, const char* what) {
  if (t.scalar_type() != dtype || t.dim() != 2 || t.size(0) != n || t.size(1) != c || (c > 1 && t.stride(1) != 1) ||
      (n > 1 && t.stride(0) < c))
    refuse(std::string(what) + " must be a " + c10::toString(dtype) + " [" + std::to_string(n) + ", " +
           std::to_string(c) + "] tensor with unit inner stride");
  call.on_device(t, what);
  return n > 1 ? t.stride(0) : c;
}

int32_t dtype_code(at::ScalarType t, const char* what) {
  if (t == at::kBFloat16) return H3_DTYPE_BF16;
  if (t == at::kHalf) return H3_DTYPE_F16;
  if (t == at::kFloat) return H3_DTYPE_F32;
  refuse(std::string(what) + " must be bf16, fp16 or fp32");
}

at::ScalarType dtype_of(int64_t code) {
  return code == H3_DTYPE_BF16 ? at::kBFloat16 : code == H3_DTYPE_F16 ? at::kHalf : at::kFloat;
}

int32_t as_int32(int64_t v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " is too large");
  return static_cast<int32_t>(v);
}

// The caller's workspace of at least `need` bytes, or a new one.
at::Tensor workspace(const Call& c, int i, uint64_t need) {
  if (!c.given(i)) return c.empty({static_cast<int64_t>(need)}, at::kByte);
  const at::Tensor& w = c.tensor(i, "workspace");
  if (w.scalar_type() != at::kByte || !w.is_contiguous() || static_cast<uint64_t>(w.numel()) < need)
    refuse("workspace must be a contiguous uint8 tensor of at least " + std::to_string(need) + " bytes");
  c.on_device(w, "workspace");
  return w;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* none() { Py_RETURN_NONE; }

PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// An output tensor that the caller gave (argument i), else a new one shaped as `like`.
at::Tensor given_or_like(const Call& c, int i, const at::Tensor& like, const char* what) {
  return c.given(i) ? c.tensor(i, what) : c.empty(like.sizes(), like.scalar_type());
}

// ------------------------------------------------------------- the calls ----

// q, k, coords, q_out, k_out, inverse, theta, sec_t, sec_h, sec_w, pair_layout, freq_rule, stream
PyObject* rotate(const Call& c) {
  h3_rope_cfg cfg{c.number(6), 128, as_int32(c.integer(7), "section"), as_int32(c.integer(8), "section"),
                  as_int32(c.integer(9), "section"), as_int32(c.integer(10), "pair_layout"),
                  as_int32(c.integer(11), "freq_rule")};
  Heads in[2] = {}, out[2] = {};
  at::Tensor outs[2];
  int64_t rows = -1, batch = 0;
  for (int i = 0; i < 2; ++i) {
    if (!c.given(i)) {
      if (c.given(3 + i)) refuse("an output without its input");
      continue;
    }
    const at::Tensor& x = c.tensor(i, "q and k");
    in[i] = heads_of(c, x, "q and k");
    if (rows >= 0 && (rows != in[i].rows || batch != in[i].batch)) refuse("q and k differ in their rows");
    rows = in[i].rows;
    batch = in[i].batch;
    outs[i] = given_or_like(c, 3 + i, x, "outputs");
    out[i] = heads_of(c, outs[i], "outputs");
    if (!out[i].same(in[i])) refuse("outputs must have the inputs' shape");
  }
  if (rows < 0) refuse("neither q nor k given");
  const int64_t n = rows * batch;
  const float* coords = plain<float>(c, c.tensor(2, "coords"), at::kFloat, 3 * n, "coords");
  const bool inverse = c.flag(5);
  c.run([&] {
    return h3_mmrope_rotate(in[0].ptr, in[1].ptr, out[0].ptr, out[1].ptr, coords, n, static_cast<int32_t>(in[0].heads),
                            static_cast<int32_t>(in[1].heads), in[0].stride, in[1].stride, out[0].stride, out[1].stride,
                            &cfg, inverse, c.stream());
  });
  return tuple({outs[0].defined() ? wrap(outs[0]) : none(), outs[1].defined() ? wrap(outs[1]) : none()});
}

// doc_starts, n_rows, mode, prefix, out, stream
PyObject* key_ranges(const Call& c) {
  const at::Tensor& starts = c.tensor(0, "doc_starts");
  if (starts.dim() != 1 || starts.numel() < 1) refuse("doc_starts must be a contiguous int32 [documents + 1] tensor");
  const int64_t docs = starts.numel() - 1, n = c.integer(1);
  if (n < 0) refuse("n_rows must not be negative");
  const int32_t* s = plain<int32_t>(c, starts, at::kInt, docs + 1, "doc_starts");
  const int32_t* p = c.given(3) ? plain<int32_t>(c, c.tensor(3, "prefix"), at::kInt, docs, "prefix") : nullptr;
  at::Tensor out = c.given(4) ? c.tensor(4, "out") : c.empty({n, 2}, at::kInt);
  int32_t* o = plain<int32_t>(c, out, at::kInt, 2 * n, "out");
  const int32_t mode = as_int32(c.integer(2), "mode"), n_docs = as_int32(docs, "documents");
  c.run([&] { return h3_build_key_ranges(s, p, n_docs, n, mode, o, c.stream()); });
  return wrap(out);
}

// The sizes that q, k, v and the intervals give.
struct Problem {
  Heads q, k, v;
  const int32_t* ranges;
  h3_attn_shape shape;
};

Problem problem_of(const Call& c, int iq, int iranges, double scale) {
  Problem p;
  p.q = heads_of(c, c.tensor(iq, "q"), "q");
  p.k = heads_of(c, c.tensor(iq + 1, "k"), "k");
  p.v = heads_of(c, c.tensor(iq + 2, "v"), "v");
  if (!p.v.same(p.k) || p.k.batch != p.q.batch) refuse("k and v must have one shape and q's batch");
  if (p.q.heads < 1 || p.k.heads < 1 || p.q.heads % p.k.heads != 0)
    refuse("the query heads must be a multiple of the K/V heads");
  const at::Tensor& r = c.tensor(iranges, "key_ranges");
  if (r.dim() < 2 || r.size(-1) != 2) refuse("key_ranges must be contiguous int32 [rows, 2]");
  p.ranges = plain<int32_t>(c, r, at::kInt, 2 * p.q.batch * p.q.rows, "key_ranges");
  p.shape = {p.q.rows,
             p.k.rows,
             as_int32(p.q.batch, "batch"),
             as_int32(p.q.heads, "heads"),
             as_int32(p.k.heads, "heads"),
             128,
             static_cast<float>(scale)};
  return p;
}

// q, k, v, key_ranges, out, lse, softmax_scale, stream
PyObject* attention(const Call& c) {
  const Problem p = problem_of(c, 0, 3, c.number(6));
  at::Tensor out = given_or_like(c, 4, c.tensor(0, "q"), "out");
  const Heads o = heads_of(c, out, "out");
  if (!o.same(p.q)) refuse("output must have q's shape");
  float* lse = c.given(5) ? plain<float>(c, c.tensor(5, "lse"), at::kFloat, p.q.batch * p.q.heads * p.q.rows, "lse")
                          : nullptr;
  c.run([&] {
    return h3_masked_attention(p.q.ptr, p.k.ptr, p.v.ptr, o.ptr, lse, p.ranges, &p.shape, p.q.stride, p.k.stride,
                               p.v.stride, o.stride, c.stream());
  });
  return wrap(out);
}

// dout, q, k, v, out, lse, key_ranges, dq, dk, dv, softmax_scale, workspace, stream
PyObject* attention_backward(const Call& c) {
  const Problem p = problem_of(c, 1, 6, c.number(10));
  auto like = [&](const at::Tensor& t, const Heads& want, const char* what) {
    const Heads h = heads_of(c, t, what);
    if (!h.same(want)) refuse(std::string(what) + " must be shaped as the tensor it belongs to");
    return h;
  };
  const Heads dout = like(c.tensor(0, "dout"), p.q, "dout"), o = like(c.tensor(4, "out"), p.q, "out");
  const at::Tensor dq = given_or_like(c, 7, c.tensor(1, "q"), "dq"), dk = given_or_like(c, 8, c.tensor(2, "k"), "dk");
  const at::Tensor dv = given_or_like(c, 9, c.tensor(3, "v"), "dv");
  const Heads hq = like(dq, p.q, "dq"), hk = like(dk, p.k, "dk"), hv = like(dv, p.k, "dv");
  const float* lse = plain<float>(c, c.tensor(5, "lse"), at::kFloat, p.q.batch * p.q.heads * p.q.rows, "lse");
  const at::Tensor work = workspace(c, 11, h3_masked_attention_backward_workspace_bytes(&p.shape));
  const h3_attn_strides strides{p.q.stride, p.k.stride, p.v.stride, o.stride, dout.stride, hq.stride, hk.stride, hv.stride};
  void* w = work.data_ptr();
  c.run([&] {
    return h3_masked_attention_backward(dout.ptr, p.q.ptr, p.k.ptr, p.v.ptr, o.ptr, lse, p.ranges, hq.ptr, hk.ptr,
                                        hv.ptr, w, &p.shape, &strides, c.stream());
  });
  return tuple({wrap(dq), wrap(dk), wrap(dv)});
}

// x, weight, bias, eps, out, mean, rstd, stream
PyObject* layer_norm(const Call& c) {
  const at::Tensor& x = c.tensor(0, "x");
  if (x.dim() != 2) refuse("x must be [N, C]");
  const int64_t n = x.size(0), ch = x.size(1);
  const auto dtype = x.scalar_type();
  const int32_t dt = dtype_code(dtype, "x"), hidden = as_int32(ch, "C");
  const int64_t xs = row_stride(c, x, n, ch, dtype, "x");
  int32_t pdt = dt;
  const void *w = nullptr, *b = nullptr;
  at::ScalarType ptype = dtype;
  if (c.given(1)) {
    const at::Tensor& t = c.tensor(1, "weight");
    ptype = t.scalar_type();
    w = plain(c, t, ptype, ch, "weight");
    pdt = dtype_code(ptype, "weight");
  }
  if (c.given(2)) {
    const at::Tensor& t = c.tensor(2, "bias");
    if (!c.given(1)) ptype = t.scalar_type();
    b = plain(c, t, ptype, ch, "bias");
    pdt = dtype_code(ptype, "bias");
  }
  const at::Tensor out = given_or_like(c, 4, x, "out");
  const int64_t ys = row_stride(c, out, n, ch, dtype, "out");
  const at::Tensor mean = c.given(5) ? c.tensor(5, "mean") : c.empty({n}, at::kFloat);
  const at::Tensor rstd = c.given(6) ? c.tensor(6, "rstd") : c.empty({n}, at::kFloat);
  float* m = plain<float>(c, mean, at::kFloat, n, "mean");
  float* r = plain<float>(c, rstd, at::kFloat, n, "rstd");
  const float eps = static_cast<float>(c.number(3));
  const void* px = x.data_ptr();
  void* py = out.data_ptr();
  c.run([&] { return h3_layernorm(px, py, w, b, m, r, n, hidden, xs, ys, dt, pdt, eps, c.stream()); });
  return tuple({wrap(out), wrap(mean), wrap(rstd)});
}

// dy, x, mean, rstd, weight, param_dtype (a code, without a weight), dx, workspace, param_grads, stream
PyObject* layer_norm_backward(const Call& c) {
  const at::Tensor &dy = c.tensor(0, "dy"), &x = c.tensor(1, "x");
  if (x.dim() != 2) refuse("x must be [N, C]");
  const int64_t n = x.size(0), ch = x.size(1);
  const auto dtype = x.scalar_type();
  const int32_t dt = dtype_code(dtype, "x"), hidden = as_int32(ch, "C");
  const int64_t xs = row_stride(c, x, n, ch, dtype, "x"), dys = row_stride(c, dy, n, ch, dtype, "dy");
  const float* m = plain<float>(c, c.tensor(2, "mean"), at::kFloat, n, "mean");
  const float* r = plain<float>(c, c.tensor(3, "rstd"), at::kFloat, n, "rstd");
  at::ScalarType ptype = dtype_of(c.integer(5));
  const void* w = nullptr;
  if (c.given(4)) {
    const at::Tensor& t = c.tensor(4, "weight");
    ptype = t.scalar_type();
    w = plain(c, t, ptype, ch, "weight");
  }
  const int32_t pdt = dtype_code(ptype, "weight");
  const at::Tensor dx = given_or_like(c, 6, x, "dx");
  const int64_t dxs = row_stride(c, dx, n, ch, dtype, "dx");
  at::Tensor dw, db, work;
  void *pw = nullptr, *pb = nullptr, *ws = nullptr;
  if (c.flag(8)) {
    dw = c.empty({ch}, ptype);
    db = c.empty({ch}, ptype);
    work = workspace(c, 7, h3_layernorm_backward_workspace_bytes(n, hidden));
    pw = dw.data_ptr();
    pb = db.data_ptr();
    ws = work.data_ptr();
  }
  const void *pdy = dy.data_ptr(), *px = x.data_ptr();
  void* pdx = dx.data_ptr();
  c.run([&] {
    return h3_layernorm_backward(pdy, px, m, r, w, pdx, pw, pb, ws, n, hidden, dys, xs, dxs, dt, pdt, c.stream());
  });
  return tuple({wrap(dx), dw.defined() ? wrap(dw) : none(), db.defined() ? wrap(db) : none()});
}

// dy, x, timestep_index, token_tag, table, eps, dx, dtable, workspace, stream
PyObject* adaln_backward(const Call& c) {
  const at::Tensor &dy = c.tensor(0, "dy"), &x = c.tensor(1, "x"), &table = c.tensor(4, "table");
  if (x.dim() != 2 || table.dim() != 3) refuse("x must be [N, C] and table [E, 2, C]");
  const int64_t n = x.size(0), ch = x.size(1), e = table.size(0);
  if (table.size(1) != 2 || table.size(2) != ch) refuse("table must be [E, 2, C]");
  const int64_t xs = row_stride(c, x, n, ch, at::kBFloat16, "x"), dys = row_stride(c, dy, n, ch, at::kBFloat16, "dy");
  const int32_t* ts = plain<int32_t>(c, c.tensor(2, "timestep_index"), at::kInt, n, "timestep_index");
  const int32_t* tags = plain<int32_t>(c, c.tensor(3, "token_tag"), at::kInt, n, "token_tag");
  const float* tab = plain<float>(c, table, at::kFloat, 2 * e * ch, "table");
  const int32_t hidden = as_int32(ch, "C"), entries = as_int32(e, "E");
  const uint64_t need = h3_adaln_backward_workspace_bytes(n, hidden, entries);
  if (need == 0) refuse("hidden must be a multiple of 8 up to 8192, with 1 to 8192 table entries");
  const at::Tensor dx = given_or_like(c, 6, x, "dx");
  const int64_t dxs = row_stride(c, dx, n, ch, at::kBFloat16, "dx");
  const at::Tensor dtable = c.given(7) ? c.tensor(7, "dtable") : c.empty({e, 2, ch}, at::kFloat);
  float* dt = plain<float>(c, dtable, at::kFloat, 2 * e * ch, "dtable");
  const at::Tensor work = workspace(c, 8, need);
  const float eps = static_cast<float>(c.number(5));
  const void *pdy = dy.data_ptr(), *px = x.data_ptr();
  void *pdx = dx.data_ptr(), *w = work.data_ptr();
  c.run([&] {
    return h3_adaln_modulate_backward(pdy, px, ts, tags, tab, pdx, dt, w, entries, n, hidden, dys, xs, dxs, eps,
                                      c.stream());
  });
  return tuple({wrap(dx), wrap(dtable)});
}

template <PyObject* (*F)(const Call&), int N>
PyObject* entry(PyObject* name, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(Call(args, n, N, PyUnicode_AsUTF8(name)));
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_h3_error);
  g_h3_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(const Call&), int N>
void add(PyObject* m, const char* method, const char* name) {
  // the C call's name travels as the function's self
  static PyMethodDef def;
  def = {method, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
  PyObject* self = PyUnicode_FromString(name);
  PyObject* f = PyCFunction_New(&def, self);
  Py_DECREF(self);
  PyModule_AddObject(m, method, f);
}

PyMethodDef g_methods[] = {{"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensors", "Tensor binding of libh3.", -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
  PyObject* m = PyModule_Create(&g_module);
  if (m == nullptr) return nullptr;
  add<rotate, 13>(m, "rotate", "h3_mmrope_rotate");
  add<key_ranges, 6>(m, "key_ranges", "h3_build_key_ranges");
  add<attention, 8>(m, "attention", "h3_masked_attention");
  add<attention_backward, 13>(m, "attention_backward", "h3_masked_attention_backward");
  add<layer_norm, 8>(m, "layer_norm", "h3_layernorm");
  add<layer_norm_backward, 10>(m, "layer_norm_backward", "h3_layernorm_backward");
  add<adaln_backward, 10>(m, "adaln_backward", "h3_adaln_modulate_backward");
  return m;
}
