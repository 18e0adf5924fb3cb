// torch_calls.cpp -- the layer operators (norm, rotary positions, cache,
// attention) called on torch tensors, as the extension module _torch_calls.
//
// These calls are a few microseconds of GPU work in a decoding step, and their
// host side is what a step waits for: checking nine tensors, allocating the
// results and marshalling thirty arguments takes 12 to 17 us through Python and
// ctypes, and 2 to 4 us here (B200 machine).  The functions take every argument by
// position (the Python functions of the package give them names and defaults),
// check what the C ABI cannot see -- devices, types, shapes, strides --, allocate
// what the caller did not bring, and call the C ABI of libbq on the tensors'
// device and its current stream.  They return the result, or the bq_status as an
// int where the library refused the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "bq.h"

namespace {

struct Bad {                    // a ValueError or TypeError with this text
  std::string text;
  bool type = false;
};

std::string text_of(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad{std::string(name) + " must be a torch.Tensor", true};
  return THPVariable_Unpack(o);
}

// A tensor on a CUDA device, whose index is returned.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda())
    throw Bad{std::string(name) + " must be on a CUDA device (libbq has no CPU path)"};
  return t.get_device();
}

[[noreturn]] void wrong(const at::Tensor& t, const char* name, at::ScalarType type,
                        at::IntArrayRef shape, int dev) {
  if (device_of(t, name) != dev)
    throw Bad{std::string(name) + " must be on cuda:" + std::to_string(dev) + ", not " +
              t.device().str()};
  throw Bad{std::string(name) + " must be " + at::toString(type) + " " + text_of(shape) +
            ", with dense rows that do not overlap, not " + at::toString(t.scalar_type()) + " " +
            text_of(t.sizes()) + " with strides " + text_of(t.strides())};
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
           int dev) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape)
    wrong(t, name, type, shape, dev);
}

// Row stride of a [M, K] tensor with unit column stride.
int64_t rows(const at::Tensor& t, const char* name, at::ScalarType type, int64_t M, int64_t K,
             int dev) {
  check(t, name, type, {M, K}, dev);
  const int64_t ld = t.stride(0);
  if ((K > 1 && t.stride(1) != 1) || (M > 1 && ld < K)) wrong(t, name, type, {M, K}, dev);
  return ld > K ? ld : K;
}

void* dense(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
            int dev) {
  check(t, name, type, shape, dev);
  if (!t.is_contiguous()) wrong(t, name, type, shape, dev);
  return t.data_ptr();
}

struct Heads {
  void* p;
  int64_t token, head;
};

// A bf16 [T, H, D] tensor with unit last stride.
Heads heads(const at::Tensor& t, const char* name, int64_t T, int64_t H, int64_t D, int dev) {
  check(t, name, at::kBFloat16, {T, H, D}, dev);
  if (D > 1 && t.stride(2) != 1) wrong(t, name, at::kBFloat16, {T, H, D}, dev);
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad{std::string(name) + " must be a whole number within 64 bits", true};
  }
  return v;
}

// A number that a C int takes as it is, so that the library sees what was said.
int small(PyObject* o, const char* name) {
  const int64_t v = whole(o, name);
  if (v < -(1ll << 30) || v > (1ll << 30)) throw Bad{std::string(name) + " is out of range"};
  return (int)v;
}

double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad{std::string(name) + " must be a number", true};
  }
  return v;
}

// The truth of an argument; what Python raises on asking for it (a tensor of several
// elements) goes on to the caller.
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}

bool none(PyObject* o) { return o == Py_None; }

// The tensors' device as the current one while the library launches.
struct On {
  std::optional<c10::cuda::CUDAGuard> guard;
  void* stream;
  explicit On(int dev) {
    if (c10::cuda::current_device() != dev) guard.emplace((c10::DeviceIndex)dev);
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }
};

PyObject* status(bq_status st) { return PyLong_FromLong(st); }

PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts) {
  Py_ssize_t n = 0;
  for (auto t : ts) n += t->defined() ? 1 : 0;
  PyObject* out = PyTuple_New(n);
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (auto t : ts) {
    if (!t->defined()) continue;
    PyObject* o = THPVariable_Wrap(*t);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  HANDLE_TH_ERRORS
  try {
    if (got != want) throw Bad{"wrong number of arguments", true};
    return body();
  } catch (const Bad& e) {
    PyErr_SetString(e.type ? PyExc_TypeError : PyExc_ValueError, e.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, weight, eps, residual, group_k, dtype, weight_offset, want_h, q, s, res_out, h, mx (MXFP8:
// group_k and dtype unused) -> (q, s[, res_out][, h])
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int dev = device_of(x, "x");
    if (x.dim() != 2) throw Bad{"x must be bfloat16 [M, K]"};
    const int64_t M = x.size(0), K = x.size(1), group = whole(a[4], "group_k");
    const int dtype = small(a[5], "dtype");
    const bool mx = truth(a[12]);
    if (group < 1) throw Bad{"group_k must be >= 1"};
    const int64_t ldx = rows(x, "x", at::kBFloat16, M, K, dev);
    void* w = dense(tensor(a[1], "weight"), "weight", at::kBFloat16, {K}, dev);
    at::Tensor q, s, ro, h;
    int64_t ldq = K, ldr = K, ldro = K, ldh = K;
    const void* res = nullptr;
    if (none(a[8])) {
      q = fresh({M, K}, at::kByte, x);
    } else {
      q = tensor(a[8], "q");
      ldq = rows(q, "q", at::kByte, M, K, dev);
    }
    if (mx) {
      size_t bytes = 0;
      const bq_status st = bq_mx_scale_bytes(M, K, &bytes);
      if (st != BQ_OK) return status(st);
      if (none(a[9])) {
        s = fresh({(int64_t)bytes}, at::kByte, x);
      } else {
        s = tensor(a[9], "sf");
        if (!s.is_cuda() || s.get_device() != dev || s.scalar_type() != at::kByte ||
            !s.is_contiguous() || s.numel() < (int64_t)bytes)
          wrong(s, "sf", at::kByte, {(int64_t)bytes}, dev);
      }
    } else if (none(a[9])) {
      s = fresh({(K + group - 1) / group, M}, at::kFloat, x);
    } else {
      s = tensor(a[9], "s");
      dense(s, "s", at::kFloat, {(K + group - 1) / group, M}, dev);
    }
    if (!none(a[3])) {
      const at::Tensor& r = tensor(a[3], "residual");
      ldr = rows(r, "residual", at::kBFloat16, M, K, dev);
      res = r.data_ptr();
      if (none(a[10])) ro = fresh({M, K}, at::kBFloat16, x);
    }
    if (!none(a[10])) {
      ro = tensor(a[10], "res_out");
      ldro = rows(ro, "res_out", at::kBFloat16, M, K, dev);
    }
    if (!none(a[11])) {
      h = tensor(a[11], "h");
      ldh = rows(h, "h", at::kBFloat16, M, K, dev);
    } else if (truth(a[7])) {
      h = fresh({M, K}, at::kBFloat16, x);
    }
    const float eps = (float)real(a[2], "eps"), off = (float)real(a[6], "weight_offset");
    void* pro = ro.defined() ? ro.data_ptr() : nullptr;
    void* ph = h.defined() ? h.data_ptr() : nullptr;
    const On on(dev);
    const bq_status st =
        mx
            ? bq_mx_rmsnorm_quant(x.data_ptr(), ldx, res, ldr, w, off, eps, M, K, q.data_ptr(),
                                  ldq, s.data_ptr(), pro, ldro, ph, ldh, on.stream)
            : bq_rmsnorm_quant(x.data_ptr(), ldx, res, ldr, w, off, eps, M, K, group, dtype,
                               q.data_ptr(), ldq, static_cast<float*>(s.data_ptr()), pro, ldro,
                               ph, ldh, on.stream);
    return st == BQ_OK ? tuple_of({&q, &s, &ro, &h}) : status(st);
  });
}

// x, positions, freqs, layout, mscale, out -> out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int dev = device_of(x, "x");
    const at::Tensor& f = tensor(a[2], "freqs");
    if (x.dim() != 3 || f.dim() != 1)
      throw Bad{"x must be bfloat16 [T, H, D], freqs float64 [rot_dim / 2]"};
    const int64_t T = x.size(0), H = x.size(1), D = x.size(2), half = f.size(0);
    const Heads hx = heads(x, "x", T, H, D, dev);
    void* pos = dense(tensor(a[1], "positions"), "positions", at::kInt, {T}, dev);
    void* pf = dense(f, "freqs", at::kDouble, {half}, dev);
    at::Tensor out = none(a[5]) ? fresh({T, H, D}, at::kBFloat16, x) : tensor(a[5], "out");
    const Heads ho = heads(out, "out", T, H, D, dev);
    const On on(dev);
    const bq_status st =
        bq_rope(hx.p, hx.token, hx.head, static_cast<const int32_t*>(pos),
                static_cast<const double*>(pf), T, H, D, 2 * half, small(a[3], "layout"),
                (float)real(a[4], "mscale"), ho.p, ho.token, ho.head, on.stream);
    return st == BQ_OK ? THPVariable_Wrap(out) : status(st);
  });
}

struct Cache {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t n_pages, H, page, D, bt;
};

// k, v, ks, vs of a cache
Cache cache_of(PyObject* const* a, int dev) {
  const at::Tensor &k = tensor(a[0], "cache.k"), &v = tensor(a[1], "cache.v"),
                   &ks = tensor(a[2], "cache.ks"), &vs = tensor(a[3], "cache.vs");
  if (k.dim() != 4 || ks.dim() != 3)
    throw Bad{"cache codes must be uint8 [n_pages, Hkv, page_size, D], scales float32 "
              "[n_pages, Hkv, page_size / block_t]"};
  Cache c;
  c.n_pages = k.size(0); c.H = k.size(1); c.page = k.size(2); c.D = k.size(3);
  const int64_t blocks = ks.size(2);
  c.k = static_cast<uint8_t*>(dense(k, "cache.k", at::kByte, k.sizes(), dev));
  c.v = static_cast<uint8_t*>(dense(v, "cache.v", at::kByte, k.sizes(), dev));
  c.ks = static_cast<float*>(dense(ks, "cache.ks", at::kFloat, {c.n_pages, c.H, blocks}, dev));
  c.vs = static_cast<float*>(dense(vs, "cache.vs", at::kFloat, {c.n_pages, c.H, blocks}, dev));
  if (c.page < 1 || blocks < 1 || c.page % blocks != 0)
    throw Bad{"block_t must divide page_size"};
  c.bt = c.page / blocks;
  return c;
}

struct Batch {
  const int32_t *off, *lens, *table;
  int64_t ld, cols, B;
};

// seq_offsets, kv_lens, page_table
Batch batch_of(PyObject* const* a, int dev) {
  const at::Tensor &off = tensor(a[0], "seq_offsets"), &lens = tensor(a[1], "kv_lens"),
                   &table = tensor(a[2], "page_table");
  if (lens.dim() != 1 || table.dim() != 2)
    throw Bad{"kv_lens must be int32 [B], page_table int32 [B, pages]"};
  Batch b;
  b.B = lens.size(0);
  b.cols = table.size(1);
  b.lens = static_cast<int32_t*>(dense(lens, "kv_lens", at::kInt, {b.B}, dev));
  b.off = static_cast<int32_t*>(dense(off, "seq_offsets", at::kInt, {b.B + 1}, dev));
  b.ld = rows(table, "page_table", at::kInt, b.B, b.cols, dev);
  b.table = static_cast<int32_t*>(table.data_ptr());
  return b;
}

// cache k, v, ks, vs, dtype, k, v, seq_offsets, kv_lens, page_table -> None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[5], "k"), &v = tensor(a[6], "v");
    const int dev = device_of(k, "k");
    const Cache c = cache_of(a, dev);
    const Batch b = batch_of(a + 7, dev);
    const int64_t T = k.dim() ? k.size(0) : -1;
    const Heads hk = heads(k, "k", T, c.H, c.D, dev), hv = heads(v, "v", T, c.H, c.D, dev);
    const On on(dev);
    const bq_status st =
        bq_kv_append(hk.p, hk.token, hk.head, hv.p, hv.token, hv.head, b.off, b.lens, b.table,
                     b.ld, b.cols, b.B, T, c.H, c.D, c.n_pages, c.page, c.bt,
                     small(a[4], "dtype"), c.k, c.v, c.ks, c.vs, on.stream);
    if (st != BQ_OK) return status(st);
    Py_RETURN_NONE;
  });
}

// q, cache k, v, ks, vs, dtype, seq_offsets, kv_lens, page_table, max_q_len, max_kv_len,
// scale (or None), causal, window, out, lse, ws -> out
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const int dev = device_of(q, "q");
    const Cache c = cache_of(a + 1, dev);
    const Batch b = batch_of(a + 6, dev);
    if (q.dim() != 3) throw Bad{"q must be bfloat16 [T, Hq, D]"};
    const int64_t T = q.size(0), Hq = q.size(1);
    const Heads hq = heads(q, "q", T, Hq, c.D, dev);
    at::Tensor out = none(a[14]) ? fresh({T, Hq, c.D}, at::kBFloat16, q) : tensor(a[14], "out");
    const Heads ho = heads(out, "out", T, Hq, c.D, dev);
    float* lse = none(a[15]) ? nullptr
                             : static_cast<float*>(dense(tensor(a[15], "lse"), "lse", at::kFloat,
                                                         {T, Hq}, dev));
    const int64_t max_q = whole(a[9], "max_q_len"), max_kv = whole(a[10], "max_kv_len"),
                  window = whole(a[13], "window");
    const float scale = none(a[11]) ? (float)(1.0 / std::sqrt((double)c.D))
                                    : (float)real(a[11], "scale");
    const bool causal = truth(a[12]);
    size_t bytes = 0;
    bq_status st = bq_kv_attention_workspace_size(b.B, T, Hq, c.H, c.D, max_q, max_kv, c.page,
                                                  c.bt, &bytes);
    if (st != BQ_OK) return status(st);
    at::Tensor ws;
    if (!none(a[16])) {
      ws = tensor(a[16], "ws");
      if (!ws.is_cuda() || ws.get_device() != dev || !ws.is_contiguous())
        wrong(ws, "ws", at::kByte, {(int64_t)bytes}, dev);
      bytes = ws.numel() * ws.element_size();
    } else if (bytes) {
      ws = fresh({(int64_t)bytes}, at::kByte, q);
    }
    const On on(dev);
    st = bq_kv_attention(hq.p, hq.token, hq.head, b.off, b.lens, b.table, b.ld, b.cols, b.B, T, Hq,
                         c.H, c.D, max_q, max_kv, c.k, c.v, c.ks, c.vs, c.n_pages, c.page, c.bt,
                         small(a[5], "dtype"), scale, causal, window, ho.p,
                         ho.token, ho.head, lse, ws.defined() ? ws.data_ptr() : nullptr, bytes,
                         on.stream);
    return st == BQ_OK ? THPVariable_Wrap(out) : status(st);
  });
}

#define BQ_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), \
                    METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {BQ_FAST(rmsnorm), BQ_FAST(rope), BQ_FAST(kv_append),
                          BQ_FAST(kv_attention), {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_calls() {
  return PyModule_Create(&kModule);
}
