// qmm_bind.cpp -- Python entry of the key/value cache calls: checks the tensors,
// allocates what the caller does not give and calls the C ABI (include/qmm.h).
//
// These calls take a few microseconds on the GPU; through ctypes, checking and
// passing their 18 to 26 arguments took 8 to 15 us on the host. Nothing is
// computed here. Functions return what the Python functions of the same name
// return, or the library's status as an int where that is not QMM_OK; what is
// wrong with the tensors themselves is a ValueError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <string>

#include "../../include/qmm.h"

namespace {

struct Refused {
  std::string what;
};

[[noreturn]] void refuse(const char *fn, const std::string &what) { throw Refused{std::string(fn) + ": " + what}; }

const at::Tensor &tensor(const char *fn, const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) refuse(fn, std::string(name) + " is not a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(const char *fn, const char *name, PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(fn, std::string(name) + " is not an integer of 64 bits");
  }
  return v;
}

int small(const char *fn, const char *name, PyObject *o) {
  const int64_t v = integer(fn, name, o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(fn, std::string(name) + " is out of range");
  return static_cast<int>(v);
}

int element(const char *fn, const char *name, const at::Tensor &t) {
  if (t.scalar_type() == at::kFloat) return QMM_F32;
  if (t.scalar_type() == at::kBFloat16) return QMM_BF16;
  refuse(fn, std::string(name) + " is " + c10::toString(t.scalar_type()) + ", not float32 or bfloat16");
}

void on(const char *fn, const char *name, const at::Tensor &t, const at::Device &dev) {
  if (t.device() != dev) refuse(fn, std::string(name) + " is on " + t.device().str() + ", the cache on " + dev.str());
}

// A tensor of rows; the strides of its leading dims (0 where a dim is not stepped over: it is arbitrary there).
void rows(const char *fn, const char *name, const at::Tensor &t, int dims, const at::Device &dev, int64_t *strides) {
  if (t.layout() != at::kStrided || t.dim() != dims ||
      (t.stride(dims - 1) != 1 && t.size(dims - 1) != 1 && t.numel() != 0))
    refuse(fn, std::string(name) + " is not a tensor of " + std::to_string(dims) + " dims with contiguous rows");
  on(fn, name, t, dev);
  for (int i = 0; i + 1 < dims; ++i) strides[i] = t.size(i) > 1 && t.numel() != 0 ? t.stride(i) : 0;
}

void index(const char *fn, const char *name, const at::Tensor &t, at::ScalarType type, int64_t n, const at::Device &dev) {
  if (t.scalar_type() != type || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
    refuse(fn, std::string(name) + " is not a contiguous " + c10::toString(type) + " tensor of one dim" +
                   (n >= 0 ? " of " + std::to_string(n) : ""));
  on(fn, name, t, dev);
}

// Pages of a cache tensor, checked against its form; -1 with *st set where the library refuses the form.
int64_t cache_pages(const char *fn, const at::Tensor &cache, int ktype, int vtype, int64_t heads, int64_t dim, int block,
                    int64_t page, qmm_status *st) {
  if (cache.scalar_type() != at::kByte || cache.dim() != 2 || !cache.is_contiguous())
    refuse(fn, "cache is not a contiguous uint8 tensor [pages, page_bytes]");
  int64_t size = 0;
  *st = qmm_kv_page_bytes(ktype, vtype, heads, dim, block, page, &size);
  if (*st != QMM_OK) return -1;
  if (cache.size(1) != size)
    refuse(fn, "pages of " + std::to_string(cache.size(1)) + " bytes, this form has " + std::to_string(size));
  return cache.size(0);
}

// The library takes addresses: those of tensors that are not on a CUDA device are kept from it.
void on_cuda(const char *fn, const at::Device &dev) {
  if (!dev.is_cuda()) refuse(fn, "the cache is on " + dev.str() + ", not on a CUDA device");
}

qmm_stream_t stream_of(const at::Device &dev) {
  return reinterpret_cast<qmm_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

void count(const char *fn, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(fn, "takes " + std::to_string(want) + " arguments, " + std::to_string(n) + " given");
}

PyObject *status(qmm_status st) { return PyLong_FromLong(st); }

// write(cache, K, V, slots, page, ktype, vtype, block)
PyObject *write(PyObject *const *a, Py_ssize_t n) {
  const char *fn = "qmm_kv_write";
  count(fn, n, 8);
  const at::Tensor &cache = tensor(fn, "cache", a[0]), &K = tensor(fn, "K", a[1]), &V = tensor(fn, "V", a[2]),
                   &slots = tensor(fn, "slots", a[3]);
  const at::Device dev = cache.device();
  int64_t ks[2], vs[2];
  const int dtype = element(fn, "K", K);
  rows(fn, "K", K, 3, dev, ks);
  rows(fn, "V", V, 3, dev, vs);
  if (V.sizes() != K.sizes() || V.scalar_type() != K.scalar_type()) refuse(fn, "V is not of K's shape and type");
  index(fn, "slots", slots, at::kLong, K.size(0), dev);
  const int ktype = small(fn, "ktype", a[5]), vtype = small(fn, "vtype", a[6]), block = small(fn, "block", a[7]);
  const int64_t page = integer(fn, "page", a[4]);
  qmm_status st;
  const int64_t pages = cache_pages(fn, cache, ktype, vtype, K.size(1), K.size(2), block, page, &st);
  if (st != QMM_OK) return status(st);
  on_cuda(fn, dev);
  const c10::DeviceGuard guard(dev);
  st = qmm_kv_write(ktype, vtype, dtype, K.size(0), K.size(1), K.size(2), block, pages, page, K.data_ptr(), ks[0], ks[1],
                    V.data_ptr(), vs[0], vs[1], slots.data_ptr<int64_t>(), cache.data_ptr(), stream_of(dev));
  if (st != QMM_OK) return status(st);
  Py_INCREF(a[0]);
  return a[0];
}

// read(cache, slots, Hkv, D, K or None, V or None, bf16, page, ktype, vtype, block)
PyObject *read(PyObject *const *a, Py_ssize_t n) {
  const char *fn = "qmm_kv_read";
  count(fn, n, 11);
  const at::Tensor &cache = tensor(fn, "cache", a[0]), &slots = tensor(fn, "slots", a[1]);
  const at::Device dev = cache.device();
  index(fn, "slots", slots, at::kLong, -1, dev);
  const int64_t T = slots.size(0), heads = integer(fn, "Hkv", a[2]), dim = integer(fn, "D", a[3]);
  const int64_t page = integer(fn, "page", a[7]);
  const int ktype = small(fn, "ktype", a[8]), vtype = small(fn, "vtype", a[9]), block = small(fn, "block", a[10]);
  qmm_status st;
  const int64_t pages = cache_pages(fn, cache, ktype, vtype, heads, dim, block, page, &st);
  if (st != QMM_OK) return status(st);
  on_cuda(fn, dev);
  const c10::DeviceGuard guard(dev);
  at::Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    PyObject *o = a[4 + i];
    if (o == Py_None) {
      const at::ScalarType type = i ? out[0].scalar_type() : PyObject_IsTrue(a[6]) ? at::kBFloat16 : at::kFloat;
      out[i] = at::empty({T, heads, dim}, cache.options().dtype(type));
    } else {
      out[i] = tensor(fn, i ? "V" : "K", o);
      element(fn, i ? "V" : "K", out[i]);
      if (out[i].sizes() != at::IntArrayRef({T, heads, dim}) || !out[i].is_contiguous())
        refuse(fn, std::string(i ? "V" : "K") + " is not a contiguous tensor [tokens, Hkv, D]");
      on(fn, i ? "V" : "K", out[i], dev);
    }
  }
  if (out[0].scalar_type() != out[1].scalar_type()) refuse(fn, "K and V differ in type");
  st = qmm_kv_read(ktype, vtype, element(fn, "K", out[0]), T, heads, dim, block, pages, page, slots.data_ptr<int64_t>(),
                   cache.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), stream_of(dev));
  if (st != QMM_OK) return status(st);
  PyObject *pair = PyTuple_New(2);
  for (int i = 0; i < 2 && pair; ++i) {
    PyObject *o = a[4 + i];
    if (o == Py_None)
      o = THPVariable_Wrap(out[i]);
    else
      Py_INCREF(o);
    PyTuple_SET_ITEM(pair, i, o);
  }
  return pair;
}

// attn(Q, cache, table, lens, Hkv, Y or None, ws or None, page, ktype, vtype, scale or None, window, block)
PyObject *attn(PyObject *const *a, Py_ssize_t n) {
  const char *fn = "qmm_kv_attn";
  count(fn, n, 13);
  const at::Tensor &Q = tensor(fn, "Q", a[0]), &cache = tensor(fn, "cache", a[1]), &table = tensor(fn, "table", a[2]),
                   &lens = tensor(fn, "lens", a[3]);
  const at::Device dev = cache.device();
  int64_t qs[3];
  const int dtype = element(fn, "Q", Q);
  rows(fn, "Q", Q, 4, dev, qs);
  const int64_t B = Q.size(0), M = Q.size(1), Hq = Q.size(2), D = Q.size(3), heads = integer(fn, "Hkv", a[4]);
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B ||
      (table.size(1) > 1 && table.stride(1) != 1))
    refuse(fn, "table is not an int32 tensor of " + std::to_string(B) + " contiguous rows");
  on(fn, "table", table, dev);
  index(fn, "lens", lens, at::kInt, B, dev);
  const int64_t page = integer(fn, "page", a[7]), window = integer(fn, "window", a[11]);
  const int ktype = small(fn, "ktype", a[8]), vtype = small(fn, "vtype", a[9]), block = small(fn, "block", a[12]);
  qmm_status st;
  const int64_t pages = cache_pages(fn, cache, ktype, vtype, heads, D, block, page, &st);
  int64_t need = 0;
  if (st == QMM_OK) st = qmm_kv_attn_workspace(B, M, Hq, heads, D, &need);
  if (st != QMM_OK) return status(st);
  double scale = 1.0 / std::sqrt(static_cast<double>(D));
  if (a[10] != Py_None) {
    scale = PyFloat_AsDouble(a[10]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(fn, "scale is not a number");
    }
  }
  on_cuda(fn, dev);
  const c10::DeviceGuard guard(dev);
  at::Tensor Y, ws;
  if (a[5] == Py_None) {
    Y = at::empty(Q.sizes(), cache.options().dtype(Q.scalar_type()));
  } else {
    Y = tensor(fn, "Y", a[5]);
    if (Y.sizes() != Q.sizes() || Y.scalar_type() != Q.scalar_type() || !Y.is_contiguous())
      refuse(fn, "Y is not a contiguous tensor of Q's shape and type");
    on(fn, "Y", Y, dev);
  }
  if (a[6] == Py_None) {
    ws = at::empty({need}, cache.options());
  } else {
    ws = tensor(fn, "ws", a[6]);
    if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) refuse(fn, "ws is not a contiguous uint8 tensor");
    on(fn, "ws", ws, dev);
  }
  st = qmm_kv_attn(ktype, vtype, dtype, B, M, Hq, heads, D, block, pages, page, Q.data_ptr(), qs[0], qs[1], qs[2],
                   cache.data_ptr(), table.data_ptr<int32_t>(), B > 1 && table.numel() ? table.stride(0) : 0,
                   table.size(1), lens.data_ptr<int32_t>(), static_cast<float>(scale), window, Y.data_ptr(),
                   ws.data_ptr(), ws.numel(), stream_of(dev));
  if (st != QMM_OK) return status(st);
  if (a[5] == Py_None) return THPVariable_Wrap(Y);
  Py_INCREF(a[5]);
  return a[5];
}

// No C++ exception leaves the module.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (!PyErr_Occurred()) PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyMethodDef kMethods[] = {
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<write>)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<read>)), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<attn>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_qmm_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_bind(void) { return PyModule_Create(&kModule); }
