// gdp_records.cpp -- CPython extension of the binding: the gdp_tensor records
// (include/gdp.h) of torch tensors, filled in C++.
//
// records(index, *tensors) checks that every tensor lies on the GPU `index` (-1:
// the host), and returns a tuple: per tensor the address of its record, None for
// None, and last the bytes object that holds the records, to be kept alive during
// the call that reads them; record_bytes is the size of a record.  From Python a
// record costs 0.6 us, a tenth of a call on few tokens; here ten of them cost 0.3 us.

#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstring>
#include <exception>
#include <string>

#include "gdp.h"

namespace {

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return GDP_F32;
    case at::kBFloat16: return GDP_BF16;
    case at::kHalf: return GDP_F16;
    case at::kInt: return GDP_I32;
    case at::kLong: return GDP_I64;
    default: return -1;
  }
}

// Fills r; returns false with a Python error set.
bool fill(gdp_tensor *r, const at::Tensor &t, long index) {
  std::memset(r, 0, sizeof *r);
  const long where = t.is_cuda() ? (long)t.get_device() : -1;
  if (where != index) {
    const std::string want = index < 0 ? "the host" : "cuda:" + std::to_string(index);
    PyErr_Format(PyExc_ValueError, "expected a tensor on %s, got one on %s", want.c_str(), t.device().str().c_str());
    return false;
  }
  if (t.is_neg()) {  // its memory holds the values with the other sign
    PyErr_SetString(PyExc_ValueError, "lazily negated view: call resolve_neg() first");
    return false;
  }
  r->dtype = type_code(t.scalar_type());
  if (r->dtype < 0) {
    PyErr_Format(PyExc_ValueError, "unsupported dtype %s", at::toString(t.scalar_type()));
    return false;
  }
  if (t.dim() > 4) {
    PyErr_SetString(PyExc_ValueError, "at most 4 dims");
    return false;
  }
  r->ndim = (int32_t)t.dim();
  for (int d = 0; d < r->ndim; ++d) {
    r->shape[d] = t.size(d);
    r->stride[d] = t.stride(d);
  }
  r->data = t.data_ptr();
  if (!r->data) r->data = (void *)16;  // an empty tensor is still "present": a non-null dummy address
  return true;
}

PyObject *records(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n < 1) {
    PyErr_SetString(PyExc_TypeError, "records(index, *tensors)");
    return nullptr;
  }
  const long index = PyLong_AsLong(args[0]);
  if (index == -1 && PyErr_Occurred()) return nullptr;
  PyObject *holder = PyBytes_FromStringAndSize(nullptr, (n - 1) * (Py_ssize_t)sizeof(gdp_tensor));
  if (!holder) return nullptr;
  PyObject *out = PyTuple_New(n);
  if (!out) {
    Py_DECREF(holder);
    return nullptr;
  }
  PyTuple_SET_ITEM(out, n - 1, holder);
  gdp_tensor *r = reinterpret_cast<gdp_tensor *>(PyBytes_AS_STRING(holder));
  try {
    for (Py_ssize_t i = 0; i + 1 < n; ++i, ++r) {
      PyObject *o = args[i + 1], *address = Py_None;
      if (o == Py_None) {
        Py_INCREF(address);
      } else {
        if (!THPVariable_Check(o)) {
          PyErr_Format(PyExc_TypeError, "expected a torch.Tensor or None, got %s", Py_TYPE(o)->tp_name);
          Py_DECREF(out);
          return nullptr;
        }
        address = fill(r, THPVariable_Unpack(o), index) ? PyLong_FromVoidPtr(r) : nullptr;
        if (!address) {
          Py_DECREF(out);
          return nullptr;
        }
      }
      PyTuple_SET_ITEM(out, i, address);
    }
  } catch (const std::exception &e) {  // a tensor without storage
    Py_DECREF(out);
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  return out;
}

PyMethodDef methods[] = {{"records", (PyCFunction)(void *)records, METH_FASTCALL, "gdp_tensor records of tensors"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_records", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

// "3.10" of "3.10.12 (main, ...)", "2.10.0" of "2.10.0+rocm7.0"
std::string python_of(const std::string &v) { return v.substr(0, v.find('.', v.find('.') + 1)); }
std::string torch_of(const std::string &v) { return v.substr(0, v.find('+')); }

}  // namespace

PyMODINIT_FUNC PyInit__records(void) {
  // the file's name does not say what it was built for
  if (python_of(Py_GetVersion()) != python_of(PY_VERSION)) {
    PyErr_Format(PyExc_ImportError, "built for Python %s", PY_VERSION);
    return nullptr;
  }
  PyObject *torch = PyImport_ImportModule("torch");
  PyObject *version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  const char *text = version ? PyUnicode_AsUTF8(version) : nullptr;
  const bool same = text && torch_of(text) == torch_of(TORCH_VERSION);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  if (!same) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ImportError, "built for torch %s", TORCH_VERSION);
    return nullptr;
  }
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddIntConstant(m, "record_bytes", (long)sizeof(gdp_tensor)) < 0) Py_CLEAR(m);
  return m;
}
