// Lists of torch tensors as tables of moe_param_t, for the calls over many tensors (moe_adamw_step,
// moe_grad_norm). Checks and addresses cost about 20 ns a tensor here and 700 in Python, which for a model
// of some hundred small tensors was several times the GPU's work.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <vector>

#include "moe.h"

namespace {

// Whether o is a contiguous tensor on the device; false, with no error set or with Python's, if not.
bool there(PyObject* o, long dev) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  // the device as the object itself has it: a subclass (other than Parameter) may answer otherwise
  long at = -1;
  if (THPVariable_CheckExact(o)) {
    at = t.get_device();
  } else {
    PyObject* d = PyObject_CallMethod(o, "get_device", nullptr);
    if (!d) return false;
    at = PyLong_AsLong(d);
    Py_DECREF(d);
    if (at == -1 && PyErr_Occurred()) return false;
  }
  return at == dev && t.layout() == at::kStrided && t.is_contiguous();
}

// The element type of a tensor as the kernels take it, or -1 with a ValueError set.
int element_type(PyObject* o, long dev, const char* where, const char* what) {
  if (there(o, dev)) {
    const auto st = THPVariable_Unpack(o).scalar_type();
    if (st == at::kFloat || st == at::kBFloat16) return st == at::kFloat ? MOE_F32 : MOE_BF16;
  }
  if (PyErr_Occurred()) return -1;
  PyErr_Format(PyExc_ValueError, "%s: %s must be a contiguous float32 or bfloat16 tensor on CUDA device %ld", where,
               what, dev);
  return -1;
}

void* address(PyObject* o) { return const_cast<void*>(THPVariable_Unpack(o).const_data_ptr()); }

// A sequence held for the length of a call.
struct Items {
  PyObject* seq;
  explicit Items(PyObject* o, const char* say) : seq(PySequence_Fast(o, say)) {}
  ~Items() { Py_XDECREF(seq); }
  Items(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// gradients(list, device) -> (table as bytes, entries): one for every tensor, None left out
PyObject* gradients(PyObject*, PyObject* args) {
  PyObject* list;
  long dev;
  if (!PyArg_ParseTuple(args, "Ol", &list, &dev)) return nullptr;
  Items items(list, "grad_norm: the gradients must be a sequence");
  if (!items.seq) return nullptr;
  std::vector<moe_param_t> tab;
  tab.reserve(items.size());
  for (Py_ssize_t i = 0; i < items.size(); ++i) {
    PyObject* o = items[i];
    if (o == Py_None) continue;
    const int dt = element_type(o, dev, "grad_norm", "every gradient");
    if (dt < 0) return nullptr;
    moe_param_t e = {};
    e.g = address(o);
    e.n = THPVariable_Unpack(o).numel();
    e.g_dtype = dt;
    tab.push_back(e);
  }
  return Py_BuildValue("(y#n)", reinterpret_cast<const char*>(tab.data()), Py_ssize_t(tab.size() * sizeof(moe_param_t)),
                       Py_ssize_t(tab.size()));
}

// Whether a tensor is what the table says: address (which implies the device), type, size, contiguous.
bool as_it_was(PyObject* o, const void* held, int type, int64_t n) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  return address(o) == held && t.scalar_type() == (type == MOE_BF16 ? at::kBFloat16 : at::kFloat) && t.numel() == n &&
         t.is_contiguous();
}

// Whether a gradient's elements are those of its parameter, one for one: the same shape (sides of 1 apart), or one of
// them flat.
bool same_order(const at::Tensor& g, const at::Tensor& p) {
  const auto a = g.sizes(), b = p.sizes();
  if (a == b || a.size() == 1 || b.size() == 1) return true;
  size_t i = 0, j = 0;
  for (;; ++i, ++j) {
    while (i < a.size() && a[i] == 1) ++i;
    while (j < b.size() && b[j] == 1) ++j;
    if (i == a.size() || j == b.size()) return i == a.size() && j == b.size();
    if (a[i] != b[j]) return false;
  }
}

// step(table's address, sizes' address, their length, gradients, parameters, copies, device) -> whether a parameter or
// copy is not what the table says (address, type, size). Writes g, n and g_dtype (no gradient: n = 0).
PyObject* step(PyObject*, PyObject* args) {
  unsigned long long table, sizes;
  PyObject *grads, *params, *copies;
  Py_ssize_t held;
  long dev;
  if (!PyArg_ParseTuple(args, "KKnOOOl", &table, &sizes, &held, &grads, &params, &copies, &dev)) return nullptr;
  Items g(grads, "AdamW.step: the gradients must be a sequence"), p(params, "parameters"), c(copies, "copies");
  if (!g.seq || !p.seq || !c.seq) return nullptr;
  if (g.size() != p.size()) {
    PyErr_Format(PyExc_ValueError, "AdamW.step: %zd gradients for %zd parameters", g.size(), p.size());
    return nullptr;
  }
  moe_param_t* tab = reinterpret_cast<moe_param_t*>(table);
  const int64_t* n = reinterpret_cast<const int64_t*>(sizes);
  if (p.size() != held || c.size() != held) return PyErr_Format(PyExc_ValueError, "AdamW.step: the lists of parameters or copies are not what they were");
  bool moved = false;
  for (Py_ssize_t i = 0; i < g.size(); ++i) {
    moe_param_t& e = tab[i];
    if (!as_it_was(p[i], e.p, e.p_dtype, n[i])) {
      if (element_type(p[i], dev, "AdamW.step", "every parameter") < 0) return nullptr;
      moved = true;
    }
    if (c[i] == Py_None) {
      moved |= e.copy != nullptr;
    } else if (!as_it_was(c[i], e.copy, MOE_BF16, n[i])) {
      if (element_type(c[i], dev, "AdamW.step", "every copy") < 0) return nullptr;
      moved = true;
    }
    if (g[i] == Py_None) {
      e.g = nullptr;
      e.n = 0;
      e.g_dtype = MOE_F32;
      continue;
    }
    const int dt = element_type(g[i], dev, "AdamW.step", "every gradient");
    if (dt < 0) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(g[i]);
    if (t.numel() != n[i]) {
      PyErr_Format(PyExc_ValueError, "AdamW.step: gradient %zd has %lld elements and its parameter %lld", i,
                   (long long)t.numel(), (long long)n[i]);
      return nullptr;
    }
    if (!same_order(t, THPVariable_Unpack(p[i]))) {
      std::ostringstream say;
      say << "AdamW.step: gradient " << i << " has shape " << t.sizes() << " and its parameter "
          << THPVariable_Unpack(p[i]).sizes();
      PyErr_SetString(PyExc_ValueError, say.str().c_str());
      return nullptr;
    }
    e.g = address(g[i]);
    e.n = n[i];
    e.g_dtype = dt;
  }
  return PyBool_FromLong(moved);
}

// state(device, elements, bits, m, v, m_scale, v_scale, clock): nothing, or a ValueError for what an optimiser of that
// many elements does not hold. They are attributes that a program may replace.
PyObject* state(PyObject*, PyObject* args) {
  long dev, bits;
  long long n;
  PyObject* t[5];
  if (!PyArg_ParseTuple(args, "lLlOOOOO", &dev, &n, &bits, t, t + 1, t + 2, t + 3, t + 4)) return nullptr;
  static const char* const name[5] = {"m", "v", "m_scale", "v_scale", "clock"};
  const bool codes = bits == 8;
  const at::ScalarType type[5] = {codes ? at::kChar : at::kFloat, codes ? at::kByte : at::kFloat, at::kFloat, at::kFloat,
                                  at::kDouble};
  const long long size[5] = {n, n, n / 256, n / 256, 3};
  for (int i = 0; i < 5; ++i) {
    if (!codes && (i == 2 || i == 3)) continue;
    if (there(t[i], dev) && THPVariable_Unpack(t[i]).scalar_type() == type[i] &&
        THPVariable_Unpack(t[i]).numel() == size[i])
      continue;
    if (!PyErr_Occurred())
      PyErr_Format(PyExc_ValueError, "AdamW: %s must be a contiguous %s tensor of %lld elements on CUDA device %ld",
                   name[i], c10::toString(type[i]), size[i], dev);
    return nullptr;
  }
  Py_RETURN_NONE;
}

// A contiguous tensor over a part of base's storage. (An allocation between two launches costs 3 to 6 us on the
// host, 1 us alone: small outputs of one call share one.)
at::Tensor part(const at::Tensor& base, int64_t offset, at::IntArrayRef sizes) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), base.dtype());
  impl->set_sizes_contiguous(sizes);
  impl->set_storage_offset(offset);
  return at::Tensor(std::move(impl));
}

PyObject* tuple_of(const std::vector<at::Tensor>& ts) {
  PyObject* out = PyTuple_New(Py_ssize_t(ts.size()));
  for (size_t i = 0; out && i < ts.size(); ++i) {
    PyObject* t = THPVariable_Wrap(ts[i]);
    if (!t) Py_CLEAR(out);
    else PyTuple_SET_ITEM(out, Py_ssize_t(i), t);
  }
  return out;
}

constexpr int64_t kShared = 1 << 20;  // bytes up to which outputs share a storage

// outputs(device, type, columns, rows, ..): tensors [rows, columns] (columns 0: [rows]) on the CUDA device, from the
// current stream's pool; type MOE_F32 or MOE_BF16
PyObject* outputs(PyObject*, PyObject* args) {
  long dev, type;
  long long cols, rows[4];
  const Py_ssize_t n = PyTuple_GET_SIZE(args) - 3;
  if (n < 1 || n > 4) return PyErr_Format(PyExc_TypeError, "outputs: device, type, columns and one to four rows");
  PyObject* head = PyTuple_GetSlice(args, 0, 3);
  const bool parsed = head && PyArg_ParseTuple(head, "llL", &dev, &type, &cols);
  Py_XDECREF(head);
  if (!parsed) return nullptr;
  const int64_t eb = type == MOE_BF16 ? 2 : 4, width = cols ? cols : 1, unit = 256 / eb;
  int64_t all = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    rows[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(args, i + 3));
    if (rows[i] == -1 && PyErr_Occurred()) return nullptr;
    all += (rows[i] * width + unit - 1) / unit * unit;
  }
  const auto options = at::TensorOptions()
                           .dtype(type == MOE_BF16 ? at::kBFloat16 : at::kFloat)
                           .device(at::Device(at::kCUDA, c10::DeviceIndex(dev)));
  const bool shared = n > 1 && all * eb <= kShared;
  at::Tensor base;
  if (shared) base = at::empty({all}, options);
  std::vector<at::Tensor> ts;
  int64_t at = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const int64_t two[2] = {rows[i], cols};
    const at::IntArrayRef sizes(two, cols ? 2 : 1);
    ts.push_back(shared ? part(base, at, sizes) : at::empty(sizes, options));
    at += (rows[i] * width + unit - 1) / unit * unit;
  }
  return tuple_of(ts);
}

// No C++ exception leaves the module: torch's own become what torch raises for them (no memory, no device); a tensor
// that cannot be read (one without storage throws) is the caller's ValueError.
PyObject* allocated(PyObject* self, PyObject* args) {
  HANDLE_TH_ERRORS
  return outputs(self, args);
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject*, PyObject*)>
PyObject* guarded(PyObject* self, PyObject* args) {
  try {
    return F(self, args);
  } catch (const std::bad_alloc&) {
    return PyErr_NoMemory();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a tensor of the list cannot be read");
  }
  return nullptr;
}

PyMethodDef methods[] = {{"gradients", guarded<gradients>, METH_VARARGS, nullptr},
                         {"step", guarded<step>, METH_VARARGS, nullptr},
                         {"state", guarded<state>, METH_VARARGS, nullptr},
                         {"outputs", allocated, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists() {
  PyObject* m = PyModule_Create(&module);
  if (m) PyModule_AddStringConstant(m, "built_for", BUILT_FOR);
  return m;
}
