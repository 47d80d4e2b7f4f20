// state_space_binding.cpp -- packs torch tensors into the operand lists of the
// state space entry points of include/rk.h.
//
// A single token's kernel takes a few microseconds, so the host's time for a
// call is what such a step costs.  Checking and packing a dozen tensors in
// Python takes three times as long as the launch (20 to 26 us per call,
// measured); here it is done with torch's C++ tensors.  A Plan holds what one
// operator expects for one problem; run() checks, allocates what is wanted
// and calls the C entry.  Nothing of an operator's arithmetic is here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <vector>

namespace {

// One operand: where its entry starts in the operand list (in 8-byte words),
// and the tensor it has to be.
struct Entry {
  PyObject* name;
  int at;
  bool rows, required, output;
  at::ScalarType type;
  std::vector<int64_t> shape;
};

using Call = int32_t (*)(void*, const void*, const void*, void*);
using ScratchCall = int32_t (*)(void*, const void*, const void*, const void*, void*);
using NeededCall = int64_t (*)(const void*, const void*);

struct Plan {
  PyObject_HEAD
  std::vector<Entry>* entries;
  std::string* problem;
  void* encode;
  int64_t scratch;  // floats; -1: the entry takes no scratch
  void* needed;     // what a call's operands take of it, or null: all
};

constexpr int kMaxOperands = 21, kWords = 5 * kMaxOperands;
// The operand that run() takes by itself is a plan's first.

const Entry* find(const Plan* p, PyObject* name) {
  for (const Entry& e : *p->entries)
    if (e.name == name) return &e;
  for (const Entry& e : *p->entries)
    if (PyUnicode_Check(name) && PyUnicode_Compare(e.name, name) == 0) return &e;
  PyErr_SetObject(PyExc_KeyError, name);
  return nullptr;
}

// Distances in elements between the rows of t along its last but one
// dimension and its first (0 in a matrix), and the elements it spans.
// Dimensions of one row lie any distance apart.  False: not rows.
bool pitches(const at::Tensor& t, int64_t* pitch, int64_t* outer, int64_t* span) {
  const int64_t d = t.dim(), inner = t.size(d - 1);
  if (inner > 1 && t.stride(d - 1) != 1) return false;
  *pitch = t.size(d - 2) > 1 ? t.stride(d - 2) : inner;
  *outer = d == 3 && t.size(0) > 1 ? t.stride(0) : 0;
  if (*pitch < inner || (*outer < inner && d == 3 && t.size(0) > 1)) return false;
  *span = (t.size(d - 2) - 1) * *pitch + (t.size(0) - 1) * *outer + inner;
  return true;
}

// Checks a tensor and writes its entry.
bool pack(const Entry& e, PyObject* obj, c10::Device device, int64_t* words) {
  if (!THPVariable_Check(obj)) {
    PyErr_Format(PyExc_TypeError, "%U: expected a tensor, got %s", e.name, Py_TYPE(obj)->tp_name);
    return false;
  }
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (t.scalar_type() != e.type) {
    PyErr_Format(PyExc_TypeError, "%U: expected %s, got %s", e.name, c10::toString(e.type),
                 c10::toString(t.scalar_type()));
    return false;
  }
  if (t.device() != device || t.layout() != at::kStrided) {
    PyErr_Format(PyExc_ValueError, "%U: expected a dense tensor on %s, got one on %s", e.name, device.str().c_str(),
                 t.device().str().c_str());
    return false;
  }
  if (t.sizes() != at::IntArrayRef(e.shape)) {
    PyObject* shape = PyTuple_New((Py_ssize_t)e.shape.size());
    if (shape == nullptr) return false;
    for (size_t i = 0; i < e.shape.size(); ++i) PyTuple_SET_ITEM(shape, i, PyLong_FromLongLong(e.shape[i]));
    PyObject* got = PyObject_GetAttrString(obj, "shape");
    if (got != nullptr) PyErr_Format(PyExc_ValueError, "%U: expected shape %S, got %S", e.name, shape, got);
    Py_XDECREF(got);
    Py_DECREF(shape);
    return false;
  }
  int64_t* w = words + e.at;
  w[2] = t.numel();
  if (!t.is_contiguous()) {
    if (!e.rows) {
      PyErr_Format(PyExc_ValueError, "%U: must be contiguous", e.name);
      return false;
    }
    if (!pitches(t, &w[3], &w[4], &w[2])) {
      PyErr_Format(PyExc_ValueError, "%U: the last dimension must be dense and rows must not overlap", e.name);
      return false;
    }
  }
  w[0] = reinterpret_cast<int64_t>(t.data_ptr());
  return true;
}

// run(handle, X, want, tensors): the outputs as a dict, or the entry's error code.  X: the first operand.
PyObject* plan_run(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Plan* p = reinterpret_cast<Plan*>(self);
  if (n != 4 || !PyDict_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "run(handle, X, want, tensors)");
    return nullptr;
  }
  void* handle = PyLong_AsVoidPtr(args[0]);
  if (handle == nullptr) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "the layer is closed");
    return nullptr;
  }
  const Entry* const first = p->entries->data();
  if (!THPVariable_Check(args[1]) || !THPVariable_Unpack(args[1]).is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%U: expected a CUDA tensor", first->name);
    return nullptr;
  }
  const c10::Device device = THPVariable_Unpack(args[1]).device();
  c10::cuda::OptionalCUDAGuard guard;
  if (device.index() != c10::cuda::current_device()) guard.set_device(device);

  int64_t words[kWords] = {};
  const Entry* e = first;
  if (!pack(*e, args[1], device, words)) return nullptr;
  uint32_t seen = 1u << (e - p->entries->data());
  PyObject *key, *value;
  for (Py_ssize_t pos = 0; PyDict_Next(args[3], &pos, &key, &value);) {
    if ((e = find(p, key)) == nullptr) return nullptr;
    if (value == Py_None) continue;
    if (!pack(*e, value, device, words)) return nullptr;
    seen |= 1u << (e - p->entries->data());
  }
  for (const Entry& r : *p->entries) {
    if (r.required && !(seen >> (&r - p->entries->data()) & 1)) {
      PyErr_Format(PyExc_ValueError, "%U: required", r.name);
      return nullptr;
    }
  }

  THPObjectPtr out(PyDict_New());
  THPObjectPtr want(PySequence_Fast(args[2], "want: expected names"));
  if (!out || !want) return nullptr;
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(want.get()); ++i) {
    PyObject* name = PySequence_Fast_GET_ITEM(want.get(), i);
    if ((e = find(p, name)) == nullptr) return nullptr;
    PyObject* given = e == first ? args[1] : PyDict_GetItemWithError(args[3], name);
    if (given != nullptr && given != Py_None) {
      if (PyDict_SetItem(out, name, given) != 0) return nullptr;
      continue;
    }
    if (!e->output) {
      PyErr_Format(PyExc_ValueError, "%U: wanted, but an input of this operator that was not passed", e->name);
      return nullptr;
    }
    const at::Tensor t(at::detail::empty_cuda(e->shape, e->type, device, std::nullopt));
    words[e->at] = reinterpret_cast<int64_t>(t.data_ptr());
    words[e->at + 2] = t.numel();
    THPObjectPtr obj(THPVariable_Wrap(t));
    if (!obj || PyDict_SetItem(out, name, obj) != 0) return nullptr;
  }
  void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  int32_t st;
  if (p->scratch < 0) {
    st = reinterpret_cast<Call>(p->encode)(handle, p->problem->data(), words, stream);
  } else {
    // from torch's allocator: the stream's own memory, and a graph's where one is captured
    c10::DataPtr memory;
    int64_t work[3] = {};
    int64_t scratch = p->scratch;
    if (p->needed != nullptr) scratch = std::max<int64_t>(reinterpret_cast<NeededCall>(p->needed)(p->problem->data(), words), 0);
    if (scratch > 0) {
      memory = c10::cuda::CUDACachingAllocator::get()->allocate((size_t)scratch * sizeof(float));
      work[0] = reinterpret_cast<int64_t>(memory.get());
      work[2] = scratch;
    }
    st = reinterpret_cast<ScratchCall>(p->encode)(handle, p->problem->data(), words, work, stream);
  }
  return st != 0 ? PyLong_FromLong(st) : out.release();
  END_HANDLE_TH_ERRORS
}

// Plan(encode address, problem bytes, scratch floats or -1,
//      [(name, word, rows, required, output, type code, shape)][, address of
//      the scratch that operands need, or 0]); type codes: 0 float32, 1 Half,
//      2 bfloat16, 3 int32.
PyObject* plan_new(PyTypeObject* type, PyObject* args, PyObject*) {
  HANDLE_TH_ERRORS
  unsigned long long encode, needed = 0;
  const char* bytes;
  Py_ssize_t length;
  long long scratch;
  PyObject* list;
  if (!PyArg_ParseTuple(args, "Ky#LO!|K", &encode, &bytes, &length, &scratch, &PyList_Type, &list, &needed)) return nullptr;
  std::vector<Entry> entries;
  for (Py_ssize_t i = 0; i < PyList_GET_SIZE(list); ++i) {
    PyObject *name, *shape;
    int at, rows, required, output, code;
    if (!PyArg_ParseTuple(PyList_GET_ITEM(list, i), "UipppiO!", &name, &at, &rows, &required, &output, &code,
                          &PyTuple_Type, &shape))
      return nullptr;
    constexpr at::ScalarType kTypes[] = {at::kFloat, at::kHalf, at::kBFloat16, at::kInt};
    if (i >= kMaxOperands || at < 0 || at + (rows ? 5 : 3) > kWords || code < 0 || code > 3) {
      PyErr_SetString(PyExc_ValueError, "Plan: entry out of range");
      return nullptr;
    }
    Entry e{name, at, rows != 0, required != 0, output != 0, kTypes[code], {}};
    for (Py_ssize_t d = 0; d < PyTuple_GET_SIZE(shape); ++d) {
      e.shape.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d)));
      if (PyErr_Occurred()) return nullptr;
    }
    entries.push_back(std::move(e));
  }
  if (entries.empty()) {
    PyErr_SetString(PyExc_ValueError, "Plan: no entries");
    return nullptr;
  }
  Plan* p = reinterpret_cast<Plan*>(type->tp_alloc(type, 0));
  if (p == nullptr) return nullptr;
  for (Entry& e : entries) {
    Py_INCREF(e.name);
    PyUnicode_InternInPlace(&e.name);
  }
  p->entries = new std::vector<Entry>(std::move(entries));
  p->problem = new std::string(bytes, (size_t)length);
  p->encode = reinterpret_cast<void*>(encode);
  p->scratch = scratch;
  p->needed = reinterpret_cast<void*>(needed);
  return reinterpret_cast<PyObject*>(p);
  END_HANDLE_TH_ERRORS
}

void plan_dealloc(PyObject* self) {
  Plan* p = reinterpret_cast<Plan*>(self);
  if (p->entries)
    for (Entry& e : *p->entries) Py_DECREF(e.name);
  delete p->entries;
  delete p->problem;
  Py_TYPE(self)->tp_free(self);
}

// row_pitches(t): (pitch, outer pitch, elements spanned), or None.
PyObject* row_pitches(PyObject*, PyObject* obj) {
  HANDLE_TH_ERRORS
  int64_t pitch, outer, span;
  if (!THPVariable_Check(obj) || THPVariable_Unpack(obj).dim() < 2) {
    PyErr_SetString(PyExc_TypeError, "row_pitches: expected a tensor of rows");
    return nullptr;
  }
  if (!pitches(THPVariable_Unpack(obj), &pitch, &outer, &span)) Py_RETURN_NONE;
  return Py_BuildValue("LLL", (long long)pitch, (long long)outer, (long long)span);
  END_HANDLE_TH_ERRORS
}

PyMethodDef plan_methods[] = {
    {"run", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan_run)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyTypeObject plan_type = {PyVarObject_HEAD_INIT(nullptr, 0)};
PyMethodDef methods[] = {{"row_pitches", row_pitches, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "state_space_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_state_space_binding() {
  plan_type.tp_name = "state_space_binding.Plan";
  plan_type.tp_basicsize = sizeof(Plan);
  plan_type.tp_flags = Py_TPFLAGS_DEFAULT;
  plan_type.tp_new = plan_new;
  plan_type.tp_dealloc = plan_dealloc;
  plan_type.tp_methods = plan_methods;
  if (PyType_Ready(&plan_type) < 0) return nullptr;
  PyObject* m = PyModule_Create(&module);
  if (m == nullptr) return nullptr;
  Py_INCREF(&plan_type);
  if (PyModule_AddObject(m, "Plan", reinterpret_cast<PyObject*>(&plan_type)) < 0) {
    Py_DECREF(&plan_type);
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
