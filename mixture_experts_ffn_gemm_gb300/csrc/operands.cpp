// operands.cpp -- the quick way from torch tensors to an entry point of the library: one call that compares each
// operand with its spec, collects the addresses and calls the C function.  The same comparisons in Python cost
// more than a small launch does (9 us a call against 4).  Anything but the plain, accepted case is left to
// binding.py, which takes or refuses it with its reasons; nothing is computed or kept here.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

namespace {

constexpr Py_ssize_t kMaxOperands = 8;

// What a call expects of an operand.  pitched: a [rows][width] tensor, rows `pitch` elements apart; else
// least..most consecutive elements.
struct Spec {
  int64_t type, least, most, pitched, rows, width, pitch;
};

bool plain(PyObject* o, const Spec& s, int64_t device, uint64_t* address) {
  if (o == Py_None) {
    *address = 0;
    return true;
  }
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.get_device() != device ||
      static_cast<int64_t>(t.scalar_type()) != s.type)
    return false;
  if (s.pitched) {
    if (t.dim() != 2 || t.size(0) != s.rows || t.size(1) != s.width) return false;
    if ((t.stride(1) != 1 && s.width > 1) || (t.stride(0) != s.pitch && s.rows > 1)) return false;
  } else {
    if (t.numel() < s.least || t.numel() > s.most || !t.is_contiguous()) return false;
  }
  *address = reinterpret_cast<uint64_t>(t.data_ptr());
  return true;
}

typedef uint64_t U;
int call_with(U fn, const void* c, Py_ssize_t n, const U* a, U ws, U bytes, U st) {
  switch (n) {
    case 4: return reinterpret_cast<int (*)(const void*, U, U, U, U, U, U, U)>(fn)(
        c, a[0], a[1], a[2], a[3], ws, bytes, st);
    case 5: return reinterpret_cast<int (*)(const void*, U, U, U, U, U, U, U, U)>(fn)(
        c, a[0], a[1], a[2], a[3], a[4], ws, bytes, st);
    case 6: return reinterpret_cast<int (*)(const void*, U, U, U, U, U, U, U, U, U)>(fn)(
        c, a[0], a[1], a[2], a[3], a[4], a[5], ws, bytes, st);
    case 8: return reinterpret_cast<int (*)(const void*, U, U, U, U, U, U, U, U, U, U, U)>(fn)(
        c, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], ws, bytes, st);
  }
  return -1;
}

// call(function address, configuration bytes, spec bytes, operands tuple, workspace, device, stream):
// the function's status, or None when an operand is not the plain case (nothing has been called then).
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 7 || !PyBytes_Check(args[1]) || !PyBytes_Check(args[2]) || !PyTuple_Check(args[3]) ||
      !THPVariable_Check(args[4])) {
    PyErr_SetString(PyExc_TypeError, "call(function, configuration, specs, operands, ws, device, stream)");
    return nullptr;
  }
  const U fn = PyLong_AsUnsignedLongLong(args[0]);
  const int64_t device = PyLong_AsLongLong(args[5]);
  const U stream = args[6] == Py_None ? 0 : PyLong_AsUnsignedLongLong(args[6]);
  if (PyErr_Occurred()) return nullptr;
  const Py_ssize_t n = PyTuple_GET_SIZE(args[3]);
  if (n > kMaxOperands || PyBytes_GET_SIZE(args[2]) != n * static_cast<Py_ssize_t>(sizeof(Spec)))
    Py_RETURN_NONE;
  const Spec* specs = reinterpret_cast<const Spec*>(PyBytes_AS_STRING(args[2]));
  U address[kMaxOperands], base, bytes;
  try {  // tensors without storage or of irregular sizes throw when asked; binding.py refuses them
    for (Py_ssize_t i = 0; i < n; ++i)
      if (!plain(PyTuple_GET_ITEM(args[3], i), specs[i], device, &address[i])) Py_RETURN_NONE;
    const at::Tensor& ws = THPVariable_Unpack(args[4]);
    if (!ws.defined() || !ws.is_cuda() || ws.get_device() != device || !ws.is_contiguous()) Py_RETURN_NONE;
    base = reinterpret_cast<U>(ws.data_ptr());
    bytes = ws.nbytes();
  } catch (const std::exception&) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const void* cfg = PyBytes_AS_STRING(args[1]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = call_with(fn, cfg, n, address, base, bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

// The number by which specs name a torch.dtype.
PyObject* type_code(PyObject*, PyObject* dtype) {
  if (!THPDtype_Check(dtype)) {
    PyErr_SetString(PyExc_TypeError, "expected a torch.dtype");
    return nullptr;
  }
  return PyLong_FromLong(static_cast<long>(reinterpret_cast<THPDtype*>(dtype)->scalar_type));
}

PyMethodDef kMethods[] = {
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr},
    {"type_code", type_code, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_operands", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__operands(void) { return PyModule_Create(&kModule); }
