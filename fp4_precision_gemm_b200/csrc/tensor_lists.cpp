// Reads Python lists of torch tensors into fp8q_grad_item records, for the binding: through Python a tensor's
// address, size, type, device and contiguity cost five attribute reads, 0.3 us, and lists of hundreds of small
// tensors then cost more on the host than their kernels do on the device.  The tensors are asked through
// DLPack's C exchange interface (a table of functions that torch publishes for this, looked up once).
// Loaded with ctypes.PyDLL: the interpreter's lock is held, so the lists do not change under the loop.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/dlpack.h>

#include <cstdint>

#include "../../include/fp8q.h"

namespace {

struct Read {
  const DLPackExchangeAPI* api;
  PyTypeObject *tensor, *parameter;
  int device_type, device;

  // Address, elements and type of one contiguous tensor; false for anything else (other classes too, which
  // may not be what their memory says).
  bool operator()(PyObject* o, void** data, int64_t* numel, int64_t* dtype) {
    if (Py_TYPE(o) != tensor && Py_TYPE(o) != parameter) return false;
    DLTensor t;
    if (api->dltensor_from_py_object_no_sync(o, &t) != 0) {
      PyErr_Clear();
      return false;
    }
    if (t.device.device_type != device_type || t.dtype.lanes != 1) return false;
    if (device < 0) device = t.device.device_id;
    if (t.device.device_id != device) return false;
    if (t.dtype.code == kDLBfloat && t.dtype.bits == 16) *dtype = FP8Q_BF16;
    else if (t.dtype.code == kDLFloat && t.dtype.bits == 32) *dtype = FP8Q_FP32;
    else return false;
    int64_t n = 1;
    bool contiguous = true;
    for (int d = t.ndim - 1; d >= 0; --d) {
      contiguous &= t.strides == nullptr || t.shape[d] == 1 || t.strides[d] == n;
      n *= t.shape[d];
    }
    if (n != 0 && !contiguous) return false;
    *data = static_cast<char*>(t.data) + t.byte_offset;
    *numel = n;
    return true;
  }
};

}  // namespace

// The table behind a class's __dlpack_c_exchange_api__, NULL if it is of another version than this file knows.
extern "C" const void* fp8q_lists_api(PyObject* capsule) {
  const auto* api = static_cast<const DLPackExchangeAPI*>(PyCapsule_GetPointer(capsule, "dlpack_exchange_api"));
  if (api == nullptr) PyErr_Clear();
  return api != nullptr && api->header.version.major == DLPACK_MAJOR_VERSION ? api : nullptr;
}

// items[i] of the lists grads and outs (None: grads), whose tensors are all contiguous FP32 or BF16 on one device
// of `device_type` (a kDL... value), a tensor of outs of its gradient's type and size.  Returns the device's
// index, or -1 where one of this does not hold.
extern "C" int64_t fp8q_lists_grads(const void* api, PyObject* tensor, PyObject* parameter, PyObject* grads,
                                    PyObject* outs, int32_t device_type, fp8q_grad_item* items) {
  if (!PyList_CheckExact(grads) || (outs != Py_None && !PyList_CheckExact(outs))) return -1;
  Read read{static_cast<const DLPackExchangeAPI*>(api), reinterpret_cast<PyTypeObject*>(tensor),
            reinterpret_cast<PyTypeObject*>(parameter), device_type, -1};
  const Py_ssize_t n = PyList_GET_SIZE(grads);
  if (outs != Py_None && PyList_GET_SIZE(outs) != n) return -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    fp8q_grad_item& it = items[i];
    void* data = nullptr;
    if (!read(PyList_GET_ITEM(grads, i), &data, &it.numel, &it.dtype)) return -1;
    it.grad = it.out = data;
    if (outs == Py_None) continue;
    int64_t numel = 0, dtype = 0;
    if (!read(PyList_GET_ITEM(outs, i), &it.out, &numel, &dtype) || numel != it.numel || dtype != it.dtype) return -1;
  }
  return read.device;
}
