// Reads torch tensors for the training classes: checks a call's arguments and takes their
// addresses.  From Python the same checks cost a small call more than its launch does (a norm of
// one token 3.6 us of 7.2), and those of an optimizer's list several times its step (250
// tensors 80 us).  Called through ctypes with the interpreter's lock held; linked to torch, and
// so kept out of libmoeskew.so.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "moeskew_train.h"

namespace {

// What is wrong with an argument.
enum { ARG_OK = 0, ARG_LIST = 1, ARG_TYPE = 2, ARG_DEVICE = 3, ARG_SIZE = 4, ARG_MISSING = 5 };

// Element types: MOET_F32, MOET_BF16, MOET_E4M3, and those of indices and masks.
enum { TYPE_I32 = 3, TYPE_U8 = 4 };
int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOET_F32;
    case at::kBFloat16: return MOET_BF16;
    case at::kFloat8_e4m3fn: return MOET_E4M3;
    case at::kInt: return TYPE_I32;
    case at::kByte: return TYPE_U8;
    default: return -1;
  }
}

// A strided, contiguous CUDA tensor on `device` with n elements, or with more of them in one
// dimension when `flat` (what MoeLayer owns).
int check(const at::Tensor& t, int device, int64_t n, bool flat) {
  if (!t.is_cuda() || t.get_device() != device) return ARG_DEVICE;
  if (t.layout() != at::kStrided || !t.is_contiguous()) return ARG_SIZE;
  if (t.numel() != n && !(flat && t.dim() == 1 && t.numel() > n)) return ARG_SIZE;
  return ARG_OK;
}

int64_t length(PyObject* list) {
  return PyList_Check(list) ? PyList_GET_SIZE(list)
         : PyTuple_Check(list) ? PyTuple_GET_SIZE(list) : -1;
}
PyObject* item(PyObject* list, int64_t i) {
  return PyList_Check(list) ? PyList_GET_ITEM(list, i) : PyTuple_GET_ITEM(list, i);
}

}  // namespace

// One argument: its element type and size, and whether None may stand for it.
struct moet_arg {
  int32_t type, optional;
  int64_t n;
};

#define MOET_HOST extern "C" __attribute__((visibility("default")))

// The addresses of `count` arguments (a list or tuple of tensors and None) after their checks
// against `args`; NULL for None.  Returns 0, or 8 i + what is wrong with argument i.
MOET_HOST int64_t moet_read_arguments(PyObject* list, int64_t count, int32_t device,
                                      const moet_arg* args, const void** out) {
  if (length(list) != count) return ARG_LIST;
  int64_t i = 0;
  try {
    for (; i < count; ++i) {
      PyObject* o = item(list, i);
      out[i] = nullptr;
      if (o == Py_None) {
        if (!args[i].optional) return 8 * i + ARG_MISSING;
        continue;
      }
      if (!THPVariable_Check(o)) return 8 * i + ARG_DEVICE;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (const int bad = check(t, device, args[i].n, true)) return 8 * i + bad;
      if (type_of(t) != args[i].type) return 8 * i + ARG_TYPE;
      out[i] = t.const_data_ptr();
    }
  } catch (...) {  // a tensor without storage
    return 8 * i + ARG_DEVICE;
  }
  return ARG_OK;
}

// The weights and gradients of an optimizer's step: weights of the descriptors' types, gradients
// fp32 or bf16, each of sizes[i] elements; their addresses (a weight's storage may have been
// exchanged since the last step) and the gradients' types go into the descriptors.  Returns 0,
// or 8 i + what is wrong with gradient i, or 8 (count + i) + what is wrong with weight i (the
// descriptors before it are filled then, and no step has been made).
MOET_HOST int64_t moet_read_step(PyObject* grads, PyObject* weights, int64_t count,
                                 int32_t device, const int64_t* sizes,
                                 moet_adamw_tensor* descriptors) {
  if (length(grads) != count) return ARG_LIST;
  if (length(weights) != count) return 8 * count + ARG_LIST;
  int64_t at = 0;
  try {
    for (int64_t i = 0; i < count; ++i) {
      at = 8 * i;
      PyObject* o = item(grads, i);
      if (!THPVariable_Check(o)) return at + ARG_TYPE;
      const at::Tensor& g = THPVariable_Unpack(o);
      const int type = type_of(g);
      if (type != MOET_F32 && type != MOET_BF16) return at + ARG_TYPE;
      if (const int bad = check(g, device, sizes[i], false)) return at + bad;
      at = 8 * (count + i);
      o = item(weights, i);
      if (!THPVariable_Check(o)) return at + ARG_TYPE;
      const at::Tensor& p = THPVariable_Unpack(o);
      if (type_of(p) != descriptors[i].p_dtype) return at + ARG_TYPE;
      if (const int bad = check(p, device, sizes[i], false)) return at + bad;
      descriptors[i].g = g.const_data_ptr();
      descriptors[i].g_dtype = type;
      descriptors[i].p = p.data_ptr();
    }
  } catch (...) {
    return at + ARG_TYPE;
  }
  return ARG_OK;
}
