// Reads torch tensors for the training classes: checks a call's arguments and takes their
// addresses.  From Python the same checks cost a small call more than its launch does (a norm of
// one token 3.6 us of 7.2), and those of an optimizer's list several times its step (250
// tensors 80 us).  Called through ctypes with the interpreter's lock held; linked to torch, and
// so kept out of libmoeskew.so.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "moeskew_train.h"

// For the build, which reads it from the file: another torch or interpreter lays out its objects
// in another way.
extern "C" __attribute__((used)) const char moeskew_args_built_for[] =
    "moeskew_args built for [" MOESKEW_BUILT_FOR "]";

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
// dimension when `flat`.
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

// One argument: its element type and size, whether None may stand for it (ARG_OPTIONAL), and
// whether a longer one-dimensional buffer may (ARG_FLAT: MoeLayer's buffers are such).
enum { ARG_OPTIONAL = 1, ARG_FLAT = 2 };
struct moet_arg {
  int32_t type, flags;
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
        if (!(args[i].flags & ARG_OPTIONAL)) return 8 * i + ARG_MISSING;
        continue;
      }
      if (!THPVariable_Check(o)) return 8 * i + ARG_DEVICE;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (const int bad = check(t, device, args[i].n, args[i].flags & ARG_FLAT))
        return 8 * i + bad;
      if (type_of(t) != args[i].type) return 8 * i + ARG_TYPE;
      out[i] = t.const_data_ptr();
    }
  } catch (...) {  // a tensor without storage
    return 8 * i + ARG_DEVICE;
  }
  return ARG_OK;
}

namespace {

// A tensor of a step: its address as the step finds it (a storage may have been exchanged since
// the last one), noting whether it moved.
template <class T>
inline int take(PyObject* o, int type, int device, int64_t n, T** out, bool* moved) {
  if (!THPVariable_Check(o)) return ARG_TYPE;
  const at::Tensor& t = THPVariable_Unpack(o);
  const c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  const caffe2::TypeMeta f32 = caffe2::TypeMeta::Make<float>(),
                         bf16 = caffe2::TypeMeta::Make<at::BFloat16>(),
                         e4m3 = caffe2::TypeMeta::Make<at::Float8_e4m3fn>();
  if (impl->dtype() != (type == MOET_F32 ? f32 : type == MOET_BF16 ? bf16 : e4m3)) return ARG_TYPE;
  if (*out && impl->has_storage() && impl->numel() == n && impl->is_contiguous()) {
    // where the last step found it, what `check` asks has the answers of that step
    const int64_t size = type == MOET_F32 ? 4 : type == MOET_BF16 ? 2 : 1;
    if (static_cast<char*>(impl->unsafe_storage().mutable_data()) + impl->storage_offset() * size ==
        reinterpret_cast<char*>(*out))
      return ARG_OK;
  }
  if (const int bad = check(t, device, n, false)) return bad;
  T* p = static_cast<T*>(t.data_ptr());
  *moved |= p != *out;
  *out = p;
  return ARG_OK;
}

}  // namespace

// The tensors of an optimizer's step: gradients (fp32 or bf16, of sizes[i] elements), weights of
// the descriptors' types, and `states`, a tuple of the lists m, v, m_scale, v_scale and master
// (None where there is none; () for none at all: the descriptors keep theirs).  Their addresses
// and the gradients' types go into the descriptors, and the weights' versions are raised.  Returns
// 0, -1 if an address other than a gradient's changed, or 8 (j count + i) + what is wrong with
// tensor i of list j: gradients, weights, then the states' five (the descriptors before it are
// filled then, and no step has been made).
MOET_HOST int64_t moet_read_step(PyObject* grads, PyObject* weights, PyObject* states,
                                 int64_t count, int32_t device, const int64_t* sizes,
                                 moet_adamw_tensor* descriptors) {
  enum { M = 0, V = 1, M_SCALE = 2, V_SCALE = 3, MASTER = 4, LISTS = 5 };
  PyObject** list[LISTS] = {};
  if (length(grads) != count) return ARG_LIST;
  if (length(weights) != count) return 8 * count + ARG_LIST;
  const bool with_states = length(states) == LISTS;
  if (with_states) {
    for (int64_t j = 0; j < LISTS; ++j) {
      PyObject* l = item(states, j);
      if (l == Py_None) continue;
      if (length(l) != count) return 8 * (j + 2) * count + ARG_LIST;
      list[j] = PySequence_Fast_ITEMS(l);
    }
  }
  PyObject** const g_list = PySequence_Fast_ITEMS(grads);
  PyObject** const p_list = PySequence_Fast_ITEMS(weights);
  int64_t at = 0;
  bool changed = false;
  try {
    for (int64_t i = 0; i < count; ++i) {
      moet_adamw_tensor& d = descriptors[i];
      const int64_t n = sizes[i], blocks = (n + MOET_ADAMW_BLOCK - 1) / MOET_ADAMW_BLOCK;
      at = 8 * i;
      PyObject* o = g_list[i];
      if (!THPVariable_Check(o)) return at + ARG_TYPE;
      const at::Tensor& g = THPVariable_Unpack(o);
      const int type = type_of(g);
      if (type != MOET_F32 && type != MOET_BF16) return at + ARG_TYPE;
      if (const int bad = check(g, device, n, false)) return at + bad;
      d.g = g.const_data_ptr();
      d.g_dtype = type;
      at = 8 * (count + i);
      if (const int bad = take(p_list[i], d.p_dtype, device, n, &d.p, &changed)) return at + bad;
      if (!with_states) continue;
      // one of the states: none (any more) where its list is, or a master where it is None itself
      const auto state = [&](int64_t j, int type, int64_t size, auto** out) -> int {
        at = 8 * ((j + 2) * count + i);
        if (list[j] && !(j == MASTER && list[j][i] == Py_None))
          return take(list[j][i], type, device, size, out, &changed);
        *out = nullptr;
        return ARG_OK;
      };
      if (const int bad = state(M, d.state_dtype, n, &d.m)) return at + bad;
      if (const int bad = state(V, d.state_dtype, n, &d.v)) return at + bad;
      if (const int bad = state(M_SCALE, MOET_F32, blocks, &d.m_scale)) return at + bad;
      if (const int bad = state(V_SCALE, MOET_F32, blocks, &d.v_scale)) return at + bad;
      if (const int bad = state(MASTER, MOET_F32, n, &d.master)) return at + bad;
    }
    // the step changes the weights behind autograd's back: a backward that saved one has to know
    for (int64_t i = 0; i < count; ++i) {
      at = 8 * (count + i);
      const at::Tensor& p = THPVariable_Unpack(p_list[i]);
      if (!p.is_inference()) p.unsafeGetTensorImpl()->bump_version();
    }
  } catch (...) {
    return at + ARG_TYPE;
  }
  return changed ? -1 : ARG_OK;
}
