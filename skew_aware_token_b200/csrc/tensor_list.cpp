// Reads a list of torch tensors into the descriptors of an optimizer's step: for hundreds of
// tensors the same checks from Python take several times the step itself (250 tensors: 80 us).
// Called through ctypes with the interpreter's lock held; linked to torch, and so kept out of
// libmoeskew.so.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "moeskew_train.h"

enum { LIST_OK = 0, LIST_LENGTH = 1, LIST_TYPE = 2, LIST_DEVICE = 3, LIST_SIZE = 4 };

// For tensor i of `list` (a Python list or tuple) of `count`: its checks (fp32 or bf16, on
// CUDA device `device`, contiguous, sizes[i] elements), then its address and element type
// into descriptors[i].g and .g_dtype.  Returns LIST_OK, or 8 i + what is wrong with tensor i
// (the descriptors before it are filled then, and no step has been made).
extern "C" __attribute__((visibility("default"))) int64_t
moet_read_gradients(PyObject* list, int64_t count, int32_t device, const int64_t* sizes,
                    moet_adamw_tensor* descriptors) {
  const bool is_list = PyList_Check(list);
  if (!is_list && !PyTuple_Check(list)) return LIST_LENGTH;
  if ((is_list ? PyList_GET_SIZE(list) : PyTuple_GET_SIZE(list)) != count) return LIST_LENGTH;
  int64_t i = 0;
  try {
    for (; i < count; ++i) {
      PyObject* item = is_list ? PyList_GET_ITEM(list, i) : PyTuple_GET_ITEM(list, i);
      if (!THPVariable_Check(item)) return 8 * i + LIST_TYPE;
      const at::Tensor& t = THPVariable_Unpack(item);
      const auto type = t.scalar_type();
      if (type != at::kFloat && type != at::kBFloat16) return 8 * i + LIST_TYPE;
      if (!t.is_cuda() || t.get_device() != device) return 8 * i + LIST_DEVICE;
      if (t.layout() != at::kStrided || t.numel() != sizes[i] || !t.is_contiguous())
        return 8 * i + LIST_SIZE;
      descriptors[i].g = t.const_data_ptr();
      descriptors[i].g_dtype = type == at::kFloat ? MOET_F32 : MOET_BF16;
    }
  } catch (...) {  // a tensor without storage
    return 8 * i + LIST_TYPE;
  }
  return LIST_OK;
}
