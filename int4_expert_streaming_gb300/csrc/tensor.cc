// tensor.cc -- what binding.c asks of a torch tensor, read from the tensor
// itself.  Its Python attributes say the same at 30 to 80 ns each, 270 ns a
// tensor (on Grace); this takes 4.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tensor.h"

// The torch and Python whose headers this was compiled with: the parts of a tensor stand where these say.
extern "C" const char* moe_tensor_built_for(void) { return MOE_BUILT_FOR; }

// 1: filled.  0: not a torch tensor, or one without plain strides or memory of its own.
extern "C" int moe_tensor_of(PyObject* o, moe_tensor* v) {
    try {
        if (!THPVariable_Check(o)) return 0;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.defined() || t.layout() != at::kStrided) return 0;
        switch (t.scalar_type()) {
            case at::kFloat: v->type = MOE_TENSOR_F32; break;
            case at::kBFloat16: v->type = MOE_TENSOR_BF16; break;
            case at::kInt: v->type = MOE_TENSOR_I32; break;
            case at::kByte: v->type = MOE_TENSOR_U8; break;
            default: v->type = MOE_TENSOR_OTHER;
        }
        v->device = t.is_cuda() ? t.get_device() : -1;
        const auto shape = t.sizes(), stride = t.strides();
        v->dims = (int)shape.size();
        for (int i = 0; i < v->dims && i < MOE_TENSOR_DIMS; ++i) v->shape[i] = shape[i], v->stride[i] = stride[i];
        v->numel = t.numel();
        v->contiguous = t.is_contiguous();
        v->p = t.data_ptr();
        return 1;
    } catch (...) {
        return 0;  // its attributes then say why
    }
}
