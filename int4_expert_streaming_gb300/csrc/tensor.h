// tensor.h -- a tensor as binding.c sees it.
#ifndef MOE_TENSOR_H
#define MOE_TENSOR_H

#include <Python.h>
#include <stdint.h>

enum { MOE_TENSOR_OTHER = -1, MOE_TENSOR_F32, MOE_TENSOR_BF16, MOE_TENSOR_I32, MOE_TENSOR_U8 };
#define MOE_TENSOR_DIMS 4 /* of which shape and stride are kept */

typedef struct {
    void* p;
    int64_t shape[MOE_TENSOR_DIMS], stride[MOE_TENSOR_DIMS], numel;
    int device; /* -1: not on a GPU */
    int type, dims, contiguous;
} moe_tensor;

#ifdef __cplusplus
extern "C" {
#endif
int moe_tensor_of(PyObject* o, moe_tensor* v);
const char* moe_tensor_built_for(void);
#ifdef __cplusplus
}
#endif

#endif
