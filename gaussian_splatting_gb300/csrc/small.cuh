// The linear layer's small calls (linear_small.cu): whether a call is one, and the call.
#pragma once

#include "dense.cuh"

namespace gs {

bool small_fwd_takes(const gs_linear_desc* d);
gs_status small_fwd(const gs_linear_desc* d, const void* x, const void* w, const void* bias, const void* residual, void* y,
                    void* z, cudaStream_t st, const char* where);

bool small_bwd_takes(const gs_linear_desc* d);
size_t small_bwd_workspace(const gs_linear_desc* d);
gs_status small_bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                    void* dbias, void* workspace, cudaStream_t st, const char* where);

}  // namespace gs
