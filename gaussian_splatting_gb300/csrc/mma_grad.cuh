// dz, its column sums and dx of a narrow bfloat16 layer in one pass (mma_grad.cu).
#pragma once

#include "mma.cuh"

namespace gs {

// Whether the sizes, types and alignment are this kernel's.  Not a question of whether dx is wanted, which must not change
// the order in which the bias gradient is added up.
bool grad_takes(const gs_linear_desc* d, const void* dy, const void* z);
// Whether it can also write dx; else the products read the dz that it writes.
bool grad_takes_dx(const gs_linear_desc* d, const void* w, const void* dx);
// blocks, each of which writes a row of out_features column sums to `part`
int grad_parts(int64_t rows);
// dz (rows of lddz), dx and part may each be NULL: not wanted
gs_status grad_run(const gs_linear_desc* d, const void* dy, const void* z, const void* w, void* dz, int64_t lddz, void* dx,
                   float* part, int32_t* status, cudaStream_t st, const char* where);

}  // namespace gs
