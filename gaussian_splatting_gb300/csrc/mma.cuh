// The tensor-core product behind the linear layer (mma.cu).
#pragma once

#include <cuda.h>

#include "dense.cuh"

namespace gs {

// C(m, n) = sum over k of A(m, k) B(n, k), then y = act(C + bias) + residual, z = C + bias.
// An operand lies in memory as [m][k] with `ld` elements between rows, or, `*_mn`, as [k][m].
struct MmaProduct {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  bool a_mn, b_mn;
  int64_t m, n, k;
  const void* bias;
  const void* residual;
  void* y;
  void* z;
  int64_t ldr, ldy, ldz;
  int act;
  int64_t a_pad = 0, b_pad = 0;  // zeros that follow each of the operand's rows in memory
  ColumnFold also = {};          // sums to fold when the product is done, in the launch that folds its splits if any
};

// bfloat16 whose rows start anywhere (mma_staged.cu).
size_t staged_workspace(int64_t m, int64_t n, int64_t k);
gs_status staged_run(const MmaProduct& p, void* workspace, int32_t* status, cudaStream_t st, const char* where);

// float32 in full precision (mma_f32.cu).
size_t f32_workspace(int64_t m, int64_t n, int64_t k);
gs_status f32_run(const MmaProduct& p, void* workspace, int32_t* status, cudaStream_t st, const char* where);

// A tensor map of a [rows][cols] matrix in boxes of box_rows rows x 128 (or 64) bytes, swizzled over them; false
// if the driver refuses it.
bool encode_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, int32_t dtype,
                int row_bytes = 128);

// the bound of a device-side wait in microseconds: the number of iterations that the sorts' waits have
inline int wait_us() {
  const int64_t n = wait_limit();
  return n < 0x7fffffff ? (int)n : 0x7fffffff;
}

// whether TMA takes every array of the product (bfloat16)
bool mma_takes(const MmaProduct& p);
// bytes of scratch for a product of these sizes (0: none), whatever its arrays
size_t mma_workspace(int64_t m, int64_t n, int64_t k);
gs_status mma_run(const MmaProduct& p, void* workspace, int32_t* status, cudaStream_t st, const char* where);

}  // namespace gs
