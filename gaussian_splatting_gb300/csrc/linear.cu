// The linear layer y = act(x w^T + bias) + residual and its gradient (gs_linear_fwd, gs_linear_bwd).
//
// Three products, each C(m, n) = sum over k of A(m, k) B(n, k) on the tensor cores:
//   forward  z  = x w^T    A = x,  B = w
//   dx       dx = dz w     A = dz, B = w along its other axis
//   dw       dw = dz^T x   A = dz and B = x, both along their other axes
// bfloat16 arrays whose rows start and end on 16-byte boundaries go to mma.cu, other bfloat16 ones to mma_staged.cu,
// float32 to mma_f32.cu; small calls to linear_small.cu.
// dz = dy act'(z) is formed once, in a pass over dy and z that also takes the bias gradient's column
// sums, and kept in the workspace for the two products that read it.  A narrow bfloat16 layer's pass computes
// dx as well (mma_grad.cu), with up to 256 inputs and outputs: the dw product's operands are then all that is
// read twice (300K x 256 -> 256 with GELU 174 us, 211 as separate passes; 3M x 64 -> 64 358 and 510; the two
// meet at 500 rows, 20 us).
#include "mma.cuh"
#include "mma_grad.cuh"
#include "small.cuh"

namespace {

constexpr int kThreads = 256;

// dz = dy act'(z) to `dz` (if wanted; a row's last 16 bytes are filled up with zeros), and its column sums over this
// block's rows to part[blockIdx.x].  In bfloat16 dz is rounded here, once, and the sums are taken before: the tensor core
// multiplies bfloat16, and a second part for what the rounding leaves would double both products and dz's traffic.
// What it costs: dx and dw of 300K x 256 -> 256 and of 15,965 x 1024 -> 4096 with GELU are off by 2.3e-3 of their norm
// against 64 bits, where dz in 32 bits and the rounding of the results alone gives 1.7e-3.  (Few rows, thin and narrow
// layers on the FP32 pipe, linear_small.cu, keep dz in 32 bits.)  A thread owns VE columns; CX threads lie along a row, kThreads / CX rows side by
// side.  (ACT is the compiler's: a branch for each element would keep their evaluations from overlapping; 15,965 x 4096
// bf16 with GELU 60 us, 63.5 with branches.  Four blocks to an SM, or that layer's whole backward takes 241 us, not 235.)
template <typename T, bool VEC, int CX, int ACT>
__device__ __forceinline__ void act_grad_rows(const T* dy, const T* z, int64_t rows, int n, int64_t lddy, int64_t ldz, T* dz,
                                              int64_t lddz, int c, int ry, float* sum) {
  constexpr int VE = 16 / sizeof(T), kRows = kThreads / CX;
  using IO = VecIO<T, VE>;
#pragma unroll 2
  for (int64_t r = (int64_t)blockIdx.x * kRows + ry; r < rows; r += (int64_t)gridDim.x * kRows) {
    float d[VE], v[VE];
    if (VEC) {
      const auto rd = IO::load(dy + r * lddy + c);
      if (ACT != GS_ACT_NONE) {
        const auto rz = IO::load(z + r * ldz + c);
        IO::unpack(rz, v);
      }
      IO::unpack(rd, d);
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        d[e] = c + e < n ? to_f32<T>(dy[r * lddy + c + e]) : 0.f;
        if (ACT != GS_ACT_NONE) v[e] = c + e < n ? to_f32<T>(z[r * ldz + c + e]) : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if (ACT != GS_ACT_NONE) d[e] *= act_slope(v[e], ACT);
      sum[e] += d[e];
    }
    if (dz) IO::store(dz + r * lddz + c, d);
  }
}
template <typename T, bool VEC, int CX>
__global__ void __launch_bounds__(kThreads, 4) k_act_grad(const T* dy, const T* z, int64_t rows, int n, int64_t lddy,
                                                          int64_t ldz, int act, T* dz, int64_t lddz, float* part) {
  follow();
  constexpr int VE = 16 / sizeof(T), kRows = kThreads / CX;
  const int cx = threadIdx.x % CX, ry = threadIdx.x / CX;
  const int c = (blockIdx.y * CX + cx) * VE;
  float sum[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) sum[e] = 0.f;
  if (c < n) {
    if (act == GS_ACT_GELU) act_grad_rows<T, VEC, CX, GS_ACT_GELU>(dy, z, rows, n, lddy, ldz, dz, lddz, c, ry, sum);
    else if (act == GS_ACT_SILU) act_grad_rows<T, VEC, CX, GS_ACT_SILU>(dy, z, rows, n, lddy, ldz, dz, lddz, c, ry, sum);
    else if (act == GS_ACT_RELU) act_grad_rows<T, VEC, CX, GS_ACT_RELU>(dy, z, rows, n, lddy, ldz, dz, lddz, c, ry, sum);
    else act_grad_rows<T, VEC, CX, GS_ACT_NONE>(dy, z, rows, n, lddy, ldz, dz, lddz, c, ry, sum);
  }
  if (!part) return;
  __shared__ float fold[kRows][CX * VE + 1];
#pragma unroll
  for (int e = 0; e < VE; ++e) fold[ry][cx * VE + e] = sum[e];
  __syncthreads();
  for (int k = threadIdx.x; k < CX * VE; k += kThreads) {
    const int col = blockIdx.y * CX * VE + k;
    if (col >= n) continue;
    float t = 0.f;
#pragma unroll 8
    for (int r = 0; r < kRows; ++r) t += fold[r][k];
    part[(int64_t)blockIdx.x * n + col] = t;
  }
}

// ---------------------------------------------------------------- host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// threads along a row of n columns in k_act_grad, and its blocks down the rows
template <typename T>
int row_threads(int n) {
  const int nv = (int)ceil_div(n, 16 / sizeof(T));
  return nv <= 4 ? 4 : nv <= 8 ? 8 : nv <= 16 ? 16 : 32;
}
template <typename T>
int act_grad_parts(int64_t rows, int n) {
  const int cx = row_threads<T>(n);
  const int64_t across = ceil_div(n, cx * (16 / (int64_t)sizeof(T)));
  int64_t s = ceil_div(4 * 152, across);
  const int64_t most = ceil_div(rows, 4 * (kThreads / cx));
  return (int)(s < most ? s : most);
}
int parts_of(const gs_linear_desc* d) {
  return d->dtype == GS_F32 ? act_grad_parts<float>(d->rows, d->out_features)
                            : act_grad_parts<__nv_bfloat16>(d->rows, d->out_features);
}

template <typename T>
gs_status run_act_grad(const gs_linear_desc* d, const T* dy, const T* z, T* dz, int64_t lddz, float* part, cudaStream_t st,
                       const char* where) {
  const int n = d->out_features, parts = act_grad_parts<T>(d->rows, n);
  const bool vec = gs::rows_aligned16(dy, d->rows, d->ldy, d->dtype) && n % (16 / sizeof(T)) == 0 &&
                   (!z || gs::rows_aligned16(z, d->rows, d->ldz, d->dtype));
  const int cx = row_threads<T>(n);
  const dim3 grid(parts, (unsigned)ceil_div(n, cx * (16 / (int64_t)sizeof(T))));
  // Launched only when the kernel before it is done: blocks placed while another kernel holds part of some SMs
  // lie unevenly, and each block has the same share of the rows (300K x 128 -> 59 f32 backward 147 us, 149 with
  // gs::launch).
#define GS_GO(V, CX)                                                                                                  \
  k_act_grad<T, V, CX><<<grid, kThreads, 0, st>>>(dy, z, d->rows, n, d->ldy, d->ldz, d->act, dz, lddz, part)
  if (vec) {
    if (cx == 4) GS_GO(true, 4);
    else if (cx == 8) GS_GO(true, 8);
    else if (cx == 16) GS_GO(true, 16);
    else GS_GO(true, 32);
  } else {
    if (cx == 4) GS_GO(false, 4);
    else if (cx == 8) GS_GO(false, 8);
    else if (cx == 16) GS_GO(false, 16);
    else GS_GO(false, 32);
  }
#undef GS_GO
  return gs::check_launch(where);
}

gs_status run_product(const gs::MmaProduct& q, int32_t dtype, void* workspace, int32_t* status, cudaStream_t st,
                      const char* where) {
  if (dtype == GS_F32) return gs::f32_run(q, workspace, status, st, where);
  if (gs::mma_takes(q)) return gs::mma_run(q, workspace, status, st, where);
  return gs::staged_run(q, workspace, status, st, where);
}

// scratch of a product of these sizes, whichever kernel its arrays' alignment takes it to
size_t product_space(int64_t m, int64_t n, int64_t k, int32_t dtype) {
  if (dtype == GS_F32) return gs::f32_workspace(m, n, k);
  const size_t a = gs::staged_workspace(m, n, k), b = gs::mma_workspace(m, n, k);
  return a > b ? a : b;
}

// The backward's scratch: a copy of dz, its rows filled up with zeros to 16 bytes (after an activation, or
// where rows of dy do not start and end on 16-byte boundaries), the bias gradient's parts, the products' parts.
struct BwdSpace {
  size_t dz, bias, part, total;
  int64_t lddz;
};
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
BwdSpace bwd_space(const gs_linear_desc* d) {
  BwdSpace s{};
  s.lddz = ceil_div(d->out_features, 8) * 8;
  const int unit = 16 / (int)gs::dtype_size(d->dtype);
  const bool copy = d->act != GS_ACT_NONE || d->ldy % unit != 0 || d->out_features % unit != 0;
  s.dz = copy ? up256((size_t)d->rows * s.lddz * gs::dtype_size(d->dtype)) : 0;
  const int parts = parts_of(d), fused = gs::grad_parts(d->rows);
  s.bias = up256((size_t)(parts > fused ? parts : fused) * d->out_features * sizeof(float));
  const size_t a = product_space(d->rows, d->in_features, d->out_features, d->dtype);
  const size_t b = product_space(d->out_features, d->in_features, d->rows, d->dtype);
  s.part = a > b ? a : b;
  s.total = s.dz + s.bias + s.part;
  return s;
}

template <typename T>
gs_status run_bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                  void* dbias, void* workspace, int32_t* status, cudaStream_t st) {
  const char* where = "gs_linear_bwd";
  const BwdSpace space = bwd_space(d);
  unsigned char* at = static_cast<unsigned char*>(workspace);
  // float32 without an activation: a copy with filled-up rows pays for itself when both products read it (300K x
  // 128 -> 59: 150 us against 163; the input gradient alone 83 against 69)
  const bool worth = d->act != GS_ACT_NONE || d->dtype == GS_BF16 ? dx || dw : dx && dw;
  T* copy = space.dz && worth ? reinterpret_cast<T*>(at) : nullptr;
  float* bias_part = reinterpret_cast<float*>(at + space.dz);
  void* part = at + space.dz + space.bias;
  const void* dz = copy ? copy : dy;
  const int64_t lddz = copy ? space.lddz : d->ldy;
  const int64_t unit = 16 / (int64_t)sizeof(T), pad = copy ? ceil_div(d->out_features, unit) * unit - d->out_features : 0;
  int parts = act_grad_parts<T>(d->rows, d->out_features);
  // (without an activation there is nothing to form, and it is used for the sums' sake alone)
  const bool fused = (z || dbias) && gs::grad_takes(d, dy, z), fused_dx = fused && dx && gs::grad_takes_dx(d, w, dx);
  if (fused) {
    parts = gs::grad_parts(d->rows);
    if (gs_status s = gs::grad_run(d, dy, z, w, dw || !fused_dx ? copy : nullptr, space.lddz, fused_dx ? dx : nullptr,
                                   dbias ? bias_part : nullptr, status, st, where))
      return s;
  } else if (copy || dbias) {
    if (gs_status s = run_act_grad<T>(d, static_cast<const T*>(dy), static_cast<const T*>(z), copy, lddz,
                                      dbias ? bias_part : nullptr, st, where))
      return s;
  }
  if (dx && !fused_dx) {
    const gs::MmaProduct q{dz, w, lddz, d->ldw, false, true, d->rows, d->in_features, d->out_features,
                           nullptr, nullptr, dx, nullptr, 0, d->lddx, 0, GS_ACT_NONE, pad};
    if (gs_status s = run_product(q, d->dtype, part, status, st, where)) return s;
  }
  const ColumnFold sums{dbias ? bias_part : nullptr, parts, d->out_features, dbias};
  if (dw) {
    const gs::MmaProduct q{dz, x, lddz, d->ldx, true, true, d->out_features, d->in_features, d->rows,
                           nullptr, nullptr, dw, nullptr, 0, d->lddw, 0, GS_ACT_NONE, pad, 0, sums};
    return run_product(q, d->dtype, part, status, st, where);
  }
  if (dbias) {
    launch_column_fold<T>(sums, st);
    return gs::check_launch(where);
  }
  return GS_OK;
}

gs_status check_desc(const char* where, const gs_linear_desc* d) {
  if (!d) return gs::set_error(GS_ERR_INVALID, "%s: descriptor is NULL", where);
  if (d->rows < 0 || d->rows > 0x7fffffffll || d->in_features < 1 || d->in_features > (1 << 20) || d->out_features < 1 ||
      d->out_features > (1 << 20))
    return gs::set_error(GS_ERR_INVALID, "%s: bad size %lld x %d -> %d", where, (long long)d->rows, d->in_features,
                         d->out_features);
  if (d->dtype != GS_F32 && d->dtype != GS_BF16)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown element type %d", where, d->dtype);
  if (d->act < GS_ACT_NONE || d->act > GS_ACT_SILU)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown activation %d", where, d->act);
  return GS_OK;
}

gs_status check_workspace(const char* where, const void* workspace, size_t have, size_t need) {
  if (need == 0) return GS_OK;
  if (!workspace || !gs::aligned16(workspace))
    return gs::set_error(GS_ERR_INVALID, "%s: workspace is NULL or misaligned", where);
  if (have < need) return gs::set_error(GS_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", where, have, need);
  return GS_OK;
}

}  // namespace

extern "C" size_t gs_linear_fwd_workspace_size(const gs_linear_desc* d) {
  if (check_desc("gs_linear_fwd_workspace_size", d) || d->rows == 0) return 0;
  return gs::small_fwd_takes(d) ? 0 : product_space(d->rows, d->out_features, d->in_features, d->dtype);
}

extern "C" gs_status gs_linear_fwd(const gs_linear_desc* d, const void* x, const void* w, const void* bias,
                                   const void* residual, void* y, void* z, void* workspace, size_t workspace_bytes,
                                   int32_t* status, void* stream) {
  const char* where = "gs_linear_fwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (d->rows == 0) return GS_OK;
  if (gs_status s = gs::check_matrix(where, "x", x, d->rows, d->in_features, d->ldx, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "w", w, d->out_features, d->in_features, d->ldw, d->dtype)) return s;
  if (bias)
    if (gs_status s = gs::check_matrix(where, "bias", bias, 1, d->out_features, d->out_features, d->dtype)) return s;
  if (residual)
    if (gs_status s = gs::check_matrix(where, "residual", residual, d->rows, d->out_features, d->ldr, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "y", y, d->rows, d->out_features, d->ldy, d->dtype)) return s;
  if (z)
    if (gs_status s = gs::check_matrix(where, "z", z, d->rows, d->out_features, d->ldz, d->dtype)) return s;
  if (gs_status s = check_workspace(where, workspace, workspace_bytes, gs_linear_fwd_workspace_size(d))) return s;
  if (gs::small_fwd_takes(d)) return gs::small_fwd(d, x, w, bias, residual, y, z, gs::as_stream(stream), where);
  const gs::MmaProduct q{x, w, d->ldx, d->ldw, false, false, d->rows, d->out_features, d->in_features,
                         bias, residual, y, z, d->ldr, d->ldy, d->ldz, d->act};
  return run_product(q, d->dtype, workspace, status, gs::as_stream(stream), where);
}

extern "C" size_t gs_linear_bwd_workspace_size(const gs_linear_desc* d) {
  if (check_desc("gs_linear_bwd_workspace_size", d) || d->rows == 0) return 0;
  return gs::small_bwd_takes(d) ? gs::small_bwd_workspace(d) : bwd_space(d).total;
}

extern "C" gs_status gs_linear_bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z,
                                   void* dx, void* dw, void* dbias, void* workspace, size_t workspace_bytes,
                                   int32_t* status, void* stream) {
  const char* where = "gs_linear_bwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (!dx && !dw && !dbias) return GS_OK;
  cudaStream_t st = gs::as_stream(stream);
  const size_t size = gs::dtype_size(d->dtype);
  if (dw)
    if (gs_status s = gs::check_matrix(where, "dw", dw, d->out_features, d->in_features, d->lddw, d->dtype)) return s;
  if (dbias)
    if (gs_status s = gs::check_matrix(where, "dbias", dbias, 1, d->out_features, d->out_features, d->dtype)) return s;
  if (d->rows == 0) {
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemset2DAsync(dw, (d->out_features > 1 ? d->lddw : d->in_features) * size, 0, d->in_features * size,
                                  d->out_features, st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, d->out_features * size, st);
    return e == cudaSuccess ? GS_OK : gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  }
  if (gs_status s = gs::check_matrix(where, "dy", dy, d->rows, d->out_features, d->ldy, d->dtype)) return s;
  if (dw)
    if (gs_status s = gs::check_matrix(where, "x", x, d->rows, d->in_features, d->ldx, d->dtype)) return s;
  if (dx) {
    if (gs_status s = gs::check_matrix(where, "w", w, d->out_features, d->in_features, d->ldw, d->dtype)) return s;
    if (gs_status s = gs::check_matrix(where, "dx", dx, d->rows, d->in_features, d->lddx, d->dtype)) return s;
  }
  if (d->act == GS_ACT_NONE) z = nullptr;
  else if (gs_status s = gs::check_matrix(where, "z", z, d->rows, d->out_features, d->ldz, d->dtype)) return s;
  if (gs_status s = check_workspace(where, workspace, workspace_bytes, gs_linear_bwd_workspace_size(d))) return s;
  if (gs::small_bwd_takes(d)) return gs::small_bwd(d, dy, x, w, z, dx, dw, dbias, workspace, st, where);
  if (d->dtype == GS_F32) return run_bwd<float>(d, dy, x, w, z, dx, dw, dbias, workspace, status, st);
  return run_bwd<__nv_bfloat16>(d, dy, x, w, z, dx, dw, dbias, workspace, status, st);
}
