// The linear layer y = act(x w^T + bias) + residual and its gradient (gs_linear_fwd, gs_linear_bwd).
//
// Three products share one kernel, C(m, n) = sum over k of A(m, k) B(n, k) with A and B given by
// their two strides:
//   forward  z  = x w^T    A = x,  B = w
//   dx       dx = dz w     A = dz, B = w read along its other axis
//   dw       dw = dz^T x   A = dz and x both read along their other axes
// with dz = dy act'(z) formed as its elements are loaded.
#include "dense.cuh"

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float act_value(float v, int act) {
  switch (act) {
    case GS_ACT_RELU: return v < 0.f ? 0.f : v;
    case GS_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case GS_ACT_SILU: return v / (1.f + expf(-v));
    default: return v;
  }
}

__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case GS_ACT_RELU: return v > 0.f ? 1.f : 0.f;
    case GS_ACT_GELU:
      return 0.5f * (1.f + erff(v * 0.70710678118654752f)) + v * expf(-0.5f * v * v) * 0.39894228040143268f;
    case GS_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-v));
      return s * (1.f + v * (1.f - s));
    }
    default: return 1.f;
  }
}

struct Product {
  const void* a;   // A(m, k) = a[m * am + k * ak], times act'(az(m, k)) if az
  const void* az;
  const void* b;   // B(n, k) = b[n * bn + k * bk]
  int64_t am, ak, azm, azk, bn, bk;
  int64_t m, n, k;
  int64_t k_per_split;
  int act;
  // epilogue, when there is one split; otherwise C goes to part[split][m][n] as it is
  const void* bias;
  const void* residual;
  void* y;
  void* z;
  int64_t ldr, ldy, ldz;
  float* part;
};

template <typename T>
__device__ __forceinline__ void finish(const Product& p, int64_t m, int64_t n, float v) {
  if (p.bias) v += to_f32<T>(static_cast<const T*>(p.bias)[n]);
  if (p.z) static_cast<T*>(p.z)[m * p.ldz + n] = from_f32<T>(v);
  v = act_value(v, p.act);
  if (p.residual) v += to_f32<T>(static_cast<const T*>(p.residual)[m * p.ldr + n]);
  static_cast<T*>(p.y)[m * p.ldy + n] = from_f32<T>(v);
}

// 64 x 64 tile of C per block, 16 of k at a time through shared memory, 4 x 4 sums per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_product(const Product p, int slope_act) {
  __shared__ float sa[16][65], sb[16][65];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
  const int64_t k_lo = (int64_t)blockIdx.z * p.k_per_split;
  const int64_t k_hi = k_lo + p.k_per_split < p.k ? k_lo + p.k_per_split : p.k;
  float c[4][4] = {};
  for (int64_t k0 = k_lo; k0 < k_hi; k0 += 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + i * kThreads;
      // the axis with unit stride runs over neighbouring threads
      const int ka = p.ak == 1 ? e % 16 : e / 64, ma = p.ak == 1 ? e / 16 : e % 64;
      const int kb = p.bk == 1 ? e % 16 : e / 64, nb = p.bk == 1 ? e / 16 : e % 64;
      float va = 0.f, vb = 0.f;
      if (m0 + ma < p.m && k0 + ka < k_hi) {
        va = to_f32<T>(static_cast<const T*>(p.a)[(m0 + ma) * p.am + (k0 + ka) * p.ak]);
        if (p.az) va *= act_slope(to_f32<T>(static_cast<const T*>(p.az)[(m0 + ma) * p.azm + (k0 + ka) * p.azk]), slope_act);
      }
      if (n0 + nb < p.n && k0 + kb < k_hi)
        vb = to_f32<T>(static_cast<const T*>(p.b)[(n0 + nb) * p.bn + (k0 + kb) * p.bk]);
      sa[ka][ma] = va;
      sb[kb][nb] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = sa[k][ty + 16 * i], b[i] = sb[k][tx + 16 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(a[i], b[j], c[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.m || n >= p.n) continue;
      if (gridDim.z > 1) p.part[((int64_t)blockIdx.z * p.m + m) * p.n + n] = c[i][j];
      else finish<T>(p, m, n, c[i][j]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_product_fold(const Product p, int splits) {
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (e >= p.m * p.n) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += p.part[s * p.m * p.n + e];
  finish<T>(p, e / p.n, e % p.n, v);
}

// column sums of dz: 32 columns by 8 rows per block, gridDim.y row ranges
template <typename T>
__global__ void __launch_bounds__(kThreads) k_bias_grad(const T* dy, const T* z, int64_t rows, int n, int64_t lddy,
                                                        int64_t ldz, int act, float* part) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < n)
    for (int64_t r = (int64_t)blockIdx.y * 8 + w; r < rows; r += (int64_t)gridDim.y * 8) {
      const float d = to_f32<T>(dy[r * lddy + c]);
      v += z ? d * act_slope(to_f32<T>(z[r * ldz + c]), act) : d;
    }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < n) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][lane];
    part[(int64_t)blockIdx.y * n + c] = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_bias_fold(const float* part, int parts, int n, T* out) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= n) return;
  float v = 0.f;
  for (int p = 0; p < parts; ++p) v += part[(int64_t)p * n + c];
  out[c] = from_f32<T>(v);
}

// ---------------------------------------------------------------- host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// splits of the k axis: enough blocks for the device, at least 512 of k each
int splits_of(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = ceil_div(m, 64) * ceil_div(n, 64);
  int64_t s = ceil_div(4 * 152, tiles);
  if (s > k / 512) s = k / 512;
  return (int)(s < 1 ? 1 : s > 256 ? 256 : s);
}

size_t part_bytes(int64_t m, int64_t n, int64_t k) {
  const int s = splits_of(m, n, k);
  return s > 1 ? (size_t)s * m * n * sizeof(float) : 0;
}

int bias_parts(int64_t rows, int n) {
  int64_t s = ceil_div(4 * 152, ceil_div(n, 32));
  if (s > ceil_div(rows, 64)) s = ceil_div(rows, 64);
  return (int)(s < 1 ? 1 : s);
}

template <typename T>
gs_status run_product(Product& p, int slope_act, void* workspace, cudaStream_t st, const char* where) {
  const int splits = splits_of(p.m, p.n, p.k);
  p.k_per_split = ceil_div(ceil_div(p.k, splits), 16) * 16;
  p.part = static_cast<float*>(workspace);
  dim3 grid((unsigned)ceil_div(p.m, 64), (unsigned)ceil_div(p.n, 64), splits);
  k_product<T><<<grid, kThreads, 0, st>>>(p, slope_act);
  if (gs_status s = gs::check_launch(where)) return s;
  if (splits > 1) {
    k_product_fold<T><<<(unsigned)ceil_div(p.m * p.n, kThreads), kThreads, 0, st>>>(p, splits);
    return gs::check_launch(where);
  }
  return GS_OK;
}

template <typename T>
gs_status run_fwd(const gs_linear_desc* d, const void* x, const void* w, const void* bias, const void* residual, void* y,
                  void* z, void* workspace, cudaStream_t st) {
  Product p{};
  p.a = x, p.am = d->ldx, p.ak = 1;
  p.b = w, p.bn = d->ldw, p.bk = 1;
  p.m = d->rows, p.n = d->out_features, p.k = d->in_features;
  p.act = d->act, p.bias = bias, p.residual = residual, p.ldr = d->ldr;
  p.y = y, p.ldy = d->ldy, p.z = z, p.ldz = d->ldz;
  return run_product<T>(p, GS_ACT_NONE, workspace, st, "gs_linear_fwd");
}

template <typename T>
gs_status run_bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                  void* dbias, void* workspace, cudaStream_t st) {
  const char* where = "gs_linear_bwd";
  if (dx) {
    Product p{};
    p.a = dy, p.am = d->ldy, p.ak = 1, p.az = z, p.azm = d->ldz, p.azk = 1;
    p.b = w, p.bn = 1, p.bk = d->ldw;
    p.m = d->rows, p.n = d->in_features, p.k = d->out_features;
    p.y = dx, p.ldy = d->lddx;
    if (gs_status s = run_product<T>(p, d->act, workspace, st, where)) return s;
  }
  if (dw) {
    Product p{};
    p.a = dy, p.am = 1, p.ak = d->ldy, p.az = z, p.azm = 1, p.azk = d->ldz;
    p.b = x, p.bn = 1, p.bk = d->ldx;
    p.m = d->out_features, p.n = d->in_features, p.k = d->rows;
    p.y = dw, p.ldy = d->lddw;
    if (gs_status s = run_product<T>(p, d->act, workspace, st, where)) return s;
  }
  if (dbias) {
    const int n = d->out_features, parts = bias_parts(d->rows, n);
    float* part = static_cast<float*>(workspace);
    k_bias_grad<T><<<dim3((unsigned)ceil_div(n, 32), parts), kThreads, 0, st>>>(
        (const T*)dy, (const T*)z, d->rows, n, d->ldy, d->ldz, d->act, part);
    if (gs_status s = gs::check_launch(where)) return s;
    k_bias_fold<T><<<(unsigned)ceil_div(n, kThreads), kThreads, 0, st>>>(part, parts, n, (T*)dbias);
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
  return part_bytes(d->rows, d->out_features, d->in_features);
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
  if (d->dtype == GS_F32) return run_fwd<float>(d, x, w, bias, residual, y, z, workspace, gs::as_stream(stream));
  return run_fwd<__nv_bfloat16>(d, x, w, bias, residual, y, z, workspace, gs::as_stream(stream));
}

extern "C" size_t gs_linear_bwd_workspace_size(const gs_linear_desc* d) {
  if (check_desc("gs_linear_bwd_workspace_size", d) || d->rows == 0) return 0;
  const size_t a = part_bytes(d->rows, d->in_features, d->out_features);
  const size_t b = part_bytes(d->out_features, d->in_features, d->rows);
  const size_t c = (size_t)bias_parts(d->rows, d->out_features) * d->out_features * sizeof(float);
  const size_t ab = a > b ? a : b;
  return ab > c ? ab : c;
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
  if (d->dtype == GS_F32) return run_bwd<float>(d, dy, x, w, z, dx, dw, dbias, workspace, st);
  return run_bwd<__nv_bfloat16>(d, dy, x, w, z, dx, dw, dbias, workspace, st);
}
