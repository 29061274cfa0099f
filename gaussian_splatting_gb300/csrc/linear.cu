// The linear layer y = act(x w^T + bias) + residual and its gradient (gs_linear_fwd, gs_linear_bwd).
//
// Three products share one kernel, C(m, n) = sum over k of A(m, k) B(n, k) with A and B given by
// their two strides:
//   forward  z  = x w^T    A = x,  B = w
//   dx       dx = dz w     A = dz, B = w read along its other axis
//   dw       dw = dz^T x   A = dz and x both read along their other axes
// with dz = dy act'(z) formed as its elements are loaded.
#include "mma.cuh"

namespace {

constexpr int kThreads = 256;

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

// dz = dy act'(z) to `dz` (if wanted), and its column sums over this block's rows to part[blockIdx.x].
// A thread owns VE columns; CX threads lie along a row, kThreads / CX rows side by side.
template <typename T, bool VEC, int CX>
__global__ void __launch_bounds__(kThreads) k_act_grad(const T* dy, const T* z, int64_t rows, int n, int64_t lddy,
                                                       int64_t ldz, int act, T* dz, int64_t lddz, float* part) {
  constexpr int VE = 16 / sizeof(T), kRows = kThreads / CX;
  using IO = VecIO<T, VE>;
  const int cx = threadIdx.x % CX, ry = threadIdx.x / CX;
  const int c = (blockIdx.y * CX + cx) * VE;
  const bool in = c < n;
  float sum[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) sum[e] = 0.f;
  if (in) {
#pragma unroll 2
    for (int64_t r = (int64_t)blockIdx.x * kRows + ry; r < rows; r += (int64_t)gridDim.x * kRows) {
      float d[VE], v[VE];
      if (VEC) {
        const auto rd = IO::load(dy + r * lddy + c);
        if (z) {
          const auto rz = IO::load(z + r * ldz + c);
          IO::unpack(rz, v);
        }
        IO::unpack(rd, d);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          d[e] = c + e < n ? to_f32<T>(dy[r * lddy + c + e]) : 0.f;
          v[e] = z && c + e < n ? to_f32<T>(z[r * ldz + c + e]) : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if (z) d[e] *= act_slope(v[e], act);
        sum[e] += d[e];
      }
      if (dz) IO::store(dz + r * lddz + c, d);
    }
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

template <typename T>
__global__ void __launch_bounds__(kThreads) k_bias_fold(const float* part, int parts, int n, T* out) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < n)
    for (int p = w; p < parts; p += 8) v += part[(int64_t)p * n + c];
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < n) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][lane];
    out[c] = from_f32<T>(v);
  }
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
  int64_t s = ceil_div(8 * 152, across);
  const int64_t most = ceil_div(rows, 4 * (kThreads / cx));
  return (int)(s < most ? s : most);
}
int parts_of(const gs_linear_desc* d) {
  return d->dtype == GS_F32 ? act_grad_parts<float>(d->rows, d->out_features)
                            : act_grad_parts<__nv_bfloat16>(d->rows, d->out_features);
}

template <typename T>
gs_status run_act_grad(const gs_linear_desc* d, const T* dy, const T* z, T* dz, int64_t lddz, float* part, T* dbias,
                       cudaStream_t st, const char* where) {
  const int n = d->out_features, parts = act_grad_parts<T>(d->rows, n);
  const bool vec = gs::rows_aligned16(dy, d->rows, d->ldy, d->dtype) && n % (16 / sizeof(T)) == 0 &&
                   (!z || gs::rows_aligned16(z, d->rows, d->ldz, d->dtype));
  const int cx = row_threads<T>(n);
  const dim3 grid(parts, (unsigned)ceil_div(n, cx * (16 / (int64_t)sizeof(T))));
#define GS_GO(V, CX)                                                                                                  \
  k_act_grad<T, V, CX><<<grid, kThreads, 0, st>>>(dy, z, d->rows, n, d->ldy, d->ldz, d->act, dz, lddz, dbias ? part : nullptr)
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
  if (gs_status s = gs::check_launch(where)) return s;
  if (!dbias) return GS_OK;
  k_bias_fold<T><<<(unsigned)ceil_div(n, 32), kThreads, 0, st>>>(part, parts, n, dbias);
  return gs::check_launch(where);
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
                  void* z, void* workspace, int32_t* status, cudaStream_t st) {
  if (d->dtype == GS_BF16) {
    const gs::MmaProduct q{x, w, d->ldx, d->ldw, false, false, d->rows, d->out_features, d->in_features,
                           bias, residual, y, z, d->ldr, d->ldy, d->ldz, d->act};
    if (gs::mma_takes(q)) return gs::mma_run(q, workspace, status, st, "gs_linear_fwd");
  }
  Product p{};
  p.a = x, p.am = d->ldx, p.ak = 1;
  p.b = w, p.bn = d->ldw, p.bk = 1;
  p.m = d->rows, p.n = d->out_features, p.k = d->in_features;
  p.act = d->act, p.bias = bias, p.residual = residual, p.ldr = d->ldr;
  p.y = y, p.ldy = d->ldy, p.z = z, p.ldz = d->ldz;
  return run_product<T>(p, GS_ACT_NONE, workspace, st, "gs_linear_fwd");
}

// The backward's scratch: dz where the products read a copy of it (bfloat16: after an activation, or where
// dy's rows do not start on 16-byte boundaries), the bias gradient's parts, the products' parts.
struct BwdSpace {
  size_t dz, bias, part, total;
  int64_t lddz;
};
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
BwdSpace bwd_space(const gs_linear_desc* d) {
  BwdSpace s{};
  s.lddz = ceil_div(d->out_features, 8) * 8;
  const bool copy = d->dtype == GS_BF16 && (d->act != GS_ACT_NONE || (d->ldy * 2) % 16 != 0);
  s.dz = copy ? up256((size_t)d->rows * s.lddz * 2) : 0;
  s.bias = up256((size_t)parts_of(d) * d->out_features * sizeof(float));
  auto most = [](size_t a, size_t b) { return a > b ? a : b; };
  s.part = most(part_bytes(d->rows, d->in_features, d->out_features), part_bytes(d->out_features, d->in_features, d->rows));
  if (d->dtype == GS_BF16)
    s.part = most(s.part, most(gs::mma_workspace(d->rows, d->in_features, d->out_features),
                               gs::mma_workspace(d->out_features, d->in_features, d->rows)));
  s.total = s.dz + s.bias + s.part;
  return s;
}

template <typename T>
gs_status run_bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                  void* dbias, void* workspace, int32_t* status, cudaStream_t st) {
  const char* where = "gs_linear_bwd";
  const BwdSpace space = bwd_space(d);
  unsigned char* at = static_cast<unsigned char*>(workspace);
  T* dz_copy = space.dz ? reinterpret_cast<T*>(at) : nullptr;
  float* bias_part = reinterpret_cast<float*>(at + space.dz);
  void* part = at + space.dz + space.bias;
  const void* dz = dz_copy ? dz_copy : dy;
  const int64_t lddz = dz_copy ? space.lddz : d->ldy;
  gs::MmaProduct qx{}, qw{};
  bool mx = false, mw = false;
  if (d->dtype == GS_BF16) {
    if (dx) {
      qx = {dz, w, lddz, d->ldw, false, true, d->rows, d->in_features, d->out_features,
            nullptr, nullptr, dx, nullptr, 0, d->lddx, 0, GS_ACT_NONE};
      mx = gs::mma_takes(qx);
    }
    if (dw) {
      qw = {dz, x, lddz, d->ldx, true, true, d->out_features, d->in_features, d->rows,
            nullptr, nullptr, dw, nullptr, 0, d->lddw, 0, GS_ACT_NONE};
      mw = gs::mma_takes(qw);
    }
  }
  T* write_dz = dz_copy && (mx || mw) ? dz_copy : nullptr;
  if (write_dz || dbias)
    if (gs_status s = run_act_grad<T>(d, static_cast<const T*>(dy), static_cast<const T*>(z), write_dz, lddz, bias_part,
                                      static_cast<T*>(dbias), st, where))
      return s;
  if (mx)
    if (gs_status s = gs::mma_run(qx, part, status, st, where)) return s;
  if (mw)
    if (gs_status s = gs::mma_run(qw, part, status, st, where)) return s;
  if (dx && !mx) {
    Product p{};
    p.a = dy, p.am = d->ldy, p.ak = 1, p.az = z, p.azm = d->ldz, p.azk = 1;
    p.b = w, p.bn = 1, p.bk = d->ldw;
    p.m = d->rows, p.n = d->in_features, p.k = d->out_features;
    p.y = dx, p.ldy = d->lddx;
    if (gs_status s = run_product<T>(p, d->act, part, st, where)) return s;
  }
  if (dw && !mw) {
    Product p{};
    p.a = dy, p.am = 1, p.ak = d->ldy, p.az = z, p.azm = 1, p.azk = d->ldz;
    p.b = x, p.bn = 1, p.bk = d->ldx;
    p.m = d->out_features, p.n = d->in_features, p.k = d->rows;
    p.y = dw, p.ldy = d->lddw;
    if (gs_status s = run_product<T>(p, d->act, part, st, where)) return s;
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
  const size_t a = part_bytes(d->rows, d->out_features, d->in_features);
  const size_t b = d->dtype == GS_BF16 ? gs::mma_workspace(d->rows, d->out_features, d->in_features) : 0;
  return a > b ? a : b;
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
  if (d->dtype == GS_F32) return run_fwd<float>(d, x, w, bias, residual, y, z, workspace, status, gs::as_stream(stream));
  return run_fwd<__nv_bfloat16>(d, x, w, bias, residual, y, z, workspace, status, gs::as_stream(stream));
}

extern "C" size_t gs_linear_bwd_workspace_size(const gs_linear_desc* d) {
  if (check_desc("gs_linear_bwd_workspace_size", d) || d->rows == 0) return 0;
  return bwd_space(d).total;
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
  if (d->dtype == GS_F32) return run_bwd<float>(d, dy, x, w, z, dx, dw, dbias, workspace, status, st);
  return run_bwd<__nv_bfloat16>(d, dy, x, w, z, dx, dw, dbias, workspace, status, st);
}
