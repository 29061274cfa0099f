// The linear layer's small calls, where a launch's latency is the cost, on the FP32 pipe.
//
//   forward: a group of lanes per output column reads a weight row once and keeps the sums of eight rows in
//     registers (k_few_fwd); few_takes says for which calls
//   backward of few rows (at most 16): columns of the input gradient summed over slices of the outputs (k_few_dx);
//     the weight gradient as a sum of at most 16 outer products (k_few_dw).  Bound by reading or writing w.
//   backward of narrow layers (64 x 64 at most) over up to 4,864 rows: dz, its column sums, dx and the
//     block's part of dw from one read of dy, z and x (k_small_bwd), then the parts in order; of thin ones (16 x 16)
//     over any number beyond (k_thin_bwd)
// All sums in 32 bits in a fixed order.
#include "small.cuh"

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T>
struct Fwd {
  const T* x;
  const T* w;
  const T* bias;
  const T* residual;
  T* y;
  T* z;
  int64_t ldx, ldw, ldr, ldy, ldz;
  int rows, in, out, act;
};

template <typename T>
__device__ __forceinline__ void finish(const Fwd<T>& p, int r, int n, float v) {
  if (p.bias) v += to_f32<T>(p.bias[n]);
  if (p.z) p.z[r * p.ldz + n] = from_f32<T>(v);
  v = act_value(v, p.act);
  if (p.residual) v += to_f32<T>(p.residual[r * p.ldr + n]);
  p.y[r * p.ldy + n] = from_f32<T>(v);
}

// ---------------------------------------------------------------- few rows
constexpr int kFew = 8;  // rows of a block

// LANES lanes per column, VE elements per lane and step
template <typename T, int VE, int LANES>
__global__ void __launch_bounds__(kThreads) k_few_fwd(const Fwd<T> p) {
  follow();
  using IO = VecIO<T, VE>;
  const int lane = threadIdx.x % LANES, n = (blockIdx.x * kThreads + threadIdx.x) / LANES, r0 = blockIdx.y * kFew;
  const int rows = min(kFew, p.rows - r0);
  float acc[kFew];
#pragma unroll
  for (int r = 0; r < kFew; ++r) acc[r] = 0.f;
  if (n < p.out) {
    const T* w = p.w + n * p.ldw;
    const T* x = p.x + r0 * p.ldx;
#pragma unroll 2
    for (int k = lane * VE; k < p.in; k += LANES * VE) {
      float wf[VE];
      IO::unpack(IO::load(w + k), wf);
#pragma unroll
      for (int r = 0; r < kFew; ++r) {
        if (r >= rows) break;
        float xf[VE];
        IO::unpack(IO::load(x + r * p.ldx + k), xf);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[r] = fmaf(wf[e], xf[e], acc[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kFew; ++r)
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
#pragma unroll
  for (int r = 0; r < kFew; ++r)  // row r by the group's lane r
    if (r == lane && r < rows && n < p.out) finish(p, r0 + r, n, acc[r]);
}

template <typename T>
struct Bwd {
  const T* dy;
  const T* x;
  const T* w;
  const T* z;
  T* dx;
  T* dw;
  T* db;
  int64_t ldy, ldx, ldw, ldz, lddx, lddw;
  int rows, in, out, act;
};

template <typename T>
__device__ __forceinline__ float dz_at(const Bwd<T>& p, int64_t r, int n) {
  const float d = to_f32<T>(p.dy[r * p.ldy + n]);
  return p.z ? d * act_slope(to_f32<T>(p.z[r * p.ldz + n]), p.act) : d;
}

// dx of kFew rows and 4 VE columns: 64 slices of the outputs per block, added over the slices at the end
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads) k_few_dx(const Bwd<T> p) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int kChunk = 512, kSlices = kThreads / 4;
  __shared__ float dz[kFew][kChunk];
  __shared__ float part[kThreads / 32][4][kFew * VE];
  const int tx = threadIdx.x % 4, slice = threadIdx.x / 4, r0 = blockIdx.y * kFew;
  const int rows = min(kFew, p.rows - r0), k = (blockIdx.x * 4 + tx) * VE;
  float acc[kFew][VE];
#pragma unroll
  for (int r = 0; r < kFew; ++r)
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[r][e] = 0.f;
  for (int n0 = 0; n0 < p.out; n0 += kChunk) {
    const int len = min(kChunk, p.out - n0);
    __syncthreads();
    for (int i = threadIdx.x; i < kFew * kChunk; i += kThreads) {
      const int r = i / kChunk, n = i % kChunk;
      dz[r][n] = r < rows && n < len ? dz_at(p, r0 + r, n0 + n) : 0.f;
    }
    __syncthreads();
    if (k < p.in) {
#pragma unroll 4
      for (int n = slice; n < len; n += kSlices) {
        float wf[VE];
        IO::unpack(IO::load(p.w + (int64_t)(n0 + n) * p.ldw + k), wf);
#pragma unroll
        for (int r = 0; r < kFew; ++r)
#pragma unroll
          for (int e = 0; e < VE; ++e) acc[r][e] = fmaf(dz[r][n], wf[e], acc[r][e]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kFew; ++r)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) acc[r][e] += __shfl_xor_sync(0xffffffffu, acc[r][e], o);
      if ((threadIdx.x & 31) < 4) part[threadIdx.x / 32][tx][r * VE + e] = acc[r][e];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * kFew * VE; i += kThreads) {
    const int t = i / (kFew * VE), r = i / VE % kFew, e = i % VE, col = (blockIdx.x * 4 + t) * VE + e;
    if (r >= rows || col >= p.in) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += part[w][t][r * VE + e];
    p.dx[(r0 + r) * p.lddx + col] = from_f32<T>(v);
  }
}

// dw of 32 outputs x 32 VE inputs, and their bias gradient in the first block across
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads) k_few_dw(const Bwd<T> p) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int kRows = 2 * kFew, kOut = 32, kPer = kOut / (kThreads / 32);
  __shared__ float dz[kRows][kOut];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n0 = blockIdx.y * kOut, k = (blockIdx.x * 32 + lane) * VE;
  for (int i = threadIdx.x; i < kRows * kOut; i += kThreads) {
    const int r = i / kOut, n = n0 + i % kOut;
    dz[r][i % kOut] = r < p.rows && n < p.out ? dz_at(p, r, n) : 0.f;
  }
  __syncthreads();
  if (p.db && blockIdx.x == 0 && threadIdx.x < kOut && n0 + threadIdx.x < p.out) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) v += dz[r][threadIdx.x];
    p.db[n0 + threadIdx.x] = from_f32<T>(v);
  }
  if (!p.dw || k >= p.in) return;
  float acc[kPer][VE];
#pragma unroll
  for (int j = 0; j < kPer; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[j][e] = 0.f;
#pragma unroll 4
  for (int r = 0; r < p.rows; ++r) {
    float xf[VE];
    IO::unpack(IO::load(p.x + r * p.ldx + k), xf);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[j][e] = fmaf(dz[r][warp * kPer + j], xf[e], acc[j][e]);
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (n0 + warp * kPer + j < p.out) IO::store(p.dw + (int64_t)(n0 + warp * kPer + j) * p.lddw + k, acc[j]);
}

// ---------------------------------------------------------------- narrow layers
constexpr int kTileR = 32;
constexpr int kNarrow = 64;

// parts: [gridDim.x][kNarrow + 1][kNarrow], the bias gradient's in the last row
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_small_bwd(const Bwd<T> p, float* parts) {
  follow();
  __shared__ float dz[kTileR][kNarrow + 1], xs[kTileR][kNarrow + 1], ws[kNarrow][kNarrow + 1];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16, c = tid % kNarrow, rr = tid / kNarrow;
  float aw[4][4] = {}, ab = 0.f;
  if (p.dx) {
#pragma unroll
    for (int i = 0; i < kNarrow * kNarrow / kThreads; ++i) {
      const int n = rr + i * (kThreads / kNarrow);
      ws[n][c] = n < p.out && c < p.in ? to_f32<T>(p.w[n * p.ldw + c]) : 0.f;
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kTileR; r0 < p.rows; r0 += (int64_t)gridDim.x * kTileR) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileR * kNarrow / kThreads; ++i) {
      const int r = rr + i * (kThreads / kNarrow);
      const bool in = r0 + r < p.rows;
      dz[r][c] = in && c < p.out ? dz_at(p, r0 + r, c) : 0.f;
      xs[r][c] = p.x && in && c < p.in ? to_f32<T>(p.x[(r0 + r) * p.ldx + c]) : 0.f;
    }
    __syncthreads();
    if (p.dx) {
      float acc[2][4] = {};
#pragma unroll 8
      for (int n = 0; n < kNarrow; ++n) {
        float a[2], b[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = dz[ty + 16 * i][n];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = ws[n][tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r0 + ty + 16 * i < p.rows && tx + 16 * j < p.in)
            p.dx[(r0 + ty + 16 * i) * p.lddx + tx + 16 * j] = from_f32<T>(acc[i][j]);
    }
#pragma unroll 8
    for (int r = 0; r < kTileR; ++r) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = dz[r][ty + 16 * i], b[i] = xs[r][tx + 16 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) aw[i][j] = fmaf(a[i], b[j], aw[i][j]);
    }
    if (tid < kNarrow) {
#pragma unroll 8
      for (int r = 0; r < kTileR; ++r) ab += dz[r][tid];
    }
  }
  float* out = parts + (int64_t)blockIdx.x * (kNarrow + 1) * kNarrow;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) out[(ty + 16 * i) * kNarrow + tx + 16 * j] = aw[i][j];
  if (tid < kNarrow) out[kNarrow * kNarrow + tid] = ab;
}

// Thin layers (16 x 16 at most) over any number of rows: 256 rows of dz and x at a time in shared memory, in which a
// thread owns an entry of dw, then a row of dx.  parts as above; of a row only the first `in` are written.
constexpr int kThin = 16;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_thin_bwd(const Bwd<T> p, float* parts) {
  follow();
  __shared__ float dz[kThreads][kThin + 1], xs[kThreads][kThin + 1], ws[kThin][kThin];
  const int tid = threadIdx.x, n = tid / kThin, c = tid % kThin;
  const bool own = n < p.out && c < p.in;
  if (p.dx) ws[n][c] = own ? to_f32<T>(p.w[n * p.ldw + c]) : 0.f;
  float aw = 0.f, ab = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * kThreads; r0 < p.rows; r0 += (int64_t)gridDim.x * kThreads) {
    const int m = p.rows - r0 < kThreads ? (int)(p.rows - r0) : kThreads;
    __syncthreads();
#pragma unroll 4
    for (int e = tid; e < kThreads * p.out; e += kThreads) {
      const int r = e / p.out, k = e - r * p.out;
      dz[r][k] = r < m ? dz_at(p, r0 + r, k) : 0.f;
    }
    if (p.x) {
#pragma unroll 4
      for (int e = tid; e < kThreads * p.in; e += kThreads) {
        const int r = e / p.in, k = e - r * p.in;
        xs[r][k] = r < m ? to_f32<T>(p.x[(r0 + r) * p.ldx + k]) : 0.f;
      }
    }
    __syncthreads();
    if (own && p.x) {
#pragma unroll 8
      for (int r = 0; r < kThreads; ++r) aw = fmaf(dz[r][n], xs[r][c], aw);
    }
    if (tid < p.out) {
#pragma unroll 8
      for (int r = 0; r < kThreads; ++r) ab += dz[r][tid];
    }
    if (!p.dx) continue;
    __syncthreads();
    float acc[kThin] = {};
    for (int k = 0; k < p.out; ++k) {
      const float d = dz[tid][k];
#pragma unroll
      for (int j = 0; j < kThin; ++j) acc[j] = fmaf(d, ws[k][j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < kThin; ++j) xs[tid][j] = acc[j];
    __syncthreads();
#pragma unroll 4
    for (int e = tid; e < m * p.in; e += kThreads) {
      const int r = e / p.in, k = e - r * p.in;
      p.dx[(r0 + r) * p.lddx + k] = from_f32<T>(xs[r][k]);
    }
  }
  float* out = parts + (int64_t)blockIdx.x * (kNarrow + 1) * kNarrow;
  if (own) out[n * kNarrow + c] = aw;
  if (tid < p.out) out[kNarrow * kNarrow + tid] = ab;
}

// a row of dw (or, last, db) per block: 64 columns by 4 interleaved sets of parts
template <typename T>
__global__ void __launch_bounds__(kThreads) k_small_bwd_fold(const float* parts, int n_parts, int in, int out, T* dw, int64_t lddw,
                                                             T* db) {
  follow();
  __shared__ float s[4][kNarrow];
  const int c = threadIdx.x % kNarrow, way = threadIdx.x / kNarrow, row = blockIdx.x < out ? blockIdx.x : kNarrow;
  float v = 0.f;
#pragma unroll 8
  for (int i = way; i < n_parts; i += 4) v += parts[((int64_t)i * (kNarrow + 1) + row) * kNarrow + c];
  s[way][c] = v;
  __syncthreads();
  if (way) return;
  v = ((s[0][c] + s[1][c]) + s[2][c]) + s[3][c];
  if (row < kNarrow) {
    if (dw && c < in) dw[row * lddw + c] = from_f32<T>(v);
  } else if (db && c < out) {
    db[c] = from_f32<T>(v);
  }
}

// ---------------------------------------------------------------- host side
constexpr int kFewRows = 2 * kFew;
constexpr int kNarrowRows = 152 * kTileR;  // one tile of k_small_bwd per block

bool vec_ok(const void* p, int64_t rows, int64_t ld, int width, int32_t dtype) {
  return width % (16 / (int)gs::dtype_size(dtype)) == 0 && gs::rows_aligned16(p, rows, ld, dtype);
}

int small_bwd_grid(const gs_linear_desc* d) {
  const bool thin = d->rows > kNarrowRows;
  const int64_t tiles = ceil_div(d->rows, thin ? kThreads : kTileR), most = thin ? 4 * 152 : 152;
  return (int)(tiles < most ? tiles : most);
}

// Whether 16-byte vectors lie whole in every row of [rows][width] matrices `ld` apart, by what the descriptor says.
bool whole(int64_t rows, int64_t ld, int width, int32_t dtype) {
  const int ve = 16 / (int)gs::dtype_size(dtype);
  return width % ve == 0 && (rows <= 1 || ld % ve == 0);
}

// Whether a backward of at most 16 rows is the plain kernels', of which k_few_dx walks over all outputs for eight rows at a
// time, and not the tensor cores'.  Alone, in us, here and there:
//   float32          256 -> 256, 16 rows: 13, 21; 1024 -> 1024, 16: 22, 23; 4096 -> 1024, 8: 25, 31, 16: 39, 31; 1024 -> 4096, 1: 27, 30,
//                    4: 37, 29; 8192 -> 64, 8: 17, 19, 16: 25, 19; off 16-byte rows 145 -> 952, 16: 19, 26; 60 -> 2001, 4: 21, 23, 8: 29, 23
//   bfloat16 by TMA  256 -> 256, 16: 14, 19; 1024 -> 1024, 2: 16, 17, 8: 21, 17; 1024 -> 4096, 1: 29, 19; 8 -> 1016, 2: 15, 15, 8: 20, 15;
//                    8192 -> 64, 1: 13, 15, 8: 17, 14
//   others           145 -> 952, 16: 19, 23; 2047 -> 100, 16: 17, 20; 60 -> 2001, 4: 20, 21, 8: 27, 21
bool few_bwd_takes(const gs_linear_desc* d) {
  const bool tma = d->in_features % (16 / (int)gs::dtype_size(d->dtype)) == 0 && whole(d->rows, d->ldy, d->out_features, d->dtype);
  const int64_t deep = (d->rows < kFew ? d->rows : kFew) * d->out_features, across = d->rows * d->in_features;
  const int64_t work = across * d->out_features;
  if (d->dtype == GS_F32)
    return deep <= (tma ? 8192 : 12288) && work <= (1 << 25) && (d->rows <= kFew || d->in_features <= 4096);
  return tma ? deep <= 2048 && across <= 16384 && d->in_features <= 8192 : deep <= 8192 && work <= (1 << 23);
}

// Whether k_few_fwd takes a forward call, and not the tensor cores.  It takes 2.6 us and 0.24 us for each step of a lane,
// a vector of w against one of its rows, while no more than four blocks are on an SM (independent calls: 64 rows of
// 64 -> 64 float32 4.9, 256 -> 256 6.9, 16 rows of 1024 -> 1024 14.7).  The tensor cores' products take
//   float32               7 to 10 us (8.2, 10.5 and 9.6 for the same layers), 11 from 4096 inputs on
//     off 16-byte rows    10 to 13 (255 -> 257: 4 rows 9.0 here, 10.6 there, 8 rows 14.3 and 10.8)
//   bfloat16 by TMA       3 to 4, 7 from 1024 inputs on (256 -> 256: 16 rows 5.0 and 4.1, 1 row 2.1 and 3.9)
//     others              5.5 with few inputs, else 7 to 10 (9 -> 5: 512 rows 3.9 and 5.3; 60 -> 64: 16 rows 7.5 and 5.8; 236 -> 23: 2 rows
//                         5.1 and 7.4, 8 rows 13.4 and 7.9)
// and where there are more blocks (float32 64 -> 64: 512 rows 5.7 and 8.6, 1,024 rows 9.8 and 8.7) they take the call.
// Of eight rows at most w is read once, and a float32 product of many columns has fewer blocks on the tensor cores than
// here (2048 -> 16384: 8 rows 97 and 117, 16 rows 208 and 116; 8192 -> 8192: 1 row 75 and 95, 4 rows 200 and 95).
bool few_takes(const gs_linear_desc* d) {
  const int ve = 16 / (int)gs::dtype_size(d->dtype);
  const bool vec = whole(d->rows, d->ldx, d->in_features, d->dtype) && whole(d->out_features, d->ldw, d->in_features, d->dtype);
  const bool tma = vec && whole(d->rows, d->ldy, d->out_features, d->dtype);
  const int lanes = vec && d->in_features <= 8 * ve ? 8 : 32;
  const int64_t groups = ceil_div(d->rows, kFew), blocks = groups * ceil_div((int64_t)d->out_features * lanes, kThreads);
  const int64_t steps = (d->rows < kFew ? d->rows : kFew) * ceil_div(d->in_features, lanes * (vec ? ve : 1));
  if (d->dtype == GS_F32 && groups == 1 && d->out_features >= 8192) return steps <= 128;
  int64_t most;
  if (d->dtype == GS_F32) most = tma ? 16 + d->in_features / 128 : 40;
  else most = tma ? 4 + d->in_features / 128 : d->in_features < 192 ? 8 + d->in_features / 8 : 32;
  return d->in_features <= 4096 && steps <= most && blocks <= 4 * 152;
}

template <typename T>
gs_status fwd(const gs_linear_desc* d, const void* x, const void* w, const void* bias, const void* residual, void* y, void* z,
              cudaStream_t st, const char* where) {
  const Fwd<T> p{(const T*)x, (const T*)w, (const T*)bias, (const T*)residual, (T*)y, (T*)z,
                 d->ldx, d->ldw, d->ldr, d->ldy, d->ldz, (int)d->rows, d->in_features, d->out_features, d->act};
  constexpr int VE = 16 / sizeof(T);
  const unsigned groups = (unsigned)ceil_div(d->rows, kFew);
  const bool vec = vec_ok(x, d->rows, d->ldx, d->in_features, d->dtype) &&
                   vec_ok(w, d->out_features, d->ldw, d->in_features, d->dtype);
  auto grid = [&](int lanes) { return dim3((unsigned)ceil_div((int64_t)d->out_features * lanes, kThreads), groups); };
  if (!vec) gs::launch(k_few_fwd<T, 1, 32>, grid(32), kThreads, 0, st, p);
  else if (d->in_features <= 8 * VE) gs::launch(k_few_fwd<T, VE, 8>, grid(8), kThreads, 0, st, p);
  else gs::launch(k_few_fwd<T, VE, 32>, grid(32), kThreads, 0, st, p);
  return gs::check_launch(where);
}

template <typename T>
gs_status bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
              void* dbias, void* workspace, cudaStream_t st, const char* where) {
  // x is read for dw alone
  const Bwd<T> p{(const T*)dy, dw ? (const T*)x : nullptr, (const T*)w, (const T*)z, (T*)dx, (T*)dw, (T*)dbias,
                 d->ldy, d->ldx, d->ldw, d->ldz, d->lddx, d->lddw, (int)d->rows, d->in_features, d->out_features, d->act};
  constexpr int VE = 16 / sizeof(T);
  if (d->rows <= kFewRows) {
    if (dx) {
      const bool vec = vec_ok(w, d->out_features, d->ldw, d->in_features, d->dtype);
      const dim3 grid((unsigned)ceil_div(d->in_features, 4 * (vec ? VE : 1)), (unsigned)ceil_div(d->rows, kFew));
      if (vec) gs::launch(k_few_dx<T, VE>, grid, kThreads, 0, st, p);
      else gs::launch(k_few_dx<T, 1>, grid, kThreads, 0, st, p);
      if (gs_status s = gs::check_launch(where)) return s;
    }
    if (dw || dbias) {
      const bool vec = !dw || (vec_ok(x, d->rows, d->ldx, d->in_features, d->dtype) &&
                               vec_ok(dw, d->out_features, d->lddw, d->in_features, d->dtype));
      const dim3 grid(dw ? (unsigned)ceil_div(d->in_features, 32 * (vec ? VE : 1)) : 1, (unsigned)ceil_div(d->out_features, 32));
      gs::launch(vec ? k_few_dw<T, VE> : k_few_dw<T, 1>, grid, kThreads, 0, st, p);
    }
    return gs::check_launch(where);
  }
  const int grid = small_bwd_grid(d);
  float* parts = static_cast<float*>(workspace);
  // only when the kernel before it is done, as k_act_grad (2,048 x 64 f32: 12.3 us, 13.2 with gs::launch)
  if (d->rows > kNarrowRows) k_thin_bwd<T><<<grid, kThreads, 0, st>>>(p, parts);
  else k_small_bwd<T><<<grid, kThreads, 0, st>>>(p, parts);
  if (gs_status s = gs::check_launch(where)) return s;
  if (!dw && !dbias) return GS_OK;
  gs::launch(k_small_bwd_fold<T>, dim3(d->out_features + 1), kThreads, 0, st, (const float*)parts, grid,
             (int)d->in_features, (int)d->out_features, (T*)dw, (int64_t)d->lddw, (T*)dbias);
  return gs::check_launch(where);
}

}  // namespace

namespace gs {

bool small_fwd_takes(const gs_linear_desc* d) {
  return few_takes(d);
}
gs_status small_fwd(const gs_linear_desc* d, const void* x, const void* w, const void* bias, const void* residual, void* y,
                    void* z, cudaStream_t st, const char* where) {
  return d->dtype == GS_F32 ? fwd<float>(d, x, w, bias, residual, y, z, st, where)
                            : fwd<bf16>(d, x, w, bias, residual, y, z, st, where);
}

bool small_bwd_takes(const gs_linear_desc* d) {
  if (d->rows <= kFewRows) return few_bwd_takes(d);
  // (By what every call reads: which outputs are wanted, and their strides, must not change the sums' order.)
  const bool vectors = d->dtype == GS_BF16 && d->in_features % 8 == 0 && d->out_features % 8 == 0 && d->ldy % 8 == 0 &&
                       (d->act == GS_ACT_NONE || d->ldz % 8 == 0);
  // A round of tiles takes k_small_bwd 9 to 11 us whatever the layer; two rounds take as long as the tensor cores (64 -> 64
  // float32: 4,096 rows 11.5 us here, 17.8 there; 8,192 rows 19.4 and 19.0; 32,768 rows 88 and 28), but for bfloat16
  // layers of 16-byte vectors, which mma_grad.cu passes over as fast from the start (64 -> 64: 512 rows 11.2 and 10.0;
  // 2,048 rows 10.9 and 11.5; 4,096 rows 12.2 and 10.8).
  if (d->rows <= kNarrowRows) return d->in_features <= kNarrow && d->out_features <= kNarrow && !vectors;
  // Thin layers over more rows, for which the tensor cores' tiles are nearly empty (GELU, 3M rows: 9 -> 5 bfloat16 254 us
  // here, 808 there; float32 8 -> 8 292 and 709, 16 -> 16 516 and 734; from 8,192 rows on: 16 -> 16 14.9 and 16.3); of the
  // vectors of bfloat16 only the narrowest (8 -> 8 285 and 335; 8 -> 16 444 and 332; 16 -> 16 506 and 279).
  return d->in_features <= kThin && d->out_features <= kThin && !(vectors && d->in_features * d->out_features > 64);
}
size_t small_bwd_workspace(const gs_linear_desc* d) {
  return d->rows <= kFewRows ? 0 : (size_t)small_bwd_grid(d) * (kNarrow + 1) * kNarrow * sizeof(float);
}
gs_status small_bwd(const gs_linear_desc* d, const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                    void* dbias, void* workspace, cudaStream_t st, const char* where) {
  return d->dtype == GS_F32 ? bwd<float>(d, dy, x, w, z, dx, dw, dbias, workspace, st, where)
                            : bwd<bf16>(d, dy, x, w, z, dx, dw, dbias, workspace, st, where);
}

}  // namespace gs
