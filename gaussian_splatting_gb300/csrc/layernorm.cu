// Layer normalisation over the rows of a strided matrix, forward and backward
// (gs_layernorm_fwd, gs_layernorm_bwd).
//
// Mathematics, for a row x of `width` values:
//   forward   mean = sum(x) / width, var = sum((x - mean)^2) / width, rstd = (var + eps)^-1/2,
//             h = (x - mean) rstd, y = h gamma + beta
//   backward  g = dy gamma, dx = rstd (g - mean(g) - h mean(g h)) + skip,
//             dgamma = sum over rows of dy h, dbeta = sum over rows of dy
// All of it in 32 bits whatever the element type, rounded once when stored.
//
// Both directions are bound by memory (about 8 and 14 operations per element against 4 to 16
// bytes), so every array is read once and written once: a row stays in the registers of the G
// threads that own it (G = 8 to 32 lanes of a warp, or a block of 256 threads for wide rows)
// between the sums and the output, which also lets the variance be taken about the mean itself
// instead of as E[x^2] - mean^2 (no cancellation when the mean is large).  The backward's two
// column sums are kept in the registers of the threads that own the columns over all rows of a
// persistent block, folded over the block's warps in shared memory, written as one partial row
// per block and added up by a second kernel in block order: no atomics, the same bits each run.
#include "dense.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct FwdArgs {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, ldx, ldy;
  int width;
  float eps;
};

struct BwdArgs {
  const void* dy;
  const void* x;
  const void* gamma;
  const float* mean;
  const float* rstd;
  const void* skip;
  void* dx;
  float* partials;  // [gridDim.x][2][width], or NULL when neither column sum is wanted
  int64_t rows, lddy, ldx, ldskip, lddx;
  int width;
};

// Sums over the G threads that share a row.  A sum over several warps alternates between two buffers,
// so that one barrier per sum is enough.
__shared__ float2 s_fold[2][kWarps];
template <int G>
struct RowSum {
  int turn = 0;
  __device__ __forceinline__ void operator()(float& a, float& b) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (G > 32) {
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) s_fold[turn][warp] = make_float2(a, b);
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int w = 0; w < G / 32; ++w) {
        const float2 f = s_fold[turn][warp / (G / 32) * (G / 32) + w];
        a += f.x, b += f.y;
      }
      turn ^= 1;
    }
  }
};

// G threads per row, IT vectors of VE elements per thread, U rows in flight per thread.
template <typename T, int VE, int G, int IT, int U>
__global__ void __launch_bounds__(kThreads) k_layernorm_fwd(const FwdArgs a) {
  using IO = VecIO<T, VE>;
  constexpr int kRows = kThreads / G;  // rows a block takes side by side
  const int lane = threadIdx.x % G, sub = threadIdx.x / G;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  typename IO::Raw rg[IT], rb[IT];
  bool in[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (lane + i * G) * VE;
    in[i] = c < a.width;
    rg[i] = in[i] ? IO::load(static_cast<const T*>(a.gamma) + c) : IO::zero();
    rb[i] = in[i] ? IO::load(static_cast<const T*>(a.beta) + c) : IO::zero();
  }
  const float inv = 1.f / (float)a.width;
  RowSum<G> sum;
  for (int64_t r0 = (int64_t)blockIdx.x * (kRows * U); r0 < a.rows; r0 += (int64_t)gridDim.x * (kRows * U)) {
    typename IO::Raw rx[U][IT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * kRows + sub;
#pragma unroll
      for (int i = 0; i < IT; ++i)
        rx[u][i] = in[i] && r < a.rows ? IO::load(x + r * a.ldx + (lane + i * G) * VE) : IO::zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * kRows + sub;
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float f[VE];
        IO::unpack(rx[u][i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) s += f[e];  // values beyond the width are zero
      }
      sum(s, q);
      const float mean = __fmul_rn(s, inv);  // the value that is stored: not folded into the differences below
      q = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float f[VE];
        IO::unpack(rx[u][i], f);
        if (in[i]) {
#pragma unroll
          for (int e = 0; e < VE; ++e) q = fmaf(f[e] - mean, f[e] - mean, q);
        }
      }
      s = 0.f;
      sum(q, s);
      const float rstd = 1.f / sqrtf(q * inv + a.eps);
      if (r < a.rows) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          if (!in[i]) continue;
          float f[VE], g[VE], b[VE];
          IO::unpack(rx[u][i], f);
          IO::unpack(rg[i], g);
          IO::unpack(rb[i], b);
#pragma unroll
          for (int e = 0; e < VE; ++e) f[e] = fmaf((f[e] - mean) * rstd, g[e], b[e]);
          IO::store(y + r * a.ldy + (lane + i * G) * VE, f);
        }
        if (lane == 0) {
          if (a.mean) a.mean[r] = mean;
          if (a.rstd) a.rstd[r] = rstd;
        }
      }
    }
  }
}

// Rows wider than a block's registers: one block per row, the row read again for each sum
// (the second and third time mostly from L2).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_layernorm_fwd_wide(const FwdArgs a) {
  const T* gamma = static_cast<const T*>(a.gamma);
  const T* beta = static_cast<const T*>(a.beta);
  const float inv = 1.f / (float)a.width;
  RowSum<kThreads> sum;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    T* y = static_cast<T*>(a.y) + r * a.ldy;
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) s += to_f32<T>(x[c]);
    sum(s, q);
    const float mean = __fmul_rn(s, inv);  // the value that is stored: not folded into the differences below
    q = 0.f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      const float d = to_f32<T>(x[c]) - mean;
      q = fmaf(d, d, q);
    }
    s = 0.f;
    sum(q, s);
    const float rstd = 1.f / sqrtf(q * inv + a.eps);
    for (int c = threadIdx.x; c < a.width; c += kThreads)
      y[c] = from_f32<T>(fmaf((to_f32<T>(x[c]) - mean) * rstd, to_f32<T>(gamma[c]), to_f32<T>(beta[c])));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <typename T, int VE, int G, int IT, int U>
__global__ void __launch_bounds__(kThreads) k_layernorm_bwd(const BwdArgs a) {
  using IO = VecIO<T, VE>;
  constexpr int kRows = kThreads / G;
  const int lane = threadIdx.x % G, sub = threadIdx.x / G;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const T* skip = static_cast<const T*>(a.skip);
  T* dx = static_cast<T*>(a.dx);
  typename IO::Raw rg[IT];
  bool in[IT];
  float ag[IT][VE], ab[IT][VE];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (lane + i * G) * VE;
    in[i] = c < a.width;
    rg[i] = in[i] ? IO::load(static_cast<const T*>(a.gamma) + c) : IO::zero();
#pragma unroll
    for (int e = 0; e < VE; ++e) ag[i][e] = ab[i][e] = 0.f;
  }
  const float inv = 1.f / (float)a.width;
  RowSum<G> sum;
  for (int64_t r0 = (int64_t)blockIdx.x * (kRows * U); r0 < a.rows; r0 += (int64_t)gridDim.x * (kRows * U)) {
    typename IO::Raw rx[U][IT], ry[U][IT], rs[U][IT];
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * kRows + sub;
      const bool ok = r < a.rows;
      mean[u] = ok ? a.mean[r] : 0.f;
      rstd[u] = ok ? a.rstd[r] : 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (lane + i * G) * VE;
        rx[u][i] = in[i] && ok ? IO::load(x + r * a.ldx + c) : IO::zero();
        ry[u][i] = in[i] && ok ? IO::load(dy + r * a.lddy + c) : IO::zero();
        rs[u][i] = in[i] && ok && skip ? IO::load(skip + r * a.ldskip + c) : IO::zero();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * kRows + sub;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float f[VE], d[VE], g[VE];
        IO::unpack(rx[u][i], f);
        IO::unpack(ry[u][i], d);
        IO::unpack(rg[i], g);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float h = (f[e] - mean[u]) * rstd[u], ge = d[e] * g[e];
          s1 += ge;  // beyond the width and the rows dy is zero: nothing is added
          s2 = fmaf(ge, h, s2);
          ag[i][e] = fmaf(d[e], h, ag[i][e]);
          ab[i][e] += d[e];
        }
      }
      sum(s1, s2);
      s1 *= inv;
      s2 *= inv;
      if (dx && r < a.rows) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          if (!in[i]) continue;
          float f[VE], d[VE], g[VE], k[VE];
          IO::unpack(rx[u][i], f);
          IO::unpack(ry[u][i], d);
          IO::unpack(rg[i], g);
          IO::unpack(rs[u][i], k);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float h = (f[e] - mean[u]) * rstd[u];
            f[e] = fmaf(rstd[u], d[e] * g[e] - s1 - h * s2, k[e]);
          }
          IO::store(dx + r * a.lddx + (lane + i * G) * VE, f);
        }
      }
    }
  }
  if (!a.partials) return;
  // fold the column sums over the block's rows: the groups of a warp by shuffles, the warps in
  // shared memory, in a fixed order
  float* out = a.partials + (int64_t)blockIdx.x * 2 * a.width;
#pragma unroll
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        ag[i][e] += __shfl_xor_sync(0xffffffffu, ag[i][e], o);
        ab[i][e] += __shfl_xor_sync(0xffffffffu, ab[i][e], o);
      }
  }
  if constexpr (G == kThreads) {  // a column belongs to one thread
#pragma unroll
    for (int i = 0; i < IT; ++i)
      if (in[i]) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          out[(lane + i * G) * VE + e] = ag[i][e];
          out[a.width + (lane + i * G) * VE + e] = ab[i][e];
        }
      }
  } else {
    // one slot per group of threads that owns all columns: a warp's groups are folded already
    constexpr int kSlots = G < 32 ? kWarps : kRows, kOwners = G;
    __shared__ float fold[kSlots][2][kOwners * VE];
    const int slot = G < 32 ? threadIdx.x >> 5 : sub;
    for (int i = 0; i < IT; ++i) {
      __syncthreads();
      // register arrays are indexed by constants only: the unrolled select keeps them there
#pragma unroll
      for (int j = 0; j < IT; ++j)
        if (j == i && (threadIdx.x & 31) < G) {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            fold[slot][0][lane * VE + e] = ag[j][e];
            fold[slot][1][lane * VE + e] = ab[j][e];
          }
        }
      __syncthreads();
      for (int k = threadIdx.x; k < 2 * G * VE; k += kThreads) {
        const int which = k / (G * VE), e = k % (G * VE), c = i * G * VE + e;
        if (c < a.width) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < kSlots; ++w) s += fold[w][which][e];
          out[which * a.width + c] = s;
        }
      }
    }
  }
}

// Wide rows: as the forward; the block keeps its column sums in its own partial row.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_layernorm_bwd_wide(const BwdArgs a) {
  const T* gamma = static_cast<const T*>(a.gamma);
  float* out = a.partials ? a.partials + (int64_t)blockIdx.x * 2 * a.width : nullptr;
  const float inv = 1.f / (float)a.width;
  RowSum<kThreads> sum;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      const float d = to_f32<T>(dy[c]), h = (to_f32<T>(x[c]) - mean) * rstd, g = d * to_f32<T>(gamma[c]);
      s1 += g;
      s2 = fmaf(g, h, s2);
      if (out) {  // a column belongs to one thread of the block
        const bool first = r == blockIdx.x;
        out[c] = fmaf(d, h, first ? 0.f : out[c]);
        out[a.width + c] = d + (first ? 0.f : out[a.width + c]);
      }
    }
    sum(s1, s2);
    s1 *= inv;
    s2 *= inv;
    if (a.dx) {
      const T* skip = a.skip ? static_cast<const T*>(a.skip) + r * a.ldskip : nullptr;
      T* dx = static_cast<T*>(a.dx) + r * a.lddx;
      for (int c = threadIdx.x; c < a.width; c += kThreads) {
        const float h = (to_f32<T>(x[c]) - mean) * rstd;
        dx[c] = from_f32<T>(fmaf(rstd, to_f32<T>(dy[c]) * to_f32<T>(gamma[c]) - s1 - h * s2,
                                 skip ? to_f32<T>(skip[c]) : 0.f));
      }
    }
  }
}

// out[c] = sum over the partial rows: 32 columns by 32 interleaved sets of rows per block, in order.
template <typename T>
__global__ void __launch_bounds__(1024) k_layernorm_fold(const float* __restrict__ partials, int n_part, int width,
                                                         T* __restrict__ dgamma, T* __restrict__ dbeta) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < 2 * width) {
#pragma unroll 8
    for (int p = warp; p < n_part; p += 32) v += partials[(int64_t)p * 2 * width + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  // warp w: column w of the block
  v = s[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane != 0 || col >= 2 * width) return;
  if (col < width) {
    if (dgamma) dgamma[col] = from_f32<T>(v);
  } else if (dbeta) {
    dbeta[col - width] = from_f32<T>(v);
  }
}

// ---------------------------------------------------------------- host side
// Which form a width takes: G threads per row, IT vectors per thread (0: the wide kernel).
struct Form {
  int vec, g, it;
};

// Forward: a row gets as few threads as hold it in at most four 16-byte vectors (eight single elements)
// each, so that narrow rows keep whole warps busy; beyond a warp's reach a block shares it.
Form fwd_form(int width, bool vec, int32_t dtype) {
  const int ve = vec ? (dtype == GS_F32 ? 4 : 8) : 1;
  const int n = width / ve, most = vec ? 4 : 8;
  for (int g : {8, 16, 32})
    if (n <= g) return {vec, g, 1};
  for (int it = 2; it <= most; it *= 2)
    if (n <= 32 * it) return {vec, 32, it};
  for (int it = 1; it <= (vec ? 4 : 16); it *= 2)
    if (n <= kThreads * it) return {vec, kThreads, it};
  return {vec, kThreads, 0};
}
// Backward: every value a thread holds also has two sums in its registers, so a row is spread over as
// many threads as it has vectors before any thread takes a second one.
Form bwd_form(int width, bool vec, int32_t dtype) {
  const int n = width / (vec ? (dtype == GS_F32 ? 4 : 8) : 1);
  for (int g : {8, 16, 32, 64, 128})
    if (n <= g) return {vec, g, 1};
  for (int it = 1; it <= (vec ? 4 : 16); it *= 2)
    if (n <= kThreads * it) return {vec, kThreads, it};
  return {vec, kThreads, 0};
}

// blocks that fill the device at 8 resident blocks per SM, or fewer when the rows are few
int grid_of(int64_t rows, int rows_per_block, int per_sm) {
  const int64_t need = (rows + rows_per_block - 1) / rows_per_block;
  const int64_t most = (int64_t)gs::num_sms() * per_sm;
  return (int)(need < most ? (need > 0 ? need : 1) : most);
}

constexpr int kFwdPerSm = 8, kBwdPerSm = 4;

template <typename T, int VE, int G, int IT>
void launch_fwd(const FwdArgs& a, cudaStream_t st) {
  constexpr int U = G == kThreads ? 1 : IT == 1 ? 2 : 1;
  k_layernorm_fwd<T, VE, G, IT, U><<<grid_of(a.rows, kThreads / G * U, kFwdPerSm), kThreads, 0, st>>>(a);
}
template <typename T>
void run_fwd(const FwdArgs& a, Form f, cudaStream_t st) {
  constexpr int VE = 16 / sizeof(T);
  if (f.it == 0) {
    k_layernorm_fwd_wide<T><<<grid_of(a.rows, 1, kFwdPerSm), kThreads, 0, st>>>(a);
    return;
  }
  const int key = (f.vec ? 10000 : 0) + f.g * 20 + f.it;
  switch (key) {
#define GS_FORM(v, g, it) \
  case (v ? 10000 : 0) + g * 20 + it: launch_fwd<T, v ? VE : 1, g, it>(a, st); break;
    GS_FORM(1, 8, 1) GS_FORM(1, 16, 1) GS_FORM(1, 32, 1) GS_FORM(1, 32, 2) GS_FORM(1, 32, 4)
    GS_FORM(1, 256, 1) GS_FORM(1, 256, 2) GS_FORM(1, 256, 4)
    GS_FORM(0, 8, 1) GS_FORM(0, 16, 1) GS_FORM(0, 32, 1) GS_FORM(0, 32, 2) GS_FORM(0, 32, 4) GS_FORM(0, 32, 8)
    GS_FORM(0, 256, 2) GS_FORM(0, 256, 4) GS_FORM(0, 256, 8) GS_FORM(0, 256, 16)
#undef GS_FORM
  }
}

template <typename T>
void run_bwd(const BwdArgs& a, Form f, int grid, cudaStream_t st) {
  constexpr int VE = 16 / sizeof(T);
  if (f.it == 0) {
    k_layernorm_bwd_wide<T><<<grid, kThreads, 0, st>>>(a);
    return;
  }
  const int key = (f.vec ? 10000 : 0) + f.g * 20 + f.it;
  switch (key) {
#define GS_FORM(v, g, it) \
  case (v ? 10000 : 0) + g * 20 + it: k_layernorm_bwd<T, v ? VE : 1, g, it, 1><<<grid, kThreads, 0, st>>>(a); break;
    GS_FORM(1, 8, 1) GS_FORM(1, 16, 1) GS_FORM(1, 32, 1) GS_FORM(1, 64, 1) GS_FORM(1, 128, 1)
    GS_FORM(1, 256, 1) GS_FORM(1, 256, 2) GS_FORM(1, 256, 4)
    GS_FORM(0, 8, 1) GS_FORM(0, 16, 1) GS_FORM(0, 32, 1) GS_FORM(0, 64, 1) GS_FORM(0, 128, 1)
    GS_FORM(0, 256, 1) GS_FORM(0, 256, 2) GS_FORM(0, 256, 4) GS_FORM(0, 256, 8) GS_FORM(0, 256, 16)
#undef GS_FORM
  }
}

gs_status check_desc(const char* where, const gs_layernorm_desc* d) {
  if (!d) return gs::set_error(GS_ERR_INVALID, "%s: descriptor is NULL", where);
  if (d->rows < 0 || d->width < 1 || d->width > (1 << 24))
    return gs::set_error(GS_ERR_INVALID, "%s: bad size %lld x %d", where, (long long)d->rows, d->width);
  if (d->dtype != GS_F32 && d->dtype != GS_BF16)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown element type %d", where, d->dtype);
  return GS_OK;
}

// blocks of the backward: the number of partial rows
// (rows too wide for registers: no more than keep the partials within 256 MiB)
int bwd_grid(int64_t rows, Form f, int width) {
  const int g = grid_of(rows, f.it == 0 ? 1 : kThreads / f.g, kBwdPerSm);
  const int fit = (1 << 25) / width;
  return f.it == 0 && g > fit ? fit : g;
}

}  // namespace

extern "C" gs_status gs_layernorm_fwd(const gs_layernorm_desc* d, const void* x, const void* gamma, const void* beta,
                                      void* y, float* mean, float* rstd, void* stream) {
  const char* where = "gs_layernorm_fwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (!(d->eps >= 0.f)) return gs::set_error(GS_ERR_INVALID, "%s: eps must be >= 0", where);
  if (d->rows == 0) return GS_OK;
  if (gs_status s = gs::check_matrix(where, "x", x, d->rows, d->width, d->ldx, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "y", y, d->rows, d->width, d->ldy, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "gamma", gamma, 1, d->width, d->width, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "beta", beta, 1, d->width, d->width, d->dtype)) return s;
  const int ve = 16 / (int)gs::dtype_size(d->dtype);
  const bool vec = d->width % ve == 0 && gs::rows_aligned16(x, d->rows, d->ldx, d->dtype) &&
                   gs::rows_aligned16(y, d->rows, d->ldy, d->dtype) && gs::aligned16(gamma) && gs::aligned16(beta);
  const FwdArgs a{x, gamma, beta, y, mean, rstd, d->rows, d->ldx, d->ldy, d->width, d->eps};
  const Form f = fwd_form(d->width, vec, d->dtype);
  if (d->dtype == GS_F32) run_fwd<float>(a, f, gs::as_stream(stream));
  else run_fwd<__nv_bfloat16>(a, f, gs::as_stream(stream));
  return gs::check_launch(where);
}

extern "C" size_t gs_layernorm_bwd_workspace_size(const gs_layernorm_desc* d) {
  if (!d || d->rows < 0 || d->width < 1 || d->width > (1 << 24)) return 0;
  // the scalar and the vector form need not have the same number of blocks: the larger
  int most = 1;
  for (int vec = 0; vec < 2; ++vec) {
    const int g = bwd_grid(d->rows, bwd_form(d->width, vec, d->dtype), d->width);
    most = g > most ? g : most;
  }
  return sizeof(float) * 2 * (size_t)d->width * most;
}

extern "C" gs_status gs_layernorm_bwd(const gs_layernorm_desc* d, const void* dy, const void* x, const void* gamma,
                                      const float* mean, const float* rstd, const void* skip, void* dx, void* dgamma,
                                      void* dbeta, void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "gs_layernorm_bwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (!dx && !dgamma && !dbeta) return GS_OK;
  const size_t size = gs::dtype_size(d->dtype);
  cudaStream_t st = gs::as_stream(stream);
  if (dgamma && reinterpret_cast<uintptr_t>(dgamma) % size)
    return gs::set_error(GS_ERR_INVALID, "%s: dgamma is misaligned for its type", where);
  if (dbeta && reinterpret_cast<uintptr_t>(dbeta) % size)
    return gs::set_error(GS_ERR_INVALID, "%s: dbeta is misaligned for its type", where);
  if (d->rows == 0) {
    if (dgamma && cudaMemsetAsync(dgamma, 0, size * d->width, st) != cudaSuccess) return gs::check_launch(where);
    if (dbeta && cudaMemsetAsync(dbeta, 0, size * d->width, st) != cudaSuccess) return gs::check_launch(where);
    return GS_OK;
  }
  if (gs_status s = gs::check_matrix(where, "dy", dy, d->rows, d->width, d->lddy, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "x", x, d->rows, d->width, d->ldx, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "gamma", gamma, 1, d->width, d->width, d->dtype)) return s;
  if (skip)
    if (gs_status s = gs::check_matrix(where, "skip", skip, d->rows, d->width, d->ldskip, d->dtype)) return s;
  if (dx)
    if (gs_status s = gs::check_matrix(where, "dx", dx, d->rows, d->width, d->lddx, d->dtype)) return s;
  if (!mean || !rstd) return gs::set_error(GS_ERR_INVALID, "%s: mean or rstd is NULL", where);
  const bool sums = dgamma || dbeta;
  if (sums) {
    const size_t need = gs_layernorm_bwd_workspace_size(d);
    if (!workspace || !gs::aligned16(workspace))
      return gs::set_error(GS_ERR_INVALID, "%s: workspace is NULL or misaligned", where);
    if (workspace_bytes < need)
      return gs::set_error(GS_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", where, workspace_bytes, need);
  }
  const int ve = 16 / (int)size;
  const bool vec = d->width % ve == 0 && gs::rows_aligned16(x, d->rows, d->ldx, d->dtype) &&
                   gs::rows_aligned16(dy, d->rows, d->lddy, d->dtype) && gs::aligned16(gamma) &&
                   (!skip || gs::rows_aligned16(skip, d->rows, d->ldskip, d->dtype)) &&
                   (!dx || gs::rows_aligned16(dx, d->rows, d->lddx, d->dtype));
  const Form f = bwd_form(d->width, vec, d->dtype);
  const int grid = bwd_grid(d->rows, f, d->width);
  float* part = sums ? static_cast<float*>(workspace) : nullptr;
  const BwdArgs a{dy, x, gamma, mean, rstd, skip, dx, part, d->rows, d->lddy, d->ldx, d->ldskip, d->lddx, d->width};
  if (d->dtype == GS_F32) run_bwd<float>(a, f, grid, st);
  else run_bwd<__nv_bfloat16>(a, f, grid, st);
  if (gs_status s = gs::check_launch(where)) return s;
  if (!sums) return GS_OK;
  const int blocks = (2 * d->width + 31) / 32;
  if (d->dtype == GS_F32)
    k_layernorm_fold<float><<<blocks, 1024, 0, st>>>(part, grid, d->width, (float*)dgamma, (float*)dbeta);
  else
    k_layernorm_fold<__nv_bfloat16><<<blocks, 1024, 0, st>>>(part, grid, d->width, (__nv_bfloat16*)dgamma,
                                                                 (__nv_bfloat16*)dbeta);
  return gs::check_launch(where);
}
