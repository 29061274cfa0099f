// Group normalisation with an activation over channels-last maps, forward and backward (gs_groupnorm_fwd,
// gs_groupnorm_bwd).
//
// Mathematics, for the values x of one map's group (its rows times width / groups channels):
//   forward   mean, var = mean of (x - mean)^2, rstd = (var + eps)^-1/2, z = (x - mean) rstd gamma + beta, y = act(z)
//   backward  h = (x - mean) rstd, dz = dy act'(z), g = dz gamma, dx = rstd (g - mean(g) - h mean(g h)) + skip,
//             dgamma = sum of dz h, dbeta = sum of dz, per channel over all rows of all maps
// All of it in 32 bits, rounded once when stored.
//
// Both directions are bound by memory, and both need two passes over a map: one for its sums, one for its output.  Blocks
// take chunks of a map's rows; a thread owns one vector of neighbouring channels and walks down the rows, so that gamma, beta and
// the statistics stay in registers and every access of a warp is a run of whole sectors.  The variance is taken about a value of the
// thread's own rows (their first), so that it loses nothing where the mean is far from zero: a pivot p among n values with
// squared distances M from their mean has n (p - mean)^2 <= n M.  Chunks' sums are joined about the joint mean, in a fixed order.
// What a block of the second pass needs of the chunks' sums it adds up by itself, a few kilobytes from L2, which is
// cheaper than a kernel between the two.
#include <algorithm>
#include <cmath>

#include "dense.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A map's rows in chunks of blocks, its channels in slabs of columns.
struct Shape {
  int64_t samples, rows;
  int width, groups, per;  // per: channels of a group
  int chunks;              // of a map's rows
  int64_t chunk;           // rows of one (the last may have fewer)
  int slabs, cols;         // slabs of the width, columns of one
  int tx;                  // threads side by side: vectors of a slab
  int span;                // groups that a slab may touch
};
struct FwdArgs {
  Shape s;
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  float2* part;  // [samples][slabs][span][chunks]: mean and squared distances
  int64_t ldx, ldy;
  float eps;
};
struct BwdArgs {
  Shape s;
  const void* dy;
  const void* x;
  const void* gamma;
  const void* beta;
  const float* mean;
  const float* rstd;
  const void* skip;
  void* dx;
  float2* part;  // as the forward's: sums of g and of g h
  float* cols;   // [2][samples * chunks][width]: sums of dz and of dz h, or NULL
  int64_t lddy, ldx, ldskip, lddx;
};

// What a block works on.
struct Place {
  int64_t sample, row, end;  // rows of the matrix
  int chunk, slab, col0, col1;  // its slab's columns
  int g0, g1;                   // and the groups that they touch
  __device__ __forceinline__ Place(const Shape& s, unsigned block) {
    sample = block / s.chunks, chunk = block % s.chunks, slab = blockIdx.y;
    row = sample * s.rows + chunk * s.chunk;
    end = min(row + s.chunk, (sample + 1) * s.rows);
    col0 = slab * s.cols, col1 = min(col0 + s.cols, s.width);
    g0 = col0 / s.per, g1 = (col1 - 1) / s.per + 1;
  }
};

__device__ __forceinline__ float2 warp_sum(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// Mean and rstd of a group, from the parts of all chunks and slabs, by a warp.
__device__ __forceinline__ float2 group_stats(const FwdArgs& a, int64_t sample, int group) {
  const Shape& s = a.s;
  const int first = group * s.per / s.cols, last = ((group + 1) * s.per - 1) / s.cols;
  const int lane = threadIdx.x & 31;
  const float total = (float)s.rows * (float)s.per;
  float mean = 0.f, m2 = 0.f;
  for (int turn = 0; turn < 2; ++turn) {
    float2 sum = make_float2(0.f, 0.f);
    for (int b = first; b <= last; ++b) {
      const int wide = min((group + 1) * s.per, (b + 1) * s.cols) - max(group * s.per, b * s.cols);
      const float2* part = a.part + ((sample * s.slabs + b) * s.span + (group - b * s.cols / s.per)) * s.chunks;
      for (int c = lane; c < s.chunks; c += 32) {
        const float n = (float)(min(s.chunk, s.rows - c * s.chunk) * wide);
        const float2 p = part[c];
        if (turn == 0) sum.x = fmaf(n, p.x, sum.x);
        else sum.x += fmaf(n * (p.x - mean), p.x - mean, p.y);
      }
    }
    sum = warp_sum(sum);
    if (turn == 0) mean = sum.x / total;
    else m2 = sum.x;
  }
  return make_float2(mean, 1.f / sqrtf(m2 / total + a.eps));
}

template <typename T, int VE>
__global__ void __launch_bounds__(kThreads) k_groupnorm_stats(const FwdArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int U = 8;
  __shared__ float2 s_part[kThreads * VE];
  const Shape& s = a.s;
  const Place at(s, blockIdx.x);
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE;
  const T* x = static_cast<const T*>(a.x) + col;
  if (ty < ny && col < s.width) {
    float pivot[VE], s1[VE], s2[VE];
    int64_t r = at.row + ty;
    const int count = r < at.end ? (int)((at.end - r + ny - 1) / ny) : 0;
    if (count) IO::unpack(IO::load(x + r * a.ldx), pivot);
#pragma unroll
    for (int e = 0; e < VE; ++e) s1[e] = s2[e] = 0.f;
    auto add = [&](const typename IO::Raw& v) {
      float f[VE];
      IO::unpack(v, f);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = f[e] - pivot[e];
        s1[e] += d;
        s2[e] = fmaf(d, d, s2[e]);
      }
    };
    int i = 0;
    for (; i + U <= count; i += U, r += (int64_t)U * ny) {
      typename IO::Raw v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = IO::load(x + (r + (int64_t)u * ny) * a.ldx);
#pragma unroll
      for (int u = 0; u < U; ++u) add(v[u]);
    }
    for (; i < count; ++i, r += ny) add(IO::load(x + r * a.ldx));
    const float inv = count ? 1.f / (float)count : 0.f;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      s_part[ty * s.tx * VE + tx * VE + e] =
          count ? make_float2(fmaf(s1[e], inv, pivot[e]), fmaxf(fmaf(-s1[e] * inv, s1[e], s2[e]), 0.f)) : make_float2(0.f, 0.f);
  }
  __syncthreads();
  // the slab's part of each group: all threads' means about their mean
  const int lane = threadIdx.x & 31, rows = (int)(at.end - at.row);
  for (int g = at.g0 + (threadIdx.x >> 5); g < at.g1; g += kWarps) {
    const int c0 = max(g * s.per, at.col0), c1 = min((g + 1) * s.per, at.col1), wide = c1 - c0;
    float mean = 0.f;
    for (int turn = 0; turn < 2; ++turn) {
      float2 sum = make_float2(0.f, 0.f);
      for (int i = lane; i < wide * ny; i += 32) {
        const int y = i / wide, c = c0 - at.col0 + i % wide;
        const float2 p = s_part[y * s.tx * VE + c];
        const float n = (float)(y < rows ? (rows - y + ny - 1) / ny : 0);
        if (turn == 0) sum.x = fmaf(n, p.x, sum.x);
        else sum.x += fmaf(n * (p.x - mean), p.x - mean, p.y);
      }
      sum = warp_sum(sum);
      if (turn == 0) mean = sum.x / ((float)rows * (float)wide);
      else if (lane == 0)
        a.part[((at.sample * s.slabs + at.slab) * s.span + (g - at.g0)) * s.chunks + at.chunk] = make_float2(mean, sum.x);
    }
  }
}

template <typename T, int VE, int ACT>
__global__ void __launch_bounds__(kThreads) k_groupnorm_write(const FwdArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int U = 4;
  __shared__ float2 s_stat[kThreads * VE + 1];  // of the slab's groups
  const Shape& s = a.s;
  const Place at(s, gridDim.x - 1 - blockIdx.x);  // the rows that were read last are still in L2
  for (int g = at.g0 + (threadIdx.x >> 5); g < at.g1; g += kWarps) {
    const float2 st = group_stats(a, at.sample, g);
    if ((threadIdx.x & 31) == 0) {
      s_stat[g - at.g0] = st;
      if (at.chunk == 0 && g * s.per >= at.col0) {  // (one block of those that know it)
        if (a.mean) a.mean[at.sample * s.groups + g] = st.x;
        if (a.rstd) a.rstd[at.sample * s.groups + g] = st.y;
      }
    }
  }
  __syncthreads();
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE;
  if (ty >= ny || col >= s.width) return;
  float mean[VE], scale[VE], beta[VE];
  {
    float gamma[VE];
    IO::unpack(IO::load(static_cast<const T*>(a.gamma) + col), gamma);
    IO::unpack(IO::load(static_cast<const T*>(a.beta) + col), beta);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float2 st = s_stat[(col + e) / s.per - at.g0];
      mean[e] = st.x, scale[e] = st.y * gamma[e];
    }
  }
  const T* x = static_cast<const T*>(a.x) + col;
  T* y = static_cast<T*>(a.y) + col;
  for (int64_t r0 = at.row + ty; r0 < at.end; r0 += (int64_t)U * ny) {
    typename IO::Raw v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * ny;
      v[u] = r < at.end ? IO::load(x + r * a.ldx) : IO::zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * ny;
      if (r >= at.end) break;
      float f[VE];
      IO::unpack(v[u], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = act_value(fmaf(f[e] - mean[e], scale[e], beta[e]), ACT);
      IO::store(y + r * a.ldy, f);
    }
  }
}

// ------------------------------------------------------------------ backward
// A thread's channels: h = (x - mean) rstd, z = h gamma + beta.
template <typename T, int VE>
struct Channels {
  float mean[VE], rstd[VE], gamma[VE], beta[VE];
  __device__ __forceinline__ void load(const BwdArgs& a, const Place& at, int col) {
    using IO = VecIO<T, VE>;
    IO::unpack(IO::load(static_cast<const T*>(a.gamma) + col), gamma);
    IO::unpack(IO::load(static_cast<const T*>(a.beta) + col), beta);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int64_t g = at.sample * a.s.groups + (col + e) / a.s.per;
      mean[e] = a.mean[g], rstd[e] = a.rstd[g];
    }
  }
};

template <typename T, int VE, int ACT>
__global__ void __launch_bounds__(kThreads) k_groupnorm_grad_sums(const BwdArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int U = 4;
  __shared__ float2 s_part[kThreads * VE];
  const Shape& s = a.s;
  const Place at(s, blockIdx.x);
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE;
  if (ty < ny && col < s.width) {
    Channels<T, VE> ch;
    ch.load(a, at, col);
    const T* x = static_cast<const T*>(a.x) + col;
    const T* dy = static_cast<const T*>(a.dy) + col;
    float sz[VE], sh[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) sz[e] = sh[e] = 0.f;
    for (int64_t r0 = at.row + ty; r0 < at.end; r0 += (int64_t)U * ny) {
      typename IO::Raw vx[U], vd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + (int64_t)u * ny;
        vx[u] = r < at.end ? IO::load(x + r * a.ldx) : IO::zero();
        vd[u] = r < at.end ? IO::load(dy + r * a.lddy) : IO::zero();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + (int64_t)u * ny >= at.end) break;
        float f[VE], d[VE];
        IO::unpack(vx[u], f);
        IO::unpack(vd[u], d);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float h = (f[e] - ch.mean[e]) * ch.rstd[e];
          float dz = d[e];
          if constexpr (ACT != GS_ACT_NONE) dz *= act_slope(fmaf(h, ch.gamma[e], ch.beta[e]), ACT);
          sz[e] += dz;
          sh[e] = fmaf(dz, h, sh[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) s_part[ty * s.tx * VE + tx * VE + e] = make_float2(sz[e], sh[e]);
  }
  __syncthreads();
  // columns: over the rows of threads; the first row of them keeps the sums, times gamma
  const int cols = at.col1 - at.col0;
  const int64_t part = at.sample * s.chunks + at.chunk;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    float2 t = s_part[c];
    for (int y = 1; y < ny; ++y) {
      const float2 p = s_part[y * s.tx * VE + c];
      t.x += p.x, t.y += p.y;
    }
    if (a.cols) {
      a.cols[part * s.width + at.col0 + c] = t.x;
      a.cols[(s.samples * s.chunks + part) * s.width + at.col0 + c] = t.y;
    }
    const float gamma = to_f32<T>(static_cast<const T*>(a.gamma)[at.col0 + c]);
    s_part[c] = make_float2(t.x * gamma, t.y * gamma);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int g = at.g0 + (threadIdx.x >> 5); g < at.g1; g += kWarps) {
    const int c0 = max(g * s.per, at.col0) - at.col0, c1 = min((g + 1) * s.per, at.col1) - at.col0;
    float2 t = make_float2(0.f, 0.f);
    for (int c = c0 + lane; c < c1; c += 32) t.x += s_part[c].x, t.y += s_part[c].y;
    t = warp_sum(t);
    if (lane == 0) a.part[((at.sample * s.slabs + at.slab) * s.span + (g - at.g0)) * s.chunks + at.chunk] = t;
  }
}

template <typename T, int VE, int ACT>
__global__ void __launch_bounds__(kThreads) k_groupnorm_grad_write(const BwdArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int U = 2;
  __shared__ float2 s_mean[kThreads * VE + 1];  // of g and of g h, by the slab's groups
  const Shape& s = a.s;
  const Place at(s, gridDim.x - 1 - blockIdx.x);
  const float inv = 1.f / ((float)s.rows * (float)s.per);
  for (int g = at.g0 + (threadIdx.x >> 5); g < at.g1; g += kWarps) {
    const int first = g * s.per / s.cols, last = ((g + 1) * s.per - 1) / s.cols;
    float2 t = make_float2(0.f, 0.f);
    for (int b = first; b <= last; ++b) {
      const float2* part = a.part + ((at.sample * s.slabs + b) * s.span + (g - b * s.cols / s.per)) * s.chunks;
      for (int c = threadIdx.x & 31; c < s.chunks; c += 32) t.x += part[c].x, t.y += part[c].y;
    }
    t = warp_sum(t);
    if ((threadIdx.x & 31) == 0) s_mean[g - at.g0] = make_float2(t.x * inv, t.y * inv);
  }
  __syncthreads();
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE;
  if (ty >= ny || col >= s.width) return;
  Channels<T, VE> ch;
  ch.load(a, at, col);
  float2 mean[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) mean[e] = s_mean[(col + e) / s.per - at.g0];
  const T* x = static_cast<const T*>(a.x) + col;
  const T* dy = static_cast<const T*>(a.dy) + col;
  const T* skip = a.skip ? static_cast<const T*>(a.skip) + col : nullptr;
  T* dx = static_cast<T*>(a.dx) + col;
  for (int64_t r0 = at.row + ty; r0 < at.end; r0 += (int64_t)U * ny) {
    typename IO::Raw vx[U], vd[U], vs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * ny;
      vx[u] = r < at.end ? IO::load(x + r * a.ldx) : IO::zero();
      vd[u] = r < at.end ? IO::load(dy + r * a.lddy) : IO::zero();
      vs[u] = r < at.end && skip ? IO::load(skip + r * a.ldskip) : IO::zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + (int64_t)u * ny;
      if (r >= at.end) break;
      float f[VE], d[VE], k[VE];
      IO::unpack(vx[u], f);
      IO::unpack(vd[u], d);
      IO::unpack(vs[u], k);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float h = (f[e] - ch.mean[e]) * ch.rstd[e];
        float g = d[e] * ch.gamma[e];
        if constexpr (ACT != GS_ACT_NONE) g *= act_slope(fmaf(h, ch.gamma[e], ch.beta[e]), ACT);
        f[e] = fmaf(ch.rstd[e], g - mean[e].x - h * mean[e].y, k[e]);
      }
      IO::store(dx + r * a.lddx, f);
    }
  }
}

// dbeta, then dgamma, from the chunks' column sums
template <typename T>
__global__ void __launch_bounds__(1024) k_groupnorm_fold(const ColumnFold dbeta, const ColumnFold dgamma) {
  follow();
  const int half = gridDim.x / 2;
  if ((int)blockIdx.x < half) {
    if (dbeta.out) column_fold<T, 1024>(dbeta, blockIdx.x);
  } else if (dgamma.out) {
    column_fold<T, 1024>(dgamma, blockIdx.x - half);
  }
}

__global__ void k_groupnorm_empty(float* mean, float* rstd, int64_t n, float value) {
  follow();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    if (mean) mean[i] = 0.f;
    if (rstd) rstd[i] = value;
  }
}

// ------------------------------------------------------------------ host
// Blocks of all maps' chunks that fill the device twice over (152 SMs, 8 blocks each); a chunk's threads take 8 rows at least.
Shape shape_of(const gs_groupnorm_desc* d, int ve) {
  Shape s{};
  s.samples = d->samples, s.rows = d->rows, s.width = d->width, s.groups = d->groups, s.per = d->width / d->groups;
  const int vectors = d->width / ve;
  s.tx = vectors < kThreads ? vectors : kThreads;
  s.cols = s.tx * ve;
  s.slabs = (d->width + s.cols - 1) / s.cols;
  s.span = std::min(s.groups, s.cols / s.per + 2);
  const int ny = kThreads / s.tx;
  const int64_t want = std::max<int64_t>(1, 2 * 152 * 8 / (s.samples * s.slabs));
  s.chunk = std::max<int64_t>((d->rows + want - 1) / want, (int64_t)8 * ny);
  s.chunks = (int)((d->rows + s.chunk - 1) / s.chunk);
  return s;
}
size_t part_bytes(const Shape& s) {
  return (sizeof(float2) * (size_t)s.samples * s.slabs * s.span * s.chunks + 255) / 256 * 256;
}
// over the vectors that the arrays' alignment may lead to
template <typename F>
size_t most_bytes(const gs_groupnorm_desc* d, F f) {
  size_t most = 0;
  for (int ve : {1, 2, 4, 8})
    if (d->width % ve == 0 && ve * gs::dtype_size(d->dtype) <= 16) most = std::max(most, f(shape_of(d, ve)));
  return most;
}

gs_status check_desc(const char* where, const gs_groupnorm_desc* d) {
  if (!d) return gs::set_error(GS_ERR_INVALID, "%s: descriptor is NULL", where);
  if (d->samples < 0 || d->rows < 0 || d->width < 1 || d->width > (1 << 20) || d->samples > INT32_MAX || d->rows > INT32_MAX ||
      d->samples * d->rows > INT32_MAX)
    return gs::set_error(GS_ERR_INVALID, "%s: bad size %lld x %lld x %d", where, (long long)d->samples, (long long)d->rows, d->width);
  if (d->groups < 1 || d->width % d->groups)
    return gs::set_error(GS_ERR_INVALID, "%s: %d channels in %d groups", where, d->width, d->groups);
  if (d->dtype != GS_F32 && d->dtype != GS_BF16)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown element type %d", where, d->dtype);
  if (d->act < GS_ACT_NONE || d->act > GS_ACT_SILU) return gs::set_error(GS_ERR_INVALID, "%s: unknown activation %d", where, d->act);
  return GS_OK;
}
gs_status check_workspace(const char* where, const void* workspace, size_t bytes, size_t need) {
  if (need && (!workspace || !gs::aligned16(workspace)))
    return gs::set_error(GS_ERR_INVALID, "%s: workspace is NULL or misaligned", where);
  if (bytes < need) return gs::set_error(GS_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", where, bytes, need);
  return GS_OK;
}

template <typename Aligned>
int vector_of(int width, int32_t dtype, Aligned at) {
  const int full = 16 / (int)gs::dtype_size(dtype);
  if (width % full == 0 && at(16)) return full;
  return dtype == GS_BF16 && width % 2 == 0 && at(4) ? 2 : 1;
}

// f of an element type, a vector's length and an activation
template <typename F>
void by_form(const gs_groupnorm_desc* d, int ve, F f) {
  auto act = [&](auto t, auto v) {
    switch (d->act) {
      case GS_ACT_RELU: return f(t, v, std::integral_constant<int, GS_ACT_RELU>{});
      case GS_ACT_GELU: return f(t, v, std::integral_constant<int, GS_ACT_GELU>{});
      case GS_ACT_SILU: return f(t, v, std::integral_constant<int, GS_ACT_SILU>{});
      default: return f(t, v, std::integral_constant<int, GS_ACT_NONE>{});
    }
  };
  if (d->dtype == GS_F32) {
    if (ve == 4) act(float{}, std::integral_constant<int, 4>{});
    else act(float{}, std::integral_constant<int, 1>{});
  } else {
    if (ve == 8) act(__nv_bfloat16{}, std::integral_constant<int, 8>{});
    else if (ve == 2) act(__nv_bfloat16{}, std::integral_constant<int, 2>{});
    else act(__nv_bfloat16{}, std::integral_constant<int, 1>{});
  }
}

}  // namespace

extern "C" size_t gs_groupnorm_fwd_workspace_size(const gs_groupnorm_desc* d) {
  if (check_desc("gs_groupnorm_fwd_workspace_size", d) || d->samples * d->rows == 0) return 0;
  return most_bytes(d, part_bytes);
}

extern "C" gs_status gs_groupnorm_fwd(const gs_groupnorm_desc* d, const void* x, const void* gamma, const void* beta, void* y,
                                      float* mean, float* rstd, void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "gs_groupnorm_fwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (!(d->eps >= 0.f)) return gs::set_error(GS_ERR_INVALID, "%s: eps must be >= 0", where);
  if ((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) % 4)
    return gs::set_error(GS_ERR_INVALID, "%s: mean or rstd is misaligned", where);
  const int64_t rows = d->samples * d->rows, stats = d->samples * d->groups;
  cudaStream_t st = gs::as_stream(stream);
  if (rows == 0) {
    if (stats == 0 || (!mean && !rstd)) return GS_OK;
    gs::launch(k_groupnorm_empty, dim3((unsigned)std::min<int64_t>((stats + 255) / 256, 1216)), 256, 0, st, mean, rstd, stats,
               1.f / std::sqrt(d->eps));
    return gs::check_launch(where);
  }
  if (gs_status s = gs::check_matrix(where, "x", x, rows, d->width, d->ldx, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "y", y, rows, d->width, d->ldy, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "gamma", gamma, 1, d->width, d->width, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "beta", beta, 1, d->width, d->width, d->dtype)) return s;
  if (gs_status s = check_workspace(where, workspace, workspace_bytes, gs_groupnorm_fwd_workspace_size(d))) return s;
  const int ve = vector_of(d->width, d->dtype, [&](int bytes) {
    return gs::rows_aligned(x, rows, d->ldx, d->dtype, bytes) && gs::rows_aligned(y, rows, d->ldy, d->dtype, bytes) &&
           gs::rows_aligned(gamma, 1, 0, d->dtype, bytes) && gs::rows_aligned(beta, 1, 0, d->dtype, bytes);
  });
  const FwdArgs a{shape_of(d, ve), x, gamma, beta, y, mean, rstd, static_cast<float2*>(workspace), d->ldx, d->ldy, d->eps};
  by_form(d, ve, [&](auto t, auto v, auto act) {
    using T = decltype(t);
    constexpr int VE = decltype(v)::value, ACT = decltype(act)::value;
    const dim3 grid((unsigned)(a.s.samples * a.s.chunks), a.s.slabs);
    gs::launch(k_groupnorm_stats<T, VE>, grid, kThreads, 0, st, a);
    gs::launch(k_groupnorm_write<T, VE, ACT>, grid, kThreads, 0, st, a);
  });
  return gs::check_launch(where);
}

extern "C" size_t gs_groupnorm_bwd_workspace_size(const gs_groupnorm_desc* d) {
  if (check_desc("gs_groupnorm_bwd_workspace_size", d) || d->samples * d->rows == 0) return 0;
  return most_bytes(d, [&](const Shape& s) {
    return part_bytes(s) + sizeof(float) * 2 * (size_t)s.samples * s.chunks * s.width;
  });
}

extern "C" gs_status gs_groupnorm_bwd(const gs_groupnorm_desc* d, const void* dy, const void* x, const void* gamma,
                                      const void* beta, const float* mean, const float* rstd, const void* skip, void* dx,
                                      void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "gs_groupnorm_bwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (!dx && !dgamma && !dbeta) return GS_OK;
  const size_t size = gs::dtype_size(d->dtype);
  cudaStream_t st = gs::as_stream(stream);
  if (reinterpret_cast<uintptr_t>(dgamma) % size)
    return gs::set_error(GS_ERR_INVALID, "%s: dgamma is misaligned for its type", where);
  if (reinterpret_cast<uintptr_t>(dbeta) % size)
    return gs::set_error(GS_ERR_INVALID, "%s: dbeta is misaligned for its type", where);
  const int64_t rows = d->samples * d->rows;
  if (rows == 0) {
    if (dgamma && cudaMemsetAsync(dgamma, 0, size * d->width, st) != cudaSuccess) return gs::check_launch(where);
    if (dbeta && cudaMemsetAsync(dbeta, 0, size * d->width, st) != cudaSuccess) return gs::check_launch(where);
    return GS_OK;
  }
  if (gs_status s = gs::check_matrix(where, "dy", dy, rows, d->width, d->lddy, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "x", x, rows, d->width, d->ldx, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "gamma", gamma, 1, d->width, d->width, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "beta", beta, 1, d->width, d->width, d->dtype)) return s;
  if (skip)
    if (gs_status s = gs::check_matrix(where, "skip", skip, rows, d->width, d->ldskip, d->dtype)) return s;
  if (dx)
    if (gs_status s = gs::check_matrix(where, "dx", dx, rows, d->width, d->lddx, d->dtype)) return s;
  if (!mean || !rstd || (reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) % 4)
    return gs::set_error(GS_ERR_INVALID, "%s: mean or rstd is NULL or misaligned", where);
  if (gs_status s = check_workspace(where, workspace, workspace_bytes, gs_groupnorm_bwd_workspace_size(d))) return s;
  const int ve = vector_of(d->width, d->dtype, [&](int bytes) {
    return gs::rows_aligned(x, rows, d->ldx, d->dtype, bytes) && gs::rows_aligned(dy, rows, d->lddy, d->dtype, bytes) &&
           gs::rows_aligned(gamma, 1, 0, d->dtype, bytes) && gs::rows_aligned(beta, 1, 0, d->dtype, bytes) &&
           (!skip || gs::rows_aligned(skip, rows, d->ldskip, d->dtype, bytes)) &&
           (!dx || gs::rows_aligned(dx, rows, d->lddx, d->dtype, bytes));
  });
  const Shape s = shape_of(d, ve);
  float* cols = dgamma || dbeta ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(s)) : nullptr;
  const BwdArgs a{s, dy, x, gamma, beta, mean, rstd, skip, dx, static_cast<float2*>(workspace), cols, d->lddy, d->ldx, d->ldskip, d->lddx};
  const int parts = (int)(s.samples * s.chunks);
  by_form(d, ve, [&](auto t, auto v, auto act) {
    using T = decltype(t);
    constexpr int VE = decltype(v)::value, ACT = decltype(act)::value;
    const dim3 grid((unsigned)parts, s.slabs);
    gs::launch(k_groupnorm_grad_sums<T, VE, ACT>, grid, kThreads, 0, st, a);
    if (dx) gs::launch(k_groupnorm_grad_write<T, VE, ACT>, grid, kThreads, 0, st, a);
    if (cols) {
      const ColumnFold b{cols, parts, s.width, dbeta}, g{cols + (int64_t)parts * s.width, parts, s.width, dgamma};
      gs::launch(k_groupnorm_fold<T>, dim3(2 * ((s.width + 31) / 32)), 1024, 0, st, b, g);
    }
  });
  return gs::check_launch(where);
}
