// Group normalisation with an activation over channels-last maps, forward and backward (gs_groupnorm_fwd,
// gs_groupnorm_bwd).
//
// Mathematics, for the values x of one map's group (its rows times width / groups channels):
//   forward   mean, var = mean of (x - mean)^2, rstd = (var + eps)^-1/2, z = (x - mean) rstd gamma + beta, y = act(z)
//   backward  h = (x - mean) rstd, dz = dy act'(z), g = dz gamma, dx = rstd (g - mean(g) - h mean(g h)) + skip,
//             dgamma = sum of dz h, dbeta = sum of dz, per channel over all rows of all maps
// All of it in 32 bits, rounded once when stored.
//
// Both directions are bound by memory, and both need two passes over a map: one for its sums, one for its output (but a small
// map's group fits in a block's registers, and one kernel does: 16 maps of 32 x 32 x 64 float32 6.2 us, 10.2 in two).  Blocks
// take chunks of a map's rows; a thread owns one vector of neighbouring channels and walks down the rows, so that gamma, beta and
// the statistics stay in registers and every access of a warp is a run of whole sectors.  The variance is taken about a value of the
// thread's own rows (their first), so that a mean far from zero costs nothing: a pivot p among a thread's n values with
// squared distances M from their mean has n (p - mean)^2 <= n M, which costs log2(n) / 2 digits where the spread is p's alone (n
// is some 64, of rows off 16 bytes some 500).  Threads', columns' and chunks' sums are joined about their joint mean, in a fixed order.
// What a block of the second pass needs of the chunks' sums it adds up by itself, a few kilobytes from L2, or a small kernel
// between the passes does.
//
// 16 maps of 15,965 x 256 bfloat16, SiLU: 69 us, 58 for two readings and a writing at the copy's rate (in one pass, a slab of
// groups held in the shared memory of a cluster of blocks, it took 124: 16 to 24 warps an SM do not hide the arithmetic's
// latency).  4 images of 1236 x 820 x 64 bfloat16 backward: 395 us, 382 for the two passes' bytes.
#include <algorithm>
#include <cmath>

#include "dense.cuh"

namespace {

constexpr int kThreads = 256;

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
  float2* part;    // [samples][slabs][span][chunks]: mean and squared distances
  float2* joined;  // [samples][groups]: means and rstds, or NULL: every block joins the parts by itself
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
  float2 *part, *joined;  // as the forward's: sums of g and of g h, their means
  float* cols;   // [2][samples * chunks][width]: sums of dz and of dz h, or NULL
  int64_t lddy, ldx, ldskip, lddx;
};

// What a block works on: a chunk, by its number.
struct Place {
  int64_t sample, row, end;     // rows of the matrix
  int chunk, slab, col0, col1;  // its slab's columns
  int g0, g1;                   // and the groups that they touch
  __device__ __forceinline__ Place(const Shape& s, unsigned number) {
    sample = number / s.chunks, chunk = number % s.chunks, slab = blockIdx.y;
    row = sample * s.rows + chunk * s.chunk;
    end = min(row + s.chunk, (sample + 1) * s.rows);
    col0 = slab * s.cols, col1 = min(col0 + s.cols, s.width);
    g0 = col0 / s.per, g1 = (col1 - 1) / s.per + 1;
  }
};
// The index of the first of a slab's parts of a group in the array of parts.
__device__ __forceinline__ int64_t parts_of(const Shape& s, int64_t sample, int slab, int group) {
  return ((sample * s.slabs + slab) * s.span + (group - slab * s.cols / s.per)) * s.chunks;
}

// The second pass's kernel copies its first rows before it waits for the first one's sums.  What it reads then is the call's
// input, which the kernel before the first pass may have written: the first pass lets the second begin only when that one is
// done.  (Copies of 16 bytes, which go past L1; shorter ones wait.)
__device__ __forceinline__ void wait_for_inputs() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename R>
__device__ __forceinline__ void start_and_follow(R& r, int count) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (sizeof(typename R::Raw) == 16) r.start(count);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if constexpr (sizeof(typename R::Raw) != 16) r.start(count);
}

// The rows of a thread in A arrays, through a ring of its own in shared memory: D rows ahead are copied asynchronously, which
// takes no registers and, as nobody else reads the thread's slots, no barriers.
extern __shared__ __align__(16) char s_ring[];
constexpr int kRing = 40 << 10;  // with the group's statistics no more than a block has without asking
template <int BYTES, int A>
constexpr int ring_depth() {
  constexpr int d = kRing / (kThreads * BYTES * A);
  return d > 12 ? 12 : d;
}
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}
template <typename T, int VE, int A>
struct Rows {
  using IO = VecIO<T, VE>;
  using Raw = typename IO::Raw;
  static constexpr bool kAsync = sizeof(Raw) >= 4;  // no copies of two bytes: those rows are read in batches
  static constexpr int D = kAsync ? ring_depth<sizeof(Raw), A>() : 8;
  const T* at[A];
  int64_t step[A];
  int count, next;
  __device__ __forceinline__ Raw& slot(int stage, int i) {
    return reinterpret_cast<Raw*>(s_ring)[(stage * A + i) * kThreads + threadIdx.x];
  }
  __device__ __forceinline__ void issue(int stage) {
    if (next < count) {
#pragma unroll
      for (int i = 0; i < A; ++i) {
        copy_async<sizeof(Raw)>(&slot(stage, i), at[i]);
        at[i] += step[i];
      }
    }
    ++next;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void start(int n) {
    count = n, next = 0;
    if constexpr (kAsync) {
#pragma unroll
      for (int u = 0; u < D; ++u) issue(u);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    for (int i = 0; i < count; i += D) {
      Raw v[kAsync ? 1 : D][A];
      if constexpr (!kAsync) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
#pragma unroll
          for (int k = 0; k < A; ++k) {
            v[u][k] = i + u < count ? IO::load(at[k]) : IO::zero();
            at[k] += step[k];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < D; ++u) {
        if (i + u >= count) break;
        if constexpr (kAsync) {
          asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
#pragma unroll
          for (int k = 0; k < A; ++k) v[0][k] = slot(u, k);
        }
        f(v[kAsync ? 0 : u]);
        if constexpr (kAsync) issue(u);
      }
    }
  }
};
// A vector's values as pairs, which sm_100 adds and multiplies in one instruction, or as one value (VE = 1).
template <int VE>
struct Pairs {
  using E = F2;
  static constexpr int N = VE / 2;
  static __device__ __forceinline__ E of(const float* f, int i) { return F2(f[2 * i], f[2 * i + 1]); }
  static __device__ __forceinline__ void get(const E& v, float* f, int i) { v.get(f[2 * i], f[2 * i + 1]); }
};
template <>
struct Pairs<1> {
  using E = float;
  static constexpr int N = 1;
  static __device__ __forceinline__ E of(const float* f, int) { return f[0]; }
  static __device__ __forceinline__ void get(const E& v, float* f, int) { f[0] = v; }
};
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }

// 1 / (1 + exp(-v)) of two values by one reciprocal, of the product of the denominators: a third fewer special-function
// operations, which bound the activation (16 a cycle and SM).  The denominators are scaled by 2^-63 (exactly), so that the
// product of two of up to 2^126.5 is a float whose reciprocal is one, and nobody's value is lost to a neighbour far below zero.
// Exponents are held to 126.5: a result below 2^-126 becomes zero, as logistic's does, so that z times it vanishes.
__device__ __forceinline__ F2 logistic_of(F2 v) {
  float a, b, r;
  mul2(v, F2(-1.4426950408889634f)).get(a, b);
  const F2 d = fma2(F2(fast_exp2(fminf(a, 126.5f)), fast_exp2(fminf(b, 126.5f))), F2(0x1p-63f), F2(0x1p-63f));
  d.get(a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
  F2 s;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(s.v) : "l"(F2(r).v), "l"(mul2(F2(b, a), F2(0x1p-63f)).v));
  return s;
}
template <int ACT>
__device__ __forceinline__ F2 activate(F2 z) {
  if constexpr (ACT == GS_ACT_SILU) return mul2(z, logistic_of(z));
  float a, b;
  z.get(a, b);
  act_value2(a, b, ACT);
  return F2(a, b);
}
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  return act_value(z, ACT);
}
template <int ACT>
__device__ __forceinline__ F2 slope_of(F2 z) {
  if constexpr (ACT == GS_ACT_SILU) {
    const F2 s = logistic_of(z);
    return mul2(s, fma2(z, fma2(s, F2(-1.f), F2(1.f)), F2(1.f)));
  } else {
    float a, b;
    z.get(a, b);
    return F2(act_slope(a, ACT), act_slope(b, ACT));
  }
}
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
  return act_slope(z, ACT);
}

// Threads to each of n items, a power of two: all items at once if the block has as many.
__device__ __forceinline__ int side_by_side(int n) {
  int k = 32;
  while (k > 1 && n * k > kThreads) k >>= 1;
  return k;
}
__device__ __forceinline__ float sum_among(float v, int k) {
  for (int o = k / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ forward
// at least zero, or NaN
__device__ __forceinline__ float not_negative(float v) { return v < 0.f ? 0.f : v; }

// a + b as a float, and what that float lacks
__device__ __forceinline__ float2 exact_sum(float a, float b) {
  const float sum = a + b, up = sum - a;
  return make_float2(sum, (a - (sum - up)) + (b - up));
}
// A group's mean and rstd by `lanes` lanes, from the parts of all chunks and slabs: their joint mean first, as a distance from
// the first part's, then the squares about it and the distances' own mean, by which it is corrected (about the first part's mean,
// a first chunk far from the others would cost as many digits as there are chunks).
__device__ __forceinline__ float2 join_stats(const FwdArgs& a, int64_t sample, int g, int lane, int lanes) {
  const Shape& s = a.s;
  const int first = g * s.per / s.cols, last = ((g + 1) * s.per - 1) / s.cols;
  auto each = [&](auto add) {
    for (int b = first; b <= last; ++b) {
      const int wide = min((g + 1) * s.per, (b + 1) * s.cols) - max(g * s.per, b * s.cols);
      const float2* part = a.part + parts_of(s, sample, b, g);
      const float full = (float)s.chunk * (float)wide, rest = (float)(s.rows - (s.chunks - 1) * s.chunk) * (float)wide;
#pragma unroll 8
      for (int c = lane; c < s.chunks; c += lanes) add(part[c], c == s.chunks - 1 ? rest : full);
    }
  };
  const float k = a.part[parts_of(s, sample, first, g)].x, total = (float)s.rows * (float)s.per;
  float s1 = 0.f, s2 = 0.f;
  each([&](float2 p, float n) { s1 = fmaf(n, p.x - k, s1); });
  const float2 mean = exact_sum(k, sum_among(s1, lanes) / total);
  s1 = 0.f;
  each([&](float2 p, float n) {
    const float d = p.x - mean.x - mean.y;
    s1 = fmaf(n, d, s1);
    s2 += fmaf(n * d, d, p.y);
  });
  s1 = sum_among(s1, lanes) / total, s2 = sum_among(s2, lanes) / total;
  return make_float2(mean.x + (mean.y + s1), 1.f / sqrtf(not_negative(fmaf(-s1, s1, s2)) + a.eps));
}
__device__ __forceinline__ void keep_stats(const FwdArgs& a, int64_t sample, int g, float2 st) {
  if (a.mean) a.mean[sample * a.s.groups + g] = st.x;
  if (a.rstd) a.rstd[sample * a.s.groups + g] = st.y;
}
// of the block's groups
__device__ __forceinline__ void group_stats(const FwdArgs& a, const Place& at, float2* s_stat) {
  const int groups = at.g1 - at.g0;
  if (a.joined) {
    for (int g = threadIdx.x; g < groups; g += kThreads) s_stat[g] = a.joined[at.sample * a.s.groups + at.g0 + g];
    return;
  }
  const int lanes = side_by_side(groups), lane = threadIdx.x % lanes;
  for (int g0 = 0; g0 < groups; g0 += kThreads / lanes) {
    const int g = at.g0 + min(g0 + (int)threadIdx.x / lanes, groups - 1);
    const float2 st = join_stats(a, at.sample, g, lane, lanes);
    if (lane == 0 && g0 + (int)threadIdx.x / lanes < groups) {
      s_stat[g - at.g0] = st;
      if (at.chunk == 0 && g * a.s.per >= at.col0) keep_stats(a, at.sample, g, st);  // (one block of those that know it)
    }
  }
}
// of all groups, a warp to each
__global__ void __launch_bounds__(kThreads) k_groupnorm_join(const FwdArgs a) {
  follow();
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= a.s.samples * a.s.groups) return;
  const int64_t sample = i / a.s.groups;
  const int g = (int)(i % a.s.groups), lane = threadIdx.x & 31;
  const float2 st = join_stats(a, sample, g, lane, 32);
  if (lane) return;
  a.joined[i] = st;
  keep_stats(a, sample, g, st);
}

template <typename T, int VE>
__device__ __forceinline__ void sum_chunk(const FwdArgs& a, const Place& at) {
  using IO = VecIO<T, VE>;
  const Shape& s = a.s;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE, rows = (int)(at.end - at.row);
  const bool mine = ty < ny && col < s.width;
  const int count = mine && ty < rows ? (rows - ty + ny - 1) / ny : 0;
  const T* x = static_cast<const T*>(a.x) + (at.row + ty) * a.ldx + col;
  Rows<T, VE, 1> r{{x}, {(int64_t)ny * a.ldx}};
  r.start(count);
  using V = Pairs<VE>;
  float pivot[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) pivot[e] = 0.f;
  if (count) IO::unpack(IO::load(x), pivot);
  typename V::E less[V::N], s1[V::N], s2[V::N];
#pragma unroll
  for (int i = 0; i < V::N; ++i) {
    less[i] = mul2(V::of(pivot, i), typename V::E(-1.f));
    s1[i] = s2[i] = typename V::E(0.f);
  }
  r.each([&](const typename IO::Raw (&v)[1]) {
    float f[VE];
    IO::unpack(v[0], f);
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      const auto d = add2(V::of(f, i), less[i]);
      s1[i] = add2(s1[i], d);
      s2[i] = fma2(d, d, s2[i]);
    }
  });
  __syncthreads();
  // threads' means and squared distances; then columns', over the rows of threads; then groups', over their columns
  float2* s_part = reinterpret_cast<float2*>(s_ring);
  const float inv = count ? 1.f / (float)count : 0.f;
  if (mine) {
    float f1[VE], f2[VE];
#pragma unroll
    for (int i = 0; i < V::N; ++i) V::get(s1[i], f1, i), V::get(s2[i], f2, i);
#pragma unroll
    for (int e = 0; e < VE; ++e)
      s_part[(ty * s.tx + tx) * VE + e] =
          make_float2(fmaf(f1[e], inv, pivot[e]), not_negative(fmaf(-f1[e] * inv, f1[e], f2[e])));
  }
  __syncthreads();
  const int cols = at.col1 - at.col0, lanes = side_by_side(cols), lane = threadIdx.x % lanes;
  const float by_rows = 1.f / (float)rows, few = (float)(rows / ny);  // rows of a thread; the first `more` have one more
  const int more = rows % ny;
  for (int c0 = 0; c0 < cols; c0 += kThreads / lanes) {
    const int c = c0 + (int)threadIdx.x / lanes, many = c < cols ? ny : 0;
    // about the first thread's mean, and the groups' about their first column's: like values have exactly theirs
    const float k = many ? s_part[c].x : 0.f;
    float off = 0.f, m2 = 0.f;
    for (int y = lane; y < many; y += lanes) off = fmaf(y < more ? few + 1.f : few, s_part[y * s.tx * VE + c].x - k, off);
    off = sum_among(off, lanes) * by_rows;
    for (int y = lane; y < many; y += lanes) {
      const float2 p = s_part[y * s.tx * VE + c];
      const float d = p.x - k - off;
      m2 += fmaf((y < more ? few + 1.f : few) * d, d, p.y);
    }
    m2 = sum_among(m2, lanes);
    // (row 0 of the threads has been read by this column's threads alone)
    if (lane == 0 && c < cols) s_part[c] = make_float2(k + off, m2);
  }
  __syncthreads();
  const int groups = at.g1 - at.g0, glanes = side_by_side(groups), gl = threadIdx.x % glanes;
  for (int g0 = 0; g0 < groups; g0 += kThreads / glanes) {
    const int g = at.g0 + min(g0 + (int)threadIdx.x / glanes, groups - 1);
    const int c0 = max(g * s.per, at.col0) - at.col0, c1 = min((g + 1) * s.per, at.col1) - at.col0;
    const float k = s_part[c0].x;
    float off = 0.f, m2 = 0.f;
    for (int c = c0 + gl; c < c1; c += glanes) off += s_part[c].x - k;
    off = sum_among(off, glanes) / (float)(c1 - c0);
    for (int c = c0 + gl; c < c1; c += glanes) {
      const float2 p = s_part[c];
      const float d = p.x - k - off;
      m2 += fmaf((float)rows * d, d, p.y);
    }
    m2 = sum_among(m2, glanes);
    if (gl == 0 && g0 + (int)threadIdx.x / glanes < groups)
      a.part[parts_of(s, at.sample, at.slab, g) + at.chunk] = make_float2(k + off, m2);
  }
}

// ONE: a vector's channels are of one group
template <typename T, int VE, bool ONE, int ACT>
__device__ __forceinline__ void write_chunk(const FwdArgs& a, const Place& at) {
  using IO = VecIO<T, VE>;
  const Shape& s = a.s;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE, rows = (int)(at.end - at.row);
  const int count = ty < ny && col < s.width && ty < rows ? (rows - ty + ny - 1) / ny : 0;
  Rows<T, VE, 1> r{{static_cast<const T*>(a.x) + (at.row + ty) * a.ldx + col}, {(int64_t)ny * a.ldx}};
  start_and_follow(r, count);
  float2* s_stat = reinterpret_cast<float2*>(s_ring + kRing);
  group_stats(a, at, s_stat);
  __syncthreads();
  if (!count) return;
  using V = Pairs<VE>;
  using E = typename V::E;
  E less[ONE ? 1 : V::N], scale[V::N], beta[V::N];
  {
    float gamma[VE], b[VE], m[VE], q[VE];
    IO::unpack(IO::load(static_cast<const T*>(a.gamma) + col), gamma);
    IO::unpack(IO::load(static_cast<const T*>(a.beta) + col), b);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float2 st = s_stat[(ONE ? col : col + e) / s.per - at.g0];
      m[e] = -st.x, q[e] = st.y * gamma[e];
    }
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      if (!ONE || i == 0) less[ONE ? 0 : i] = V::of(m, i);
      scale[i] = V::of(q, i), beta[i] = V::of(b, i);
    }
  }
  T* y = static_cast<T*>(a.y) + (at.row + ty) * a.ldy + col;
  const int64_t sy = (int64_t)ny * a.ldy;
  r.each([&](const typename IO::Raw (&v)[1]) {
    float f[VE];
    IO::unpack(v[0], f);
#pragma unroll
    for (int i = 0; i < V::N; ++i)
      V::get(activate<ACT>(fma2(add2(V::of(f, i), less[ONE ? 0 : i]), scale[i], beta[i])), f, i);
    IO::store(y, f);
    y += sy;
  });
}

template <typename T, int VE>
__global__ void __launch_bounds__(kThreads, 4) k_groupnorm_sums(const FwdArgs a) {
  wait_for_inputs();
  sum_chunk<T, VE>(a, Place(a.s, blockIdx.x));
}
// (backwards: the rows that were read last are still in L2)
template <typename T, int VE, bool ONE, int ACT>
__global__ void __launch_bounds__(kThreads, 4) k_groupnorm_write(const FwdArgs a) {
  write_chunk<T, VE, ONE, ACT>(a, Place(a.s, gridDim.x - 1 - blockIdx.x));
}

// ------------------------------------------------------------------ forward, small maps
// One kernel: a block takes a map's group and holds it in registers, up to small_rows vectors a thread, from the mean to the
// variance (about that mean, in two floats) to the output.
struct SmallArgs {
  FwdArgs f;
  int tx;  // threads side by side: vectors of a group
};
constexpr int kSmallThreads = 512;
constexpr int small_rows(int ve) { return ve >= 4 ? 8 : 32; }  // 32 registers
// Of the block's threads, in a fixed order; s: a float for each warp.
__device__ __forceinline__ void sum_of_warp(float v, float* s) {
  v = sum_among(v, 32);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
}
__device__ __forceinline__ float sum_of_warps(const float* s) {
  return sum_among((threadIdx.x & 31) < blockDim.x / 32 ? s[threadIdx.x & 31] : 0.f, 32);
}
template <typename T, int VE, int ACT>
__global__ void __launch_bounds__(kSmallThreads) k_groupnorm_small(const SmallArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int K = small_rows(VE);
  __shared__ float s_sum[3][32];
  const Shape& s = a.f.s;
  const int g = blockIdx.x % s.groups, tx = threadIdx.x % a.tx, ty = threadIdx.x / a.tx, ny = blockDim.x / a.tx;
  const int64_t sample = blockIdx.x / s.groups, row = sample * s.rows + ty;
  const int col = g * s.per + tx * VE, count = ty < ny && ty < s.rows ? ((int)s.rows - ty + ny - 1) / ny : 0;
  const T* x = static_cast<const T*>(a.f.x) + row * a.f.ldx + col;
  typename IO::Raw v[K];
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = k < count ? IO::load(x + (int64_t)k * ny * a.f.ldx) : IO::zero();
  // about the group's first value, so that a mean far from zero costs no digits of the spread
  const float pivot = to_f32<T>(static_cast<const T*>(a.f.x)[sample * s.rows * a.f.ldx + g * s.per]);
  float gamma[VE], beta[VE], sum = 0.f;
  IO::unpack(IO::load(static_cast<const T*>(a.f.gamma) + col), gamma);
  IO::unpack(IO::load(static_cast<const T*>(a.f.beta) + col), beta);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float f[VE];
    IO::unpack(v[k], f);
#pragma unroll
    for (int e = 0; e < VE; ++e) sum += k < count ? f[e] - pivot : 0.f;
  }
  sum_of_warp(sum, s_sum[0]);
  __syncthreads();
  const float n = (float)s.rows * (float)s.per, off = sum_of_warps(s_sum[0]) / n;
  // the mean as a float and what that float lacks, to which the distances' own mean is added: the first value may be the one
  // that is far from the others
  const float2 two = exact_sum(pivot, off);
  const float mean = two.x;
  float low = two.y, squares = 0.f;
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float f[VE];
    IO::unpack(v[k], f);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float d = k < count ? f[e] - mean - low : 0.f;
      sum += d;
      squares = fmaf(d, d, squares);
    }
  }
  sum_of_warp(sum, s_sum[1]), sum_of_warp(squares, s_sum[2]);
  __syncthreads();
  const float more = sum_of_warps(s_sum[1]) / n;
  const float rstd = 1.f / sqrtf(not_negative(fmaf(-more, more, sum_of_warps(s_sum[2]) / n)) + a.f.eps);
  low += more;
  if (threadIdx.x == 0) keep_stats(a.f, sample, g, make_float2(mean + low, rstd));
  using V = Pairs<VE>;
  typename V::E scale[V::N], shift[V::N];
#pragma unroll
  for (int e = 0; e < VE; ++e) gamma[e] *= rstd;
#pragma unroll
  for (int i = 0; i < V::N; ++i) scale[i] = V::of(gamma, i), shift[i] = V::of(beta, i);
  T* y = static_cast<T*>(a.f.y) + row * a.f.ldy + col;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k >= count) break;
    float f[VE];
    IO::unpack(v[k], f);
#pragma unroll
    for (int i = 0; i < V::N; ++i)
      V::get(activate<ACT>(fma2(add2(add2(V::of(f, i), typename V::E(-mean)), typename V::E(-low)), scale[i], shift[i])), f, i);
    IO::store(y + (int64_t)k * ny * a.f.ldy, f);
  }
}

// ------------------------------------------------------------------ backward
// With d = x - mean and q = rstd gamma: z = d q + beta, h = d rstd.
template <typename T, int VE, bool ONE, int ACT>
__device__ __forceinline__ void grad_sums(const BwdArgs& a, const Place& at) {
  using IO = VecIO<T, VE>;
  const Shape& s = a.s;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE, rows = (int)(at.end - at.row);
  const bool mine = ty < ny && col < s.width;
  const int count = mine && ty < rows ? (rows - ty + ny - 1) / ny : 0;
  Rows<T, VE, 2> r{{static_cast<const T*>(a.x) + (at.row + ty) * a.ldx + col, static_cast<const T*>(a.dy) + (at.row + ty) * a.lddy + col},
                   {(int64_t)ny * a.ldx, (int64_t)ny * a.lddy}};
  r.start(count);
  using V = Pairs<VE>;
  using E = typename V::E;
  E less[ONE ? 1 : V::N], q[V::N], beta[V::N], sz[V::N], sd[V::N];
  float rstd[ONE ? 1 : VE];
  if (mine) {
    float gamma[VE], b[VE], m[VE];
    IO::unpack(IO::load(static_cast<const T*>(a.gamma) + col), gamma);
    IO::unpack(IO::load(static_cast<const T*>(a.beta) + col), b);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int64_t g = at.sample * s.groups + (ONE ? col : col + e) / s.per;
      m[e] = -a.mean[g], rstd[ONE ? 0 : e] = a.rstd[g];
      gamma[e] *= rstd[ONE ? 0 : e];
    }
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      if (!ONE || i == 0) less[ONE ? 0 : i] = V::of(m, i);
      q[i] = V::of(gamma, i), beta[i] = V::of(b, i);
    }
  }
#pragma unroll
  for (int i = 0; i < V::N; ++i) sz[i] = sd[i] = E(0.f);
  r.each([&](const typename IO::Raw (&v)[2]) {
    float f[VE], g[VE];
    IO::unpack(v[0], f);
    IO::unpack(v[1], g);
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      const E d = add2(V::of(f, i), less[ONE ? 0 : i]);
      E dz = V::of(g, i);
      if constexpr (ACT != GS_ACT_NONE) dz = mul2(dz, slope_of<ACT>(fma2(d, q[i], beta[i])));
      sz[i] = add2(sz[i], dz);
      sd[i] = fma2(dz, d, sd[i]);
    }
  });
  __syncthreads();
  // threads' sums; then columns', over the rows of threads; then groups', of the columns' times gamma
  float2* s_part = reinterpret_cast<float2*>(s_ring);
  if (mine) {
    float fz[VE], fd[VE];
#pragma unroll
    for (int i = 0; i < V::N; ++i) V::get(sz[i], fz, i), V::get(sd[i], fd, i);
#pragma unroll
    for (int e = 0; e < VE; ++e) s_part[(ty * s.tx + tx) * VE + e] = make_float2(fz[e], fd[e] * rstd[ONE ? 0 : e]);
  }
  __syncthreads();
  const int cols = at.col1 - at.col0, lanes = side_by_side(cols), lane = threadIdx.x % lanes;
  const int64_t part = at.sample * s.chunks + at.chunk;
  for (int c0 = 0; c0 < cols; c0 += kThreads / lanes) {
    const int c = c0 + (int)threadIdx.x / lanes, many = c < cols ? ny : 0;
    float2 t = make_float2(0.f, 0.f);
    for (int y = lane; y < many; y += lanes) {
      const float2 p = s_part[y * s.tx * VE + c];
      t.x += p.x, t.y += p.y;
    }
    t.x = sum_among(t.x, lanes), t.y = sum_among(t.y, lanes);
    if (lane == 0 && c < cols) {
      if (a.cols) {
        a.cols[part * s.width + at.col0 + c] = t.x;
        a.cols[(s.samples * s.chunks + part) * s.width + at.col0 + c] = t.y;
      }
      const float gamma = to_f32<T>(static_cast<const T*>(a.gamma)[at.col0 + c]);
      s_part[c] = make_float2(t.x * gamma, t.y * gamma);
    }
  }
  __syncthreads();
  const int groups = at.g1 - at.g0, glanes = side_by_side(groups), gl = threadIdx.x % glanes;
  for (int g0 = 0; g0 < groups; g0 += kThreads / glanes) {
    const int g = at.g0 + min(g0 + (int)threadIdx.x / glanes, groups - 1);
    const int c0 = max(g * s.per, at.col0) - at.col0, c1 = min((g + 1) * s.per, at.col1) - at.col0;
    float2 t = make_float2(0.f, 0.f);
    for (int c = c0 + gl; c < c1; c += glanes) t.x += s_part[c].x, t.y += s_part[c].y;
    t.x = sum_among(t.x, glanes), t.y = sum_among(t.y, glanes);
    if (gl == 0 && g0 + (int)threadIdx.x / glanes < groups) a.part[parts_of(s, at.sample, at.slab, g) + at.chunk] = t;
  }
}

// A group's means of g and of g h by `lanes` lanes; of the block's groups; of all groups, a warp to each.
__device__ __forceinline__ float2 join_means(const BwdArgs& a, int64_t sample, int g, int lane, int lanes) {
  const Shape& s = a.s;
  const int first = g * s.per / s.cols, last = ((g + 1) * s.per - 1) / s.cols;
  float2 t = make_float2(0.f, 0.f);
  for (int b = first; b <= last; ++b) {
    const float2* part = a.part + parts_of(s, sample, b, g);
#pragma unroll 8
    for (int c = lane; c < s.chunks; c += lanes) {
      const float2 p = part[c];
      t.x += p.x, t.y += p.y;
    }
  }
  const float inv = 1.f / ((float)s.rows * (float)s.per);
  return make_float2(sum_among(t.x, lanes) * inv, sum_among(t.y, lanes) * inv);
}
__device__ __forceinline__ void grad_means(const BwdArgs& a, const Place& at, float2* s_mean) {
  const int groups = at.g1 - at.g0;
  if (a.joined) {
    for (int g = threadIdx.x; g < groups; g += kThreads) s_mean[g] = a.joined[at.sample * a.s.groups + at.g0 + g];
    return;
  }
  const int lanes = side_by_side(groups), lane = threadIdx.x % lanes;
  for (int g0 = 0; g0 < groups; g0 += kThreads / lanes) {
    const int g = at.g0 + min(g0 + (int)threadIdx.x / lanes, groups - 1);
    const float2 t = join_means(a, at.sample, g, lane, lanes);
    if (lane == 0 && g0 + (int)threadIdx.x / lanes < groups) s_mean[g - at.g0] = t;
  }
}
__global__ void __launch_bounds__(kThreads) k_groupnorm_grad_join(const BwdArgs a) {
  follow();
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= a.s.samples * a.s.groups) return;
  const float2 t = join_means(a, i / a.s.groups, (int)(i % a.s.groups), threadIdx.x & 31, 32);
  if ((threadIdx.x & 31) == 0) a.joined[i] = t;
}

// dx = dz q - (rstd mean(g) + d rstd^2 mean(g h)) + skip; A = 3: with skip
template <typename T, int VE, bool ONE, int ACT, int A>
__device__ __forceinline__ void grad_write(const BwdArgs& a, const Place& at) {
  using IO = VecIO<T, VE>;
  const Shape& s = a.s;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx, ny = kThreads / s.tx;
  const int col = at.col0 + tx * VE, rows = (int)(at.end - at.row);
  const int count = ty < ny && col < s.width && ty < rows ? (rows - ty + ny - 1) / ny : 0;
  const int64_t row = at.row + ty;
  Rows<T, VE, A> r;
  r.at[0] = static_cast<const T*>(a.x) + row * a.ldx + col, r.step[0] = (int64_t)ny * a.ldx;
  r.at[1] = static_cast<const T*>(a.dy) + row * a.lddy + col, r.step[1] = (int64_t)ny * a.lddy;
  if constexpr (A == 3) r.at[2] = static_cast<const T*>(a.skip) + row * a.ldskip + col, r.step[2] = (int64_t)ny * a.ldskip;
  start_and_follow(r, count);
  float2* s_mean = reinterpret_cast<float2*>(s_ring + kRing);  // of g and of g h, by the slab's groups
  grad_means(a, at, s_mean);
  __syncthreads();
  if (!count) return;
  using V = Pairs<VE>;
  using E = typename V::E;
  E less[ONE ? 1 : V::N], c1[ONE ? 1 : V::N], c2[ONE ? 1 : V::N], q[V::N], beta[V::N];
  {
    float gamma[VE], b[VE], m[VE], f1[VE], f2[VE];
    IO::unpack(IO::load(static_cast<const T*>(a.gamma) + col), gamma);
    IO::unpack(IO::load(static_cast<const T*>(a.beta) + col), b);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int group = (ONE ? col : col + e) / s.per;
      const float rstd = a.rstd[at.sample * s.groups + group];
      const float2 t = s_mean[group - at.g0];
      m[e] = -a.mean[at.sample * s.groups + group];
      f1[e] = -rstd * t.x, f2[e] = -rstd * rstd * t.y;
      gamma[e] *= rstd;
    }
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      if (!ONE || i == 0) less[ONE ? 0 : i] = V::of(m, i), c1[ONE ? 0 : i] = V::of(f1, i), c2[ONE ? 0 : i] = V::of(f2, i);
      q[i] = V::of(gamma, i), beta[i] = V::of(b, i);
    }
  }
  T* dx = static_cast<T*>(a.dx) + row * a.lddx + col;
  const int64_t so = (int64_t)ny * a.lddx;
  r.each([&](const typename IO::Raw (&v)[A]) {
    float f[VE], g[VE], k[VE];
    IO::unpack(v[0], f);
    IO::unpack(v[1], g);
    if constexpr (A == 3) IO::unpack(v[2], k);
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      const E d = add2(V::of(f, i), less[ONE ? 0 : i]);
      E dz = V::of(g, i);
      if constexpr (ACT != GS_ACT_NONE) dz = mul2(dz, slope_of<ACT>(fma2(d, q[i], beta[i])));
      E out = fma2(dz, q[i], fma2(d, c2[ONE ? 0 : i], c1[ONE ? 0 : i]));
      if constexpr (A == 3) out = add2(out, V::of(k, i));
      V::get(out, f, i);
    }
    IO::store(dx, f);
    dx += so;
  });
}

// dbeta and dgamma from the chunks' column sums: a block adds the parts of 8 columns of either, 32 of them side by side.
struct SumFold {
  const float* cols;
  void* dbeta;
  void* dgamma;
  int64_t parts;
  int width;
};
inline unsigned fold_blocks(int width) { return 2 * (unsigned)((width + 7) / 8); }
template <typename T>
__device__ __forceinline__ void fold(const SumFold& a, unsigned block) {
  float(*s)[8] = reinterpret_cast<float(*)[8]>(s_ring);
  void* out = block & 1 ? a.dgamma : a.dbeta;
  if (!out) return;
  const int c = (int)(block >> 1) * 8 + threadIdx.x % 8;
  const float* from = a.cols + (block & 1 ? a.parts * a.width : 0) + c;
  float v = 0.f;
  if (c < a.width) {
#pragma unroll 16
    for (int64_t p = threadIdx.x / 8; p < a.parts; p += kThreads / 8) v += from[p * a.width];
  }
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if ((threadIdx.x & 31) < 8) s[threadIdx.x >> 5][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x >= 8 || c >= a.width) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += s[w][threadIdx.x];
  static_cast<T*>(out)[c] = from_f32<T>(v);
}
template <typename T>
__global__ void __launch_bounds__(kThreads) k_groupnorm_fold(const SumFold f) {
  follow();
  fold<T>(f, blockIdx.x);
}

// blocks to an SM that the registers allow without spilling
constexpr int grad_blocks(int ve, bool one) { return ve == 8 ? (one ? 3 : 2) : ve == 1 ? 3 : one ? 4 : 3; }
template <typename T, int VE, bool ONE, int ACT>
__global__ void __launch_bounds__(kThreads, grad_blocks(VE, ONE)) k_groupnorm_grad_sums(const BwdArgs a) {
  wait_for_inputs();
  grad_sums<T, VE, ONE, ACT>(a, Place(a.s, blockIdx.x));
}
template <typename T, int VE, bool ONE, int ACT, int A>
__global__ void __launch_bounds__(kThreads, grad_blocks(VE, ONE)) k_groupnorm_grad_write(const BwdArgs a, const SumFold f, const unsigned folds) {
  if (blockIdx.x < folds) {  // beside the chunks, rather than behind them
    follow();
    if (blockIdx.y == 0) fold<T>(f, blockIdx.x);
    return;
  }
  grad_write<T, VE, ONE, ACT, A>(a, Place(a.s, gridDim.x - 1 - blockIdx.x));
}

__global__ void k_groupnorm_empty(float* mean, float* rstd, int64_t n, float value) {
  follow();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    if (mean) mean[i] = 0.f;
    if (rstd) rstd[i] = value;
  }
}

// ------------------------------------------------------------------ host
// Chunks of about 256 KB of input, but as many as the device holds blocks of (152 SMs, 4 each, of the gradient's 3; 4 maps of
// 3,927 x 200 float32 backward: 21 us with 3, 28 with 4), and of at least 4 rows a thread: a block's beginning and
// end take some 4 us, which smaller chunks repeat too often (16 maps of 15,965 x 256 bfloat16: 71 us with chunks of 215 KB, 93 with
// 54, 156 with 27), and the SMs do not get equal shares of the memory's rate, which larger ones do not even out (4 images of 1236 x
// 820 x 64 backward: 404 us with 284 KB, 416 with 1.1 MB).
constexpr int64_t kChunkBytes = 256 << 10;
Shape shape_of(const gs_groupnorm_desc* d, int ve, int arrays) {
  Shape s{};
  s.samples = d->samples, s.rows = d->rows, s.width = d->width, s.groups = d->groups, s.per = d->width / d->groups;
  const int vectors = d->width / ve;
  s.tx = std::min(vectors, kThreads);
  // forward, slabs of a width that leaves few of a block's threads without a vector, of 32 vectors and 256 bytes at least (12 maps
  // of 3,141 x 834 bfloat16 in 5 slabs of 84 vectors: 53 us, 73 in slabs of 256 and 161; backward the narrower rows cost more than
  // the idle threads, 3 maps of 34,302 x 262 float32 223 us in 4 slabs, 199 in 2)
  double best = (double)vectors / ((vectors + s.tx - 1) / s.tx * kThreads) * (kThreads / s.tx);
  for (int slabs = (vectors + kThreads - 1) / kThreads, k = 0; arrays == 1 && k < 8; ++slabs, ++k) {
    const int tx = (vectors + slabs - 1) / slabs;
    const double busy = (double)vectors / (slabs * (double)kThreads) * (kThreads / tx);
    if (tx < 32 || tx * ve * (int)gs::dtype_size(d->dtype) < 256 || busy < 1.05 * best) continue;
    best = busy, s.tx = tx;
  }
  while (s.tx * ve / s.per > 960) s.tx /= 2;  // (their statistics' place beside the ring)
  s.cols = s.tx * ve;
  s.slabs = (d->width + s.cols - 1) / s.cols;
  s.span = std::min(s.groups, s.cols / s.per + 2);
  const int ny = kThreads / s.tx;
  const double bytes = (double)d->samples * d->rows * d->width * gs::dtype_size(d->dtype) * arrays;
  const int64_t wave = 152 * (arrays == 1 ? 4 : 3), waves = std::max<int64_t>(1, (int64_t)(bytes / (kChunkBytes * wave) + 0.5));
  // (one wave has room for the blocks that fold: 4 maps of 3,927 x 200 float32 backward 21.9 us without, 18.5 with)
  const int64_t room = arrays == 2 && waves == 1 ? std::min(fold_blocks(d->width), 76u) : 0;
  const int64_t want = std::max<int64_t>(1, (waves * wave - room) / (s.samples * s.slabs));
  s.chunk = std::max<int64_t>((d->rows + want - 1) / want, (int64_t)4 * ny);
  s.chunks = (int)((d->rows + s.chunk - 1) / s.chunk);
  return s;
}
size_t part_bytes(const Shape& s) {
  return (sizeof(float2) * (size_t)s.samples * s.slabs * s.span * s.chunks + 255) / 256 * 256;
}
size_t joined_bytes(const Shape& s) { return (sizeof(float2) * (size_t)s.samples * s.groups + 255) / 256 * 256; }
// Whether a kernel between the passes joins the parts.  It costs a launch, some 3 us; without it a block waits for the parts in
// turns of eight loads a lane (12 maps of 13,604 x 952 float32 backward, 390 chunks of 119 groups: 25 turns, 471 us with it and
// 683 without; 4 images of 1236 x 820 x 64, 1,026 chunks of 8 groups: 5 turns, 394 and 392).
bool joins(const Shape& s) {
  int lanes = 32;
  while (lanes > 1 && s.span * lanes > kThreads) lanes /= 2;
  return (s.chunks + 8 * lanes - 1) / (8 * lanes) * ((s.span * lanes + kThreads - 1) / kThreads) > 5;
}
dim3 join_grid(const Shape& s) { return dim3((unsigned)((s.samples * s.groups + kThreads / 32 - 1) / (kThreads / 32))); }
// over the vectors that the arrays' alignment may lead to
template <typename F>
size_t most_bytes(const gs_groupnorm_desc* d, int arrays, F f) {
  size_t most = 0;
  for (int ve : {1, 2, 4, 8})
    if (d->width % ve == 0 && ve * gs::dtype_size(d->dtype) <= 16) most = std::max(most, f(shape_of(d, ve, arrays)));
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

// f of an element type, a vector's length, whether its channels are of one group, and an activation
template <typename F>
void by_form(const gs_groupnorm_desc* d, int ve, F f) {
  auto act = [&](auto t, auto v, auto one) {
    switch (d->act) {
      case GS_ACT_RELU: return f(t, v, one, std::integral_constant<int, GS_ACT_RELU>{});
      case GS_ACT_GELU: return f(t, v, one, std::integral_constant<int, GS_ACT_GELU>{});
      case GS_ACT_SILU: return f(t, v, one, std::integral_constant<int, GS_ACT_SILU>{});
      default: return f(t, v, one, std::integral_constant<int, GS_ACT_NONE>{});
    }
  };
  auto vector = [&](auto t, auto v) {
    if constexpr (decltype(v)::value == 1) act(t, v, std::true_type{});
    else if (d->width / d->groups % decltype(v)::value == 0) act(t, v, std::true_type{});
    else act(t, v, std::false_type{});
  };
  if (d->dtype == GS_F32) {
    if (ve == 4) vector(float{}, std::integral_constant<int, 4>{});
    else vector(float{}, std::integral_constant<int, 1>{});
  } else {
    if (ve == 8) vector(__nv_bfloat16{}, std::integral_constant<int, 8>{});
    else if (ve == 2) vector(__nv_bfloat16{}, std::integral_constant<int, 2>{});
    else vector(__nv_bfloat16{}, std::integral_constant<int, 1>{});
  }
}

// Whether the kernel for small maps takes a call, with how many threads to a block.  Up to 16 MB, whose blocks come in a
// wave or two, and not where a block would have next to nothing (us with it and without: 16 maps of 32 x 32 x 64 float32 in 8
// groups 5.6 and 8.5, of 1,024 x 256 in 32 groups 7.2 and 13.0, of 300 x 834 bfloat16 in 278 groups 18.5 and 25.8; 64 of
// 1,024 x 256 bfloat16, 32 MB, 23.4 and 20.8; 8 of 16 x 1,024 float32 in as many groups 8.7 and 6.3).
constexpr int64_t kSmallBytes = 16 << 20, kSmallBlocks = 152 * 40;
template <typename Aligned>
bool small_takes(const gs_groupnorm_desc* d, Aligned aligned, int& ve, int& tx, int& threads) {
  const int per = d->width / d->groups;
  if (d->samples * d->groups > kSmallBlocks || d->samples * d->rows * d->width * (int64_t)gs::dtype_size(d->dtype) > kSmallBytes)
    return false;
  ve = vector_of(per, d->dtype, aligned);
  tx = per / ve;
  if (tx > kSmallThreads) return false;
  threads = 32;
  auto rows = [&] { return (d->rows + threads / tx - 1) / (threads / tx); };
  while (threads < kSmallThreads && (threads < tx || rows() > (ve >= 4 ? 8 : 16))) threads *= 2;
  return rows() <= small_rows(ve);
}
// whatever the arrays' alignment
bool small_takes(const gs_groupnorm_desc* d) {
  int ve, tx, threads;
  for (int bytes : {16, 4, 0})
    if (!small_takes(d, [&](int b) { return b <= bytes; }, ve, tx, threads)) return false;
  return true;
}

}  // namespace

extern "C" size_t gs_groupnorm_fwd_workspace_size(const gs_groupnorm_desc* d) {
  if (check_desc("gs_groupnorm_fwd_workspace_size", d) || d->samples * d->rows == 0 || small_takes(d)) return 0;
  return most_bytes(d, 1, [](const Shape& s) { return part_bytes(s) + joined_bytes(s); });
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
  auto aligned = [&](int bytes) {
    return gs::rows_aligned(x, rows, d->ldx, d->dtype, bytes) && gs::rows_aligned(y, rows, d->ldy, d->dtype, bytes) &&
           gs::rows_aligned(gamma, 1, 0, d->dtype, bytes) && gs::rows_aligned(beta, 1, 0, d->dtype, bytes);
  };
  int tx, threads, small_ve;
  if (small_takes(d, aligned, small_ve, tx, threads)) {
    SmallArgs a{};
    a.f.s.rows = d->rows, a.f.s.groups = d->groups, a.f.s.per = d->width / d->groups, a.tx = tx;
    a.f.x = x, a.f.gamma = gamma, a.f.beta = beta, a.f.y = y, a.f.mean = mean, a.f.rstd = rstd;
    a.f.ldx = d->ldx, a.f.ldy = d->ldy, a.f.eps = d->eps;
    by_form(d, small_ve, [&](auto t, auto v, auto one, auto act) {
      if constexpr (decltype(one)::value)
        gs::launch(k_groupnorm_small<decltype(t), decltype(v)::value, decltype(act)::value>, dim3((unsigned)(d->samples * d->groups)),
                   threads, 0, st, a);
    });
    return gs::check_launch(where);
  }
  if (gs_status s = check_workspace(where, workspace, workspace_bytes, gs_groupnorm_fwd_workspace_size(d))) return s;
  const int ve = vector_of(d->width, d->dtype, aligned);
  const Shape s = shape_of(d, ve, 1);
  float2* parts = static_cast<float2*>(workspace);
  const FwdArgs a{s, x, gamma, beta, y, mean, rstd, parts, joins(s) ? parts + part_bytes(s) / sizeof(float2) : nullptr,
                  d->ldx, d->ldy, d->eps};
  const dim3 grid((unsigned)(s.samples * s.chunks), s.slabs);
  const size_t smem = kRing + sizeof(float2) * s.span;
  by_form(d, ve, [&](auto t, auto v, auto one, auto act) {
    using T = decltype(t);
    constexpr int VE = decltype(v)::value;
    gs::launch(k_groupnorm_sums<T, VE>, grid, kThreads, smem, st, a);
    if (a.joined) gs::launch(k_groupnorm_join, join_grid(s), kThreads, 0, st, a);
    gs::launch(k_groupnorm_write<T, VE, decltype(one)::value, decltype(act)::value>, grid, kThreads, smem, st, a);
  });
  return gs::check_launch(where);
}

extern "C" size_t gs_groupnorm_bwd_workspace_size(const gs_groupnorm_desc* d) {
  if (check_desc("gs_groupnorm_bwd_workspace_size", d) || d->samples * d->rows == 0) return 0;
  return most_bytes(d, 2, [&](const Shape& s) {
    return part_bytes(s) + joined_bytes(s) + sizeof(float) * 2 * (size_t)s.samples * s.chunks * s.width;
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
  const Shape s = shape_of(d, ve, 2);
  float* cols = dgamma || dbeta ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(s) + joined_bytes(s)) : nullptr;
  float2* parts = static_cast<float2*>(workspace);
  const BwdArgs a{s, dy, x, gamma, beta, mean, rstd, skip, dx, parts, joins(s) ? parts + part_bytes(s) / sizeof(float2) : nullptr, cols, d->lddy, d->ldx, d->ldskip, d->lddx};
  const dim3 grid((unsigned)(s.samples * s.chunks), s.slabs);
  const size_t smem = kRing + sizeof(float2) * s.span;
  by_form(d, ve, [&](auto t, auto v, auto one, auto act) {
    using T = decltype(t);
    constexpr int VE = decltype(v)::value, ACT = decltype(act)::value;
    constexpr bool ONE = decltype(one)::value;
    gs::launch(k_groupnorm_grad_sums<T, VE, ONE, ACT>, grid, kThreads, smem, st, a);
    if (dx && a.joined) gs::launch(k_groupnorm_grad_join, join_grid(s), kThreads, 0, st, a);
    const SumFold f{cols, dbeta, dgamma, s.samples * s.chunks, s.width};
    const unsigned all = cols ? fold_blocks(s.width) : 0u, folds = dx && grid.x + all <= INT32_MAX ? all : 0u;
    const dim3 more(grid.x + folds, grid.y);
    if (dx && skip) gs::launch(k_groupnorm_grad_write<T, VE, ONE, ACT, 3>, more, kThreads, smem, st, a, f, folds);
    else if (dx) gs::launch(k_groupnorm_grad_write<T, VE, ONE, ACT, 2>, more, kThreads, smem, st, a, f, folds);
    if (all != folds) gs::launch(k_groupnorm_fold<T>, dim3(all), kThreads, smem, st, f);
  });
  return gs::check_launch(where);
}
