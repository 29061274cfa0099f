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
#include <atomic>

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
  __device__ __forceinline__ void operator()(float& a) {
    if constexpr (G <= 32) {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    } else {
      float none = 0.f;
      (*this)(a, none);
    }
  }
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
__global__ void __launch_bounds__(kThreads, U == 4 ? 2 : 1) k_layernorm_fwd(const FwdArgs a) {
  follow();
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
  const int64_t step = (int64_t)gridDim.x * (kRows * U);
  typename IO::Raw rx[U][IT], next[U][IT];
  auto load = [&](int64_t r0, typename IO::Raw (&to)[U][IT]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * kRows + sub;
#pragma unroll
      for (int i = 0; i < IT; ++i)
        to[u][i] = in[i] && r < a.rows ? IO::load(x + r * a.ldx + (lane + i * G) * VE) : IO::zero();
    }
  };
  auto sum_rows = [&](float (&v)[U]) {  // two rows at a time
#pragma unroll
    for (int u = 0; u + 1 < U; u += 2) sum(v[u], v[u + 1]);
    if constexpr (U == 1) sum(v[0]);
  };
  int64_t r0 = (int64_t)blockIdx.x * (kRows * U);
  load(r0, rx);
  for (; r0 < a.rows; r0 += step) {
    load(r0 + step, next);  // in flight while these rows are summed and written
    float mean[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float f[VE];
        IO::unpack(rx[u][i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) mean[u] += f[e];  // values beyond the width are zero
      }
    }
    sum_rows(mean);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = __fmul_rn(mean[u], inv);  // the value that is stored: not folded into the differences below
      q[u] = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float f[VE];
        IO::unpack(rx[u][i], f);
        if (in[i]) {
#pragma unroll
          for (int e = 0; e < VE; ++e) q[u] = fmaf(f[e] - mean[u], f[e] - mean[u], q[u]);
        }
      }
    }
    sum_rows(q);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * kRows + sub;
      const float rstd = 1.f / sqrtf(q[u] * inv + a.eps);
      if (r < a.rows) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          if (!in[i]) continue;
          float f[VE], g[VE], b[VE];
          IO::unpack(rx[u][i], f);
          IO::unpack(rg[i], g);
          IO::unpack(rb[i], b);
#pragma unroll
          for (int e = 0; e < VE; ++e) f[e] = fmaf((f[e] - mean[u]) * rstd, g[e], b[e]);
          IO::store(y + r * a.ldy + (lane + i * G) * VE, f);
        }
        if (lane == 0) {
          if (a.mean) a.mean[r] = mean[u];
          if (a.rstd) a.rstd[r] = rstd;
        }
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) rx[u][i] = next[u][i];
    }
  }
}

// Rows wider than a block's registers: one block per row, the row read again for each sum
// (the second and third time mostly from L2).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_layernorm_fwd_wide(const FwdArgs a) {
  follow();
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

template <typename T, int VE, int G, int IT>
__global__ void __launch_bounds__(kThreads, VE == 8 && IT == 1 ? 2 : VE * IT <= 4 ? (IT == 1 && G <= 32 ? 4 : 3) : 1) k_layernorm_bwd(const BwdArgs a) {
  follow();
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
  struct Row {
    typename IO::Raw x[IT], dy[IT], skip[IT];
    float mean, rstd;
  } cur, next;
  auto load = [&](int64_t r, Row& to) {
    const bool ok = r < a.rows;
    to.mean = ok ? a.mean[r] : 0.f;
    to.rstd = ok ? a.rstd[r] : 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (lane + i * G) * VE;
      to.x[i] = in[i] && ok ? IO::load(x + r * a.ldx + c) : IO::zero();
      to.dy[i] = in[i] && ok ? IO::load(dy + r * a.lddy + c) : IO::zero();
      to.skip[i] = in[i] && ok && skip ? IO::load(skip + r * a.ldskip + c) : IO::zero();
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r0 = (int64_t)blockIdx.x * kRows;
  load(r0 + sub, cur);
  for (; r0 < a.rows; r0 += step) {
    const int64_t r = r0 + sub;
    load(r + step, next);  // in flight while this row is summed and written
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float f[VE], d[VE], g[VE];
      IO::unpack(cur.x[i], f);
      IO::unpack(cur.dy[i], d);
      IO::unpack(rg[i], g);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float h = (f[e] - cur.mean) * cur.rstd, ge = d[e] * g[e];
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
        IO::unpack(cur.x[i], f);
        IO::unpack(cur.dy[i], d);
        IO::unpack(rg[i], g);
        IO::unpack(cur.skip[i], k);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float h = (f[e] - cur.mean) * cur.rstd;
          f[e] = fmaf(cur.rstd, d[e] * g[e] - s1 - h * s2, k[e]);
        }
        IO::store(dx + r * a.lddx + (lane + i * G) * VE, f);
      }
    }
    cur = next;
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
  follow();
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
  follow();
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
// Which form a width takes: VE elements per vector, G threads per row, IT vectors per thread (0: the wide
// kernel).  The vector is 16 bytes where every array's rows and the width allow it, else a pair of bfloat16,
// else one element.
struct Form {
  int ve, g, it;
};

// A row gets as few threads as hold it in one vector each, then whole warps, then the block; a thread takes a
// second vector only where that keeps the row's sums inside a warp (64 vectors), or beyond 256.  Rows of pairs
// or single elements hold more of them per thread before they leave the warp: a thread's work would otherwise
// be mostly the sums (1M x 100 bfloat16 backward with single elements: 533 us at one per thread).  The
// backward, which keeps two sums per value in registers, prefers more threads to a second 16-byte vector.
Form form_of(int width, int ve, int32_t dtype, bool backward) {
  const bool full = ve == 16 / (int)gs::dtype_size(dtype);
  const int n = (width + ve - 1) / ve;
  for (int g : {8, 16, 32})
    if (n <= g) return {ve, g, 1};
  if (full) {
    if (n <= 64) return backward ? Form{ve, 64, 1} : Form{ve, 32, 2};
    // (forward, float32: 423 us per 700K x 512 with four vectors per lane, 459 with one for each of 128 threads;
    // bfloat16, twice as many values per vector: 234 and 216 us per 300K x 1024)
    if (n <= 128) return !backward && dtype == GS_F32 ? Form{ve, 32, 4} : Form{ve, 128, 1};
  } else {
    for (int it : {2, 4, 8})
      if (n <= 32 * it) return {ve, 32, it};
  }
  for (int it = full ? 1 : 2; it <= (full ? 4 : backward && ve == 2 ? 8 : 16); it *= 2)  // what the registers hold
    if (n <= kThreads * it) return {ve, kThreads, it};
  return {ve, kThreads, 0};
}

// blocks for these rows, no more than are resident at once: a persistent block takes the rest of the rows
int grid_of(int64_t rows, int rows_per_block, int per_sm) {
  const int64_t need = (rows + rows_per_block - 1) / rows_per_block;
  const int64_t most = (int64_t)gs::num_sms() * per_sm;
  return (int)(need < most ? (need > 0 ? need : 1) : most);
}

// Resident blocks of a kernel per SM, asked for once per kernel (a property of its code: devices of one
// architecture do not differ).
template <typename Args, void (*K)(const Args)>
int resident() {
  static std::atomic<int> known{0};
  int n = known.load();
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, K, kThreads, 0) != cudaSuccess || n < 1) n = 1;
    known.store(n);
  }
  return n;
}

constexpr int kFwdPerSm = 8, kBwdPerSm = 4;  // at most; the backward's is what its workspace is sized for

template <typename T, int VE, int G, int IT>
void launch_fwd(const FwdArgs& a, cudaStream_t st) {
  // rows in flight per thread: narrow rows need several for the memory's latency
  constexpr int U = IT == 1 ? 4 : IT == 2 ? 2 : 1;
  const int per_sm = resident<FwdArgs, k_layernorm_fwd<T, VE, G, IT, U>>();
  const int grid = grid_of(a.rows, kThreads / G * U, per_sm < kFwdPerSm ? per_sm : kFwdPerSm);
  gs::launch(k_layernorm_fwd<T, VE, G, IT, U>, dim3(grid), kThreads, 0, st, a);
}
// returns the number of blocks: the partial rows that it writes
template <typename T, int VE, int G, int IT>
int launch_bwd(const BwdArgs& a, cudaStream_t st) {
  const int per_sm = resident<BwdArgs, k_layernorm_bwd<T, VE, G, IT>>();
  const int grid = grid_of(a.rows, kThreads / G, per_sm < kBwdPerSm ? per_sm : kBwdPerSm);
  gs::launch(k_layernorm_bwd<T, VE, G, IT>, dim3(grid), kThreads, 0, st, a);
  return grid;
}

// The forms of 16-byte vectors, and of smaller ones.
#define GS_FULL_FORMS(F) F(8, 1) F(16, 1) F(32, 1) F(256, 1) F(256, 2) F(256, 4)
#define GS_PART_FORMS(F) \
  F(8, 1) F(16, 1) F(32, 1) F(32, 2) F(32, 4) F(32, 8) F(256, 2) F(256, 4) F(256, 8)

template <typename T, int VE>
void run_fwd_ve(const FwdArgs& a, Form f, cudaStream_t st) {
#define GS_FORM(G, IT) \
  if (f.g == G && f.it == IT) return launch_fwd<T, VE, G, IT>(a, st);
  if constexpr (VE * sizeof(T) == 16) {
    GS_FULL_FORMS(GS_FORM) GS_FORM(32, 2)
    if constexpr (sizeof(T) == 4) { GS_FORM(32, 4) } else { GS_FORM(128, 1) }
  } else {
    GS_PART_FORMS(GS_FORM) GS_FORM(256, 16)
  }
#undef GS_FORM
}

template <typename T>
void run_fwd(const FwdArgs& a, Form f, cudaStream_t st) {
  if (f.it == 0) gs::launch(k_layernorm_fwd_wide<T>, dim3(grid_of(a.rows, 1, kFwdPerSm)), kThreads, 0, st, a);
  else if (f.ve == 1) run_fwd_ve<T, 1>(a, f, st);
  else if (f.ve == 16 / (int)sizeof(T)) run_fwd_ve<T, 16 / sizeof(T)>(a, f, st);
  else if constexpr (sizeof(T) == 2) run_fwd_ve<T, 2>(a, f, st);
}

// the most blocks that a backward launches, each with a partial row
// (rows too wide for registers: no more than keep the partials within 256 MiB)
int bwd_most(int64_t rows, Form f, int width) {
  const int g = grid_of(rows, f.it == 0 ? 1 : kThreads / f.g, kBwdPerSm);
  const int fit = (1 << 25) / width;
  return f.it == 0 && g > fit ? fit : g;
}

template <typename T, int VE>
int run_bwd_ve(const BwdArgs& a, Form f, cudaStream_t st) {
#define GS_FORM(G, IT) \
  if (f.g == G && f.it == IT) return launch_bwd<T, VE, G, IT>(a, st);
  if constexpr (VE * sizeof(T) == 16) {
    GS_FULL_FORMS(GS_FORM) GS_FORM(64, 1) GS_FORM(128, 1)
  } else {
    GS_PART_FORMS(GS_FORM)
    if constexpr (VE == 1) { GS_FORM(256, 16) }
  }
#undef GS_FORM
  return 0;
}

template <typename T>
int run_bwd(const BwdArgs& a, Form f, cudaStream_t st) {
  if (f.it == 0) {
    const int grid = bwd_most(a.rows, f, a.width);
    gs::launch(k_layernorm_bwd_wide<T>, dim3(grid), kThreads, 0, st, a);
    return grid;
  }
  if (f.ve == 1) return run_bwd_ve<T, 1>(a, f, st);
  if (f.ve == 16 / (int)sizeof(T)) return run_bwd_ve<T, 16 / sizeof(T)>(a, f, st);
  if constexpr (sizeof(T) == 2) return run_bwd_ve<T, 2>(a, f, st);
  return 0;
}

// elements per vector: what the width, and the alignment that `at` tells of (16 or 4 bytes), allow
template <typename Aligned>
int vector_of(int width, int32_t dtype, Aligned at) {
  const int full = 16 / (int)gs::dtype_size(dtype);
  if (width % full == 0 && at(16)) return full;
  return dtype == GS_BF16 && width % 2 == 0 && at(4) ? 2 : 1;
}

gs_status check_desc(const char* where, const gs_layernorm_desc* d) {
  if (!d) return gs::set_error(GS_ERR_INVALID, "%s: descriptor is NULL", where);
  if (d->rows < 0 || d->width < 1 || d->width > (1 << 24))
    return gs::set_error(GS_ERR_INVALID, "%s: bad size %lld x %d", where, (long long)d->rows, d->width);
  if (d->dtype != GS_F32 && d->dtype != GS_BF16)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown element type %d", where, d->dtype);
  return GS_OK;
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
  const int ve = vector_of(d->width, d->dtype, [&](int bytes) {
    return gs::rows_aligned(x, d->rows, d->ldx, d->dtype, bytes) && gs::rows_aligned(y, d->rows, d->ldy, d->dtype, bytes) &&
           gs::rows_aligned(gamma, 1, 0, d->dtype, bytes) && gs::rows_aligned(beta, 1, 0, d->dtype, bytes);
  });
  const FwdArgs a{x, gamma, beta, y, mean, rstd, d->rows, d->ldx, d->ldy, d->width, d->eps};
  const Form f = form_of(d->width, ve, d->dtype, false);
  if (d->dtype == GS_F32) run_fwd<float>(a, f, gs::as_stream(stream));
  else run_fwd<__nv_bfloat16>(a, f, gs::as_stream(stream));
  return gs::check_launch(where);
}

extern "C" size_t gs_layernorm_bwd_workspace_size(const gs_layernorm_desc* d) {
  if (!d || d->rows < 0 || d->width < 1 || d->width > (1 << 24)) return 0;
  // the forms that the arrays' alignment may lead to need not have the same number of blocks: the largest
  int most = 1;
  for (int ve : {1, 2, 4, 8}) {
    if (d->width % ve || ve > 16 / (int)gs::dtype_size(d->dtype)) continue;
    const int g = bwd_most(d->rows, form_of(d->width, ve, d->dtype, true), d->width);
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
  const int ve = vector_of(d->width, d->dtype, [&](int bytes) {
    return gs::rows_aligned(x, d->rows, d->ldx, d->dtype, bytes) && gs::rows_aligned(dy, d->rows, d->lddy, d->dtype, bytes) &&
           gs::rows_aligned(gamma, 1, 0, d->dtype, bytes) && (!skip || gs::rows_aligned(skip, d->rows, d->ldskip, d->dtype, bytes)) &&
           (!dx || gs::rows_aligned(dx, d->rows, d->lddx, d->dtype, bytes));
  });
  const Form f = form_of(d->width, ve, d->dtype, true);
  float* part = sums ? static_cast<float*>(workspace) : nullptr;
  const BwdArgs a{dy, x, gamma, mean, rstd, skip, dx, part, d->rows, d->lddy, d->ldx, d->ldskip, d->lddx, d->width};
  const int grid = d->dtype == GS_F32 ? run_bwd<float>(a, f, st) : run_bwd<__nv_bfloat16>(a, f, st);
  if (gs_status s = gs::check_launch(where)) return s;
  if (!sums) return GS_OK;
  const int blocks = (2 * d->width + 31) / 32;
  if (d->dtype == GS_F32)
    gs::launch(k_layernorm_fold<float>, dim3(blocks), 1024, 0, st, (const float*)part, grid, (int)d->width, (float*)dgamma,
               (float*)dbeta);
  else
    gs::launch(k_layernorm_fold<__nv_bfloat16>, dim3(blocks), 1024, 0, st, (const float*)part, grid, (int)d->width,
               (__nv_bfloat16*)dgamma, (__nv_bfloat16*)dbeta);
  return gs::check_launch(where);
}
