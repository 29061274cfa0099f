// What the dense-layer kernels (linear.cu, layernorm.cu) share: the two element types, vector
// access with 32-bit arithmetic, the argument checks of a strided matrix.
#pragma once

#include <cuda_bf16.h>

#include <utility>

#include "common.cuh"

namespace gs {

inline size_t dtype_size(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }

// a matrix of `rows` x `width` with `ld` elements between rows: NULL, stride and alignment
inline gs_status check_matrix(const char* where, const char* what, const void* p, int64_t rows, int64_t width, int64_t ld,
                              int32_t dtype) {
  if (!p) return set_error(GS_ERR_INVALID, "%s: %s is NULL", where, what);
  if (reinterpret_cast<uintptr_t>(p) % dtype_size(dtype))
    return set_error(GS_ERR_INVALID, "%s: %s is misaligned for its type", where, what);
  if (ld < width && rows > 1)
    return set_error(GS_ERR_INVALID, "%s: row stride %lld of %s < its width %lld", where, (long long)ld, what, (long long)width);
  // the last byte's offset fits 62 bits
  if (rows > 0 && (ld > (int64_t(1) << 40) || rows > (int64_t(1) << 40) ||
                   (ld > 0 && rows > (int64_t(1) << 59) / ld)))
    return set_error(GS_ERR_INVALID, "%s: %s is too large", where, what);
  return GS_OK;
}

// whether every row of a matrix starts at a multiple of `bytes`
inline bool rows_aligned(const void* p, int64_t rows, int64_t ld, int32_t dtype, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || (ld * (int64_t)dtype_size(dtype)) % bytes == 0);
}
inline bool rows_aligned16(const void* p, int64_t rows, int64_t ld, int32_t dtype) {
  return rows_aligned(p, rows, ld, dtype, 16);
}
// Whether tiled bulk copies (TMA) may move a matrix: its rows also end on such boundaries.  Where the last
// 16 bytes of a row are only in part its own, a store fills them all (a 59-wide view of 60-float rows lost
// its 60th column), so neither direction is trusted with them.
inline bool tma_takes(const void* p, int64_t rows, int64_t width, int64_t ld, int32_t dtype) {
  return rows_aligned16(p, rows, ld, dtype) && (width * (int64_t)dtype_size(dtype)) % 16 == 0;
}

// Launches a dense-layer kernel: its blocks may start while the kernel before it on the stream ends, if that is
// another of these (programmatic dependent launch), and wait for its results in follow().  About 4 us pass from
// one kernel to the next otherwise, of which this saves half or more.  (Kernels that end up slower with their blocks
// placed early are launched with <<<>>>, which waits for everything before them, and say so there.)
template <typename... P, typename... A>
inline cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid, c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

}  // namespace gs

// ------------------------------------------------------------------ device helpers
// First in every dense-layer kernel: lets the kernel after it be set up, and waits until the one before it is done and
// its writes are visible (at once where there is none to wait for).  Nothing in memory is touched before.
__device__ __forceinline__ void follow() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// two bfloat16 in a word, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// VE consecutive elements of type T as 32-bit floats: one 16-byte access (VE = 16 / sizeof T)
// a pair of bfloat16, or one element (VE = 1)
template <typename T, int VE>
struct VecIO {
  using Raw = T;
  static __device__ __forceinline__ Raw load(const T* p) { return *p; }
  static __device__ __forceinline__ Raw zero() { return from_f32<T>(0.f); }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = to_f32<T>(r); }
  static __device__ __forceinline__ void store(T* p, const float* f) { *p = from_f32<T>(f[0]); }
};
template <>
struct VecIO<__nv_bfloat16, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }
  static __device__ __forceinline__ Raw zero() { return 0u; }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = bf16_lo(r), f[1] = bf16_hi(r); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(f[0], f[1]);
  }
};
template <>
struct VecIO<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const float4*>(p); }
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct VecIO<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) {
    f[0] = bf16_lo(r.x), f[1] = bf16_hi(r.x), f[2] = bf16_lo(r.y), f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z), f[5] = bf16_hi(r.z), f[6] = bf16_lo(r.w), f[7] = bf16_hi(r.w);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
};

// ------------------------------------------------------------------ activations and their slopes
// Phi(v) and exp(-v^2 / 2).  Phi(-|v|) = P(t) exp(-v^2 / 2), t = 1 / (1 + 0.3275911 |v| / sqrt 2), with the
// five-term polynomial of Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26, halved: off
// by at most 7.5e-8, and without the cancellation of 1 + erf for negative v.  Two special-function
// operations and 13 others, and the slope gets its exponential with it: the epilogues that evaluate it
// are bound by instructions, and erff with expf took three times as many (300K x 256 bf16 slopes with
// the bias gradient's sums: 119 us with them).  float32 pays with about a bit of GELU: on normal inputs it is off by
// 5.5e-8 root mean square (2.5e-8 by 1 + erff), between -4 and -2 by up to 2.1e-7 (1.2e-7), below -4 by half as much as
// 1 + erff, whose cancellation it has not.
__device__ __forceinline__ float gauss_cdf(float v, float& e) {
  e = fast_exp2(v * v * -0.72134752044448170f);  // -log2(e) / 2
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(v), 0.23164189f, 1.f)));
  float q = fmaf(t, 0.5307027145f, -0.7265760135f);
  q = fmaf(t, q, 0.7107068705f);
  q = fmaf(t, q, -0.142248368f);
  q = fmaf(t, q, 0.127414796f);
  const float h = q * t * e;
  return v < 0.f ? h : 1.f - h;
}
// 1 / (1 + exp(-v)).  The approximate exponential and reciprocal are off by 2e-7 of the result near zero, 4e-6 at v = -85,
// where the rounding of the exponent's argument shows; v logistic(v) is as good as by expf and a division to 20 %.
__device__ __forceinline__ float logistic(float v) {
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + fast_exp2(v * -1.4426950408889634f)));
  return s;
}

__device__ __forceinline__ float act_value(float v, int act) {
  float e;
  switch (act) {
    case GS_ACT_RELU: return v < 0.f ? 0.f : v;
    case GS_ACT_GELU: return v * gauss_cdf(v, e);
    case GS_ACT_SILU: return v * logistic(v);
    default: return v;
  }
}

__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case GS_ACT_RELU: return v > 0.f ? 1.f : 0.f;
    case GS_ACT_GELU: {
      float e;
      const float c = gauss_cdf(v, e);
      return fmaf(v * 0.39894228040143268f, e, c);
    }
    case GS_ACT_SILU: {
      const float s = logistic(v);
      return s * (1.f + v * (1.f - s));
    }
    default: return 1.f;
  }
}

// The same for pairs of elements: sm_100 adds, multiplies and fma's two floats in one instruction.  For the epilogues
// of mma_staged.cu (300K x 255 -> 257 bf16 with GELU and z: 7 % less) and of mma.cu's pairs of blocks; the
// other kernels, whose registers are all taken, lose by the pairs' alignment.  The roundings are those of one element
// at a time.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 exp2_2(F2 x) {
  float a, b;
  x.get(a, b);
  return F2(fast_exp2(a), fast_exp2(b));
}
__device__ __forceinline__ F2 recip2(F2 x) {
  float a, b;
  x.get(a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b));
  return F2(a, b);
}
// gauss_cdf as step + tail, which are (v < 0 ? 0 : 1) and (v < 0 ? Phi(v) : -Phi(-v)): no rounding of a small tail
// against a half
__device__ __forceinline__ void gauss_cdf2(float va, float vb, F2& step, F2& tail) {
  const F2 v(va, vb), e = exp2_2(mul2(mul2(v, v), F2(-0.72134752044448170f)));
  const F2 t = recip2(fma2(F2(fabsf(va), fabsf(vb)), F2(0.23164189f), F2(1.f)));
  F2 q = fma2(t, F2(0.5307027145f), F2(-0.7265760135f));
  q = fma2(t, q, F2(0.7107068705f));
  q = fma2(t, q, F2(-0.142248368f));
  q = fma2(t, q, F2(0.127414796f));
  float a, b;
  mul2(mul2(q, t), e).get(a, b);
  auto signed_as = [](float h, float v) {  // -h, or h where v is negative
    return __uint_as_float(__float_as_uint(h) ^ (~__float_as_uint(v) & 0x80000000u));
  };
  tail = F2(signed_as(a, va), signed_as(b, vb));
  step = F2(va < 0.f ? 0.f : 1.f, vb < 0.f ? 0.f : 1.f);
}
__device__ __forceinline__ F2 logistic2(F2 v) { return recip2(add2(exp2_2(mul2(v, F2(-1.4426950408889634f))), F2(1.f))); }

__device__ __forceinline__ void act_value2(float& a, float& b, int act) {
  if (act == GS_ACT_GELU) {
    F2 step, tail;
    gauss_cdf2(a, b, step, tail);
    mul2(F2(a, b), add2(step, tail)).get(a, b);
  } else if (act == GS_ACT_SILU) {
    const F2 v(a, b);
    mul2(v, logistic2(v)).get(a, b);
  } else {
    a = act_value(a, act), b = act_value(b, act);
  }
}
// ------------------------------------------------------------------ folds of split sums
// Column sums in parts ([parts][n], 32 bits) added in order: 32 columns by 32 interleaved sets of parts a block, the
// same sums for any whole number of warps.  part NULL: nothing.
struct ColumnFold {
  const float* part;
  int parts, n;
  void* out;
};
template <typename T, int THREADS>
__device__ __forceinline__ void column_fold(const ColumnFold& a, int block) {
  constexpr int kWarps = THREADS / 32, kEach = 32 / kWarps;
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = block * 32 + lane;
  float v[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) v[j] = 0.f;
  if (c < a.n) {
#pragma unroll 8
    for (int p = warp; p < a.parts; p += 32) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)  // sets warp, warp + kWarps, ..
        if (p + j * kWarps < a.parts) v[j] += a.part[(int64_t)(p + j * kWarps) * a.n + c];
    }
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) s[warp + j * kWarps][lane] = v[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j) {  // columns warp, warp + kWarps, .. of the block
    float t = s[lane][warp + j * kWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = block * 32 + warp + j * kWarps;
    if (lane == 0 && col < a.n) static_cast<T*>(a.out)[col] = from_f32<T>(t);
  }
}
template <typename T>
__global__ void __launch_bounds__(1024) k_column_fold(const ColumnFold a) {
  follow();
  column_fold<T, 1024>(a, blockIdx.x);
}
template <typename T>
inline void launch_column_fold(const ColumnFold& a, cudaStream_t st) {
  gs::launch(k_column_fold<T>, dim3((unsigned)((a.n + 31) / 32)), 1024, 0, st, a);
}

// The splits' parts [splits][m][ldp] (32-bit sums) added in order, then z = sum + bias, y = act(z) + residual;
// `transposed`: the parts hold the transpose of what is written.  The first `more`
// blocks add up `also`, if there is one.
// A block takes 128 neighbouring sums, or several times as many; WAYS warps each add every WAYS-th split of them, four
// a lane, and the warps' sums are added in order.
template <typename T>
struct FoldArgs {
  const float* part;
  const T* bias;
  const T* residual;
  T* y;
  T* z;
  int64_t m, ldp, ldr, ldy, ldz;
  int splits, n, act;
  bool transposed;
  ColumnFold also;
};
constexpr int fold_threads(int ways) { return ways > 8 ? 32 * ways : 256; }
template <typename T, int WAYS>
__global__ void __launch_bounds__(fold_threads(WAYS)) k_fold(const FoldArgs<T> a, unsigned more) {
  constexpr int kThreads = fold_threads(WAYS), kGroups = kThreads / 32 / WAYS;  // groups of 128 sums per block
  __shared__ float4 s[kThreads / 32][32];
  follow();
  if (blockIdx.x < more) {
    column_fold<T, kThreads>(a.also, blockIdx.x);
    return;
  }
  const unsigned block = blockIdx.x - more;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, way = warp % WAYS;
  const int64_t size = a.m * a.ldp, at = ((int64_t)block * kGroups + warp / WAYS) * 128 + lane * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at < size) {
#pragma unroll 8
    for (int i = way; i < a.splits; i += WAYS) {
      const float4 f = *reinterpret_cast<const float4*>(a.part + i * size + at);
      v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
    }
  }
  s[warp][lane] = v;
  __syncthreads();
  for (int e = threadIdx.x; e < kGroups * 128; e += kThreads) {
    const int64_t i = (int64_t)block * kGroups * 128 + e;
    if (i >= size) break;
    int64_t row = i / a.ldp, col = i % a.ldp;
    if (col >= a.n) continue;
    if (a.transposed) {
      const int64_t r = row;
      row = col, col = r;
    }
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < WAYS; ++w) t += reinterpret_cast<const float*>(s[e / 128 * WAYS + w])[e % 128];
    if (a.bias) t += to_f32<T>(a.bias[col]);
    if (a.z) a.z[row * a.ldz + col] = from_f32<T>(t);
    t = act_value(t, a.act);
    if (a.residual) t += to_f32<T>(a.residual[row * a.ldr + col]);
    a.y[row * a.ldy + col] = from_f32<T>(t);
  }
}
// (32 ways where the sums are too few to fill the device otherwise: 59 x 128 in 152 parts)
template <typename T>
inline void launch_fold(const FoldArgs<T>& a, cudaStream_t st) {
  const int64_t groups = (a.m * a.ldp + 127) / 128;
  const unsigned more = a.also.part ? (unsigned)((a.also.n + 31) / 32) : 0;
  auto go = [&](auto kernel, int ways) {
    const int per = fold_threads(ways) / 32 / ways;
    gs::launch(kernel, dim3((unsigned)((groups + per - 1) / per) + more), fold_threads(ways), 0, st, a, more);
  };
  if (a.splits >= 64 && groups <= 2 * 152) go(k_fold<T, 32>, 32);
  else if (a.splits >= 16) go(k_fold<T, 8>, 8);
  else go(k_fold<T, 2>, 2);
}
