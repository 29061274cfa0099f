// What the dense-layer kernels (linear.cu, layernorm.cu) share: the two element types, vector
// access with 32-bit arithmetic, the argument checks of a strided matrix.
#pragma once

#include <cuda_bf16.h>

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

// whether 16-byte accesses at multiples of 16 bytes reach every row of a matrix
inline bool rows_aligned16(const void* p, int64_t rows, int64_t ld, int32_t dtype) {
  return aligned16(p) && (rows <= 1 || (ld * (int64_t)dtype_size(dtype)) % 16 == 0);
}

}  // namespace gs

// ------------------------------------------------------------------ device helpers
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
// or one element (VE = 1)
template <typename T, int VE>
struct VecIO {
  using Raw = T;
  static __device__ __forceinline__ Raw load(const T* p) { return *p; }
  static __device__ __forceinline__ Raw zero() { return from_f32<T>(0.f); }
  static __device__ __forceinline__ void unpack(const Raw& r, float* f) { f[0] = to_f32<T>(r); }
  static __device__ __forceinline__ void store(T* p, const float* f) { *p = from_f32<T>(f[0]); }
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
