// One AdamW step over many tensors (gs_adamw), moments in 32 bits or in 8 with a scale for each run of 256 values.
//
// Mathematics, per value: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
//   p = p keep - m step / (sqrt(v) root + eps), with keep = 1 - lr decay, step = lr / (1 - b1^t) and
//   root = (1 - b2^t)^-1/2 from the host in 64 bits.  keep comes as two floats, since lr decay may be less than the last place
//   of one: what the second adds to p joins the step, and that sum p keep, with one rounding of p's size.
// An 8-bit moment is code x scale; v is kept as its root, whose range the type holds (2^-9 to 448: of v 2^35).
//
// Bound by memory: 28 bytes a value with 32-bit moments and gradients (80M values: 316 us, 330 at the copy's rate), 16.1 with 8-bit
// moments (176M values: 430 us, 417 at the copy's rate; 17M with bfloat16 gradients and copies: 48 and 40).  Tensors off 16 bytes
// take one value an access: 20M values 87 us with 32-bit moments and 74 with 8-bit ones (83 and 47 at the copy's rate).  The tensors' addresses are
// launch parameters (no table in device memory to fill and wait for), a block looks its tensor up in them.  A warp takes
// runs of 256 values, eight a lane: the run's largest magnitudes, by which its scales go, are one reduction over the warp.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>
#include <vector>

#include "dense.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kRun = 256;                   // values that share a scale
constexpr int kTile = kThreads / 32 * kRun; // values of a block
constexpr float kTop = 448.f;               // the largest float8 e4m3

struct Tensor {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  __nv_bfloat16* copy;
  int64_t n;
  uint32_t tile;  // the launch's first tile of this tensor
  uint32_t place; // of its first value, for the random bits
  float keep, rest, step;  // keep + rest: 1 - lr decay
  int wide;       // whether every array is aligned to four of its values
};
// Launch parameters hold up to 32,764 bytes; the small form keeps the copying of them short.
constexpr int kFew = 40, kMany = 340;
template <int MOST>
struct Args {
  Tensor t[MOST];
  int count;
  float b1, c1, b2, c2, eps, root;
  uint32_t key;
  const int64_t* counts;
  int n_counts;
};
static_assert(sizeof(Args<kMany>) <= 32764, "launch parameters");

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* f);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float* f) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float* f) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
}
// four codes in a word
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"((uint16_t)(w >> (16 * h))));
    asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;}"
        : "=f"(f[2 * h]), "=f"(f[2 * h + 1]) : "r"(half2));
  }
}
__device__ __forceinline__ uint32_t encode4(const float* f) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
  return (uint32_t)hi << 16 | lo;
}
__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x6A09E667u;
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}
// To four significant bits, up where 16 random bits carry from the 16 below them.  (The type has fewer below 2^-6, which the
// conversion then rounds to the nearest of: a moment fades no further than to 2^-7 or, its root, 2^-6 of a scale that stays.)  The largest value's quotient may be
// a unit in the last place above 448, and what that is rounded up to is saturated by the conversion.
__device__ __forceinline__ float at_random(float q, uint32_t noise) {
  return __uint_as_float((__float_as_uint(q) + (noise << 4)) & 0xfff00000u);
}
// the larger of two magnitudes, NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// (b is a normal float, infinite, or zero where eps is: eps is raised to 2^-126, and the root of the smallest float is 2^-74.5.
// Beyond 2^126, where only eps or an overflowing root can be, the result is flushed to zero.)
__device__ __forceinline__ float recip(float b) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
  return r;
}

__device__ __forceinline__ void add_each(F2 x, F2 y, float& a, float& b) {
  float x0, x1, y0, y1;
  x.get(x0, x1), y.get(y0, y1);
  a = __fadd_rn(x0, y0), b = __fadd_rn(x1, y1);
}
// A run by a warp, eight values a lane: two fours (WIDE), or every 32nd one, what lies beyond the tensor taken as zeros.
template <typename G, int BITS, bool WIDE>
__device__ __forceinline__ void run_of_256(const Tensor& t, int64_t at, int lane, const float b1, const float c1, const float b2,
                                           const float c2, const float eps, const float root, const uint32_t key) {
  const G* gp = static_cast<const G*>(t.g);
  float p[8], g[8], m[8], v[8];
  [[maybe_unused]] const int left = (int)min(t.n - at, (int64_t)kRun) - lane;  // 32 i < left: the lane has an i-th value
  uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
  if constexpr (WIDE) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t e = at + lane * 4 + k * 128;
      load4(gp + e, g + 4 * k);
      if constexpr (BITS == 32) {
        load4(static_cast<const float*>(t.m) + e, m + 4 * k);
        load4(static_cast<const float*>(t.v) + e, v + 4 * k);
      } else {
        mc[k] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + e);
        vc[k] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + e);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = 32 * i < left;
      const int64_t e = at + lane + 32 * i;
      g[i] = in ? to_f32<G>(gp[e]) : 0.f;
      if constexpr (BITS == 32) {
        m[i] = in ? static_cast<const float*>(t.m)[e] : 0.f;
        v[i] = in ? static_cast<const float*>(t.v)[e] : 0.f;
      } else if (in) {
        mc[i >> 2] |= (uint32_t) static_cast<const uint8_t*>(t.m)[e] << (8 * (i & 3));
        vc[i >> 2] |= (uint32_t) static_cast<const uint8_t*>(t.v)[e] << (8 * (i & 3));
      }
    }
  }
  [[maybe_unused]] const int64_t run = at / kRun;
  if constexpr (BITS == 8) {
    const float ms = t.ms[run], vs = t.vs[run];
    decode4(mc[0], m), decode4(mc[1], m + 4);
    decode4(vc[0], v), decode4(vc[1], v + 4);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      mul2(F2(m[i], m[i + 1]), F2(ms)).get(m[i], m[i + 1]);
      const F2 r = mul2(F2(v[i], v[i + 1]), F2(vs));
      mul2(r, r).get(v[i], v[i + 1]);
    }
  }
  // (pairs of values, which sm_100 multiplies in one instruction; the sums are of one value at a time, since the compiler
  // makes one rounding of a product and a sum of pairs, and the bits of 8-bit moments are those of two)
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const F2 gi(g[i], g[i + 1]);
    add_each(mul2(F2(m[i], m[i + 1]), F2(b1)), mul2(gi, F2(c1)), m[i], m[i + 1]);
    add_each(mul2(F2(v[i], v[i + 1]), F2(b2)), mul2(mul2(gi, gi), F2(c2)), v[i], v[i + 1]);
    s[i] = __fsqrt_rn(v[i]), s[i + 1] = __fsqrt_rn(v[i + 1]);
  }
  if constexpr (WIDE) {  // (in flight while the moments are rounded)
#pragma unroll
    for (int k = 0; k < 2; ++k) load4(t.p + at + lane * 4 + k * 128, p + 4 * k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = 32 * i < left ? t.p[at + lane + 32 * i] : 0.f;
  }
  uint32_t qm[2], qv[2];
  if constexpr (BITS == 8) {
    float am = 0.f, av = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = max_nan(am, fabsf(m[i])), av = max_nan(av, s[i]);
    // the bits of magnitudes order as their values do, NaN above all
    const uint32_t bm = __reduce_max_sync(0xffffffffu, __float_as_uint(am)), bv = __reduce_max_sync(0xffffffffu, __float_as_uint(av));
    constexpr uint32_t kLeast = (127 - 100) << 23;  // 2^-100
    const float tm = bm >= kLeast ? __uint_as_float(bm) : 0.f, tv = bv >= kLeast ? __uint_as_float(bv) : 0.f;
    const float im = tm != 0.f ? __fmul_rn(__frcp_rn(tm), kTop) : 0.f, iv = tv != 0.f ? __fmul_rn(__frcp_rn(tv), kTop) : 0.f;
    const float least = tv != 0.f ? 0x1p-9f : 0.f;
    const uint32_t base = (t.place + (uint32_t)at + (WIDE ? lane * 4 : lane)) * 0x9E3779B1u + key;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * k + j;
        const uint32_t h = mix(base + (WIDE ? (uint32_t)(k * 128 + j) : (uint32_t)(32 * i)) * 0x9E3779B1u);
        a[j] = at_random(__fmul_rn(m[i], im), h & 0xffffu);
        b[j] = at_random(__fmul_rn(s[i], iv), h >> 16);
        if (s[i] > 0.f) b[j] = fmaxf(b[j], least);
      }
      qm[k] = encode4(a), qv[k] = encode4(b);
    }
    if (lane == 0) {
      t.ms[run] = __fmul_rn(tm, 1.f / kTop);
      t.vs[run] = __fmul_rn(tv, 1.f / kTop);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float d0, d1;
    fma2(F2(s[i], s[i + 1]), F2(root), F2(eps)).get(d0, d1);
    const F2 old(p[i], p[i + 1]), less = fma2(mul2(F2(m[i], m[i + 1]), F2(-t.step)), F2(recip(d0), recip(d1)), mul2(old, F2(t.rest)));
    fma2(old, F2(t.keep), less).get(p[i], p[i + 1]);
  }
  if constexpr (WIDE) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t e = at + lane * 4 + k * 128;
      *reinterpret_cast<float4*>(t.p + e) = make_float4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
      if (t.copy)
        *reinterpret_cast<uint2*>(t.copy + e) =
            make_uint2(pack_bf16(p[4 * k], p[4 * k + 1]), pack_bf16(p[4 * k + 2], p[4 * k + 3]));
      if constexpr (BITS == 32) {
        *reinterpret_cast<float4*>(static_cast<float*>(t.m) + e) = make_float4(m[4 * k], m[4 * k + 1], m[4 * k + 2], m[4 * k + 3]);
        *reinterpret_cast<float4*>(static_cast<float*>(t.v) + e) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      } else {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + e) = qm[k];
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + e) = qv[k];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (32 * i >= left) continue;
      const int64_t e = at + lane + 32 * i;
      t.p[e] = p[i];
      if constexpr (BITS == 32) {
        static_cast<float*>(t.m)[e] = m[i];
        static_cast<float*>(t.v)[e] = v[i];
      } else {
        static_cast<uint8_t*>(t.m)[e] = (uint8_t)(qm[i >> 2] >> (8 * (i & 3)));
        static_cast<uint8_t*>(t.v)[e] = (uint8_t)(qv[i >> 2] >> (8 * (i & 3)));
      }
      if (t.copy) t.copy[e] = __float2bfloat16_rn(p[i]);
    }
  }
}

// 40 warps to an SM for 8-bit moments, 48 registers: instructions bound that form as much as memory does, and more warps hide
// both (176M values: 428 us, 464 with 32 warps and 64 registers).
template <typename G, int BITS, int MOST>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 10 : 8) k_adamw(const __grid_constant__ Args<MOST> a) {
  follow();
  for (int i = 0; i < a.n_counts; ++i)
    if (a.counts[2 * i + 1] != 0) return;
  int lo = 0, hi = a.count - 1;  // the last tensor that starts at or before this tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.t[mid].tile <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const Tensor& t = a.t[lo];
  const int64_t at = (int64_t)(blockIdx.x - t.tile) * kTile + (threadIdx.x >> 5) * kRun;
  if (at >= t.n) return;
  if (t.wide && at + kRun <= t.n)
    run_of_256<G, BITS, true>(t, at, threadIdx.x & 31, a.b1, a.c1, a.b2, a.c2, a.eps, a.root, a.key);
  else
    run_of_256<G, BITS, false>(t, at, threadIdx.x & 31, a.b1, a.c1, a.b2, a.c2, a.eps, a.root, a.key);
}

template <int MOST>
void launch_some(const gs_adamw_desc* d, Args<MOST>& a, unsigned tiles, cudaStream_t st) {
  auto go = [&](auto kernel) { gs::launch(kernel, dim3(tiles), kThreads, 0, st, a); };
  if (d->grad_dtype == GS_F32) d->state_bits == 32 ? go(k_adamw<float, 32, MOST>) : go(k_adamw<float, 8, MOST>);
  else d->state_bits == 32 ? go(k_adamw<__nv_bfloat16, 32, MOST>) : go(k_adamw<__nv_bfloat16, 8, MOST>);
}

// Launches over as many tensors as the parameters hold, each of at most 2^31 - 1 tiles.
template <int MOST>
gs_status run_all(const char* where, const gs_adamw_desc* d, const gs_adamw_tensor* tensors, int count, const int64_t* counts,
                  int n_counts, cudaStream_t st) {
  Args<MOST> a;
  a.b1 = (float)d->beta1, a.c1 = (float)(1.0 - d->beta1), a.b2 = (float)d->beta2, a.c2 = (float)(1.0 - d->beta2);
  a.eps = d->eps > 0.0 ? std::max((float)d->eps, FLT_MIN) : 0.f;
  const double bc1 = 1.0 - std::pow(d->beta1, (double)d->step), bc2 = 1.0 - std::pow(d->beta2, (double)d->step);
  a.root = (float)(1.0 / std::sqrt(bc2));
  a.key = d->seed * 0x6A09E667u + (uint32_t)d->step * 0xBB67AE85u;
  a.counts = counts, a.n_counts = n_counts, a.count = 0;
  uint64_t tiles = 0, place = 0;
  auto flush = [&] {
    if (!a.count) return GS_OK;
    launch_some(d, a, (unsigned)tiles, st);
    a.count = 0, tiles = 0;
    return gs::check_launch(where);
  };
  for (int i = 0; i < count; ++i) {
    const gs_adamw_tensor& s = tensors[i];
    if (s.n == 0) continue;
    const uint64_t need = (uint64_t)(s.n + kTile - 1) / kTile;
    if (a.count == MOST || tiles + need > INT32_MAX)
      if (gs_status e = flush()) return e;
    auto at4 = [](const void* p, size_t size) { return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0; };
    const size_t ss = d->state_bits / 8;
    const bool wide = at4(s.param, 4) && at4(s.grad, gs::dtype_size(d->grad_dtype)) && at4(s.exp_avg, ss) &&
                      at4(s.exp_avg_sq, ss) && at4(s.copy, 2);
    // keep's float towards zero, so that what it lacks has its sign and an infinite parameter stays what it is; nothing is the
    // smallest float then, which no finite parameter notices
    const double exact = 1.0 - s.lr * s.weight_decay;
    float keep = (float)exact;
    if (std::fabs((double)keep) > std::fabs(exact)) keep = std::nextafter(keep, 0.f);
    float rest = (float)(exact - keep);
    if (rest == 0.f && keep != 0.f) rest = std::copysign(FLT_TRUE_MIN, keep);
    a.t[a.count++] = Tensor{s.param, s.grad, s.exp_avg, s.exp_avg_sq, s.exp_avg_scale, s.exp_avg_sq_scale,
                            static_cast<__nv_bfloat16*>(s.copy), s.n, (uint32_t)tiles, (uint32_t)place,
                            keep, rest, (float)(s.lr / bc1), wide};
    tiles += need;
    place += (uint64_t)(s.n + kRun - 1) / kRun * kRun;
  }
  return flush();
}

// Whether an array that is written shares memory with any other: their updates would race.
constexpr int kKinds = 7;
struct Range {
  uintptr_t begin, end;
  bool written;
};
// f(kind, array's range) of a tensor's arrays
template <typename F>
void each_array(const gs_adamw_desc* d, const gs_adamw_tensor& t, F f) {
  const size_t n = t.n, grad = gs::dtype_size(d->grad_dtype), state = d->state_bits / 8;
  auto one = [&](int kind, const void* p, size_t bytes) { f(kind, Range{(uintptr_t)p, (uintptr_t)p + bytes, kind != 1}); };
  if (!n) return;
  one(0, t.param, 4 * n), one(1, t.grad, grad * n), one(2, t.exp_avg, state * n), one(3, t.exp_avg_sq, state * n);
  if (d->state_bits == 8) one(4, t.exp_avg_scale, 4 * ((n + kRun - 1) / kRun)), one(5, t.exp_avg_sq_scale, 4 * ((n + kRun - 1) / kRun));
  if (t.copy) one(6, t.copy, 2 * n);
}
bool overlap(const gs_adamw_desc* d, const gs_adamw_tensor* tensors, int count) {
  // Arrays of a kind mostly ascend, as parts of a buffer or as they were allocated, and kinds often lie apart.
  Range span[kKinds] = {};
  bool apart = true;
  for (int i = 0; i < count; ++i)
    each_array(d, tensors[i], [&](int kind, Range r) {
      apart &= r.begin >= span[kind].end;
      if (!span[kind].end) span[kind].begin = r.begin;
      span[kind].end = r.end;
    });
  for (int i = 0; i < kKinds; ++i)
    for (int j = 0; j < i; ++j) apart &= span[i].begin >= span[j].end || span[j].begin >= span[i].end;
  if (apart) return false;
  std::vector<Range> all;
  all.reserve((size_t)count * kKinds);
  for (int i = 0; i < count; ++i) each_array(d, tensors[i], [&](int, Range r) { all.push_back(r); });
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t end = 0, written = 0;  // of those so far, and of those that are written
  for (const Range& r : all) {
    if (r.begin < (r.written ? end : written)) return true;
    end = std::max(end, r.end);
    if (r.written) written = std::max(written, r.end);
  }
  return false;
}

}  // namespace

extern "C" gs_status gs_adamw(const gs_adamw_desc* d, const gs_adamw_tensor* tensors, int count, const int64_t* counts,
                              int n_counts, void* stream) {
  const char* where = "gs_adamw";
  if (!d) return gs::set_error(GS_ERR_INVALID, "%s: descriptor is NULL", where);
  if (count < 0 || (count > 0 && !tensors)) return gs::set_error(GS_ERR_INVALID, "%s: bad tensors", where);
  if (n_counts < 0 || (n_counts > 0 && !counts)) return gs::set_error(GS_ERR_INVALID, "%s: bad counts", where);
  if (reinterpret_cast<uintptr_t>(counts) % 8) return gs::set_error(GS_ERR_INVALID, "%s: counts is misaligned", where);
  if (!(d->beta1 >= 0.0 && d->beta1 < 1.0) || !(d->beta2 >= 0.0 && d->beta2 < 1.0))
    return gs::set_error(GS_ERR_INVALID, "%s: betas must be in [0, 1)", where);
  if (!(d->eps >= 0.0)) return gs::set_error(GS_ERR_INVALID, "%s: eps must be >= 0", where);
  if (d->step < 1) return gs::set_error(GS_ERR_INVALID, "%s: step must be >= 1", where);
  if (d->grad_dtype != GS_F32 && d->grad_dtype != GS_BF16)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown gradient type %d", where, d->grad_dtype);
  if (d->state_bits != 32 && d->state_bits != 8)
    return gs::set_error(GS_ERR_INVALID, "%s: state_bits must be 32 or 8, got %d", where, d->state_bits);
  for (int i = 0; i < count; ++i) {
    const gs_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t(1) << 40)) return gs::set_error(GS_ERR_INVALID, "%s: bad size of tensor %d", where, i);
    if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay))
      return gs::set_error(GS_ERR_INVALID, "%s: lr or weight_decay of tensor %d is not finite", where, i);
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq)
      return gs::set_error(GS_ERR_INVALID, "%s: an array of tensor %d is NULL", where, i);
    const uintptr_t f = (uintptr_t)t.param | (uintptr_t)t.exp_avg_scale | (uintptr_t)t.exp_avg_sq_scale |
                        (d->state_bits == 32 ? (uintptr_t)t.exp_avg | (uintptr_t)t.exp_avg_sq : 0);
    if (f % 4 || (uintptr_t)t.grad % gs::dtype_size(d->grad_dtype) || (uintptr_t)t.copy % 2)
      return gs::set_error(GS_ERR_INVALID, "%s: an array of tensor %d is misaligned for its type", where, i);
    if (d->state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale))
      return gs::set_error(GS_ERR_INVALID, "%s: 8-bit moments of tensor %d need their scales", where, i);
  }
  try {
    if (overlap(d, tensors, count))
      return gs::set_error(GS_ERR_INVALID, "%s: arrays overlap of which at least one is written", where);
  } catch (const std::bad_alloc&) {
    return gs::set_error(GS_ERR_INVALID, "%s: no host memory for %d tensors", where, count);
  }
  cudaStream_t st = gs::as_stream(stream);
  if (count <= kFew) return run_all<kFew>(where, d, tensors, count, counts, n_counts, st);
  return run_all<kMany>(where, d, tensors, count, counts, n_counts, st);
}
