// float32 products in full precision on the tensor cores.
//
// C(m, n) = sum over k of A(m, k) B(n, k), then the linear layer's epilogue, as in mma.cu.  A value is split
// into three bfloat16 parts, a = a0 + a1 + a2 (each the rounding of what the ones before it leave: 8 + 8 + 8
// significant bits, the 24 of the value), and the product is summed from the six pairs whose weight is 2^-16
// or more,
//   a0 b0 | a0 b1 + a1 b0 + a1 b1 + a0 b2 + a2 b0
// each exact in 32 bits; what is left out is below 2^-25 of |a b|.  The tensor core adds a product of
// 16 terms to its sum with the low bits cut off (measured: 2.3e-7 of the result after 256 terms, 4.4e-6
// after 4096, always towards zero), so the pairs of the second group, 2^-8 smaller, have an accumulator of
// their own, and every 256 of k both are read back and added in registers with ordinary rounding.  Six
// bfloat16 products at 2.2 PFLOP/s nominal leave about 375 TFLOP/s; the FP32 pipe has 75.
//
// One persistent block per SM; its warps:
//   warp 17       copies pieces of 32 of k of A and B, float32 as they are, to a ring of raw buffers by TMA
//   warps 8 - 15  split a raw piece into the three parts and store them to a stage in the tensor core's
//                 swizzled layout.  An operand whose rows do not start on 16-byte boundaries they also copy,
//                 word by word with cp.async, several pieces ahead.  B's parts stay resident where all of
//                 its k fits.  (Loading straight to registers instead kept 16 KB in flight per SM: 312 us for
//                 the 300,000 x 59 x 128 weight gradient.)
//   warp 16       issues tcgen05.mma
//   warps 0 - 7   add up the accumulators and write C: 32 x 32 pieces through shared memory, so that the
//                 epilogue reads and writes whole rows of 32 columns at any alignment; the residual is
//                 copied ahead while the tile is being summed
// Every wait is bounded (see tc::Guard).
#include <cuda.h>

#include "mma.cuh"
#include "tcgen05.cuh"

namespace {

constexpr int kEpiWarps = 8, kSplitWarps = 8;
constexpr int kSplitters = 32 * kSplitWarps;
constexpr int kMmaWarp = 16, kCopyWarp = 17;
constexpr int kThreads = 32 * 18;
constexpr int kTileM = 128, kTileK = 32;
constexpr int kStages = 2;         // of split parts
constexpr int kMaxRaw = 6;
constexpr int kSmemMost = 232448;  // 227 KB
constexpr int kSmemCtl = 1024;
constexpr int kPitch = 33;         // floats per row of an epilogue buffer: rows and columns both hit distinct banks
constexpr int kBufBytes = 32 * kPitch * 4;
constexpr int kChunk = 8;          // k blocks between two additions in registers

struct Ctl {
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t full[kStages], empty[kStages];
  uint64_t resident, acc_full[2], acc_empty[2], drain;
  uint32_t tmem, dead;
};
static_assert(sizeof(Ctl) <= kSmemCtl, "control block");

struct Args {
  CUtensorMap map_a, map_b;
  const float* a;
  const float* b;
  int64_t lda, ldb;
  int64_t m, n, k;
  int m_tiles, n_tiles, splits, kblocks, kb_per_split;
  int raws, resident;
  int a_mn, b_mn, a_tma, b_tma;
  const float* bias;
  const float* residual;
  float* y;
  float* z;
  int64_t ldr, ldy, ldz;
  int act;
  float* part;  // [splits][m][ldp] when splits > 1: no epilogue
  int64_t ldp;
  int32_t* status;
  int wait_limit;
  int drop;
};

__device__ __forceinline__ void tile_of(const Args& p, int bn, int t, int64_t& m0, int64_t& n0, int& split) {
  const int nt = t % p.n_tiles, rest = t / p.n_tiles;
  n0 = (int64_t)nt * bn;
  m0 = (int64_t)(rest % p.m_tiles) * kTileM;
  split = rest / p.m_tiles;
}

// cp.async of one word, or a zero
__device__ __forceinline__ void copy_word(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// One operand: pieces of EXT (m or n) x 32 (k).
//  raw    [x][k]: rows of 128 bytes; [k][x]: EXT / 32 boxes of 32 rows of 128 bytes.  16-byte units of a row are
//         swizzled (unit ^ row % 8), by TMA's 128-byte mode or by the copying threads.
//  parts  [x][k]: rows of 64 bytes, 64-byte swizzle; [k][x]: EXT / 64 chunks of 32 rows of 128 bytes, 128-byte swizzle.
template <int EXT>
struct Operand {
  static constexpr int kRaw = EXT * 128, kPlane = EXT * 64;
  static constexpr int kUnits = EXT * 4 / kSplitters;  // of 8 values, per thread and piece
  const float* p;
  int64_t ld, ext, k;
  bool mn;

  // the copy of one piece by TMA
  __device__ __forceinline__ void copy_tma(const CUtensorMap* map, int64_t x0, int kb, uint32_t dst, uint32_t full) const {
    if (!mn) tc::tma_load_2d(dst, map, kb * kTileK, (int)x0, full);
    else
      for (int c = 0; c < EXT; c += 32) tc::tma_load_2d(dst + c * 128, map, (int)x0 + c, kb * kTileK, full);
  }
  // and by the splitters, a word per thread at a time: rows outside of the matrix are left as they are
  __device__ __forceinline__ void copy_words(int tid, int64_t x0, int kb, uint32_t dst) const {
    const int lane = tid & 31;
    const int64_t k0 = (int64_t)kb * kTileK;
    if (!mn) {
      const bool in = k0 + lane < k;
      const float* src = p + x0 * ld + k0 + lane;
#pragma unroll 4
      for (int r = tid >> 5; r < EXT; r += kSplitWarps) {
        if (x0 + r >= ext) break;
        copy_word(dst + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4, in ? src + r * ld : p, in);
      }
    } else {
#pragma unroll 4
      for (int i = tid >> 5; i < EXT; i += kSplitWarps) {
        const int r = i & 31, c = i & ~31;  // row of k, first column of the box
        const bool in = k0 + r < k && x0 + c + lane < ext;
        copy_word(dst + c * 128 + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4,
                  in ? p + (k0 + r) * ld + x0 + c + lane : p, in);
      }
    }
  }
  // this thread's units of a raw piece, split: 8 values to 16 bytes in each of three planes
  __device__ __forceinline__ void split(int tid, const unsigned char* raw, unsigned char* parts) const {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int j = tid + i * kSplitters;
      int from0, from1, to;
      if (!mn) {
        const int x = j >> 2, u = j & 3;
        from0 = x * 128 + (((2 * u) ^ (x & 7)) << 4);
        from1 = x * 128 + (((2 * u + 1) ^ (x & 7)) << 4);
        to = x * 64 + ((u ^ (x >> 1 & 3)) << 4);
      } else {
        const int u = j % (EXT / 8), r = j / (EXT / 8);
        const int at = (u >> 2) * 4096 + r * 128, v = 2 * (u & 3);
        from0 = at + ((v ^ (r & 7)) << 4);
        from1 = at + (((v + 1) ^ (r & 7)) << 4);
        to = (u >> 3) * 4096 + r * 128 + (((u & 7) ^ (r & 7)) << 4);
      }
      float f[8];
      // neighbouring boxes read their two halves in opposite order: distinct banks
      const bool swap = mn && ((j % (EXT / 8)) >> 2 & 1);
      const float4 s = *reinterpret_cast<const float4*>(raw + (swap ? from1 : from0));
      const float4 t = *reinterpret_cast<const float4*>(raw + (swap ? from0 : from1));
      const float4 lo = swap ? t : s, hi = swap ? s : t;
      f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w, f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint4 o;
        uint32_t* w = &o.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
          if (q < 2) {
            f[2 * e] -= bf16_lo(w[e]);  // exact: what the rounding left
            f[2 * e + 1] -= bf16_hi(w[e]);
          }
        }
        *reinterpret_cast<uint4*>(parts + q * kPlane + to) = o;
      }
    }
  }
};

// Where a copy stands: tile t, k block kb of [.., k_hi).
struct Cursor {
  int64_t m0, n0;
  int t, kb, k_hi;
};
__device__ __forceinline__ void seek(const Args& p, int bn, Cursor& c, int total) {
  if (c.t >= total) return;
  int split;
  tile_of(p, bn, c.t, c.m0, c.n0, split);
  c.kb = split * p.kb_per_split;
  c.k_hi = min(c.kb + p.kb_per_split, p.kblocks);
}
__device__ __forceinline__ void advance(const Args& p, int bn, Cursor& c, int total) {
  if (++c.kb == c.k_hi) {
    c.t += gridDim.x;
    seek(p, bn, c, total);
  }
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) k_mma_f32(const __grid_constant__ Args p) {
  using OpA = Operand<kTileM>;
  using OpB = Operand<BN>;
  constexpr int kAPlane = OpA::kPlane, kBPlane = OpB::kPlane;
  constexpr int kABytes = 3 * kAPlane, kBBytes = 3 * kBPlane;
  constexpr int kTmem = BN * 4;  // two accumulators of two chunks of k
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
  unsigned char* res_b = smem + kSmemCtl;
  unsigned char* ring = res_b + (p.resident ? kBBytes * p.kblocks : 0);
  const int stage_bytes = kABytes + (p.resident ? 0 : kBBytes);
  unsigned char* raws = ring + stage_bytes * kStages;
  const int raw_bytes = OpA::kRaw + (p.resident ? 0 : OpB::kRaw);
  unsigned char* epi = raws + raw_bytes * p.raws;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return tc::smem_addr(&b); };
  const bool a_words = !p.a_tma, b_words = !p.b_tma && !p.resident;
  const bool words = a_words || b_words;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.raws; ++s) {
      tc::mbar_init(bar(ctl.raw_full[s]), 1 + (words ? kSplitters : 0));
      tc::mbar_init(bar(ctl.raw_empty[s]), kSplitWarps);
    }
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar(ctl.full[s]), kSplitWarps);
      tc::mbar_init(bar(ctl.empty[s]), 1);
    }
    tc::mbar_init(bar(ctl.resident), kSplitWarps);
    tc::mbar_init(bar(ctl.drain), 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(ctl.acc_full[i]), 1);
      tc::mbar_init(bar(ctl.acc_empty[i]), kEpiWarps);
    }
    ctl.dead = 0;
    tc::fence_mbar_init();
  }
  const tc::Guard g{&ctl.dead, p.status, p.wait_limit};
  const int total = p.m_tiles * p.n_tiles * p.splits;
  if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_addr(&ctl.tmem), kTmem);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = ctl.tmem;
  const OpA a{p.a, p.lda, p.m, p.k, p.a_mn != 0};
  const OpB b{p.b, p.ldb, p.n, p.k, p.b_mn != 0};

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ raw copies by TMA
    if (lane == 0 && !p.drop) {
      Cursor c;
      c.t = blockIdx.x;
      seek(p, BN, c, total);
      const uint32_t bytes = (p.a_tma ? OpA::kRaw : 0) + (p.b_tma && !p.resident ? OpB::kRaw : 0);
      int s = 0, it = 0;
      uint32_t parity = 1;
      bool ok = true;
      while (c.t < total) {
        ok = tc::mbar_wait(bar(ctl.raw_empty[s]), parity, g);
        if (!ok) break;
        const uint32_t dst = tc::smem_addr(raws) + raw_bytes * s, full = bar(ctl.raw_full[s]);
        if (bytes) tc::mbar_expect_tx(full, bytes);
        else tc::mbar_arrive(full);
        if (p.a_tma) a.copy_tma(&p.map_a, c.m0, c.kb, dst, full);
        if (p.b_tma && !p.resident) b.copy_tma(&p.map_b, c.n0, c.kb, dst + OpA::kRaw, full);
        advance(p, BN, c, total);
        ++it;
        if (++s == p.raws) s = 0, parity ^= 1;
      }
      if (!ok && bytes) {  // gave up: no copy may be in flight when the block ends
        for (int i = it < p.raws ? 0 : it - p.raws; i < it; ++i)
          for (int j = 0; j < p.wait_limit && !tc::mbar_try(bar(ctl.raw_full[i % p.raws]), (uint32_t)(i / p.raws & 1)); ++j) {}
      }
    }
  } else if (warp >= kEpiWarps && warp < kEpiWarps + kSplitWarps) {
    // ------------------------------------------------------------ splitters
    const int tid = threadIdx.x - 32 * kEpiWarps;
    if (!p.drop) {
      if (p.resident && (int)blockIdx.x < total) {
        // B's parts, once, its words a piece at a time through the room of the epilogue, which waits for it
        const int64_t n0 = (int64_t)(blockIdx.x % p.n_tiles) * BN;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          unsigned char* to = res_b + kBBytes * kb;
          b.copy_words(tid, n0, kb, tc::smem_addr(epi));
          asm volatile("cp.async.wait_all;" ::: "memory");
          asm volatile("bar.sync 1, %0;" ::"n"(kSplitters) : "memory");
          b.split(tid, epi, to);
          asm volatile("bar.sync 1, %0;" ::"n"(kSplitters) : "memory");
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.resident));
      }
      Cursor cur;
      cur.t = blockIdx.x;
      seek(p, BN, cur, total);
      Cursor ahead = cur;
      int ahead_s = 0;
      uint32_t ahead_parity = 1;
      bool ok = true;
      // the next piece's words, when its raw buffer is free; its arrival follows the words
      auto copy_ahead = [&]() {
        if (!words || ahead.t >= total || !ok) return;
        ok = tc::mbar_wait_warp(bar(ctl.raw_empty[ahead_s]), ahead_parity, g);
        if (!ok) return;
        const uint32_t dst = tc::smem_addr(raws) + raw_bytes * ahead_s;
        if (a_words) a.copy_words(tid, ahead.m0, ahead.kb, dst);
        if (b_words) b.copy_words(tid, ahead.n0, ahead.kb, dst + OpA::kRaw);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(ctl.raw_full[ahead_s])) : "memory");
        advance(p, BN, ahead, total);
        if (++ahead_s == p.raws) ahead_s = 0, ahead_parity ^= 1;
      };
      for (int i = 0; i + 1 < p.raws; ++i) copy_ahead();
      int r = 0, s = 0;
      uint32_t r_parity = 0, s_parity = 1;
      while (cur.t < total) {
        copy_ahead();
        ok = ok && tc::mbar_wait_warp(bar(ctl.raw_full[r]), r_parity, g);
        ok = ok && tc::mbar_wait_warp(bar(ctl.empty[s]), s_parity, g);
        if (!ok) break;
        unsigned char* to = ring + stage_bytes * s;
        const unsigned char* from = raws + raw_bytes * r;
        a.split(tid, from, to);
        if (!p.resident) b.split(tid, from + OpA::kRaw, to + kABytes);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar(ctl.raw_empty[r]));
          tc::mbar_arrive(bar(ctl.full[s]));
        }
        advance(p, BN, cur, total);
        if (++r == p.raws) r = 0, r_parity ^= 1;
        if (++s == kStages) s = 0, s_parity ^= 1;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ matrix instructions
    if (lane == 0) {
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)p.a_mn << 15 | (uint32_t)p.b_mn << 16 |
                             (uint32_t)(BN >> 3) << 17 | (uint32_t)(kTileM >> 4) << 24;
      // 16 of k further: 32 bytes along a row, or 16 rows of 128 bytes; rows of 64 or of 128 bytes
      const uint32_t a_step = p.a_mn ? 16 * 128 : 32, b_step = p.b_mn ? 16 * 128 : 32;
      const uint64_t a_desc = p.a_mn ? tc::smem_desc(0, 4096, 1024) : tc::smem_desc_64(0, 512);
      const uint64_t b_desc = p.b_mn ? tc::smem_desc(0, 4096, 1024) : tc::smem_desc_64(0, 512);
      int s = 0, n_acc = 0;
      uint32_t parity = 0;
      bool ok = true;
      if (p.resident && (int)blockIdx.x < total) ok = tc::mbar_wait(bar(ctl.resident), 0, g);
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        int64_t m0, n0;
        int split;
        tile_of(p, BN, t, m0, n0, split);
        int kb = split * p.kb_per_split;
        const int k_hi = min(kb + p.kb_per_split, p.kblocks);
        for (; ok && kb < k_hi; ++n_acc) {  // a chunk of k: one pair of accumulators
          const int acc = n_acc & 1, c_hi = min(kb + kChunk, k_hi);
          ok = tc::mbar_wait(bar(ctl.acc_empty[acc]), (uint32_t)(n_acc >> 1 & 1) ^ 1, g);
          if (!ok) break;
          tc::fence_after();
          const uint32_t d = tmem + acc * (kTmem / 2);
          for (bool first = true; kb < c_hi; ++kb, first = false) {
            ok = tc::mbar_wait(bar(ctl.full[s]), parity, g);
            if (!ok) break;
            tc::fence_after();
            const uint32_t as = tc::smem_addr(ring) + stage_bytes * s;
            const uint32_t bs = p.resident ? tc::smem_addr(res_b) + kBBytes * kb : as + kABytes;
#pragma unroll
            for (int i = 0; i < kTileK / 16; ++i) {
              uint64_t da[3], db[3];
#pragma unroll
              for (int q = 0; q < 3; ++q) {
                da[q] = a_desc | ((as + q * kAPlane + i * a_step) & 0x3ffff) >> 4;
                db[q] = b_desc | ((bs + q * kBPlane + i * b_step) & 0x3ffff) >> 4;
              }
              const uint32_t add = !first || i > 0;
              tc::mma_bf16(d, da[0], db[0], idesc, add);
              tc::mma_bf16(d + BN, da[0], db[2], idesc, add);
              tc::mma_bf16(d + BN, da[2], db[0], idesc, 1);
              tc::mma_bf16(d + BN, da[1], db[1], idesc, 1);
              tc::mma_bf16(d + BN, da[0], db[1], idesc, 1);
              tc::mma_bf16(d + BN, da[1], db[0], idesc, 1);
            }
            tc::mma_commit(bar(ctl.empty[s]));
            if (++s == kStages) s = 0, parity ^= 1;
          }
          if (ok) tc::mma_commit(bar(ctl.acc_full[acc]));
        }
      }
      if (!ok) {  // gave up: nothing may be in flight when the tensor memory is freed
        tc::mma_commit(bar(ctl.drain));
        for (int j = 0; j < p.wait_limit && !tc::mbar_try(bar(ctl.drain), 0); ++j) {}
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int kCols = BN / 2;  // of this warp: 32 rows x kCols
    const int quad = warp & 3, half = warp >> 2;
    float* buf = reinterpret_cast<float*>(epi + warp * kBufBytes);
    float* res_buf = reinterpret_cast<float*>(epi + (kEpiWarps + warp) * kBufBytes);
    int n_acc = 0;
    bool ok = true;
    if (p.resident && (int)blockIdx.x < total) ok = tc::mbar_wait_warp(bar(ctl.resident), 0, g);
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      int64_t m0, n0;
      int split;
      tile_of(p, BN, t, m0, n0, split);
      const int k_lo = split * p.kb_per_split, k_hi = min(k_lo + p.kb_per_split, p.kblocks);
      const int64_t row0 = m0 + quad * 32, col0 = n0 + half * kCols;
      const bool in = row0 < p.m && col0 < (p.part ? p.ldp : p.n);
      const int rows = (int)min((int64_t)32, p.m - row0);
      // the residual of 32 columns from c on, a column per lane
      auto copy_residual = [&](int c) {
        const bool ci = col0 + c + lane < p.n;
        const float* src = p.residual + row0 * p.ldr + col0 + c + lane;
        const uint32_t dst = tc::smem_addr(res_buf) + lane * 4;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) copy_word(dst + r * (kPitch * 4), ci ? src + r * p.ldr : p.residual, ci);
      };
      if (in && !p.part && p.residual) copy_residual(0);
      float sum[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) sum[i] = 0.f;
      for (int kb = k_lo; kb < k_hi; kb += kChunk, ++n_acc) {
        const int acc = n_acc & 1;
        ok = tc::mbar_wait_warp(bar(ctl.acc_full[acc]), (uint32_t)(n_acc >> 1 & 1), g);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = tmem + acc * (kTmem / 2) + ((uint32_t)(quad * 32) << 16) + half * kCols;
        if (in) {
#pragma unroll
          for (int c = 0; c < kCols; c += 8) {
            float v[8];
            tc::tmem_load8(d + BN + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[c + i] += v[i];
            tc::tmem_load8(d + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[c + i] += v[i];
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.acc_empty[acc]));
      }
      if (!ok || !in) continue;
      if (p.part) {
        const int64_t row = row0 + lane;
        if (row < p.m) {
          float* out = p.part + ((int64_t)split * p.m + row) * p.ldp + col0;
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            if (col0 + c < p.ldp) *reinterpret_cast<float4*>(out + c) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
        }
        continue;
      }
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        const int64_t col = col0 + c + lane;
        const bool ci = col < p.n;
        const float bias = p.bias && ci ? p.bias[col] : 0.f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) buf[lane * kPitch + i] = sum[c + i] + __shfl_sync(0xffffffffu, bias, i);
        __syncwarp();
        // a lane owns a column; short separate loops keep the sums of the other pieces in registers
        if (ci && (p.act != GS_ACT_NONE || p.z)) {
          float* z = p.z + row0 * p.ldz + col;
#pragma unroll 1
          for (int r = 0; r < rows; ++r) {
            const float v = buf[r * kPitch + lane];
            if (p.z) z[r * p.ldz] = v;
            buf[r * kPitch + lane] = act_value(v, p.act);
          }
        }
        if (p.residual) {  // a lane reads the words that it copied itself
          asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 8
          for (int r = 0; r < rows; ++r) buf[r * kPitch + lane] += res_buf[r * kPitch + lane];
          if (c + 32 < kCols) copy_residual(c + 32);
        }
        if (ci) {
          float* y = p.y + row0 * p.ldy + col;
#pragma unroll 8
          for (int r = 0; r < rows; ++r) y[r * p.ldy] = buf[r * kPitch + lane];
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmem);
}

// ---------------------------------------------------------------- host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int bn, m_tiles, n_tiles, splits, kblocks, kb_per_split;
  int64_t ldp;
};

constexpr int kSms = 152;  // the device's; only speed depends on it

// Tiles of 128 columns where there are more than 64 and the tiles, or their ranges of k (at least four
// blocks, 128, each), are enough for the device; else of 64.
Plan plan_of(int64_t m, int64_t n, int64_t k) {
  Plan p;
  p.m_tiles = (int)ceil_div(m, kTileM);
  p.kblocks = (int)ceil_div(k, kTileK);
  const int64_t ranges = p.kblocks / 4 > 1 ? p.kblocks / 4 : 1;
  p.bn = n <= 64 || (int64_t)p.m_tiles * ceil_div(n, 128) * ranges < kSms ? 64 : 128;
  p.n_tiles = (int)ceil_div(n, p.bn);
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  int64_t splits = tiles >= kSms ? 1 : kSms / tiles;
  if (splits > ranges) splits = ranges;
  p.kb_per_split = (int)ceil_div(p.kblocks, splits);
  p.splits = (int)ceil_div(p.kblocks, p.kb_per_split);
  p.ldp = ceil_div(n, 4) * 4;
  return p;
}

template <int BN>
gs_status launch(Args& p, const Plan& pl, cudaStream_t st, const char* where) {
  constexpr int kA = 3 * Operand<kTileM>::kPlane, kB = 3 * Operand<BN>::kPlane;
  const int total = pl.m_tiles * pl.n_tiles * pl.splits;
  int grid = total < gs::num_sms() ? total : gs::num_sms();
  const int epi = kEpiWarps * kBufBytes * (p.residual && !p.part ? 2 : 1);
  const int room = kSmemMost - 1024 - kSmemCtl - epi;
  // resident B: one range of columns per block, and at least three raw buffers of A beside it
  if (pl.splits == 1 && pl.n_tiles <= 4 && total >= 2 * grid &&
      (int64_t)kB * pl.kblocks + kStages * kA + 3 * Operand<kTileM>::kRaw <= room) {
    p.resident = 1;
    grid -= grid % pl.n_tiles;
  }
  const int fixed = p.resident ? kB * pl.kblocks + kStages * kA : kStages * (kA + kB);
  const int raw = Operand<kTileM>::kRaw + (p.resident ? 0 : Operand<BN>::kRaw);
  const int raws = (room - fixed) / raw;
  p.raws = raws < kMaxRaw ? raws : kMaxRaw;
  const int smem = kSmemMost - room + fixed + p.raws * raw;
  const cudaError_t e = gs::max_dynamic_smem((const void*)k_mma_f32<BN>, kSmemMost);
  if (e != cudaSuccess) return gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  k_mma_f32<BN><<<grid, kThreads, smem, st>>>(p);
  return gs::check_launch(where);
}

}  // namespace

namespace gs {

size_t f32_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_of(m, n, k);
  return p.splits > 1 ? (size_t)p.splits * m * p.ldp * sizeof(float) : 0;
}

gs_status f32_run(const MmaProduct& q, void* workspace, int32_t* status, cudaStream_t st, const char* where) {
  const Plan pl = plan_of(q.m, q.n, q.k);
  if ((int64_t)pl.m_tiles * pl.n_tiles * pl.splits > 0x7fffffff) return set_error(GS_ERR_INVALID, "%s: too many tiles", where);
  Args p{};
  p.a = static_cast<const float*>(q.a), p.b = static_cast<const float*>(q.b), p.lda = q.lda, p.ldb = q.ldb;
  p.m = q.m, p.n = q.n, p.k = q.k;
  p.m_tiles = pl.m_tiles, p.n_tiles = pl.n_tiles, p.splits = pl.splits, p.kblocks = pl.kblocks;
  p.kb_per_split = pl.kb_per_split;
  p.a_mn = q.a_mn, p.b_mn = q.b_mn;
  p.a_tma = rows_aligned16(q.a, q.a_mn ? q.k : q.m, q.lda, GS_F32);
  p.b_tma = rows_aligned16(q.b, q.b_mn ? q.k : q.n, q.ldb, GS_F32);
  bool ok = true;
  if (p.a_tma)
    ok = q.a_mn ? encode_map(&p.map_a, q.a, q.k, q.m, q.lda, 32, GS_F32) : encode_map(&p.map_a, q.a, q.m, q.k, q.lda, kTileM, GS_F32);
  if (p.b_tma)
    ok = ok && (q.b_mn ? encode_map(&p.map_b, q.b, q.k, q.n, q.ldb, 32, GS_F32)
                       : encode_map(&p.map_b, q.b, q.n, q.k, q.ldb, pl.bn, GS_F32));
  if (!ok) return set_error(GS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", where);
  p.bias = static_cast<const float*>(q.bias), p.residual = static_cast<const float*>(q.residual);
  p.y = static_cast<float*>(q.y), p.z = static_cast<float*>(q.z), p.ldr = q.ldr, p.ldy = q.ldy, p.ldz = q.ldz;
  p.act = q.act;
  p.part = pl.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  p.ldp = pl.ldp;
  p.status = status, p.wait_limit = wait_tries(), p.drop = 0;
  if (gs_status s = pl.bn == 64 ? launch<64>(p, pl, st, where) : launch<128>(p, pl, st, where)) return s;
  if (!p.part) return GS_OK;
  launch_fold(FoldArgs<float>{p.part, p.bias, p.residual, p.y, p.z, q.m, pl.ldp, q.ldr, q.ldy, q.ldz, pl.splits, (int)q.n, q.act},
              st);
  return check_launch(where);
}

}  // namespace gs
