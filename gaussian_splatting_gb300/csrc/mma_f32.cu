// float32 products in full precision on the tensor cores.
//
// C(m, n) = sum over k of A(m, k) B(n, k), then the linear layer's epilogue, as in mma.cu.  A value is split
// into three bfloat16 parts, a = a0 + a1 + a2 (each the rounding of what the ones before it leave: 8 + 8 + 8
// significant bits, the 24 of the value), and the product is summed from the six pairs whose weight is 2^-16
// or more,
//   a0 b0 | a0 b1 + a1 b0 + a1 b1 + a0 b2 + a2 b0
// each exact in 32 bits; what is left out, a1 b2 + a2 b1 + a2 b2, is at most about 2^-24 of |a b| (a1 is at most 2^-8
// of a, a2 2^-17), half a unit in the last place of a product.  The tensor core adds a product of
// 16 terms to its sum with the low bits cut off (measured: 2.3e-7 of the result after 256 terms, 4.4e-6
// after 4096, always towards zero), so the pairs of the second group, 2^-8 smaller, have an accumulator of
// their own, and every 256 of k both are read back and added in registers with ordinary rounding.  Six
// bfloat16 products at 2.2 PFLOP/s nominal leave about 375 TFLOP/s; the FP32 pipe has 75.
//
// A value whose first part is not finite (infinities, NaN, and from 2^128 - 2^119 on, which rounds to infinity) has no
// such parts: what the first leaves is inf - inf, and its sums come out as NaN.  A sum that is NaN is therefore taken
// once more on the FP32 pipe (plain_sums), from the values themselves: an infinity stays one, the largest values give
// what they should, and a true NaN stays.  The test for it costs 2 to 6 % of a product of few inputs.
//
// One persistent block per SM; its warps:
//   warp 17       copies pieces of 32 of k of A and B, float32 as they are, to a ring of raw buffers by TMA
//   warps 8 - 15  split a raw piece into the three parts and store them to a stage in the tensor core's
//                 swizzled layout.  An operand whose rows do not start on 16-byte boundaries they also copy,
//                 word by word with cp.async, several pieces ahead.  B's parts stay resident where all of
//                 its k fits.  (Loading straight to registers instead kept 16 KB in flight per SM: 312 us for
//                 the 300,000 x 59 x 128 weight gradient.)
//   warp 16       issues tcgen05.mma
//   warps 0 - 7   add up the accumulators and write C in 32 x 32 pieces through shared memory: by bulk copies
//                 where the arrays' layout allows (see Way), a column per lane where not; the residual is
//                 copied ahead while the tile before is written
// Every wait is bounded (see tc::Guard).
#include <cuda.h>

#include <utility>

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
constexpr int kBufBytes = 32 * 32 * 4;  // an epilogue warp's 32 x 32 piece
constexpr int kChunk = 8;          // k blocks between two additions in registers

// How an array of the epilogue is read or written: a column per lane; 32 x 32 boxes by TMA, where its rows start
// and end on 16-byte boundaries; or 32 whole rows at a time as one run of bytes, where they follow each other without
// gaps and one tile holds all columns (a 59-column record).
enum Way { kPlain, kBox, kDense };

struct Ctl {
  uint64_t res[kEpiWarps];
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t full[kStages], empty[kStages];
  uint64_t resident, acc_full[2], acc_empty[2], drain;
  uint32_t tmem, dead;
};
static_assert(sizeof(Ctl) <= kSmemCtl, "control block");

struct Args {
  CUtensorMap map_a, map_b, map_y, map_z, map_r;
  int y_way, z_way, r_way;
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
  int wait_limit;  // microseconds
  int drop;        // test hook: nothing is copied in, every wait for it runs out
};

__device__ __forceinline__ void tile_of(const Args& p, int bn, int t, int64_t& m0, int64_t& n0, int& split) {
  int nt = 0, mt = t;
  split = 0;
  if (p.n_tiles > 1) {
    mt = t / p.n_tiles;
    nt = t - mt * p.n_tiles;
  }
  if (p.splits > 1) {
    split = mt / p.m_tiles;
    mt -= split * p.m_tiles;
  }
  n0 = (int64_t)nt * bn;
  m0 = (int64_t)mt * kTileM;
}

// barrier of one team
template <int TEAM>
__device__ __forceinline__ void team_sync(int group) {
  if (group == 0) asm volatile("bar.sync 1, %0;" ::"n"(TEAM) : "memory");
  else asm volatile("bar.sync 2, %0;" ::"n"(TEAM) : "memory");
}

// cp.async of one word, or a zero
__device__ __forceinline__ void copy_word(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// One operand: pieces of EXT (m or n) x 32 (k).
//  raw    [x][k]: rows of 128 bytes; [k][x]: EXT / 32 boxes of 32 rows of 128 bytes.  16-byte units of a row are
//         swizzled (unit ^ row % 8), by TMA's 128-byte mode or by the copying threads.
//  parts  [x][k]: rows of 64 bytes, 64-byte swizzle; [k][x]: EXT / 64 chunks of 32 rows of 128 bytes, 128-byte swizzle.
template <int EXT, int TEAM>
struct Operand {
  static constexpr int kRaw = EXT * 128, kPlane = EXT * 64;
  static constexpr int kUnits = EXT * 4 / TEAM;  // of 8 values, per thread and piece
  const float* p;
  int64_t ld, ext, k;
  bool mn;

  // the copy of one piece by TMA
  __device__ __forceinline__ void copy_tma(const CUtensorMap* map, int64_t x0, int kb, uint32_t dst, uint32_t full) const {
    if (!mn) tc::tma_load_2d(dst, map, kb * kTileK, (int)x0, full);
    else
      for (int c = 0; c < EXT; c += 32) tc::tma_load_2d(dst + c * 128, map, (int)x0 + c, kb * kTileK, full);
  }
  // and by a team of splitters, a word per thread at a time, neighbouring threads along a row; rows outside of
  // the matrix are left as they are, k outside of it becomes zero
  __device__ __forceinline__ void copy_words(int tid, int64_t x0, int kb, uint32_t dst) const {
    constexpr int kWarps = TEAM / 32;
    const int lane = tid & 31, w = tid >> 5;
    const int64_t k0 = (int64_t)kb * kTileK;
    // rows w, w + kWarps, ...: their swizzle has at most two forms
    uint32_t at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) at[h] = dst + w * 128 + (((lane >> 2) ^ ((w + kWarps * h) & 7)) << 4) + (lane & 3) * 4;
    const int64_t step = ld * kWarps;
    if (!mn) {
      const bool in = k0 + lane < k;
      const float* src = in ? p + (x0 + w) * ld + k0 + lane : p;
      const int64_t by = in ? step : 0;
      const int rows = (int)min((int64_t)EXT, ext - x0) - w;
#pragma unroll 8
      for (int t = 0; t < EXT / kWarps; ++t, src += by)
        if (t * kWarps < rows) copy_word(at[t & 1] + t * (kWarps * 128), src, in);
    } else {
      const int rows = (int)min((int64_t)32, k - k0) - w;
      for (int c = 0; c < EXT && x0 + c < ext; c += 32) {
        const bool ci = x0 + c + lane < ext;
        const float* src = ci ? p + (k0 + w) * ld + x0 + c + lane : p;
        const int64_t by = ci ? step : 0;
#pragma unroll 4
        for (int t = 0; t < 32 / kWarps; ++t, src += by) {
          const bool in = t * kWarps < rows;
          copy_word(at[t & 1] + c * 128 + t * (kWarps * 128), in ? src : p, in && ci);
        }
      }
    }
  }
  // this thread's units of a raw piece, split: 8 values to 16 bytes in each of three planes
  __device__ __forceinline__ void split(int tid, int64_t x0, const unsigned char* raw, unsigned char* parts) const {
    // unit i lies a fixed distance from unit 0: the swizzles repeat every 8 rows
    int from, to, from_step, to_step;
    bool swap = false;
    if (!mn) {
      const int x = tid >> 2, u = tid & 3;
      from = x * 128 + (((2 * u) ^ (x & 7)) << 4);
      to = x * 64 + ((u ^ (x >> 1 & 3)) << 4);
      from_step = TEAM / 4 * 128, to_step = TEAM / 4 * 64;
    } else {
      const int u = tid % (EXT / 8), r = tid / (EXT / 8), v = 2 * (u & 3);
      if (x0 + u * 8 >= ext) return;  // reaches only sums that are not stored
      from = (u >> 2) * 4096 + r * 128 + ((v ^ (r & 7)) << 4);
      to = (u >> 3) * 4096 + r * 128 + (((u & 7) ^ (r & 7)) << 4);
      from_step = to_step = TEAM / (EXT / 8) * 128;
      swap = u >> 2 & 1;  // neighbouring boxes read their two halves in opposite order: distinct banks
    }
    float4 f[kUnits][2];
    const int first = swap ? from ^ 16 : from;  // the two halves differ in the unit's lowest bit
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      f[i][0] = *reinterpret_cast<const float4*>(raw + first + i * from_step);
      f[i][1] = *reinterpret_cast<const float4*>(raw + (first ^ 16) + i * from_step);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const float4 lo = swap ? f[i][1] : f[i][0], hi = swap ? f[i][0] : f[i][1];
      float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint4 o;
        uint32_t* w = &o.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
          if (q < 2) {
            v[2 * e] -= bf16_lo(w[e]);  // exact: what the rounding left
            v[2 * e + 1] -= bf16_hi(w[e]);
          }
        }
        *reinterpret_cast<uint4*>(parts + q * kPlane + to + i * to_step) = o;
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

// The sums of this lane's row and COLS columns that are NaN, again over the k blocks [kb, k_hi) by the FP32 pipe.  The
// warp does it together, eight columns at a time; rows and columns outside of C take the last one's values.  It is slow
// (counted: 1,600 cycles per k and tile of 64 columns, 3,200 per tile of 128, where every row has a NaN), but inside the
// waits' limit of 4 s up to a million of k.  Where all sums are NaN in earnest it ends with the first (20,000 x 1024 ->
// 1024 of NaN alone: 0.72 ms, 16 to their ends; clean 0.28).
template <int COLS>
__device__ __forceinline__ void plain_sums(const Args& p, float* sum, uint32_t row, uint32_t col0, int kb, int k_hi) {
  constexpr int kAt = 8;
  const uint32_t r = min(row, (uint32_t)p.m - 1);
  float all[COLS];  // indexed by a variable, so in memory: its registers are the loop's
#pragma unroll
  for (int i = 0; i < COLS; ++i) all[i] = sum[i];
#pragma unroll 1
  for (int c = 0; c < COLS; c += kAt) {
    float v[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) v[j] = 0.f;
#pragma unroll 1
    for (uint32_t k = (uint32_t)kb * kTileK; k < min((uint32_t)k_hi * kTileK, (uint32_t)p.k); ++k) {
      const float f = p.a[p.a_mn ? k * p.lda + r : r * p.lda + k];
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const uint32_t col = min(col0 + c + j, (uint32_t)p.n - 1);
        v[j] = fmaf(f, p.b[p.b_mn ? k * p.ldb + col : col * p.ldb + k], v[j]);
      }
      if (k % 32 == 31) {
        bool lost = true;  // a NaN stays one
#pragma unroll
        for (int j = 0; j < kAt; ++j) lost = lost && isnan(v[j]);
        if (__all_sync(0xffffffffu, lost)) break;
      }
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j)
      if (isnan(all[c + j])) all[c + j] = v[j];
  }
#pragma unroll
  for (int i = 0; i < COLS; ++i) sum[i] = all[i];
}

// Whether one of the first `count` of COLS sums is NaN, or two are infinities of either sign: the sum of all is NaN.  Two at
// a time, on the pipe that the splitters leave alone (106,489 x 8 -> 848 input gradient, whose tiles are all epilogue: 13 us
// of 207; 17 by largest values of three, 28 by comparisons).
template <int COLS>
__device__ __forceinline__ bool any_nan(const float* sum, int count) {
  float r;
  if (count >= COLS) {
    F2 v[2] = {F2(0.f), F2(0.f)};
#pragma unroll
    for (int i = 0; i < COLS; i += 4) v[0] = add2(v[0], F2(sum[i], sum[i + 1])), v[1] = add2(v[1], F2(sum[i + 2], sum[i + 3]));
    float a, b;
    add2(v[0], v[1]).get(a, b);
    r = a + b;
  } else {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < COLS - 1; ++i)
      if (i < count) v[i & 3] += sum[i];
    r = (v[0] + v[1]) + (v[2] + v[3]);
  }
  return isnan(r);
}

template <int ACT>
__device__ __forceinline__ void activate(float* v) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], ACT);
}

// GROUPS: the splitters work as one or two teams that take the pieces in turn.  Two hide a team's latency
// behind the other's, but each wants two raw buffers of its own.
// DENSE: arrays of the epilogue may take whole rows (tiles of 64 columns only).  A kernel of its own, so that the others
// do without the barriers between its warps (the 59-column record with residual 57.6 us, 60.5 by one kernel for all).
template <int BN, int GROUPS, bool DENSE>
__global__ void __launch_bounds__(kThreads, 1) k_mma_f32(const __grid_constant__ Args p) {
  constexpr int TEAM = kSplitters / GROUPS;
  static_assert(kStages % GROUPS == 0, "stages per team");
  using OpA = Operand<kTileM, TEAM>;
  using OpB = Operand<BN, TEAM>;
  constexpr int kAPlane = OpA::kPlane, kBPlane = OpB::kPlane;
  constexpr int kABytes = 3 * kAPlane, kBBytes = 3 * kBPlane;
  // Accumulators of a chunk of k, two chunks in flight: a0 b0, and one (128 columns) or two (64 columns) for the
  // smaller pairs
  constexpr int kAccs = BN == 64 ? 3 : 2, kTmem = 512;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
  unsigned char* res_b = smem + kSmemCtl;
  unsigned char* ring = res_b + (p.resident ? kBBytes * p.kblocks : 0);
  const int stage_bytes = kABytes + (p.resident ? 0 : kBBytes);
  unsigned char* raws = ring + stage_bytes * kStages;
  const int raw_bytes = OpA::kRaw + (p.resident ? 0 : OpB::kRaw);
  unsigned char* epi = raws + raw_bytes * p.raws;
  const int warp = tc::warp_index(), lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return tc::smem_addr(&b); };
  const bool a_words = !p.a_tma, b_words = !p.b_tma && !p.resident;
  const bool words = a_words || b_words;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.raws; ++s) {
      tc::mbar_init(bar(ctl.raw_full[s]), 1 + (words ? TEAM : 0));
      tc::mbar_init(bar(ctl.raw_empty[s]), TEAM / 32);
    }
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar(ctl.full[s]), TEAM / 32);
      tc::mbar_init(bar(ctl.empty[s]), 1);
    }
    tc::mbar_init(bar(ctl.resident), kSplitWarps);
    tc::mbar_init(bar(ctl.drain), 1);
    for (int i = 0; i < kEpiWarps; ++i) tc::mbar_init(bar(ctl.res[i]), 1);
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
  follow();
  const OpA a{p.a, p.lda, p.m, p.k, p.a_mn != 0};
  const OpB b{p.b, p.ldb, p.n, p.k, p.b_mn != 0};

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ raw copies by TMA
    if (!p.drop) {
      Cursor c;
      c.t = blockIdx.x;
      seek(p, BN, c, total);
      const uint32_t bytes = (p.a_tma ? OpA::kRaw : 0) + (p.b_tma && !p.resident ? OpB::kRaw : 0);
      int s = 0, it = 0;
      uint32_t parity = 1;
      bool ok = true;
      while (c.t < total) {
        ok = tc::mbar_wait_warp(bar(ctl.raw_empty[s]), parity, g);
        if (!ok) break;
        if (tc::elect_one()) {
          const uint32_t dst = tc::smem_addr(raws) + raw_bytes * s, full = bar(ctl.raw_full[s]);
          if (bytes) tc::mbar_expect_tx(full, bytes);
          else tc::mbar_arrive(full);
          if (p.a_tma) a.copy_tma(&p.map_a, c.m0, c.kb, dst, full);
          if (p.b_tma && !p.resident) b.copy_tma(&p.map_b, c.n0, c.kb, dst + OpA::kRaw, full);
        }
        __syncwarp();
        advance(p, BN, c, total);
        ++it;
        if (++s == p.raws) s = 0, parity ^= 1;
      }
      if (!ok && bytes) {  // gave up: no copy may be in flight when the block ends
        for (int i = it < p.raws ? 0 : it - p.raws; i < it; ++i)
          tc::mbar_drain(bar(ctl.raw_full[i % p.raws]), (uint32_t)(i / p.raws & 1), p.wait_limit);
      }
    }
  } else if (warp >= kEpiWarps && warp < kEpiWarps + kSplitWarps) {
    // ------------------------------------------------------------ splitters
    const int group = (warp - kEpiWarps) / (TEAM / 32), tid = (threadIdx.x - 32 * kEpiWarps) % TEAM;
    if (!p.drop) {
      if (p.resident && (int)blockIdx.x < total) {
        // B's parts, once, its words a piece at a time through the room of the epilogue, which waits for it
        const int64_t n0 = (int64_t)(blockIdx.x % p.n_tiles) * BN;
        unsigned char* room = epi + group * OpB::kRaw;
        for (int kb = group; kb < p.kblocks; kb += GROUPS) {
          b.copy_words(tid, n0, kb, tc::smem_addr(room));
          asm volatile("cp.async.wait_all;" ::: "memory");
          team_sync<TEAM>(group);
          b.split(tid, n0, room, res_b + kBBytes * kb);
          team_sync<TEAM>(group);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.resident));
      }
      // a place in a ring that this group's pieces take GROUPS further each time
      struct Ring {
        int s;
        uint32_t parity;
        __device__ __forceinline__ void step(int n, int size) {
          s += n;
          while (s >= size) s -= size, parity ^= 1;
        }
      };
      Cursor cur;
      cur.t = blockIdx.x;
      seek(p, BN, cur, total);
      Ring from{0, 0}, to{0, 1}, next{0, 1};
      auto skip = [&](Cursor& c, int n) {
        for (int i = 0; i < n && c.t < total; ++i) advance(p, BN, c, total);
      };
      skip(cur, group);
      from.step(group, p.raws), to.step(group, kStages), next.step(group, p.raws);
      Cursor ahead = cur;
      bool ok = true;
      // the next piece's words, when its raw buffer is free; its arrival follows the words
      auto copy_ahead = [&]() {
        if (!words || ahead.t >= total || !ok) return;
        ok = tc::mbar_wait_warp(bar(ctl.raw_empty[next.s]), next.parity, g);
        if (!ok) return;
        const uint32_t dst = tc::smem_addr(raws) + raw_bytes * next.s;
        if (a_words) a.copy_words(tid, ahead.m0, ahead.kb, dst);
        if (b_words) b.copy_words(tid, ahead.n0, ahead.kb, dst + OpA::kRaw);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(ctl.raw_full[next.s])) : "memory");
        skip(ahead, GROUPS);
        next.step(GROUPS, p.raws);
      };
      // its share of the ring, less the piece that is being split
      for (int i = 0; i < p.raws / GROUPS - 1; ++i) copy_ahead();
      while (cur.t < total) {
        copy_ahead();
        ok = ok && tc::mbar_wait_warp(bar(ctl.raw_full[from.s]), from.parity, g);
        ok = ok && tc::mbar_wait_warp(bar(ctl.empty[to.s]), to.parity, g);
        if (!ok) break;
        unsigned char* st = ring + stage_bytes * to.s;
        const unsigned char* raw = raws + raw_bytes * from.s;
        a.split(tid, cur.m0, raw, st);
        if (!p.resident) b.split(tid, cur.n0, raw + OpA::kRaw, st + kABytes);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar(ctl.raw_empty[from.s]));
          tc::mbar_arrive(bar(ctl.full[to.s]));
        }
        skip(cur, GROUPS);
        from.step(GROUPS, p.raws), to.step(GROUPS, kStages);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ matrix instructions
    {
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)p.a_mn << 15 | (uint32_t)p.b_mn << 16 |
                             (uint32_t)(BN >> 3) << 17 | (uint32_t)(kTileM >> 4) << 24;
      constexpr uint32_t kStepN = (uint32_t)(BN >> 3) << 17;  // BN columns more
      // 16 of k further: 32 bytes along a row, or 16 rows of 128 bytes; rows of 64 or of 128 bytes
      const uint32_t a_step = p.a_mn ? 16 * 128 : 32, b_step = p.b_mn ? 16 * 128 : 32;
      const uint64_t a_desc = p.a_mn ? tc::smem_desc(0, 4096, 1024) : tc::smem_desc_64(0, 512);
      const uint64_t b_desc = p.b_mn ? tc::smem_desc(0, 4096, 1024) : tc::smem_desc_64(0, 512);
      int s = 0, n_acc = 0;
      uint32_t parity = 0;
      bool ok = true;
      if (p.resident && (int)blockIdx.x < total) ok = tc::mbar_wait_warp(bar(ctl.resident), 0, g);
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        int64_t m0, n0;
        int split;
        tile_of(p, BN, t, m0, n0, split);
        int kb = split * p.kb_per_split;
        const int k_hi = min(kb + p.kb_per_split, p.kblocks);
        for (; ok && kb < k_hi; ++n_acc) {  // a chunk of k: one pair of accumulators
          const int acc = n_acc & 1, c_hi = min(kb + kChunk, k_hi);
          ok = tc::mbar_wait_warp(bar(ctl.acc_empty[acc]), (uint32_t)(n_acc >> 1 & 1) ^ 1, g);
          if (!ok) break;
          tc::fence_after();
          const uint32_t d = tmem + acc * (kTmem / 2);
          for (bool first = true; kb < c_hi; ++kb, first = false) {
            ok = tc::mbar_wait_warp(bar(ctl.full[s]), parity, g);
            if (!ok) break;
            tc::fence_after();
            const uint32_t as = tc::smem_addr(ring) + stage_bytes * s;
            const uint32_t bs = p.resident ? tc::smem_addr(res_b) + kBBytes * kb : as + kABytes;
            if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < kTileK / 16; ++i) {
              uint64_t da[3], db[3];
#pragma unroll
              for (int q = 0; q < 3; ++q) {
                da[q] = a_desc | ((as + q * kAPlane + i * a_step) & 0x3ffff) >> 4;
                db[q] = b_desc | ((bs + q * kBPlane + i * b_step) & 0x3ffff) >> 4;
              }
              // B's parts lie one behind the other, as one operand of up to 256 columns: several pairs per
              // instruction, and A read from shared memory half as often
              const uint32_t add = !first || i > 0;
              if constexpr (BN == 64) {
                tc::mma_bf16(d, da[0], db[0], idesc + 2 * kStepN, add);           // a0 (b0 b1 b2)
                tc::mma_bf16(d + BN, da[1], db[0], idesc + kStepN, 1);            // a1 (b0 b1)
                tc::mma_bf16(d + 2 * BN, da[2], db[0], idesc, 1);                 // a2 b0
              } else {
                tc::mma_bf16(d, da[0], db[0], idesc + kStepN, add);               // a0 (b0 b1)
                tc::mma_bf16(d + BN, da[1], db[0], idesc, 1);
                tc::mma_bf16(d + BN, da[0], db[2], idesc, 1);
                tc::mma_bf16(d + BN, da[1], db[1], idesc, 1);
                tc::mma_bf16(d + BN, da[2], db[0], idesc, 1);
              }
            }
            tc::mma_commit(bar(ctl.empty[s]));
            }
            __syncwarp();
            if (++s == kStages) s = 0, parity ^= 1;
          }
          if (ok && tc::elect_one()) tc::mma_commit(bar(ctl.acc_full[acc]));
          __syncwarp();
        }
      }
      if (!ok) {  // gave up: nothing may be in flight when the tensor memory is freed
        if (tc::elect_one()) tc::mma_commit(bar(ctl.drain));
        __syncwarp();
        tc::mbar_drain(bar(ctl.drain), 0, p.wait_limit);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int kCols = BN / 2;  // of this warp: 32 rows x kCols
    constexpr int kLoad = BN == 64 ? 32 : 8;  // columns per read of an accumulator: what the registers hold
    const int quad = warp & 3, half = warp >> 2, n = (int)p.n, m = (int)p.m;  // below 2^31
    // y, the residual, z: 32 KB each, 8 KB for the two warps that share 32 rows, 4 KB of it for this one
    unsigned char* const y_buf = epi + quad * (2 * kBufBytes);
    unsigned char* const r_buf = y_buf + kEpiWarps * kBufBytes;
    // (z and the residual: tiles of 64 columns only)
    unsigned char* const z_buf = r_buf + (p.residual ? kEpiWarps * kBufBytes : 0);
    const bool with_res = BN == 64 && p.residual && !p.part;
    const uint32_t res_bar = bar(ctl.res[DENSE ? quad : warp]);
    auto quad_sync = [&]() {
      __syncwarp();
      asm volatile("bar.sync %0, 64;" ::"r"(4 + quad) : "memory");
    };
    // Dense rows are written by the two warps of a quadrant together, which meet at a barrier without a limit.  Each
    // of them may give up in a wait of its own, so they agree after every such wait on whether they go on: the other
    // would wait for ever for one that has left.
    auto quad_agree = [&](bool mine) {
      uint32_t both;
      __syncwarp();
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 p, %2, 0;\n\t"
          "bar.red.and.pred q, %1, 64, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(both)
          : "r"(4 + quad), "r"((uint32_t)mine)
          : "memory");
      return both != 0;
    };
    int n_acc = 0, res_used = 0;
    bool res_flying = false;
    bool ok = true;
    if (p.resident && (int)blockIdx.x < total) ok = tc::mbar_wait_warp(bar(ctl.resident), 0, g);
    if (DENSE) ok = quad_agree(ok);
    // this warp's piece of tile t
    auto place = [&](int t, uint32_t& row0, uint32_t& col0, int& split) {
      int64_t m0, n0;
      tile_of(p, BN, t, m0, n0, split);
      row0 = (uint32_t)m0 + quad * 32;
      col0 = (uint32_t)n0 + half * kCols;
    };
    // the residual of tile t on its way to the buffer, while the tile before is written
    auto ask_residual = [&](int t) {
      if (t >= total) return;
      uint32_t row0, col0;
      int split;
      place(t, row0, col0, split);
      const int rows = min(32, (int)((int64_t)m - row0));
      if (rows <= 0) return;
      if (DENSE && p.r_way == kDense) {
        if (rows < 32) return;  // read where it is used
        if (half == 0 && tc::elect_one()) {
          tc::mbar_expect_tx(res_bar, 128 * n);
          tc::bulk_load(tc::smem_addr(r_buf), p.residual + (int64_t)row0 * n, 128 * n, res_bar);
        }
        res_flying = true;
      } else if (col0 < (uint32_t)n) {
        if (!DENSE && p.r_way == kBox) {
          if (tc::elect_one()) {
            tc::mbar_expect_tx(res_bar, kBufBytes);
            tc::tma_load_2d(tc::smem_addr(r_buf) + half * kBufBytes, &p.map_r, (int)col0, (int)row0, res_bar);
          }
          res_flying = true;
        } else if (col0 + lane < (uint32_t)n) {
          const float* src = p.residual + (int64_t)row0 * p.ldr + col0 + lane;
          const uint32_t dst = tc::smem_addr(r_buf) + half * kBufBytes;
#pragma unroll 8
          for (int r = 0; r < 32; ++r, src += p.ldr)
            if (r < rows) copy_word(dst + r * 128 + (lane ^ r) * 4, src, true);
        }
      }
      __syncwarp();
    };
    if (with_res && ok) ask_residual(blockIdx.x);
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      uint32_t row0, col0;
      int split;
      place(t, row0, col0, split);
      const int k_lo = split * p.kb_per_split, k_hi = min(k_lo + p.kb_per_split, p.kblocks);
      const bool in = row0 < (uint32_t)m && (DENSE || col0 < (uint32_t)(p.part ? p.ldp : n));
      const int rows = min(32, (int)((int64_t)m - row0));
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
          for (int c = 0; c < kCols; c += kLoad) {
            float v[kLoad];
#pragma unroll
            for (int q = kAccs - 1; q >= 0; --q) {
              tc::tmem_load<kLoad>(d + q * BN + c, v);
#pragma unroll
              for (int i = 0; i < kLoad; ++i) sum[c + i] += v[i];
            }
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.acc_empty[acc]));
      }
      if (DENSE) {
        // stores of the last tile have read the buffers (as below) before either warp writes to them
        if (tc::elect_one()) tc::bulk_wait_read0();
        ok = quad_agree(ok);
      }
      if (!ok) break;
      if (!in) {
        if (with_res) ask_residual(t + gridDim.x);
        continue;
      }
      if (__any_sync(0xffffffffu, row0 + lane < (uint32_t)m && any_nan<kCols>(sum, (int)(n - col0))))  // of what is stored
        plain_sums<kCols>(p, sum, row0 + lane, col0, k_lo, k_hi);
      if (p.part) {
        const int64_t row = row0 + lane;
        if (row < m) {
          float* out = p.part + ((int64_t)split * m + row) * p.ldp + col0;
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            if (col0 + c < p.ldp) *reinterpret_cast<float4*>(out + c) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
        }
        continue;
      }
      // a piece v (a lane: 32 columns of a row) through a buffer to its array
      auto write_piece = [&](const float* v, int way, unsigned char* b8, const CUtensorMap* map, float* out, int64_t ld, int c) {
        float* b = reinterpret_cast<float*>(b8 + half * kBufBytes);
        if (!DENSE && way == kBox) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(reinterpret_cast<unsigned char*>(b) + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          tc::fence_async_smem();
          __syncwarp();
          if (col0 + c < (uint32_t)n && tc::elect_one()) {
            tc::tma_store_2d(map, (int)col0 + c, (int)row0, tc::smem_addr(b));
            tc::bulk_commit();
          }
          __syncwarp();
        } else if (DENSE && way == kDense) {
          float* d = reinterpret_cast<float*>(b8) + lane * n + half * 32;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (half * 32 + i < n) d[i] = v[i];
          tc::fence_async_smem();
          quad_sync();
          out += (int64_t)row0 * n;
          if (rows == 32) {
            if (half == 0 && tc::elect_one()) {
              tc::bulk_store(out, tc::smem_addr(b8), 128 * n);
              tc::bulk_commit();
            }
            __syncwarp();
          } else {
            for (int e = half * 32 + lane; e < rows * n; e += 64) out[e] = reinterpret_cast<const float*>(b8)[e];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) b[lane * 32 + (i ^ lane)] = v[i];
          __syncwarp();
          if (col0 + c + lane < (uint32_t)n) {
            out += (int64_t)row0 * ld + col0 + c + lane;
#pragma unroll 4
            for (int r = 0; r < 32; ++r, out += ld)
              if (r < rows) *out = b[r * 32 + (lane ^ r)];
          }
          __syncwarp();
        }
      };
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        if (col0 + c >= (uint32_t)n && !DENSE) break;
        // stores of the last piece have read the buffers; a bulk store is its issuer's to wait for, and the
        // same lane of a warp issues all of that warp's
        if (!DENSE) {
          if (tc::elect_one()) tc::bulk_wait_read0();
          __syncwarp();
        }
        float* v = sum + c;
        if (p.bias) {
          const float bias = col0 + c + lane < (uint32_t)n ? p.bias[col0 + c + lane] : 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, bias, i);
        }
        if (BN == 64 && p.z) write_piece(v, p.z_way, z_buf, &p.map_z, p.z, p.ldz, c);
        if (p.act == GS_ACT_RELU) activate<GS_ACT_RELU>(v);
        else if (p.act == GS_ACT_GELU) activate<GS_ACT_GELU>(v);
        else if (p.act == GS_ACT_SILU) activate<GS_ACT_SILU>(v);
        if (with_res) {
          const float* b = reinterpret_cast<const float*>(r_buf + half * kBufBytes);
          if (DENSE && p.r_way == kDense && rows < 32) {
            const float* src = p.residual + (int64_t)(row0 + lane) * n + col0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (lane < rows && col0 + i < (uint32_t)n) v[i] += src[i];
          } else {
            if (p.r_way == kPlain) {
              asm volatile("cp.async.wait_all;" ::: "memory");
              __syncwarp();
              int l = lane;  // not to be known: the 32 addresses would be kept from tile to tile, on the stack
              asm volatile("" : "+r"(l));
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += b[l * 32 + (i ^ l)];
            } else {
              if (DENSE || col0 < (uint32_t)n) {
                ok = tc::mbar_wait_warp(res_bar, (uint32_t)(res_used & 1), g);
                if (ok) {
                  ++res_used;
                  res_flying = false;
                }
              }
              if (!DENSE && !ok) break;  // (what a dense tile's warp reads below without its residual is not used)
              if (DENSE) {
                const float* d = reinterpret_cast<const float*>(r_buf) + lane * n + half * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (half * 32 + i < n) v[i] += d[i];
              } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  const float4 f = *reinterpret_cast<const float4*>(reinterpret_cast<const unsigned char*>(b) + lane * 128 +
                                                                    ((q ^ (lane & 7)) << 4));
                  v[4 * q] += f.x, v[4 * q + 1] += f.y, v[4 * q + 2] += f.z, v[4 * q + 3] += f.w;
                }
              }
            }
          }
          tc::fence_async_smem();  // the reads above come before the next copy into the buffer
          if (DENSE) ok = quad_agree(ok);
          else __syncwarp();
          if (!ok) break;
          ask_residual(t + gridDim.x);
        }
        write_piece(v, p.y_way, y_buf, &p.map_y, p.y, p.ldy, c);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok)  // gave up: the copies in flight land before the block ends
      if (res_flying)
        tc::mbar_drain(res_bar, (uint32_t)(res_used & 1), p.wait_limit);
    if (tc::elect_one()) tc::bulk_wait0();
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
  bool swap;  // A and B change places: the parts hold C transposed
};

constexpr int kSms = 152;  // the device's; only speed depends on it

// Tiles of 128 columns where there are more than 64 and the tiles, or their ranges of k (at least four
// blocks, 128, each), are enough for the device; else of 64.
Plan plan_as(int64_t m, int64_t n, int64_t k) {
  Plan p;
  p.swap = false;
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

// With ranges of k the sums go through the fold kernel, which can as well transpose: then the operands stand
// so that the tiles' padding is least (a 59 x 128 weight gradient: one tile of 128 x 64, not of 128 x 128).
Plan plan_of(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_as(m, n, k);
  Plan q = plan_as(n, m, k);
  q.swap = true;
  auto area = [](const Plan& r) { return (int64_t)r.m_tiles * r.n_tiles * r.bn; };
  return p.splits > 1 && q.splits > 1 && area(q) < area(p) ? q : p;
}

// The shared memory of a launch: bytes of everything but the raw buffers, and how many of those fit.
struct Room {
  int fixed, raw, raws;
};
Room room_of(const Plan& pl, bool resident, int bufs) {
  const int a = 3 * kTileM * 64, b = 3 * pl.bn * 64;  // bytes of a block's parts
  Room r;
  r.fixed = 1024 + kSmemCtl + kEpiWarps * kBufBytes * bufs;
  const int64_t parts = resident ? (int64_t)b * pl.kblocks + kStages * a : kStages * (a + b);
  r.raw = kTileM * 128 + (resident ? 0 : pl.bn * 128);
  if (parts > kSmemMost - r.fixed) return {0, 0, 0};
  r.fixed += (int)parts;
  r.raws = (kSmemMost - r.fixed) / r.raw;
  if (r.raws > kMaxRaw) r.raws = kMaxRaw;
  return r;
}

template <int BN, int GROUPS, bool DENSE>
gs_status launch(Args& p, const Room& r, int grid, cudaStream_t st, const char* where) {
  // every team of splitters has raw buffers of its own: a wait for a buffer's next phase is then always made
  // by those who have seen the phase before it, as the phases' one bit of parity demands
  p.raws = r.raws - r.raws % GROUPS;
  if (p.raws < GROUPS) return gs::set_error(GS_ERR_INVALID, "%s: no room for raw buffers", where);
  cudaError_t e = gs::max_dynamic_smem((const void*)k_mma_f32<BN, GROUPS, DENSE>, kSmemMost);
  if (e == cudaSuccess) e = gs::launch(k_mma_f32<BN, GROUPS, DENSE>, dim3(grid), kThreads, r.fixed + p.raws * r.raw, st, p);
  return e == cudaSuccess ? GS_OK : gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

// (cols: of the rows that are written, in the end)
gs_status launch_any(Args& p, const Plan& pl, int64_t cols, cudaStream_t st, const char* where) {
  const int total = pl.m_tiles * pl.n_tiles * pl.splits;
  int grid = total < gs::num_sms() ? total : gs::num_sms();
  const int bufs = p.part ? 0 : 1 + (p.residual != nullptr) + (p.z != nullptr);
  Room r = room_of(pl, true, bufs);
  // resident B: one range of columns per block, and three raw buffers of A beside it
  if (pl.splits == 1 && pl.n_tiles <= 4 && total >= 2 * grid && r.raws >= 3) {
    p.resident = 1;
    grid -= grid % pl.n_tiles;
  } else {
    r = room_of(pl, false, bufs);
  }
  // Ranges of k write no array, and take the kernel that the other product of a backward takes, whose instructions are at
  // hand: both write rows of as many columns (575 x 7 -> 214 backward 24.2 us, 28.3 by two kernels; 151,069 x 10 -> 67 79
  // and 85).
  const bool dense = p.part ? cols % 4 != 0 && cols <= 64 : p.y_way == kDense || p.z_way == kDense || p.r_way == kDense;
  if (pl.bn == 128) return launch<128, 1, false>(p, r, grid, st, where);
  if (dense) return r.raws >= 4 ? launch<64, 2, true>(p, r, grid, st, where) : launch<64, 1, true>(p, r, grid, st, where);
  return r.raws >= 4 ? launch<64, 2, false>(p, r, grid, st, where) : launch<64, 1, false>(p, r, grid, st, where);
}

}  // namespace

namespace gs {

size_t f32_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_of(m, n, k);
  return p.splits > 1 ? (size_t)p.splits * (p.swap ? n : m) * p.ldp * sizeof(float) : 0;
}

gs_status f32_run(const MmaProduct& product, void* workspace, int32_t* status, cudaStream_t st, const char* where) {
  MmaProduct q = product;
  Plan pl = plan_of(q.m, q.n, q.k);
  if (pl.swap) {
    std::swap(q.a, q.b);
    std::swap(q.lda, q.ldb);
    std::swap(q.a_mn, q.b_mn);
    std::swap(q.m, q.n);
    std::swap(q.a_pad, q.b_pad);
  }
  if (pl.bn == 128 && pl.splits == 1 && (q.residual || q.z)) {  // their buffers and registers leave no room for 128 columns
    pl.bn = 64;
    pl.n_tiles = (int)ceil_div(q.n, 64);
  }
  if ((int64_t)pl.m_tiles * pl.n_tiles * pl.splits > 0x7fffffff) return set_error(GS_ERR_INVALID, "%s: too many tiles", where);
  Args p{};
  p.a = static_cast<const float*>(q.a), p.b = static_cast<const float*>(q.b), p.lda = q.lda, p.ldb = q.ldb;
  p.m = q.m, p.n = q.n, p.k = q.k;
  p.m_tiles = pl.m_tiles, p.n_tiles = pl.n_tiles, p.splits = pl.splits, p.kblocks = pl.kblocks;
  p.kb_per_split = pl.kb_per_split;
  p.a_mn = q.a_mn, p.b_mn = q.b_mn;
  p.a_tma = tma_takes(q.a, q.a_mn ? q.k : q.m, (q.a_mn ? q.m : q.k) + q.a_pad, q.lda, GS_F32);
  p.b_tma = tma_takes(q.b, q.b_mn ? q.k : q.n, (q.b_mn ? q.n : q.k) + q.b_pad, q.ldb, GS_F32);
  bool ok = true;
  if (p.a_tma)
    ok = q.a_mn ? encode_map(&p.map_a, q.a, q.k, q.m + q.a_pad, q.lda, 32, GS_F32)
                : encode_map(&p.map_a, q.a, q.m, q.k + q.a_pad, q.lda, kTileM, GS_F32);
  if (p.b_tma)
    ok = ok && (q.b_mn ? encode_map(&p.map_b, q.b, q.k, q.n + q.b_pad, q.ldb, 32, GS_F32)
                       : encode_map(&p.map_b, q.b, q.n, q.k + q.b_pad, q.ldb, pl.bn, GS_F32));
  if (!ok) return set_error(GS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", where);
  p.bias = static_cast<const float*>(q.bias), p.residual = static_cast<const float*>(q.residual);
  p.y = static_cast<float*>(q.y), p.z = static_cast<float*>(q.z), p.ldr = q.ldr, p.ldy = q.ldy, p.ldz = q.ldz;
  p.act = q.act;
  p.part = pl.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  p.ldp = pl.ldp;
  if (!p.part) {
    auto way = [&](const void* at, int64_t ld, CUtensorMap* map, int& w) {
      w = kPlain;
      if (!at) return true;
      if (tma_takes(at, q.m, q.n, ld, GS_F32)) {
        w = kBox;
        return encode_map(map, at, q.m, q.n, ld, 32, GS_F32);
      }
      if (pl.bn == 64 && pl.n_tiles == 1 && ld == q.n && aligned16(at)) w = kDense;
      return true;
    };
    if (!way(q.y, q.ldy, &p.map_y, p.y_way) || !way(q.z, q.ldz, &p.map_z, p.z_way) || !way(q.residual, q.ldr, &p.map_r, p.r_way))
      return set_error(GS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", where);
  }
  p.status = status, p.wait_limit = wait_us(), p.drop = take_drop_copy();
  if (gs_status s = launch_any(p, pl, product.n, st, where)) return s;
  if (!p.part) {
    if (q.also.part) launch_column_fold<float>(q.also, st);
    return check_launch(where);
  }
  launch_fold(FoldArgs<float>{p.part, p.bias, p.residual, p.y, p.z, q.m, pl.ldp, q.ldr, q.ldy, q.ldz, pl.splits, (int)q.n, q.act, pl.swap,
                              q.also},
              st);
  return check_launch(where);
}

}  // namespace gs
