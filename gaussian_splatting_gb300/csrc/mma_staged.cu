// bfloat16 products whose operands pass through registers on their way to the tensor cores: those whose
// rows do not start on 16-byte boundaries, which TMA cannot copy.
//
// C(m, n) = sum over k of A(m, k) B(n, k) and the epilogue as in mma.cu.
// Warps of the one persistent block per SM:
//   warps 8 - 15  load pieces of A and B (16-byte loads where rows start on such boundaries, single
//                 elements where not) and store them to a shared-memory stage in the tensor core's
//                 128-byte-swizzled layout; the next pieces' loads are in flight meanwhile.  B stays
//                 resident where all of its k fits.
//   warp 16       issues tcgen05.mma
//   warps 0 - 7   read the accumulators and write C: 32 x 32 pieces through shared memory, so that the
//                 epilogue reads and writes whole rows of 32 columns at any alignment
#include "mma.cuh"
#include "tcgen05.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kEpiWarps = 8, kLoadWarps = 8;
constexpr int kLoaders = 32 * kLoadWarps;
constexpr int kThreads = 32 * (kEpiWarps + kLoadWarps + 1);
constexpr int kTileM = 128, kTileK = 64;
constexpr int kMaxStages = 6;
constexpr int kSmemMost = 232448;  // 227 KB
constexpr int kSmemCtl = 1024;
constexpr int kPitch = 33;         // floats per row of an epilogue buffer: rows and columns both hit distinct banks
constexpr int kBufBytes = 32 * kPitch * 4;

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t resident, acc_full[2], acc_empty[2], drain;
  uint32_t tmem, dead;
};

struct Args {
  const bf16* a;
  const bf16* b;
  int64_t lda, ldb;
  int64_t m, n, k;
  int m_tiles, n_tiles, splits, kblocks, kb_per_split;
  int stages, resident;
  int a_mn, b_mn, a_vec, b_vec;
  const bf16* bias;
  const bf16* residual;
  bf16* y;
  bf16* z;
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

// 8 consecutive elements at p, those at or past `left` as zeros
__device__ __forceinline__ uint4 load8(const bf16* p, int64_t left, bool vec) {
  if (vec && left >= 8) return *reinterpret_cast<const uint4*>(p);
  uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < left ? reinterpret_cast<const uint16_t*>(p)[i] : 0;
  return make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                    e[6] | (uint32_t)e[7] << 16);
}

// One operand as the loaders see it: pieces of EXT (m or n) x 16 (one step of the tensor core), a unit
// of 8 elements per thread.
constexpr int kPieces = kTileK / 16;  // of a k block
constexpr int kDepth = 3;             // pieces of a thread in registers, all but one of them in flight

template <int EXT>
struct Operand {
  static_assert(EXT * 2 <= kLoaders, "one unit per thread");
  const bf16* p;
  int64_t ld, ext, k;
  bool mn, vec;

  // the unit of thread tid: its row or column x, its k, and its place in a plane; whether it has one
  __device__ __forceinline__ bool place(int tid, int piece, int& x, int& kk, int& at) const {
    if (!mn) {
      x = tid >> 1;
      const int u = (tid & 1) + 2 * piece;
      kk = u * 8;
      at = x * 128 + ((u ^ (x & 7)) << 4);
    } else {
      const int u = tid % (EXT / 8);
      kk = tid / (EXT / 8) + 16 * piece;
      x = u * 8;
      at = (u >> 3) * (kTileK * 128) + kk * 128 + (((u & 7) ^ (kk & 7)) << 4);
    }
    return tid < EXT * 2;
  }
  __device__ __forceinline__ uint4 load(int tid, int piece, int64_t x0, int64_t k0) const {
    int x, kk, at;
    const bool mine = place(tid, piece, x, kk, at);
    const int64_t gx = x0 + x, gk = k0 + kk;
    if (!mine || gx >= ext) return make_uint4(0u, 0u, 0u, 0u);
    if (!mn) return load8(p + gx * ld + gk, k - gk, vec);
    return load8(p + gk * ld + gx, gk < k ? ext - gx : 0, vec);
  }
  // Rows and columns outside of the matrix are not written: they only reach sums that are not stored.
  __device__ __forceinline__ void store(int tid, int piece, int64_t x0, unsigned char* stage, uint4 v) const {
    int x, kk, at;
    if (place(tid, piece, x, kk, at) && x0 + x < ext) *reinterpret_cast<uint4*>(stage + at) = v;
  }
};

// Where a loader stands: tile t, k block kb of [.., k_hi), piece h.
struct Cursor {
  int64_t m0, n0;
  int t, kb, k_hi, h;
};

__device__ __forceinline__ void seek(const Args& p, int bn, Cursor& c, int total) {
  if (c.t >= total) return;
  int split;
  tile_of(p, bn, c.t, c.m0, c.n0, split);
  c.kb = split * p.kb_per_split;
  c.k_hi = min(c.kb + p.kb_per_split, p.kblocks);
  c.h = 0;
}

__device__ __forceinline__ void advance(const Args& p, int bn, Cursor& c, int total) {
  if (++c.h < kPieces) return;
  c.h = 0;
  if (++c.kb == c.k_hi) {
    c.t += gridDim.x;
    seek(p, bn, c, total);
  }
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) k_mma_staged(const __grid_constant__ Args p) {
  constexpr int kABytes = kTileM * kTileK * 2, kBBytes = BN * kTileK * 2;
  constexpr int kTmem = BN * 2;  // columns, two tiles in flight
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
  unsigned char* res_b = smem + kSmemCtl;
  unsigned char* ring = res_b + (p.resident ? (size_t)kBBytes * p.kblocks : 0);
  const int stage_bytes = kABytes + (p.resident ? 0 : kBBytes);
  unsigned char* epi = ring + (size_t)stage_bytes * p.stages;
  const int warp = tc::warp_index(), lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return tc::smem_addr(&b); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(bar(ctl.full[s]), kLoadWarps);
      tc::mbar_init(bar(ctl.empty[s]), 1);
    }
    tc::mbar_init(bar(ctl.resident), kLoadWarps);
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
  if (warp == kEpiWarps + kLoadWarps) tc::tmem_alloc(tc::smem_addr(&ctl.tmem), kTmem);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = ctl.tmem;

  if (warp >= kEpiWarps && warp < kEpiWarps + kLoadWarps) {
    // ------------------------------------------------------------ loaders
    const int tid = threadIdx.x - 32 * kEpiWarps;
    const Operand<kTileM> a{p.a, p.lda, p.m, p.k, p.a_mn != 0, p.a_vec != 0};
    const Operand<BN> b{p.b, p.ldb, p.n, p.k, p.b_mn != 0, p.b_vec != 0};
    if (!p.drop) {
      if (p.resident) {
        const int64_t n0 = (int64_t)(blockIdx.x % p.n_tiles) * BN;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          uint4 f[kPieces];
#pragma unroll
          for (int h = 0; h < kPieces; ++h) f[h] = b.load(tid, h, n0, (int64_t)kb * kTileK);
#pragma unroll
          for (int h = 0; h < kPieces; ++h) b.store(tid, h, n0, res_b + (size_t)kBBytes * kb, f[h]);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.resident));
      }
      Cursor cur;
      cur.t = blockIdx.x;
      seek(p, BN, cur, total);
      Cursor ahead = cur;
      uint4 fa[kDepth], fb[kDepth];
      auto load = [&](int w) {
        if (ahead.t >= total) return;
        fa[w] = a.load(tid, ahead.h, ahead.m0, (int64_t)ahead.kb * kTileK);
        if (!p.resident) fb[w] = b.load(tid, ahead.h, ahead.n0, (int64_t)ahead.kb * kTileK);
        advance(p, BN, ahead, total);
      };
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
#pragma unroll
      for (int w = 0; w + 1 < kDepth; ++w) load(w);
      while (ok && cur.t < total) {
#pragma unroll
        for (int w = 0; w < kDepth; ++w) {  // the register sets alternate
          if (!ok || cur.t >= total) break;
          load((w + kDepth - 1) % kDepth);
          if (cur.h == 0) ok = tc::mbar_wait_warp(bar(ctl.empty[s]), parity, g);
          if (!ok) break;
          unsigned char* st = ring + (size_t)stage_bytes * s;
          a.store(tid, cur.h, cur.m0, st, fa[w]);
          if (!p.resident) b.store(tid, cur.h, cur.n0, st + kABytes, fb[w]);
          if (cur.h == kPieces - 1) {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(ctl.full[s]));
            if (++s == p.stages) s = 0, parity ^= 1;
          }
          advance(p, BN, cur, total);
        }
      }
    }
  } else if (warp == kEpiWarps + kLoadWarps) {
    // ------------------------------------------------------------ matrix instructions
    {
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)p.a_mn << 15 | (uint32_t)p.b_mn << 16 |
                             (uint32_t)(BN >> 3) << 17 | (uint32_t)(kTileM >> 4) << 24;
      const uint32_t a_step = p.a_mn ? 16 * 128 : 32, b_step = p.b_mn ? 16 * 128 : 32;
      int it = 0, n_acc = 0;
      bool ok = true;
      if (p.resident && blockIdx.x < total) ok = tc::mbar_wait_warp(bar(ctl.resident), 0, g);
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        int64_t m0, n0;
        int split;
        tile_of(p, BN, t, m0, n0, split);
        int kb = split * p.kb_per_split;
        const int k_hi = min(kb + p.kb_per_split, p.kblocks);
        const int acc = n_acc & 1;
        ok = tc::mbar_wait_warp(bar(ctl.acc_empty[acc]), (uint32_t)(n_acc >> 1 & 1) ^ 1, g);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = tmem + acc * BN;
        for (bool first = true; kb < k_hi; ++kb, ++it, first = false) {
          const int s = it % p.stages;
          ok = tc::mbar_wait_warp(bar(ctl.full[s]), (uint32_t)(it / p.stages & 1), g);
          if (!ok) break;
          tc::fence_after();
          const uint32_t as = tc::smem_addr(ring) + stage_bytes * s;
          const uint32_t bs = p.resident ? tc::smem_addr(res_b) + kBBytes * kb : as + kABytes;
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < kTileK / 16; ++i)
            tc::mma_bf16(d, tc::smem_desc(as + i * a_step, kTileK * 128, 1024), tc::smem_desc(bs + i * b_step, kTileK * 128, 1024),
                         idesc, !first || i > 0);
            tc::mma_commit(bar(ctl.empty[s]));
          }
          __syncwarp();
        }
        if (ok && tc::elect_one()) tc::mma_commit(bar(ctl.acc_full[acc]));
        __syncwarp();
        ++n_acc;
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
    const int quad = warp & 3, half = warp >> 2;
    float* buf = reinterpret_cast<float*>(epi + warp * kBufBytes);
    int n_acc = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      int64_t m0, n0;
      int split;
      tile_of(p, BN, t, m0, n0, split);
      const int64_t row0 = m0 + quad * 32, col0 = n0 + half * kCols;
      const bool in = row0 < p.m && col0 < (p.part ? p.ldp : p.n);
      const int acc = n_acc & 1;
      ok = tc::mbar_wait_warp(bar(ctl.acc_full[acc]), (uint32_t)(n_acc >> 1 & 1), g);
      if (!ok) break;
      ++n_acc;
      tc::fence_after();
      const uint32_t d = tmem + acc * BN + ((uint32_t)(quad * 32) << 16) + half * kCols;
      const int rows = (int)min((int64_t)32, p.m - row0);
      for (int c = 0; in && c < kCols; c += 32) {
        float sum[32];
        tc::tmem_load32(d + c, sum);
        if (p.part) {
          const int64_t row = row0 + lane;
          if (row < p.m) {
            float* out = p.part + ((int64_t)split * p.m + row) * p.ldp + col0 + c;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              if (col0 + c + i < p.ldp)
                *reinterpret_cast<float4*>(out + i) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
          }
          continue;
        }
        // a lane owns a column from here on
        const int64_t col = col0 + c + lane;
        const bool ci = col < p.n;
        const float bias = p.bias && ci ? __bfloat162float(p.bias[col]) : 0.f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) buf[lane * kPitch + i] = sum[i];
        __syncwarp();
        if (!ci) continue;
        const bf16* res = p.residual + row0 * p.ldr + col;
        bf16* y = p.y + row0 * p.ldy + col;
        bf16* z = p.z + row0 * p.ldz + col;
        for (int r0 = 0; r0 < rows; r0 += 8) {
          bf16 rr[8];  // loads in flight
          if (p.residual) {
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (r0 + r < rows) rr[r] = res[(r0 + r) * p.ldr];
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            if (r0 + r >= rows) break;
            float v = buf[(r0 + r) * kPitch + lane] + bias;
            if (p.z) z[(r0 + r) * p.ldz] = __float2bfloat16_rn(v);
            v = act_value(v, p.act);
            if (p.residual) v += __bfloat162float(rr[r]);
            y[(r0 + r) * p.ldy] = __float2bfloat16_rn(v);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(ctl.acc_empty[acc]));
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kEpiWarps + kLoadWarps) tc::tmem_dealloc(tmem, kTmem);
}

// ---------------------------------------------------------------- host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int bn, m_tiles, n_tiles, splits, kblocks, kb_per_split;
  int64_t ldp;
};

constexpr int kSms = 152;  // the device's; only speed depends on it

// 128 columns per tile where there are more than 64 and enough tiles; ranges of k of at least two blocks
// (128) where there are too few tiles for the device.
Plan plan_of(int64_t m, int64_t n, int64_t k) {
  Plan p;
  p.m_tiles = (int)ceil_div(m, kTileM);
  p.kblocks = (int)ceil_div(k, kTileK);
  p.bn = n <= 64 || (int64_t)p.m_tiles * ceil_div(n, 128) < kSms / 2 ? 64 : 128;
  p.n_tiles = (int)ceil_div(n, p.bn);
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  int64_t splits = tiles >= kSms ? 1 : kSms / tiles;
  if (splits > p.kblocks / 2) splits = p.kblocks / 2;
  if (splits < 1) splits = 1;
  p.kb_per_split = (int)ceil_div(p.kblocks, splits);
  p.splits = (int)ceil_div(p.kblocks, p.kb_per_split);
  p.ldp = ceil_div(n, 4) * 4;
  return p;
}

template <int BN>
gs_status launch(Args& p, const Plan& pl, cudaStream_t st, const char* where) {
  constexpr int kA = kTileM * kTileK * 2, kB = BN * kTileK * 2;
  const int64_t total = (int64_t)pl.m_tiles * pl.n_tiles * pl.splits;
  int grid = (int)(total < gs::num_sms() ? total : gs::num_sms());
  const int room = kSmemMost - 1024 - kSmemCtl - kEpiWarps * kBufBytes;
  // resident B: one range of columns per block, and at least two stages of A beside it
  if (pl.splits == 1 && pl.n_tiles <= 4 && total >= 2 * grid && (int64_t)kB * pl.kblocks + 2 * kA <= room) {
    p.resident = 1;
    grid -= grid % pl.n_tiles;
  }
  const int stage = kA + (p.resident ? 0 : kB);
  const int stages = (room - (p.resident ? kB * pl.kblocks : 0)) / stage;
  p.stages = stages < kMaxStages ? stages : kMaxStages;
  const int smem = kSmemMost - room + (p.resident ? kB * pl.kblocks : 0) + p.stages * stage;
  const cudaError_t e = gs::max_dynamic_smem((const void*)k_mma_staged<BN>, kSmemMost);
  if (e != cudaSuccess) return gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  k_mma_staged<BN><<<grid, kThreads, smem, st>>>(p);
  return gs::check_launch(where);
}

}  // namespace

namespace gs {

size_t staged_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_of(m, n, k);
  return p.splits > 1 ? (size_t)p.splits * m * p.ldp * sizeof(float) : 0;
}

gs_status staged_run(const MmaProduct& q, void* workspace, int32_t* status, cudaStream_t st, const char* where) {
  const Plan pl = plan_of(q.m, q.n, q.k);
  if ((int64_t)pl.m_tiles * pl.n_tiles * pl.splits > 0x7fffffff)
    return set_error(GS_ERR_INVALID, "%s: too many tiles", where);
  Args p{};
  p.a = static_cast<const bf16*>(q.a), p.b = static_cast<const bf16*>(q.b), p.lda = q.lda, p.ldb = q.ldb, p.m = q.m, p.n = q.n, p.k = q.k;
  p.m_tiles = pl.m_tiles, p.n_tiles = pl.n_tiles, p.splits = pl.splits, p.kblocks = pl.kblocks;
  p.kb_per_split = pl.kb_per_split;
  p.a_mn = q.a_mn, p.b_mn = q.b_mn;
  p.a_vec = rows_aligned16(q.a, q.a_mn ? q.k : q.m, q.lda, GS_BF16);
  p.b_vec = rows_aligned16(q.b, q.b_mn ? q.k : q.n, q.ldb, GS_BF16);
  p.bias = static_cast<const bf16*>(q.bias), p.residual = static_cast<const bf16*>(q.residual);
  p.y = static_cast<bf16*>(q.y), p.z = static_cast<bf16*>(q.z), p.ldr = q.ldr, p.ldy = q.ldy, p.ldz = q.ldz;
  p.act = q.act;
  p.part = pl.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  p.ldp = pl.ldp;
  p.status = status, p.wait_limit = wait_us(), p.drop = take_drop_copy();
  if (gs_status s = pl.bn == 64 ? launch<64>(p, pl, st, where) : launch<128>(p, pl, st, where)) return s;
  if (!p.part) return GS_OK;
  launch_fold(FoldArgs<bf16>{p.part, p.bias, p.residual, p.y, p.z, q.m, pl.ldp, q.ldr, q.ldy, q.ldz, pl.splits, (int)q.n, q.act, false},
              st);
  return check_launch(where);
}

}  // namespace gs
