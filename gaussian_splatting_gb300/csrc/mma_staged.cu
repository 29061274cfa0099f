// bfloat16 products whose operands TMA cannot copy: those whose rows do not start and end on 16-byte boundaries.
//
// C(m, n) = sum over k of A(m, k) B(n, k) and the epilogue as in mma.cu.
// Warps of the one persistent block per SM:
//   warps 8 - 15  load segments of 64 neighbouring elements of A and B by words (a word per lane, coalesced), shift
//                 them to the segment's alignment and store them to a stage in the tensor core's
//                 128-byte-swizzled layout; the next k block's words are in flight meanwhile.  B stays
//                 resident where all of its k fits.
//   warp 16       issues tcgen05.mma
//   warps 0 - 7   read the accumulators and write C: 32 x 32 pieces through shared memory, so that the
//                 epilogue reads and writes whole rows of 32 columns at any alignment
// (What did not do, 300K x 255 -> 257: eight elements per lane, loaded one by one, 16 cache lines per load, 634 us;
// cp.async by words, one per 13 cycles and SM, 481 us without epilogue.)
#include "mma.cuh"
#include "tcgen05.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kEpiWarps = 8, kLoadWarps = 8;
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
  int stages;
  int a_mn, b_mn;
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

// One operand as the loaders see it.  A k block of EXT (m or n) x 64 (k) is EXT segments of 64 neighbouring
// elements in memory, 128 bytes of the stage each: a row each of an operand stored [x][k]; of one stored
// [k][x], 64 rows of each 64 columns.  Warp w has the segments w, w + 8, ...: eight of each 64.
constexpr int kSegs = 64 / kLoadWarps;

template <int EXT>
struct Operand {
  static constexpr int kGroups = EXT / 64;
  // a warp's words of a k block: word l of a segment in lane l, the 33rd of segment i in lane i
  struct Words {
    uint32_t word[kGroups][kSegs], last[kGroups];
  };
  const bf16* p;
  int64_t ld, ext, k;
  bool mn;
  uintptr_t lo, hi;  // the array's bytes

  // Where a warp's segments of the tile at x0 start, and what is left of the operand from there on (m or n).
  // Kept by the loaders from block to block.
  struct Spot {
    uintptr_t at;
    int rest;
  };
  __device__ __forceinline__ Spot spot(int warp, int64_t x0) const {
    if (!mn) return {reinterpret_cast<uintptr_t>(p + (x0 + warp) * ld), (int)(ext - x0) - warp};
    return {reinterpret_cast<uintptr_t>(p + warp * ld + x0), (int)(ext - x0)};
  }
  // A warp's segments of the c-th 64 of k block kb: the first one's address, the bytes between two, how many
  // elements of each are in the matrix, how many segments are.  `skip`: those that are not would only reach sums
  // that are not stored, and are not written; else they are zeros.
  struct View {
    uintptr_t at;
    int64_t step;
    int left, rows;
    bool skip, inside;  // inside: all segments are there, and all their words lie in the array
  };
  __device__ __forceinline__ View view(int warp, const Spot& o, int c, int kb) const {
    View v;
    v.step = ld * (2 * kLoadWarps);
    const int k_left = (int)k - kb * kTileK;
    const int along = (mn ? o.rest : k_left) - (mn ? c * 64 : 0), across = mn ? k_left - warp : o.rest - c * 64;
    v.left = min(along, 64);
    v.rows = v.left <= 0 ? 0 : max(0, min((across + kLoadWarps - 1) / kLoadWarps, kSegs));
    v.skip = !mn || v.left <= 0;
    // 64 further along k, 64 further along the tile: bytes in a row, or rows
    v.at = o.at + (mn ? (int64_t)kb * (kTileK / kLoadWarps) * v.step + c * 128 : (int64_t)kb * 128 + c * (64 / kLoadWarps) * v.step);
    v.inside = v.rows == kSegs && v.at >= lo + 2 && v.at + (kSegs - 1) * v.step + 2 * 64 + 4 <= hi;
    return v;
  }
  __device__ __forceinline__ void load(int warp, int lane, const Spot& o, int kb, Words& f) const {
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      const View v = view(warp, o, c, kb);
      uintptr_t at = v.at;
      if (v.inside) {
        // (elements past `left` are read too where they lie in the array, and cut off later)
#pragma unroll
        for (int i = 0; i < kSegs; ++i, at += v.step)
          f.word[c][i] = *reinterpret_cast<const uint32_t*>((at & ~uintptr_t(3)) + 4 * lane);
        if (lane < kSegs)
          f.last[c] = *reinterpret_cast<const uint32_t*>(((v.at + lane * v.step) & ~uintptr_t(3)) + 128);
      } else {
        // words that lie in the array as a whole; the two that may not are seen to in shift()
#pragma unroll
        for (int i = 0; i < kSegs; ++i, at += v.step) {
          const uintptr_t word = (at & ~uintptr_t(3)) + 4 * lane;
          f.word[c][i] = 0;
          if (i < v.rows && word >= lo && word + 4 <= hi) f.word[c][i] = *reinterpret_cast<const uint32_t*>(word);
        }
        const uintptr_t word = ((v.at + lane * v.step) & ~uintptr_t(3)) + 128;
        f.last[c] = 0;
        if (lane < v.rows && word + 4 <= hi) f.last[c] = *reinterpret_cast<const uint32_t*>(word);
      }
    }
  }
  __device__ __forceinline__ void shift(int warp, int lane, const Spot& o, int kb, const Words& f, uint32_t stage) const {
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      const View v = view(warp, o, c, kb);
      if (v.skip && v.rows == 0) continue;
      uintptr_t at = v.at;
      // segments 8 further have the same swizzle
      const uint32_t to = stage + (c * 64 + warp) * 128 + (((lane >> 2) ^ (warp & 7)) << 4) + (lane & 3) * 4;
      const uint32_t keep = 2 * lane + 1 < v.left ? 0xffffffffu : 2 * lane < v.left ? 0xffffu : 0u;
      uint32_t e[kSegs];  // all of them before the first is stored: the shuffles overlap
#pragma unroll
      for (int i = 0; i < kSegs; ++i, at += v.step) {
        uint32_t next = __shfl_down_sync(0xffffffffu, f.word[c][i], 1);
        const uint32_t last = __shfl_sync(0xffffffffu, f.last[c], i);
        if (lane == 31) next = last;
        e[i] = __funnelshift_r(f.word[c][i], next, (uint32_t)(at & 2) * 8) & keep;
      }
      if (!v.inside) {
        at = v.at;
#pragma unroll
        for (int i = 0; i < kSegs; ++i, at += v.step) {
          if (i >= v.rows) {
            e[i] = 0;
          } else if ((at & ~uintptr_t(3)) < lo || at + 2 * v.left + 2 > hi) {
            // a segment with the array's first or last word: element by element
            const uint16_t* q = reinterpret_cast<const uint16_t*>(at) + 2 * lane;
            e[i] = 2 * lane < v.left ? q[0] : 0;
            if (2 * lane + 1 < v.left) e[i] |= (uint32_t)q[1] << 16;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kSegs; ++i)
        if (i < v.rows || !v.skip)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + i * (kLoadWarps * 128)), "r"(e[i]) : "memory");
    }
  }
};

// Where a loader stands: tile t, k block kb of [.., k_hi), its segments' places.
template <int BN>
struct Cursor {
  typename Operand<kTileM>::Spot a;
  typename Operand<BN>::Spot b;
  int t, kb, k_hi;

  __device__ __forceinline__ void seek(const Args& p, const Operand<kTileM>& oa, const Operand<BN>& ob, int warp, int total) {
    if (t >= total) return;
    int64_t m0, n0;
    int split;
    tile_of(p, BN, t, m0, n0, split);
    kb = split * p.kb_per_split;
    k_hi = min(kb + p.kb_per_split, p.kblocks);
    a = oa.spot(warp, m0);
    b = ob.spot(warp, n0);
  }
  __device__ __forceinline__ void advance(const Args& p, const Operand<kTileM>& oa, const Operand<BN>& ob, int warp, int total) {
    if (++kb < k_hi) return;
    t += gridDim.x;
    seek(p, oa, ob, warp, total);
  }
};

template <int ACT>
__device__ __forceinline__ void activate(float* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) act_value2(v[i], v[i + 1], ACT);
}

// RESIDENT: B's parts are in shared memory from the start, and the loaders hold two k blocks of A's words in
// turn; else one of A's and B's.
template <int BN, bool RESIDENT>
__global__ void __launch_bounds__(kThreads, 1) k_mma_staged(const __grid_constant__ Args p) {
  constexpr int kABytes = kTileM * kTileK * 2, kBBytes = BN * kTileK * 2;
  constexpr int kTmem = BN * 2;  // columns, two tiles in flight
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
  unsigned char* res_b = smem + kSmemCtl;
  unsigned char* ring = res_b + (RESIDENT ? (size_t)kBBytes * p.kblocks : 0);
  const int stage_bytes = kABytes + (RESIDENT ? 0 : kBBytes);
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
  follow();

  if (warp >= kEpiWarps && warp < kEpiWarps + kLoadWarps) {
    // ------------------------------------------------------------ loaders
    const int lw = warp - kEpiWarps;
    auto operand = [](auto op, const bf16* q, int64_t ld, int64_t ext, int64_t k, bool mn) {
      op.p = q, op.ld = ld, op.ext = ext, op.k = k, op.mn = mn;
      op.lo = reinterpret_cast<uintptr_t>(q);
      op.hi = reinterpret_cast<uintptr_t>(q + ((mn ? k : ext) - 1) * ld + (mn ? ext : k));
      return op;
    };
    using OpA = Operand<kTileM>;
    using OpB = Operand<BN>;
    const OpA a = operand(OpA{}, p.a, p.lda, p.m, p.k, p.a_mn != 0);
    const OpB b = operand(OpB{}, p.b, p.ldb, p.n, p.k, p.b_mn != 0);
    if (!p.drop) {
      if (RESIDENT && (int)blockIdx.x < total) {
        const auto spot = b.spot(lw, (int64_t)(blockIdx.x % p.n_tiles) * BN);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          typename OpB::Words f;
          b.load(lw, lane, spot, kb, f);
          b.shift(lw, lane, spot, kb, f, tc::smem_addr(res_b) + kBBytes * kb);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.resident));
      }
      Cursor<BN> cur;
      cur.t = blockIdx.x;
      cur.seek(p, a, b, lw, total);
      Cursor<BN> ahead = cur;
      constexpr int kSets = RESIDENT ? 2 : 1;
      typename OpA::Words fa[kSets];
      typename OpB::Words fb;
      auto load = [&](int w) {
        if (ahead.t >= total) return;
        a.load(lw, lane, ahead.a, ahead.kb, fa[w]);
        if (!RESIDENT) b.load(lw, lane, ahead.b, ahead.kb, fb);
        ahead.advance(p, a, b, lw, total);
      };
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      load(0);
      while (ok && cur.t < total) {
#pragma unroll
        for (int w = 0; w < kSets; ++w) {
          if (!ok || cur.t >= total) break;
          if constexpr (kSets == 2) load(w ^ 1);
          ok = tc::mbar_wait_warp(bar(ctl.empty[s]), parity, g);
          if (!ok) break;
          const uint32_t st = tc::smem_addr(ring) + stage_bytes * s;
          a.shift(lw, lane, cur.a, cur.kb, fa[w], st);
          if (!RESIDENT) b.shift(lw, lane, cur.b, cur.kb, fb, st + kABytes);
          if constexpr (kSets == 1) load(0);
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(ctl.full[s]));
          if (++s == p.stages) s = 0, parity ^= 1;
          cur.advance(p, a, b, lw, total);
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
      if (RESIDENT && (int)blockIdx.x < total) ok = tc::mbar_wait_warp(bar(ctl.resident), 0, g);
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
          const uint32_t bs = RESIDENT ? tc::smem_addr(res_b) + kBBytes * kb : as + kABytes;
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
      for (int c = 0; in && c < kCols && col0 + c < (p.part ? p.ldp : p.n); c += 32) {
        float v[32];
        __syncwarp();  // the load is the whole warp's: the lanes that left the piece before early are waited for
        tc::tmem_load32(d + c, v);
        if (p.part) {
          const int64_t row = row0 + lane;
          if (row < p.m) {
            float* out = p.part + ((int64_t)split * p.m + row) * p.ldp + col0 + c;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              if (col0 + c + i < p.ldp) *reinterpret_cast<float4*>(out + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
          continue;
        }
        // a lane owns a column from here on; all 32 rows at each step, so that their accesses overlap
        const int64_t col = col0 + c + lane;
        const bool ci = col < p.n;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) buf[lane * kPitch + i] = v[i];
        __syncwarp();
        if (!ci) continue;
        bf16 rr[32];
        if (p.residual) {
          const bf16* res = p.residual + row0 * p.ldr + col;
#pragma unroll
          for (int r = 0; r < 32; ++r, res += p.ldr)
            if (r < rows) rr[r] = *res;
        }
        const float bias = p.bias ? __bfloat162float(p.bias[col]) : 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r] = buf[r * kPitch + lane] + bias;
        if (p.z) {
          bf16* z = p.z + row0 * p.ldz + col;
#pragma unroll
          for (int r = 0; r < 32; ++r, z += p.ldz)
            if (r < rows) *z = __float2bfloat16_rn(v[r]);
        }
        if (p.act == GS_ACT_RELU) activate<GS_ACT_RELU>(v);
        else if (p.act == GS_ACT_GELU) activate<GS_ACT_GELU>(v);
        else if (p.act == GS_ACT_SILU) activate<GS_ACT_SILU>(v);
        bf16* y = p.y + row0 * p.ldy + col;
#pragma unroll
        for (int r = 0; r < 32; ++r, y += p.ldy)
          if (r < rows) *y = __float2bfloat16_rn(p.residual ? v[r] + __bfloat162float(rr[r]) : v[r]);
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

// Ranges of k of at least two blocks (128) where there are too few tiles for the device.
Plan plan_as(int bn, int64_t m, int64_t n, int64_t k) {
  Plan p;
  p.m_tiles = (int)ceil_div(m, kTileM);
  p.kblocks = (int)ceil_div(k, kTileK);
  p.bn = bn;
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
// Tiles of 64 columns: the words of both operands' blocks fit a loader's registers twice.
Plan plan_of(int64_t m, int64_t n, int64_t k) { return plan_as(64, m, n, k); }

// bytes of shared memory beside the stages, with B resident or not
template <int BN>
int64_t fixed_bytes(const Plan& pl, bool resident) {
  return (int64_t)1024 + kSmemCtl + kEpiWarps * kBufBytes + (resident ? (int64_t)BN * kTileK * 2 * pl.kblocks : 0);
}
// resident B: one range of columns per block, and at least three stages of A beside it
template <int BN>
bool fits_resident(const Plan& pl) {
  return pl.splits == 1 && pl.n_tiles <= 4 && (int64_t)pl.m_tiles * pl.n_tiles >= 2 * gs::num_sms() &&
         fixed_bytes<BN>(pl, true) + 3 * kTileM * kTileK * 2 <= kSmemMost;
}

template <int BN, bool RESIDENT>
gs_status launch(Args& p, const Plan& pl, cudaStream_t st, const char* where) {
  const int64_t total = (int64_t)pl.m_tiles * pl.n_tiles * pl.splits;
  int grid = (int)(total < gs::num_sms() ? total : gs::num_sms());
  if (RESIDENT) grid -= grid % pl.n_tiles;
  const int64_t fixed = fixed_bytes<BN>(pl, RESIDENT);
  const int stage = (kTileM + (RESIDENT ? 0 : BN)) * kTileK * 2, stages = (int)((kSmemMost - fixed) / stage);
  p.stages = stages < kMaxStages ? stages : kMaxStages;
  cudaError_t e = gs::max_dynamic_smem((const void*)k_mma_staged<BN, RESIDENT>, kSmemMost);
  if (e == cudaSuccess)
    e = gs::launch(k_mma_staged<BN, RESIDENT>, dim3(grid), kThreads, (size_t)fixed + p.stages * stage, st, p);
  return e == cudaSuccess ? GS_OK : gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

}  // namespace

namespace gs {

size_t staged_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_of(m, n, k);
  return p.splits > 1 ? (size_t)p.splits * m * p.ldp * sizeof(float) : 0;
}

gs_status staged_run(const MmaProduct& q, void* workspace, int32_t* status, cudaStream_t st, const char* where) {
  // of 128 where B stays resident, and is no part of what they hold
  Plan pl = plan_of(q.m, q.n, q.k);
  const Plan wide = plan_as(128, q.m, q.n, q.k);
  const bool resident = q.n > 64 && fits_resident<128>(wide);
  if (resident) pl = wide;
  if ((int64_t)pl.m_tiles * pl.n_tiles * pl.splits > 0x7fffffff)
    return set_error(GS_ERR_INVALID, "%s: too many tiles", where);
  Args p{};
  p.a = static_cast<const bf16*>(q.a), p.b = static_cast<const bf16*>(q.b), p.lda = q.lda, p.ldb = q.ldb, p.m = q.m, p.n = q.n, p.k = q.k;
  p.m_tiles = pl.m_tiles, p.n_tiles = pl.n_tiles, p.splits = pl.splits, p.kblocks = pl.kblocks;
  p.kb_per_split = pl.kb_per_split;
  p.a_mn = q.a_mn, p.b_mn = q.b_mn;
  p.bias = static_cast<const bf16*>(q.bias), p.residual = static_cast<const bf16*>(q.residual);
  p.y = static_cast<bf16*>(q.y), p.z = static_cast<bf16*>(q.z), p.ldr = q.ldr, p.ldy = q.ldy, p.ldz = q.ldz;
  p.act = q.act;
  p.part = pl.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  p.ldp = pl.ldp;
  p.status = status, p.wait_limit = wait_us(), p.drop = take_drop_copy();
  if (gs_status s = resident                  ? launch<128, true>(p, pl, st, where)
                    : fits_resident<64>(pl) ? launch<64, true>(p, pl, st, where)
                                            : launch<64, false>(p, pl, st, where))
    return s;
  if (!p.part) {
    if (q.also.part) launch_column_fold<bf16>(q.also, st);
    return check_launch(where);
  }
  launch_fold(FoldArgs<bf16>{p.part, p.bias, p.residual, p.y, p.z, q.m, pl.ldp, q.ldr, q.ldy, q.ldz, pl.splits, (int)q.n, q.act, false,
                             q.also},
              st);
  return check_launch(where);
}

}  // namespace gs
