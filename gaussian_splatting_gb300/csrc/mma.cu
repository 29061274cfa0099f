// bfloat16 products on the 5th-generation tensor cores, with the linear layer's epilogue.
//
// C(m, n) = sum over k of A(m, k) B(n, k), 32-bit sums, then z = C + bias, y = act(z) + residual.
// One persistent block per SM walks over 128 x BN tiles of C (BN = 64 .. 256, and ranges of k where
// there are few tiles).  Its warps work as a pipeline:
//   warp 16       issues TMA copies of 128 x 64 (A) and BN x 64 (B) pieces into a ring of shared-memory
//                 stages (128-byte swizzle).  An operand stored along its other axis ([k][m]) is copied
//                 as 64 x 64 boxes and handed to the tensor core as it lies: no transpose.  B stays
//                 resident where all of its k fits: the weights are then read once per block.
//   warp 17       issues tcgen05.mma, 128 x BN x 16 each, into one of two accumulators in TMEM
//   warps 0 - 15  read the finished accumulator in pieces of 32 rows x 32 columns and write them through
//                 shared memory with TMA stores while the next tile is being summed; the residual's piece
//                 is copied in one piece ahead.  The epilogue is latency: with eight warps it took longer
//                 than the products (16,384 x 1024 -> 4096 with GELU and z: 114 us, the products alone 82)
// Every wait is bounded (see tc::Guard).
#include <cuda.h>

#include <atomic>

#include "mma.cuh"
#include "tcgen05.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kEpiWarps = 16;         // four to a quadrant of 32 rows
constexpr int kParts = kEpiWarps / 4;  // which take its pieces of 32 columns in turn
constexpr int kLoadWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kTileM = 128, kTileK = 64;
constexpr int kMaxStages = 8;
constexpr int kABytes = kTileM * kTileK * 2;
constexpr int kBufCols = 32;          // columns of one warp's piece
constexpr int kBufBytes = 32 * 64;    // and its bytes: 32 rows of 64, 64-byte swizzle
constexpr int kSmemMost = 232448;     // 227 KB
constexpr int kSmemCtl = 1024;        // barriers, TMEM address, dead flag

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t resident, acc_full[2], acc_empty[2], drain;
  uint64_t res[kEpiWarps];
  uint32_t tmem, dead;
};
static_assert(sizeof(Ctl) <= kSmemCtl, "control block");

struct Args {
  CUtensorMap a, b, y, z, r;
  int64_t m, n;
  int m_tiles, n_tiles, splits, kblocks, kb_per_split;
  int bn, stages, tmem_cols;
  int a_mn, b_mn, resident;
  int bufs_y, has_z, has_r, act;  // bufs_y: buffers per warp for y and the residual (1, or 2 with a residual)
  const bf16* bias;
  float* part;  // [splits][m][ldp] when splits > 1: no epilogue
  int64_t ldp;
  int32_t* status;
  int wait_limit;  // microseconds
  int drop;        // test hook: nothing is copied in, every wait for it runs out
};

// ---------------------------------------------------------------- epilogue
// y and z of 8 columns of a row from the sums v: bias (already 32 bits), activation, residual.
// (Activations in pairs of elements in the pairs of blocks: 15,965 x 1024 -> 4096 with GELU and z 103 us, 108 one by one.
// A single block's epilogue has no registers left for them, and its products are bound by memory.)
template <int CTAS, int ACT>
__device__ __forceinline__ void epilogue8(const float* v, const float* bias, const uint4* res, uint4& y, uint4& z) {
  float t[8], r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = v[i] + bias[i];
  z = make_uint4(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]), pack_bf16(t[4], t[5]), pack_bf16(t[6], t[7]));
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if (CTAS == 2) act_value2(t[i], t[i + 1], ACT);
    else t[i] = act_value(t[i], ACT), t[i + 1] = act_value(t[i + 1], ACT);
  }
  if (res) {
    VecIO<bf16, 8>::unpack(*res, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] += r[i];
  }
  y = make_uint4(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]), pack_bf16(t[4], t[5]), pack_bf16(t[6], t[7]));
}

struct EpiState {
  uint32_t buf;        // this warp's buffers in shared memory (address)
  unsigned char* ptr;  // the same, generic
  bf16* bias;          // 32 values of this warp's own
  uint32_t res_bar;
  uint32_t loads, issued;  // residual pieces waited for and asked for so far
  int lane, quad, part;
  int rank, step;      // of the block in its pair; tiles between two of this pair
};

// The tile t of a pair (or, CTAS = 1, a block): the rows of the block of this rank.
template <int CTAS>
__device__ __forceinline__ void tile_of(const Args& p, int rank, int t, int64_t& m0, int64_t& n0, int& split) {
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
  n0 = (int64_t)nt * p.bn;
  m0 = ((int64_t)mt * CTAS + rank) * kTileM;
}

// whether this warp writes anything of chunk c of the tile at (m0, n0)
__device__ __forceinline__ bool chunk_in(const Args& p, const EpiState& e, int64_t m0, int64_t n0, int c) {
  return m0 + e.quad * 32 < p.m && n0 + c * kBufCols < p.n;
}

template <int CTAS, int ACT>
__device__ bool epilogue_tile(const Args& p, EpiState& e, const tc::Guard& g, int t, int total, uint32_t tmem,
                              uint32_t acc_full, uint32_t parity) {
  int64_t m0, n0;
  int split;
  tile_of<CTAS>(p, e.rank, t, m0, n0, split);
  bool waited = false;
  for (int c = e.part; c * kBufCols < p.bn; c += kParts) {
    const bool in = chunk_in(p, e, m0, n0, c);
    uint32_t slot = 0;
    if (in) {
      const int64_t col = n0 + c * kBufCols + e.lane;
      const bf16 bias = p.bias && col < p.n ? p.bias[col] : __float2bfloat16_rn(0.f);
      // every store that reads these buffers is done reading
      if (tc::elect_one()) tc::bulk_wait_read0();
      __syncwarp();
      e.bias[e.lane] = bias;
      if (p.has_r) {
        slot = e.loads & 1;
        // the residual piece of the next chunk goes to the other buffer
        int64_t nm = 0, nn = 0;
        int t2 = t, c2 = c, s2;
        do {  // skips the chunks that lie outside of C
          c2 += kParts;
          if (c2 * kBufCols >= p.bn) c2 = e.part, t2 += e.step;
          if (t2 >= total) break;
          tile_of<CTAS>(p, e.rank, t2, nm, nn, s2);
        } while (!chunk_in(p, e, nm, nn, c2));
        if (t2 < total) {
          if (tc::elect_one()) {
            tc::mbar_expect_tx(e.res_bar + 8 * (slot ^ 1), kBufBytes);
            tc::tma_load_2d(e.buf + (slot ^ 1) * kBufBytes, &p.r, (int)nn + c2 * kBufCols, (int)(nm + e.quad * 32),
                            e.res_bar + 8 * (slot ^ 1));
          }
          ++e.issued;
        }
        if (!tc::mbar_wait_warp(e.res_bar + 8 * slot, (e.loads >> 1) & 1, g)) return false;
        ++e.loads;
      }
      __syncwarp();
    }
    if (!waited) {
      if (!tc::mbar_wait_warp(acc_full, parity, g)) return false;
      tc::fence_after();
      waited = true;
    }
    if (!in) continue;
    unsigned char* yb = e.ptr + slot * kBufBytes;
    unsigned char* zb = e.ptr + p.bufs_y * kBufBytes;
    float v[32];
    tc::tmem_load32(tmem + ((uint32_t)(e.quad * 32) << 16) + c * kBufCols, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int at = e.lane * 64 + ((q ^ (e.lane >> 1 & 3)) << 4);
      float b[8];
      VecIO<bf16, 8>::unpack(reinterpret_cast<const uint4*>(e.bias)[q], b);
      uint4 y, z, r;
      if (p.has_r) r = *reinterpret_cast<uint4*>(yb + at);
      epilogue8<CTAS, ACT>(v + q * 8, b, p.has_r ? &r : nullptr, y, z);
      *reinterpret_cast<uint4*>(yb + at) = y;
      if (p.has_z) *reinterpret_cast<uint4*>(zb + at) = z;
    }
    tc::fence_async_smem();
    __syncwarp();
    if (tc::elect_one()) {
      tc::tma_store_2d(&p.y, (int)n0 + c * kBufCols, (int)(m0 + e.quad * 32), e.buf + slot * kBufBytes);
      if (p.has_z)
        tc::tma_store_2d(&p.z, (int)n0 + c * kBufCols, (int)(m0 + e.quad * 32), e.buf + p.bufs_y * kBufBytes);
      tc::bulk_commit();
    }
    __syncwarp();
  }
  if (!waited && !tc::mbar_wait_warp(acc_full, parity, g)) return false;
  return true;
}

// A range of k: the sums as they are, 32 bits, to this split's part (rows of ldp, a multiple of 8).
template <int CTAS>
__device__ bool partial_tile(const Args& p, const EpiState& e, const tc::Guard& g, int t, uint32_t tmem,
                             uint32_t acc_full, uint32_t parity) {
  int64_t m0, n0;
  int split;
  tile_of<CTAS>(p, e.rank, t, m0, n0, split);
  if (!tc::mbar_wait_warp(acc_full, parity, g)) return false;
  tc::fence_after();
  const int64_t row = m0 + e.quad * 32 + e.lane;
  float* out = p.part + ((int64_t)split * p.m + row) * p.ldp + n0;
  for (int c = e.part; c * 32 < p.bn; c += kParts) {
    if (n0 + c * 32 >= p.ldp) break;
    float v[32];
    __syncwarp();  // the load is the whole warp's: the lanes without a row of the piece before wait for the others
    tc::tmem_load32(tmem + ((uint32_t)(e.quad * 32) << 16) + c * 32, v);
    if (row < p.m) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (n0 + c * 32 + q * 4 < p.ldp)
          *reinterpret_cast<float4*>(out + c * 32 + q * 4) = make_float4(v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]);
    }
  }
  return true;
}

template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) k_mma(const __grid_constant__ Args p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
  const uint32_t base = tc::smem_addr(smem);
  const int rank = CTAS == 2 ? (int)tc::cluster_rank() : 0, first = blockIdx.x / CTAS, step = gridDim.x / CTAS;
  const uint32_t b_bytes = (uint32_t)p.bn / CTAS * kTileK * 2;  // this block's part of B
  const uint32_t res_b = base + kSmemCtl;
  const uint32_t ring = res_b + (p.resident ? b_bytes * p.kblocks : 0);
  const uint32_t stage_bytes = kABytes + (p.resident ? 0 : b_bytes);
  const uint32_t epi = ring + stage_bytes * p.stages;
  const int warp = tc::warp_index(), lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return tc::smem_addr(&b); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(bar(ctl.full[s]), 1);
      tc::mbar_init(bar(ctl.empty[s]), 1);
    }
    tc::mbar_init(bar(ctl.resident), 1);
    tc::mbar_init(bar(ctl.drain), 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(ctl.acc_full[i]), 1);
      tc::mbar_init(bar(ctl.acc_empty[i]), kEpiWarps * CTAS);
    }
    ctl.dead = 0;
    tc::fence_mbar_init();
  }
  const tc::Guard g{&ctl.dead, p.status, p.wait_limit};
  const int total = p.m_tiles * p.n_tiles * p.splits;
  if (warp == kMmaWarp) tc::tmem_alloc<CTAS>(bar(reinterpret_cast<uint64_t&>(ctl.tmem)), p.tmem_cols);
  tc::fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = ctl.tmem;
  follow();

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ producer
    if (!p.drop) {
      // in a pair, the barriers that count the copies of both blocks are those of rank 0
      auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t full) {
        if constexpr (CTAS == 2) tc::tma_load_2d_pair(dst, map, x, y, full);
        else tc::tma_load_2d(dst, map, x, y, full);
      };
      auto lead = [&](uint32_t b) { return CTAS == 2 ? tc::map_rank(b, 0) : b; };
      auto load_b = [&](uint32_t dst, int64_t n0, int kb, uint32_t full) {
        n0 += rank * (p.bn / CTAS);
        if (!p.b_mn) load(dst, &p.b, kb * kTileK, (int)n0, full);
        else
          for (int c = 0; c < p.bn / CTAS; c += 64) load(dst + c * 128, &p.b, (int)n0 + c, kb * kTileK, full);
      };
      int it = 0, s = 0;
      uint32_t parity = 1;
      bool ok = true;
      if (p.resident && first < total && tc::elect_one()) {
        if (rank == 0) tc::mbar_expect_tx(bar(ctl.resident), b_bytes * p.kblocks * CTAS);
        for (int kb = 0; kb < p.kblocks; ++kb)
          load_b(res_b + b_bytes * kb, (int64_t)(first % p.n_tiles) * p.bn, kb, lead(bar(ctl.resident)));
      }
      __syncwarp();
      for (int t = first; ok && t < total; t += step) {
        int64_t m0, n0;
        int split;
        tile_of<CTAS>(p, rank, t, m0, n0, split);
        const int k_lo = split * p.kb_per_split;
        const int k_hi = min(k_lo + p.kb_per_split, p.kblocks);
        for (int kb = k_lo; kb < k_hi; ++kb, ++it) {
          ok = tc::mbar_wait_warp(bar(ctl.empty[s]), parity, g);
          if (!ok) break;
          if (tc::elect_one()) {
            const uint32_t dst = ring + stage_bytes * s, full = lead(bar(ctl.full[s]));
            if (rank == 0) tc::mbar_expect_tx(bar(ctl.full[s]), stage_bytes * CTAS);
            if (!p.a_mn) load(dst, &p.a, kb * kTileK, (int)m0, full);
            else
              for (int c = 0; c < kTileM; c += 64) load(dst + c * 128, &p.a, (int)m0 + c, kb * kTileK, full);
            if (!p.resident) load_b(dst + kABytes, n0, kb, full);
          }
          __syncwarp();
          if (++s == p.stages) s = 0, parity ^= 1;
        }
      }
      if (!ok && rank == 0) {  // gave up: no copy, of either block, may be in flight when it ends
        for (int i = it < p.stages ? 0 : it - p.stages; i < it; ++i)
          tc::mbar_drain(bar(ctl.full[i % p.stages]), (uint32_t)(i / p.stages & 1), p.wait_limit);
        if (p.resident)
          tc::mbar_drain(bar(ctl.resident), 0, p.wait_limit);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ matrix instructions
    if (rank == 0) {
      // bfloat16 operands, f32 sums, 128 (256) x bn
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)p.a_mn << 15 | (uint32_t)p.b_mn << 16 |
                             (uint32_t)(p.bn >> 3) << 17 | (uint32_t)(kTileM * CTAS >> 4) << 24;
      // 16 of k further: 32 bytes along a row, or 16 rows of 128 bytes
      const uint32_t a_step = p.a_mn ? 16 * 128 : 32, b_step = p.b_mn ? 16 * 128 : 32;
      int s = 0, n_acc = 0;
      uint32_t parity = 0;
      bool ok = true;
      if (p.resident && first < total) ok = tc::mbar_wait_warp(bar(ctl.resident), 0, g);
      for (int t = first; ok && t < total; t += step, ++n_acc) {
        int64_t m0, n0;
        int split;
        tile_of<CTAS>(p, rank, t, m0, n0, split);
        const int k_lo = split * p.kb_per_split;
        const int k_hi = min(k_lo + p.kb_per_split, p.kblocks);
        const int acc = (int)(n_acc & 1);
        ok = tc::mbar_wait_warp(bar(ctl.acc_empty[acc]), (uint32_t)(n_acc >> 1 & 1) ^ 1, g);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = tmem + acc * (p.tmem_cols / 2);
        for (int kb = k_lo; kb < k_hi; ++kb) {
          ok = tc::mbar_wait_warp(bar(ctl.full[s]), parity, g);
          if (!ok) break;
          tc::fence_after();
          const uint32_t a = ring + stage_bytes * s;
          const uint32_t b = p.resident ? res_b + b_bytes * kb : a + kABytes;
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < kTileK / 16; ++i) {
              const uint64_t da = tc::smem_desc(a + i * a_step, 64 * 128, 1024), db = tc::smem_desc(b + i * b_step, 64 * 128, 1024);
              if constexpr (CTAS == 2) tc::mma_bf16_pair(d, da, db, idesc, kb > k_lo || i > 0);
              else tc::mma_bf16(d, da, db, idesc, kb > k_lo || i > 0);
            }
            tc::mma_commit<CTAS>(bar(ctl.empty[s]));
          }
          __syncwarp();
          if (++s == p.stages) s = 0, parity ^= 1;
        }
        if (ok && tc::elect_one()) tc::mma_commit<CTAS>(bar(ctl.acc_full[acc]));
        __syncwarp();
      }
      if (!ok) {  // gave up: nothing may be in flight when the tensor memory is freed
        if (tc::elect_one()) tc::mma_commit<CTAS>(bar(ctl.drain));
        __syncwarp();
        tc::mbar_drain(bar(ctl.drain), 0, p.wait_limit);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    EpiState e;
    e.lane = lane, e.quad = warp & 3, e.part = warp >> 2, e.rank = rank, e.step = step;
    const int bufs = p.bufs_y + p.has_z;
    e.buf = epi + warp * bufs * kBufBytes;
    e.ptr = smem + (e.buf - base);
    e.bias = reinterpret_cast<bf16*>(smem + (epi - base) + kEpiWarps * bufs * kBufBytes) + warp * 32;
    e.res_bar = bar(ctl.res[0]) + warp * 16;
    e.loads = e.issued = 0;
    int n_acc = 0;
    bool ok = true;
    if (p.has_r) {
      // the first chunk's residual piece
      if (lane == 0) {
        tc::mbar_init(e.res_bar, 1);
        tc::mbar_init(e.res_bar + 8, 1);
        tc::fence_mbar_init();
        tc::fence_async_smem();
      }
      __syncwarp();
      int c = e.part;
      for (int t = first; t < total; t += step) {
        int64_t m0, n0;
        int split;
        tile_of<CTAS>(p, rank, t, m0, n0, split);
        for (c = e.part; c * kBufCols < p.bn && !chunk_in(p, e, m0, n0, c);) c += kParts;
        if (c * kBufCols >= p.bn) continue;
        if (tc::elect_one()) {
          tc::mbar_expect_tx(e.res_bar, kBufBytes);
          tc::tma_load_2d(e.buf, &p.r, (int)n0 + c * kBufCols, (int)(m0 + e.quad * 32), e.res_bar);
        }
        e.issued = 1;
        break;
      }
    }
    for (int t = first; ok && t < total; t += step, ++n_acc) {
      const int acc = (int)(n_acc & 1);
      const uint32_t parity = (uint32_t)(n_acc >> 1 & 1), d = tmem + acc * (p.tmem_cols / 2), full = bar(ctl.acc_full[acc]);
      if (p.part) ok = partial_tile<CTAS>(p, e, g, t, d, full, parity);
      else if (p.act == GS_ACT_RELU) ok = epilogue_tile<CTAS, GS_ACT_RELU>(p, e, g, t, total, d, full, parity);
      else if (p.act == GS_ACT_GELU) ok = epilogue_tile<CTAS, GS_ACT_GELU>(p, e, g, t, total, d, full, parity);
      else if (p.act == GS_ACT_SILU) ok = epilogue_tile<CTAS, GS_ACT_SILU>(p, e, g, t, total, d, full, parity);
      else ok = epilogue_tile<CTAS, GS_ACT_NONE>(p, e, g, t, total, d, full, parity);
      tc::fence_before();
      __syncwarp();
      if (lane == 0 && ok) {
        if constexpr (CTAS == 2) tc::mbar_arrive_cluster(tc::map_rank(bar(ctl.acc_empty[acc]), 0));
        else tc::mbar_arrive(bar(ctl.acc_empty[acc]));
      }
    }
    if (!ok && lane == 0) {  // gave up: the pieces in flight land before the block ends
      for (uint32_t i = e.loads; i < e.issued; ++i)
        tc::mbar_drain(e.res_bar + 8 * (i & 1), i >> 1 & 1, p.wait_limit);
    }
    if (tc::elect_one()) tc::bulk_wait0();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) tc::cluster_sync();  // nothing of this block is in use by the other any more
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc<CTAS>(tmem, p.tmem_cols);
}

// ---------------------------------------------------------------- host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's encoder, asked for once per process (a function's address, the same for every device)
EncodeFn encoder() {
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn f = cached.load();
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeFn>(p);
  cached.store(f);
  return f;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int ctas, bn, m_tiles, n_tiles, splits, kblocks, kb_per_split;
  int64_t ldp;
};

constexpr int kSms = 152;  // the device's; only speed depends on it

// A pair of blocks takes a 256-row tile together where the tiles, or their ranges of k, are enough for all
// pairs: each then holds half of B, and shared memory, which a single block's 128 x 256 tile keeps busy for
// 768 cycles per 512 of the tensor core, is no longer what bounds it.  Tiles as wide as they go (256 columns:
// the fewest reads of A); with fewer tiles than that single blocks, narrower tiles, then ranges of k of at
// least four blocks (256).
Plan plan_as(int ctas, int64_t m, int64_t n, int64_t k) {
  Plan p;
  p.ctas = ctas;
  const int units = kSms / ctas;
  p.m_tiles = (int)ceil_div(m, kTileM * ctas);
  p.kblocks = (int)ceil_div(k, kTileK);
  const int n_tiles = (int)ceil_div(n, 256), grain = 64 * ctas;
  int bn = (int)(ceil_div(ceil_div(n, n_tiles), grain) * grain);
  while (ctas == 1 && bn > 64 && (int64_t)p.m_tiles * ceil_div(n, bn) < units / 2 && p.kblocks < 16) bn -= 64;
  p.bn = bn;
  p.n_tiles = (int)ceil_div(n, bn);
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  int64_t splits = tiles >= units ? 1 : units / tiles;
  if (splits > p.kblocks / 4) splits = p.kblocks / 4;
  if (splits < 1) splits = 1;
  p.kb_per_split = (int)ceil_div(p.kblocks, splits);
  p.splits = (int)ceil_div(p.kblocks, p.kb_per_split);
  p.ldp = ceil_div(n, 8) * 8;
  return p;
}
Plan plan_of(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_as(2, m, n, k);
  // (short k: the copies of x and y bound it, and two blocks that wait for each other gain nothing: 300K x 256 ->
  // 256 with residual, 114 us by single blocks, 128 us by pairs)
  return n > 64 && m > 128 && p.kblocks >= 8 && (int64_t)p.m_tiles * p.n_tiles * p.splits * 5 >= kSms / 2 * 4 ? p : plan_as(1, m, n, k);
}

template <int CTAS>
gs_status launch(const Args& p, int grid, int smem, cudaStream_t st, const char* where) {
  cudaError_t e = gs::max_dynamic_smem((const void*)k_mma<CTAS>, kSmemMost);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid), c.blockDim = dim3(kThreads), c.dynamicSmemBytes = smem, c.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CTAS, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as gs::launch
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at + (CTAS == 1), c.numAttrs = CTAS;
    e = cudaLaunchKernelEx(&c, k_mma<CTAS>, p);
  }
  return e == cudaSuccess ? GS_OK : gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

}  // namespace

namespace gs {

bool encode_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, int32_t dtype,
                int row_bytes) {
  const EncodeFn f = encoder();
  if (!f) return false;
  const int size = (int)dtype_size(dtype), unit = 16 / size;
  if (rows == 1) ld = (cols + unit - 1) / unit * unit;  // the stride of a single row is never used
  const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)ld * size};
  const cuuint32_t box[2] = {(cuuint32_t)(row_bytes / size), (cuuint32_t)box_rows}, step[2] = {1, 1};
  return f(map, dtype == GS_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
           const_cast<void*>(base), dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool mma_takes(const MmaProduct& p) {
  return tma_takes(p.a, p.a_mn ? p.k : p.m, (p.a_mn ? p.m : p.k) + p.a_pad, p.lda, GS_BF16) &&
         tma_takes(p.b, p.b_mn ? p.k : p.n, (p.b_mn ? p.n : p.k) + p.b_pad, p.ldb, GS_BF16) &&
         tma_takes(p.y, p.m, p.n, p.ldy, GS_BF16) && (!p.z || tma_takes(p.z, p.m, p.n, p.ldz, GS_BF16)) &&
         (!p.residual || tma_takes(p.residual, p.m, p.n, p.ldr, GS_BF16));
}

size_t mma_workspace(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_of(m, n, k);
  return p.splits > 1 ? (size_t)p.splits * m * p.ldp * sizeof(float) : 0;
}

gs_status mma_run(const MmaProduct& q, void* workspace, int32_t* status, cudaStream_t st, const char* where) {
  const Plan pl = plan_of(q.m, q.n, q.k);
  if ((int64_t)pl.m_tiles * pl.n_tiles * pl.splits > 0x7fffffff) return set_error(GS_ERR_INVALID, "%s: too many tiles", where);
  Args p{};
  p.m = q.m, p.n = q.n;
  p.m_tiles = pl.m_tiles, p.n_tiles = pl.n_tiles, p.splits = pl.splits, p.kblocks = pl.kblocks;
  p.kb_per_split = pl.kb_per_split, p.bn = pl.bn;
  p.a_mn = q.a_mn, p.b_mn = q.b_mn;
  p.tmem_cols = pl.bn <= 64 ? 128 : pl.bn <= 128 ? 256 : 512;
  p.act = q.act, p.bias = static_cast<const bf16*>(q.bias);
  p.status = status, p.wait_limit = wait_us(), p.drop = take_drop_copy();
  p.ldp = pl.ldp;
  p.bufs_y = 1;
  if (pl.splits > 1) p.part = static_cast<float*>(workspace);
  else p.has_z = q.z != nullptr, p.has_r = q.residual != nullptr, p.bufs_y = q.residual ? 2 : 1;
  // shared memory: control, epilogue buffers, then resident weights if they leave three stages, then stages
  const int epi = p.part ? 0 : kEpiWarps * ((p.bufs_y + p.has_z) * kBufBytes + 64);
  const int room = kSmemMost - 1024 - kSmemCtl - epi;
  const int b_bytes = pl.bn / pl.ctas * kTileK * 2;
  const int64_t total = (int64_t)pl.m_tiles * pl.n_tiles * pl.splits;
  const int units = num_sms() / pl.ctas;
  int grid = (int)(total < units ? total : units);  // blocks, or pairs
  p.resident = 0;
  if (pl.splits == 1 && pl.n_tiles <= 4 && total >= 2 * grid && (int64_t)b_bytes * pl.kblocks + 3 * kABytes <= room) {
    p.resident = 1;
    grid -= grid % pl.n_tiles;  // a block keeps to one range of columns
  }
  const int stage = kABytes + (p.resident ? 0 : b_bytes);
  int stages = (room - (p.resident ? b_bytes * pl.kblocks : 0)) / stage;
  p.stages = stages < kMaxStages ? stages : kMaxStages;
  const int smem = 1024 + kSmemCtl + (p.resident ? b_bytes * pl.kblocks : 0) + p.stages * stage + epi;
  bool ok = q.a_mn ? encode_map(&p.a, q.a, q.k, q.m + q.a_pad, q.lda, 64, GS_BF16)
                   : encode_map(&p.a, q.a, q.m, q.k + q.a_pad, q.lda, kTileM, GS_BF16);
  ok = ok && (q.b_mn ? encode_map(&p.b, q.b, q.k, q.n + q.b_pad, q.ldb, 64, GS_BF16)
                    : encode_map(&p.b, q.b, q.n, q.k + q.b_pad, q.ldb, pl.bn / pl.ctas, GS_BF16));
  if (!p.part) {
    ok = ok && encode_map(&p.y, q.y, q.m, q.n, q.ldy, 32, GS_BF16, 64);
    if (q.z) ok = ok && encode_map(&p.z, q.z, q.m, q.n, q.ldz, 32, GS_BF16, 64);
    if (q.residual) ok = ok && encode_map(&p.r, q.residual, q.m, q.n, q.ldr, 32, GS_BF16, 64);
  }
  if (!ok) return set_error(GS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", where);
  if (gs_status s = pl.ctas == 2 ? launch<2>(p, 2 * grid, smem, st, where) : launch<1>(p, grid, smem, st, where)) return s;
  if (!p.part) {
    if (q.also.part) launch_column_fold<bf16>(q.also, st);
    return check_launch(where);
  }
  launch_fold(FoldArgs<bf16>{p.part, p.bias, static_cast<const bf16*>(q.residual), static_cast<bf16*>(q.y),
                             static_cast<bf16*>(q.z), q.m, pl.ldp, q.ldr, q.ldy, q.ldz, pl.splits, (int)q.n, q.act, false, q.also},
              st);
  return check_launch(where);
}

}  // namespace gs
