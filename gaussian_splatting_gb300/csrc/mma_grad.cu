// The first half of a narrow linear layer's backward in one pass, bfloat16: dz = dy act'(z), its column sums
// (the bias gradient) and dx = dz w.
//
// With at most 256 outputs and 256 inputs a row of dz and all of w fit a block's shared memory, so that dz, on
// its way from the registers that form it to memory, passes through there as the product's operand: dx then
// costs its own store only, and not another read of dz.  One persistent block per SM walks over tiles of 128
// rows:
//   warps 0 - 15   read dy and z (four vectors of 16 bytes of each in flight per thread), form dz, round it to
//                  bfloat16 once, write it to memory and, swizzled, to shared memory, and add the columns up.
//                  Where w leaves no room for a second buffer of dz they work in four groups, one for each 64 of
//                  the outputs, and a group waits only for the products of its own block of k: together they would
//                  stand still for all of a tile's products
//   warps 16 - 19  write the finished accumulator through shared memory with TMA stores
//   warp 20        issues tcgen05.mma, 128 x in x 16 each, into one of two accumulators
//   warp 21        copies w in, once
// Bound by memory: 300K x 256 -> 256 with GELU reads 307 MB and writes as much.
#include "mma_grad.cuh"

#include "tcgen05.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kFormWarps = 16, kEpiWarps = 4;
constexpr int kMmaWarp = kFormWarps + kEpiWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kForm = 32 * kFormWarps, kThreads = 32 * (kLoadWarp + 1);
constexpr int kTileM = 128, kTileK = 64, kMost = 256;
constexpr int kABytes = kTileM * kTileK * 2;
constexpr int kBufCols = 32, kBufBytes = 32 * 64;  // a warp's piece of dx: 32 rows of 64 bytes, 64-byte swizzle
constexpr int kEpiBytes = kEpiWarps * 2 * kBufBytes, kFoldBytes = kForm * 8 * 4;
constexpr int kSmemMost = 232448, kSmemCtl = 1024;
constexpr int kSms = 152;  // the most blocks; only speed depends on it

struct Ctl {
  uint64_t w, a_full[2][4], a_empty[2][4], acc_full[2], acc_empty[2], drain;
  uint32_t tmem, dead;
};
static_assert(sizeof(Ctl) <= kSmemCtl, "control block");

struct Args {
  CUtensorMap w, dx;
  const bf16* dy;
  const bf16* z;   // NULL: dz = dy
  bf16* dz;        // NULL: not wanted
  float* part;     // [blocks][n]; NULL: no sums
  int64_t rows, ldy, ldz, lddz;
  int n, cols, act, tiles, kblocks, bn, bufs, tmem_cols;  // n outputs, cols inputs
  int has_dx;
  int32_t* status;
  int wait_limit, drop;  // microseconds; test hook: w is not copied in
};

// GROUPS groups of warps side by side, CX threads of each along a row, with a vector of 8 columns each
template <int CX, int GROUPS>
__device__ void form(const Args& p, Ctl& ctl, unsigned char* a, float* fold, const tc::Guard& g) {
  constexpr int kSize = kForm / GROUPS, kRows = kSize / CX, kSteps = kTileM / kRows, kAhead = 4;
  using IO = VecIO<bf16, 8>;
  const int group = threadIdx.x / kSize, cx = threadIdx.x % CX, ry = threadIdx.x % kSize / CX, c = (group * CX + cx) * 8;
  const int lane = threadIdx.x & 31;
  const bool in = c < p.n, used = c < p.kblocks * kTileK;  // the last block of k is filled up with zeros
  const int steps = (p.tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * kSteps;
  auto row_of = [&](int i) {
    return ((int64_t)blockIdx.x + (int64_t)(i / kSteps) * gridDim.x) * kTileM + i % kSteps * kRows + ry;
  };
  uint4 d[kAhead], z[kAhead];
  auto fetch = [&](int i, uint4& rd, uint4& rz) {
    const int64_t r = row_of(i);
    rd = rz = make_uint4(0u, 0u, 0u, 0u);
    if (in && i < steps && r < p.rows) {
      rd = IO::load(p.dy + r * p.ldy + c);
      if (p.z) rz = IO::load(p.z + r * p.ldz + c);
    }
  };
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch(u, d[u], z[u]);
  unsigned char* mine = a + c / kTileK * kABytes;
  bool ok = true;
  int buf = 0;
  uint32_t parity = 1;
  for (int i0 = 0; ok && i0 < steps; i0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u, s = i % kSteps;
      if (i >= steps || !ok) break;
      float f[8];
      IO::unpack(d[u], f);
      if (p.z) {
        float v[8];
        IO::unpack(z[u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= act_slope(v[e], p.act);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f[e];
      const int64_t r = row_of(i);
      fetch(i + kAhead, d[u], z[u]);
      uint4 q;
      IO::store(reinterpret_cast<bf16*>(&q), f);
      if (p.dz && in && r < p.rows) *reinterpret_cast<uint4*>(p.dz + r * p.lddz + c) = q;
      if (!p.has_dx) continue;
      if (s == 0) {
        ok = tc::mbar_wait_warp(tc::smem_addr(&ctl.a_empty[buf][group]), parity, g);
        if (!ok) break;
      }
      const int row = s * kRows + ry;
      if (used) *reinterpret_cast<uint4*>(mine + buf * p.kblocks * kABytes + row * 128 + (((cx ^ row) & 7) << 4)) = q;
      if (s == kSteps - 1) {
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_addr(&ctl.a_full[buf][group]));
        if (++buf == p.bufs) buf = 0, parity ^= 1;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) fold[ry * GROUPS * CX * 8 + c + e] = sum[e];
}

template <int CX, int GROUPS>
__global__ void __launch_bounds__(kThreads, 1) k_mma_grad(const __grid_constant__ Args p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
  const uint32_t w_bytes = (uint32_t)p.bn * kTileK * 2;  // of a block of k
  unsigned char* w = smem + kSmemCtl;
  unsigned char* a = w + (p.has_dx ? w_bytes * p.kblocks : 0);
  unsigned char* epi = a + (p.has_dx ? p.bufs * p.kblocks * kABytes : 0);
  float* fold = reinterpret_cast<float*>(epi + kEpiBytes);
  const int warp = tc::warp_index(), lane = threadIdx.x & 31;
  auto bar = [&](const uint64_t& b) { return tc::smem_addr(&b); };
  if (threadIdx.x == 0) {
    tc::mbar_init(bar(ctl.w), 1);
    tc::mbar_init(bar(ctl.drain), 1);
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < GROUPS; ++j) {
        tc::mbar_init(bar(ctl.a_full[i][j]), kFormWarps / GROUPS);
        tc::mbar_init(bar(ctl.a_empty[i][j]), 1);
      }
      tc::mbar_init(bar(ctl.acc_full[i]), 1);
      tc::mbar_init(bar(ctl.acc_empty[i]), kEpiWarps);
    }
    ctl.dead = 0;
    tc::fence_mbar_init();
  }
  const tc::Guard g{&ctl.dead, p.status, p.wait_limit};
  if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_addr(&ctl.tmem), p.tmem_cols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = ctl.tmem;
  follow();

  if (warp < kFormWarps) {
    form<CX, GROUPS>(p, ctl, a, fold, g);
  } else if (!p.has_dx) {
  } else if (warp == kLoadWarp) {
    if (!p.drop) {
      if (tc::elect_one()) {
        tc::mbar_expect_tx(bar(ctl.w), w_bytes * p.kblocks);
        for (int kb = 0; kb < p.kblocks; ++kb)
          for (int c = 0; c < p.bn; c += 64)
            tc::tma_load_2d(tc::smem_addr(w) + w_bytes * kb + c * 128, &p.w, c, kb * kTileK, bar(ctl.w));
      }
      __syncwarp();
      tc::mbar_drain(bar(ctl.w), 0, p.wait_limit);  // no copy is in flight when the block ends
    }
  } else if (warp == kMmaWarp) {
    // bfloat16 operands, f32 sums, 128 x bn, w along its other axis
    const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 16 | (uint32_t)(p.bn >> 3) << 17 | (uint32_t)(kTileM >> 4) << 24;
    int buf = 0, acc = 0;
    uint32_t parity = 0, acc_parity = 1;
    bool ok = tc::mbar_wait_warp(bar(ctl.w), 0, g);
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
      ok = tc::mbar_wait_warp(bar(ctl.acc_empty[acc]), acc_parity, g);
      const uint32_t d = tmem + acc * (p.tmem_cols / 2);
      for (int kb = 0; kb < p.kblocks; ++kb) {
        const int group = kb * 8 / CX;
        if (ok) ok = tc::mbar_wait_warp(bar(ctl.a_full[buf][group]), parity, g);
        if (!ok) break;
        tc::fence_after();
        if (tc::elect_one()) {
          const uint32_t at = tc::smem_addr(a) + (buf * p.kblocks + kb) * kABytes, bt = tc::smem_addr(w) + w_bytes * kb;
#pragma unroll
          for (int i = 0; i < kTileK / 16; ++i)
            tc::mma_bf16(d, tc::smem_desc(at + i * 32, 64 * 128, 1024), tc::smem_desc(bt + i * 16 * 128, 64 * 128, 1024), idesc,
                         kb > 0 || i > 0);
          if (kb + 1 == p.kblocks || (kb + 1) * 8 / CX != group) tc::mma_commit(bar(ctl.a_empty[buf][group]));
        }
        __syncwarp();
      }
      if (ok && tc::elect_one()) tc::mma_commit(bar(ctl.acc_full[acc]));
      __syncwarp();
      if (++buf == p.bufs) buf = 0, parity ^= 1;
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
    if (!ok) {  // gave up: nothing may be in flight when the tensor memory is freed
      if (tc::elect_one()) tc::mma_commit(bar(ctl.drain));
      __syncwarp();
      tc::mbar_drain(bar(ctl.drain), 0, p.wait_limit);
    }
  } else {
    const int quad = warp & 3;
    unsigned char* out = epi + quad * 2 * kBufBytes;
    int acc = 0, slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
      ok = tc::mbar_wait_warp(bar(ctl.acc_full[acc]), parity, g);
      if (!ok) break;
      tc::fence_after();
      const int64_t row = (int64_t)t * kTileM + quad * 32;
      for (int c = 0; row < p.rows && c < p.cols; c += kBufCols, slot ^= 1) {
        float v[32];
        tc::tmem_load32(tmem + acc * (p.tmem_cols / 2) + ((uint32_t)(quad * 32) << 16) + c, v);
        if (tc::elect_one()) tc::bulk_wait_read1();  // the store that reads this buffer is done reading
        __syncwarp();
        unsigned char* at = out + slot * kBufBytes + lane * 64;
#pragma unroll
        for (int q = 0; q < 4; ++q) VecIO<bf16, 8>::store(reinterpret_cast<bf16*>(at + ((q ^ (lane >> 1 & 3)) << 4)), v + q * 8);
        tc::fence_async_smem();
        __syncwarp();
        if (tc::elect_one()) {
          tc::tma_store_2d(&p.dx, c, (int)row, tc::smem_addr(out + slot * kBufBytes));
          tc::bulk_commit();
        }
        __syncwarp();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(ctl.acc_empty[acc]));
      acc ^= 1;
      if (acc == 0) parity ^= 1;
    }
    if (tc::elect_one()) tc::bulk_wait0();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, p.tmem_cols);
  if (p.part && threadIdx.x < p.n) {
    float t = 0.f;
#pragma unroll 8
    for (int r = 0; r < kForm / (GROUPS * CX); ++r) t += fold[r * GROUPS * CX * 8 + threadIdx.x];
    p.part[(int64_t)blockIdx.x * p.n + threadIdx.x] = t;
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int grid_of(int64_t rows) {
  const int64_t tiles = ceil_div(rows, kTileM);
  return (int)(tiles < kSms ? tiles : kSms);
}

template <int CX, int GROUPS>
gs_status launch(const Args& p, int grid, int smem, cudaStream_t st, const char* where) {
  cudaError_t e = gs::max_dynamic_smem((const void*)k_mma_grad<CX, GROUPS>, kSmemMost);
  if (e == cudaSuccess) e = gs::launch(k_mma_grad<CX, GROUPS>, dim3(grid), kThreads, smem, st, p);
  return e == cudaSuccess ? GS_OK : gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

}  // namespace

namespace gs {

int grad_parts(int64_t rows) { return grid_of(rows); }

bool grad_takes(const gs_linear_desc* d, const void* dy, const void* z, const void* w, const void* dx) {
  return d->dtype == GS_BF16 && d->out_features <= kMost && d->in_features <= kMost && d->out_features % 8 == 0 &&
         rows_aligned16(dy, d->rows, d->ldy, GS_BF16) && (!z || rows_aligned16(z, d->rows, d->ldz, GS_BF16)) &&
         (!dx || (tma_takes(w, d->out_features, d->in_features, d->ldw, GS_BF16) &&
                  tma_takes(dx, d->rows, d->in_features, d->lddx, GS_BF16)));
}

gs_status grad_run(const gs_linear_desc* d, const void* dy, const void* z, const void* w, void* dz, int64_t lddz, void* dx,
                   float* part, int32_t* status, cudaStream_t st, const char* where) {
  Args p{};
  p.dy = static_cast<const bf16*>(dy), p.z = static_cast<const bf16*>(z), p.dz = static_cast<bf16*>(dz);
  p.part = part;
  p.rows = d->rows, p.ldy = d->ldy, p.ldz = d->ldz, p.lddz = lddz;
  p.n = d->out_features, p.cols = d->in_features, p.act = d->act, p.tiles = (int)ceil_div(d->rows, kTileM);
  p.kblocks = (int)ceil_div(p.n, kTileK), p.bn = (int)ceil_div(d->in_features, 64) * 64;
  p.tmem_cols = p.bn <= 64 ? 128 : p.bn <= 128 ? 256 : 512;
  p.has_dx = dx != nullptr;
  p.status = status, p.wait_limit = wait_us(), p.drop = dx ? take_drop_copy() : 0;
  // two buffers of dz where they fit: the next tile's is written while this one's products run
  const int fixed = 1024 + kSmemCtl + kEpiBytes + kFoldBytes + (dx ? p.kblocks * p.bn * kTileK * 2 : 0);
  p.bufs = fixed + 2 * p.kblocks * kABytes <= kSmemMost ? 2 : 1;
  const int smem = fixed + (dx ? p.bufs * p.kblocks * kABytes : 0);
  if (dx && !(encode_map(&p.w, w, p.n, d->in_features, d->ldw, 64, GS_BF16) &&
              encode_map(&p.dx, dx, d->rows, d->in_features, d->lddx, 32, GS_BF16, 64)))
    return set_error(GS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", where);
  const int grid = grid_of(d->rows);
  // as many threads along a row as its blocks of k have columns (256 -> 256 with one buffer: 191 us in groups, 197
  // without; 128 -> 256 with two: 382 and 365 for 1.2M rows)
  if (p.n <= 64) return launch<8, 1>(p, grid, smem, st, where);
  if (p.n <= 128) return launch<16, 1>(p, grid, smem, st, where);
  return p.bufs == 1 && p.kblocks == 4 ? launch<8, 4>(p, grid, smem, st, where) : launch<32, 1>(p, grid, smem, st, where);
}

}  // namespace gs
