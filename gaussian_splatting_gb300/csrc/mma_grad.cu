// The first half of a narrow linear layer's backward in one pass, bfloat16: dz = dy act'(z), its column sums
// (the bias gradient) and dx = dz w.
//
// With at most 256 outputs and 256 inputs a row of dz and all of w fit a block's shared memory, so that dz, on
// its way from the registers that form it to memory, passes through there as the product's operand: dx then
// costs its own store only, and not another read of dz.  One persistent block per SM walks over tiles of 128
// rows:
//   warps 0 - 15   read dy and z (four vectors of 16 bytes of each in flight per thread), form dz, round it to
//                  bfloat16 once (the operand's type; what that costs stands in linear.cu), write it to memory and, swizzled, to shared memory, and add the columns up.
//                  Where w leaves no room for a second buffer of dz they work in four groups, one for each 64 of
//                  the outputs, and a group waits only for the products of its own block of k: together they would
//                  stand still for all of a tile's products
//   warps 16 - 19  write the finished accumulator through shared memory with TMA stores
//   warp 20        copies w in, once, and issues tcgen05.mma, 128 x in x 16 each, into one of two accumulators
// Bound by memory: 300K x 256 -> 256 with GELU reads 307 MB and writes as much in 105 us, 0.88 of the rate of a copy.
#include "mma_grad.cuh"

#include "tcgen05.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kFormWarps = 16, kEpiWarps = 4, kMmaWarp = kFormWarps + kEpiWarps;
constexpr int kForm = 32 * kFormWarps, kThreads = 32 * (kMmaWarp + 1);
constexpr int kTileM = 128, kTileK = 64, kMost = 256;
constexpr int kABytes = kTileM * kTileK * 2;
constexpr int kBufCols = 32, kBufBytes = 32 * 64;  // a warp's piece of dx: 32 rows of 64 bytes, 64-byte swizzle
constexpr int kEpiBytes = kEpiWarps * 2 * kBufBytes, kFoldBytes = kForm * 8 * 4;
constexpr int kSmemMost = 232448, kSmemCtl = 1024;
constexpr int kSms = 152;  // the most blocks; only speed depends on it
static_assert(1024 + kSmemCtl + kEpiBytes + kFoldBytes + 3 * (kMost * kTileK * 2 + 2 * kABytes) <= kSmemMost, "shared memory");

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
  uint32_t rows, dy_bytes, z_bytes, dz_bytes;  // of a row, to the next
  int n, cols, act, tiles, kblocks, bn, tmem_cols;  // n outputs, cols inputs
  int has_dx;
  int32_t* status;
  int wait_limit, drop;  // microseconds; test hook: w is not copied in
};

// Buffers of dz: two, so that the next tile's is written while this one's products run, or one and groups
template <int GROUPS>
constexpr int kBufs = GROUPS == 1 ? 2 : 1;

// GROUPS groups of warps side by side, CX threads of each along a row, with a vector of 8 columns each.  (ACT is the
// compiler's: a branch for each element would keep their evaluations from overlapping.)
template <int CX, int GROUPS, int ACT>
__device__ void form(const Args& p, Ctl& ctl, unsigned char* a, float* fold, const tc::Guard& g) {
  constexpr int kSize = kForm / GROUPS, kRows = kSize / CX, kSteps = kTileM / kRows, kAhead = 4;
  using IO = VecIO<bf16, 8>;
  const int group = threadIdx.x / kSize, cx = threadIdx.x % CX, ry = threadIdx.x % kSize / CX, c = (group * CX + cx) * 8;
  const int lane = threadIdx.x & 31;
  // the last block of k is filled up with zeros; of 256 columns it may be the third
  const bool used = CX < 32 || c < p.kblocks * kTileK;
  // the row of the next step: kRows further with each, and to this block's next tile with the last of a tile
  const uint32_t rows = c < p.n ? p.rows : 0, next = gridDim.x * kTileM;
  uint32_t at = blockIdx.x * kTileM + ry;
  auto row_of = [&](const bf16* base, uint32_t r, uint32_t row_bytes) {
    return reinterpret_cast<const bf16*>(reinterpret_cast<const unsigned char*>(base + c) + (uint64_t)r * row_bytes);
  };
  uint4 d[kAhead], z[kAhead];
  auto fetch = [&](uint32_t r, uint4& rd, uint4& rz) {
    rd = rz = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      rd = IO::load(row_of(p.dy, r, p.dy_bytes));
      if (ACT != GS_ACT_NONE) rz = IO::load(row_of(p.z, r, p.z_bytes));
    }
  };
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch(at + u % kSteps * kRows + u / kSteps * next, d[u], z[u]);
  static_assert(kRows % 8 == 0, "the swizzle of a thread's rows is the same");
  unsigned char* mine = a + c / kTileK * kABytes + ry * 128 + (((cx ^ ry) & 7) << 4);
  int buf = 0;
  uint32_t parity = 1;
  const uint32_t end = (uint32_t)p.tiles * kTileM;
  for (int i0 = 0; at < end; i0 ^= kSteps > kAhead ? kAhead : 0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {  // a tile's steps, half of them, or those of two tiles
      const int s = (i0 + u) % kSteps;
      if (u > 0 && u % kSteps == 0 && at >= end) break;
      uint32_t q[4] = {d[u].x, d[u].y, d[u].z, d[u].w}, zw[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo = bf16_lo(q[e]), hi = bf16_hi(q[e]);
        if (ACT != GS_ACT_NONE) lo *= act_slope(bf16_lo(zw[e]), ACT), hi *= act_slope(bf16_hi(zw[e]), ACT);
        sum[2 * e] += lo, sum[2 * e + 1] += hi;
        if (ACT != GS_ACT_NONE) q[e] = pack_bf16(lo, hi);
      }
      const uint4 dz = make_uint4(q[0], q[1], q[2], q[3]);
      // keeps the steps' evaluations apart, which with this many of a tile's steps need more than the 80 registers
      // that there are; the others gain by overlapping them (1.2M x 256 -> 256: 326 us, 342 apart)
      if (CX == 16) __syncwarp();
      fetch(at + (kSteps > kAhead ? kAhead * kRows + (i0 ? next - kTileM : 0) : kAhead / kSteps * next), d[u], z[u]);
      if (p.dz && at < rows) *reinterpret_cast<uint4*>(const_cast<bf16*>(row_of(p.dz, at, p.dz_bytes))) = dz;
      at += kRows + (s == kSteps - 1 ? next - kTileM : 0);
      if (!p.has_dx) continue;
      if (s == 0) {
        if (!tc::mbar_wait_warp(tc::smem_addr(&ctl.a_empty[buf][group]), parity, g)) {
          at = end;
          break;
        }
      }
      if (used) *reinterpret_cast<uint4*>(mine + buf * p.kblocks * kABytes + s * kRows * 128) = dz;
      if (s == kSteps - 1) {
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_addr(&ctl.a_full[buf][group]));
        if (++buf == kBufs<GROUPS>) buf = 0, parity ^= 1;
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
  unsigned char* epi = a + (p.has_dx ? kBufs<GROUPS> * p.kblocks * kABytes : 0);
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
    if (p.act == GS_ACT_GELU) form<CX, GROUPS, GS_ACT_GELU>(p, ctl, a, fold, g);
    else if (p.act == GS_ACT_SILU) form<CX, GROUPS, GS_ACT_SILU>(p, ctl, a, fold, g);
    else if (p.act == GS_ACT_RELU) form<CX, GROUPS, GS_ACT_RELU>(p, ctl, a, fold, g);
    else form<CX, GROUPS, GS_ACT_NONE>(p, ctl, a, fold, g);
  } else if (!p.has_dx) {
  } else if (warp == kMmaWarp) {
    if (!p.drop && tc::elect_one()) {
      tc::mbar_expect_tx(bar(ctl.w), w_bytes * p.kblocks);
      for (int kb = 0; kb < p.kblocks; ++kb)
        for (int c = 0; c < p.bn; c += 64)
          tc::tma_load_2d(tc::smem_addr(w) + w_bytes * kb + c * 128, &p.w, c, kb * kTileK, bar(ctl.w));
    }
    __syncwarp();
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
          if (kb + 1 == p.kblocks) tc::mma_commit(bar(ctl.acc_full[acc]));
        }
        __syncwarp();
      }
      if (++buf == kBufs<GROUPS>) buf = 0, parity ^= 1;
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
    if (!ok) {  // gave up: nothing may be in flight when the block ends and the tensor memory is freed
      if (tc::elect_one()) tc::mma_commit(bar(ctl.drain));
      __syncwarp();
      tc::mbar_drain(bar(ctl.drain), 0, p.wait_limit);
      if (!p.drop) tc::mbar_drain(bar(ctl.w), 0, p.wait_limit);
    }
  } else {
    const int quad = warp & 3;
    unsigned char* out = epi + quad * 2 * kBufBytes;
    int acc = 0, slot = 0;
    uint32_t parity = 0;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x) {
      if (!tc::mbar_wait_warp(bar(ctl.acc_full[acc]), parity, g)) break;
      tc::fence_after();
      const uint32_t row = (uint32_t)t * kTileM + quad * 32;
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

int smem_of(const Args& p, int bufs) {
  return 1024 + kSmemCtl + kEpiBytes + kFoldBytes + (p.has_dx ? p.kblocks * (p.bn * kTileK * 2 + bufs * kABytes) : 0);
}

template <int CX, int GROUPS>
gs_status launch(const Args& p, int grid, cudaStream_t st, const char* where) {
  cudaError_t e = gs::max_dynamic_smem((const void*)k_mma_grad<CX, GROUPS>, kSmemMost);
  if (e == cudaSuccess) e = gs::launch(k_mma_grad<CX, GROUPS>, dim3(grid), kThreads, smem_of(p, kBufs<GROUPS>), st, p);
  return e == cudaSuccess ? GS_OK : gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

}  // namespace

namespace gs {

int grad_parts(int64_t rows) { return grid_of(rows); }

bool grad_takes(const gs_linear_desc* d, const void* dy, const void* z) {
  // (32 bits for the bytes from one row to the next keep the addresses at one instruction each)
  auto near = [&](int64_t ld) { return d->rows <= 1 || ld < (int64_t(1) << 31); };
  return d->dtype == GS_BF16 && d->out_features <= kMost && d->in_features <= kMost && d->out_features % 8 == 0 &&
         near(d->ldy) && rows_aligned16(dy, d->rows, d->ldy, GS_BF16) &&
         (!z || (near(d->ldz) && rows_aligned16(z, d->rows, d->ldz, GS_BF16)));
}
bool grad_takes_dx(const gs_linear_desc* d, const void* w, const void* dx) {
  return tma_takes(w, d->out_features, d->in_features, d->ldw, GS_BF16) &&
         tma_takes(dx, d->rows, d->in_features, d->lddx, GS_BF16);
}

gs_status grad_run(const gs_linear_desc* d, const void* dy, const void* z, const void* w, void* dz, int64_t lddz, void* dx,
                   float* part, int32_t* status, cudaStream_t st, const char* where) {
  Args p{};
  p.dy = static_cast<const bf16*>(dy), p.z = static_cast<const bf16*>(z), p.dz = static_cast<bf16*>(dz);
  p.part = part;
  p.rows = (uint32_t)d->rows;
  p.dy_bytes = (uint32_t)(2 * d->ldy), p.z_bytes = (uint32_t)(2 * d->ldz), p.dz_bytes = (uint32_t)(2 * lddz);
  p.n = d->out_features, p.cols = d->in_features, p.act = d->act, p.tiles = (int)ceil_div(d->rows, kTileM);
  p.kblocks = (int)ceil_div(p.n, kTileK), p.bn = (int)ceil_div(d->in_features, 64) * 64;
  p.tmem_cols = p.bn <= 64 ? 128 : p.bn <= 128 ? 256 : 512;
  p.has_dx = dx != nullptr;
  p.status = status, p.wait_limit = wait_us(), p.drop = dx ? take_drop_copy() : 0;
  if (dx && !(encode_map(&p.w, w, p.n, d->in_features, d->ldw, 64, GS_BF16) &&
              encode_map(&p.dx, dx, d->rows, d->in_features, d->lddx, 32, GS_BF16, 64)))
    return set_error(GS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", where);
  const int grid = grid_of(d->rows);
  // As many threads along a row as its blocks of k have columns; in groups only where two buffers do not fit (an
  // earlier form of the kernel, 300K x 256 -> 256, one buffer: 191 us in groups, 197 without; 1.2M x 128 -> 256, two
  // buffers: 382 and 365).  Two buffers of up to three blocks always fit.
  if (p.n <= 64) return launch<8, 1>(p, grid, st, where);
  if (p.n <= 128) return launch<16, 1>(p, grid, st, where);
  return smem_of(p, 2) <= kSmemMost ? launch<32, 1>(p, grid, st, where) : launch<8, 4>(p, grid, st, where);
}

}  // namespace gs
