// Rows of a table by their indices, scaled (gs_embedding_fwd), and the table's gradient by sorted rows
// (gs_embedding_bwd).
//
// Mathematics: y[r] = scale table[idx[r]]; dtable[v] = scale sum over {r: idx[r] = v} of dy[r].
//
// Both are bound by memory.  The forward reads the indices and what it needs of the table, and writes y once: a thread
// holds 16 bytes of a row, four times in flight (10M rows of 64 bfloat16: 230 us, 196 at the copy's rate; 242 with stores
// that stay in L2).
//
// The backward must not add in whatever order atomics come, and one code may have any number of rows, so the rows are
// first sorted by code, stably, and then added up in equal parts of the sorted rows by groups of lanes ("walkers"), in registers
// as long as the code stays the same.  A code whose rows lie inside one walker's part is written at once; the sums at a
// part's ends are joined in order, first among the walkers of a block in shared memory, then among blocks by another kernel.
// The parts follow from the sizes, the indices and the vector that strides and alignment allow, so the same call gives the
// same bits.  Three forms, by size:
//   few rows     one kernel, whose blocks own runs of codes, pick their rows out of all indices and sort them in shared memory;
//   more         a radix sort of (code, row) pairs, up to eight bits a pass, each pass three kernels (digit counts of tiles,
//                their scan by digit, a scatter through shared memory), then the sums;
//   many         one such pass into up to 2,048 buckets of neighbouring codes; the rest of the sort is done in shared memory by
//                the blocks that add a bucket up.  11M rows of 32 float32, 2M codes: 396 us against 675 by the sort, of which
//                the sums take 300 (their bytes at the copy's rate: 258), the pairs' scatter 62, counts and their scan 27.
#include <algorithm>

#include "dense.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPartThreads = 512;  // of the backward's kernels by buckets

// ------------------------------------------------------------------ forward
// Outputs of this size or more are not held by L2 (129 MB) until they are read: they are stored first to be evicted, and leave
// it to the table, in vectors of 16 bytes (shorter ones take longer so).
constexpr int64_t kStreamBytes = 64 << 20;
__device__ __forceinline__ void store_first_out(float* p, const float* f) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
}
__device__ __forceinline__ void store_first_out(__nv_bfloat16* p, const float* f) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
}
struct FwdArgs {
  const void* table;
  const void* idx;
  void* y;
  int64_t rows, n, ldt, ldy;
  uint32_t per_row, magic;  // units of a row; 2^32 / per_row rounded up
  uint32_t width;
  float scale;
};

// Vectors of a thread's unit: two of less than 16 bytes share the arithmetic of their place (300K rows of 394 bfloat16: 87 us,
// 117 with four, 114 alone; of 393 float32: 162, 150 with four, 263 alone; 332K of 393 bfloat16: 164, 290 with eight, 274 alone).
constexpr int unit_of(int vector_bytes) { return vector_bytes == 16 ? 1 : 2; }
template <typename T, int VE, bool STREAM, typename I>
__global__ void __launch_bounds__(kThreads) k_embedding_fwd(const FwdArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int K = unit_of(sizeof(typename IO::Raw)), U = 4;
  const int64_t first = (int64_t)blockIdx.x * (kThreads * U);
  const int64_t r0 = first / a.per_row;
  const uint32_t c0 = (uint32_t)(first - r0 * a.per_row);
  const T* table = static_cast<const T*>(a.table);
  const I* idx = static_cast<const I*>(a.idx);
  T* y = static_cast<T*>(a.y);
  int64_t row[U];
  uint32_t col[U];
  I code[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t o = c0 + u * kThreads + threadIdx.x;  // < per_row + 1024
    // rows of more than 1024 units: at most one further row; else o per_row < 2^22 and the product is exact
    const uint32_t q = a.per_row > 1024 ? (o >= a.per_row) : a.per_row == 1 ? o : __umulhi(o, a.magic);
    row[u] = r0 + q, col[u] = (o - q * a.per_row) * (K * VE);
    const bool in = row[u] < a.rows;
    code[u] = in ? idx[row[u]] : (I)-1;
  }
  typename IO::Raw v[U][K];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool there = code[u] >= 0 && code[u] < a.n;
    const T* from = table + (there ? (int64_t)code[u] : (int64_t)0) * a.ldt + col[u];
#pragma unroll
    for (int k = 0; k < K; ++k) v[u][k] = there && (K == 1 || col[u] + k * VE < a.width) ? IO::load(from + k * VE) : IO::zero();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= a.rows) continue;
    const bool there = code[u] >= 0 && code[u] < a.n;
    T* to = y + row[u] * a.ldy + col[u];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float f[VE];
      IO::unpack(v[u][k], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = there ? f[e] * a.scale : 0.f;
      if constexpr (STREAM) store_first_out(to, f);
      else if (K == 1 || col[u] + k * VE < a.width) IO::store(to + k * VE, f);
    }
  }
}

// ------------------------------------------------------------------ backward: the sort
struct SortArgs {
  const void* idx;           // first pass
  const uint32_t* keys;      // later ones
  const uint32_t* rows_in;
  uint32_t* keys_out;
  uint32_t* rows_out;
  uint32_t* counts;          // [digits][tiles]
  uint32_t* totals;          // [256]
  uint32_t* bitmap;          // of the codes that have rows: cleared by the first pass, set by the sums
  int64_t rows, n;
  int tiles, shift, bits;
};

// The lanes of the warp with the same digit, by a table of the warp's own that is zero before and after.
__device__ __forceinline__ uint32_t peers_of(uint32_t* table, uint32_t digit, bool in) {
  const int lane = threadIdx.x & 31;
  if (in) atomicOr(table + digit, 1u << lane);
  __syncwarp();
  const uint32_t same = in ? table[digit] : 0u;
  __syncwarp();
  if (in) table[digit] = 0u;  // (the next call's first addition comes behind its caller's __syncwarp)
  return same;
}

// What does not name a code is the code n, behind all others.
template <typename I>
__device__ __forceinline__ uint32_t code_of(const void* idx, int64_t r, int64_t n) {
  const I v = static_cast<const I*>(idx)[r];
  return v >= 0 && v < n ? (uint32_t)v : (uint32_t)n;
}
// I: the first pass reads indices of this type; char: a later pass
template <typename I>
__device__ __forceinline__ uint32_t key_at(const SortArgs& a, int64_t r) {
  if constexpr (sizeof(I) == 1) return a.keys[r];
  else return code_of<I>(a.idx, r, a.n);
}

// Exclusive sum over the block's threads; `total` of all of them.  `sums`: a word for each warp.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    before += w < warp ? sums[w] : 0u;
    total += sums[w];
  }
  return before + x - v;
}

// Tiles of 256 ITEMS pairs.  ITEMS is 16, or 4 where those would be too few to fill the device (300,000 rows: a pass of 74
// tiles took 35 us).
template <typename I, int ITEMS>
__global__ void __launch_bounds__(kThreads) k_embedding_count(const SortArgs a) {
  follow();
  __shared__ uint32_t s[256];
  s[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t mask = (1u << a.bits) - 1;
  const int lane = threadIdx.x & 31;
  const int64_t base = (int64_t)blockIdx.x * (kThreads * ITEMS) + (threadIdx.x >> 5) * (32 * ITEMS) + lane;
  uint32_t key[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) key[i] = base + i * 32 < a.rows ? key_at<I>(a, base + i * 32) : 0u;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const bool in = base + i * 32 < a.rows;
    const uint32_t d = in ? (key[i] >> a.shift) & mask : 256u;
    int alike;  // a common code would be added 32 times one after the other
    __match_all_sync(0xffffffffu, d, &alike);
    if (alike) {
      if (in && lane == 0) atomicAdd(s + d, 32u);
    } else if (in) {
      atomicAdd(s + d, 1u);
    }
  }
  if constexpr (sizeof(I) != 1) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (a.n + 31) / 32; i += (int64_t)gridDim.x * kThreads)
      a.bitmap[i] = 0u;
  }
  __syncthreads();
  if (threadIdx.x <= mask) a.counts[(int64_t)threadIdx.x * a.tiles + blockIdx.x] = s[threadIdx.x];
}

// A block for each digit: the exclusive sums of its counts over the tiles.
__global__ void __launch_bounds__(kThreads) k_embedding_scan(const SortArgs a) {
  follow();
  __shared__ uint32_t s_sums[kWarps];
  uint32_t* c = a.counts + (int64_t)blockIdx.x * a.tiles;
  uint32_t run = 0;
  for (int t0 = 0; t0 < a.tiles; t0 += kThreads * 4) {  // four counts a thread
    uint32_t v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + threadIdx.x * 4 + i;
      v[i] = t < a.tiles ? c[t] : 0u;
      sum += v[i];
    }
    uint32_t total, before = run + block_scan<kThreads>(sum, s_sums, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + threadIdx.x * 4 + i;
      if (t < a.tiles) c[t] = before;
      before += v[i];
    }
    run += total;
  }
  if (threadIdx.x == 0) a.totals[blockIdx.x] = run;
}

template <typename I, int ITEMS>
__global__ void __launch_bounds__(kThreads, ITEMS == 16 ? 2 : 3) k_embedding_scatter(const SortArgs a) {
  follow();
  __shared__ uint32_t s_count[kWarps][256];  // of each warp's digits; then where its first of them goes in the tile
  __shared__ uint32_t s_start[256];          // where a digit's run begins in the tile
  __shared__ uint32_t s_out[256];            // and in the output, less s_start
  __shared__ uint32_t s_sums[kWarps];
  __shared__ uint32_t s_key[kThreads * ITEMS > kWarps * 256 ? kThreads * ITEMS : kWarps * 256], s_row[kThreads * ITEMS];
  uint32_t* peers = s_key + (threadIdx.x >> 5) * 256;  // (the tables of peers, before the pairs are placed)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int i = threadIdx.x; i < kWarps * 256; i += kThreads) s_count[i / 256][i % 256] = 0, s_key[i] = 0;
  const int64_t base = (int64_t)blockIdx.x * (kThreads * ITEMS) + warp * (32 * ITEMS) + lane;
  uint32_t key[ITEMS], row[ITEMS], rank[ITEMS / 2];  // (16 bits are enough for a rank)
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t r = base + i * 32;
    key[i] = r < a.rows ? key_at<I>(a, r) : 0u;
    if constexpr (sizeof(I) == 1) row[i] = r < a.rows ? a.rows_in[r] : 0u;
    else row[i] = (uint32_t)r;
  }
  const uint32_t total_of_digit = threadIdx.x <= mask ? a.totals[threadIdx.x] : 0u;
  const uint32_t here = threadIdx.x <= mask ? a.counts[(int64_t)threadIdx.x * a.tiles + blockIdx.x] : 0u;
  uint32_t total;
  const uint32_t digit_base = block_scan<kThreads>(total_of_digit, s_sums, total);  // (its barriers also end the clearing above)
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const bool in = base + i * 32 < a.rows;
    const uint32_t d = (key[i] >> a.shift) & mask;
    const uint32_t same = peers_of(peers, d, in);
    const uint32_t before = s_count[warp][d];
    const uint32_t mine = before + __popc(same & ((1u << lane) - 1));
    rank[i / 2] = i % 2 ? rank[i / 2] | mine << 16 : mine;
    __syncwarp();
    if (in) s_count[warp][d] = before + __popc(same);  // (every peer stores the same)
    __syncwarp();
  }
  __syncthreads();
  uint32_t sum = 0;
  if (threadIdx.x <= mask) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t t = s_count[w][threadIdx.x];
      s_count[w][threadIdx.x] = sum;
      sum += t;
    }
  }
  const uint32_t start = block_scan<kThreads>(sum, s_sums, total);
  if (threadIdx.x <= mask) {
    s_start[threadIdx.x] = start;
    s_out[threadIdx.x] = digit_base + here - start;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (base + i * 32 >= a.rows) continue;
    const uint32_t d = (key[i] >> a.shift) & mask, at = s_start[d] + s_count[warp][d] + (rank[i / 2] >> (i % 2 * 16) & 0xffffu);
    s_key[at] = key[i], s_row[at] = row[i];
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < total; i += kThreads) {
    const uint32_t k = s_key[i], to = s_out[(k >> a.shift) & mask] + i;
    a.keys_out[to] = k, a.rows_out[to] = s_row[i];
  }
}

// ------------------------------------------------------------------ backward: the sums
struct SumArgs {
  const void* dy;
  const void* idx;          // few rows only
  const uint32_t* keys;     // sorted
  const uint32_t* order;    // and the rows
  uint32_t* bitmap;
  void* dtable;
  float* ends;              // [blocks][2][ldp]: sums that go on from the block before, into the block after
  uint32_t* flags;          // [blocks]: kHead, kThrough, kTail
  uint32_t* tail_code;      // [blocks]
  int64_t rows, n, ldy, ldt, ldp;
  int per_walker, width;
  unsigned blocks;
  float scale;
};
// A part's first code has rows before the part (head; through: behind it too), its last code has rows behind it (tail).
constexpr uint32_t kHead = 1, kThrough = 2, kTail = 4;

template <typename T, int VE>
__device__ __forceinline__ void write_sum(const SumArgs& a, uint32_t code, int col, const float* acc) {
  if (col >= a.width) return;
  float f[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) f[e] = acc[e] * a.scale;
  VecIO<T, VE>::store(static_cast<T*>(a.dtable) + (int64_t)code * a.ldt + col, f);
}

constexpr int kBatch = 8;  // a walker's part begins at a multiple of it
// A walker's rows, a lane's vector of each, by their sorted positions in lists that are padded to kBatch (what lies behind the
// last row is not used).  A position has a key, or `none` from `end` on; rows with the key `none` read as zeros.
// Lists in global memory: eight rows at once in registers, and the next eight's keys while these are added up.
template <typename T, int VE, typename P>
struct ListedRows {
  using IO = VecIO<T, VE>;
  using Pos = P;
  static constexpr int B = 8;
  const uint32_t *keys, *order;
  const T* dy;  // at the lane's column
  int64_t ldy;
  Pos end;
  uint32_t none;
  bool there;  // such a column
  uint32_t next_k[B], next_o[B], k[B];
  typename IO::Raw v[B];
  __device__ __forceinline__ void ahead(Pos p) {
#pragma unroll
    for (int h = 0; h < B; h += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(keys + p + h), o = *reinterpret_cast<const uint4*>(order + p + h);
      next_k[h] = q.x, next_k[h + 1] = q.y, next_k[h + 2] = q.z, next_k[h + 3] = q.w;
      next_o[h] = o.x, next_o[h + 1] = o.y, next_o[h + 2] = o.z, next_o[h + 3] = o.w;
    }
  }
  __device__ __forceinline__ void start(Pos p) { ahead(p); }
  __device__ __forceinline__ void batch(Pos p) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      k[u] = p + u < end ? next_k[u] : none;
      v[u] = k[u] != none && there ? IO::load(dy + (int64_t)next_o[u] * ldy) : IO::zero();
    }
    if (p + B < end) ahead(p + B);
  }
  __device__ __forceinline__ uint32_t key(int u) const { return k[u]; }
  __device__ __forceinline__ typename IO::Raw value(int u) { return v[u]; }
  __device__ __forceinline__ void done(int) {}
};

__device__ __forceinline__ void copy_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
// Lists in shared memory: four rows are always in flight, through a ring of the thread's own in shared memory, which takes no
// registers (16 bytes a vector; shorter ones take the registers of a batch of eight).
template <typename T, int VE>
struct RingRows {
  using IO = VecIO<T, VE>;
  using Pos = int;
  using Raw = typename IO::Raw;
  static constexpr bool kRing = sizeof(Raw) == 16;
  static constexpr int B = kRing ? 4 : 8;
  const uint16_t* keys;
  const uint32_t* order;
  const T* dy;
  int64_t ldy;
  int end;
  bool there;
  Raw* ring;  // [B][threads], at the thread's
  uint32_t k[B], o[B];
  Raw v[kRing ? 1 : B];
  __device__ __forceinline__ void rows_at(int p) {
#pragma unroll
    for (int h = 0; h < B; h += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(order + p + h);
      o[h] = q.x, o[h + 1] = q.y, o[h + 2] = q.z, o[h + 3] = q.w;
    }
  }
  __device__ __forceinline__ void issue(int p, int u) {
    if (p + u < end && there) copy_async16(ring + u * kPartThreads, dy + (int64_t)o[u] * ldy);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  int now;
  __device__ __forceinline__ void start(int p) {
    if constexpr (kRing) {
      rows_at(p);
#pragma unroll
      for (int u = 0; u < B; ++u) issue(p, u);
    }
  }
  __device__ __forceinline__ void batch(int p) {
#pragma unroll
    for (int h = 0; h < B; h += 4) {
      const uint2 q = *reinterpret_cast<const uint2*>(keys + p + h);
      k[h] = q.x & 0xffffu, k[h + 1] = q.x >> 16, k[h + 2] = q.y & 0xffffu, k[h + 3] = q.y >> 16;
    }
#pragma unroll
    for (int u = 0; u < B; ++u) k[u] = p + u < end ? k[u] : 0xffffu;
    now = p;
    if constexpr (kRing) {
      if (p + B < end) rows_at(p + B);
    } else {
      rows_at(p);
#pragma unroll
      for (int u = 0; u < B; ++u) v[u] = p + u < end && there ? IO::load(dy + (int64_t)o[u] * ldy) : IO::zero();
    }
  }
  __device__ __forceinline__ uint32_t key(int u) const { return k[u]; }
  __device__ __forceinline__ Raw value(int u) {
    if constexpr (kRing) {
      asm volatile("cp.async.wait_group 3;" ::: "memory");
      return now + u < end && there ? ring[u * kPartThreads] : IO::zero();
    } else {
      return v[u];
    }
  }
  __device__ __forceinline__ void done(int u) {
    if constexpr (kRing) issue(now + B, u);
  }
};

// A walker's part [begin, end) of sorted rows, of `total` in all: codes inside it are summed up and put(code, sums), the
// sums at its ends go to `head` and `tail` (the lane's own VE floats).  Returns the flags; `code` is the last one.  `none`:
// the key of rows without a code, behind all others; seen(code): the part has the code's first row.
template <typename T, int VE, typename R, typename Key, typename Put, typename Seen>
__device__ __forceinline__ uint32_t walk(R& rows, const Key* keys, typename R::Pos begin, typename R::Pos total, uint32_t none,
                                         float* head, float* tail, uint32_t& code, Put put, Seen seen) {
  using IO = VecIO<T, VE>;
  const typename R::Pos end = rows.end;
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.f;
  uint32_t flag = 0;
  code = none;
  if (begin >= end) return 0;
  rows.start(begin);
  code = keys[begin];
  bool from_before = begin > 0 && code != none && keys[begin - 1] == code;
  if (!from_before && code != none) seen(code);
  for (typename R::Pos p = begin; p < end; p += R::B) {
    rows.batch(p);
#pragma unroll
    for (int u = 0; u < R::B; ++u) {
      const uint32_t k = rows.key(u);
      if (p + u < end && k != code) {  // the sum of `code` is complete here
        if (from_before) {
#pragma unroll
          for (int e = 0; e < VE; ++e) head[e] = acc[e];
          flag |= kHead;
          from_before = false;
        } else {
          put(code, acc);
        }
        code = k;
        if (code != none) seen(code);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] = 0.f;
      }
      float f[VE];
      IO::unpack(rows.value(u), f);
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += f[e];
      rows.done(u);
    }
  }
  if (code != none) {
    const bool goes_on = end < total && keys[end] == code;
    if (from_before || goes_on) {
      float* to = from_before ? head : tail;
#pragma unroll
      for (int e = 0; e < VE; ++e) to[e] = acc[e];
      flag |= from_before ? (goes_on ? kHead | kThrough : kHead) : kTail;
    } else {
      put(code, acc);
    }
  }
  return flag;
}

// The sum of a walker's open end (its tail, or walker 0's head) and the heads behind it, in acc; returns whether it is still
// open behind the last walker.  (A lane reads its own columns only.)
template <int VE>
__device__ __forceinline__ bool join(const float* from, const float* heads, const uint32_t* flags, bool open, int walker,
                                     int walkers, int g, int lane, float* acc) {
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = from[e];
  for (int w = walker + 1; w < walkers && open; ++w) {
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] += heads[(w * g + lane) * VE + e];
    open = flags[w] & kThrough;
  }
  return open;
}

constexpr int sum_blocks(int ve) { return ve >= 4 ? 2 : 3; }  // of an SM, by the registers
// G lanes to a walker, a vector each; gridDim.y slabs of columns.
template <typename T, int VE, int G>
__global__ void __launch_bounds__(kThreads, sum_blocks(VE)) k_embedding_sum(const SumArgs a) {
  follow();
  constexpr int kWalkers = kThreads / G;
  __shared__ float s_end[2][kThreads * VE];  // heads and tails
  __shared__ uint32_t s_flag[kWalkers], s_block;
  const int lane = threadIdx.x % G, walker = threadIdx.x / G;
  const int col = ((int)blockIdx.y * G + lane) * VE;
  const int64_t from = ((int64_t)blockIdx.x * kWalkers + walker) * a.per_walker;
  const int begin = (int)min(from, a.rows), end = (int)min(from + a.per_walker, a.rows);  // (at most 2^31 - 1024 rows)
  float *head = s_end[0] + threadIdx.x * VE, *tail = s_end[1] + threadIdx.x * VE;
  uint32_t code, word = 0, bits = 0;  // codes seen, gathered to words of the bitmap
  const bool tells = lane == 0 && blockIdx.y == 0;
  ListedRows<T, VE, int> list;
  list.keys = a.keys, list.order = a.order, list.dy = static_cast<const T*>(a.dy) + col, list.ldy = a.ldy, list.end = end;
  list.none = (uint32_t)a.n, list.there = col < a.width;
  const uint32_t flag = walk<T, VE>(
      list, a.keys, begin, (int)a.rows, (uint32_t)a.n, head, tail, code,
      [&](uint32_t c, const float* sum) { write_sum<T, VE>(a, c, col, sum); },
      [&](uint32_t c) {
        if (c >> 5 != word) {
          if (tells && bits) atomicOr(a.bitmap + word, bits);
          word = c >> 5, bits = 0;
        }
        bits |= 1u << (c & 31);
      });
  if (tells && bits) atomicOr(a.bitmap + word, bits);
  if (lane == 0) s_flag[walker] = flag;
  if (threadIdx.x == 0) s_block = 0;
  __syncthreads();
  float acc[VE];
  auto keep = [&](int end_of, uint32_t flags) {  // for the kernel that joins the blocks
    float* to = a.ends + ((int64_t)blockIdx.x * 2 + end_of) * a.ldp + col;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (col + e < a.width) to[e] = acc[e];
    if (lane == 0) atomicOr(&s_block, flags);
  };
  if (flag & kTail) {
    if (join<VE>(tail, s_end[0], s_flag, true, walker, kWalkers, G, lane, acc)) {
      keep(1, kTail);
      if (lane == 0) a.tail_code[blockIdx.x] = code;
    } else {
      write_sum<T, VE>(a, code, col, acc);
    }
  }
  if (walker == 0 && flag & kHead)
    keep(0, join<VE>(head, s_end[0], s_flag, flag & kThrough, 0, kWalkers, G, lane, acc) ? kHead | kThrough : kHead);
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = s_block;
}

// Zeros for the codes without rows among the 32 of a word; a warp, G lanes to a row.
template <typename T, int VE>
__device__ __forceinline__ void write_zeros(const SumArgs& a, uint32_t empty, int64_t first, int g, int slab) {
  const int lane = threadIdx.x & 31, col = (slab * g + lane % g) * VE;
  const float none[VE] = {};
  if (col >= a.width || lane >= 32 / g * g) return;
  for (int r = lane / g; r < 32; r += 32 / g)
    if ((empty >> r) & 1u) VecIO<T, VE>::store(static_cast<T*>(a.dtable) + (first + r) * a.ldt + col, none);
}

// A block for each block of the sums: its tail and the heads behind it, every kWalkers-th to a walker.  The blocks behind
// those write the zeros.
template <typename T, int VE, int G>
__global__ void __launch_bounds__(kThreads) k_embedding_join(const SumArgs a) {
  follow();
  if (blockIdx.x >= a.blocks) {
    const int64_t word = (int64_t)(blockIdx.x - a.blocks) * kWarps + (threadIdx.x >> 5);
    if (word * 32 >= a.n) return;
    uint32_t empty = ~a.bitmap[word];
    if (a.n - word * 32 < 32) empty &= (1u << (a.n - word * 32)) - 1;
    if (empty) write_zeros<T, VE>(a, empty, word * 32, G, blockIdx.y);
    return;
  }
  if (!(a.flags[blockIdx.x] & kTail)) return;
  constexpr int kWalkers = kThreads / G;
  __shared__ float s[kThreads * VE];
  __shared__ unsigned s_first;
  const int lane = threadIdx.x % G, walker = threadIdx.x / G;
  const int col = ((int)blockIdx.y * G + lane) * VE;
  unsigned last = blockIdx.x + 1;  // the first block that the code does not go through
  for (;; last += kThreads) {
    const unsigned b = last + threadIdx.x;
    if (threadIdx.x == 0) s_first = kThreads;
    __syncthreads();
    if (b >= a.blocks || !(a.flags[b] & kThrough)) atomicMin(&s_first, threadIdx.x);
    __syncthreads();
    const unsigned first = s_first;
    __syncthreads();
    if (first < kThreads) {
      last += first;
      break;
    }
  }
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.f;
  if (walker == 0) {
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (col + e < a.width) acc[e] = a.ends[((int64_t)blockIdx.x * 2 + 1) * a.ldp + col + e];
  }
#pragma unroll 4
  for (unsigned b = blockIdx.x + 1 + walker; b <= last; b += kWalkers) {
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (col + e < a.width) acc[e] += a.ends[(int64_t)b * 2 * a.ldp + col + e];
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) s[threadIdx.x * VE + e] = acc[e];
  __syncthreads();
  if (walker != 0) return;
  for (int w = 1; w < kWalkers && blockIdx.x + 1 + w <= last; ++w) {
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] += s[(w * G + lane) * VE + e];
  }
  write_sum<T, VE>(a, a.tail_code[blockIdx.x], col, acc);
}

// ------------------------------------------------------------------ backward: buckets
// One pass of a sort puts (code, row) pairs into up to 2,048 buckets of 2^shift neighbouring codes each, in the order of the
// rows.  A block of the second step takes a bucket, or a part of `cap` rows of one that has more, sorts it in shared memory
// and sums it up as above.  Whole buckets are written at once, zeros included; the sums of parts go to the workspace, for a
// third step that joins them in order.
// Parts' sums take a place for each of a bucket's codes, and most buckets may have little more rows than a part: places for all of
// these would be two thirds as many sums as dy has rows.  Where that is much, there are places for one part of every bucket that can
// have several and an eighth more; where the indices are such that these are too few, parts have 2, 4, .. times `cap` rows, which a
// block takes in turn.
constexpr int kPartWarps = kPartThreads / 32, kPartItems = 16;  // pairs of a thread in a tile
constexpr int kMostBuckets = 2048, kMostCodes = 2048;  // a thread has four of either
constexpr int kMostRows = 6144;                        // of a part
struct Part {
  uint32_t bucket, begin, end, slot;  // its pairs; where the sums go, or kWhole
};
struct Bucket {  // of more than `cap` rows
  uint32_t bucket, slot, parts, unused;
};
constexpr uint32_t kWhole = 0xffffffffu;
struct PartArgs {
  SumArgs s;
  uint2* pairs;        // codes and rows
  uint32_t* counts;    // [tiles][padded buckets]
  uint32_t* totals;    // of the buckets
  Part* parts;
  Bucket* many;        // buckets of more than `cap` rows
  uint32_t* numbers;   // of parts and of those buckets
  float* sums;         // [slots][codes][ldp]
  uint32_t* seen;      // [slots][words]: codes that have rows
  int tiles, buckets, padded, shift, codes, cap, slots;
};

// How many pairs with the same digit the warp had before, in its row of counters: what an atomic addition returns, unless
// lanes share a digit, whose order is then that of the lanes.  (Votes on each bit of the digit, 50 instructions, took 88 us
// for the scatter of 11M rows into 1,954 buckets.)
__device__ __forceinline__ uint32_t rank_of(uint16_t* counters, uint32_t digit, bool in) {
  const int shift = digit % 2 * 16;
  uint32_t rank = 0, now = 0;
  if (in) rank = atomicAdd(reinterpret_cast<uint32_t*>(counters) + digit / 2, 1u << shift) >> shift & 0xffffu;
  __syncwarp();
  if (in) now = *reinterpret_cast<volatile uint16_t*>(counters + digit);
  uint32_t left = __ballot_sync(0xffffffffu, in && rank + 1 != now);  // a lane at least of each shared digit
  while (left) {
    const uint32_t d = __shfl_sync(0xffffffffu, digit, __ffs(left) - 1);
    const uint32_t same = __ballot_sync(0xffffffffu, in && digit == d);
    if (in && digit == d) rank = now - __popc(same) + __popc(same & ((1u << (threadIdx.x & 31)) - 1));
    left &= ~same;
  }
  __syncwarp();
  return rank;
}
// The warps' counters of the thread's four digits, from counts to how many the warps before have; `total`: of the four.
__device__ __forceinline__ uint4 four_totals(uint16_t* counters, int digits) {
  uint2 sum = make_uint2(0u, 0u);
  if ((int)threadIdx.x * 4 < digits) {
#pragma unroll
    for (int w = 0; w < kPartWarps; ++w) {
      uint2* p = reinterpret_cast<uint2*>(counters + w * digits) + threadIdx.x;
      const uint2 v = *p;
      *p = sum;
      sum.x += v.x, sum.y += v.y;  // (no sum passes 16 bits)
    }
  }
  return make_uint4(sum.x & 0xffffu, sum.x >> 16, sum.y & 0xffffu, sum.y >> 16);
}
__device__ __forceinline__ uint4 four_starts(uint4 t, uint32_t* s_sums, uint32_t& total) {
  const uint32_t b = block_scan<kPartThreads>(t.x + t.y + t.z + t.w, s_sums, total);
  return make_uint4(b, b + t.x, b + t.x + t.y, b + t.x + t.y + t.z);
}

template <typename I>
__global__ void __launch_bounds__(kPartThreads) k_embedding_bucket_count(const PartArgs a) {
  follow();
  __shared__ uint32_t s[kMostBuckets];
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < a.padded; i += kPartThreads) s[i] = 0;
  __syncthreads();
  // (in any order: four neighbours a thread)
  const int64_t base = (int64_t)blockIdx.x * (kPartThreads * kPartItems) + threadIdx.x * 4;
  uint32_t key[kPartItems];
  if (base - threadIdx.x * 4 + kPartThreads * kPartItems <= a.s.rows && reinterpret_cast<uintptr_t>(a.s.idx) % (4 * sizeof(I)) == 0) {
#pragma unroll
    for (int i = 0; i < kPartItems; i += 4) {
      struct alignas(sizeof(I) == 4 ? 16 : 32) Four { I v[4]; };
      const Four f = *reinterpret_cast<const Four*>(static_cast<const I*>(a.s.idx) + base + i * kPartThreads);
#pragma unroll
      for (int j = 0; j < 4; ++j) key[i + j] = code_of<I>(f.v, j, a.s.n);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPartItems; ++i) {
      const int64_t r = base + i / 4 * (4 * kPartThreads) + i % 4;
      key[i] = r < a.s.rows ? code_of<I>(a.s.idx, r, a.s.n) : (uint32_t)a.s.n;
    }
  }
#pragma unroll
  for (int i = 0; i < kPartItems; ++i) {
    const bool in = key[i] < (uint32_t)a.s.n;
    const uint32_t d = in ? key[i] >> a.shift : kMostBuckets;
    int alike;  // a common bucket would be added to 32 times one after the other
    __match_all_sync(0xffffffffu, d, &alike);
    if (alike) {
      if (in && lane == 0) atomicAdd(s + d, 32u);
    } else if (in) {
      atomicAdd(s + d, 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.padded; i += kPartThreads) a.counts[(int64_t)blockIdx.x * a.padded + i] = s[i];
}

// Exclusive sums of the counts over the tiles: a block has 8 buckets, 128 runs of 8 tiles side by side.
__global__ void __launch_bounds__(1024) k_embedding_bucket_scan(const PartArgs a) {
  follow();
  constexpr int kRun = 8;
  __shared__ uint32_t s[2][32][8];
  const int d = threadIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bucket = blockIdx.x * 8 + d;
  uint32_t* c = a.counts + bucket;
  const int tiles = bucket < a.padded ? a.tiles : 0;
  uint32_t carry = 0;
  for (int r0 = 0, half = 0; r0 < a.tiles; r0 += 128 * kRun, half ^= 1) {
    const int t0 = r0 + (threadIdx.x >> 3) * kRun;
    uint32_t v[kRun], sum = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = t0 + i < tiles ? c[(int64_t)(t0 + i) * a.padded] : 0u;
#pragma unroll
    for (int i = 0; i < kRun; ++i) sum += v[i];
    uint32_t x = sum;  // inclusive over the warp's four runs
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane >= 24) s[half][warp][d] = x;
    __syncthreads();
    uint32_t before = carry + x - sum;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const uint32_t y = s[half][w][d];
      before += w < warp ? y : 0u;
      carry += y;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (t0 + i < tiles) c[(int64_t)(t0 + i) * a.padded] = before;
      before += v[i];
    }
  }
  if (threadIdx.x < 8 && tiles) a.totals[bucket] = carry;
}

// The list of parts, for the next step: of the thread's four buckets' sizes and beginnings.  (A call of its
// own: inlined, it makes the kernel spill.)
__device__ __noinline__ void list_parts(const PartArgs& a, uint4 sizes, uint4 first, uint32_t* s_sums) {
  const uint32_t size[4] = {sizes.x, sizes.y, sizes.z, sizes.w}, from[4] = {first.x, first.y, first.z, first.w};
  uint32_t parts[4], all, several, buckets, sum_several;
  uint32_t slot;
  for (uint32_t cap = a.cap;; cap *= 2) {  // (as large as all rows at last: one for each such bucket, which fits)
    all = several = buckets = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      parts[j] = (int)threadIdx.x * 4 + j >= a.buckets ? 0u : size[j] <= (uint32_t)a.cap ? 1u : (size[j] - 1) / cap + 1;
      all += parts[j];
      if (size[j] > (uint32_t)a.cap) several += parts[j], ++buckets;
    }
    slot = block_scan<kPartThreads>(several, s_sums, sum_several);
    if (sum_several <= (uint32_t)a.slots || cap >> 31) break;
  }
  uint32_t sum_all, sum_buckets;
  uint32_t to = block_scan<kPartThreads>(all, s_sums, sum_all), list = block_scan<kPartThreads>(buckets, s_sums, sum_buckets);
  if (threadIdx.x == 0) a.numbers[0] = sum_all, a.numbers[1] = sum_buckets;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t d = threadIdx.x * 4 + j, n = parts[j];
    const bool whole = size[j] <= (uint32_t)a.cap;
    if (n && !whole) a.many[list++] = Bucket{d, slot, n, 0u};
    const uint32_t rows = n ? (size[j] + n - 1) / n : 0u;
    for (uint32_t p = 0; p < n; ++p)
      a.parts[to++] = Part{d, from[j] + min(p * rows, size[j]), from[j] + min((p + 1) * rows, size[j]), whole ? kWhole : slot++};
  }
}

size_t scatter_bytes(int padded) {
  return std::max<size_t>((size_t)2 * kPartWarps * padded, (size_t)8 * kPartThreads * kPartItems) + (size_t)8 * padded;
}
template <typename I>
__global__ void __launch_bounds__(kPartThreads, 2) k_embedding_bucket_scatter(const PartArgs a) {
  follow();
  extern __shared__ __align__(16) uint32_t s_dyn[];
  __shared__ uint32_t s_sums[kPartWarps];
  uint32_t *s_start = s_dyn, *s_out = s_dyn + a.padded;  // where a bucket's run begins in the tile; in the pairs, less s_start
  uint16_t* counters = reinterpret_cast<uint16_t*>(s_dyn + 2 * a.padded);  // [warps][padded]
  uint2* s_pair = reinterpret_cast<uint2*>(counters);                      // and, once they have been read, the tile's pairs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kPartWarps * a.padded / 8; i += kPartThreads) reinterpret_cast<uint4*>(counters)[i] = uint4{};
  const uint32_t base = blockIdx.x * (kPartThreads * kPartItems) + warp * (32 * kPartItems) + lane, rows = (uint32_t)a.s.rows;  // (rows < 2^31)
  uint32_t key[kPartItems], at[kPartItems / 2];  // (16 bits are enough for a place in the tile)
#pragma unroll
  for (int i = 0; i < kPartItems; ++i)
    key[i] = base + i * 32 < rows ? code_of<I>(a.s.idx, base + i * 32, a.s.n) : (uint32_t)a.s.n;
  const bool mine = (int)threadIdx.x * 4 < a.padded;  // four buckets
  uint32_t total;
  {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u), in_all = mine ? reinterpret_cast<const uint4*>(a.totals)[threadIdx.x] : none;
    uint4 before = none;
    if (mine && (int)blockIdx.x < a.tiles) before = reinterpret_cast<const uint4*>(a.counts + (int64_t)blockIdx.x * a.padded)[threadIdx.x];
    const uint4 first = four_starts(in_all, s_sums, total);  // (its barriers also end the clearing above)
    if ((int)blockIdx.x == a.tiles) return list_parts(a, in_all, first, s_sums);
    if (mine)
      reinterpret_cast<uint4*>(s_out)[threadIdx.x] = make_uint4(first.x + before.x, first.y + before.y, first.z + before.z, first.w + before.w);
  }
#pragma unroll
  for (int i = 0; i < kPartItems; ++i) {
    const uint32_t rank = rank_of(counters + warp * a.padded, key[i] >> a.shift, key[i] < (uint32_t)a.s.n);
    at[i / 2] = i % 2 ? at[i / 2] | rank << 16 : rank;
  }
  __syncthreads();
  const uint4 start = four_starts(four_totals(counters, a.padded), s_sums, total);
  if (mine) {
    reinterpret_cast<uint4*>(s_start)[threadIdx.x] = start;
    const uint4 to = reinterpret_cast<uint4*>(s_out)[threadIdx.x];
    reinterpret_cast<uint4*>(s_out)[threadIdx.x] = make_uint4(to.x - start.x, to.y - start.y, to.z - start.z, to.w - start.w);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPartItems; ++i) {
    const uint32_t d = key[i] >> a.shift;
    if (key[i] < (uint32_t)a.s.n) at[i / 2] += (s_start[d] + counters[warp * a.padded + d]) << (i % 2 * 16);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPartItems; ++i)
    if (key[i] < (uint32_t)a.s.n) s_pair[at[i / 2] >> (i % 2 * 16) & 0xffffu] = make_uint2(key[i], base + i * 32);
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < total; i += kPartThreads) {
    const uint2 p = s_pair[i];
    a.pairs[s_out[p.x >> a.shift] + i] = p;
  }
}

// Shared memory of a block that sums a part up: where the codes' rows begin; the warps' counters and, once they have been
// read, the sorted codes and rows and the walkers' ends.
size_t part_bytes(int cap, int codes, int ve) {
  const size_t digits = std::max(codes, 4), list = cap + 8;
  const size_t ring = 4 * 16 * kPartThreads;  // (not used where vectors are shorter)
  return 4 * (digits + 4) + std::max(2 * kPartWarps * digits, 6 * list + 4 * kPartThreads * (2 * (size_t)ve + 1) + ring);
}
// `m` rows of a part from pair `from` on, `cap` at most.  TURNS: there may be more of the part; s_seen: those of its codes that had
// rows before these.
template <typename T, int VE, bool TURNS>
__device__ __forceinline__ void sum_rows(const PartArgs& p, const int g, const Part& part, const uint32_t from, const int m,
                                         uint32_t* s_seen) {
  extern __shared__ __align__(16) uint32_t s_dyn[];
  __shared__ uint32_t s_sums[kPartWarps];
  const SumArgs& a = p.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = max(p.codes, 4), list = p.cap + 8;
  uint32_t* s_start = s_dyn;
  uint16_t* counters = reinterpret_cast<uint16_t*>(s_dyn + digits + 4);
  uint32_t* s_row = s_dyn + digits + 4;
  float* ends = reinterpret_cast<float*>(s_row + list);  // [2][threads VE]
  using Raw = typename VecIO<T, VE>::Raw;
  Raw* ring = reinterpret_cast<Raw*>(ends + 2 * kPartThreads * VE);
  uint32_t* flags = reinterpret_cast<uint32_t*>(ends + 2 * kPartThreads * VE) + 16 * kPartThreads;
  uint16_t* s_key = reinterpret_cast<uint16_t*>(flags + kPartThreads);
  for (int i = threadIdx.x; i < kPartWarps * digits / 8; i += kPartThreads) reinterpret_cast<uint4*>(counters)[i] = uint4{};
  constexpr int kItems = kMostRows / kPartThreads;
  const int share = (m + kPartThreads - 1) / kPartThreads * 32, i0 = warp * share + lane;  // a warp's pairs
  uint32_t key[kItems];  // local codes, their ranks above them (rows are read when they are placed: registers)
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    key[i] = 0u;
    if (i * 32 < share && i0 + i * 32 < m) {
      const uint32_t v = p.pairs[from + i0 + i * 32].x;
      key[i] = v & (uint32_t)(p.codes - 1);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (i * 32 < share) key[i] |= rank_of(counters + warp * digits, key[i], i0 + i * 32 < m) << 16;
  __syncthreads();
  uint32_t total;
  const uint4 start = four_starts(four_totals(counters, digits), s_sums, total);
  if ((int)threadIdx.x * 4 < digits) reinterpret_cast<uint4*>(s_start)[threadIdx.x] = start;
  if (threadIdx.x == 0) s_start[digits] = (uint32_t)m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (i * 32 < share && i0 + i * 32 < m) {
      const uint32_t k = key[i] & 0xffffu;
      key[i] += (s_start[k] + counters[warp * digits + k]) << 16;
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (i * 32 < share && i0 + i * 32 < m) {
      const uint32_t to = key[i] >> 16;
      s_key[to] = (uint16_t)key[i], s_row[to] = p.pairs[from + i0 + i * 32].y;
    }
  __syncthreads();
  // the sums
  const bool whole = part.slot == kWhole;
  const uint32_t code0 = part.bucket << p.shift;  // (n <= 2^22)
  const int walkers = kPartThreads / g, wl = threadIdx.x % g, walker = threadIdx.x / g;  // (threads may be left over)
  const int col = ((int)blockIdx.y * g + wl) * VE;
  const int per = (m + walkers * kBatch - 1) / (walkers * kBatch) * kBatch;
  const int begin = walker < walkers ? min(walker * per, m) : m, end = min(begin + per, m);
  float *head = ends + threadIdx.x * VE, *tail = ends + (kPartThreads + threadIdx.x) * VE;
  auto put = [&](uint32_t c, const float* sum) {
    if (whole) {
      write_sum<T, VE>(a, code0 + c, col, sum);
    } else if (col < a.width) {
      float* to = p.sums + ((int64_t)part.slot * p.codes + c) * a.ldp + col;
      float f[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = sum[e];
      if (TURNS && from != part.begin && (s_seen[c >> 5] >> (c & 31) & 1u)) {
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = to[e] + f[e];
      }
      if constexpr (VE >= 4) {  // (rows of `ldp`, a multiple of 8)
#pragma unroll
        for (int e = 0; e < VE; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) to[e] = f[e];
      }
    }
  };
  uint32_t code;
  RingRows<T, VE> rows;
  rows.keys = s_key, rows.order = s_row, rows.dy = static_cast<const T*>(a.dy) + col, rows.ldy = a.ldy, rows.end = end;
  rows.there = col < a.width, rows.ring = ring + threadIdx.x;
  const uint32_t flag = walk<T, VE>(rows, s_key, begin, m, 0xffffu, head, tail, code, put, [](uint32_t) {});
  if (wl == 0 && walker < walkers) flags[walker] = flag;
  // codes without rows
  const int words = (p.codes + 31) / 32;
  auto have = [&](int w, bool there) {
    const int c = w * 32 + lane;
    return __ballot_sync(0xffffffffu, there && s_start[min(c, digits - 1)] != s_start[min(c, digits - 1) + 1]);
  };
  for (int w = warp; (whole || !TURNS) && w < words; w += kPartWarps) {
    const int c = w * 32 + lane;
    const bool there = c < p.codes && code0 + c < (uint32_t)a.n;
    const uint32_t now = have(w, there);
    if (whole) {
      const uint32_t empty = __ballot_sync(0xffffffffu, there) & ~now;
      if (empty) write_zeros<T, VE>(a, empty, code0 + w * 32, g, blockIdx.y);
    } else if (lane == 0 && blockIdx.y == 0) {
      p.seen[(int64_t)part.slot * words + w] = now;
    }
  }
  __syncthreads();
  if (flag & kTail) {
    float acc[VE];
    join<VE>(tail, ends, flags, true, walker, walkers, g, wl, acc);
    put(code, acc);
  }
  if (!TURNS || whole) return;
  __syncthreads();
  for (int w = warp; w < words; w += kPartWarps) {
    const uint32_t now = have(w, w * 32 + lane < p.codes);
    if (lane == 0) s_seen[w] = from != part.begin ? s_seen[w] | now : now;
  }
}
// TURNS: parts may have more than `cap` rows.  (11M rows of 32 float32, 2M codes: 396 us either way.  Where most buckets have two
// parts, which then are one in two turns: 11M of 32 float32, codes from 600K of 2M, 567 and 513 us; 8M of 64 bfloat16, 600K codes, 427
// and 439.)
template <typename T, int VE, bool TURNS>
__global__ void __launch_bounds__(kPartThreads, 2) k_embedding_part(const PartArgs p, const int g) {
  follow();
  if (blockIdx.x >= p.numbers[0]) return;
  const Part part = p.parts[blockIdx.x];
  if constexpr (!TURNS) {
    sum_rows<T, VE, false>(p, g, part, part.begin, (int)(part.end - part.begin), nullptr);
  } else {
    __shared__ uint32_t s_seen[kMostCodes / 32];
    for (uint32_t from = part.begin;; from += p.cap) {
      sum_rows<T, VE, true>(p, g, part, from, (int)min(part.end - from, (uint32_t)p.cap), s_seen);
      if (part.end - from <= (uint32_t)p.cap) break;
      __syncthreads();  // (the next rows take the same memory)
    }
    if (part.slot == kWhole || blockIdx.y != 0) return;
    __syncthreads();
    const int words = (p.codes + 31) / 32;
    for (int w = threadIdx.x; w < words; w += kPartThreads) p.seen[(int64_t)part.slot * words + w] = s_seen[w];
  }
}

// The buckets of several parts: their parts' sums in order, every `per`-th to a walker.
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads) k_embedding_part_join(const PartArgs p, const int g) {
  follow();
  __shared__ float s[kThreads * VE];
  const SumArgs& a = p.s;
  const int walkers = kThreads / g, wl = threadIdx.x % g, walker = threadIdx.x / g;
  const int col = ((int)blockIdx.y * g + wl) * VE;
  const int per = max(walkers / p.codes, 1), codes = walkers / per, sub = walker % per;  // (powers of two)
  const int runs = (p.codes + codes - 1) / codes, words = (p.codes + 31) / 32;
  const uint32_t items = p.numbers[1] * (uint32_t)runs;
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const Bucket b = p.many[item / runs];
    const int c = (int)(item % runs) * codes + walker / per;
    const int64_t code = ((int64_t)b.bucket << p.shift) + c;
    const bool there = c < p.codes && code < a.n && col < a.width;
    float acc[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = 0.f;
    const uint32_t* seen = p.seen + (int64_t)b.slot * words + (c >> 5);
    const float* from = p.sums + ((int64_t)b.slot * p.codes + c) * a.ldp + col;
    for (uint32_t q0 = sub; there && q0 < b.parts; q0 += 4 * per) {
      uint32_t have[4];
      float v[4][VE];
#pragma unroll
      for (int u = 0; u < 4; ++u) have[u] = q0 + u * per < b.parts ? (seen[(int64_t)(q0 + u * per) * words] >> (c & 31)) & 1u : 0u;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[u][e] = have[u] ? from[(int64_t)(q0 + u * per) * p.codes * a.ldp + e] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += v[u][e];
      }
    }
    if (per > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VE; ++e) s[threadIdx.x * VE + e] = acc[e];
      __syncthreads();
      for (int w = 1; w < per && sub == 0; ++w) {
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += s[(threadIdx.x + w * g) * VE + e];
      }
    }
    if (there && sub == 0) write_sum<T, VE>(a, (uint32_t)code, col, acc);
  }
}

// ------------------------------------------------------------------ backward: few rows
// One launch: each block takes the codes of every gridDim.x-th run of `run` neighbours (so that common codes, which
// often are neighbours, spread), picks their rows out of all indices, sorts them in shared memory, and sums and writes as
// above.  No block waits for another.
constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32;
constexpr int64_t kFewRows = 8192;
constexpr int kFewItems = kFewRows / kFewThreads;  // indices of a lane
struct FewArgs {
  SumArgs s;
  int log_run;     // codes of a run, a power of two (32 at most)
  int bits;        // of a block's own numbers of codes
  int local;       // codes of a block at most
  int g;           // lanes of a walker
  int index_bits;
};
size_t few_bytes(int64_t rows, int local, int ve) {
  const size_t list = (size_t)(rows + 8) / 8 * 8;
  return 4 * (4 * list + (local + 31) / 32 + 2 * kFewWarps * 256 + 256 + kFewThreads + 2 * (size_t)kFewThreads * ve);
}

template <typename T, int VE>
__global__ void __launch_bounds__(kFewThreads) k_embedding_few(const FewArgs f) {
  follow();
  extern __shared__ __align__(16) uint32_t s_few[];
  __shared__ uint32_t s_sums[kFewWarps];
  const SumArgs& a = f.s;
  const int rows = (int)a.rows, list = (rows + 8) / 8 * 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t *key[2] = {s_few, s_few + 2 * list}, *row[2] = {s_few + list, s_few + 3 * list};
  uint32_t* bitmap = s_few + 4 * list;                       // of the block's codes
  uint32_t* count = bitmap + (f.local + 31) / 32;            // [warps][256]
  uint32_t* peers = count + kFewWarps * 256 + warp * 256;    // [warps][256]
  uint32_t* start = count + 2 * kFewWarps * 256;             // [256]
  uint32_t* flags = start + 256;                             // [threads]
  float* ends = reinterpret_cast<float*>(flags + kFewThreads);  // [2][threads VE]
  for (int i = threadIdx.x; i < (f.local + 31) / 32 + 2 * kFewWarps * 256; i += kFewThreads) bitmap[i] = 0u;
  // the block's own number of a code, or none: runs of codes go round the blocks
  const uint32_t none = (uint32_t)f.local, blocks = gridDim.x;
  auto local_of = [&](int64_t v) -> uint32_t {
    if (v < 0 || v >= a.n) return none;
    const uint32_t run = (uint32_t)v >> f.log_run;
    if (run % blocks != blockIdx.x) return none;
    return (run / blocks << f.log_run) | ((uint32_t)v & ((1u << f.log_run) - 1));
  };
  auto to_code = [&](uint32_t k) { return ((((k >> f.log_run) * blocks + blockIdx.x) << f.log_run) | (k & ((1u << f.log_run) - 1))); };
  // a warp's share of the rows, in their order: counted, then listed
  const int share = (rows + 32 * kFewWarps - 1) / (32 * kFewWarps) * 32, first = warp * share;
  uint32_t mine[kFewItems];
  uint32_t found = 0;
#pragma unroll
  for (int i = 0; i < kFewItems; ++i) {
    const int r = first + i * 32 + lane;
    mine[i] = none;
    if (i * 32 < share && r < rows)
      mine[i] = local_of(f.index_bits == 32 ? (int64_t) static_cast<const int32_t*>(a.idx)[r] : static_cast<const int64_t*>(a.idx)[r]);
  }
#pragma unroll
  for (int i = 0; i < kFewItems; ++i) found += __popc(__ballot_sync(0xffffffffu, mine[i] != none));
  uint32_t m, at = block_scan<kFewThreads>(lane == 0 ? found : 0u, s_sums, m);
  at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
  for (int i = 0; i < kFewItems; ++i) {
    const uint32_t have = __ballot_sync(0xffffffffu, mine[i] != none);
    if (mine[i] != none) {
      const uint32_t to = at + __popc(have & ((1u << lane) - 1));
      key[0][to] = mine[i], row[0][to] = first + i * 32 + lane;
      atomicOr(bitmap + (mine[i] >> 5), 1u << (mine[i] & 31));
    }
    at += __popc(have);
  }
  __syncthreads();
  // the list sorted by code, up to eight bits a pass
  int from = 0;
  const int part = ((int)m + 32 * kFewWarps - 1) / (32 * kFewWarps) * 32, p0 = warp * part;  // a warp's
  for (int shift = 0; shift < f.bits; shift += 8, from ^= 1) {
    const uint32_t *k = key[from], *r = row[from];
    uint16_t rank[kFewItems];
#pragma unroll
    for (int i = 0; i < kFewItems; ++i) {
      if (i * 32 >= part) break;
      const int p = p0 + i * 32 + lane;
      const bool in = p < (int)m;
      const uint32_t d = in ? (k[p] >> shift) & 255u : 0u;
      const uint32_t same = peers_of(peers, d, in);
      const uint32_t before = count[warp * 256 + d];
      rank[i] = (uint16_t)(before + __popc(same & ((1u << lane) - 1)));
      __syncwarp();
      if (in) count[warp * 256 + d] = before + __popc(same);
      __syncwarp();
    }
    __syncthreads();
    uint32_t sum = 0, total;
    if (threadIdx.x < 256) {
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const uint32_t t = count[w * 256 + threadIdx.x];
        count[w * 256 + threadIdx.x] = sum;
        sum += t;
      }
    }
    const uint32_t begin = block_scan<kFewThreads>(sum, s_sums, total);
    if (threadIdx.x < 256) start[threadIdx.x] = begin;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewItems; ++i) {
      if (i * 32 >= part) break;
      const int p = p0 + i * 32 + lane;
      if (p >= (int)m) break;
      const uint32_t d = (k[p] >> shift) & 255u, to = start[d] + count[warp * 256 + d] + rank[i];
      key[from ^ 1][to] = k[p], row[from ^ 1][to] = r[p];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kFewWarps * 256; i += kFewThreads) count[i] = 0u;
    __syncthreads();
  }
  // sums
  const int g = f.g, walkers = kFewThreads / g, wl = threadIdx.x % g, walker = threadIdx.x / g;
  const int col = ((int)blockIdx.y * g + wl) * VE;
  const int per = ((int)m + walkers * kBatch - 1) / (walkers * kBatch) * kBatch;
  const int begin = min(walker * per, (int)m), end = min(begin + per, (int)m);
  float *head = ends + threadIdx.x * VE, *tail = ends + (kFewThreads + threadIdx.x) * VE;
  uint32_t code;
  ListedRows<T, VE, int64_t> rows_of;  // (32 bits spill)
  rows_of.keys = key[from], rows_of.order = row[from], rows_of.dy = static_cast<const T*>(a.dy) + col, rows_of.ldy = a.ldy;
  rows_of.end = end, rows_of.none = none, rows_of.there = col < a.width;
  const uint32_t flag = walk<T, VE>(
      rows_of, key[from], begin, m, none, head, tail, code,
      [&](uint32_t c, const float* sum) { write_sum<T, VE>(a, to_code(c), col, sum); }, [](uint32_t) {});
  if (wl == 0) flags[walker] = flag;
  __syncthreads();
  if (flag & kTail) {
    float acc[VE];
    join<VE>(tail, ends, flags, true, walker, walkers, g, wl, acc);
    write_sum<T, VE>(a, to_code(code), col, acc);
  }
  // zeros, by words of the block's codes (whole runs)
  for (int w = warp; w < (f.local + 31) / 32; w += kFewWarps) {
    const int run = 1 << f.log_run;
    for (int k0 = w * 32; k0 < min(w * 32 + 32, f.local); k0 += run) {
      const int64_t v0 = to_code(k0);
      if (v0 >= a.n) continue;
      uint32_t empty = ~bitmap[w] >> (k0 & 31);
      if (run < 32) empty &= (1u << run) - 1;
      if (a.n - v0 < run) empty &= (1u << (a.n - v0)) - 1;
      if (empty) write_zeros<T, VE>(a, empty, v0, g, blockIdx.y);
    }
  }
}

// ------------------------------------------------------------------ host
gs_status check_desc(const char* where, const gs_embedding_desc* d) {
  if (!d) return gs::set_error(GS_ERR_INVALID, "%s: descriptor is NULL", where);
  if (d->rows < 0 || d->rows > INT32_MAX - 1023 || d->n < 0 || d->n > INT32_MAX - 1 || d->width < 1 || d->width > (1 << 20))
    return gs::set_error(GS_ERR_INVALID, "%s: bad size %lld of %lld x %d", where, (long long)d->rows, (long long)d->n, d->width);
  if (d->dtype != GS_F32 && d->dtype != GS_BF16)
    return gs::set_error(GS_ERR_INVALID, "%s: unknown element type %d", where, d->dtype);
  if (d->index_bits != 32 && d->index_bits != 64)
    return gs::set_error(GS_ERR_INVALID, "%s: index_bits must be 32 or 64, got %d", where, d->index_bits);
  return GS_OK;
}
gs_status check_idx(const char* where, const gs_embedding_desc* d, const void* idx) {
  if (!idx || reinterpret_cast<uintptr_t>(idx) % (d->index_bits / 8))
    return gs::set_error(GS_ERR_INVALID, "%s: idx is NULL or misaligned", where);
  return GS_OK;
}

// elements of a vector: what the width and the two matrices' alignment allow
int vector_of(const gs_embedding_desc* d, const void* table, const void* rows) {
  auto fit = [&](int ve) {
    const int bytes = ve * (int)gs::dtype_size(d->dtype);
    return d->width % ve == 0 && gs::rows_aligned(table, d->n, d->ldt, d->dtype, bytes) &&
           gs::rows_aligned(rows, d->rows, d->ldy, d->dtype, bytes);
  };
  const int full = 16 / (int)gs::dtype_size(d->dtype);
  return fit(full) ? full : d->dtype == GS_BF16 && fit(2) ? 2 : 1;
}

template <typename F>
void by_vector(const gs_embedding_desc* d, int ve, F f) {
  if (d->dtype == GS_F32) {
    if (ve == 4) f(float{}, std::integral_constant<int, 4>{});
    else f(float{}, std::integral_constant<int, 1>{});
  } else {
    if (ve == 8) f(__nv_bfloat16{}, std::integral_constant<int, 8>{});
    else if (ve == 2) f(__nv_bfloat16{}, std::integral_constant<int, 2>{});
    else f(__nv_bfloat16{}, std::integral_constant<int, 1>{});
  }
}

// The backward's sizes, from the descriptor alone but for the vectors.
struct Plan {
  int bits, passes, items, tiles;
  int64_t padded;  // rows, to whole batches
  int64_t words;   // of the bitmap
  int64_t ldp;
};
Plan plan_of(const gs_embedding_desc* d) {
  Plan p{};
  while (p.bits < 32 && (d->n >> p.bits)) ++p.bits;  // of the codes 0..n
  if (p.bits < 1) p.bits = 1;
  p.passes = (p.bits + 7) / 8;
  p.items = d->rows <= (int64_t)152 * 4 * kThreads * 16 ? 4 : 16;
  p.tiles = (int)((d->rows + kThreads * p.items - 1) / (kThreads * p.items));
  p.padded = (d->rows + 7) / 8 * 8;
  p.words = (d->n + 31) / 32;
  p.ldp = (d->width + 7) / 8 * 8;
  return p;
}
// Rows of a walker: whole batches, blocks for 8 times what the device holds (152 SMs), or for once where a walker would have
// few.
int per_walker_of(int64_t rows, int walkers, int ve) {
  const int64_t blocks = 152 * sum_blocks(ve);
  int64_t want = (rows + blocks * walkers - 1) / (blocks * walkers);
  if (want > 64) want = std::max<int64_t>(64, want / 8);
  return (int)((want + kBatch - 1) / kBatch * kBatch);
}
int lanes_of(int width, int ve) {
  const int v = (width + ve - 1) / ve;
  return v <= 2 ? 2 : v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : 32;
}
int64_t blocks_of(int64_t rows, int g, int ve) {
  const int walkers = kThreads / g;
  const int64_t per = (int64_t)per_walker_of(rows, walkers, ve) * walkers;
  return (rows + per - 1) / per;
}

struct Buckets {
  int shift, count, padded, codes, cap, tiles;
  bool turns;  // parts may have several times `cap` rows
  int64_t parts, slots, many, words;  // at most: parts, buckets of more than `cap` rows; places of their parts' sums; of a part's codes
};
// Whether the buckets take a call, and how.  They save passes over the pairs, but the sort's shorter kernels are done sooner
// where there is little to sort.  Us by the sort and by buckets: 4,096 codes of 64 bfloat16 1M rows 60 and 66, 2M 107 and 94,
// 10M 462 and 356; 100K codes of 32 float32 1M rows 73 and 82, 2M 125 and 118, 10M 524 and 421; 1M codes of 32 float32 1M rows 91
// and 104, 2M 150 and 139, 10M 567 and 437; codes that the sort does in one pass (100 of 32 float32) 2M rows 87 and 101.
bool buckets_take(const gs_embedding_desc* d, Buckets& b) {
  if (d->n <= 256 || d->n > (int64_t)kMostBuckets * kMostCodes || d->rows < (3 << 19)) return false;
  int least = 0;  // codes to a bucket, as a shift, by the number of buckets
  while ((d->n - 1) >> least >= kMostBuckets) ++least;
  // parts of up to 6,144 rows, or fewer, so that there are 608 of them (152 SMs, 2 blocks each, twice), but of several times a
  // bucket's codes: the sums of parts are kept for each of these
  b.cap = (int)std::min<int64_t>(std::max<int64_t>((d->rows / 608 + 511) / 512 * 512, 4 << least), kMostRows);
  // codes to a bucket so that an average one is nearly a part
  b.shift = least;
  while (b.shift < 11 && (d->rows << (b.shift + 1)) / d->n <= b.cap * 15 / 16 && (8 << b.shift) <= b.cap) ++b.shift;
  b.count = (int)((d->n - 1) >> b.shift) + 1, b.padded = (b.count + 3) / 4 * 4, b.codes = 1 << b.shift;
  b.tiles = (int)((d->rows + kPartThreads * kPartItems - 1) / (kPartThreads * kPartItems));
  b.many = std::min<int64_t>(d->rows / b.cap, b.count);
  // places for any number of parts (two for each that can be full) where they take little space beside dy
  b.slots = 2 * (d->rows / b.cap);
  const int64_t sums = 4 * b.slots * b.codes * ((d->width + 7) / 8 * 8), dy = d->rows * d->width * (int64_t)gs::dtype_size(d->dtype);
  if (sums > std::max<int64_t>(64 << 20, dy / 4))
    b.turns = true, b.slots = b.many + d->rows / b.cap / 8;
  b.parts = b.count + std::min(b.slots, d->rows / b.cap);  // (a bucket of more than `cap` rows has one more than it can fill)
  b.words = (b.codes + 31) / 32;
  return true;
}
size_t carve(PartArgs* a, char* base, const gs_embedding_desc* d, const Buckets& b) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = base + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  PartArgs t{};
  const int64_t ldp = (d->width + 7) / 8 * 8;
  t.pairs = (uint2*)take(8 * (size_t)d->rows);
  t.counts = (uint32_t*)take(4 * (size_t)b.tiles * b.padded);
  t.totals = (uint32_t*)take(4 * (size_t)b.padded);
  t.parts = (Part*)take(sizeof(Part) * (size_t)b.parts);
  t.many = (Bucket*)take(sizeof(Bucket) * (size_t)b.many);
  t.numbers = (uint32_t*)take(8);
  t.sums = (float*)take(4 * (size_t)b.slots * b.codes * ldp);
  t.seen = (uint32_t*)take(4 * (size_t)b.slots * b.words);
  if (a) {
    t.s = a->s;
    t.s.ldp = ldp;
    t.tiles = b.tiles, t.buckets = b.count, t.padded = b.padded, t.shift = b.shift, t.codes = b.codes, t.cap = b.cap, t.slots = (int)b.slots;
    *a = t;
  }
  return at;
}

struct Space {
  uint32_t *keys[2], *order[2], *counts, *totals, *bitmap, *flags, *tail_code;
  float* ends;
};
size_t carve(Space* s, char* base, const gs_embedding_desc* d) {
  const Plan p = plan_of(d);
  int64_t blocks = 0;  // the most that any vector leads to
  for (int ve : {1, 2, 4, 8}) blocks = std::max(blocks, blocks_of(d->rows, lanes_of(d->width, ve), ve));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = base + at;
    at += (bytes + 255) / 256 * 256;
    return q;
  };
  Space t;
  for (int i = 0; i < 2; ++i) {
    t.keys[i] = (uint32_t*)take(4 * p.padded);
    t.order[i] = (uint32_t*)take(4 * p.padded);
  }
  t.counts = (uint32_t*)take(4 * 256 * (size_t)p.tiles);
  t.totals = (uint32_t*)take(4 * 256);
  t.bitmap = (uint32_t*)take(4 * p.words);
  t.flags = (uint32_t*)take(4 * blocks);
  t.tail_code = (uint32_t*)take(4 * blocks);
  t.ends = (float*)take(4 * 2 * p.ldp * blocks);
  if (s) *s = t;
  return at;
}

template <typename I>
void launch_pass(const SortArgs& a, int items, cudaStream_t st) {
  auto go = [&](auto count, auto scatter) {
    gs::launch(count, dim3(a.tiles), kThreads, 0, st, a);
    gs::launch(k_embedding_scan, dim3(1u << a.bits), kThreads, 0, st, a);
    gs::launch(scatter, dim3(a.tiles), kThreads, 0, st, a);
  };
  if (items == 4) go(k_embedding_count<I, 4>, k_embedding_scatter<I, 4>);
  else go(k_embedding_count<I, 16>, k_embedding_scatter<I, 16>);
}

// Whether one launch takes a call, and how: few enough rows that a block which gets all of them is done in time (2 MB: 25 us
// against the sort's 35).
constexpr int64_t kFewBytes = 2 << 20;
constexpr int kFewLocal = 1 << 17;  // codes of a block
bool few_takes(const gs_embedding_desc* d, FewArgs& f) {
  if (d->rows > kFewRows || d->rows * d->width * 4 > kFewBytes) return false;
  f.log_run = 0;
  while (f.log_run < 5 && (d->n >> (f.log_run + 1)) >= 152) ++f.log_run;
  const int64_t runs = (d->n + (1 << f.log_run) - 1) >> f.log_run;
  const int64_t blocks = std::min<int64_t>(runs, 152), local = (runs + blocks - 1) / blocks << f.log_run;
  if (local > kFewLocal) return false;
  f.local = (int)local;
  f.s.blocks = (unsigned)blocks;
  f.bits = 0;
  while ((local - 1) >> f.bits) ++f.bits;
  f.index_bits = d->index_bits;
  return true;
}
template <typename T, int VE>
gs_status launch_few(const char* where, FewArgs& f, cudaStream_t st) {
  const int vectors = (f.s.width + VE - 1) / VE;
  f.g = lanes_of(f.s.width, VE);
  const size_t smem = few_bytes(f.s.rows, f.local, VE);
  const cudaError_t e = gs::max_dynamic_smem((const void*)k_embedding_few<T, VE>, (int)few_bytes(kFewRows, kFewLocal, VE));
  if (e != cudaSuccess) return gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  gs::launch(k_embedding_few<T, VE>, dim3(f.s.blocks, (vectors + f.g - 1) / f.g), kFewThreads, smem, st, f);
  return gs::check_launch(where);
}

template <typename I>
gs_status launch_buckets(const char* where, const PartArgs& a, cudaStream_t st) {
  const cudaError_t e = gs::max_dynamic_smem((const void*)k_embedding_bucket_scatter<I>, (int)scatter_bytes(kMostBuckets));
  if (e != cudaSuccess) return gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  gs::launch(k_embedding_bucket_count<I>, dim3(a.tiles), kPartThreads, 0, st, a);
  gs::launch(k_embedding_bucket_scan, dim3((a.padded + 7) / 8), 1024, 0, st, a);
  gs::launch(k_embedding_bucket_scatter<I>, dim3(a.tiles + 1), kPartThreads, scatter_bytes(a.padded), st, a);
  return gs::check_launch(where);
}
template <typename T, int VE>
gs_status launch_parts(const char* where, const PartArgs& a, const Buckets& b, cudaStream_t st) {
  const int vectors = (a.s.width + VE - 1) / VE;
  const auto kernel = b.turns ? k_embedding_part<T, VE, true> : k_embedding_part<T, VE, false>;
  const cudaError_t e = gs::max_dynamic_smem((const void*)kernel, (int)part_bytes(kMostRows, kMostCodes, VE));
  if (e != cudaSuccess) return gs::set_error(GS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  // as many lanes to a walker as a row has vectors, or equal slabs of up to 32
  const int slabs = (vectors + 31) / 32, lanes = (vectors + slabs - 1) / slabs;
  gs::launch(kernel, dim3((unsigned)b.parts, (unsigned)slabs), kPartThreads, part_bytes(b.cap, b.codes, VE), st, a, lanes);
  if (b.many) {
    const int g = lanes_of(a.s.width, VE), walkers = kThreads / g, codes = std::min(walkers, b.codes);
    const int64_t runs = b.many * ((b.codes + codes - 1) / codes);
    gs::launch(k_embedding_part_join<T, VE>, dim3((unsigned)std::min<int64_t>(runs, 152 * 8), (unsigned)((vectors + g - 1) / g)), kThreads, 0,
               st, a, g);
  }
  return gs::check_launch(where);
}

template <typename T, int VE>
void launch_sums(SumArgs& a, cudaStream_t st) {
  const int g = lanes_of(a.width, VE), vectors = (a.width + VE - 1) / VE;
  a.per_walker = per_walker_of(a.rows, kThreads / g, VE);
  a.blocks = (unsigned)blocks_of(a.rows, g, VE);
  const unsigned slabs = (vectors + g - 1) / g;
  const unsigned zeros = (unsigned)((a.n + kWarps * 32 - 1) / (kWarps * 32));
  auto go = [&](auto sum, auto join) {
    gs::launch(sum, dim3(a.blocks, slabs), kThreads, 0, st, a);
    gs::launch(join, dim3(a.blocks + zeros, slabs), kThreads, 0, st, a);
  };
  if (g == 2) go(k_embedding_sum<T, VE, 2>, k_embedding_join<T, VE, 2>);
  else if (g == 4) go(k_embedding_sum<T, VE, 4>, k_embedding_join<T, VE, 4>);
  else if (g == 8) go(k_embedding_sum<T, VE, 8>, k_embedding_join<T, VE, 8>);
  else if (g == 16) go(k_embedding_sum<T, VE, 16>, k_embedding_join<T, VE, 16>);
  else go(k_embedding_sum<T, VE, 32>, k_embedding_join<T, VE, 32>);
}

}  // namespace

extern "C" gs_status gs_embedding_fwd(const gs_embedding_desc* d, const void* table, const void* idx, void* y, void* stream) {
  const char* where = "gs_embedding_fwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (d->rows == 0) return GS_OK;
  if (d->n > 0)
    if (gs_status s = gs::check_matrix(where, "table", table, d->n, d->width, d->ldt, d->dtype)) return s;
  if (gs_status s = gs::check_matrix(where, "y", y, d->rows, d->width, d->ldy, d->dtype)) return s;
  if (gs_status s = check_idx(where, d, idx)) return s;
  const int ve = vector_of(d, table, y);
  const int k = unit_of(ve * (int)gs::dtype_size(d->dtype));
  const int64_t per_row = (d->width + k * ve - 1) / (k * ve), units = d->rows * per_row;
  const bool large = k == 1 && d->rows * d->width * (int64_t)gs::dtype_size(d->dtype) >= kStreamBytes;
  const int64_t of_block = kThreads * 4;
  const int64_t blocks = (units + of_block - 1) / of_block;
  if (blocks > INT32_MAX) return gs::set_error(GS_ERR_INVALID, "%s: y is too large", where);
  const FwdArgs a{table, idx, y, d->rows, d->n, d->ldt, d->ldy, (uint32_t)per_row,
                  (uint32_t)(((uint64_t(1) << 32) + per_row - 1) / per_row), (uint32_t)d->width, d->scale};
  by_vector(d, ve, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int VE = decltype(v)::value;
    auto go = [&](auto kernel) { gs::launch(kernel, dim3((unsigned)blocks), kThreads, 0, gs::as_stream(stream), a); };
    if constexpr (VE * sizeof(T) == 16) {
      if (large) return d->index_bits == 32 ? go(k_embedding_fwd<T, VE, true, int32_t>) : go(k_embedding_fwd<T, VE, true, int64_t>);
    }
    d->index_bits == 32 ? go(k_embedding_fwd<T, VE, false, int32_t>) : go(k_embedding_fwd<T, VE, false, int64_t>);
  });
  return gs::check_launch(where);
}

extern "C" size_t gs_embedding_bwd_workspace_size(const gs_embedding_desc* d) {
  FewArgs f{};
  if (check_desc("gs_embedding_bwd_workspace_size", d) || d->rows == 0 || d->n == 0 || few_takes(d, f)) return 0;
  Buckets b{};
  return buckets_take(d, b) ? carve(nullptr, nullptr, d, b) : carve(nullptr, nullptr, d);
}

extern "C" gs_status gs_embedding_bwd(const gs_embedding_desc* d, const void* dy, const void* idx, void* dtable, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  const char* where = "gs_embedding_bwd";
  if (gs_status s = check_desc(where, d)) return s;
  if (d->n == 0) return GS_OK;
  if (gs_status s = gs::check_matrix(where, "dtable", dtable, d->n, d->width, d->ldt, d->dtype)) return s;
  cudaStream_t st = gs::as_stream(stream);
  const size_t size = gs::dtype_size(d->dtype);
  if (d->rows == 0) {
    const size_t ld = d->n > 1 ? d->ldt : d->width;
    if (cudaMemset2DAsync(dtable, ld * size, 0, d->width * size, d->n, st) != cudaSuccess) return gs::check_launch(where);
    return GS_OK;
  }
  if (gs_status s = gs::check_matrix(where, "dy", dy, d->rows, d->width, d->ldy, d->dtype)) return s;
  if (gs_status s = check_idx(where, d, idx)) return s;
  const int ve = vector_of(d, dtable, dy);
  FewArgs f{};
  f.s.dy = dy, f.s.idx = idx, f.s.dtable = dtable, f.s.rows = d->rows, f.s.n = d->n, f.s.ldy = d->ldy, f.s.ldt = d->ldt;
  f.s.width = d->width, f.s.scale = d->scale;
  if (few_takes(d, f)) {
    gs_status status = GS_OK;
    by_vector(d, ve, [&](auto t, auto v) { status = launch_few<decltype(t), decltype(v)::value>(where, f, st); });
    return status;
  }
  const size_t need = gs_embedding_bwd_workspace_size(d);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256)  // (a call of few rows needs none)
    return gs::set_error(GS_ERR_INVALID, "%s: workspace is NULL or misaligned", where);
  if (workspace_bytes < need)
    return gs::set_error(GS_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", where, workspace_bytes, need);
  Buckets b{};
  if (buckets_take(d, b)) {
    PartArgs a{};
    a.s = f.s;
    carve(&a, static_cast<char*>(workspace), d, b);
    if (gs_status s = d->index_bits == 32 ? launch_buckets<int32_t>(where, a, st) : launch_buckets<int64_t>(where, a, st))
      return s;
    gs_status status = GS_OK;
    by_vector(d, ve, [&](auto t, auto v) { status = launch_parts<decltype(t), decltype(v)::value>(where, a, b, st); });
    return status;
  }
  Space w;
  carve(&w, static_cast<char*>(workspace), d);
  const Plan p = plan_of(d);
  SortArgs a{idx, nullptr, nullptr, nullptr, nullptr, w.counts, w.totals, w.bitmap, d->rows, d->n, p.tiles, 0, 0};
  int from = 1;
  for (int i = 0; i < p.passes; ++i) {
    a.bits = (p.bits - a.shift + p.passes - i - 1) / (p.passes - i);
    a.keys = w.keys[from], a.rows_in = w.order[from];
    from ^= 1;
    a.keys_out = w.keys[from], a.rows_out = w.order[from];
    if (i > 0) launch_pass<char>(a, p.items, st);
    else if (d->index_bits == 32) launch_pass<int32_t>(a, p.items, st);
    else launch_pass<int64_t>(a, p.items, st);
    a.shift += a.bits;
  }
  if (gs_status s = gs::check_launch(where)) return s;
  SumArgs u = f.s;
  u.keys = w.keys[from], u.order = w.order[from], u.bitmap = w.bitmap, u.ends = w.ends, u.flags = w.flags;
  u.tail_code = w.tail_code, u.ldp = p.ldp;
  by_vector(d, ve, [&](auto t, auto v) { launch_sums<decltype(t), decltype(v)::value>(u, st); });
  return gs::check_launch(where);
}
