// Rows of a table by their indices, scaled (gs_embedding_fwd), and the table's gradient by sorted rows
// (gs_embedding_bwd).
//
// Mathematics: y[r] = scale table[idx[r]]; dtable[v] = scale sum over {r: idx[r] = v} of dy[r].
//
// Both are bound by memory.  The forward reads the indices and what it needs of the table, and writes y once: a thread
// holds one vector of a row, four of them in flight.
//
// The backward must not add in whatever order atomics come, and one code may have any number of rows, so the rows are
// first sorted by code: a radix sort of (code, row) pairs, stable, of up to eight bits a pass, each pass three kernels
// (digit counts of tiles, their scan by digit, a scatter through shared memory).  Then equal parts of the sorted rows go to
// groups of lanes ("walkers"), which add rows up in registers as long as the code stays the same.  A code whose rows lie
// inside one walker's part is written at once; the sums at a part's ends are joined in order, first among the walkers of a
// block in shared memory, then among blocks by a second kernel.  The part's length follows from the sizes alone, so the
// same call gives the same bits.  Codes without rows are found in a bitmap that the first pass fills and are set to zero by
// blocks of the summing kernel's launch.
#include <algorithm>

#include "dense.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------------ forward
struct FwdArgs {
  const void* table;
  const void* idx;
  void* y;
  int64_t rows, n, ldt, ldy;
  uint32_t per_row, magic;  // vectors of a row; 2^32 / per_row rounded up
  float scale;
};

template <typename T, int VE, typename I>
__global__ void __launch_bounds__(kThreads) k_embedding_fwd(const FwdArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int U = 4;
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
    // rows of more than 1024 vectors: at most one further row; else o per_row < 2^22 and the product is exact
    const uint32_t q = a.per_row > 1024 ? (o >= a.per_row) : a.per_row == 1 ? o : __umulhi(o, a.magic);
    row[u] = r0 + q, col[u] = o - q * a.per_row;
    const bool in = row[u] < a.rows;
    code[u] = in ? idx[row[u]] : (I)-1;
  }
  typename IO::Raw v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    v[u] = code[u] >= 0 && code[u] < a.n ? IO::load(table + (int64_t)code[u] * a.ldt + col[u] * VE) : IO::zero();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= a.rows) continue;
    float f[VE];
    IO::unpack(v[u], f);
    const bool there = code[u] >= 0 && code[u] < a.n;
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = there ? f[e] * a.scale : 0.f;
    IO::store(y + row[u] * a.ldy + col[u] * VE, f);
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
__global__ void __launch_bounds__(kThreads, 3) k_embedding_scatter(const SortArgs a) {
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
  uint32_t key[ITEMS], row[ITEMS];
  uint16_t rank[ITEMS];
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
    rank[i] = (uint16_t)(before + __popc(same & ((1u << lane) - 1)));
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
    const uint32_t d = (key[i] >> a.shift) & mask, at = s_start[d] + s_count[warp][d] + rank[i];
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

constexpr int kBatch = 8;  // rows in flight

// A walker's part [begin, end) of sorted rows, of `total` in all: codes inside it are written, the sums at its ends go to
// `head` and `tail` (the lane's own VE floats).  Returns the flags; `code` is the last one.  `none`: the key of rows without a
// code, behind all others; to_code: keys to codes; seen(code): the part has the code's first row.
// (Parts begin at multiples of kBatch; the arrays are padded to one: what lies behind the last row is not used.)
template <typename T, int VE, typename Code, typename Seen>
__device__ __forceinline__ uint32_t walk(const SumArgs& a, const uint32_t* keys, const uint32_t* order, int64_t begin, int64_t end,
                                         int64_t total, uint32_t none, int col, float* head, float* tail, uint32_t& code,
                                         Code to_code, Seen seen) {
  using IO = VecIO<T, VE>;
  const T* dy = static_cast<const T*>(a.dy);
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.f;
  uint32_t flag = 0;
  code = none;
  if (begin >= end) return 0;
  uint4 k4[2], o4[2];
  auto load = [&](int64_t p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      k4[h] = *reinterpret_cast<const uint4*>(keys + p + 4 * h);
      o4[h] = *reinterpret_cast<const uint4*>(order + p + 4 * h);
    }
  };
  load(begin);
  code = k4[0].x;
  bool from_before = begin > 0 && code != none && keys[begin - 1] == code;
  if (!from_before && code != none) seen(code);
  for (int64_t p = begin; p < end; p += kBatch) {
    uint32_t k[kBatch] = {k4[0].x, k4[0].y, k4[0].z, k4[0].w, k4[1].x, k4[1].y, k4[1].z, k4[1].w};
    const uint32_t o[kBatch] = {o4[0].x, o4[0].y, o4[0].z, o4[0].w, o4[1].x, o4[1].y, o4[1].z, o4[1].w};
    typename IO::Raw v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (p + u >= end) k[u] = none;
      v[u] = k[u] != none && col < a.width ? IO::load(dy + (int64_t)o[u] * a.ldy + col) : IO::zero();
    }
    if (p + kBatch < end) load(p + kBatch);  // in flight while these rows are added
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (p + u < end && k[u] != code) {  // the sum of `code` is complete here
        if (from_before) {
#pragma unroll
          for (int e = 0; e < VE; ++e) head[e] = acc[e];
          flag |= kHead;
          from_before = false;
        } else {
          write_sum<T, VE>(a, to_code(code), col, acc);
        }
        code = k[u];
        if (code != none) seen(code);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] = 0.f;
      }
      float f[VE];
      IO::unpack(v[u], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += f[e];
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
      write_sum<T, VE>(a, to_code(code), col, acc);
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

// G lanes to a walker, a vector each; gridDim.y slabs of columns.
template <typename T, int VE, int G>
__global__ void __launch_bounds__(kThreads, VE == 8 ? 2 : 3) k_embedding_sum(const SumArgs a) {
  follow();
  constexpr int kWalkers = kThreads / G;
  __shared__ float s_end[2][kThreads * VE];  // heads and tails
  __shared__ uint32_t s_flag[kWalkers], s_block;
  const int lane = threadIdx.x % G, walker = threadIdx.x / G;
  const int col = ((int)blockIdx.y * G + lane) * VE;
  const int64_t begin = ((int64_t)blockIdx.x * kWalkers + walker) * a.per_walker;
  const int64_t end = begin + a.per_walker < a.rows ? begin + a.per_walker : a.rows;
  float *head = s_end[0] + threadIdx.x * VE, *tail = s_end[1] + threadIdx.x * VE;
  uint32_t code, word = 0, bits = 0;  // codes seen, gathered to words of the bitmap
  const bool tells = lane == 0 && blockIdx.y == 0;
  const uint32_t flag = walk<T, VE>(
      a, a.keys, a.order, begin, end, a.rows, (uint32_t)a.n, col, head, tail, code, [](uint32_t c) { return c; },
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
  if (col >= a.width) return;
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
  const uint32_t flag = walk<T, VE>(a, key[from], row[from], begin, end, m, none, col, head, tail, code, to_code, [](uint32_t) {});
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
// Rows of a walker: whole batches, blocks for 8 times what the device holds (152 SMs, 3 blocks each), or for once where
// a walker would have few.
constexpr int64_t kBlocks = 152 * 3;
int per_walker_of(int64_t rows, int walkers) {
  int64_t want = (rows + kBlocks * walkers - 1) / (kBlocks * walkers);
  if (want > 64) want = std::max<int64_t>(64, want / 8);
  return (int)((want + kBatch - 1) / kBatch * kBatch);
}
int lanes_of(int width, int ve) {
  const int v = (width + ve - 1) / ve;
  return v <= 2 ? 2 : v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : 32;
}
int64_t blocks_of(int64_t rows, int g) {
  const int walkers = kThreads / g;
  const int64_t per = (int64_t)per_walker_of(rows, walkers) * walkers;
  return (rows + per - 1) / per;
}

struct Space {
  uint32_t *keys[2], *order[2], *counts, *totals, *bitmap, *flags, *tail_code;
  float* ends;
};
size_t carve(Space* s, char* base, const gs_embedding_desc* d) {
  const Plan p = plan_of(d);
  int64_t blocks = 0;  // the most that any vector leads to
  for (int ve : {1, 2, 4, 8}) blocks = std::max(blocks, blocks_of(d->rows, lanes_of(d->width, ve)));
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

template <typename T, int VE>
void launch_sums(SumArgs& a, cudaStream_t st) {
  const int g = lanes_of(a.width, VE), vectors = (a.width + VE - 1) / VE;
  a.per_walker = per_walker_of(a.rows, kThreads / g);
  a.blocks = (unsigned)blocks_of(a.rows, g);
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
  const int64_t per_row = d->width / ve, vectors = d->rows * per_row;
  const int64_t blocks = (vectors + kThreads * 4 - 1) / (kThreads * 4);
  if (blocks > INT32_MAX) return gs::set_error(GS_ERR_INVALID, "%s: y is too large", where);
  const FwdArgs a{table, idx, y, d->rows, d->n, d->ldt, d->ldy, (uint32_t)per_row,
                  (uint32_t)(((uint64_t(1) << 32) + per_row - 1) / per_row), d->scale};
  by_vector(d, ve, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int VE = decltype(v)::value;
    if (d->index_bits == 32) gs::launch(k_embedding_fwd<T, VE, int32_t>, dim3((unsigned)blocks), kThreads, 0, gs::as_stream(stream), a);
    else gs::launch(k_embedding_fwd<T, VE, int64_t>, dim3((unsigned)blocks), kThreads, 0, gs::as_stream(stream), a);
  });
  return gs::check_launch(where);
}

extern "C" size_t gs_embedding_bwd_workspace_size(const gs_embedding_desc* d) {
  FewArgs f{};
  if (check_desc("gs_embedding_bwd_workspace_size", d) || d->rows == 0 || d->n == 0 || few_takes(d, f)) return 0;
  return carve(nullptr, nullptr, d);
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
