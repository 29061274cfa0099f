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
constexpr int kItems = 16;
constexpr int kTile = kThreads * kItems;  // pairs of a block

struct SortArgs {
  const void* idx;           // first pass
  const uint32_t* keys;      // later ones
  const uint32_t* rows_in;
  uint32_t* keys_out;
  uint32_t* rows_out;
  uint32_t* counts;          // [digits][tiles]
  uint32_t* totals;          // [256]
  uint32_t* bitmap;          // codes that have rows (first pass)
  int64_t rows, n;
  int tiles, shift, bits;
};

// The lanes of the warp with the same digit.
__device__ __forceinline__ uint32_t peers_of(uint32_t digit, int bits, uint32_t among) {
  uint32_t same = among;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(0xffffffffu, (digit >> b) & 1u);
    same &= (digit >> b) & 1u ? set : ~set;
  }
  return same;
}

// What does not name a code is the code n, behind all others.
template <typename I>
__device__ __forceinline__ uint32_t code_of(const void* idx, int64_t r, int64_t n) {
  const I v = static_cast<const I*>(idx)[r];
  return v >= 0 && v < n ? (uint32_t)v : (uint32_t)n;
}
// I: the first pass reads indices of this type; void: a later pass
template <typename I>
__device__ __forceinline__ uint32_t key_at(const SortArgs& a, int64_t r) {
  if constexpr (sizeof(I) == 1) return a.keys[r];
  else return code_of<I>(a.idx, r, a.n);
}

template <typename I>
__global__ void __launch_bounds__(kThreads) k_embedding_count(const SortArgs a) {
  follow();
  __shared__ uint32_t s[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kWarps * 256; i += kThreads) s[i / 256][i % 256] = 0;
  __syncthreads();
  const uint32_t mask = (1u << a.bits) - 1;
  const int64_t base = (int64_t)blockIdx.x * kTile + warp * (32 * kItems) + lane;
  uint32_t key[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) key[i] = base + i * 32 < a.rows ? key_at<I>(a, base + i * 32) : 0u;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const bool in = base + i * 32 < a.rows;
    const uint32_t among = __ballot_sync(0xffffffffu, in), d = (key[i] >> a.shift) & mask;
    const uint32_t same = peers_of(d, a.bits, among);
    if (in && lane == __ffs(same) - 1) s[warp][d] += __popc(same);
    if constexpr (sizeof(I) != 1) {
      if (in && key[i] < a.n) {
        const uint32_t bit = 1u << (key[i] & 31);
        uint32_t* word = a.bitmap + (key[i] >> 5);
        if (!(*reinterpret_cast<volatile uint32_t*>(word) & bit)) atomicOr(word, bit);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (threadIdx.x <= mask) {
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s[w][threadIdx.x];
    a.counts[(int64_t)threadIdx.x * a.tiles + blockIdx.x] = t;
  }
}

// exclusive sum over the block's threads; `total` of all of them
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t& total) {
  __shared__ uint32_t sums[kWarps];
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
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? sums[w] : 0u;
    total += sums[w];
  }
  return before + x - v;
}

// A block for each digit: the exclusive sums of its counts over the tiles.
__global__ void __launch_bounds__(kThreads) k_embedding_scan(const SortArgs a) {
  follow();
  uint32_t* c = a.counts + (int64_t)blockIdx.x * a.tiles;
  uint32_t run = 0;
  for (int t0 = 0; t0 < a.tiles; t0 += kThreads) {
    const int t = t0 + threadIdx.x;
    const uint32_t v = t < a.tiles ? c[t] : 0u;
    uint32_t total;
    const uint32_t before = block_scan(v, total);
    if (t < a.tiles) c[t] = run + before;
    run += total;
  }
  if (threadIdx.x == 0) a.totals[blockIdx.x] = run;
}

template <typename I>
__global__ void __launch_bounds__(kThreads) k_embedding_scatter(const SortArgs a) {
  follow();
  __shared__ uint32_t s_count[kWarps][256];  // of each warp's digits; then where its first of them goes in the tile
  __shared__ uint32_t s_start[256];          // where a digit's run begins in the tile
  __shared__ uint32_t s_out[256];            // and in the output, less s_start
  __shared__ uint32_t s_key[kTile], s_row[kTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int i = threadIdx.x; i < kWarps * 256; i += kThreads) s_count[i / 256][i % 256] = 0;
  const int64_t base = (int64_t)blockIdx.x * kTile + warp * (32 * kItems) + lane;
  uint32_t key[kItems], row[kItems], rank[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int64_t r = base + i * 32;
    key[i] = r < a.rows ? key_at<I>(a, r) : 0u;
    if constexpr (sizeof(I) == 1) row[i] = r < a.rows ? a.rows_in[r] : 0u;
    else row[i] = (uint32_t)r;
  }
  uint32_t total_of_digit = threadIdx.x <= mask ? a.totals[threadIdx.x] : 0u;
  const uint32_t here = threadIdx.x <= mask ? a.counts[(int64_t)threadIdx.x * a.tiles + blockIdx.x] : 0u;
  uint32_t total;
  const uint32_t digit_base = block_scan(total_of_digit, total);  // (its barriers also end the clearing above)
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const bool in = base + i * 32 < a.rows;
    const uint32_t among = __ballot_sync(0xffffffffu, in), d = (key[i] >> a.shift) & mask;
    const uint32_t same = peers_of(d, a.bits, among);
    const uint32_t before = s_count[warp][d];
    rank[i] = before + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) s_count[warp][d] = before + __popc(same);
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
  const uint32_t start = block_scan(sum, total);
  if (threadIdx.x <= mask) {
    s_start[threadIdx.x] = start;
    s_out[threadIdx.x] = digit_base + here - start;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
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
  const uint32_t* keys;     // sorted
  const uint32_t* order;    // and the rows
  const uint32_t* bitmap;
  void* dtable;
  float* ends;              // [blocks][2][ldp]: sums that go on from the block before, into the block after
  uint32_t* flags;          // [blocks]: kHead, kThrough, kTail
  uint32_t* tail_code;      // [blocks]
  int64_t rows, n, ldy, ldt, ldp;
  int per_walker, width;
  unsigned blocks;          // that add; the others write zeros
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

// G lanes to a walker, a vector each; gridDim.y slabs of columns.
template <typename T, int VE, int G>
__global__ void __launch_bounds__(kThreads) k_embedding_sum(const SumArgs a) {
  follow();
  using IO = VecIO<T, VE>;
  constexpr int kWalkers = kThreads / G, kBatch = 8;
  if (blockIdx.x >= a.blocks) {
    const int lane = threadIdx.x & 31;
    const int64_t word = (int64_t)(blockIdx.x - a.blocks) * kWarps + (threadIdx.x >> 5);
    if (word * 32 >= a.n) return;
    uint32_t empty = ~a.bitmap[word];
    if (a.n - word * 32 < 32) empty &= (1u << (a.n - word * 32)) - 1;
    constexpr int kSide = 32 / G;  // rows side by side
    const int col = ((int)blockIdx.y * G + lane % G) * VE;
    const float none[VE] = {};
#pragma unroll 4
    for (int r = lane / G; r < 32; r += kSide)
      if ((empty >> r) & 1u && col < a.width)
        IO::store(static_cast<T*>(a.dtable) + (word * 32 + r) * a.ldt + col, none);
    return;
  }
  __shared__ float s_end[2][kThreads * VE];  // heads and tails
  __shared__ uint32_t s_flag[kWalkers], s_block;
  const int lane = threadIdx.x % G, walker = threadIdx.x / G;
  const int col = ((int)blockIdx.y * G + lane) * VE;
  const T* dy = static_cast<const T*>(a.dy);
  const int64_t begin = ((int64_t)blockIdx.x * kWalkers + walker) * a.per_walker;
  const int64_t end = begin + a.per_walker < a.rows ? begin + a.per_walker : a.rows;
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.f;
  uint32_t flag = 0, code = (uint32_t)a.n;
  if (begin < end) {
    code = a.keys[begin];
    bool from_before = begin > 0 && code != (uint32_t)a.n && a.keys[begin - 1] == code;
    for (int64_t p = begin; p < end; p += kBatch) {
      uint32_t k[kBatch];
      typename IO::Raw v[kBatch];
      // (parts are whole batches and the arrays are padded to one: what lies behind the last row is not used)
      const uint4 k0 = *reinterpret_cast<const uint4*>(a.keys + p), k1 = *reinterpret_cast<const uint4*>(a.keys + p + 4);
      const uint4 o0 = *reinterpret_cast<const uint4*>(a.order + p), o1 = *reinterpret_cast<const uint4*>(a.order + p + 4);
      k[0] = k0.x, k[1] = k0.y, k[2] = k0.z, k[3] = k0.w, k[4] = k1.x, k[5] = k1.y, k[6] = k1.z, k[7] = k1.w;
      const uint32_t o[kBatch] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (p + u >= end) k[u] = (uint32_t)a.n;
        v[u] = k[u] != (uint32_t)a.n && col < a.width ? IO::load(dy + (int64_t)o[u] * a.ldy + col) : IO::zero();
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (p + u < end && k[u] != code) {  // the sum of `code` is complete here
          if (from_before) {
#pragma unroll
            for (int e = 0; e < VE; ++e) s_end[0][threadIdx.x * VE + e] = acc[e];
            flag |= kHead;
            from_before = false;
          } else {
            write_sum<T, VE>(a, code, col, acc);
          }
          code = k[u];
#pragma unroll
          for (int e = 0; e < VE; ++e) acc[e] = 0.f;
        }
        float f[VE];
        IO::unpack(v[u], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += f[e];
      }
    }
    if (code != (uint32_t)a.n) {
      const bool goes_on = end < a.rows && a.keys[end] == code;
      if (from_before || goes_on) {
#pragma unroll
        for (int e = 0; e < VE; ++e) s_end[from_before ? 0 : 1][threadIdx.x * VE + e] = acc[e];
        flag |= from_before ? (goes_on ? kHead | kThrough : kHead) : kTail;
      } else {
        write_sum<T, VE>(a, code, col, acc);
      }
    }
  }
  if (lane == 0) s_flag[walker] = flag;
  if (threadIdx.x == 0) s_block = 0;
  __syncthreads();
  // A tail is joined by the heads behind it.  (A lane reads its own columns only.)
  if (flag & kTail) {
    bool open = true;
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = s_end[1][threadIdx.x * VE + e];
    for (int w = walker + 1; w < kWalkers && open; ++w) {
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += s_end[0][(w * G + lane) * VE + e];
      open = s_flag[w] & kThrough;
    }
    if (open) {
      float* to = a.ends + ((int64_t)blockIdx.x * 2 + 1) * a.ldp + col;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (col + e < a.width) to[e] = acc[e];
      if (lane == 0) {
        a.tail_code[blockIdx.x] = code;
        atomicOr(&s_block, kTail);
      }
    } else {
      write_sum<T, VE>(a, code, col, acc);
    }
  }
  if (walker == 0 && flag & kHead) {
    bool open = flag & kThrough;
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = s_end[0][threadIdx.x * VE + e];
    for (int w = 1; w < kWalkers && open; ++w) {
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += s_end[0][(w * G + lane) * VE + e];
      open = s_flag[w] & kThrough;
    }
    float* to = a.ends + (int64_t)blockIdx.x * 2 * a.ldp + col;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (col + e < a.width) to[e] = acc[e];
    if (lane == 0) atomicOr(&s_block, open ? kHead | kThrough : kHead);
  }
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = s_block;
}

// A block for each block of the sums: its tail and the heads behind it, every kWalkers-th to a walker.
template <typename T, int VE, int G>
__global__ void __launch_bounds__(kThreads) k_embedding_join(const SumArgs a) {
  follow();
  if (!(a.flags[blockIdx.x] & kTail)) return;
  constexpr int kWalkers = kThreads / G;
  __shared__ float s[kThreads * VE];
  const int lane = threadIdx.x % G, walker = threadIdx.x / G;
  const int col = ((int)blockIdx.y * G + lane) * VE;
  unsigned last = blockIdx.x + 1;  // the first block that the code does not go through
  for (;; last += kThreads) {
    const unsigned b = last + threadIdx.x;
    __shared__ unsigned s_first;
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
  for (int w = 1; w < kWalkers; ++w) {
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] += s[(w * G + lane) * VE + e];
  }
  write_sum<T, VE>(a, a.tail_code[blockIdx.x], col, acc);
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
  int bits, passes, tiles;
  int64_t padded;  // rows, to whole batches
  int64_t words;   // of the bitmap
  int64_t ldp;
};
Plan plan_of(const gs_embedding_desc* d) {
  Plan p{};
  while (p.bits < 32 && (d->n >> p.bits)) ++p.bits;  // of the codes 0..n
  if (p.bits < 1) p.bits = 1;
  p.passes = (p.bits + 7) / 8;
  p.tiles = (int)((d->rows + kTile - 1) / kTile);
  p.padded = (d->rows + 7) / 8 * 8;
  p.words = (d->n + 31) / 32;
  p.ldp = (d->width + 7) / 8 * 8;
  return p;
}
// Rows of a walker: whole batches, enough blocks to fill the device twice over (152 SMs, 8 blocks each).
constexpr int64_t kBlocks = 2 * 152 * 8;
int per_walker_of(int64_t rows, int walkers) {
  const int64_t want = (rows + kBlocks * walkers - 1) / (kBlocks * walkers);
  return (int)((want + 7) / 8 * 8);
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
void launch_pass(const SortArgs& a, cudaStream_t st) {
  gs::launch(k_embedding_count<I>, dim3(a.tiles), kThreads, 0, st, a);
  gs::launch(k_embedding_scan, dim3(1u << a.bits), kThreads, 0, st, a);
  gs::launch(k_embedding_scatter<I>, dim3(a.tiles), kThreads, 0, st, a);
}

template <typename T, int VE>
void launch_sums(SumArgs& a, cudaStream_t st) {
  const int g = lanes_of(a.width, VE), vectors = (a.width + VE - 1) / VE;
  a.per_walker = per_walker_of(a.rows, kThreads / g);
  a.blocks = (unsigned)blocks_of(a.rows, g);
  const unsigned slabs = (vectors + g - 1) / g;
  const unsigned zeros = (unsigned)((a.n + kWarps * 32 - 1) / (kWarps * 32));
  auto go = [&](auto sum, auto join) {
    gs::launch(sum, dim3(a.blocks + zeros, slabs), kThreads, 0, st, a);
    if (a.blocks > 1) gs::launch(join, dim3(a.blocks, slabs), kThreads, 0, st, a);
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
  if (check_desc("gs_embedding_bwd_workspace_size", d) || d->rows == 0 || d->n == 0) return 0;
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
  const size_t need = gs_embedding_bwd_workspace_size(d);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256)
    return gs::set_error(GS_ERR_INVALID, "%s: workspace is NULL or misaligned", where);
  if (workspace_bytes < need)
    return gs::set_error(GS_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", where, workspace_bytes, need);
  Space w;
  carve(&w, static_cast<char*>(workspace), d);
  const Plan p = plan_of(d);
  if (cudaMemsetAsync(w.bitmap, 0, 4 * p.words, st) != cudaSuccess) return gs::check_launch(where);
  SortArgs a{idx, nullptr, nullptr, nullptr, nullptr, w.counts, w.totals, w.bitmap, d->rows, d->n, p.tiles, 0, 0};
  int from = 1;
  for (int i = 0; i < p.passes; ++i) {
    a.bits = (p.bits - a.shift + p.passes - i - 1) / (p.passes - i);
    a.keys = w.keys[from], a.rows_in = w.order[from];
    from ^= 1;
    a.keys_out = w.keys[from], a.rows_out = w.order[from];
    if (i > 0) launch_pass<char>(a, st);
    else if (d->index_bits == 32) launch_pass<int32_t>(a, st);
    else launch_pass<int64_t>(a, st);
    a.shift += a.bits;
  }
  if (gs_status s = gs::check_launch(where)) return s;
  SumArgs u{dy, w.keys[from], w.order[from], w.bitmap, dtable, w.ends, w.flags, w.tail_code, d->rows, d->n, d->ldy, d->ldt, p.ldp,
            0, d->width, 0, d->scale};
  by_vector(d, vector_of(d, dtable, dy), [&](auto t, auto v) { launch_sums<decltype(t), decltype(v)::value>(u, st); });
  return gs::check_launch(where);
}
