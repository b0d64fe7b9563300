// Embedding of tokens (atom species, vocabulary entries) into feature rows,
// and the table's gradient by sorted tokens, for sm_100a.
//
//   out[k][:]        = scale * table[tok[k]][:]        (0 when tok[k] is no row)
//   grad_table[v][:] = scale * sum_{k: tok[k] = v} grad_out[k][:]
//
// Both move data and compute next to nothing: n x width values read and
// written (forward), read once with n_rows x width written (backward).
//
// The gradient sums rows in the order of a stable sort of the tokens, so every
// sum has one fixed order (no floating-point atomics): the sorted positions
// are cut into chunks of equal length, one worker (a group of lanes) walks one
// chunk and writes each run that lies inside it; a run that crosses chunk
// borders leaves one partial sum per chunk, joined by a second kernel.
// Equal chunks balance the work whatever the tokens' frequencies are: one row
// that takes every token and as many rows as tokens cost the same reads.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "train_ops.h"

namespace cgtp {
namespace {

// ------------------------------------------------------------------ sort
// Least-significant-digit radix sort of (key, position), 8 bits a pass, where
// the key of a token outside [0, n_rows) is n_rows (so those come last).
// Every warp ranks a stretch of consecutive tokens: lanes with equal digits find
// one another by a ballot per bit, in position order, which keeps the sort
// stable.
//
// Up to kBlockTokens tokens: one block, all passes in shared memory, one launch
// (7 680 tokens of 16 species: 8.0 us; the tiles take 5 us on the GPU in two launches, which
// such a small batch does not hide).  Beyond: tiles of kSortTile tokens.  The
// first launch counts each tile's digits; each pass is one more, in which every
// tile adds up the counts of the tiles before it (and of smaller digits)
// itself, places its tokens, and counts the next pass's digits as it does
// (integer atomics: the counts do not depend on their order).  Beyond
// kSortScanTiles tiles that sum over tiles, which every tile repeats, would
// grow with their square: one more launch a pass then turns the counts into
// prefixes first (400 000 tokens, 196 tiles, two passes: 22.9 us without, 23.2
// with; 600 000: 30.1, 27.3).  200 003 tokens of 50 021 rows take 20 us: count
// 3, two passes of 8, mostly latency from one launch to the next and in its
// chain of loads, ranks, prefix and scattered stores.
constexpr int kSortThreads = 512;
constexpr int kSortItems = 4;
constexpr int kSortTile = kSortThreads * kSortItems;  // tokens per tile
constexpr int kDigits = 256;
constexpr int kSortScanTiles = 200;
constexpr int kSortGroups = kSortThreads / (kDigits / 4);  // of threads that add up the tiles' counts
constexpr int kBlockThreads = 1024;
constexpr int kBlockItems = 8;
constexpr int kBlockTokens = kBlockThreads * kBlockItems;

__device__ __forceinline__ int token_key(int t, int n_rows) { return (unsigned)t < (unsigned)n_rows ? t : n_rows; }

// Bits of the digit at `shift` that the largest key, n_rows, can have.
__device__ __forceinline__ int digit_bits(int n_rows, int shift) { return min(8, 32 - __clz(n_rows >> shift)); }

// Ranks of a warp's ITEMS x 32 keys (key < 0: none) among its equal digits of
// `bits` bits, in position order; count [digit], zero before, receives the warp's counts.
template <int ITEMS>
__device__ __forceinline__ void rank_digits(const int (&key)[ITEMS], int shift, int bits, int* count,
                                            int (&rank)[ITEMS]) {
  const int lane = threadIdx.x & 31;
  unsigned same[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) same[i] = __ballot_sync(0xffffffffu, key[i] >= 0);
#pragma unroll 1
  for (int b = shift; b < shift + bits; ++b) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const bool set = (key[i] >> b) & 1;
      const unsigned m = __ballot_sync(0xffffffffu, set);
      same[i] &= set ? m : ~m;
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int d = (key[i] >> shift) & (kDigits - 1), lower = __popc(same[i] & ((1u << lane) - 1u));
    int seen = 0;
    if (key[i] >= 0) seen = count[d];
    __syncwarp();
    if (key[i] >= 0 && lower == 0) count[d] = seen + __popc(same[i]);
    __syncwarp();
    rank[i] = seen + lower;
  }
}
// Exclusive prefix of v over threads 0..255 (every thread of the block calls).
__device__ __forceinline__ int prefix_digits(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31 && w < kDigits / 32) warp_sums[w] = incl;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int q = 0; q < kDigits / 32; ++q)
    if (q < w) base += warp_sums[q];
  return base + incl - v;
}

template <int ITEMS>
__global__ void __launch_bounds__(kBlockThreads)
    sort_block_kernel(int n, int n_rows, int passes, const int* __restrict__ tokens, int* __restrict__ order,
                      int* __restrict__ sorted) {
  extern __shared__ int block_smem[];
  int* keys = block_smem;
  int* places = keys + kBlockThreads * ITEMS;
  int(*count)[kDigits] = (int(*)[kDigits])(places + kBlockThreads * ITEMS);  // [warp][digit]
  __shared__ int warp_sums[kDigits / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, base = w * 32 * ITEMS, warps = (n + 32 * ITEMS - 1) / (32 * ITEMS);
  int key[ITEMS], pos[ITEMS], rank[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    pos[i] = base + 32 * i + lane;
    key[i] = pos[i] < n ? token_key(tokens[pos[i]], n_rows) : -1;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = 8 * p;
    for (int d = lane; d < kDigits; d += 32) count[w][d] = 0;
    __syncwarp();
    rank_digits(key, shift, digit_bits(n_rows, shift), count[w], rank);
    __syncthreads();
    int total = 0;
    if (tid < kDigits)
#pragma unroll 8
      for (int q = 0; q < warps; ++q) total += count[q][tid];
    int run = prefix_digits(total, warp_sums);
    if (tid < kDigits)
#pragma unroll 8
      for (int q = 0; q < warps; ++q) {
        const int c = count[q][tid];
        count[q][tid] = run;
        run += c;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (key[i] >= 0) {
        const int to = count[w][(key[i] >> shift) & (kDigits - 1)] + rank[i];
        keys[to] = key[i];
        places[to] = pos[i];
      }
    __syncthreads();
    if (p + 1 < passes) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int k = base + 32 * i + lane;
        if (k < n) {
          key[i] = keys[k];
          pos[i] = places[k];
        }
      }
    }
  }
  for (int k = tid; k < n; k += kBlockThreads) {
    sorted[k] = keys[k];
    order[k] = places[k];
  }
}

// counts: [pass][tile][digit], the passes behind the first cleared here.
__global__ void __launch_bounds__(kSortThreads)
    sort_count_kernel(int n, int n_rows, int passes, long long per_pass, const int* __restrict__ tokens,
                      int* __restrict__ counts) {
  grid_dependents_launch();
  __shared__ int c[kDigits];
  if (threadIdx.x < kDigits) c[threadIdx.x] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * kSortTile;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const long long k = base + i * kSortThreads + threadIdx.x;
    if (k < n) atomicAdd(&c[token_key(tokens[k], n_rows) & (kDigits - 1)], 1);
  }
  __syncthreads();
  if (threadIdx.x < kDigits)
    for (int p = 0; p < passes; ++p)
      counts[p * per_pass + (long long)blockIdx.x * kDigits + threadIdx.x] = p == 0 ? c[threadIdx.x] : 0;
}

// One block per digit: the counts of its digit become the sums over earlier
// tiles, and their total goes behind the last tile's counts.
__global__ void __launch_bounds__(kSortThreads) sort_prefix_kernel(int tiles, int* __restrict__ counts) {
  grid_dependents_launch();
  grid_dependency_wait();
  __shared__ int warp_sums[kSortThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < tiles; b0 += kSortThreads) {
    int* c = counts + (long long)(b0 + tid) * kDigits + blockIdx.x;
    const int v = b0 + tid < tiles ? *c : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[w] = incl;
    __syncthreads();
    int base = carry;
    for (int q = 0; q < kSortThreads / 32; ++q) {
      if (q < w) base += warp_sums[q];
      carry += warp_sums[q];
    }
    if (b0 + tid < tiles) *c = base + incl - v;
    __syncthreads();
  }
  if (tid == 0) counts[(long long)tiles * kDigits + blockIdx.x] = carry;
}

// One pass over digit bits [shift, shift + 8).  keys_in = nullptr: the first
// pass, keys from the tokens and positions 0..n-1.  next_counts (nullable): the
// next pass's tile counts.
__global__ void __launch_bounds__(kSortThreads)
    sort_scatter_kernel(int n, int n_rows, int shift, const int* __restrict__ tokens, const int* __restrict__ keys_in,
                        const int* __restrict__ pos_in, const int* __restrict__ counts, int* __restrict__ keys_out,
                        int* __restrict__ pos_out, int* __restrict__ next_counts) {
  grid_dependents_launch();
  __shared__ int count[kSortThreads / 32][kDigits];
  __shared__ __align__(16) int part[kSortGroups][2][kDigits];  // [share of the tiles][before, all][digit]
  __shared__ int warp_sums[kDigits / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int d = lane; d < kDigits; d += 32) count[w][d] = 0;
  int key[kSortItems], pos[kSortItems], rank[kSortItems];
  const long long base = (long long)blockIdx.x * kSortTile + w * (32 * kSortItems);
  if (keys_in == nullptr) {  // the tokens, which no launch of this call writes: before the wait
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      pos[i] = (int)(base + 32 * i + lane);
      key[i] = base + 32 * i + lane < n ? token_key(tokens[base + 32 * i + lane], n_rows) : -1;
    }
    grid_dependency_wait();
  } else {
    grid_dependency_wait();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const long long k = base + 32 * i + lane;
      key[i] = k < n ? keys_in[k] : -1;
      pos[i] = k < n ? pos_in[k] : 0;
    }
  }
  // start of each digit of this tile: smaller digits of every tile, then the
  // same digit of earlier tiles; 64 threads of four digits each take every
  // kSortGroups-th tile
  const int d = tid & (kDigits - 1), tiles = gridDim.x;
  const bool scanned = tiles > kSortScanTiles;  // the counts are prefixes already
  if (!scanned) {
    const int group = tid / (kDigits / 4), quad = tid % (kDigits / 4);
    const int4* c = reinterpret_cast<const int4*>(counts) + quad;
    int4 before = make_int4(0, 0, 0, 0), all = before;
#pragma unroll 8
    for (int b = group; b < tiles; b += kSortGroups) {
      const int4 v = c[b * (kDigits / 4)];
      all = make_int4(all.x + v.x, all.y + v.y, all.z + v.z, all.w + v.w);
      if (b < (int)blockIdx.x) before = make_int4(before.x + v.x, before.y + v.y, before.z + v.z, before.w + v.w);
    }
    reinterpret_cast<int4*>(part[group][0])[quad] = before;
    reinterpret_cast<int4*>(part[group][1])[quad] = all;
  }
  __syncwarp();
  rank_digits(key, shift, digit_bits(n_rows, shift), count[w], rank);
  __syncthreads();
  int before = 0, all = 0;
  if (tid < kDigits) {
    if (scanned) {
      before = counts[(long long)blockIdx.x * kDigits + d];
      all = counts[(long long)tiles * kDigits + d];
    } else {
#pragma unroll
      for (int g = 0; g < kSortGroups; ++g) {
        before += part[g][0][d];
        all += part[g][1][d];
      }
    }
  }
  int run = prefix_digits(all, warp_sums);
  if (tid < kDigits) {  // the warps' counts become their starts
    run += before;
#pragma unroll
    for (int q = 0; q < kSortThreads / 32; ++q) {
      const int c = count[q][d];
      count[q][d] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    if (key[i] < 0) continue;
    const int to = count[w][(key[i] >> shift) & (kDigits - 1)] + rank[i];
    keys_out[to] = key[i];
    pos_out[to] = pos[i];
    if (next_counts != nullptr)
      atomicAdd(next_counts + (long long)(to / kSortTile) * kDigits + ((key[i] >> (shift + 8)) & (kDigits - 1)), 1);
  }
}

int sort_passes(int n_rows) {  // digits of the largest key, n_rows itself
  int p = 1;
  while (p < 4 && ((unsigned)n_rows >> (8 * p)) != 0) ++p;
  return p;
}
long long sort_tiles(int n) { return ((long long)n + kSortTile - 1) / kSortTile; }

// --------------------------------------------------------------- gradient
// A worker is a group of LPR lanes (a power of two) that covers LPR vectors
// of VEC columns of one row; a warp holds 32 / LPR workers.
template <int VEC>
struct Vec {
  float v[VEC];
};
template <int VEC>
__device__ __forceinline__ Vec<VEC> load_vec(const float* p) {
  Vec<VEC> r;
  if constexpr (VEC == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    r.v[0] = q.x;
    r.v[1] = q.y;
    r.v[2] = q.z;
    r.v[3] = q.w;
  } else {
    r.v[0] = *p;
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const Vec<VEC>& a) {
  if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
  else *p = a.v[0];
}

struct EmbedBwdArgs {
  int n, n_rows, width, chunk, n_chunks, lpr, slices;
  const int *order, *sorted;
  const float* grad_out;
  long long grad_stride;
  float scale;
  float* grad_table;
  float *head, *tail;  // [n_chunks][width] partial sums of runs that cross chunk borders
};

constexpr int kEmbedThreads = 256;
constexpr int kEmbedUnroll = 8;

// The first clear_blocks blocks write zeros into the rows that no token has,
// found by a search of the sorted tokens; in the others, one worker takes one
// (chunk, column slice).
// Eight rows at a time in registers: 46 us of 200 003 x 256, with the memory at 65 % and
// warps waiting for an index and then for its row.  Measured and not kept: indexes
// fetched a batch ahead (65 us in all, 53 so: fewer blocks fit), rows by asynchronous copies through
// shared memory (59 us).
template <int VEC>
__global__ void __launch_bounds__(kEmbedThreads, 4) embed_bwd_kernel(EmbedBwdArgs a, int clear_blocks) {
  grid_dependents_launch();
  const int lane = threadIdx.x & (a.lpr - 1);
  if ((int)blockIdx.x < clear_blocks) {
    const long long stride = (long long)clear_blocks * (kEmbedThreads / 32);
    const int wl = threadIdx.x & 31;
    for (long long r0 = ((long long)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5)) * 32; r0 < a.n_rows;
         r0 += stride * 32) {
      // each lane searches one of 32 rows, then the warp clears the empty ones together
      const int r = (int)(r0 + wl);
      bool empty = false;
      if (r0 + wl < a.n_rows) {
        int lo = 0, hi = a.n;  // first position with sorted >= r
        while (lo < hi) {
          const int mid = lo + (hi - lo) / 2;
          if (a.sorted[mid] < r) lo = mid + 1;
          else hi = mid;
        }
        empty = lo >= a.n || a.sorted[lo] != r;
      }
      const unsigned empties = __ballot_sync(0xffffffffu, empty);
      const Vec<VEC> z{};
      if (empties == 0xffffffffu) {  // 32 rows in one piece: few tokens for the table
        float* rows = a.grad_table + r0 * (long long)a.width;
#pragma unroll 4
        for (long long c = wl * VEC; c < 32LL * a.width; c += 32 * VEC) store_vec<VEC>(rows + c, z);
        continue;
      }
      for (unsigned m = empties; m != 0; m &= m - 1) {
        float* row = a.grad_table + (r0 + __ffs(m) - 1) * (long long)a.width;
        for (int c = wl * VEC; c < a.width; c += 32 * VEC) store_vec<VEC>(row + c, z);
      }
    }
    return;
  }
  const long long worker = ((long long)(blockIdx.x - clear_blocks) * kEmbedThreads + threadIdx.x) / a.lpr;
  const int chunk = (int)(worker / a.slices), slice = (int)(worker % a.slices);
  const int col = (slice * a.lpr + lane) * VEC;
  if (chunk >= a.n_chunks || col >= a.width) return;
  const int p0 = chunk * a.chunk, p1 = min(a.n - p0, a.chunk) + p0;
  int run = a.sorted[p0];
  bool from_before = p0 > 0 && a.sorted[p0 - 1] == run;
  Vec<VEC> acc{};
  auto finish = [&](int key) {  // the run ends inside the chunk
    if (from_before) {
      store_vec<VEC>(a.head + (long long)chunk * a.width + col, acc);
    } else if ((unsigned)key < (unsigned)a.n_rows) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc.v[j] *= a.scale;
      store_vec<VEC>(a.grad_table + (long long)key * a.width + col, acc);
    }
  };
  for (int p = p0; p < p1; p += kEmbedUnroll) {
    int key[kEmbedUnroll];
    Vec<VEC> g[kEmbedUnroll];
#pragma unroll
    for (int i = 0; i < kEmbedUnroll; ++i) {
      key[i] = -1;
      g[i] = Vec<VEC>{};
      if (p + i < p1) {
        key[i] = a.sorted[p + i];
        const int k = a.order[p + i];
        if ((unsigned)k < (unsigned)a.n && (unsigned)key[i] < (unsigned)a.n_rows)
          g[i] = load_vec<VEC>(a.grad_out + (long long)k * a.grad_stride + col);
      }
    }
#pragma unroll
    for (int i = 0; i < kEmbedUnroll; ++i) {
      if (p + i >= p1) break;
      if (key[i] != run) {
        finish(run);
        run = key[i];
        from_before = false;
        acc = Vec<VEC>{};
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc.v[j] += g[i].v[j];
    }
  }
  const bool goes_on = p1 < a.n && a.sorted[p1] == run;
  if (goes_on && !from_before) store_vec<VEC>(a.tail + (long long)chunk * a.width + col, acc);
  else finish(run);
}

// Joins the runs that cross chunk borders.  The first kJoinShort threads of a
// block are a worker per chunk, which adds up a run that starts there and ends
// within the next short_run chunks, all side by side; all of the block's workers take the
// longer ones together, one after the other, and their sums meet in shared memory in a
// fixed order.  Narrow rows have more chunks in a block, and so longer queues: 200 000
// tokens of 1 000 rows x 8 take 77 us with 4 chunks a worker, 33 with 16, 24 with 32;
// 7 680 tokens of 16 rows x 128 8.0 with 16, 12 with 32.
// The width alone says what counts as long and over how many stripes of its chunks a long run is
// summed: rows off a 16-byte boundary, whose workers have STRIPES = up to four times the lanes, take
// as many stripes a worker and join them first, so that alignments change no bit (200 003 tokens of
// 50 021 rows x 8 with an odd stride: 12 us, x 16: 15; with orders of their own 10 and 13).
constexpr int kJoinShort = 256, kJoinLong = 1024;
template <int VEC, int STRIPES>
__global__ void __launch_bounds__(kJoinLong) embed_join_kernel(EmbedBwdArgs a) {
  __shared__ Vec<VEC> part[kJoinLong];
  __shared__ int2 long_run[kJoinShort];  // by chunk of the block: the row of a long run, or -1, and its last chunk
  const int lane = threadIdx.x & (a.lpr - 1), worker = threadIdx.x / a.lpr, workers = blockDim.x / a.lpr;
  const int col = (blockIdx.y * a.lpr + lane) * VEC, chunks = kJoinShort / a.lpr;
  const bool on = col < a.width;
  const int short_run = a.lpr >= 8 * STRIPES ? 16 : 32;
  const int chunk0 = blockIdx.x * chunks, chunk = chunk0 + worker;
  auto add = [](Vec<VEC>& x, const Vec<VEC>& y) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x.v[j] += y.v[j];
  };
  auto finish = [&](int row, Vec<VEC> s) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) s.v[j] *= a.scale;
    store_vec<VEC>(a.grad_table + (long long)row * a.width + col, s);
  };
  // what there is to join, from the sorted tokens alone: before the wait for the partial sums
  int run = -1, is_long = -1, last = chunk;
  if (worker < chunks && chunk < a.n_chunks - 1) {
    const int p0 = chunk * a.chunk, p1 = p0 + a.chunk, key = a.sorted[p1 - 1];
    // the run goes on behind this chunk and starts in it
    if (a.sorted[p1] == key && (unsigned)key < (unsigned)a.n_rows && (p0 == 0 || a.sorted[p0 - 1] != key)) {
      const int far = chunk + 1 + short_run;
      if (far < a.n_chunks && a.sorted[far * a.chunk] == key) {
        is_long = key;
        int hi = a.n_chunks - 1;  // the last chunk that begins inside the run
        last = far;
        while (last < hi) {
          const int mid = last + (hi - last + 1) / 2;
          if (a.sorted[mid * a.chunk] == key) last = mid;
          else hi = mid - 1;
        }
      } else {
        run = key;
        for (int c = chunk + 1; c < far; ++c)  // chunks that begin inside the run
          if (c < a.n_chunks && a.sorted[c * a.chunk] == key) last = c;
      }
    }
  }
  grid_dependency_wait();
  if (run >= 0 && on) {
    Vec<VEC> s = load_vec<VEC>(a.tail + (long long)chunk * a.width + col);
#pragma unroll 8
    for (int c = chunk + 1; c <= last; ++c) add(s, load_vec<VEC>(a.head + (long long)c * a.width + col));
    finish(run, s);
  }
  if (lane == 0 && worker < chunks) long_run[worker] = make_int2(is_long, last);
  if (!__syncthreads_or(is_long >= 0)) return;
  for (int w = 0; w < chunks; ++w) {
    const int row = long_run[w].x, lo = long_run[w].y, first = chunk0 + w;
    if (row < 0) continue;  // the same for every thread
    Vec<VEC> s[STRIPES] = {};
    if (on) {
      if (worker == 0) s[0] = load_vec<VEC>(a.tail + (long long)first * a.width + col);
#pragma unroll 4
      for (int c = first + 1 + worker; c <= lo; c += STRIPES * workers)
#pragma unroll
        for (int i = 0; i < STRIPES; ++i)
          if (i == 0 || c + i * workers <= lo)
            add(s[i], load_vec<VEC>(a.head + (long long)(c + i * workers) * a.width + col));
#pragma unroll
      for (int o = STRIPES >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) add(s[i], s[i + o]);
    }
    part[threadIdx.x] = s[0];
    __syncthreads();
    for (int o = workers >> 1; o > 0; o >>= 1) {
      if (worker < o) add(part[threadIdx.x], part[threadIdx.x + o * a.lpr]);
      __syncthreads();
    }
    if (worker == 0 && on) finish(row, part[threadIdx.x]);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- forward
constexpr int kFwdRows = 4;  // rows per worker: four independent row reads in flight a lane

template <int VEC>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_fwd_kernel(int n, int n_rows, int width, int lpr, int slices, const int* __restrict__ tokens,
                     const float* __restrict__ table, float scale, float* __restrict__ out, long long out_stride) {
  const int lane = threadIdx.x & (lpr - 1);
  const long long worker = ((long long)blockIdx.x * kEmbedThreads + threadIdx.x) / lpr;
  const long long k0 = worker / slices * kFwdRows;
  const int col = ((int)(worker % slices) * lpr + lane) * VEC;
  if (col >= width) return;
  Vec<VEC> v[kFwdRows];
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    v[i] = Vec<VEC>{};
    if (k0 + i < n) {
      const int t = tokens[k0 + i];
      if ((unsigned)t < (unsigned)n_rows) v[i] = load_vec<VEC>(table + (long long)t * width + col);
    }
  }
#pragma unroll
  for (int i = 0; i < kFwdRows; ++i) {
    if (k0 + i < n) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i].v[j] *= scale;
      store_vec<VEC>(out + (k0 + i) * out_stride + col, v[i]);
    }
  }
}

bool vec4_rows(const void* p, long long stride, int width) {
  return width % 4 == 0 && stride % 4 == 0 && ((uintptr_t)p & 15u) == 0;
}
int lanes_per_row(int width, int vec) {
  const int need = (width + vec - 1) / vec;
  int l = 1;
  while (l < 32 && l < need) l <<= 1;
  return l;
}
// Lanes of a row on a 16-byte boundary, by the width alone.
int order_lanes(int width) { return lanes_per_row(width, width % 4 == 0 ? 4 : 1); }

// Sorted positions per chunk, a function of the sizes alone (the sums' order
// does not depend on the device or on alignments).  Of the four blocks that an
// SM holds, three are for chunks and one for the clearing, so that no block
// starts late and runs alone at the end (200 003 x 256 of 50 021 rows: 417 + 148
// blocks 48 us, with 417 + 196 5 us more; x 128: 391 + 196 blocks 3 us less than
// 521 + 196).  At least 16 positions, so that the partial sums stay a small part of the
// reads.
int embed_chunk(int n, int width) {
  const int vec = width % 4 == 0 ? 4 : 1, lpr = order_lanes(width);
  const long long slices = (width + lpr * vec - 1) / (lpr * vec), workers = 148LL * 3 * kEmbedThreads / lpr;
  const long long c = ((n * slices + workers - 1) / workers + 7) / 8 * 8;
  return c < 16 ? 16 : c > 256 ? 256 : (int)c;
}

}  // namespace

size_t token_sort_workspace(int n, int n_rows) {
  if (n <= kBlockTokens) return 0;
  const int p = sort_passes(n_rows);
  const size_t counts = sizeof(int) * (size_t)(sort_tiles(n) + 1) * kDigits;
  return (size_t)p * counts + (p > 1 ? 2 * pad256(sizeof(int) * (size_t)n) : 0);
}

template <int ITEMS>
static cudaError_t sort_block(int n, int n_rows, int passes, const int* tokens, int* order, int* sorted,
                              cudaStream_t stream) {
  constexpr int bytes = sizeof(int) * (2 * kBlockThreads * ITEMS + kBlockThreads / 32 * kDigits);
  if (bytes > 48 * 1024) {  // more than a block gets unasked
    const cudaError_t e =
        cudaFuncSetAttribute(sort_block_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  sort_block_kernel<ITEMS><<<1, kBlockThreads, bytes, stream>>>(n, n_rows, passes, tokens, order, sorted);
  return cudaGetLastError();
}

cudaError_t launch_token_sort(int n, int n_rows, const int* tokens, int* order, int* sorted, void* ws,
                              cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const int passes = sort_passes(n_rows);
  if (n <= kBlockTokens) {
    // as few positions a thread as hold the tokens
    if (n <= kBlockThreads) return sort_block<1>(n, n_rows, passes, tokens, order, sorted, stream);
    if (n <= 4 * kBlockThreads) return sort_block<4>(n, n_rows, passes, tokens, order, sorted, stream);
    return sort_block<kBlockItems>(n, n_rows, passes, tokens, order, sorted, stream);
  }
  const unsigned tiles = (unsigned)sort_tiles(n);
  const long long per_pass = ((long long)tiles + 1) * kDigits;
  int* counts = (int*)ws;
  int* tmp_keys = (int*)((char*)ws + sizeof(int) * (size_t)passes * per_pass);
  int* tmp_pos = (int*)((char*)tmp_keys + pad256(sizeof(int) * (size_t)n));
  sort_count_kernel<<<tiles, kSortThreads, 0, stream>>>(n, n_rows, passes, per_pass, tokens, counts);
  cudaError_t e = cudaGetLastError();
  const int *keys = nullptr, *pos = nullptr;
  for (int p = 0; p < passes && e == cudaSuccess; ++p) {
    // the last pass writes the results; the passes before it alternate with the temporaries
    const bool to_out = (passes - 1 - p) % 2 == 0;
    int* ko = to_out ? sorted : tmp_keys;
    int* po = to_out ? order : tmp_pos;
    int* here = counts + p * per_pass;
    if (tiles > kSortScanTiles)
      e = launch_kernel(sort_prefix_kernel, dim3(kDigits), dim3(kSortThreads), 0, stream, true, (int)tiles, here);
    if (e == cudaSuccess)
      e = launch_kernel(sort_scatter_kernel, dim3(tiles), dim3(kSortThreads), 0, stream, true, n, n_rows, 8 * p, tokens,
                        keys, pos, (const int*)here, ko, po, p + 1 < passes ? here + per_pass : (int*)nullptr);
    keys = ko;
    pos = po;
  }
  return e;
}

cudaError_t launch_embed_fwd(int n, int n_rows, int width, const int* tokens, const float* table, float scale,
                             float* out, long long out_stride, cudaStream_t stream) {
  if (n == 0 || width == 0) return cudaSuccess;
  const bool v4 = vec4_rows(table, width, width) && vec4_rows(out, out_stride, width);
  const int vec = v4 ? 4 : 1, lpr = lanes_per_row(width, vec), slices = (width + lpr * vec - 1) / (lpr * vec);
  const long long threads = ((long long)n + kFwdRows - 1) / kFwdRows * slices * lpr;
  const long long blocks = (threads + kEmbedThreads - 1) / kEmbedThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (v4)
    embed_fwd_kernel<4><<<(unsigned)blocks, kEmbedThreads, 0, stream>>>(n, n_rows, width, lpr, slices, tokens, table,
                                                                        scale, out, out_stride);
  else
    embed_fwd_kernel<1><<<(unsigned)blocks, kEmbedThreads, 0, stream>>>(n, n_rows, width, lpr, slices, tokens, table,
                                                                        scale, out, out_stride);
  return cudaGetLastError();
}

size_t embed_bwd_workspace(int n, int width) {
  const size_t chunks = ((size_t)n + embed_chunk(n, width) - 1) / embed_chunk(n, width);
  return 2 * pad256(sizeof(float) * chunks * (size_t)width);
}

template <int VEC>
static cudaError_t embed_bwd(EmbedBwdArgs a, cudaStream_t stream) {
  a.lpr = lanes_per_row(a.width, VEC);
  a.slices = (a.width + a.lpr * VEC - 1) / (a.lpr * VEC);
  const long long blocks = ((long long)a.n_chunks * a.slices * a.lpr + kEmbedThreads - 1) / kEmbedThreads;
  // a block searches kEmbedThreads rows at a time; one an SM while that takes each at most twice
  long long clear = ((long long)a.n_rows + kEmbedThreads - 1) / kEmbedThreads;
  if (clear > 148) clear = clear <= 2 * 148 ? 148 : clear > 1024 ? 1024 : clear;
  if (blocks + clear > 0x7fffffffLL || a.slices > 65535) return cudaErrorInvalidValue;
  embed_bwd_kernel<VEC><<<(unsigned)(blocks + clear), kEmbedThreads, 0, stream>>>(a, (int)clear);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.n_chunks < 2) return e;
  // large blocks where the average row crosses more than 128 chunks (200 000 tokens of one row x 128: 54 us with
  // blocks of 256 threads, 33 us with 1 024; of 16 rows x 64: 20, 17; 100 000 of 50 rows x 16, 125 chunks each: 12, 15)
  const int chunks = kJoinShort / a.lpr;
  const bool long_runs = a.n / a.n_rows > 128 * a.chunk;
  const int stripes = a.lpr / order_lanes(a.width);
  const auto join = VEC == 4 || stripes == 1 ? embed_join_kernel<VEC, 1>
                    : stripes == 2           ? embed_join_kernel<1, 2>
                                             : embed_join_kernel<1, 4>;
  return launch_kernel(join, dim3((unsigned)((a.n_chunks - 2) / chunks + 1), (unsigned)a.slices),
                       dim3(long_runs ? kJoinLong : kJoinShort), 0, stream, true, a);
}

cudaError_t launch_embed_bwd(int n, int n_rows, int width, const int* order, const int* sorted, const float* grad_out,
                             long long grad_stride, float scale, float* grad_table, void* ws, cudaStream_t stream) {
  if (n_rows == 0 || width == 0) return cudaSuccess;
  if (n == 0) return cudaMemsetAsync(grad_table, 0, sizeof(float) * (size_t)n_rows * width, stream);
  EmbedBwdArgs a{};
  a.n = n;
  a.n_rows = n_rows;
  a.width = width;
  a.chunk = embed_chunk(n, width);
  a.n_chunks = (int)(((long long)n + a.chunk - 1) / a.chunk);
  a.order = order;
  a.sorted = sorted;
  a.grad_out = grad_out;
  a.grad_stride = grad_stride;
  a.scale = scale;
  a.grad_table = grad_table;
  a.head = (float*)ws;
  a.tail = (float*)((char*)ws + pad256(sizeof(float) * (size_t)a.n_chunks * width));
  if (vec4_rows(grad_out, grad_stride, width) && vec4_rows(grad_table, width, width)) return embed_bwd<4>(a, stream);
  return embed_bwd<1>(a, stream);
}

}  // namespace cgtp
