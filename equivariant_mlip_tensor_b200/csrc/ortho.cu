// Orthogonalisation of a stack of matrices by Newton-Schulz products, for
// sm_100a (as the Muon optimiser applies to an update before it is taken).
//
//   X <- G / (|G|_F + 1e-7), transposed if it has more rows than columns
//   steps times:  A = X X^T,  X <- a X + (b A + c A A) X,   (a, b, c) = (3.4445, -4.7750, 2.0315)
//   out = scale X (transposed back)
//
// On the singular values each step is the polynomial a s + b s^3 + c s^5,
// which lifts small values by a and keeps every value in [0, 1.21]: it stays
// bounded for any number of steps.
//
// All but the smallest matrices (which sum in fp32) have their products on the
// tensor cores in fp16 pairs: x 2^k = high + low holds 22
// bits of x, and low high + high low + high high, summed in fp32, leaves out
// only low low (2^-22 of a product and less), so three fp16 products give a
// product of fp32 accuracy.  That the values stay bounded makes fixed powers
// of two fit: entries of X and of X X^T are at most 1.21 and 1.45 (x 2^14 <
// 65504), those of a + b A + c A A at most 3.45 (x 2^13).  Norms and sums stay
// in fp32 and above; a X is taken into the last product by adding a to the diagonal of
// b A + c A A.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tc.cuh"
#include "train_ops.h"

namespace cgtp {
namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr double kNsEps = 1e-7;

// ---------------------------------------------------------- the short side up to 128
// All steps of one matrix in one launch: a cluster of 1, 2, 4 or 8 blocks holds
// X, each its own columns, as fp16 pairs in shared memory from the first step
// to the last; A and then b A + c A A (at most 128 x 128) are in every block.
// The same tile of X is read along its rows for X X^T and down its rows for
// the last product.  Between the products the fp32 values of A and X stay in tensor
// memory beside the accumulators, each thread its own, so that only operands
// are converted.  With more than one block, each sends its part of
// X X^T to the blocks that own the entries, which sum them in a fixed order and
// send A to all: stores that count their bytes on the receiver's mbarrier, so a
// block waits for its data alone (barriers of the whole cluster around loads from
// the other blocks took 4 us a step at 64 x 1920).
//
// The diagonals of A and of P = b A + c A A stay out of the operands and are
// applied in fp32: with A = D + R, A A = D D + D R + R D + R R, and P X likewise.
// A tensor-core accumulator rounds towards zero at every addition, so a large
// diagonal term would come out too small by the same 2e-7 everywhere, and
// a X + P X loses most of its leading digits when the values are near 1
// (64 x 1920: 3.4e-6 of the result with the diagonals inside, 5.5e-7 so).
constexpr int kSmallThreads = 512;  // and one more warp, which issues the products
constexpr int kSmallSide = 128;     // rows of X
constexpr int kSmallColumns = 256;  // columns of X in one block
constexpr float kXScale = 16384.f, kPScale = 8192.f;

struct SmallArgs {
  int rows, cols, steps, m, n, tall, vec4;
  int mp, nj;  // rows (padded to 16) and columns of X per block (a multiple of 16)
  int parts;   // accumulators of X X^T
  float scale;
  const float* g;
  float* out;
};

// Shared memory of a block: X as two sets of 64-column tiles, then A as two sets,
// then the fp32 parts that a block of a cluster receives: [block][its units of
// 8 columns]; a full set of 128 rows behind the last tile is always inside the
// allocation, because an operand of M = 128 rows reads that far (those rows of
// the result are not used).
struct SmallLayout {
  int x_set, a_set, part_at, bytes;
};
__host__ __device__ inline SmallLayout small_layout(int mp, int nj, int blocks) {
  SmallLayout L;
  L.x_set = (nj + 63) / 64 * mp * 128;
  L.a_set = (mp + 63) / 64 * mp * 128;
  L.part_at = 2 * L.x_set + 2 * L.a_set;
  const int part = blocks > 1 ? mp * mp * 4 : 0, over = (kSmallSide - mp) * 128;
  L.bytes = L.part_at + (part > over ? part : over) + 1024;
  return L;
}

// Eight elements of X before scaling from column c on: of row r of G, or of its column r where G is tall.
__device__ __forceinline__ void small_input(const SmallArgs& a, const float* g, int r, int c, float (&v)[8]) {
  if (a.vec4 && r < a.m && c + 8 <= a.n) {
    const float4* p = reinterpret_cast<const float4*>(g + (long long)r * a.cols + c);
    const float4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    return;
  }
  const float* p = a.tall ? g + (long long)c * a.cols + r : g + (long long)r * a.cols + c;
  const long long next = a.tall ? a.cols : 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r < a.m && c + i < a.n ? p[i * next] : 0.f;
}

// The products of one contraction in the order low high, high low, high high:
// small terms before large ones.  da, db: descriptors of the high parts;
// la, lb: offsets of the low ones; sb: advance of b per step of 16; jump: the
// extra advance from a tile's end to the next (all in 16-byte units).  Run by a
// whole warp, issued by one lane.
__device__ __forceinline__ void issue_products(uint32_t tmem, uint64_t da, uint64_t db, uint32_t la, uint32_t lb,
                                               uint32_t jump, uint32_t sb, uint32_t jb, int first, int last,
                                               uint32_t idesc, uint32_t issue) {
#pragma unroll 1
  for (int i = first; i < last; ++i) {
    const uint64_t x = da + 2 * i + (i >> 2) * jump, y = db + sb * i + (i >> 2) * jb;
    tc::mma(tmem, x + la, y, idesc, i > first, issue);
    tc::mma(tmem, x, y + lb, idesc, true, issue);
  }
#pragma unroll 1
  for (int i = first; i < last; ++i)
    tc::mma(tmem, da + 2 * i + (i >> 2) * jump, db + sb * i + (i >> 2) * jb, idesc, true, issue);
}

__global__ void __launch_bounds__(kSmallThreads + 32, 1) ortho_small_kernel(SmallArgs a, int blocks) {
  extern __shared__ uint8_t raw[];
  __shared__ double sums[kSmallThreads / 32];
  __shared__ double block_sum;
  __shared__ __align__(16) float a_diag[kSmallSide];  // diagonal of A
  __shared__ float p_diag[kSmallSide];  // diagonal of P
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t bars[4];
  const SmallLayout L = small_layout(a.mp, a.nj, blocks);
  uint8_t* base = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  uint8_t* xs = base;
  uint8_t* as = base + 2 * L.x_set;
  const uint32_t x_addr = tc::smem_addr(xs), a_addr = tc::smem_addr(as);
  const uint32_t done = tc::smem_addr(&bars[0]), ready = tc::smem_addr(&bars[1]);
  const uint32_t parts_in = tc::smem_addr(&bars[2]), a_in = tc::smem_addr(&bars[3]);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const bool issuer = warp == kSmallThreads / 32;
  const int rank = blockIdx.x % blocks, matrix = blockIdx.x / blocks;
  const int c0 = rank * a.nj;
  const float* g = a.g + (long long)matrix * a.rows * a.cols;
  float* out = a.out + (long long)matrix * a.rows * a.cols;
  // tensor memory: the accumulators of X X^T, then A in place of the first and R R behind it, then P X over both;
  // and X
  const int square_at = a.mp * (a.parts > 1 ? a.parts - 1 : 1);
  const int x_at = square_at + a.mp > a.nj ? square_at + a.mp : a.nj;
  uint32_t columns = 32;
  while ((int)columns < x_at + a.nj) columns <<= 1;

  if (issuer) {
    tc::tmem_alloc(tc::smem_addr(&tmem_slot), columns);
    if (lane == 0) {
      tc::mbar_init(done, 1);
      tc::mbar_init(ready, kSmallThreads / 32);
      tc::mbar_init(parts_in, 1);
      tc::mbar_init(a_in, 1);
    }
  }
  // X once from memory; the Frobenius norm from squares in 64 bits, which
  // neither overflow nor vanish
  constexpr int kMost = kSmallSide * kSmallColumns / 8 / kSmallThreads;  // 8-column units a thread
  const int units = a.nj / 8, all_units = issuer ? 0 : a.mp * units;
  float v[kMost][8];
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (k * kSmallThreads >= all_units) break;
    const int q = tid + k * kSmallThreads;
    const int r = a.tall ? q % a.mp : q / units, u = a.tall ? q / a.mp : q % units;
    small_input(a, g, q < all_units ? r : a.m, c0 + 8 * u, v[k]);
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (k * kSmallThreads >= all_units) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma((double)v[k][i], (double)v[k][i], s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && !issuer) sums[warp] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / 32; ++w) s += sums[w];
  if (blocks > 1) {
    if (tid == 0) block_sum = s;
    tc::cluster_sync();
    s = 0.0;
    for (int k = 0; k < blocks; ++k) s += tc::peer_load_double(tc::peer_addr(tc::smem_addr(&block_sum), k));
  }
  // 2^14 / norm as f 2^(e1 + e2), each factor a normal fp32 number
  int e;
  const float f = (float)frexp(kXScale / (sqrt(s) + kNsEps), &e);
  const float s1 = ldexpf(1.f, e / 2), s2 = ldexpf(f, e - e / 2);
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (k * kSmallThreads >= all_units) break;
    const int q = tid + k * kSmallThreads;
    if (q >= all_units) continue;
    const int r = a.tall ? q % a.mp : q / units, u = a.tall ? q / a.mp : q % units;
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_float2(v[k][2 * i] * s1 * s2, v[k][2 * i + 1] * s1 * s2);
    uint4 hi, lo;
    tc::split8(w, hi, lo);
    const uint32_t at = (u >> 3) * a.mp * 128 + tc::tile_unit(r, u & 7);
    *reinterpret_cast<uint4*>(xs + at) = hi;
    *reinterpret_cast<uint4*>(xs + L.x_set + at) = lo;
  }
  tc::fence_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot, row_set = a.mp * 128;
  uint32_t done_parity = 0, ready_parity = 0;
  bool ok = true;

  if (issuer) {
    const uint32_t issue = tc::elect(), jump = row_set / 16 - 8;
    const uint64_t x_k = tc::desc_k(x_addr), a_k = tc::desc_k(a_addr), x_mn = tc::desc_mn(x_addr, row_set);
    const uint32_t square = tc::instruction(a.mp, false), wide = tc::instruction(a.nj, true);
    const uint32_t xl = L.x_set / 16, al = L.a_set / 16;
    auto wait_ready = [&]() {
      if (ok) ok = tc::mbar_wait(ready, ready_parity);
      ready_parity ^= 1;
      tc::fence_after_sync();
    };
    for (int step = 0; step < a.steps; ++step) {
      if (step > 0) wait_ready();
      for (int p = 0; p < a.parts; ++p)
        issue_products(tmem + p * a.mp, x_k, x_k, xl, xl, jump, 2, jump, p * (a.nj / 16) / a.parts,
                       (p + 1) * (a.nj / 16) / a.parts, square, issue);
      tc::commit(done, issue);
      wait_ready();
      issue_products(tmem + square_at, a_k, a_k, al, al, jump, 2, jump, 0, a.mp / 16, square, issue);
      tc::commit(done, issue);
      wait_ready();
      issue_products(tmem, a_k, x_mn, al, xl, jump, 128, 0, 0, a.mp / 16, wide, issue);
      tc::commit(done, issue);
      __syncwarp();
    }
  } else {
    // this thread's row of the accumulator and its columns, 16 of every 64
    const int r = (warp & 3) * 32 + lane, first = (warp >> 2) * 16;
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool live = (warp & 3) * 32 < a.mp;  // the warp's rows hold part of the result
    const bool row_on = r < a.mp;
    auto wait_done = [&]() {
      if (ok) ok = tc::mbar_wait(done, done_parity);
      done_parity ^= 1;
      tc::fence_after_sync();
    };
    auto wrote = [&]() {  // what the warp wrote is there for the next products
      tc::fence_async();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(ready);
    };
    auto all_wrote = [&]() {  // and what the other warps wrote, for this one
      if (ok) ok = tc::mbar_wait(ready, ready_parity);
      ready_parity ^= 1;
    };
    // f(column, 16 values of the accumulator, 16 values kept at `kept`) for the thread's columns below `end`;
    // `parts` accumulators `at`, at + mp, ... are added
    auto for_columns = [&](int end, int at, int parts, int kept, auto&& f) {
      if (!live) return;
      for (int c = first; c < end; c += 64) {
        uint32_t p[16], q[16];
        tc::tmem_load16(t_row + at + c, p);
        if (kept >= 0) tc::tmem_load16(t_row + kept + c, q);
        tc::tmem_wait(p);
        if (kept >= 0) tc::tmem_wait(q);
        float2 w[8], x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1]));
          x[i] = make_float2(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1]));
        }
        for (int k = 1; k < parts; ++k) {
          tc::tmem_load16(t_row + at + k * a.mp + c, p);
          tc::tmem_wait(p);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = __fadd2_rn(w[i], make_float2(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1])));
        }
        f(c, w, x);
        __syncwarp();
      }
    };
    // the element of column `col` out of sixteen, which becomes 0
    auto take = [](float2(&w)[8], int col) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (col == 2 * i) d = w[i].x, w[i].x = 0.f;
        if (col == 2 * i + 1) d = w[i].y, w[i].y = 0.f;
      }
      return d;
    };
    // 16 columns from c on to and from the tiles
    auto place = [&](int c, int h) { return (c >> 6) * row_set + tc::tile_unit(r, ((c >> 3) + h) & 7); };
    auto put = [&](uint8_t* tiles, int set, int c, const float2(&w)[8]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 u[4] = {w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
        uint4 hi, lo;
        tc::split8(u, hi, lo);
        const uint32_t at = place(c, h);
        *reinterpret_cast<uint4*>(tiles + at) = hi;
        *reinterpret_cast<uint4*>(tiles + set + at) = lo;
      }
    };
    auto get = [&](const uint8_t* tiles, int set, int c, float2(&w)[8]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = place(c, h);
        float2 u[4];
        tc::join8(*reinterpret_cast<const uint4*>(tiles + at), *reinterpret_cast<const uint4*>(tiles + set + at), u);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * h + i] = u[i];
      }
    };
    auto pair = [](float v) { return make_float2(v, v); };
    const int own_units = a.mp * a.mp / 8 / blocks;  // 8-column units of A that a block sums
    const uint32_t part_addr = tc::smem_addr(base) + L.part_at;

    for (int step = 0; step < a.steps; ++step) {
      if (blocks > 1 && tid == 0) {  // what this step will receive
        tc::mbar_expect(parts_in, own_units * blocks * 32);
        tc::mbar_expect(a_in, 4 * a.mp * a.mp + 4 * a.mp);
      }
      // A = X X^T: the diagonal to a_diag, the rest (x 2^14) to the tiles
      wait_done();
      for_columns(a.mp, 0, a.parts, -1, [&](int c, float2(&w)[8], float2(&)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __fmul2_rn(w[i], pair(1.f / kXScale));
        if (blocks > 1) {  // to the block that owns the unit
          if (row_on)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int u = r * (a.mp / 8) + (c >> 3) + h, owner = u / own_units;
              const uint32_t to =
                  tc::peer_addr(part_addr + (rank * own_units + u - owner * own_units) * 32, owner);
              const uint32_t bar = tc::peer_addr(parts_in, owner);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float2 x = w[4 * h + 2 * i], y = w[4 * h + 2 * i + 1];
                tc::async_store16(to + 16 * i, make_uint4(__float_as_uint(x.x), __float_as_uint(x.y),
                                                          __float_as_uint(y.x), __float_as_uint(y.y)), bar);
              }
            }
          return;
        }
        const float d = (r >> 4) == (c >> 4) ? take(w, r & 15) : 0.f;
        if ((r >> 4) == (c >> 4) && row_on) a_diag[r] = d * (1.f / kXScale);
        tc::tmem_store16(t_row + c, w);
        if (row_on) put(as, L.a_set, c, w);
      });
      if (blocks == 1) tc::tmem_store_wait();
      if (blocks > 1) {
        if (ok) ok = tc::mbar_wait_cluster(parts_in, step & 1);  // every block's part is there
        // `blocks` neighbouring lanes take one unit of 8 columns: each reads one block's part, all get the
        // sum, and each sends it to one block
        const int row_units = a.mp / 8, pairs = own_units * blocks, peer = tid % blocks;
        const uint32_t bar = tc::peer_addr(a_in, peer);
        constexpr int kPairs = kSmallSide * kSmallSide / 8 / kSmallThreads;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          if (k * kSmallThreads >= pairs) break;
          const int q = tid + k * kSmallThreads, own = q / blocks, u = rank * own_units + own;
          const int rr = u / row_units, cu = u % row_units;
          float2 w[4] = {};
          if (q < pairs) {
            const float4* from = reinterpret_cast<const float4*>(base + L.part_at + (peer * own_units + own) * 32);
            const float4 x = from[0], y = from[1];
            w[0] = make_float2(x.x, x.y), w[1] = make_float2(x.z, x.w);
            w[2] = make_float2(y.x, y.y), w[3] = make_float2(y.z, y.w);
          }
          for (int o = 1; o < blocks; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i].x += __shfl_xor_sync(0xffffffffu, w[i].x, o);
              w[i].y += __shfl_xor_sync(0xffffffffu, w[i].y, o);
            }
          if (q < pairs) {
            if (rr / 8 == cu) {
              float d = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((rr & 7) == 2 * i) d = w[i].x, w[i].x = 0.f;
                if ((rr & 7) == 2 * i + 1) d = w[i].y, w[i].y = 0.f;
              }
              tc::async_store4(tc::peer_addr(tc::smem_addr(&a_diag[rr]), peer), d * (1.f / kXScale), bar);
            }
            uint4 hi, lo;
            tc::split8(w, hi, lo);
            const uint32_t to = tc::peer_addr(a_addr + (cu >> 3) * row_set + tc::tile_unit(rr, cu & 7), peer);
            tc::async_store16(to, hi, bar);
            tc::async_store16(to + L.a_set, lo, bar);
          }
        }
        if (ok) ok = tc::mbar_wait_cluster(a_in, step & 1);
      }
      wrote();
      // P = b A + c A A (x 2^13) over A: (A A)[r][c] = (R R)[r][c] + (d[r] + d[c]) R[r][c] off the diagonal
      wait_done();
      all_wrote();
      const float dr = row_on ? a_diag[r] : 0.f;
      for_columns(a.mp, square_at, 1, blocks == 1 ? 0 : -1, [&](int c, float2(&w)[8], float2(&x)[8]) {
        if (!row_on) return;
        if (blocks > 1) get(as, L.a_set, c, x);
        const bool diagonal = (r >> 4) == (c >> 4);
        if (diagonal) {
          const float d = take(w, r & 15) * (1.f / (kXScale * kXScale));
          p_diag[r] = fmaf(kNsC, fmaf(dr, dr, d), kNsB * dr);
        }
        constexpr float k = kPScale / kXScale;
        const float own = k * fmaf(kNsC, dr, kNsB);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float4 d = *reinterpret_cast<const float4*>(a_diag + c + 2 * i);
          const float2 y0 = __ffma2_rn(make_float2(d.x, d.y), pair(k * kNsC), pair(own));
          const float2 y1 = __ffma2_rn(make_float2(d.z, d.w), pair(k * kNsC), pair(own));
          w[i] = __ffma2_rn(w[i], pair(k / kXScale * kNsC), __fmul2_rn(x[i], y0));
          w[i + 1] = __ffma2_rn(w[i + 1], pair(k / kXScale * kNsC), __fmul2_rn(x[i + 1], y1));
        }
        // on the diagonal both terms are zero: x was taken there before, w just now
        put(as, L.a_set, c, w);
      });
      wrote();
      // X = (a + diagonal of P) X + (the rest of P) X
      wait_done();
      all_wrote();
      const float dx = row_on ? kNsA + p_diag[r] : 0.f;
      const bool last = step + 1 == a.steps;
      for_columns(a.nj, 0, 1, step > 0 ? x_at : -1, [&](int c, float2(&w)[8], float2(&x)[8]) {
        if (step == 0 && row_on) get(xs, L.x_set, c, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __ffma2_rn(w[i], pair(1.f / kPScale), __fmul2_rn(x[i], pair(dx)));
        if (!last) {
          tc::tmem_store16(t_row + x_at + c, w);
          if (row_on) put(xs, L.x_set, c, w);
        } else if (r < a.m) {
          const int col = c0 + c;
          const float by = ok ? a.scale / kXScale : __int_as_float(0x7fffffff);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = __fmul2_rn(w[i], pair(by));
          if (a.vec4 && col + 16 <= a.n) {
            float4* to = reinterpret_cast<float4*>(out + (long long)r * a.cols + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = make_float4(w[2 * i].x, w[2 * i].y, w[2 * i + 1].x, w[2 * i + 1].y);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (col + i < a.n)
                out[a.tall ? (long long)(col + i) * a.cols + r : (long long)r * a.cols + col + i] =
                    i & 1 ? w[i / 2].y : w[i / 2].x;
          }
        }
      });
      if (!last) {
        tc::tmem_store_wait();
        wrote();
        all_wrote();
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (issuer) tc::tmem_free(tmem, columns);
  if (blocks > 1) tc::cluster_sync();  // no block leaves while another may still read its shared memory
}

// Blocks per matrix: 1, 2, 4 or 8; 0 where they cannot hold the matrix.  One
// block as long as it holds all columns (4 x 128 x 256: 59 us, with two blocks
// 74 us, the exchange costs more than half of the columns); then so many that
// each has at most 128 (20 x 64 x 512: two blocks 53 us, four 42 us), but not
// more than run at once, and clusters do not fill the last SMs (37 and 40 x 64 x 512:
// two blocks 54 us, four 83 us; 58 x 96 x 764: four 139 us, eight 259 us).
constexpr int kSmallResident = 128;
constexpr int kSmallShared = 226 * 1024 - 512;  // of 227 KB; the rest for the kernel's own variables
int small_columns(int n, int blocks) { return ((n + blocks - 1) / blocks + 15) / 16 * 16; }
int small_blocks(int batch, int m, int n) {
  if (m > kSmallSide) return 0;
  int found = 0;
  for (int b = 1; b <= 8; b *= 2) {
    const int nj = small_columns(n, b);
    if (nj <= kSmallColumns && small_layout((m + 15) / 16 * 16, nj, b).bytes <= kSmallShared) found = b;
    if (found != 0 && (b == 1 || nj <= 128 || (long long)batch * 2 * b > kSmallResident)) break;
  }
  return found;
}

cudaError_t launch_small(int batch, int rows, int cols, int steps, float scale, const float* g, float* out,
                         cudaStream_t stream) {
  SmallArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.steps = steps;
  a.tall = rows > cols;
  a.m = a.tall ? cols : rows;
  a.n = a.tall ? rows : cols;
  const int blocks = small_blocks(batch, a.m, a.n);
  a.mp = (a.m + 15) / 16 * 16;
  a.nj = small_columns(a.n, blocks);
  // Sums of like signs (the diagonal) lose half a step each time 16 columns are
  // added: accumulators of some 64 columns, added in fp32, keep that small.  256
  // columns of tensor memory for them at most, X takes the others.
  a.parts = a.nj / 64 < 256 / a.mp ? a.nj / 64 : 256 / a.mp;
  a.parts = a.parts < 1 ? 1 : a.parts > 4 ? 4 : a.parts;
  a.vec4 = !a.tall && cols % 4 == 0 && (((uintptr_t)g | (uintptr_t)out) & 15u) == 0;
  a.scale = scale;
  a.g = g;
  a.out = out;
  const int bytes = small_layout(a.mp, a.nj, blocks).bytes;
  // the limit belongs to the kernel, not to the call: always the same one, so that no thread takes from
  // another what it is about to launch with
  cudaError_t e = cudaFuncSetAttribute(ortho_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)batch * blocks);
  cfg.blockDim = dim3(kSmallThreads + 32);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, ortho_small_kernel, a, blocks);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------- few entries
// Matrices whose products are some ten thousand multiplications: a tensor-core
// product of 128 rows and its way through tensor memory take about 1 us whatever
// they hold, plain fp32 sums in shared memory less.  One block per matrix; KP
// is the number of rows, rounded up to a power of two (the others are zero).
// X, A and P = b A + c A A lie in shared memory by rows whose strides are odd
// multiples of 16 bytes (no two of eight rows share banks); a thread sums a 2 x 2
// tile of A or P, or a 2 x 4 tile of X, with `team` threads sharing the long sums.
constexpr int kFewRows = 32;
constexpr int kFewThreads = 512;

struct FewLayout {
  int quads, stride, bytes;  // groups of four columns; floats from row to row of X
};
__host__ __device__ inline FewLayout few_layout(int kp, int n) {
  FewLayout L;
  L.quads = (n + 3) / 4;
  L.stride = 4 * (L.quads | 1);
  L.bytes = (int)sizeof(float) * (2 * kp * L.stride + 2 * kp * (kp + 4));
  return L;
}

// out(i, j, sum over the columns of x_i x_j) for all rows i, j.
template <int KP, class F>
__device__ __forceinline__ void few_gram(const float* x, int stride, int quads, int team_shift, F&& out) {
  constexpr int H = KP / 2;
  const int team = 1 << team_shift, mine = threadIdx.x & (team - 1);
  for (int t0 = 0; t0 < H * H; t0 += blockDim.x >> team_shift) {  // the same for every thread
    const int t = t0 + (threadIdx.x >> team_shift), i = t % H, j = t / H;
    float s[2][2] = {};
    if (t < H * H)
      for (int q = mine; q < quads; q += team) {
        float4 u[2], v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          u[k] = *reinterpret_cast<const float4*>(x + (i + k * H) * stride + 4 * q);
          v[k] = *reinterpret_cast<const float4*>(x + (j + k * H) * stride + 4 * q);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int l = 0; l < 2; ++l)
            s[k][l] = fmaf(u[k].w, v[l].w, fmaf(u[k].z, v[l].z, fmaf(u[k].y, v[l].y, fmaf(u[k].x, v[l].x, s[k][l]))));
      }
    for (int o = team >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k >> 1][k & 1] += __shfl_xor_sync(0xffffffffu, s[k >> 1][k & 1], o);
    if (t < H * H && mine == 0)
#pragma unroll
      for (int k = 0; k < 4; ++k) out(i + (k >> 1) * H, j + (k & 1) * H, s[k >> 1][k & 1]);
  }
}

template <int KP>
__global__ void __launch_bounds__(kFewThreads) ortho_few_kernel(SmallArgs a, int gram_shift, int square_shift) {
  extern __shared__ __align__(16) float few_smem[];
  __shared__ double sums[kFewThreads / 32];
  constexpr int H = KP / 2, kStride = KP + 4;
  const FewLayout L = few_layout(KP, a.n);
  float *x = few_smem, *y = x + KP * L.stride, *gram = y + KP * L.stride, *p = gram + KP * kStride;
  const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
  const float* g = a.g + (long long)blockIdx.x * a.rows * a.cols;
  float* out = a.out + (long long)blockIdx.x * a.rows * a.cols;
  // X once from memory; squares in 64 bits, which neither overflow nor vanish
  const int width = 4 * L.quads;
  const auto place = [&](int q, int& r, int& c) {
    if (a.tall) {
      r = q % KP;
      c = q / KP;
    } else {
      r = q / width;
      c = q - r * width;
    }
  };
  double s = 0.0;
#pragma unroll 4
  for (int q = tid; q < KP * width; q += blockDim.x) {
    int r, c;
    place(q, r, c);
    const float v = r < a.m && c < a.n ? g[a.tall ? (long long)c * a.cols + r : (long long)r * a.cols + c] : 0.f;
    x[r * L.stride + c] = v;
    s = fma((double)v, (double)v, s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sums[tid >> 5] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < warps; ++w) s += sums[w];
  // 1 / norm as f 2^(e1 + e2), each factor a normal fp32 number
  int e;
  const float f = (float)frexp(1.0 / (sqrt(s) + kNsEps), &e);
  const float s1 = ldexpf(1.f, e / 2), s2 = ldexpf(f, e - e / 2);
  for (int q = tid; q < KP * width; q += blockDim.x) {  // each thread its own
    int r, c;
    place(q, r, c);
    x[r * L.stride + c] *= s1 * s2;
  }
  for (int step = 1; step <= a.steps; ++step) {
    __syncthreads();
    few_gram<KP>(x, L.stride, L.quads, gram_shift, [&](int i, int j, float v) { gram[i * kStride + j] = v; });
    __syncthreads();
    few_gram<KP>(gram, kStride, KP / 4, square_shift, [&](int i, int j, float v) {  // A is symmetric
      p[i * kStride + j] = fmaf(kNsB, gram[i * kStride + j], kNsC * v);
    });
    __syncthreads();
    for (int t = tid; t < H * L.quads; t += blockDim.x) {
      const int i = t % H, q = t / H;
      float4 w[2] = {};
#pragma unroll
      for (int l = 0; l < KP; l += 4) {
        float4 b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) b[k] = *reinterpret_cast<const float4*>(p + (i + k * H) * kStride + l);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float4 v = *reinterpret_cast<const float4*>(x + (l + d) * L.stride + 4 * q);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float m = d == 0 ? b[k].x : d == 1 ? b[k].y : d == 2 ? b[k].z : b[k].w;
            w[k] = make_float4(fmaf(m, v.x, w[k].x), fmaf(m, v.y, w[k].y), fmaf(m, v.z, w[k].z), fmaf(m, v.w, w[k].w));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = i + k * H;
        const float4 v = *reinterpret_cast<const float4*>(x + r * L.stride + 4 * q);
        w[k] = make_float4(fmaf(kNsA, v.x, w[k].x), fmaf(kNsA, v.y, w[k].y), fmaf(kNsA, v.z, w[k].z), fmaf(kNsA, v.w, w[k].w));
        if (step < a.steps) {
          *reinterpret_cast<float4*>(y + r * L.stride + 4 * q) = w[k];
        } else if (r < a.m) {
          const float o[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int d = 0; d < 4; ++d)
            if (4 * q + d < a.n)
              out[a.tall ? (long long)(4 * q + d) * a.cols + r : (long long)r * a.cols + 4 * q + d] = a.scale * o[d];
        }
      }
    }
    float* z = x;
    x = y;
    y = z;
  }
}

// Rows of X that the kernel above is made for, or 0.  Five steps against the tensor cores', in us:
// 5 x 8 x 8: 6.0 against 15.1; 64 x 16 x 16: 7.9, 14.8; 8 x 128: 8.9, 21; 16 x 128: 13, 21; 32 x 32: 13, 17;
// 32 x 64: 17.8, 19.0; 16 x 256: 19, 30; 8 x 1024: 24, 27; beyond kFewWork 16 x 512: 31, 27; 32 x 128: 29, 23.
// Threads: 64 for the smallest (8 x 8: 5.7, 256 threads 5.9), 512 for long rows (16 x 256: 19, 256 threads 23),
// 256 between and for 32 rows, whose 2 x 2 tiles they cover (32 x 32: 13, 512 threads 16).
constexpr int kFewWork = 65536;
int few_rows(int m, int n) {
  if (m > kFewRows) return 0;
  int kp = 4;
  while (kp < m) kp *= 2;
  return (long long)kp * kp * n <= kFewWork ? kp : 0;
}

cudaError_t launch_few(int batch, int rows, int cols, int steps, float scale, const float* g, float* out,
                       cudaStream_t stream) {
  SmallArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.steps = steps;
  a.tall = rows > cols;
  a.m = a.tall ? cols : rows;
  a.n = a.tall ? rows : cols;
  a.scale = scale;
  a.g = g;
  a.out = out;
  const int kp = few_rows(a.m, a.n);
  const FewLayout L = few_layout(kp, a.n);
  const int work = kp * kp * a.n, threads = work <= 512 ? 64 : kp == 32 || work <= 8192 ? 256 : kFewThreads;
  const auto shift = [&](int quads) {  // of the threads that share a sum
    int s = 0;
    while (s < 5 && (2 << s) * (kp / 2) * (kp / 2) <= threads && (2 << s) <= quads) ++s;
    return s;
  };
  void (*kernel)(SmallArgs, int, int) = kp == 4   ? ortho_few_kernel<4>
                                        : kp == 8  ? ortho_few_kernel<8>
                                        : kp == 16 ? ortho_few_kernel<16>
                                                   : ortho_few_kernel<32>;
  if (L.bytes > 48 * 1024) {  // more than a block gets unasked: what the longest rows of the kernel take
    const int most = few_layout(kp, kFewWork / (kp * kp)).bytes;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  kernel<<<batch, threads, L.bytes, stream>>>(a, shift(L.quads), shift(kp / 4));
  return cudaGetLastError();
}

// ------------------------------------------------------------- larger matrices
// One launch per product, over 128 x 128 tiles of the result.  X, A and P lie in
// the workspace as the operands' own shared-memory tiles (128 rows x 64 columns
// of fp16, swizzled, 16 KB; the low parts a set of tiles behind the high ones),
// so a tile is one bulk copy, and the tiles that X X^T reads along their rows
// P X reads down them.  Rows and columns beyond the matrix are zero and stay so.
// A block has one warp that copies (kStages stages of 64 columns), one that
// issues the products and sixteen that turn the accumulator into the next
// operand.  The diagonal of X X^T, long sums of like signs, is summed in fp32 where
// X is made.  The launches are dependent ones (programmatic stream serialization):
// each sets up while the one before ends and waits for it before its first
// access to global memory.  Four accumulators fill the tensor memory: one for
// low high + high low, three that share the columns of high high, so that an
// accumulator is rounded towards zero a third as often (2 x 1024 x 1024: 1.7e-6
// of the result, plain fp32 products 3.1e-6; with one accumulator 4.9e-6).
// 2 x 1024 x 1024 takes 245 us, 15 products of 14 us after the set-up: 8 us the MMAs and their
// loads (6.6 at the tensor rate of 128 blocks), 6 us from one launch's last
// store to the next one's first product and the epilogue.  Measured and not kept: pairs of
// blocks that share the right operand (cta_group::2, 283 us: the pair's barriers
// cost more than the 25 % fewer bytes) and symmetric products computed by half (261 us).
constexpr int kTileBytes = 128 * 128, kStages = 3, kStageBytes = 4 * kTileBytes;
constexpr int kLargeThreads = kSmallThreads + 64;
constexpr int kLargeParts = 3;

struct LargeArgs {
  int rows, cols, m, n, tall, vec4;
  int mt, kt, nt;  // tiles: rows of X (128), columns of A with data (64), columns of X (64, even)
  float scale;
  long long x_set, a_set;  // bytes of one set of tiles of one matrix
  uint8_t *x, *x_next, *a, *p;  // [batch][2 sets][row tiles][column tiles]
  float *a_diag, *p_diag;       // [batch][mt * 128]
  float* squares;               // [batch][nt][mt * 128] sums of squares of X by row and 64-column tile
  double* sums;                 // [batch][kSumBlocks] sums of squares
  const float* g;
  float* out;
};
constexpr int kSumBlocks = 64;

// Sums of squares of a matrix, in 64 bits, one per block.
__global__ void __launch_bounds__(256) ortho_norm_kernel(LargeArgs a) {
  grid_dependents_launch();
  __shared__ double red[256];
  const long long size = (long long)a.rows * a.cols;
  const float* g = a.g + blockIdx.y * size;
  double s = 0.0;
#pragma unroll 4
  for (long long i = blockIdx.x * 256 + threadIdx.x; i < size; i += kSumBlocks * 256) s = fma((double)g[i], (double)g[i], s);
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.sums[(long long)blockIdx.y * kSumBlocks + blockIdx.x] = red[0];
}

// 2^14 X as tiles: one block per tile.
__global__ void __launch_bounds__(256) ortho_tiles_kernel(LargeArgs a) {
  const int ct = blockIdx.x, rt = blockIdx.y, z = blockIdx.z;
  grid_dependents_launch();
  grid_dependency_wait();
  double s = 0.0;
  for (int k = 0; k < kSumBlocks; ++k) s += a.sums[(long long)z * kSumBlocks + k];
  int e;
  const float f = (float)frexp(kXScale / (sqrt(s) + kNsEps), &e);
  const float s1 = ldexpf(1.f, e / 2), s2 = ldexpf(f, e - e / 2);
  const float* g = a.g + (long long)z * a.rows * a.cols;
  uint8_t* to = a.x + (2 * z * a.x_set) + ((long long)rt * a.nt + ct) * kTileBytes;
  __shared__ float sq[8][128];
  for (int q = threadIdx.x; q < 128 * 8; q += 256) {
    const int r = a.tall ? q & 127 : q >> 3, u = a.tall ? q >> 7 : q & 7;
    const int row = rt * 128 + r, col = ct * 64 + u * 8;
    float2 w[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = 0.f;
      if (row < a.m && col + i < a.n)
        v = g[a.tall ? (long long)(col + i) * a.cols + row : (long long)row * a.cols + col + i] * s1 * s2;
      if (i & 1) w[i / 2].y = v;
      else w[i / 2].x = v;
    }
    uint4 hi, lo;
    tc::split8(w, hi, lo);
    const uint32_t at = tc::tile_unit(r, u);
    *reinterpret_cast<uint4*>(to + at) = hi;
    *reinterpret_cast<uint4*>(to + a.x_set + at) = lo;
    float2 d = __fmul2_rn(w[0], w[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) d = __ffma2_rn(w[i], w[i], d);
    sq[u][r] = d.x + d.y;
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    float d = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) d += sq[u][threadIdx.x];
    a.squares[((long long)z * a.nt + ct) * a.mt * 128 + rt * 128 + threadIdx.x] = d;
  }
}

enum { kGram = 0, kSquare = 1, kApply = 2 };

// kGram: A = X X^T.  kSquare: P = b A + c A A.  kApply: X' = (a + P) X, or the output when LAST.
template <int MODE, bool LAST>
__global__ void __launch_bounds__(kLargeThreads, 1) ortho_product_kernel(LargeArgs a) {
  grid_dependents_launch();
  extern __shared__ uint8_t raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t bars[2 * kStages + 1];
  __shared__ float sq[4][128];
  uint8_t* base = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);
  const uint32_t smem = tc::smem_addr(base);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int ct = blockIdx.x, rt = blockIdx.y;  // tile of the result, 128 columns wide
  const long long z = blockIdx.z;
  uint8_t* xz = a.x + 2 * z * a.x_set;
  uint8_t* az = a.a + 2 * z * a.a_set;
  uint8_t* pz = a.p + 2 * z * a.a_set;
  const int at_cols = 2 * a.mt;  // column tiles of A
  const int chunks = MODE == kGram ? (a.n + 63) / 64 : a.kt;
  constexpr int kColumns = 128 * (kLargeParts + 1);
  const int parts = chunks < kLargeParts ? chunks : kLargeParts;
  auto full = [&](int s) { return tc::smem_addr(&bars[s]); };
  auto empty = [&](int s) { return tc::smem_addr(&bars[kStages + s]); };
  const uint32_t done = tc::smem_addr(&bars[2 * kStages]);

  if (warp == kSmallThreads / 32) {
    tc::tmem_alloc(tc::smem_addr(&tmem_slot), kColumns);
    if (lane == 0)
      for (int k = 0; k < 2 * kStages + 1; ++k) tc::mbar_init(tc::smem_addr(&bars[k]), 1);
  }
  tc::fence_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  bool ok = true;
  grid_dependency_wait();

  if (warp == kSmallThreads / 32 + 1) {
    if (lane == 0) {  // copies
      for (int c = 0; c < chunks && ok; ++c) {
        const int s = c % kStages;
        if (c >= kStages) ok = tc::mbar_wait(empty(s), (c / kStages - 1) & 1);
        if (!ok) break;
        const uint32_t to = smem + s * kStageBytes;
        tc::mbar_expect(full(s), kStageBytes);
#pragma unroll
        for (int set = 0; set < 2; ++set) {
          const uint8_t* left = MODE == kGram    ? xz + set * a.x_set + ((long long)rt * a.nt + c) * kTileBytes
                                : MODE == kSquare ? az + set * a.a_set + ((long long)rt * at_cols + c) * kTileBytes
                                                  : pz + set * a.a_set + ((long long)rt * at_cols + c) * kTileBytes;
          tc::bulk_load(to + set * kTileBytes, left, kTileBytes, full(s));
          const uint32_t right = to + (2 + set) * kTileBytes;
          if (MODE == kApply) {  // 64 rows of two column tiles
            const uint8_t* from = xz + set * a.x_set + ((long long)(c >> 1) * a.nt + 2 * ct) * kTileBytes + (c & 1) * (kTileBytes / 2);
            tc::bulk_load(right, from, kTileBytes / 2, full(s));
            tc::bulk_load(right + kTileBytes / 2, from + kTileBytes, kTileBytes / 2, full(s));
          } else {
            const uint8_t* from = MODE == kGram ? xz + set * a.x_set + ((long long)ct * a.nt + c) * kTileBytes
                                                : az + set * a.a_set + ((long long)ct * at_cols + c) * kTileBytes;
            tc::bulk_load(right, from, kTileBytes, full(s));
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kSmallThreads / 32) {  // products
    const uint32_t issue = tc::elect(), idesc = tc::instruction(128, MODE == kApply);
    constexpr uint32_t kSet = kTileBytes / 16;  // low parts, in 16-byte units
    for (int c = 0; c < chunks; ++c) {
      const int s = c % kStages;
      if (ok) ok = tc::mbar_wait(full(s), (c / kStages) & 1);
      tc::fence_after_sync();
      const uint32_t from = smem + s * kStageBytes;
      const uint64_t da = tc::desc_k(from);
      const uint64_t db = MODE == kApply ? tc::desc_mn(from + 2 * kTileBytes, kTileBytes / 2) : tc::desc_k(from + 2 * kTileBytes);
      constexpr uint32_t kStep = MODE == kApply ? 128 : 2;
      const int p = c * parts / chunks;
      const bool fresh = c == 0 || (c - 1) * parts / chunks != p;
      const uint32_t d = tmem + p * 128, cross = tmem + kLargeParts * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tc::mma(cross, da + kSet + 2 * i, db + kStep * i, idesc, c > 0 || i > 0, issue);
        tc::mma(cross, da + 2 * i, db + kSet + kStep * i, idesc, true, issue);
        tc::mma(d, da + 2 * i, db + kStep * i, idesc, !fresh || i > 0, issue);
      }
      tc::commit(empty(s), issue);
    }
    tc::commit(done, issue);
    __syncwarp();
  } else {
    const int r = (warp & 3) * 32 + lane, first = (warp >> 2) * 16, row = rt * 128 + r;
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool diagonal = MODE != kApply && rt == ct;
    const float* ad = a.a_diag + z * a.mt * 128;
    float* pd = a.p_diag + z * a.mt * 128;
    // what the tile's own elements are combined with, read while the products run
    uint4 own[MODE == kGram ? 1 : 4][2];
    const uint8_t* from = MODE == kSquare ? az + ((long long)rt * at_cols + 2 * ct) * kTileBytes
                                          : xz + ((long long)rt * a.nt + 2 * ct) * kTileBytes;
    const long long set = MODE == kApply ? a.x_set : a.a_set;
    if (MODE != kGram)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = first + (k >> 1) * 64 + (k & 1) * 8;
        const uint8_t* p = from + (c >> 6) * kTileBytes + tc::tile_unit(r, (c >> 3) & 7);
        own[k][0] = *reinterpret_cast<const uint4*>(p);
        own[k][1] = *reinterpret_cast<const uint4*>(p + set);
      }
    const float dr = MODE == kSquare ? ad[row] : MODE == kApply ? kNsA + pd[row] : 0.f;
    if (MODE == kGram && diagonal && first == 0) {  // x 2^28
      float d = 0.f;
#pragma unroll 8
      for (int k = 0; k < a.nt; ++k) d += a.squares[(z * a.nt + k) * a.mt * 128 + row];
      a.a_diag[z * a.mt * 128 + row] = d * (1.f / (kXScale * kXScale));
    }
    float2 squares = make_float2(0.f, 0.f);
    ok = tc::mbar_wait(done, 0);
    tc::fence_after_sync();
    const float fine = ok ? 1.f : __int_as_float(0x7fffffff);
    auto pair = [](float v) { return make_float2(v, v); };
    auto take = [](float2(&w)[4], int col) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col == 2 * i) d = w[i].x, w[i].x = 0.f;
        if (col == 2 * i + 1) d = w[i].y, w[i].y = 0.f;
      }
      return d;
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int c = first + half * 64;
      uint32_t v[16];
      tc::tmem_load16(t_row + kLargeParts * 128 + c, v);
      tc::tmem_wait(v);
      float2 acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
      for (int k = 0; k < parts; ++k) {
        tc::tmem_load16(t_row + k * 128 + c, v);
        tc::tmem_wait(v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[i] = __fadd2_rn(acc[i], make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cu = c + 8 * h;
        float2 w[4] = {acc[4 * h], acc[4 * h + 1], acc[4 * h + 2], acc[4 * h + 3]};
        const bool on_diagonal = diagonal && (r >> 3) == (cu >> 3);
        if (MODE == kGram) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = __fmul2_rn(w[i], pair(fine / kXScale));
          if (on_diagonal) take(w, r & 7);
        } else {
          float2 x[4];
          tc::join8(own[2 * half + h][0], own[2 * half + h][1], x);
          if (MODE == kSquare) {
            if (on_diagonal) {
              float2 y[4] = {w[0], w[1], w[2], w[3]};
              pd[row] = fmaf(kNsC, fmaf(dr, dr, take(y, r & 7) * (1.f / (kXScale * kXScale))), kNsB * dr);
            }
            const float4 d0 = *reinterpret_cast<const float4*>(ad + ct * 128 + cu);
            const float4 d1 = *reinterpret_cast<const float4*>(ad + ct * 128 + cu + 4);
            const float2 dc[4] = {make_float2(d0.x, d0.y), make_float2(d0.z, d0.w), make_float2(d1.x, d1.y),
                                  make_float2(d1.z, d1.w)};
            constexpr float k = kPScale / kXScale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 by = __ffma2_rn(dc[i], pair(k * kNsC), pair(k * fmaf(kNsC, dr, kNsB)));
              w[i] = __ffma2_rn(w[i], pair(fine * (k / kXScale * kNsC)), __fmul2_rn(x[i], by));
            }
            if (on_diagonal) take(w, r & 7);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = __ffma2_rn(w[i], pair(fine / kPScale), __fmul2_rn(x[i], pair(dr)));
              squares = __ffma2_rn(w[i], w[i], squares);
            }
          }
        }
        if (MODE == kApply && LAST) {
          const int col = ct * 128 + cu;
          if (row < a.m) {
            float* out = a.out + z * a.rows * a.cols;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __fmul2_rn(w[i], pair(a.scale / kXScale));
            if (a.vec4 && col + 8 <= a.n) {
              float4* to = reinterpret_cast<float4*>(out + (long long)row * a.cols + col);
              to[0] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
              to[1] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
            } else {
              const float o[8] = {w[0].x, w[0].y, w[1].x, w[1].y, w[2].x, w[2].y, w[3].x, w[3].y};
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (col + i < a.n)
                  out[a.tall ? (long long)(col + i) * a.cols + row : (long long)row * a.cols + col + i] = o[i];
            }
          }
        } else {  // the stages are free: tile cu / 64, high and low
          uint4 hi, lo;
          tc::split8(w, hi, lo);
          uint8_t* to = base + (cu >> 6) * 2 * kTileBytes + tc::tile_unit(r, (cu >> 3) & 7);
          *reinterpret_cast<uint4*>(to) = hi;
          *reinterpret_cast<uint4*>(to + kTileBytes) = lo;
        }
      }
    }
    if (MODE == kApply && !LAST) sq[warp >> 2][r] = squares.x + squares.y;
  }
  tc::fence_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kSmallThreads / 32) tc::tmem_free(tmem, kColumns);
  if (MODE == kApply && !LAST && tid < 128) {  // the tile's two column tiles as one
    float* to = a.squares + (z * a.nt + 2 * ct) * a.mt * 128 + rt * 128 + tid;
    to[0] = (sq[0][tid] + sq[1][tid]) + (sq[2][tid] + sq[3][tid]);
    to[a.mt * 128] = 0.f;
  }
  if (!(MODE == kApply && LAST) && tid == 0) {
    uint8_t* to = MODE == kGram    ? az + ((long long)rt * at_cols + 2 * ct) * kTileBytes
                  : MODE == kSquare ? pz + ((long long)rt * at_cols + 2 * ct) * kTileBytes
                                    : a.x_next + 2 * z * a.x_set + ((long long)rt * a.nt + 2 * ct) * kTileBytes;
    const long long set = MODE == kApply ? a.x_set : a.a_set;
    for (int k = 0; k < 4; ++k)
      tc::bulk_store(to + (k >> 1) * kTileBytes + (k & 1) * set, smem + k * kTileBytes, kTileBytes);
    tc::bulk_store_wait();
  }
}

struct LargeLayout {
  int mt, kt, nt;
  size_t x_set, a_set, bytes;
};
LargeLayout large_layout(int batch, int m, int n) {
  LargeLayout L;
  L.mt = (m + 127) / 128;
  L.kt = (m + 63) / 64;
  L.nt = (n + 127) / 128 * 2;
  L.x_set = (size_t)L.mt * L.nt * kTileBytes;
  L.a_set = (size_t)L.mt * L.mt * 2 * kTileBytes;
  L.bytes = (size_t)batch * (4 * L.x_set + 4 * L.a_set + (2 + L.nt) * L.mt * 128 * sizeof(float) + kSumBlocks * sizeof(double));
  return L;
}

template <int MODE, bool LAST>
cudaError_t launch_product(const LargeArgs& a, dim3 grid, cudaStream_t stream) {
  constexpr int bytes = kStages * kStageBytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(ortho_product_kernel<MODE, LAST>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_kernel(ortho_product_kernel<MODE, LAST>, grid, kLargeThreads, bytes, stream, true, a);
}

cudaError_t launch_large(int batch, int rows, int cols, int steps, float scale, const float* g, float* out, void* ws,
                         cudaStream_t stream) {
  LargeArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.tall = rows > cols;
  a.m = a.tall ? cols : rows;
  a.n = a.tall ? rows : cols;
  a.vec4 = !a.tall && cols % 4 == 0 && ((uintptr_t)out & 15u) == 0;
  const LargeLayout L = large_layout(batch, a.m, a.n);
  a.mt = L.mt;
  a.kt = L.kt;
  a.nt = L.nt;
  a.scale = scale;
  a.x_set = (long long)L.x_set;
  a.a_set = (long long)L.a_set;
  uint8_t* at = (uint8_t*)ws;
  a.x = at;
  a.x_next = at += 2 * batch * L.x_set;
  a.a = at += 2 * batch * L.x_set;
  a.p = at += 2 * batch * L.a_set;
  a.sums = (double*)(at += 2 * batch * L.a_set);
  a.a_diag = (float*)(a.sums + (size_t)batch * kSumBlocks);
  a.p_diag = a.a_diag + (size_t)batch * L.mt * 128;
  a.squares = a.p_diag + (size_t)batch * L.mt * 128;
  a.g = g;
  a.out = out;
  ortho_norm_kernel<<<dim3(kSumBlocks, batch), 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_kernel(ortho_tiles_kernel, dim3(L.nt, L.mt, batch), 256, 0, stream, true, a);
  const dim3 square(L.mt, L.mt, batch), wide(L.nt / 2, L.mt, batch);
  for (int s = 0; s < steps && e == cudaSuccess; ++s) {
    e = launch_product<kGram, false>(a, square, stream);
    if (e == cudaSuccess) e = launch_product<kSquare, false>(a, square, stream);
    if (e == cudaSuccess)
      e = s + 1 == steps ? launch_product<kApply, true>(a, wide, stream) : launch_product<kApply, false>(a, wide, stream);
    uint8_t* t = a.x;
    a.x = a.x_next;
    a.x_next = t;
  }
  return e;
}

}  // namespace

size_t ortho_workspace(int batch, int rows, int cols) {
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  return few_rows(m, n) > 0 || small_blocks(batch, m, n) > 0 ? 0 : pad256(large_layout(batch, m, n).bytes);
}

cudaError_t launch_ortho(int batch, int rows, int cols, int steps, float scale, const float* g, float* out, void* ws,
                         cudaStream_t stream) {
  if (batch == 0 || rows == 0 || cols == 0) return cudaSuccess;
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if (few_rows(m, n) > 0) return launch_few(batch, rows, cols, steps, scale, g, out, stream);
  if (small_blocks(batch, m, n) > 0)
    return launch_small(batch, rows, cols, steps, scale, g, out, stream);
  return launch_large(batch, rows, cols, steps, scale, g, out, ws, stream);
}

}  // namespace cgtp
