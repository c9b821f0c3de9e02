// Gated delta rule on the tensor cores: tiles, descriptors, splittings shared
// by its forward and backward kernels.
//
// Every operand tile is 128 rows x 128 columns of 16-bit values in the
// 128-byte-swizzled layout (two blocks of 64 columns, 16 KB each); tiles in the
// workspace keep that layout, so that one 32 KB bulk copy brings or stores one.
// Head sizes below 128 run with zero columns.
//
// Precision.  States and the gates' gradients are float32 results, so products
// that reach them keep float32 accuracy although their operands are 16 bits
// wide.  Operands are fp16 after a scale by a power of two: bf16 inputs are then
// exact (over a range of 2^21 below the tile's largest value), and a float32
// operand is a sum of two parts of 11 bits, x = h + l.  A part l of a value of
// order 1 reaches down to 2^-24, so the pair is off by 2^-25 of the largest
// value's order; where one scale has to last over a whole sequence, l is kept
// 2^11 times larger, in a range of its own.  The products h h', h l' and l h' are
// accumulated in float32; l l' is below 2^-22 of the result.
//
// Range.  The recurrence does not change when a key is multiplied by c, its value and
// error by c and its beta by c^-2, and the chunks are computed in the form where every
// key has its largest element in [32, 64): k = p k', p a power of two per token, with
//   beta' = beta p^2,   v' = v / p,   e' = e / p,   u' = p u,   w' = w / p,   p beta w.
// A' = K' K'^T then has no entries but for |k'| in [32, 724], whatever the lengths of the
// keys, and with beta |k|^2 <= 2 (transitions that do not grow a state) an entry of the
// inverses is at most beta'_j |k'_i| |k'_j| <= 2 x 724 / 32.  (Keys shorter than 2^-12 of
// the chunk's longest keep that p, so that their v' does not push the others' out of
// range: an entry passes fp16's range when they are shorter than 2^-16.)  u and beta w
// are at most beta |k|_1 of a state's largest element (and beta of the largest value, far
// below a state's room), so u' and p beta w at most 2 |k'|_1 / |k'|^2 <= 2 x 11.4 / 32 of it
// and have the state's room.  Where they stand in fp16 alone or without a second
// range they carry one more power of two per chunk and head, eps (Tables), which brings the
// bound to 1, so that faint writes keep their digits.
#pragma once

#include <cuda_fp16.h>

#include "gdr.cuh"
#include "sm100.cuh"

namespace llattn {
namespace gdrtc {

using namespace sm100;

constexpr int kC = 128;                  // tokens per chunk (the MMA M)
constexpr uint32_t kHalf = kC * 128;     // [128 rows x 64] block: 16 KB
constexpr uint32_t kTile = 2 * kHalf;    // 32 KB
constexpr int kSlice = 32;               // d_v columns of a scan CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kTimeoutNs = 4000000000ull;
constexpr float kLoScale = 2048.f, kLoInv = 1.f / 2048.f;  // of the low fp16 part

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp of a difference of two log decays kept as pairs of floats
__device__ __forceinline__ float exp_diff(float2 a, float2 b) { return ex2(((a.x - b.x) + (a.y - b.y)) * kLog2e); }

// Wait until all but the latest committed group of bulk stores have read their source.
__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
// 32 lanes x 8 consecutive 32-bit columns (thread i: lane base + i).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void named_bar_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// The kernels of a call follow one another closely: each lets the next one be set up
// once all of its CTAs run, and the next waits (first of all, in every CTA, so that
// "before" holds along the whole chain) until the one before has ended and its writes
// can be read.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Bounded wait (every thread): the waits of these kernels are on their own
// copies and products, which always complete.
static __device__ __noinline__ void wait_bar_long(uint64_t* bar, uint32_t par, unsigned* err) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, par)) {
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      atomicOr(err, kErrTimeout);
      return;
    }
  }
}
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t par, unsigned* err) {
  if (!mbar_try_wait(bar, par)) wait_bar_long(bar, par, err);
}

// byte offset of the 16-byte piece c8 (columns 8 c8 ..) of row r of a tile
__device__ __forceinline__ uint32_t swz16(int r, int c8) {
  return (uint32_t)(c8 >> 3) * kHalf + (uint32_t)r * 128u + ((uint32_t)((c8 & 7) ^ (r & 7)) << 4);
}
// operand descriptors of k-step kk (16 elements): K along the columns, or K along the rows
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int kk) {
  return sw128_desc(tile + (kk >> 2) * kHalf + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int kk) { return sw128_desc(tile + kk * 2048, kHalf, 1024); }

// fp16 x fp16 -> float32, 128 x N
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool a_mn, bool b_mn) {
  return idesc_bf16(128, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// The preparation and the gradient run a long sequence of phases once per chunk
// by eight warps: their code is kept short (loops, functions that are not inlined),
// because unrolled it left the instruction cache and every phase waited for its
// own instructions (the solve below: 58 thousand cycles unrolled).

// How an operand of 128 x 128 lies in shared memory: in a tile with K along its
// columns or down its rows; in slice tiles, K along the columns, 32 of them in every
// 16 KB (16-bit parts of 64 bytes side by side in a row); in a plain tile, which is
// written straight to the workspace from registers: [piece of 8 columns][row][8], a warp's
// 16-byte stores to consecutive rows being 512 bytes in a row (with the swizzled
// rows each of the 32 was a line of its own: 240 ns more a chunk of the scan).
enum Lay : int { kAlong, kDown, kSlices, kPlain, kPlainDown };
__device__ __forceinline__ uint32_t plain16(int r, int c8) { return (uint32_t)c8 * 2048u + (uint32_t)r * 16u; }
// no swizzle: blocks of 8 rows x 16 bytes; `lbo` apart along K and `sbo` along M or N, for K down the rows likewise
__device__ __forceinline__ uint64_t plain_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (sw128_desc(saddr, lbo, sbo) & ~((uint64_t)7 << 61));
}
template <int L> __device__ __forceinline__ uint64_t desc_of(uint32_t tile) {
  return L == kDown ? desc_mn(tile, 0) : L == kPlain ? plain_desc(tile, 2048, 128)
         : L == kPlainDown ? plain_desc(tile, 128, 2048) : desc_k(tile, 0);
}
template <int L> __device__ __forceinline__ uint32_t step_of(int kk) {  // of the descriptor, to k-step kk
  return (L == kDown ? kk * 2048 : L == kPlain ? kk * 4096 : L == kPlainDown ? kk * 256
          : L == kSlices ? (kk >> 1) * kHalf + (kk & 1) * 32 : (kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
}
// D (+)= A B over 128 x 128 x 128 fp16.
// (Eight instructions of about 65 cycles; a loop over them took 140 each.)
template <int AL, int BL>
static __device__ __noinline__ void mma_tile(uint32_t d, uint32_t a, uint32_t b, bool add) {
  constexpr uint32_t id = idesc_f16(128, AL == kDown || AL == kPlainDown, BL == kDown || BL == kPlainDown);
  const uint64_t da = desc_of<AL>(a), db = desc_of<BL>(b);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) umma_bf16(d, da + step_of<AL>(kk), db + step_of<BL>(kk), id, (add || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
}

// 128 rows of a [.., d] bf16 matrix into a tile (columns from d on are zeros)
__device__ __forceinline__ void load_tile(unsigned char* tile, const CUtensorMap* map, int row, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, kTile);
  tma_load_2d(tile, map, bar, 0, row);
  tma_load_2d(tile + kHalf, map, bar, 64, row);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// x0, x1 as fp16; what is left of them, times `lo`, stays in x0, x1
__device__ __forceinline__ uint32_t take_f16x2(float& x0, float& x1, float lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  x0 = (x0 - f.x) * lo;
  x1 = (x1 - f.y) * lo;
  return *reinterpret_cast<const uint32_t*>(&h);
}
// eight columns (piece c8) of row i as the high parts in one tile and the low ones in another
__device__ __forceinline__ void put_parts(unsigned char* hi, unsigned char* lo, uint32_t at, float* x, float scale_lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = take_f16x2(x[2 * e], x[2 * e + 1], scale_lo);
    l[e] = pack_f16x2(x[2 * e], x[2 * e + 1]);
  }
  *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

// What is of the size of an inverse's entries (at most beta |k| |k|, mostly far below 1) is
// split into fp16 parts times this: the low part of a value below 1/4 would be
// subnormal, with an error of 2^-25 whatever the value (gate gradients 1.3e-6 off
// instead of 7e-7, B 2, T 4096).  Entries up to 1000 fit.
constexpr float kInvUp = 64.f;

// ---- the triangular solve, float32 values and sums.  With A = SL(K K^T . G)
// of a 128-token chunk, M solves (I + A diag(beta)) M = -A, so that both inverses
// are unit triangular and exact for any beta, zero and tiny ones included:
//   (I + A diag(beta))^-1 = I + M diag(beta),  (I + diag(beta) A)^-1 = I + diag(beta) M.
// (beta here carries the inverse of a scale that A is given.)  The 8 x 8 diagonal
// blocks by forward substitution (a column per thread), then four doublings: with
// both halves' M11 and M22 known,
//   Z = A21 + [M22 diag(beta)] A21,   M21 = -(Z + [Z diag(beta)] M11).
// From 16 rows on these are products of 16-row blocks on the warp-level matrix
// instruction, a 16 x (N / 2) piece to a warp, with both operands in two fp16 parts
// made in registers.  A chunk takes 12 thousand cycles, half of its preparation:
// 1.4 to the 8 x 8 pairs, then 1.5, 3.3 and 4.9 for the doublings, each a chain of loads,
// conversions and products (two schedulers' shares of the work made equal changed
// nothing).  The last one in float32 FMAs with 4 x 4 outputs a thread took 8 thousand
// (16-byte reads of shared memory, four cycles each, bound it), and on tcgen05 6:
// 0.85 for each product, the rest for operands through shared memory and back.
//
// Both matrices are [128][128] float32 with the 16-byte pieces of a row permuted
// by the row, which keeps reads of consecutive rows at one column, and of
// consecutive columns of one row, free of bank conflicts.
constexpr uint32_t kMatB = kC * kC * 4;
__device__ __forceinline__ int mat_at(int r, int c4) { return r * kC + ((c4 ^ (r & 7)) << 2); }
__device__ __forceinline__ float4& mat4(float* m, int r, int c4) { return *reinterpret_cast<float4*>(m + mat_at(r, c4)); }
__device__ __forceinline__ float2& mat2(float* m, int r, int c) {
  return *reinterpret_cast<float2*>(m + mat_at(r, c >> 2) + (c & 3));
}
__device__ __forceinline__ float mat1(const float* m, int r, int c) { return m[mat_at(r, c >> 2) + (c & 3)]; }

// d += a b, 16 x 8 x 16 fp16
__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, const uint32_t* b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// z[n] += X Y, 16 rows, K = 16, NT tiles of 8 columns; x: this lane's row and columns
// of X (xa: its two pieces), y[n][d]: its column of Y in row 2 t + d of the block
template <int NT> struct BlockRaw {
  float2 x[4], y[NT][2];
};
template <int NT>
__device__ __forceinline__ void block_load(BlockRaw<NT>& v, const float* x, const int* xa, const float* y,
                                           const int (*yc)[2]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v.x[e] = *reinterpret_cast<const float2*>(x + xa[e >> 1] + 8 * kC * (e & 1));
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) v.y[n][e] = make_float2(y[yc[n][0] + 8 * kC * e], y[yc[n][1] + 8 * kC * e]);
}
template <int NT>
__device__ __forceinline__ void block_mma(float (*z)[4], BlockRaw<NT>& v) {
  uint32_t ah[4], al[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ah[e] = take_f16x2(v.x[e].x, v.x[e].y, 1.f);
    al[e] = pack_f16x2(v.x[e].x, v.x[e].y);
  }
  uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      bh[n][e] = take_f16x2(v.y[n][e].x, v.y[n][e].y, 1.f);
      bl[n][e] = pack_f16x2(v.y[n][e].x, v.y[n][e].y);
    }
#pragma unroll
  for (int n = 0; n < NT; ++n) mma_16816(z[n], al, bh[n]);
#pragma unroll
  for (int n = 0; n < NT; ++n) mma_16816(z[n], ah, bl[n]);
#pragma unroll
  for (int n = 0; n < NT; ++n) mma_16816(z[n], ah, bh[n]);
}

// One doubling, N >= 16 rows to a half; the places of A's finished blocks hold
// kInvUp M diag(beta).  Eight warps, barrier kSolveBar: pair, 16-row block and half of
// the columns to each.
constexpr int kSolveBar = 1;
template <int N>
static __device__ __noinline__ void tri_double(float* Ap, float* Mp, const float* beta, int warp, int lane) {
  constexpr int RB = N / 16, NT = N / 16;  // row blocks; column tiles of a warp
  const int r0 = warp / (2 * RB) * 2 * N, rb = warp / 2 % RB, c = r0 + (warp & 1) * (N / 2);
  const int row = r0 + N + 16 * rb, g = lane >> 2, t = lane & 3;
  // (pieces are permuted by the row's low three bits, and blocks of 16 start at multiples of 4 pieces)
  const int xa[2] = {(((t >> 1) ^ (g & 3)) << 2) + 2 * (t & 1), ((((t >> 1) + 2) ^ (g & 3)) << 2) + 2 * (t & 1)};
  int yc[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int d = 0; d < 2; ++d)
      yc[n][d] = (2 * t + d) * kC + ((((c >> 2) + 2 * n + (g >> 2)) ^ (2 * t + d)) << 2) + (g & 3);
  auto x_at = [&](const float* m, int k) { return m + (row + g) * kC + (((k >> 2) ^ (g & 4)) << 2); };
  float z[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 x = mat2(Ap, row + g, c + 8 * n + 2 * t), y = mat2(Ap, row + g + 8, c + 8 * n + 2 * t);
    z[n][0] = kInvUp * x.x; z[n][1] = kInvUp * x.y; z[n][2] = kInvUp * y.x; z[n][3] = kInvUp * y.y;
  }
  BlockRaw<NT> cur, nxt;  // (the next block's values are on their way during this one's products)
  block_load<NT>(nxt, x_at(Ap, r0 + N), xa, Ap + (r0 + N) * kC, yc);
#pragma unroll 1
  for (int kb = 0; kb <= rb; ++kb) {
    cur = nxt;
    const int k = r0 + N + 16 * min(kb + 1, rb);
    block_load<NT>(nxt, x_at(Ap, k), xa, Ap + k * kC, yc);
    block_mma<NT>(z, cur);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 bt = *reinterpret_cast<const float2*>(beta + c + 8 * n + 2 * t);
    mat2(Mp, row + g, c + 8 * n + 2 * t) = make_float2(bt.x * z[n][0], bt.y * z[n][1]);
    mat2(Mp, row + g + 8, c + 8 * n + 2 * t) = make_float2(bt.x * z[n][2], bt.y * z[n][3]);
  }
  named_bar_sync(kSolveBar, 256);
  const int kb0 = (c - r0) / 16;
  block_load<NT>(nxt, x_at(Mp, r0 + 16 * kb0), xa, Mp + (r0 + 16 * kb0) * kC, yc);
#pragma unroll 1
  for (int kb = kb0; kb < RB; ++kb) {
    cur = nxt;
    const int k = r0 + 16 * min(kb + 1, RB - 1);
    block_load<NT>(nxt, x_at(Mp, k), xa, Mp + k * kC, yc);
    block_mma<NT>(z, cur);
  }
  named_bar_sync(kSolveBar, 256);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int cc = c + 8 * n + 2 * t;
    mat2(Mp, row + g, cc) = make_float2(-z[n][0] / kInvUp, -z[n][1] / kInvUp);
    mat2(Mp, row + g + 8, cc) = make_float2(-z[n][2] / kInvUp, -z[n][3] / kInvUp);
    if (N < 64) {
      const float2 bt = *reinterpret_cast<const float2*>(beta + cc);
      mat2(Ap, row + g, cc) = make_float2(-bt.x * z[n][0], -bt.y * z[n][1]);
      mat2(Ap, row + g + 8, cc) = make_float2(-bt.x * z[n][2], -bt.y * z[n][3]);
    }
  }
  named_bar_sync(kSolveBar, 256);
}

// 256 threads
static __device__ __noinline__ void tri_solve(float* Ap, float* Mp, const float* beta, int t) {
  if (t < 128) {
    const int r0 = t & ~7, cc = t & 7;
    float a[8][8], acc[8];
#pragma unroll
    for (int r = 1; r < 8; ++r)
#pragma unroll
      for (int v = 0; v < (r + 3) / 4; ++v) {
        const float4 x = mat4(Ap, r0 + r, (r0 >> 2) + v);
        a[r][4 * v] = x.x; a[r][4 * v + 1] = x.y; a[r][4 * v + 2] = x.z; a[r][4 * v + 3] = x.w;
      }
    acc[0] = 0.f;
#pragma unroll
    for (int r = 1; r < 8; ++r) {
      const float y = mat1(Ap, r0 + r, r0 + cc);
      acc[r] = r > cc ? -y : 0.f;
    }
    __syncwarp();  // (the block's columns are this warp's: all have read it)
    // once row m of the column is known, it goes into the rows below
#pragma unroll
    for (int m = 1; m < 7; ++m) {
      const float c = beta[r0 + m] * acc[m];  // (zero for m <= cc)
#pragma unroll
      for (int r = m + 1; r < 8; ++r) acc[r] = fmaf(-a[r][m], c, acc[r]);
    }
    const float bc = beta[r0 + cc];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int at = mat_at(r0 + r, (r0 + cc) >> 2) + (cc & 3);
      Mp[at] = acc[r];
      Ap[at] = kInvUp * bc * acc[r];
    }
    if (r0 & 8)  // zeros above the diagonal of the 16 x 16 block (A has them)
#pragma unroll
      for (int r = 0; r < 8; ++r) Mp[mat_at(r0 - 8 + r, (r0 + cc) >> 2) + (cc & 3)] = 0.f;
  } else {  // and of the 32 x 32 blocks: the last doubling's column halves begin with both
#pragma unroll
    for (int e = 0; e < 2; ++e)
      mat4(Mp, 32 * ((t - 128) >> 5) + (t & 15), 8 * ((t - 128) >> 5) + 4 + ((t >> 4) & 1) + 2 * e) =
          make_float4(0.f, 0.f, 0.f, 0.f);
  }
  named_bar_sync(kSolveBar, 256);
  {  // 8 x 8: a pair to a warp, two outputs to a thread
    const int r0 = 16 * (t >> 5), row = r0 + 8 + ((t >> 2) & 7), c = r0 + 2 * (t & 3);
    float2 z = mat2(Ap, row, c);
    z.x *= kInvUp;
    z.y *= kInvUp;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = mat1(Ap, row, r0 + 8 + k);
      const float2 b = mat2(Ap, r0 + 8 + k, c);
      z.x = fmaf(a, b.x, z.x);
      z.y = fmaf(a, b.y, z.y);
    }
    const float2 bt = *reinterpret_cast<const float2*>(beta + c);
    mat2(Mp, row, c) = make_float2(bt.x * z.x, bt.y * z.y);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = mat1(Mp, row, r0 + k);
      const float2 b = mat2(Mp, r0 + k, c);
      z.x = fmaf(a, b.x, z.x);
      z.y = fmaf(a, b.y, z.y);
    }
    __syncwarp();
    mat2(Mp, row, c) = make_float2(-z.x / kInvUp, -z.y / kInvUp);
    mat2(Ap, row, c) = make_float2(-bt.x * z.x, -bt.y * z.y);
  }
  named_bar_sync(kSolveBar, 256);
  tri_double<16>(Ap, Mp, beta, t >> 5, t & 31);
  tri_double<32>(Ap, Mp, beta, t >> 5, t & 31);
  tri_double<64>(Ap, Mp, beta, t >> 5, t & 31);
}

// The running log decay of the chunk's tokens (`la`: this thread's, the first 128
// threads) as pairs of floats: a scan of error-free sums, since log decays of a
// hundred tokens leave a float too few digits for their differences.  Ends in
// barrier `bar` of `threads`.
__device__ __forceinline__ void chunk_decays(float la, float2* g, float2* tot, int tid, int bar, int threads) {
  float2 x = make_float2(la, 0.f);
  if (tid < kC) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float2 y = make_float2(__shfl_up_sync(0xffffffffu, x.x, o), __shfl_up_sync(0xffffffffu, x.y, o));
      if ((tid & 31) >= o) x = pair_add(x, y);
    }
    if ((tid & 31) == 31) tot[tid >> 5] = x;
  }
  named_bar_sync(bar, threads);
  if (tid < kC) {
    for (int w = 0; w < (tid >> 5); ++w) x = pair_add(x, tot[w]);
    g[tid] = x;
  }
  named_bar_sync(bar, threads);
}

// the power of two that brings values up to `amax` to at most 16 (growth up to
// 4096 times stays in fp16's range), and its inverse
__device__ __forceinline__ float2 operand_scale(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent; 0 and 255 take no scale
  if (e == 0 || e >= 255) return make_float2(1.f, 1.f);
  const int s = min(max(257 - e, 1), 253);
  return make_float2(__uint_as_float((uint32_t)s << 23), __uint_as_float((uint32_t)(254 - s) << 23));
}

// Maxima of magnitudes that decide scales leave infinities and NaN out (a bad value must not
// take range from chunks that it does not reach): of the bits without the sign plus one step of
// the exponent, which wrap (float) or turn negative (bf16 pairs) for these.
constexpr uint32_t kNoMax = 0x01000000u, kNoMax2 = 0x00800080u;
__device__ __forceinline__ uint32_t max_finite(uint32_t m, float x) { return max(m, (__float_as_uint(x) << 1) + kNoMax); }
__device__ __forceinline__ uint32_t max_bits(uint32_t m) { return (m - kNoMax) >> 1; }
__device__ __forceinline__ uint32_t max_finite2(uint32_t m, uint32_t v) { return __vmaxs2(m, (v & 0x7fff7fffu) + kNoMax2); }
__device__ __forceinline__ uint32_t max_bits2(uint32_t m) { return max(m & 0xffffu, m >> 16) - 0x80u; }

// A bf16 tile in shared memory becomes fp16, scaled as above by its largest
// value; returns the inverse scale.  Rows from n on belong to
// other sequences: they become zeros, whatever they hold.  NT threads (`t` among
// them, barrier `bar`), the tile complete before; one barrier inside, none after.
template <int NT>
static __device__ __noinline__ float tile_to_f16(unsigned char* tile, int n, uint32_t* red, int t, int bar) {
  const bool in = (t & 127) < n;
  constexpr int PC = kC * 16 / NT;
  uint32_t m2 = kNoMax2;
#pragma unroll
  for (int c = 0; c < PC; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + swz16(t & 127, PC * (t >> 7) + c));
    m2 = max_finite2(max_finite2(max_finite2(max_finite2(m2, v.x), v.y), v.z), v.w);
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, in ? max_bits2(m2) : 0u);
  if ((t & 31) == 0) red[t >> 5] = m;
  named_bar_sync(bar, NT);
#pragma unroll
  for (int w = 0; w < NT / 128; ++w) {
    const uint4 x = *reinterpret_cast<const uint4*>(red + 4 * w);
    m = max(max(m, max(x.x, x.y)), max(x.z, x.w));
  }
  const float2 sc = operand_scale(__uint_as_float(m << 16));
#pragma unroll 2
  for (int c = 0; c < PC; ++c) {
    uint4* at = reinterpret_cast<uint4*>(tile + swz16(t & 127, PC * (t >> 7) + c));
    uint4 v = *at;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16x2(in ? w[e] : 0u);
      w[e] = pack_f16x2(sc.x * f.x, sc.x * f.y);
    }
    *at = v;
  }
  fence_proxy_async_shared();
  return sc.y;
}

// The same for K, a scale to each row, and the rows' sums of absolute values.  Thread =
// part of a row (NT / 128 neighbouring threads to a row, which take its pieces in an
// order that keeps a quarter of a warp free of bank conflicts).
struct Keys {
  float p, l1;  // of the thread's row: the inverse scale, the sum over the scaled row
  float p_all;  // the longest key's p
};
template <int NT> __device__ __forceinline__ int row_piece(int t, int c) {
  constexpr int W = NT / 128, PC = 16 / W;  // threads to a row, pieces to a thread
  const int part = t % W, turn = part >= W / 2 ? W == 2 ? 4 : 2 : 0;
  return PC * part + (c ^ turn);
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }
constexpr float kKeysUp = 4.f;  // rows of K go up to 64
constexpr float kShortest = 1.f / 4096.f;
template <int NT>
static __device__ __noinline__ Keys keys_to_f16(unsigned char* tile, int n, uint32_t* red, int t, int bar) {
  constexpr int W = NT / 128, PC = 16 / W;
  const int r = t / W;
  const bool in = r < n;
  uint32_t m2 = kNoMax2;
#pragma unroll
  for (int c = 0; c < PC; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + swz16(r, row_piece<NT>(t, c)));
    m2 = max_finite2(max_finite2(max_finite2(max_finite2(m2, v.x), v.y), v.z), v.w);
  }
  uint32_t row = in ? max_bits2(m2) : 0u;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) row = max(row, __shfl_xor_sync(0xffffffffu, row, o));
  uint32_t m = __reduce_max_sync(0xffffffffu, row);
  if ((t & 31) == 0) red[t >> 5] = m;
  named_bar_sync(bar, NT);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const uint4 x = *reinterpret_cast<const uint4*>(red + 4 * w);
    m = max(max(m, max(x.x, x.y)), max(x.z, x.w));
  }
  const float all = __uint_as_float(m << 16), own = __uint_as_float(row << 16);
  float2 sc = operand_scale(row == 0 ? all : fmaxf(own, all * kShortest));
  sc.x *= kKeysUp;
  sc.y /= kKeysUp;
  float sum = 0.f;
#pragma unroll 2
  for (int c = 0; c < PC; ++c) {
    uint4* at = reinterpret_cast<uint4*>(tile + swz16(r, row_piece<NT>(t, c)));
    uint4 v = *at;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float2 f = unpack_bf16x2(in ? w[e] : 0u);
      f.x *= sc.x;
      f.y *= sc.x;
      sum += fabsf(f.x) + fabsf(f.y);
      w[e] = pack_f16x2(f.x, f.y);
    }
    *at = v;
  }
#pragma unroll
  for (int o = 1; o < W; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  fence_proxy_async_shared();
  return Keys{sc.y, sum, operand_scale(all).y / kKeysUp};
}
// And for V / p, one scale to the tile; returns its inverse.  `p` is that of the thread's row,
// relative to the longest key's (1 to kShortest: kValuesDown keeps v / p below float's end whatever
// v is), `bits` those of the largest |v| that the thread's warp sees.
constexpr float kValuesDown = 1.f / 8192.f;
template <int NT>
static __device__ __noinline__ float values_to_f16(unsigned char* tile, int n, float p, uint32_t* red, int t, int bar,
                                            uint32_t* bits) {
  constexpr int W = NT / 128, PC = 16 / W;
  const int r = t / W;
  const bool in = r < n;
  uint32_t m2 = kNoMax2;
#pragma unroll
  for (int c = 0; c < PC; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + swz16(r, row_piece<NT>(t, c)));
    m2 = max_finite2(max_finite2(max_finite2(max_finite2(m2, v.x), v.y), v.z), v.w);
  }
  const uint32_t own = in ? max_bits2(m2) << 16 : 0u;
  const float ip = pow2_inverse(p) * kValuesDown;
  *bits = __reduce_max_sync(0xffffffffu, own);
  uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(__uint_as_float(own) * ip));
  if ((t & 31) == 0) red[t >> 5] = m;
  named_bar_sync(bar, NT);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const uint4 x = *reinterpret_cast<const uint4*>(red + 4 * w);
    m = max(max(m, max(x.x, x.y)), max(x.z, x.w));
  }
  const float2 sc = operand_scale(__uint_as_float(m));
#pragma unroll 2
  for (int c = 0; c < PC; ++c) {
    uint4* at = reinterpret_cast<uint4*>(tile + swz16(r, row_piece<NT>(t, c)));
    uint4 v = *at;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16x2(in ? w[e] : 0u);
      w[e] = pack_f16x2(ip * f.x * sc.x, ip * f.y * sc.x);
    }
    *at = v;
  }
  fence_proxy_async_shared();
  return sc.y / kValuesDown;
}
// the bits of a bound of a token's rows u' and p beta w: beta p |k|_1 of a state's largest element
// (|k|_1 = p l1) and beta p of the largest value, whose own scale leaves it 4096 times more room
__device__ __forceinline__ uint32_t rows_bound(float beta, float p, float l1) {
  return __float_as_uint(fabsf(beta) * p * fmaxf(p * l1, 1.f / 128.f));
}
template <int N> __device__ __forceinline__ uint32_t max_of(const uint32_t* x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, x[i]);
  return m;
}
// eps: the power of two that brings a bound of the rows u' of a chunk to at most 1
__device__ __forceinline__ float rows_scale(uint32_t bits) {
  const int e = (int)(bits >> 23);  // the bound is below 2^(e - 126)
  return e == 0 || e >= 255 ? 1.f : __uint_as_float((uint32_t)min(max(253 - e, 1), 187) << 23);
}

// the bits of the largest of a state's n values that this thread of `threads` sees
// (16 bytes a load: with four the 64 KB took longer than a chunk's solve)
static __device__ __noinline__ uint32_t state_max(const float* x, int n, int t, int threads) {
  uint32_t m = kNoMax;
#pragma unroll 4
  for (int e = t; e < n / 4; e += threads) {
    const float4 v = reinterpret_cast<const float4*>(x)[e];
    m = max_finite(max_finite(max_finite(max_finite(m, v.x), v.y), v.z), v.w);
  }
  return max_bits(m);
}

// rows 0 .. n - 1 of a tile of 16-bit values into a [.., d] matrix, whole rows to half a warp
static __device__ __noinline__ void store_rows(void* dst, const unsigned char* tile, int n, int d, int tid, int threads) {
  const int c8 = tid & 15;
  if (c8 * 8 < d)
#pragma unroll 4
    for (int r = tid >> 4; r < n; r += threads >> 4)
      *reinterpret_cast<uint4*>(static_cast<char*>(dst) + ((size_t)r * d + c8 * 8) * 2) =
          *reinterpret_cast<const uint4*>(tile + swz16(r, c8));
}

// ---- phases of the preparation; i: the thread's row, qt: its quarter of the columns
// M's row i, 32 columns (zero above the block on the diagonal)
__device__ __forceinline__ void load_m(float* m, float* Mp, int i, int qt) {
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (32 * qt + 4 * v <= (i | 15)) x = mat4(Mp, i, 8 * qt + v);
    m[4 * v] = x.x;
    m[4 * v + 1] = x.y;
    m[4 * v + 2] = x.z;
    m[4 * v + 3] = x.w;
  }
}
// rows of kInvUp (I + M diag(beta)) in two parts, and of that times diag(f2)
__device__ __forceinline__ void put_inverse2(unsigned char* t1, unsigned char* t2, const float* m, int i, int qt,
                                             const float* beta, const float* f2) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x[8], y[8];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int j = 32 * qt + 8 * c + 4 * v;
      const float4 b4 = *reinterpret_cast<const float4*>(beta + j), f4 = *reinterpret_cast<const float4*>(f2 + j);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w}, f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[4 * v + e] = j + e == i ? kInvUp : kInvUp * b[e] * m[8 * c + 4 * v + e];
        y[4 * v + e] = x[4 * v + e] * f[e];
      }
    }
    put_parts(t1, t1 + kTile, swz16(i, 4 * qt + c), x, 1.f);
    put_parts(t2, t2 + kTile, swz16(i, 4 * qt + c), y, 1.f);
  }
}
// rows of kInvUp diag(f) (I + diag(beta) M) in two parts
__device__ __forceinline__ void put_inverse(unsigned char* hi, unsigned char* lo, const float* m, int i, int qt, float f,
                                            float beta) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (32 * qt + 8 * c + e == i ? kInvUp : kInvUp * beta * m[8 * c + e]) * f;
    put_parts(hi, lo, swz16(i, 4 * qt + c), x, 1.f);
  }
}
// an accumulator's row, times f, as [slice of 32][piece of 4][row][4] floats; returns its largest value's bits
static __device__ __noinline__ uint32_t write_rows(float* dst, uint32_t acc, int i, int qt, float f) {
  uint32_t m = kNoMax;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float x[16];
    tmem_ld16(acc + 16 * c, x);
    tmem_ld_wait();
    float4* d = reinterpret_cast<float4*>(dst) + (size_t)(8 * qt + 4 * c) * kC + i;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float4 y = make_float4(f * x[4 * v], f * x[4 * v + 1], f * x[4 * v + 2], f * x[4 * v + 3]);
      m = max_finite(max_finite(max_finite(max_finite(m, y.x), y.y), y.z), y.w);
      d[v * kC] = y;
    }
  }
  return max_bits(m);
}
// an accumulator's row, times f, in two parts: tiles hi and lo, plain ones or not
template <bool PLAIN>
static __device__ __noinline__ void write_tiles(unsigned char* hi, unsigned char* lo, uint32_t acc, int i, int qt, float f,
                                         float scale_lo) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float x[16];
    tmem_ld16(acc + 16 * c, x);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] *= f;
    const int c8 = 4 * qt + 2 * c;
    put_parts(hi, lo, PLAIN ? plain16(i, c8) : swz16(i, c8), x, scale_lo);
    put_parts(hi, lo, PLAIN ? plain16(i, c8 + 1) : swz16(i, c8 + 1), x + 8, scale_lo);
  }
}
// exp(g_i - g_j) = exp(g_i - g_m) exp(g_m - g_j), m the first row of i's 32: one factor of
// the row and one of the column, both at most 1 for j < m (log decays are at most 0),
// so that only the 32 x 32 blocks on the diagonal take an exponential per element.
// The columns' factors: of row block q = 1, 2, 3 those of the columns below 32 q.
constexpr int kColDecays = 32 + 64 + 96;
__device__ __forceinline__ int col_at(int q) { return 16 * q * (q - 1); }
__device__ __forceinline__ void column_decays(float* cf, const float2* g, int tid) {  // 192 threads
  if (tid < kColDecays) {
    const int q = tid < 32 ? 1 : tid < 96 ? 2 : 3;
    cf[tid] = exp_diff(g[32 * q], g[tid - col_at(q)]);
  }
}
// x[k] = exp(g_i - g_{j0 + k}) for N columns of a row i in row block q (0 above the diagonal)
template <int N>
__device__ __forceinline__ void row_decays(float* x, const float* cf, const float2* gs, float2 gi, int i, int q, int j0) {
  if (j0 < 32 * q) {  // (warp-uniform)
    const float f = exp_diff(gi, gs[32 * q]);
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const float4 c = *reinterpret_cast<const float4*>(cf + col_at(q) + j0 + k);
      x[k] = f * c.x;
      x[k + 1] = f * c.y;
      x[k + 2] = f * c.z;
      x[k + 3] = f * c.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = j0 + k <= i ? exp_diff(gi, gs[j0 + k]) : 0.f;
  }
}

// 16 columns j0 .. of an accumulator's row i, times f exp(g_i - g_j), zero from the column `end` on
__device__ __forceinline__ void decayed16(float* x, uint32_t acc, const float* cf, const float2* gs, float2 gi, int i, int q,
                                          int j0, int end, float f) {
  float dec[16];
  row_decays<16>(dec, cf, gs, gi, i, q, j0);
  tmem_ld16(acc, x);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = j0 + j < end ? f * x[j] * dec[j] : 0.f;
}

}  // namespace gdrtc
}  // namespace llattn
