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

// Bounded wait (every thread): the waits of these kernels are on their own
// copies and products, which always complete.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t par, unsigned* err) {
  if (mbar_try_wait(bar, par)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, par)) {
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      atomicOr(err, kErrTimeout);
      return;
    }
  }
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

// D (+)= A B over 128 x 128 x 128 fp16; x_mn: that operand's K runs along its rows
__device__ __forceinline__ void mma_tile(uint32_t d, uint32_t a, bool a_mn, uint32_t b, bool b_mn, bool add) {
  const uint32_t id = idesc_f16(128, a_mn, b_mn);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    umma_bf16(d, a_mn ? desc_mn(a, kk) : desc_k(a, kk), b_mn ? desc_mn(b, kk) : desc_k(b, kk), id,
              (add || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16u : 0u));
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
}

// rows 0 .. n - 1 of a [.., d] bf16 matrix into a tile, zeros elsewhere (by
// all `threads` threads; rows that belong to another sequence stay out, so
// that nothing of theirs, a NaN say, is multiplied by a zero)
__device__ __forceinline__ void load_tile(unsigned char* tile, const __nv_bfloat16* src, int n, int d, int tid,
                                          int threads) {
  for (int x = tid; x < kC * 16; x += threads) {
    const int r = x >> 4, c8 = x & 15;
    const bool in = r < n && c8 * 8 < d;
    cp_async16_zfill(tile + swz16(r, c8), in ? src + (size_t)r * d + c8 * 8 : src, in);
  }
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

// ---- the triangular solve, float32 on the CUDA cores.  With A = SL(K K^T . G)
// of a 128-token chunk, M solves (I + A diag(beta)) M = -A, so that both inverses
// are unit triangular and exact for any beta, zero and tiny ones included:
//   (I + A diag(beta))^-1 = I + M diag(beta),  (I + diag(beta) A)^-1 = I + diag(beta) M.
// In 16 x 16 blocks: the diagonal blocks by forward substitution (a column per
// thread); Lam_IM = (I + M_II diag(beta)) A_IM in place of A; then block diagonal
// by block diagonal, a block per warp,
//   M_IJ = -(Lam_IJ + sum_{M=J}^{I-1} Lam_IM diag(beta) M_MJ).
constexpr int kBS = 20;  // row stride (floats) of a block: conflict-free 16-byte reads
constexpr uint32_t kBlocksB = 36 * 16 * kBS * 4;
__device__ __forceinline__ int blk(int I, int J) { return (I * (I + 1) / 2 + J) * 16 * kBS; }

__device__ __forceinline__ void tri_solve(float* Ap, float* Mp, const float* beta, int tid) {  // 256 threads, ends in a barrier
  const int warp = tid >> 5, lane = tid & 31;
  if (tid < 128) {
    const int I = tid >> 4, cc = tid & 15;
    const float* Ab = Ap + blk(I, I);
    float* Mb = Mp + blk(I, I);
    float col[16];  // beta_m M_mc
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float acc = 0.f;
      if (r > cc) {
        acc = -Ab[r * kBS + cc];
#pragma unroll
        for (int m = 0; m < 16; ++m)
          if (m > cc && m < r) acc = fmaf(-Ab[r * kBS + m], col[m], acc);
      }
      col[r] = beta[16 * I + r] * acc;
      Mb[r * kBS + cc] = acc;
    }
  }
  __syncthreads();
  const int r = lane >> 1, c0 = 8 * (lane & 1);
  // acc[x] += sum_k X[r][k] beta_k Y[k][c0 + x] over one block pair (beta: of X's columns)
  auto block_fma = [&](float* acc, const float* X, const float* bt, const float* Y) {
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {
      const float4 a = *reinterpret_cast<const float4*>(X + r * kBS + 4 * k4);
      const float4 bb = *reinterpret_cast<const float4*>(bt + 4 * k4);
      const float av[4] = {a.x * bb.x, a.y * bb.y, a.z * bb.z, a.w * bb.w};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float4 b0 = *reinterpret_cast<const float4*>(Y + (4 * k4 + kk) * kBS + c0);
        const float4 b1 = *reinterpret_cast<const float4*>(Y + (4 * k4 + kk) * kBS + c0 + 4);
        acc[0] = fmaf(av[kk], b0.x, acc[0]); acc[1] = fmaf(av[kk], b0.y, acc[1]);
        acc[2] = fmaf(av[kk], b0.z, acc[2]); acc[3] = fmaf(av[kk], b0.w, acc[3]);
        acc[4] = fmaf(av[kk], b1.x, acc[4]); acc[5] = fmaf(av[kk], b1.y, acc[5]);
        acc[6] = fmaf(av[kk], b1.z, acc[6]); acc[7] = fmaf(av[kk], b1.w, acc[7]);
      }
    }
  };
  auto load_row = [&](float* acc, const float* src) {
    const float4 a = *reinterpret_cast<const float4*>(src + r * kBS + c0);
    const float4 b = *reinterpret_cast<const float4*>(src + r * kBS + c0 + 4);
    acc[0] = a.x; acc[1] = a.y; acc[2] = a.z; acc[3] = a.w;
    acc[4] = b.x; acc[5] = b.y; acc[6] = b.z; acc[7] = b.w;
  };
  auto store_row = [&](float* dst, const float* acc, float sgn) {
    *reinterpret_cast<float4*>(dst + r * kBS + c0) = make_float4(sgn * acc[0], sgn * acc[1], sgn * acc[2], sgn * acc[3]);
    *reinterpret_cast<float4*>(dst + r * kBS + c0 + 4) =
        make_float4(sgn * acc[4], sgn * acc[5], sgn * acc[6], sgn * acc[7]);
  };
  for (int b = warp; b < 28; b += 8) {
    int I = 1, M = b;
    while (M >= I) { M -= I; ++I; }  // b enumerates (I, M), M < I, row by row
    float acc[8];
    load_row(acc, Ap + blk(I, M));
    block_fma(acc, Mp + blk(I, I), beta + 16 * I, Ap + blk(I, M));
    __syncwarp();
    store_row(Ap + blk(I, M), acc, 1.f);
  }
  __syncthreads();
  for (int d = 1; d < 8; ++d) {
    if (warp < 8 - d) {
      const int J = warp, I = J + d;
      float acc[8];
      load_row(acc, Ap + blk(I, J));
      for (int M = J; M < I; ++M) block_fma(acc, Ap + blk(I, M), beta + 16 * M, Mp + blk(M, J));
      store_row(Mp + blk(I, J), acc, -1.f);
    }
    __syncthreads();
  }
}

// The running log decay of the chunk's tokens as pairs of floats, by the first
// 128 threads (float64 scan); rows >= n add nothing.  Ends in a barrier.
__device__ __forceinline__ void chunk_decays(const float* log_alpha, int n, float2* g, double* tot, int tid) {
  double x = 0.0;
  if (tid < kC) {
    x = tid < n ? (double)gdr_log(log_alpha[tid]) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if ((tid & 31) >= o) x += y;
    }
    if ((tid & 31) == 31) tot[tid >> 5] = x;
  }
  __syncthreads();
  if (tid < kC) {
    for (int w = 0; w < (tid >> 5); ++w) x += tot[w];
    const float hi = (float)x;
    g[tid] = make_float2(hi, (float)(x - (double)hi));
  }
  __syncthreads();
}

// the power of two that brings values up to `amax` to at most 16 (growth up to
// 4096 times stays in fp16's range), and its inverse
__device__ __forceinline__ float2 operand_scale(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent; 0 and 255 take no scale
  if (e == 0 || e >= 255) return make_float2(1.f, 1.f);
  const int s = min(max(257 - e, 1), 253);
  return make_float2(__uint_as_float((uint32_t)s << 23), __uint_as_float((uint32_t)(254 - s) << 23));
}

// A bf16 tile in shared memory becomes fp16, scaled as above by its largest
// value; returns the inverse scale (and that value's bits).  256 threads, the
// tile complete before; one barrier inside, none after.
__device__ __forceinline__ float tile_to_f16(unsigned char* tile, uint32_t* red, int tid, uint32_t* bits = nullptr) {
  unsigned char* at[8];
  uint4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    at[c] = tile + swz16(tid & 127, 8 * (tid >> 7) + c);
    v[c] = *reinterpret_cast<const uint4*>(at[c]);
    const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, red[w]);
  m <<= 16;
  if (bits) *bits = m;
  const float2 sc = operand_scale(__uint_as_float(m));
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v[c]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16x2(w[e]);
      w[e] = pack_f16x2(sc.x * f.x, sc.x * f.y);
    }
    *reinterpret_cast<uint4*>(at[c]) = v[c];
  }
  fence_proxy_async_shared();
  return sc.y;
}

}  // namespace gdrtc
}  // namespace llattn
