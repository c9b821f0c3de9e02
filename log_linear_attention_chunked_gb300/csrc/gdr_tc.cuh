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
// wide: an operand that is not exact in bf16 is a sum of parts,
//   bf16 x 3:  x = h + m + l, 8 bits each (any range), or
//   fp16 x 2:  x = h + l / 2^11, 11 bits each, after a power-of-two scale,
// and the products of the parts are accumulated in float32.
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

__host__ __device__ constexpr uint32_t idesc(bool bf16, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(128, N, a_mn, b_mn) & ~(bf16 ? 0u : ((1u << 7) | (1u << 10)));
}

// D (+)= A B over 128 x 128 x 128 bf16; x_mn: that operand's K runs along its rows
__device__ __forceinline__ void mma_tile(uint32_t d, uint32_t a, bool a_mn, uint32_t b, bool b_mn, bool add) {
  const uint32_t id = idesc(true, 128, a_mn, b_mn);
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

// x0, x1 -> two packed 16-bit values; the rest is left in x0, x1
__device__ __forceinline__ uint32_t take_bf16x2(float& x0, float& x1) {
  const uint32_t u = pack_bf16x2(x0, x1);
  x0 -= __uint_as_float(u << 16);
  x1 -= __uint_as_float(u & 0xffff0000u);
  return u;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t take_f16x2(float& x0, float& x1) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  x0 = (x0 - f.x) * kLoScale;
  x1 = (x1 - f.y) * kLoScale;
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- the triangular inverse, float32 on the CUDA cores: T = (I + L)^-1 of a
// 128 x 128 strictly lower L in 16 x 16 blocks.  Row block I of (I + L) T = I
// gives T_IJ = -T_II sum_{M=J}^{I-1} L_IM T_MJ (J < I): the diagonal blocks by
// forward substitution (a column per thread), Lam_IM = T_II L_IM over L's
// blocks, then the block diagonals below, a block per warp.
constexpr int kBS = 20;  // row stride (floats) of a block: conflict-free 16-byte reads
constexpr uint32_t kBlocksB = 36 * 16 * kBS * 4;
__device__ __forceinline__ int blk(int I, int J) { return (I * (I + 1) / 2 + J) * 16 * kBS; }

__device__ __forceinline__ void tri_inverse(float* Lp, float* Tp, int tid) {  // 256 threads, ends in a barrier
  const int warp = tid >> 5, lane = tid & 31;
  if (tid < 128) {
    const int I = tid >> 4, cc = tid & 15;
    const float* Lb = Lp + blk(I, I);
    float* Tb = Tp + blk(I, I);
    float col[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float acc = r == cc ? 1.f : 0.f;
      if (r > cc) {
#pragma unroll
        for (int m = 0; m < 16; ++m)
          if (m >= cc && m < r) acc = fmaf(-Lb[r * kBS + m], col[m], acc);
      }
      col[r] = acc;
      Tb[r * kBS + cc] = acc;
    }
  }
  __syncthreads();
  const int r = lane >> 1, c0 = 8 * (lane & 1);
  auto block_fma = [&](float* acc, const float* A, const float* B) {
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {
      const float4 a = *reinterpret_cast<const float4*>(A + r * kBS + 4 * k4);
      const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float4 b0 = *reinterpret_cast<const float4*>(B + (4 * k4 + kk) * kBS + c0);
        const float4 b1 = *reinterpret_cast<const float4*>(B + (4 * k4 + kk) * kBS + c0 + 4);
        acc[0] = fmaf(av[kk], b0.x, acc[0]); acc[1] = fmaf(av[kk], b0.y, acc[1]);
        acc[2] = fmaf(av[kk], b0.z, acc[2]); acc[3] = fmaf(av[kk], b0.w, acc[3]);
        acc[4] = fmaf(av[kk], b1.x, acc[4]); acc[5] = fmaf(av[kk], b1.y, acc[5]);
        acc[6] = fmaf(av[kk], b1.z, acc[6]); acc[7] = fmaf(av[kk], b1.w, acc[7]);
      }
    }
  };
  auto store_row = [&](float* dst, const float* acc, float sgn) {
    *reinterpret_cast<float4*>(dst + r * kBS + c0) = make_float4(sgn * acc[0], sgn * acc[1], sgn * acc[2], sgn * acc[3]);
    *reinterpret_cast<float4*>(dst + r * kBS + c0 + 4) =
        make_float4(sgn * acc[4], sgn * acc[5], sgn * acc[6], sgn * acc[7]);
  };
  for (int b = warp; b < 28; b += 8) {
    int I = 1, M = b;
    while (M >= I) { M -= I; ++I; }  // b enumerates (I, M), M < I, row by row
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    block_fma(acc, Tp + blk(I, I), Lp + blk(I, M));
    __syncwarp();
    store_row(Lp + blk(I, M), acc, 1.f);
  }
  __syncthreads();
  for (int d = 1; d < 8; ++d) {
    if (warp < 8 - d) {
      const int J = warp, I = J + d;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int M = J; M < I; ++M) block_fma(acc, Lp + blk(I, M), Tp + blk(M, J));
      store_row(Tp + blk(I, J), acc, -1.f);
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

}  // namespace gdrtc
}  // namespace llattn
