// The dense E4M3 product: y[t, n] = sum_g sa[t, g] sw[n / 128, g] sum_{k in g} a[t, k] w[n, k].
//
// Two launches: the rows' quantization into the workspace, and the product.
// Both operands of the product are E4M3 codes, so for a BF16 output one 16x16x128
// FP8 matrix instruction takes the whole inner sum of a block of 128 for 16
// weight rows and 16 tokens; the block's two scales multiply it in FP32 on the
// way into the accumulator.  That instruction aligns its 128 products to the
// largest and cuts them there: on random codes the sum is off by 2^-14 of the
// largest product in the mean and by 2^-10.8 at most, which a BF16 output does
// not show (an FP32 one does: 3e-5 of its 2-norm).  For an FP32 output the codes
// become FP16 values (exact) and go through four 16x16x32 FP16 instructions,
// whose sums are FP32 ones (2^-23.7 of the largest product in the mean), at half
// the rate.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"

namespace mq {
namespace {

typedef int i8v __attribute__((ext_vector_type(8)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// 16 weight rows (a) x 16 tokens (b) x 128 k; E8M0 scale 127 = 2^0 on both.
// Lane l holds row l % 16 of each operand and the same 32 of the 128 k (any,
// as long as both agree); of the result, token l % 16 and weight rows
// 4 (l / 16) + [0, 4).
__device__ __forceinline__ f4 mfma_fp8_16(const i8v &a, const i8v &b, const f4 &c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
}
__device__ __forceinline__ i8v join(u4 x, u4 y) {
  return i8v{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
}

__device__ __forceinline__ h8 half8(u4 c, int hi) { return unpack_fp8(c[2 * hi], c[2 * hi + 1]); }

// The inner sum of a block of 128: a = (a0, a1), b = (b0, b1) the lane's 32 codes.
template <bool kExact>
__device__ __forceinline__ f4 block_sum(u4 a0, u4 a1, u4 b0, u4 b1) {
  f4 p = {0.f, 0.f, 0.f, 0.f};
  if constexpr (kExact) {
#pragma unroll
    for (int i = 0; i < 2; ++i) p = mfma16(half8(a0, i), half8(b0, i), p);
#pragma unroll
    for (int i = 0; i < 2; ++i) p = mfma16(half8(a1, i), half8(b1, i), p);
    return p;
  } else {
    return mfma_fp8_16(join(a0, a1), join(b0, b1), p);
  }
}

// ---- quantization: 16 lanes take one block of 128 of one token, 8 values each
__global__ __launch_bounds__(256) void linear_quant_kernel(LinearArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t grp = id >> 4;
  if (grp >= a.T * a.G) return;  // 16 lanes at a time, so the shuffles below stay among live lanes
  const int64_t t = grp / a.G;
  const int g = (int)(grp - t * a.G), at = g * 128 + 8 * (int)(id & 15);
  const u4 v = at < a.K ? *(const u4 *)(a.x + t * a.K + at) : u4{0u, 0u, 0u, 0u};
  float m = absmax_bf16x8(v, 0.f);
#pragma unroll
  for (int s = 1; s < 16; s *= 2) m = fmaxf(m, __shfl_xor(m, s, 64));
  const float u = m * (1.f / 448.f), s = u > 0.f ? u : 1.f;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
  }
  *(u2 *)(a.codes + t * (a.G * (int64_t)128) + at) =
      u2{e4m3x4(f[0], f[1], f[2], f[3], s), e4m3x4(f[4], f[5], f[6], f[7], s)};
  if ((id & 15) == 0) a.sa[g * a.T + t] = s;
}

// out[t, n .. n + 4) = round(y + residual)
__device__ __forceinline__ void store4(const LinearArgs &a, int64_t t, int n, const float *y) {
  const int64_t at = t * a.N + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    float v = y[i];
    if (a.residual) v += bf16_to_f32(a.residual[at + i]);
    if (a.out_bf16)
      ((uint16_t *)a.out)[at + i] = f32_to_bf16_rne(v);
    else
      ((float *)a.out)[at + i] = v;
  }
}

// ---- the product: a workgroup of 4 waves takes 16 weight rows and 16 tokens,
// each wave every fourth block of K; operands straight from memory to registers.
template <bool kExact>
__global__ __launch_bounds__(256) void linear_stream_kernel(LinearArgs a) {
  __shared__ float part[4][64][4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int tiles = (a.N + 15) / 16;
  const int64_t tt = blockIdx.x / tiles;
  const int n0 = (int)(blockIdx.x - tt * tiles) * 16;
  const int64_t t = tt * 16 + r, tc = t < a.T ? t : a.T - 1;
  const int n = n0 + r < a.N ? n0 + r : a.N - 1;   // rows past the end: any row, never stored
  const uint8_t *wp = a.w + (int64_t)n * a.K, *xp = a.codes + tc * (a.G * (int64_t)128);
  const float *sw = a.scale + (int64_t)(n0 / 128) * a.G;
  f4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int g = wave; g < a.G; g += 4) {
    const int k0 = g * 128 + 16 * q, k1 = k0 + 64;
    // chunks past K: the codes are 0 there, so any chunk of the same weight row will do
    const u4 w0 = *(const u4 *)(wp + (k0 < a.K ? k0 : 0)), w1 = *(const u4 *)(wp + (k1 < a.K ? k1 : 0));
    const u4 x0 = *(const u4 *)(xp + k0), x1 = *(const u4 *)(xp + k1);
    const f4 p = block_sum<kExact>(w0, w1, x0, x1);
    const float s = a.sa[g * a.T + tc] * sw[g];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(p[i], s, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][lane][i] = acc[i];
  __syncthreads();
  if (wave == 0 && t < a.T) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (part[0][lane][i] + part[1][lane][i]) + (part[2][lane][i] + part[3][lane][i]);
    store4(a, t, n0 + 4 * q, y);
  }
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
  const int64_t quant = (a.T * a.G * 16 + 255) / 256, tiles = (int64_t)((a.N + 15) / 16) * ((a.T + 15) / 16);
  if (quant > 0x7FFFFFFF || tiles > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  linear_quant_kernel<<<dim3((unsigned)quant), dim3(256), 0, s>>>(a);
  if (a.out_bf16)
    linear_stream_kernel<false><<<dim3((unsigned)tiles), dim3(256), 0, s>>>(a);
  else
    linear_stream_kernel<true><<<dim3((unsigned)tiles), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace mq
