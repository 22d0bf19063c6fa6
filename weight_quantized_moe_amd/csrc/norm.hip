// Norms before and after a block, fused with the block's gate, the residual
// scale and the residual add (mq_norm in the C header states the formulas):
//   z  = x  or  x rsqrt(mean x^2 + eps) (offset + w_post)
//   r' = round(residual + scale gate z)
//   n  = bf16(r' rsqrt(mean r'^2 + eps) (offset + w_pre))
// One workgroup per row keeps the row in LDS in 32 bits between the steps, so
// every input is read once and every output written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"
#include "route.h"

namespace mq {

__device__ __forceinline__ float load_as_f32(const void *p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(((const uint16_t *)p)[i]) : ((const float *)p)[i];
}

// Sum of v over a workgroup of `waves` waves, in a fixed order; red: LDS floats.
__device__ __forceinline__ float block_sum(float v, float *red, int waves) {
  v = sum64f(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += red[w];
  return s;
}

__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  extern __shared__ __align__(16) float row[];  // [H]
  __shared__ float red[4];
  const int H = a.H, tid = threadIdx.x;
  const int64_t t = blockIdx.x, o = t * H;
  float ss = 0.f;
  if (a.x)
    for (int i = tid; i < H; i += 256) {
      const float v = bf16_to_f32(a.x[o + i]);
      row[i] = v;
      ss += v * v;
    }
  float inv = 1.f;
  if (a.post_w) inv = 1.f / sqrtf(block_sum(ss, red, 4) / H + a.eps);
  ss = 0.f;
  for (int i = tid; i < H; i += 256) {
    float v = 0.f;
    if (a.x) {
      v = row[i];
      if (a.post_w) v = v * inv * (a.offset + load_as_f32(a.post_w, a.w_bf16, i));
      if (a.gate_kind == MQ_GATE_CHANNEL) v *= load_as_f32(a.gate, a.gate_bf16, i);
      if (a.gate_kind == MQ_GATE_TOKEN) v *= load_as_f32(a.gate, a.gate_bf16, t);
      if (a.gate_kind == MQ_GATE_FULL) v *= load_as_f32(a.gate, a.gate_bf16, o + i);
      v *= a.scale;
    }
    if (a.residual) v = load_as_f32(a.residual, a.r_bf16, o + i) + v;
    if (a.r_bf16) {
      const uint16_t b = f32_to_bf16_rne(v);
      if (a.residual_out) ((uint16_t *)a.residual_out)[o + i] = b;
      v = bf16_to_f32(b);
    } else if (a.residual_out) {
      ((float *)a.residual_out)[o + i] = v;
    }
    row[i] = v;
    ss += v * v;
  }
  if (!a.norm_out) return;
  inv = 1.f / sqrtf(block_sum(ss, red, 4) / H + a.eps);
  for (int i = tid; i < H; i += 256)
    a.norm_out[o + i] = f32_to_bf16_rne(row[i] * inv * (a.offset + load_as_f32(a.pre_w, a.w_bf16, i)));
}

hipError_t launch_norm(const NormArgs &a, int64_t T, hipStream_t s) {
  const size_t lds = (size_t)a.H * 4;
  if (lds > 48 * 1024) raise_lds_limit((const void *)norm_kernel);
  hipLaunchKernelGGL(norm_kernel, dim3((unsigned)T), dim3(256), lds, s, a);
  return hipGetLastError();
}

}  // namespace mq
