// Queries, keys and values of new tokens on their way to the attention: the
// per-head norm, the position rotation, and the keys' and values' rows into
// their pages.  Bound by memory: every value is read and written once.
//
// A head's row of D values lies on LP lanes (a power of two, at least D / 16),
// 16 values a lane in two groups of 8 (16 bytes each): where lane j turns pairs
// (i, i + R / 2) its groups are i = 8 j + [0, 8) and R / 2 + the same, so both
// partners of a pair are in one lane; elsewhere they are neighbours.  Either
// way the lane's 8 pairs have the angles 8 j + [0, 8).  The norm's sum of squares
// crosses the LP lanes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"

namespace mq {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));

struct Row16 {
  float a[8], b[8];
};

__device__ __forceinline__ void widen8(u4 v, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
  }
}
__device__ __forceinline__ u4 narrow8(const float *f) {
  u4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)f32_to_bf16_rne(f[2 * i]) | ((uint32_t)f32_to_bf16_rne(f[2 * i + 1]) << 16);
  return o;
}
// RNE-to-E4M3(v / s) saturated to +-448, NaN kept
__device__ __forceinline__ float saturate(float v, float s) {
  const float q = v / s;
  return q != q ? q : fminf(fmaxf(q, -448.f), 448.f);
}
__device__ __forceinline__ u2 codes8(const float *f, float s) {
  u2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(f[4 * i], s), saturate(f[4 * i + 1], s), 0, false);
    o[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(saturate(f[4 * i + 2], s), saturate(f[4 * i + 3], s), w, true);
  }
  return o;
}

__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, int lp) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / lp;
  const int j = (int)(id & (lp - 1)), heads = a.Hq + 2 * a.Hk;
  const int64_t t = row / heads;
  if (t >= a.T) return;  // LP lanes at a time: the sum below stays among live lanes
  const int h = (int)(row - t * heads);
  const int slot = a.slots[t];
  const int pos = a.R ? a.positions[t] : 0;
  // padding: the same answer on all of a row's lanes
  if (slot < 0 || slot >= a.num_slots || (a.R && (pos < 0 || pos >= a.max_positions))) return;
  const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk, live = 16 * j < a.D;
  const int kh = is_q ? h : is_k ? h - a.Hq : h - a.Hq - a.Hk;
  const uint16_t *src = is_q ? a.q + t * a.q_stride : is_k ? a.k + t * a.k_stride : a.v + t * a.v_stride;
  src += (int64_t)kh * a.D;
  const bool turns = (is_q || is_k) && 16 * j < a.R;
  int ia = 16 * j, ib = 16 * j + 8;
  if (turns && !a.interleaved) {
    ia = 8 * j;
    ib = a.R / 2 + 8 * j;
  }
  Row16 x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x.a[i] = x.b[i] = 0.f;
  if (live) {
    widen8(*(const u4 *)(src + ia), x.a);
    widen8(*(const u4 *)(src + ib), x.b);
  }
  const uint16_t *norm = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
  if (norm) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x.a[i] * x.a[i] + x.b[i] * x.b[i];
    for (int d = 1; d < lp; d *= 2) s += __shfl_xor(s, d, 64);
    const float f = 1.f / sqrtf(s / (float)a.D + a.eps);
    if (live) {
      float w[8];
      widen8(*(const u4 *)(norm + ia), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x.a[i] = x.a[i] * f * w[i];
      widen8(*(const u4 *)(norm + ib), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x.b[i] = x.b[i] * f * w[i];
    }
  }
  if (turns) {
    const float *c = a.cos_sin + (int64_t)pos * a.R + 8 * j, *s = c + a.R / 2;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float *p = i < 4 ? x.a + 2 * i : x.b + 2 * (i - 4);
        const float u = p[0], v = p[1];
        p[0] = u * c[i] - v * s[i];
        p[1] = v * c[i] + u * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x.a[i], v = x.b[i];
        x.a[i] = u * c[i] - v * s[i];
        x.b[i] = v * c[i] + u * s[i];
      }
    }
  }
  if (!live) return;
  if (is_q) {
    uint16_t *o = a.q_out + (t * a.Hq + kh) * a.D;
    *(u4 *)(o + ia) = narrow8(x.a);
    *(u4 *)(o + ib) = narrow8(x.b);
    return;
  }
  const int64_t page = slot >> a.page_log2, at = slot & ((1 << a.page_log2) - 1);
  const int64_t o = (((page * a.Hk + kh) << a.page_log2) + at) * a.D;
  void *cache = is_k ? a.kc : a.vc;
  if (a.fp8) {
    const float s = is_k ? a.k_scale : a.v_scale;
    *(u2 *)((uint8_t *)cache + o + ia) = codes8(x.a, s);
    *(u2 *)((uint8_t *)cache + o + ib) = codes8(x.b, s);
  } else {
    *(u4 *)((uint16_t *)cache + o + ia) = narrow8(x.a);
    *(u4 *)((uint16_t *)cache + o + ib) = narrow8(x.b);
  }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s) {
  int lp = 1;
  while (lp * 16 < a.D) lp *= 2;
  // rows of all tokens: at most 2^24 workgroups a launch
  const int64_t heads = a.Hq + 2 * a.Hk, most = ((int64_t)1 << 24) * 256 / lp / heads;
  for (int64_t t = 0; t < a.T; t += most) {
    KvAppendArgs p = a;
    p.T = a.T - t < most ? a.T - t : most;
    p.q += t * a.q_stride; p.k += t * a.k_stride; p.v += t * a.v_stride;
    p.slots += t;
    if (p.positions) p.positions += t;
    p.q_out += t * a.Hq * a.D;
    const int64_t blocks = (p.T * heads * lp + 255) / 256;
    kv_append_kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(p, lp);
  }
  return hipGetLastError();
}

}  // namespace mq
