// Queries, keys and values of new tokens on their way to the attention: the
// per-head norm, the position rotation, and the keys' and values' rows into
// their pages.  Bound by memory: every value is read and written once (16384 tokens
// of 32 + 2 x 4 heads of 128: 344 MB in 67 us, 5.1 TB/s; a large copy moves 5.4); for few
// tokens by the call (64 tokens: kernel 4 us, call 6.5).
//
// A head's row of D values lies on LP lanes (a power of two, at least D / 16),
// 16 values a lane in two groups of 8 (16 bytes each): where lane j turns pairs
// (i, i + R / 2) its groups are i = 8 j + [0, 8) and R / 2 + the same, so both
// partners of a pair are in one lane; elsewhere they are neighbours.  Either
// way the lane's 8 pairs have the angles 8 j + [0, 8).  The norm's sum of squares
// crosses the LP lanes.
//
// A wave takes 64 / LP heads of one token at a time, and with many tokens all of
// the token's heads one after the other, so that the angles (a row of the table is
// as long as one or two heads) and norm weights are read once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"

namespace mq {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

// Waves of a call at least, where there are that many groups of heads (3001 tokens of
// 72 heads: 16.5 us with 4096, 18.9 with a wave per group; 16384 of 40: 66.2 and 69.5).
constexpr int64_t kWaves = 4096;

__device__ __forceinline__ void widen8(u4 v, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
  }
}
// to nearest even, by the conversion instruction
__device__ __forceinline__ u4 narrow8(const float *f) {
  u4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b2 v;
    v[0] = (__bf16)f[2 * i];
    v[1] = (__bf16)f[2 * i + 1];
    o[i] = __builtin_bit_cast(uint32_t, v);
  }
  return o;
}
// v / s saturated to +-448, NaN kept: the rounded reciprocal y's quotient corrected by
// its remainder, which is v / s rounded (see quotient_by)
__device__ __forceinline__ float saturated(float v, float s, float y) {
  const float q = v * y, c = __builtin_fmaf(__builtin_fmaf(-q, s, v), y, q);
  const float w = fabsf(q) < 500.f ? c : q;
  return w != w ? w : __builtin_amdgcn_fmed3f(w, -448.f, 448.f);
}
// y: quotient_by(s)
__device__ __forceinline__ u2 codes8(const float *f, float s, float y) {
  float v[8];
  if (y != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = saturated(f[i], s, y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = f[i] / s;
      v[i] = w != w ? w : __builtin_amdgcn_fmed3f(w, -448.f, 448.f);
    }
  }
  u2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
    o[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
  }
  return o;
}

// parts: waves of a token, each with `turns` groups of 64 / LP heads
template <int LP, bool FP8>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, int parts, int turns) {
  constexpr int HPW = 64 / LP;
  const int wave = (int)(blockIdx.x * 4 + (threadIdx.x >> 6)), lane = threadIdx.x & 63, j = lane & (LP - 1);
  const int t = wave / parts, part = wave - t * parts;
  if (t >= a.T) return;
  const int heads = a.Hq + 2 * a.Hk;
  int h = part * turns * HPW + lane / LP;
  const bool live = 16 * j < a.D, turned = 16 * j < a.R;
  const int ta = turned && !a.interleaved ? 8 * j : 16 * j, tb = turned && !a.interleaved ? a.R / 2 + 8 * j : 16 * j + 8;
  // row h of the token: kind 0 query, 1 key, 2 value
  auto load = [&](int h, u4 &va, u4 &vb) {
    va = vb = u4{0u, 0u, 0u, 0u};
    if (h >= heads || !live) return;
    const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hk ? 1 : 2;
    const uint16_t *src = kind == 0   ? a.q + t * a.q_stride + h * a.D
                          : kind == 1 ? a.k + t * a.k_stride + (h - a.Hq) * a.D
                                      : a.v + t * a.v_stride + (h - a.Hq - a.Hk) * a.D;
    va = *(const u4 *)(src + (kind == 2 ? 16 * j : ta));
    vb = *(const u4 *)(src + (kind == 2 ? 16 * j + 8 : tb));
  };
  u4 va, vb;
  load(h, va, vb);
  const int slot = a.slots[t], pos = a.R ? a.positions[t] : 0;
  // padding: the same answer on the whole wave
  if (slot < 0 || slot >= a.num_slots || (a.R && (pos < 0 || pos >= a.max_positions))) return;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (turned) {
    const float *row = a.cos_sin + (int64_t)pos * a.R + 8 * j;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const f4 x = *(const f4 *)(row + i), y = *(const f4 *)(row + a.R / 2 + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[i + e] = x[e];
        s[i + e] = y[e];
      }
    }
  }
  u4 wq[2], wk[2];
  if (a.q_norm && live) {
    wq[0] = *(const u4 *)(a.q_norm + ta);
    wq[1] = *(const u4 *)(a.q_norm + tb);
  }
  if (a.k_norm && live) {
    wk[0] = *(const u4 *)(a.k_norm + ta);
    wk[1] = *(const u4 *)(a.k_norm + tb);
  }
  const int64_t page = slot >> a.page_log2, at = slot & ((1 << a.page_log2) - 1);
  const int last = min(heads, (part + 1) * turns * HPW);
  for (int h0 = part * turns * HPW; h0 < last; h0 += HPW, h += HPW) {
    float xa[8], xb[8];
    widen8(va, xa);
    widen8(vb, xb);
    if (h0 + HPW < last) load(h + HPW, va, vb);
    const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hk ? 1 : 2;
    const bool norm = kind == 0 ? a.q_norm != nullptr : kind == 1 && a.k_norm != nullptr;
    if (__any(norm)) {
      auto squares = [&]() {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += xa[i] * xa[i] + xb[i] * xb[i];
#pragma unroll
        for (int d = 1; d < LP; d *= 2) sum += __shfl_xor(sum, d, 64);
        return sum;
      };
      float sum = squares(), eps = a.eps;
      const bool large = norm && sum == INFINITY;
      if (__any(large)) {
        // values of 2^60 or more: 2^-70 of the head has the same norm, and squares in range
        const float k = large ? 0x1p-70f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xa[i] *= k;
          xb[i] *= k;
        }
        sum = squares();
        eps *= k * k;
      }
      if (norm) {
        const float f = 1.f / sqrtf(sum / (float)a.D + eps);
        float w[8];
        widen8(kind ? wk[0] : wq[0], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) xa[i] = xa[i] * f * w[i];
        widen8(kind ? wk[1] : wq[1], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) xb[i] = xb[i] * f * w[i];
      }
    }
    if (turned && kind < 2) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float *p = i < 4 ? xa + 2 * i : xb + 2 * (i - 4);
          const float u = p[0], v = p[1];
          p[0] = u * c[i] - v * s[i];
          p[1] = v * c[i] + u * s[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = xa[i], v = xb[i];
          xa[i] = u * c[i] - v * s[i];
          xb[i] = v * c[i] + u * s[i];
        }
      }
    }
    if (!live || h >= heads) continue;
    const int ia = kind == 2 ? 16 * j : ta, ib = kind == 2 ? 16 * j + 8 : tb;
    if (kind == 0) {
      uint16_t *o = a.q_out + ((int64_t)t * a.Hq + h) * a.D;
      *(u4 *)(o + ia) = narrow8(xa);
      *(u4 *)(o + ib) = narrow8(xb);
    } else {
      const int kh = h - a.Hq - (kind == 2 ? a.Hk : 0);
      const int64_t o = (((page * a.Hk + kh) << a.page_log2) + at) * a.D;
      void *cache = kind == 1 ? a.kc : a.vc;
      if constexpr (FP8) {
        const float sc = kind == 1 ? a.k_scale : a.v_scale, y = kind == 1 ? a.k_inv : a.v_inv;
        *(u2 *)((uint8_t *)cache + o + ia) = codes8(xa, sc, y);
        *(u2 *)((uint8_t *)cache + o + ib) = codes8(xb, sc, y);
      } else {
        *(u4 *)((uint16_t *)cache + o + ia) = narrow8(xa);
        *(u4 *)((uint16_t *)cache + o + ib) = narrow8(xb);
      }
    }
  }
}

template <int LP>
void run_append(const KvAppendArgs &a, hipStream_t s) {
  constexpr int HPW = 64 / LP;
  const int groups = (a.Hq + 2 * a.Hk + HPW - 1) / HPW;
  // a wave per group of heads while that makes few waves, then as many groups a wave as
  // leave kWaves of them
  const int want = (int)((kWaves + a.T - 1) / a.T), most_parts = want < groups ? want : groups;
  const int turns = (groups + most_parts - 1) / most_parts, parts = (groups + turns - 1) / turns;
  // T parts is below T + kWaves, so wave numbers and lanes stay in 32 bits
  const dim3 grid((unsigned)((a.T * parts + 3) / 4)), block(256);
  if (a.fp8) kv_append_kernel<LP, true><<<grid, block, 0, s>>>(a, parts, turns);
  else kv_append_kernel<LP, false><<<grid, block, 0, s>>>(a, parts, turns);
}

}  // namespace

// The rounded 1 / s where a quotient v / s follows from it (Markstein's theorem), 0 where
// the kernel has to divide: for a reciprocal that is infinite or subnormal, a remainder
// of a quotient that has a code (2^-11 s at least) below 2^-149, and a mantissa of s of
// all ones.
static float quotient_by(float s) {
  if (!(s >= 0x1p-90f && s <= 0x1p126f) || (__builtin_bit_cast(uint32_t, s) & 0x7FFFFFu) == 0x7FFFFFu) return 0.f;
  return 1.f / s;
}

hipError_t launch_kv_append(const KvAppendArgs &args, hipStream_t s) {
  KvAppendArgs a = args;
  a.k_inv = quotient_by(a.k_scale);
  a.v_inv = quotient_by(a.v_scale);
  if (a.D <= 16) run_append<1>(a, s);
  else if (a.D <= 32) run_append<2>(a, s);
  else if (a.D <= 64) run_append<4>(a, s);
  else if (a.D <= 128) run_append<8>(a, s);
  else run_append<16>(a, s);
  return hipGetLastError();
}

}  // namespace mq
