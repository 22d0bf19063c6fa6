// Device code of the routing stage shared by the softmax top-k kernels and the
// gated ones: lane reductions, the top-k over ordered logits, the staging of
// the hidden rows, and the grouping of (token, slot) pairs by expert in one
// workgroup.
#pragma once
#include "device.h"
#include "internal.h"

namespace mq {

// Order-preserving map of an IEEE float to an unsigned integer (every bit
// pattern, NaN included, gets a position in a total order).  -0 maps to the
// key of +0: the two are equal logits, so their order falls to the expert id.
__device__ __forceinline__ uint32_t ordered_key(float v) {
  uint32_t b = __builtin_bit_cast(uint32_t, v);
  if ((b << 1) == 0u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_ordered_key(uint32_t o) {
  uint32_t b = (o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o;
  return __builtin_bit_cast(float, b);
}

// DPP lane moves inside a 16-lane row (every lane has a valid source).
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  return v;
}
template <int kCtrl>
__device__ __forceinline__ float dppf(float v) {
  return __builtin_bit_cast(float, dpp<kCtrl>(__builtin_bit_cast(uint32_t, v)));
}
__device__ __forceinline__ float sum16(float v) {
  v += dppf<kXor1>(v);
  v += dppf<kXor2>(v);
  v += dppf<kHalfMirror>(v);
  v += dppf<kMirror>(v);
  return v;
}
__device__ __forceinline__ float max16f(float v) {
  v = fmaxf(v, dppf<kXor1>(v));
  v = fmaxf(v, dppf<kXor2>(v));
  v = fmaxf(v, dppf<kHalfMirror>(v));
  v = fmaxf(v, dppf<kMirror>(v));
  return v;
}

// Top-k + softmax of token t on the 16 lanes of one DPP row (li = lane % 16).
// Keys pack (ordered logit, ~expert id): the row maximum is the largest logit
// with the lowest id.  A selected key becomes 0, below every real key (the id
// half of a real key is never 0 since E <= 512), so the k winners are always k
// distinct valid experts.  Results go to ids/wts (and the probe arrays).
template <int kPer, bool kBf16Logits>
__device__ __forceinline__ void topk16_keys(const void *__restrict__ logits, int t, int E, int li,
                                            uint64_t *key) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = li + 16 * i;
    key[i] = 0;
    if (e < E) {
      float v;
      if (kBf16Logits)
        v = bf16_to_f32(((const uint16_t *)logits)[(size_t)t * E + e]);
      else
        v = ((const float *)logits)[(size_t)t * E + e];
      key[i] = ((uint64_t)ordered_key(v) << 32) | (uint32_t)(0xFFFFFFFFu - (uint32_t)e);
    }
  }
}
template <int kPer>
__device__ __forceinline__ void topk16_select(uint64_t *key, int t, int k, int li,
                                              int32_t *__restrict__ ids, float *__restrict__ wts,
                                              int32_t *__restrict__ p_ids, float *__restrict__ p_w) {
  float sv[4] = {0.f, 0.f, 0.f, 0.f};  // slot j = li + 16 s held by this lane
  int si[4] = {0, 0, 0, 0};
  float vmax = 0.f;
  // The 64-bit maximum taken as two 32-bit ones: the largest ordered logit,
  // then the largest id half among the keys that hold it (32-bit max
  // instructions, no 64-bit compare and select chains).
  uint32_t hi[kPer], lo[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    hi[i] = (uint32_t)(key[i] >> 32);
    lo[i] = (uint32_t)key[i];
  }
  for (int j = 0; j < k; ++j) {
    uint32_t hm = hi[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) hm = max(hm, hi[i]);
    hm = max16_u32(hm);
    uint32_t lm = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) lm = max(lm, hi[i] == hm ? lo[i] : 0u);
    lm = max16_u32(lm);
    const int e = (int)(0xFFFFFFFFu - lm);
    const float v = from_ordered_key(hm);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (li + 16 * i == e) hi[i] = lo[i] = 0u;
    if (j == 0) vmax = v;
    if ((j & 15) == li) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if ((j >> 4) == s) { sv[s] = v; si[s] = e; }
    }
  }
  float p[4], sum = 0.f;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    p[s] = (li + 16 * s < k) ? expf(sv[s] - vmax) : 0.f;
    sum += p[s];
  }
  sum = sum16(sum);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int j = li + 16 * s;
    if (j < k) {
      const float w = p[s] / sum;
      ids[(size_t)t * k + j] = si[s];
      wts[(size_t)t * k + j] = w;
      if (p_ids) p_ids[(size_t)t * k + j] = si[s];
      if (p_w) p_w[(size_t)t * k + j] = w;
    }
  }
}
template <int kPer, bool kBf16Logits>
__device__ __forceinline__ void topk16(const void *__restrict__ logits, int t, int E, int k, int li,
                                       int32_t *__restrict__ ids, float *__restrict__ wts,
                                       int32_t *__restrict__ p_ids, float *__restrict__ p_w) {
  uint64_t key[kPer];
  topk16_keys<kPer, kBf16Logits>(logits, t, E, li, key);
  topk16_select<kPer>(key, t, k, li, ids, wts, p_ids, p_w);
}

// Top-k + softmax of token t on all 64 lanes of one wave (batches of at most
// 4 tokens, one per wave; every lane of the wave active).  Lane l holds the
// keys of experts l + 64 i; a round takes the same two 32-bit maxima as
// topk16_select, each a DPP maximum inside the 16-lane rows followed by the
// maximum of the four row results read with v_readlane (wave-uniform).
__device__ __forceinline__ uint32_t max64_u32(uint32_t v) {
  v = max16_u32(v);  // every lane of a row holds the row maximum
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
  const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
  const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
  return max(max(a, b), max(c, d));
}
__device__ __forceinline__ float sum64f(float v) {
  v = sum16(v);
  const float a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 0));
  const float b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16));
  const float c = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 32));
  const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 48));
  return ((a + b) + c) + d;
}
template <int kPer64, bool kBf16Logits>
__device__ __forceinline__ void topk64(const void *__restrict__ logits, int t, int E, int k, int lane,
                                       int32_t *__restrict__ ids, float *__restrict__ wts,
                                       int32_t *__restrict__ p_ids, float *__restrict__ p_w) {
  uint32_t hi[kPer64], lo[kPer64];
#pragma unroll
  for (int i = 0; i < kPer64; ++i) {
    const int e = lane + 64 * i;
    hi[i] = lo[i] = 0u;
    if (e < E) {
      const float v = kBf16Logits ? bf16_to_f32(((const uint16_t *)logits)[(size_t)t * E + e])
                                  : ((const float *)logits)[(size_t)t * E + e];
      hi[i] = ordered_key(v);
      lo[i] = 0xFFFFFFFFu - (uint32_t)e;
    }
  }
  float sv = 0.f, vmax = 0.f;  // lane j < k keeps slot j
  int si = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t hm = hi[0];
#pragma unroll
    for (int i = 1; i < kPer64; ++i) hm = max(hm, hi[i]);
    hm = max64_u32(hm);
    uint32_t lm = 0u;
#pragma unroll
    for (int i = 0; i < kPer64; ++i) lm = max(lm, hi[i] == hm ? lo[i] : 0u);
    lm = max64_u32(lm);
    const int e = (int)(0xFFFFFFFFu - lm);
    const float v = from_ordered_key(hm);
#pragma unroll
    for (int i = 0; i < kPer64; ++i)
      if (lane + 64 * i == e) hi[i] = lo[i] = 0u;
    if (j == 0) vmax = v;
    if (j == lane) { sv = v; si = e; }
  }
  const float p = lane < k ? expf(sv - vmax) : 0.f;
  const float sum = sum64f(p);
  if (lane < k) {
    const float w = p / sum;
    ids[(size_t)t * k + lane] = si;
    wts[(size_t)t * k + lane] = w;
    if (p_ids) p_ids[(size_t)t * k + lane] = si;
    if (p_w) p_w[(size_t)t * k + lane] = w;
  }
}

// Hidden rows of the wave's 4 tokens -> FP16 scaled by a power of two each,
// using all 64 lanes per row.  With max|x| mapped into [2^14, 2^15), every BF16
// value of the row above max * 2^-31 converts to FP16 exactly (BF16 has 8
// significant bits, FP16 11, and the FP16 subnormal step there is 2^-24);
// smaller entries round with an absolute error below max * 2^-39.  The GEMMs
// multiply their result rows back by 2^s.  With kPermInt4 every 8 consecutive
// values are stored in the k order of the INT4 unpack ({0,4,1,5,2,6,3,7}, see
// unpack_int4), so INT4 GEMMs use the rows as they are.  Loads of the 4 rows
// are issued together (kChunk per row per round trip).
template <bool kPermInt4, bool kWriteRows = true>
__device__ __forceinline__ void rows_to_f16(const uint16_t *__restrict__ hidden, int t0, int T,
                                            int H, int lane, _Float16 *__restrict__ x16,
                                            float *__restrict__ rowscale) {
  constexpr int kChunk = 4;  // u4 per lane per row per round trip (2048 values)
  float m[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c0 = lane * 8; c0 < H; c0 += 512 * kChunk) {
    u4 v[4][kChunk];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < kChunk; ++u)
        if (t0 + r < T && c0 + 512 * u < H)
          v[r][u] = *(const u4 *)(hidden + (size_t)(t0 + r) * H + c0 + 512 * u);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < kChunk; ++u)
        if (t0 + r < T && c0 + 512 * u < H) m[r] = absmax_bf16x8(v[r][u], m[r]);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = max16f(m[r]);
    m[r] = fmaxf(m[r], __shfl_xor(m[r], 16, 64));
    m[r] = fmaxf(m[r], __shfl_xor(m[r], 32, 64));
  }
  float down[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int sh = row_shift(m[r]);
    down[r] = pow2f(-sh);
    if (lane == 0 && t0 + r < T) rowscale[t0 + r] = pow2f(sh);
  }
  if (!kWriteRows) return;  // the power of two only (decode)
  for (int c0 = lane * 8; c0 < H; c0 += 512 * kChunk) {
    u4 v[4][kChunk];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < kChunk; ++u)
        if (t0 + r < T && c0 + 512 * u < H)
          v[r][u] = *(const u4 *)(hidden + (size_t)(t0 + r) * H + c0 + 512 * u);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < kChunk; ++u)
        if (t0 + r < T && c0 + 512 * u < H) {
          const u4 o = bf16x8_to_f16x8(v[r][u], down[r]);
          *(u4 *)(x16 + (size_t)(t0 + r) * H + c0 + 512 * u) = kPermInt4 ? perm_0415(o) : o;
        }
  }
}

// W8A8: the wave's 4 hidden rows as dynamic 1x128 FP8 activations, codes
// [T, H] and FP32 scales [T, H/128].  Each pass covers 512 columns of a row:
// lane l holds columns 8 l + [0, 8), so the 16 lanes of a DPP row hold one
// 128-wide group, whose maximum is a 4-step DPP max.
__device__ __forceinline__ void rows_to_fp8(const uint16_t *__restrict__ hidden, int t0, int T,
                                            int H, int lane, uint8_t *__restrict__ xq,
                                            float *__restrict__ xs) {
  const int G = H / 128;
  for (int r = 0; r < 4; ++r) {
    const int t = t0 + r;
    if (t >= T) break;  // wave-uniform
    for (int c0 = 0; c0 < H; c0 += 512) {
      const int c = c0 + lane * 8;
      const bool ok = c < H;  // whole 16-lane groups (H is a multiple of 128)
      const u4 v = ok ? *(const u4 *)(hidden + (size_t)t * H + c) : u4{0u, 0u, 0u, 0u};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
        f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
      }
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
      m = max16f(m);
      const float s = fp8_group_scale(m);
      if (ok) {
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        *(u2 *)(xq + (size_t)t * H + c) = u2{e4m3x4(f[0], f[1], f[2], f[3], s), e4m3x4(f[4], f[5], f[6], f[7], s)};
        if ((lane & 15) == 0) xs[(size_t)t * G + c / 128] = s;
      }
    }
  }
}

// W4A4: the wave's 4 hidden rows as NVFP4 activations with global scale g
// (see nvfp4_act_scale), written as the FP16 values e2m1(code) * s into x16
// [T, H] (exact; natural k order, the NVFP4 GEMMs' operand order), with
// rowscale[t] = 1 / g for the GEMM to apply to its sums.  Each pass covers
// 512 columns of a row: lane l holds columns 8 l + [0, 8), so lanes 2i and
// 2i + 1 hold one group of 16.
__device__ __forceinline__ void rows_to_nvfp4(const uint16_t *__restrict__ hidden, int t0, int T,
                                              int H, int lane, float g, _Float16 *__restrict__ x16,
                                              float *__restrict__ rowscale) {
  for (int r = 0; r < 4; ++r) {
    const int t = t0 + r;
    if (t >= T) break;  // wave-uniform
    if (lane == 0) rowscale[t] = 1.f / g;
    for (int c0 = 0; c0 < H; c0 += 512) {
      const int c = c0 + lane * 8;
      const bool ok = c < H;  // whole 2-lane groups (H is a multiple of 128)
      const u4 v = ok ? *(const u4 *)(hidden + (size_t)t * H + c) : u4{0u, 0u, 0u, 0u};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
        f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
      }
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
      m = fmaxf(m, __shfl_xor(m, 1, 64));
      const Nvfp4Scale sc = nvfp4_act_scale(m, g);
      u4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const h2 pr = {(_Float16)(e2m1_value(e2m1_code(f[2 * i], g, sc.s)) * sc.s),
                       (_Float16)(e2m1_value(e2m1_code(f[2 * i + 1], g, sc.s)) * sc.s)};
        o[i] = as_u32(pr);
      }
      if (ok) *(u4 *)(x16 + (size_t)t * H + c) = o;
    }
  }
}

// Decode: only the power of two of each hidden row (rowscale[t] = 2^s), for
// the wave's 4 tokens (rows of H <= kRowRegsMaxH, read once into registers).  The
// decode gate/up GEMM scales the rows into FP16 itself while staging them.
__device__ __forceinline__ void row_scale_regs(const u4 (&v)[4][4], int t0, int T, int H, int lane,
                                               float *__restrict__ rowscale, float *down = nullptr) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (t0 + r < T && lane * 8 + 512 * u < H) m[r] = absmax_bf16x8(v[r][u], m[r]);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = max16f(m[r]);
    m[r] = fmaxf(m[r], __shfl_xor(m[r], 16, 64));
    m[r] = fmaxf(m[r], __shfl_xor(m[r], 32, 64));
    const int sh = row_shift(m[r]);
    if (lane == 0 && t0 + r < T) rowscale[t0 + r] = pow2f(sh);
    if (down) down[r] = pow2f(-sh);
  }
}

// ---------------------------------------------------------------------------
// Exclusive scan of cnt[0..E) (E <= 512) by one wave; also the prefill
// M-tile counts and the table of active experts.  Writes offsets[E+1],
// mtile[E+1], einfo ({count of active experts, their 16-row chunks}, then one
// {expert, first grouped row, rows, 0} entry per active expert in ascending
// expert order),
// rcp (per active expert, the prefix of the 16-row chunks of the experts
// before it, then the total: [count + 1] entries)
// and, if given, p_offsets.  Lanes hold 8 consecutive experts.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void scan_experts_wave(const int32_t *cnt, int E, int lane,
                                                  int32_t *__restrict__ offsets,
                                                  int32_t *__restrict__ mtile,
                                                  int4 *__restrict__ einfo,
                                                  int32_t *__restrict__ rcp,
                                                  int32_t *__restrict__ p_offsets,
                                                  int32_t *cursor) {
  int c[8], s0 = 0, s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    c[i] = e < E ? cnt[e] : 0;
    s0 += c[i];
    s1 += (c[i] + kPrefillBM - 1) / kPrefillBM;
    s2 += c[i] > 0;
    s3 += (c[i] + 15) >> 4;
  }
  int i0 = s0, i1 = s1, i2 = s2, i3 = s3;  // inclusive wave scans
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int a0 = __shfl_up(i0, d, 64), a1 = __shfl_up(i1, d, 64), a2 = __shfl_up(i2, d, 64);
    const int a3 = __shfl_up(i3, d, 64);
    if (lane >= d) { i0 += a0; i1 += a1; i2 += a2; i3 += a3; }
  }
  int r0 = i0 - s0, r1 = i1 - s1, r2 = i2 - s2, r3 = i3 - s3;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    if (e < E) {
      offsets[e] = r0;
      if (p_offsets) p_offsets[e] = r0;
      if (cursor) cursor[e] = r0;
      mtile[e] = r1;
      if (c[i] > 0) {
        einfo[1 + r2] = int4{e, r0, c[i], 0};
        rcp[r2] = r3;
      }
    }
    r0 += c[i];
    r1 += (c[i] + kPrefillBM - 1) / kPrefillBM;
    r2 += c[i] > 0;
    r3 += (c[i] + 15) >> 4;
  }
  if (lane == 63) {
    offsets[E] = i0;
    if (p_offsets) p_offsets[E] = i0;
    mtile[E] = i1;
    einfo[0] = int4{i2, i3, 0, 0};
    rcp[i2] = i3;
  }
}

// NTH threads of one workgroup group the T k (token, slot) pairs whose experts
// are ids[] (ids, wts and rowscale may be in LDS or global memory).
template <int NTH>
__device__ __forceinline__ void group_small_body(
    const int32_t *ids, const float *wts, const float *rowscale, int T, int E, int k,
    int32_t *__restrict__ offsets, int32_t *__restrict__ mtile, int4 *__restrict__ einfo,
    int32_t *__restrict__ rcp, int4 *__restrict__ rowinfo,
    int32_t *__restrict__ inv_pos, int32_t *__restrict__ p_offsets, int32_t *__restrict__ p_sorted_tok,
    int32_t *__restrict__ p_inv, int32_t *sm_ids) {
  __shared__ uint64_t mask[kMaxExperts * (kSmallT / 64)];  // [E][NW]
  __shared__ int32_t cnt[kMaxExperts];
  __shared__ int32_t off[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63;
  const int NW = (T + 63) >> 6;  // mask words per expert
  for (int i = tid; i < E * NW; i += NTH) mask[i] = 0ull;
  if (sm_ids != ids)
    for (int i = tid; i < T * k; i += NTH) sm_ids[i] = ids[i];
  __syncthreads();
  for (int i = tid; i < T * k; i += NTH) {
    const int tt = i / k;
    atomicOr(&mask[sm_ids[i] * NW + (tt >> 6)], 1ull << (tt & 63));
  }
  __syncthreads();
  for (int e = tid; e < E; e += NTH) {
    int c = 0;
    for (int w = 0; w < NW; ++w) c += __popcll(mask[e * NW + w]);
    cnt[e] = c;
  }
  __syncthreads();
  if (tid < 64) scan_experts_wave(cnt, E, lane, offsets, mtile, einfo, rcp, p_offsets, off);
  __syncthreads();
  for (int i = tid; i < T * k; i += NTH) {
    const int tt = i / k, e = sm_ids[i], tw = tt >> 6, tb = tt & 63;
    const uint64_t below = tb == 0 ? 0ull : (~0ull >> (64 - tb));
    int pos = off[e] + __popcll(mask[e * NW + tw] & below);
    for (int w = 0; w < tw; ++w) pos += __popcll(mask[e * NW + w]);
    const float rs = rowscale ? rowscale[tt] : 0.f;
    rowinfo[pos] = int4{i, tt, __builtin_bit_cast(int, rs), __builtin_bit_cast(int, wts[i])};
    inv_pos[i] = pos;
    if (p_sorted_tok) p_sorted_tok[pos] = tt;
    if (p_inv) p_inv[i] = pos;
  }
}

}  // namespace mq
