// Gated routing: softmax or sigmoid scores, a balance bias that takes part in
// the selection only, groups of experts of which a few are kept, top-k,
// renormalised or raw weights (mq_gate in the C header states the formulas).
//
// The order of two selection scores next to each other decides which expert a
// token takes, so the selection runs on 64-bit scores: sigmoid(l) + bias
// rounds at 2^-54 there, against gaps of 2^-24 and less that a 32-bit score
// cannot tell apart.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"
#include "route.h"

namespace mq {

// Order-preserving map of a double to an unsigned integer; -0 maps to the key
// of +0, and no key of a number is 0 (the key of a selected or excluded expert).
__device__ __forceinline__ uint64_t ordered_key64(double v) {
  uint64_t b = __builtin_bit_cast(uint64_t, v);
  if ((b << 1) == 0ull) b = 0ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// A logit as the gate reads it: NaN counts as -inf (masked), +inf as the
// largest finite value.
__device__ __forceinline__ float gate_logit(float v) {
  v = v == v ? v : -INFINITY;
  return fminf(v, 3.402823466e38f);
}
__device__ __forceinline__ float load_gate_logit(const void *logits, int bf16, int64_t i) {
  return gate_logit(bf16 ? bf16_to_f32(((const uint16_t *)logits)[i]) : ((const float *)logits)[i]);
}

__device__ __forceinline__ uint64_t max64_u64(uint64_t v) {
  const uint32_t hi = max64_u32((uint32_t)(v >> 32));
  const uint32_t lo = max64_u32((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float max64f(float v) {
  v = max16f(v);
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}

// Weight of the slot a lane holds (wave-wide; l = -inf where the expert is
// masked or the lane has no slot).  m and z: softmax maximum and sum over all
// experts.  Written so that nothing overflows and small scores keep their
// digits: sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), and a renormalised row
// is shifted by its largest logit first.
__device__ __forceinline__ float gate_weight(const GateArgs &g, float l, float m, float z) {
  const float top = g.renormalize ? max64f(l) : 0.f;  // -inf where every slot is masked
  float s = 0.f;
  if (l > -INFINITY) {
    if (g.score == MQ_SCORE_SIGMOID)
      s = expf(fminf(l, 0.f) - (g.renormalize ? fminf(top, 0.f) : 0.f)) / (1.f + expf(-fabsf(l)));
    else
      s = g.renormalize ? expf(l - top) : expf(l - m) / z;
  }
  if (g.renormalize) {
    const float sum = sum64f(s);
    s = sum > 0.f ? s / sum : 0.f;
  }
  return s * g.scale;
}

// The power of two that brings a token's largest weight into [2^-1, 1).
__device__ __forceinline__ float weight_scale(float m) {
  if (!(m > 0.f)) return 1.f;
  const int ex = (int)(__builtin_bit_cast(uint32_t, m) >> 23) - 126;
  return pow2f(ex < -120 ? -120 : ex > 120 ? 120 : ex);
}

// Orders a wave's LDS writes before its reads of other lanes' values.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The gate of one token on all 64 lanes of a wave, in 64 bits; any number of
// groups.  Lane l holds experts l + 64 i.  sc: one double per expert, LDS of
// this wave alone.
template <int kPer>
__device__ __forceinline__ void gate_token(const GateArgs &g, const void *__restrict__ logits, int bf16, int64_t t,
                                           int lane, double *sc, const GateOut &o) {
  float l[kPer];
  uint64_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < g.E ? load_gate_logit(logits, bf16, t * g.E + e) : -INFINITY;
  }
  // softmax statistics over the live logits (M = 0 where there is none)
  float m = l[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) m = fmaxf(m, l[i]);
  m = max64f(m);
  if (m == -INFINITY) m = 0.f;
  double z = 0.0;
  if (g.score == MQ_SCORE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) z += exp((double)l[i] - (double)m);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) z += __shfl_xor(z, d, 64);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    key[i] = 0ull;
    if (e < g.E) {
      const float b = g.bias ? g.bias[e] : 0.f;
      const bool live = l[i] > -INFINITY && b > -INFINITY;
      double c = -INFINITY;
      // without a bias the order is the logits' own; the score itself is
      // needed for sums of two only
      if (live)
        c = !g.bias && g.group_top == 1 ? (double)l[i]
            : g.score == MQ_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)l[i])) + (double)b
                                          : exp((double)l[i] - (double)m) / z + (double)b;
      sc[e] = c;
      if (live && !g.bias) c = (double)l[i];
      key[i] = ordered_key64(c);
    }
  }
  if (g.groups > 1) {
    // lane = group: its score, then the number of groups that come before it
    wave_lds_fence();
    double s1 = -INFINITY, s2 = -INFINITY;
    if (lane < g.groups)
      for (int i = 0; i < g.per; ++i) {
        const double v = sc[lane * g.per + i];
        s2 = fmax(s2, fmin(s1, v));
        s1 = fmax(s1, v);
      }
    const double s = g.group_top == 2 ? s1 + s2 : s1;
    const uint64_t gk = lane < g.groups ? ordered_key64(s) : 0ull;
    int before = 0;
    for (int j = 0; j < g.groups; ++j) {
      const uint64_t o = __shfl(gk, j, 64);
      before += o > gk || (o == gk && j < lane);
    }
    const uint64_t kept = __ballot(lane < g.groups && before < g.topk_groups);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 64 * i;
      if (e < g.E && !((kept >> (e / g.per)) & 1ull)) key[i] = 0ull;
    }
  }
  int slot_id = 0;
  for (int j = 0; j < g.k; ++j) {
    uint64_t km = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) km = key[i] > km ? key[i] : km;
    km = max64_u64(km);
    uint32_t lo = 0u;  // ~id of the lowest expert that holds the maximum
#pragma unroll
    for (int i = 0; i < kPer; ++i) lo = max(lo, key[i] == km ? 0xFFFFFFFFu - (uint32_t)(lane + 64 * i) : 0u);
    const int e = (int)(0xFFFFFFFFu - max64_u32(lo));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 64 * i == e) key[i] = 0ull;
    if (j == lane) slot_id = e;
  }
  // weights of the k slots (lane = slot), in 32 bits
  float lw = -INFINITY;
  if (lane < g.k) {
    lw = load_gate_logit(logits, bf16, t * g.E + slot_id);
    const float b = g.bias ? g.bias[slot_id] : 0.f;
    if (!(b > -INFINITY)) lw = -INFINITY;
  }
  const float w = gate_weight(g, lw, m, (float)z);
  float ws = 1.f;
  if (o.wscale) {
    ws = weight_scale(max64f(fabsf(w)));
    if (lane == 0) o.wscale[t] = ws;
  }
  if (lane < g.k) {
    const int64_t at = t * g.k + lane;
    o.ids[at] = slot_id;
    o.wts[at] = w / ws;  // exact: ws is a power of two
    if (o.p_ids) o.p_ids[at] = slot_id;
    if (o.p_w) o.p_w[at] = w;
  }
}

template <int kPer>
__global__ __launch_bounds__(256) void gate_topk_kernel(GateArgs g, const void *__restrict__ logits, int bf16,
                                                        int64_t T, GateOut o) {
  __shared__ double sc[4][64 * kPer];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;  // no barrier below: each wave has its own scores
  gate_token<kPer>(g, logits, bf16, t, lane, sc[wave], o);
}

hipError_t launch_gate_topk(const GateArgs &g, const void *logits, int bf16, int64_t T, const GateOut &o,
                            hipStream_t s) {
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
  if (g.E <= 128)
    hipLaunchKernelGGL(gate_topk_kernel<2>, grid, block, 0, s, g, logits, bf16, T, o);
  else if (g.E <= 256)
    hipLaunchKernelGGL(gate_topk_kernel<4>, grid, block, 0, s, g, logits, bf16, T, o);
  else
    hipLaunchKernelGGL(gate_topk_kernel<8>, grid, block, 0, s, g, logits, bf16, T, o);
  return hipGetLastError();
}

// Hidden rows of 4 tokens per wave for a gated forward, staged as route_kernel
// stages them: FP16 rows and their powers of two (1), the powers of two alone
// (2), FP8 codes and scales (3), NVFP4 values (4), nothing (0).  Also clears the
// saturation flag.
template <bool kPermInt4>
__global__ __launch_bounds__(256) void stage_rows_kernel(const uint16_t *__restrict__ hidden, int T, int H,
                                                         _Float16 *__restrict__ x16, float *__restrict__ rowscale,
                                                         uint32_t *__restrict__ flags, int stage_rows, float act_g) {
  const int lane = threadIdx.x & 63, t0 = (blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6)) * 4;
  if (blockIdx.x == 0 && threadIdx.x == 0) flags[0] = 0u;
  if (t0 >= T) return;
  if (stage_rows == 1) rows_to_f16<kPermInt4>(hidden, t0, T, H, lane, x16, rowscale);
  if (stage_rows == 2) rows_to_f16<kPermInt4, false>(hidden, t0, T, H, lane, x16, rowscale);
  if (stage_rows == 3)
    rows_to_fp8(hidden, t0, T, H, lane, (uint8_t *)x16, (float *)((uint8_t *)x16 + (size_t)T * H));
  if (stage_rows == 4) rows_to_nvfp4(hidden, t0, T, H, lane, act_g, x16, rowscale);
}

hipError_t launch_route_gated(const LayerDims &L, const FwdPtrs &P, const Workspace &W, bool decode, int stage_rows,
                              hipStream_t s) {
  char *ws = P.ws;
  const void *logits = P.logits;
  int bf16 = P.logits_bf16;
  if (P.gate_w) {
    float *lg = P.p_logits ? P.p_logits : (float *)(ws + W.logits);
    const hipError_t e = launch_router_logits(P.hidden, P.gate_w, lg, P.T, L.H, L.E, s);
    if (e != hipSuccess) return e;
    logits = lg;
    bf16 = 0;
  }
  // the FP32 down projection of one or two tokens takes the weights as they are
  float *wscale = down_writes_output(L, P, decode) ? nullptr : (float *)(ws + W.wscale);
  const GateOut o = {(int32_t *)(ws + W.topk_ids), (float *)(ws + W.topk_w), wscale, P.p_ids, P.p_w};
  const hipError_t e = launch_gate_topk(*P.gated, logits, bf16, P.T, o, s);
  if (e != hipSuccess) return e;
  const int threads = P.T <= 256 ? 64 : 256;
  hipLaunchKernelGGL(L.fmt == FMT_INT4 ? stage_rows_kernel<true> : stage_rows_kernel<false>,
                     dim3((unsigned)((P.T + threads / 16 - 1) / (threads / 16))), dim3(threads), 0, s, P.hidden, P.T,
                     L.H, (_Float16 *)(ws + W.x16), (float *)(ws + W.rowscale), P.flags, stage_rows, P.act_g13);
  return hipGetLastError();
}

}  // namespace mq
