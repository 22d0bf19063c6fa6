// Gated routing: softmax or sigmoid scores, a balance bias that takes part in
// the selection only, groups of experts of which a few are kept, top-k,
// renormalised or raw weights (mq_gate in the C header states the formulas).
//
// The order of two selection scores next to each other decides which expert a
// token takes.  A 32-bit score cannot tell apart what differs by less than its
// rounding, so the selection is defined on 64-bit scores; the fast gate selects
// on 32-bit ones, bounds their error and looks again, in 64 bits, where the
// order lies within it.
//
// Measured (sigmoid, bias, k 8, 32-bit logits): 65536 tokens of 128 experts 17.8
// to 18.4 us (2.1 TB/s), 16384 of 256 in 8 groups, 4 kept, 10.1 to 11.3 us (1.7
// TB/s); all in 64 bits, a wave a token, 69 and 38 us.  Bound by vector
// instructions: 506 a wave of four tokens of 128 experts, issued in 76% of the
// kernel's cycles (876 of 256 with groups); finding close scores and the 64-bit
// second looks take 1.9 us of the first and 1.4 of the second.  Loops over several groups of four tokens a wave
// were slower (26 against 19 us: more registers).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.h"
#include "internal.h"
#include "route.h"

namespace mq {

constexpr float kInf = __builtin_inff();
constexpr float kMost = 3.402823466e38f;  // the largest finite value
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);
constexpr float kLn2 = 0.693147180559945309417f;

// Order-preserving map of a double to an unsigned integer; -0 maps to the key
// of +0, and no key of a number is 0 (the key of a selected or excluded expert).
__device__ __forceinline__ uint64_t ordered_key64(double v) {
  uint64_t b = __builtin_bit_cast(uint64_t, v);
  if ((b << 1) == 0ull) b = 0ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// A logit or a bias as the gate reads it: NaN counts as -inf (masked), +inf as
// the largest finite value, -0 as +0.
__device__ __forceinline__ float gate_logit(float v) {
  return v == v ? fminf(v + 0.f, kMost) : -kInf;
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

// The weight of a selected expert before its row is renormalised (0 where it is
// masked, l = -inf).  top: the row's largest selected logit (used where it is
// renormalised); m and z: softmax maximum and sum over all experts.  Written so
// that nothing overflows and small scores keep their digits: sigmoid(l) =
// exp(min(l, 0)) / (1 + exp(-|l|)), a renormalised row shifted by its largest.
// The hardware's exp2 and reciprocal are off by a unit in the last place.  The
// exponent x log2 e is a 32-bit product and its remainder, which corrects the
// power: a product alone is off by up to 2^-24 |x| log2 e, and the weight by as
// much.  What is left is the rounding of x itself where it is a difference, and
// in the denominator, which is 1 and more, a quarter of 2^-24 |l| exp(-|l|).
__device__ __forceinline__ float slot_score(const GateArgs &g, float l, float top, float m, float z) {
  const bool sigmoid = g.score == MQ_SCORE_SIGMOID;
  const float down = sigmoid ? (g.renormalize ? fminf(top, 0.f) : 0.f) : g.renormalize ? top : m;
  // exp(-200) is 0; the remainder of a product that overflows would be no number
  const float x = fmaxf((sigmoid ? fminf(l, 0.f) : l) - down, -200.f), p = x * kLog2e;
  const float rest = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -p));
  float s = __builtin_amdgcn_exp2f(p);
  s = fmaf(s * rest, kLn2, s);
  if (sigmoid)
    s *= __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(fabsf(l) * -kLog2e));
  else if (!g.renormalize)
    s *= __builtin_amdgcn_rcpf(z);
  return l > -kInf ? s : 0.f;
}
// Divides by a row's sum (0 where every slot is masked); the remainder of the
// first quotient corrects it, so one weight alone is 1.
__device__ __forceinline__ float over_sum(float s, float sum) {
  const float r = __builtin_amdgcn_rcpf(sum), q = s * r;
  return sum > 0.f ? fmaf(fmaf(-q, sum, s), r, q) : 0.f;
}

// The exponent of the power of two that brings a token's largest weight m into
// [2^-1, 1); 0 (none) for 2^-7 to 1, where every renormalised row of up to 64
// slots lies if the scale is 1: such a row's products have the range in FP16 that
// they have under the layer's own routing (digits from 2^-14 on, saturation).
__device__ __forceinline__ int weight_exponent(float m) {
  if (!(m > 0.f) || (m >= 0x1p-7f && m <= 1.f)) return 0;
  const int ex = (int)(__builtin_bit_cast(uint32_t, m) >> 23) - 126;
  return ex < -120 ? -120 : ex > 120 ? 120 : ex;
}

// at: slot t k + j (below 2^28); down: the power of two taken out of the weights
// (1 where none is).
__device__ __forceinline__ void write_slot(const GateOut &o, uint32_t at, int id, float w, float down) {
  o.ids[at] = id;
  o.wts[at] = w * down;
  if (o.p_ids) o.p_ids[at] = id;
  if (o.p_w) o.p_w[at] = w;
}

// Orders a wave's LDS writes before its reads of other lanes' values (and the
// other way round); each wave uses LDS of its own, so no barrier is needed.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------
// The gate of one token on all 64 lanes of a wave, in 64 bits; any number of
// groups, any k.  Lane l holds experts l + 64 i.  sc: one double per expert, LDS
// of this wave alone (the group scores read other lanes' experts there).  Each
// of the k rounds takes the largest key (two 32-bit maxima) and the lowest
// expert that holds it.  The exponentials stay one after the other (sched
// barriers): interleaved they would take the registers of the fast kernel.
// ---------------------------------------------------------------------------
template <int kPer>
__device__ __forceinline__ void gate_token(const GateArgs &g, const void *__restrict__ logits, int bf16, int64_t t,
                                           int lane, double *sc, const GateOut &o) {
  const int64_t at = t * g.E;
  float l[kPer], b[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < g.E ? load_gate_logit(logits, bf16, at + e) : -kInf;
    b[i] = g.bias && e < g.E ? gate_logit(g.bias[e]) : 0.f;
  }
  // softmax statistics over the live logits (M = 0 where there is none)
  float m = l[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) m = fmaxf(m, l[i]);
  m = max64f(m);
  if (m == -kInf) m = 0.f;
  const bool sigmoid = g.score == MQ_SCORE_SIGMOID;
  const bool by_logit = g.bias == nullptr;              // the logits' order is the scores'
  const bool scores = !by_logit || g.group_top == 2;    // else the order alone is enough
  double c[kPer], z = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c[i] = l[i];
    if (scores || (!sigmoid && !g.renormalize)) {
      c[i] = exp(sigmoid ? -fabs((double)l[i]) : (double)l[i] - (double)m);
      z += c[i];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (!sigmoid) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) z += __shfl_xor(z, d, 64);
  }
  uint64_t key[kPer];
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    const bool live = l[i] > -kInf && b[i] > -kInf;
    double s = l[i];
    if (scores) s = (sigmoid ? (l[i] < 0.f ? c[i] : 1.0) / (1.0 + c[i]) : c[i] / z) + (double)b[i];
    if (!live) s = -kInf;
    if (g.groups > 1 && e < g.E) sc[e] = s;
    key[i] = e < g.E ? ordered_key64(by_logit ? (double)l[i] : s) : 0ull;
    __builtin_amdgcn_sched_barrier(0);
  }
  if (g.groups > 1) {
    // lane = group: its score, then the number of groups that come before it
    wave_lds_fence();
    double s1 = -kInf, s2 = -kInf;
    if (lane < g.groups) {
#pragma unroll 4
      for (int i = 0; i < g.per; ++i) {
        const double v = sc[lane * g.per + i];
        s2 = fmax(s2, fmin(s1, v));
        s1 = fmax(s1, v);
      }
    }
    const double s = g.group_top == 2 ? s1 + s2 : s1;
    const uint64_t gk = lane < g.groups ? ordered_key64(s) : 0ull;
    int before = 0;
    for (int j = 0; j < g.groups; ++j) {
      const uint64_t other = __shfl(gk, j, 64);
      before += other > gk || (other == gk && j < lane);
    }
    const uint64_t kept = __ballot(lane < g.groups && before < g.topk_groups);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (!((kept >> (min(lane + 64 * i, g.E - 1) / g.per)) & 1ull)) key[i] = 0ull;
  }
  int slot_id = 0;
  for (int j = 0; j < g.k; ++j) {
    uint64_t mine = key[0];  // the lane's largest key, and the lowest expert that holds it
    int e_mine = lane;
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      if (key[i] > mine) {
        mine = key[i];
        e_mine = lane + 64 * i;
      }
    const uint64_t km = max64_u64(mine);
    const int e = (int)(0xFFFFFFFFu - max64_u32(mine == km ? 0xFFFFFFFFu - (uint32_t)e_mine : 0u));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 64 * i == e) key[i] = 0ull;
    if (j == lane) slot_id = e;
  }
  // weights of the k slots (lane = slot), in 32 bits
  float lw = -kInf;
  if (lane < g.k) {
    lw = load_gate_logit(logits, bf16, at + slot_id);
    if (g.bias && gate_logit(g.bias[slot_id]) == -kInf) lw = -kInf;
  }
  float w = slot_score(g, lw, g.renormalize ? max64f(lw) : 0.f, m, (float)z);
  if (g.renormalize) {
    const float sum = sum64f(w);
    w = over_sum(w, sum);
  }
  w *= g.scale;
  float down = 1.f;
  if (o.wscale) {
    const int ex = weight_exponent(max64f(fabsf(w)));
    down = pow2f(-ex);
    if (lane == 0) o.wscale[t] = pow2f(ex);
  }
  if (lane < g.k) write_slot(o, (uint32_t)t * g.k + lane, slot_id, w, down);
}

// ---------------------------------------------------------------------------
// The gate of four tokens on one wave, 16 lanes (one DPP row) per token, in 32
// bits; groups 1, 2, 4, 8 or 16 and k <= 16.  A lane's kPer experts are
// consecutive and of one group, so group scores are reductions over adjacent
// lanes and equal scores lie in expert order over the lanes.
//   1. scores as ordered integer keys, the two largest of each lane, and from
//      those the group scores and the rank of each group;
//   2. a lower bound tau of the k-th largest key: k rounds of "largest of the
//      lanes' two largest", 4 DPP steps each;
//   3. the experts at or above tau (8.2 of 256 on average for k = 8) go to LDS
//      in expert order;
//   4. each lane ranks the candidate it holds by counting those before it.
// What is not certain at 32 bits: a score is off by at most 2^-22 + 2^-24 |c|
// for a sigmoid (exponent 2^-23 |l| s(1 - s) <= 2^-25, reciprocal and sums), and
// for a softmax by 2^-22 + 2^-24 |c| and a common factor 1 + 2^-18 (its sum: at
// most 35 additions, 32 experts a lane, and the terms' own errors), so two
// scores further apart than tol = 2^-20 (1 + |c|), for a softmax 2^-17 (1 +
// |c|), are in their order with a factor of 2 to spare.  tau is lowered by tol.  Where two candidates next
// to each other in the order are within tol and not the same logit and bias,
// the row's candidates are ranked again by 64-bit scores; where a kept and a
// dropped group are within 2 tol (their sums of two, too: those add two errors), the groups are, by the 64-bit scores of each
// lane's two largest.  Without a bias the keys are the logits and exact, and
// masked experts (key of -inf) are exact always: of more than 16 candidates
// those equal to tau then count in expert order only.  What is left (more than
// 16 candidates or three scores of a lane within tol) is handed to the 64-bit
// gate: returns those tokens (rows of the wave) as a mask; the others are
// written.
// ---------------------------------------------------------------------------
constexpr int kFastK = 16;  // slots, and candidates a token may have

struct Candidates {  // of one token, in LDS
  uint64_t wide[kFastK];
  uint32_t key[kFastK];
  float l[kFastK];
  int32_t id[kFastK];
};

// The value N lanes down the 16-lane row, 0 where the row has none.
template <int N>
__device__ __forceinline__ uint32_t dpp_shr(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x110 + N, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t min16_u32(uint32_t v) {
  v = min(v, dpp<kXor1>(v));
  v = min(v, dpp<kXor2>(v));
  v = min(v, dpp<kHalfMirror>(v));
  v = min(v, dpp<kMirror>(v));
  return v;
}
__device__ __forceinline__ int sum16i(int v) {
  v += (int)dpp<kXor1>((uint32_t)v);
  v += (int)dpp<kXor2>((uint32_t)v);
  v += (int)dpp<kHalfMirror>((uint32_t)v);
  v += (int)dpp<kMirror>((uint32_t)v);
  return v;
}
// Inclusive sum over the row's lanes.
__device__ __forceinline__ int scan16i(int v) {
  v += (int)dpp_shr<1>((uint32_t)v);
  v += (int)dpp_shr<2>((uint32_t)v);
  v += (int)dpp_shr<4>((uint32_t)v);
  v += (int)dpp_shr<8>((uint32_t)v);
  return v;
}
// Key of a score that is no NaN and no -0; from_ordered_key inverts it.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
constexpr uint32_t kMaskedKey = 0x007FFFFFu;  // of -inf

// Moves and reductions of 64-bit values inside a 16-lane row.
template <int kCtrl>
__device__ __forceinline__ double dppd(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, ((uint64_t)dpp<kCtrl>((uint32_t)(b >> 32)) << 32) | dpp<kCtrl>((uint32_t)b));
}
__device__ __forceinline__ double sum16d(double v) {
  v += dppd<kXor1>(v);
  v += dppd<kXor2>(v);
  v += dppd<kHalfMirror>(v);
  v += dppd<kMirror>(v);
  return v;
}
template <int kCtrl>
__device__ __forceinline__ void top2_joind(double &a, double &b) {
  const double c = dppd<kCtrl>(a), d = dppd<kCtrl>(b);
  b = fmax(fmin(a, c), fmax(b, d));
  a = fmax(a, c);
}
// A selection score in 64 bits (live experts; zd: the softmax's sum).  A sigmoid by
// exp(-|l|), which does not overflow: exp(-l) would leave 0 below -709.
__device__ __forceinline__ double wide_score(const GateArgs &g, float l, float m, double zd, int e) {
  const bool sigmoid = g.score == MQ_SCORE_SIGMOID;
  const double p = exp(sigmoid ? -fabs((double)l) : (double)l - (double)m);
  return (sigmoid ? (l < 0.f ? p : 1.0) / (1.0 + p) : p / zd) + (g.bias ? (double)gate_logit(g.bias[e]) : 0.0);
}
// The softmax's sum over a row's experts in 64 bits.
template <int kPer>
__device__ __forceinline__ double wide_sum(const float (&l)[kPer], float m) {
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    z += exp((double)l[i] - (double)m);
    __builtin_amdgcn_sched_barrier(0);
  }
  return sum16d(z);
}

// The two largest of a pair of lanes' two largest.
template <int kCtrl>
__device__ __forceinline__ void top2_join(uint32_t &a, uint32_t &b) {
  const uint32_t c = dpp<kCtrl>(a), d = dpp<kCtrl>(b);
  b = max(min(a, c), max(b, d));
  a = max(a, c);
}
// Number of other groups in the 16-lane row whose key comes before this lane's,
// groups being `lanes` lanes wide; equal keys count where the other group is
// the lower one (bit n of lower: the lane n places down the row).
template <int N, typename Key>
__device__ __forceinline__ int groups_before(Key key, uint32_t lower, int lanes) {
  int before = 0;
  if constexpr (N < 16) {
    if ((N & (lanes - 1)) == 0) {  // uniform
      Key other = dpp<0x120 + N>((uint32_t)key);  // row_ror
      if constexpr (sizeof(Key) == 8) other |= (Key)dpp<0x120 + N>((uint32_t)((uint64_t)key >> 32)) << 32;
      before = other > key - ((lower >> N) & 1u);
    }
    before += groups_before<N + 1>(key, lower, lanes);
  }
  return before;
}

// A lane's place in the gate.
struct GateLane {
  int lanes;       // lanes of a group
  int e0, count;   // first expert of this lane, and how many
  uint32_t lower;  // bit n: the lane n places down the row is of a lower group
};
template <int kPer, bool kWhole>
__device__ __forceinline__ GateLane gate_lane(const GateArgs &g, int li) {
  GateLane a;
  const int shift = 4 - (31 - __builtin_clz(g.groups));
  a.lanes = 1 << shift;
  const int off = li & (a.lanes - 1);
  const int chunk = kWhole ? kPer : (g.per + a.lanes - 1) >> shift;
  a.e0 = kWhole ? li * kPer : min((li >> shift) * g.per + off * chunk, g.E);
  a.count = kWhole ? kPer : max(0, min(chunk, g.per - off * chunk));
  a.lower = ((2u << li) - 1u) & ~((2u << off) - 1u);
  return a;
}

// What of a gate is fixed when a kernel is compiled: the source of the order
// (logits, sigmoid or softmax plus bias) and whether there are groups.  Branches
// on these took a tenth of the kernel's time.  kWhole beside it: each lane holds
// kPer experts (E = 16 kPer), loaded 16 bytes at a time.
enum GateMode { kLogits, kSigmoid, kSoftmax, kLogitsGroups, kSigmoidGroups, kSoftmaxGroups };

template <int kPer, GateMode kMode, bool kWhole>
__device__ __forceinline__ uint32_t gate_tokens4(const GateArgs &g, const void *__restrict__ logits, int bf16,
                                                 int64_t t0, int64_t T, int lane, Candidates *cands,
                                                 const GateOut &o) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  typedef f4 f4_a4 __attribute__((aligned(4)));
  const int li = lane & 15, row = lane >> 4;
  const int rows = (int)min(T - t0, (int64_t)4);
  const bool here = row < rows;
  const int r = min(row, rows - 1);  // a row past the last token repeats it
  const uint32_t t = (uint32_t)t0 + r;
  constexpr bool kByLogit = kMode == kLogits || kMode == kLogitsGroups;
  constexpr bool kGroups = kMode >= kLogitsGroups;
  const GateLane a = gate_lane<kPer, kWhole>(g, li);
  constexpr bool by_logit = kByLogit, groups = kGroups;
  const bool softmax = by_logit ? g.score == MQ_SCORE_SOFTMAX : kMode == kSoftmax || kMode == kSoftmaxGroups;
  const bool sums = groups && g.group_top == 2;
  const float tol1 = softmax ? 0x1p-17f : 0x1p-20f;
  // without whole lanes: what a lane loads beyond its experts is some other
  // logit, and its key is 0; only the array's end must not be passed
  const int64_t left = (T - t0) * g.E;  // logits from the wave's first on
  const bool inside = left >= 4 * g.E + kPer;
  const uint32_t last = (uint32_t)min(left - 1, (int64_t)0x7FFFFFFF);
  float l[kPer];
  const uint32_t at = (uint32_t)(r * g.E + a.e0);  // from the wave's first logit on
  if (bf16) {
    const uint16_t *p = (const uint16_t *)logits + t0 * g.E + at;
    if (kWhole) {
      u2 u[kPer / 4];
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) u[i] = *(const u2 *)(p + 4 * i);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t w = u[i / 4][(i >> 1) & 1];
        l[i] = __builtin_bit_cast(float, i & 1 ? w & 0xFFFF0000u : w << 16);
      }
    } else if (inside) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) l[i] = bf16_to_f32(p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) l[i] = bf16_to_f32(((const uint16_t *)logits + t0 * g.E)[min(at + i, last)]);
    }
  } else {
    const float *p = (const float *)logits + t0 * g.E + at;
    if (kWhole) {
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) {
        const f4 u = *(const f4_a4 *)(p + 4 * i);  // logits computed here may be aligned to 4 bytes
#pragma unroll
        for (int q = 0; q < 4; ++q) l[4 * i + q] = u[q];
      }
    } else if (inside) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) l[i] = p[i];
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) l[i] = ((const float *)logits + t0 * g.E)[min(at + i, last)];
    }
  }
  if (by_logit || softmax) {  // a sigmoid's key below takes them as they are
#pragma unroll
    for (int i = 0; i < kPer; ++i) l[i] = kWhole || i < a.count ? gate_logit(l[i]) : -kInf;
  }

  // softmax statistics, where a score or a weight needs them
  float m = 0.f, z = 1.f;
  if (softmax && (!by_logit || !g.renormalize || sums)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, l[i]);
    m = max16f(m);
    if (m == -kInf) m = 0.f;
    if (!by_logit || !g.renormalize) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) z += __builtin_amdgcn_exp2f((l[i] - m) * kLog2e);
      z = sum16(z);
    }
  }
  // selection keys; 0: no expert of this lane
  uint32_t key[kPer];
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = score_key(l[i]);
  } else {
    float c[kPer];
    if (kWhole) {
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) {
        const f4 u = *(const f4_a4 *)(g.bias + a.e0 + 4 * i);
#pragma unroll
        for (int q = 0; q < 4; ++q) c[4 * i + q] = u[q];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = g.bias[min(a.e0 + i, g.E - 1)];
    }
    if (softmax) {
      const float zinv = 1.f / z;  // inf where every expert is masked: not used then
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        c[i] += __builtin_amdgcn_exp2f((l[i] - m) * kLog2e) * zinv;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        c[i] += __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[i] * -kLog2e));
    }
    // masked: a logit or a bias of -inf or NaN (a NaN is not greater than -inf)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      key[i] = l[i] > -kInf && c[i] > -kInf ? score_key(fminf(c[i], kMost)) : kMaskedKey;
  }
  uint32_t t1 = 0u, t2 = 0u;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!kWhole) key[i] = i < a.count ? key[i] : 0u;
    t2 = max(t2, min(t1, key[i]));
    t1 = max(t1, key[i]);
  }
  bool unsure = false, kept = true;
  if (groups) {
    uint32_t k1 = t1, k2 = t2;
    if (a.lanes >= 2) top2_join<kXor1>(k1, k2);
    if (a.lanes >= 4) top2_join<kXor2>(k1, k2);
    if (a.lanes >= 8) top2_join<kHalfMirror>(k1, k2);
    uint32_t gk = k1;
    float size = 0.f;
    if (sums || !by_logit) {
      float s1 = from_ordered_key(k1), s2 = from_ordered_key(max(k2, kMaskedKey));
      if (by_logit) {  // the scores of the two logits (a softmax's without its common factor 1 / z)
        s1 = s1 == -kInf ? s1 : softmax ? expf(s1 - m) : 1.f / (1.f + expf(-s1));
        s2 = s2 == -kInf ? s2 : softmax ? expf(s2 - m) : 1.f / (1.f + expf(-s2));
      }
      size = fmaxf(fabsf(s1), sums ? fabsf(s2) : 0.f);
      size = size < kInf ? size : 0.f;
      // half the sum: two of the largest numbers' must not pass for an infinity
      gk = score_key((sums ? fmaf(0.5f, s1, 0.5f * s2) : s1) + 0.f);
    }
    kept = groups_before<1>(gk, a.lower, a.lanes) < g.topk_groups;
    if ((sums || !by_logit) && g.topk_groups < g.groups) {
      const float lo = from_ordered_key(min16_u32(kept ? gk : 0xFFFFFFFFu));
      const float hi = from_ordered_key(max16_u32(kept ? 0u : gk));
      // -inf on either side is exact (masked experts): the difference is then inf or NaN
      const bool close = lo - hi <= (sums ? tol1 : 2.f * tol1) * (1.f + max16f(size));
      if (__any(close)) {
        // the 64-bit scores of the lane's two largest, which have to be its two
        // largest for certain
        int n = 0, e1 = 0, e2 = 0;
        float l1 = -kInf, l2 = -kInf;
        const float third = from_ordered_key(max(t2, kMaskedKey));
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i) {
          const float v = from_ordered_key(max(key[i], kMaskedKey));
          n += !by_logit && v > -kInf && v >= third - tol1 * (1.f + fabsf(third));
          if (key[i] == t2 && key[i] != t1) { l2 = l[i]; e2 = a.e0 + i; }
          if (key[i] == t1) {
            // equal largest keys: the first and the one after it
            if (t1 == t2) { l2 = l1; e2 = e1; }
            l1 = l[i];
            e1 = a.e0 + i;
          }
        }
        const double zd = softmax && !by_logit ? wide_sum(l, m) : 1.0;
        double d1 = -kInf, d2 = -kInf;
        if (t1 > kMaskedKey) d1 = wide_score(g, l1, m, zd, e1);
        __builtin_amdgcn_sched_barrier(0);
        if (t2 > kMaskedKey) d2 = wide_score(g, l2, m, zd, e2);
        const double lane1 = fmax(d1, d2), lane2 = fmin(d1, d2);
        d1 = lane1;
        d2 = lane2;
        if (a.lanes >= 2) top2_joind<kXor1>(d1, d2);
        if (a.lanes >= 4) top2_joind<kXor2>(d1, d2);
        if (a.lanes >= 8) top2_joind<kHalfMirror>(d1, d2);
        const bool again = groups_before<1>(ordered_key64(sums ? d1 + d2 : d1), a.lower, a.lanes) < g.topk_groups;
        kept = close ? again : kept;
        unsure = close && n > 2;
      }
    }
  }
  // a lane of a dropped group has no keys from here on
  const uint32_t drop = kept ? 0u : 0xFFFFFFFFu;
  t1 = kept ? t1 : 0u;
  t2 = kept ? t2 : 0u;
  // the least of the k largest of the lanes' two largest
  uint32_t tau = 0u, v1 = t1, v2 = t2;
  for (int j = 0; j < g.k; ++j) {
    tau = max16_u32(v1);
    const bool out = v1 == tau;  // several lanes may go at once: tau only gets lower
    v1 = out ? v2 : v1;
    v2 = out ? 0u : v2;
  }
  if (__any(tau == 0u)) {
    // all of them went: their least, or every key where they are fewer than k
    const uint32_t all = min16_u32(min(t1 ? t1 : 0xFFFFFFFFu, t2 ? t2 : 0xFFFFFFFFu));
    const bool enough = sum16i((t1 != 0u) + (t2 != 0u)) >= g.k;
    tau = tau != 0u ? tau : enough ? all : 1u;
  }
  // the least key a candidate may have: keys equal to tau are equal scores
  // where they are exact
  auto least = [&](uint32_t k0) {
    const float v = from_ordered_key(k0);
    return by_logit || k0 <= kMaskedKey ? k0 : score_key((v - tol1 * (1.f + fabsf(v))) + 0.f);
  };
  auto at_least = [&](uint32_t k0) {  // keys of this lane
    k0 |= drop;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += key[i] >= k0;
    return c;
  };
  uint32_t lo = least(tau);
  int n = at_least(lo), have = sum16i(n);
  if (__any(have > kFastK)) {
    // too many for the lanes: tau goes up to the next key while k are left.  A key
    // a round, and all of the kept groups' keys from the least on where their lanes'
    // two largest are fewer than k: 16384 tokens of 256 experts, k 8, 1 of 8 groups
    // kept (two lanes a group) 28.5 us, 4 kept 11.1; 512, 1 of 16 kept 48, 8 kept 18
    bool more = have > kFastK;
    while (__any(more)) {
      uint32_t up = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < kPer; ++i) up = min(up, key[i] > tau ? key[i] : 0xFFFFFFFFu);
      up = min16_u32(up | drop);
      more &= sum16i(at_least(up)) >= g.k;
      tau = more ? up : tau;
      lo = least(tau);
      n = at_least(lo);
      have = sum16i(n);
      more &= have > kFastK;
    }
  }
  const int pos0 = scan16i(n) - n;
  Candidates &cd = cands[row];
  wave_lds_fence();
  cd.key[li] = 0u;
  wave_lds_fence();
  bool fits = have <= kFastK;
  if (__any(!fits)) {
    // equal scores at the end of the order: those above, then those equal to
    // tau in expert order as far as there is room
    const int above = at_least(tau + 1u), before = scan16i(above) - above, all = sum16i(above);
    if (!fits) {
      fits = (by_logit || tau <= kMaskedKey) && all < g.k;
      have = kFastK;
      int pa = before, pe = all + pos0 - before;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (fits && key[i] >= (tau | drop)) {
          const int p = key[i] > tau ? pa++ : pe++;
          if (p < kFastK) {
            cd.key[p] = key[i];
            cd.l[p] = l[i];
            cd.id[p] = a.e0 + i;
          }
        }
      lo = 0xFFFFFFFFu;  // written, or left to the 64-bit gate: no key is that large
    }
  }
  unsure |= !fits;
  int pos = pos0;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (key[i] >= (lo | drop)) {
      cd.key[pos] = key[i];
      cd.l[pos] = l[i];
      cd.id[pos] = a.e0 + i;
      ++pos;
    }
  wave_lds_fence();
  const uint32_t ck = cd.key[li];  // 0: no candidate
  const float cl = ck <= kMaskedKey ? -kInf : cd.l[li];  // -inf: masked
  const int id = cd.id[li];
  int rank = 0;
  auto rank_among = [&](int first) {  // four candidates; equal keys: in expert order
#pragma unroll
    for (int p = 0; p < 4; ++p) rank += cd.key[first + p] > ck - (first + p < li ? 1u : 0u);
  };
  rank_among(0);
  rank_among(4);
  if (__any(have > 8)) rank_among(8);
  if (__any(have > 12)) rank_among(12);
  if (!by_logit) {
    // neighbours in the order, through LDS
    wave_lds_fence();
    if (ck != 0u) {
      cd.key[rank] = ck;
      cd.l[rank] = cl;
      cd.id[rank] = id;
    }
    wave_lds_fence();
    const int next = min(rank + 1, kFastK - 1);
    const float c = from_ordered_key(ck), d = from_ordered_key(cd.key[next]);
    bool close = fits && ck > kMaskedKey && rank + 1 < have && c - d <= tol1 * (1.f + fabsf(c));
    if (close) close = cl != cd.l[next] || gate_logit(g.bias[id]) != gate_logit(g.bias[cd.id[next]]);
    if (__any(close)) {
      // the candidates of the rows in question by 64-bit scores (equal ones in
      // expert order)
      const uint64_t rows = __ballot(close);
      const double zd = softmax ? wide_sum(l, m) : 1.0;
      const double s = ck > kMaskedKey ? wide_score(g, cl, m, zd, id) : -kInf;
      const uint64_t wk = ck != 0u ? ordered_key64(s) : 0ull;
      cd.wide[li] = wk;
      cd.id[li] = id;
      wave_lds_fence();
      int again = 0;
      for (int p = 0; p < kFastK; ++p) again += cd.wide[p] > wk || (cd.wide[p] == wk && cd.id[p] < id && wk != 0ull);
      if ((rows >> (16 * row)) & 0xFFFFull) rank = again;
    }
  }
  const uint64_t votes = __ballot(unsure && here);
  uint32_t redo = 0u;
#pragma unroll
  for (int r = 0; r < 4; ++r) redo |= (uint32_t)(((votes >> (16 * r)) & 0xFFFFull) != 0ull) << r;

  // weights of the selected candidates
  const bool sel = fits && ck != 0u && rank < g.k;
  const float top = g.renormalize ? max16f(sel ? cl : -kInf) : 0.f;
  float w = slot_score(g, sel ? cl : -kInf, top, m, z);
  if (g.renormalize) {
    const float sum = sum16(w);
    w = over_sum(w, sum);
  }
  w *= g.scale;
  const bool done = here && !((redo >> row) & 1u);
  float down = 1.f;
  if (o.wscale) {
    const int ex = weight_exponent(max16f(fabsf(w)));
    down = pow2f(-ex);
    if (done && li == 0) o.wscale[t] = pow2f(ex);
  }
  if (done && sel) write_slot(o, t * g.k + (uint32_t)rank, id, w, down);
  return redo;
}

// Four tokens (from t0 on) of one wave: the fast gate, then the 64-bit one for
// the tokens it could not decide.  kPer 0: the 64-bit one alone, for k above 16
// or a number of groups that does not divide a row of lanes.
union GateLds {
  Candidates cand[4];
  double sc[kMaxExperts];
};
template <int kPer, GateMode kMode, bool kWhole>
__device__ __forceinline__ void gate_wave(const GateArgs &g, const void *__restrict__ logits, int bf16, int64_t t0,
                                          int64_t T, int lane, GateLds *lds, const GateOut &o) {
  t0 = __builtin_amdgcn_readfirstlane((int)t0);  // the same in every lane: kept in scalar registers
  uint32_t redo = 0xFu;
  if constexpr (kPer > 0) redo = gate_tokens4<kPer, kMode, kWhole>(g, logits, bf16, t0, T, lane, lds->cand, o);
  constexpr int kPer64 = kPer == 0 ? kMaxExperts / 64 : kPer <= 4 ? 1 : kPer / 4;
  for (int r = 0; r < 4 && t0 + r < T; ++r)
    if ((redo >> r) & 1u) gate_token<kPer64>(g, logits, bf16, t0 + r, lane, lds->sc, o);
}

// Calls f with the kernel variant for this gate: f(kPer, mode, kWhole) as constants.
// kPer is the least of 4, 8, 12, 16, 24 and 32 that holds a lane's experts.  12 and
// 24 beside the powers of two (16384 tokens, sigmoid and bias): 192 experts 9.0 us,
// in lanes of 16 11.0; 384 12.0, in lanes of 32 22.3; 160 in 8 groups 10.4 and 11.6.
template <typename F>
static hipError_t with_gate_variant(const GateArgs &g, F f) {
  using std::integral_constant;
  const int lanes = 16 / g.groups;  // 0 above 16 groups
  if (g.k > kFastK || lanes == 0 || 16 % g.groups)
    return f(integral_constant<int, 0>{}, integral_constant<GateMode, kLogits>{}, std::false_type{});
  const int chunk = (g.per + lanes - 1) / lanes;
  auto whole = [&](auto n, auto mode) {
    return chunk * 16 == g.E && chunk == n() ? f(n, mode, std::true_type{}) : f(n, mode, std::false_type{});
  };
  auto go = [&](auto n) {
    const bool groups = g.groups > 1;
    if (!g.bias)
      return groups ? whole(n, integral_constant<GateMode, kLogitsGroups>{})
                    : whole(n, integral_constant<GateMode, kLogits>{});
    if (g.score == MQ_SCORE_SIGMOID)
      return groups ? whole(n, integral_constant<GateMode, kSigmoidGroups>{})
                    : whole(n, integral_constant<GateMode, kSigmoid>{});
    return groups ? whole(n, integral_constant<GateMode, kSoftmaxGroups>{})
                  : whole(n, integral_constant<GateMode, kSoftmax>{});
  };
  if (chunk <= 4) return go(integral_constant<int, 4>{});
  if (chunk <= 8) return go(integral_constant<int, 8>{});
  if (chunk <= 12) return go(integral_constant<int, 12>{});
  if (chunk <= 16) return go(integral_constant<int, 16>{});
  if (chunk <= 24) return go(integral_constant<int, 24>{});
  return go(integral_constant<int, 32>{});
}

}  // namespace mq
