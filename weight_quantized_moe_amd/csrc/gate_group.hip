// The gate of a few decode tokens with their grouping by expert, in one workgroup.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gate_route.h"
#include "gate_select.h"

namespace mq {

// Grouping of R = T k <= 64 slots (T <= kFusedT) without a barrier: lane i is slot
// i in every wave, and a slot's row is the number of slots before it in the order
// (expert, slot), counted over the slots.  No expert has more than kFusedT rows:
// one 16-row chunk and one M-tile each.
static_assert(kFusedT <= 16 && kFusedT <= kPrefillBM, "one chunk and one M-tile an expert");
__device__ __forceinline__ void group_few(const int32_t *ids, const float *wts, const float *rowscale, int T, int E,
                                          int k, const GroupArgs &q) {
  const int tid = threadIdx.x, lane = tid & 63, R = T * k;
  const int e = lane < R ? ids[lane] : kMaxExperts;
  int below = 0, same = 0, earlier = 0;  // slots of lower experts, of this one, of this one before this slot
  for (int j = 0; j < R; ++j) {
    const int ej = __builtin_amdgcn_readlane(e, j);
    below += ej < e;
    same += ej == e;
    earlier += ej == e && j < lane;
  }
  const uint64_t firsts = __ballot(lane < R && earlier == 0);
  const int active = __popcll(firsts);
  // every lane of a wave stays for the counting, also past E: the slots are read from all of them
  for (int x0 = __builtin_amdgcn_readfirstlane(tid & ~63); x0 <= E; x0 += 512) {
    const int x = x0 + lane;
    int rows = 0, experts = 0;
    for (int j = 0; j < R; ++j) {
      const bool lower = __builtin_amdgcn_readlane(e, j) < x;
      rows += lower;
      experts += lower && ((firsts >> j) & 1ull);
    }
    if (x <= E) {
      q.offsets[x] = rows;
      if (q.p_offsets) q.p_offsets[x] = rows;
      q.mtile[x] = experts;
    }
  }
  if (tid >= 64) return;
  int rank = 0;  // active experts below this one
  for (int j = 0; j < R; ++j) rank += __builtin_amdgcn_readlane(e, j) < e && ((firsts >> j) & 1ull);
  if (lane < R) {
    const int pos = below + earlier, t = lane / k;
    q.rowinfo[pos] = int4{lane, t, __builtin_bit_cast(int, rowscale ? rowscale[t] : 0.f),
                          __builtin_bit_cast(int, wts[lane])};
    q.inv_pos[lane] = pos;
    if (q.p_sorted_tok) q.p_sorted_tok[pos] = t;
    if (q.p_inv) q.p_inv[lane] = pos;
    if (earlier == 0) {
      q.einfo[1 + rank] = int4{e, below, same, 0};
      q.rcp[rank] = rank;
    }
  }
  if (lane == 0) {
    q.einfo[0] = int4{active, active, 0, 0};
    q.rcp[active] = active;
  }
}

// ---------------------------------------------------------------------------
// Decode batches of up to kFusedT tokens: gate, powers of two of the hidden rows
// and grouping in one workgroup (route_group_kernel's counterpart): waves 0 to 3
// take the gate of 4 tokens each, waves 4 to 7 their rows' powers of two, and
// all of them the grouping on the ids and weights in LDS.  One token of 128
// experts: 5.1 us, bound by the latency of its steps; in three launches the
// layer's step took 23.2 us, with this one 18.6, with group_few 18.2, with the
// gate's modes fixed at compile time 17.7 (17.2 to 17.5 on other cards).
// ---------------------------------------------------------------------------
template <int kPer, GateMode kMode, bool kWhole>
__global__ __launch_bounds__(512) void gate_group_kernel(GateArgs g, const void *__restrict__ logits, int bf16,
                                                         GateOut o, StageArgs a, GroupArgs q) {
  __shared__ GateLds lds[4];
  __shared__ int32_t s_ids[kFusedT * 64];
  __shared__ float s_wts[kFusedT * 64];
  __shared__ float s_rs[kFusedT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t0 = 4 * (wave & 3);
  if (threadIdx.x == 0) a.flags[0] = 0u;
  if (t0 < a.T) {
    if (wave < 4) {
      const GateOut in_lds = {s_ids, s_wts, o.wscale, o.p_ids, o.p_w};
      gate_wave<kPer, kMode, kWhole>(g, logits, bf16, t0, a.T, lane, &lds[wave], in_lds);
    } else if (a.stage_rows == 2) {
      u4 v[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[r][u] = t0 + r < a.T && lane * 8 + 512 * u < a.H
                        ? *(const u4 *)(a.hidden + (size_t)(t0 + r) * a.H + lane * 8 + 512 * u)
                        : u4{0u, 0u, 0u, 0u};
      row_scale_regs(v, t0, a.T, a.H, lane, s_rs);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * g.k; i += 512) {
    o.ids[i] = s_ids[i];
    o.wts[i] = s_wts[i];
  }
  const bool scales = a.stage_rows == 2;
  if (scales && (int)threadIdx.x < a.T) a.rowscale[threadIdx.x] = s_rs[threadIdx.x];
  if (a.T * g.k <= 64) {
    group_few(s_ids, s_wts, scales ? s_rs : nullptr, a.T, g.E, g.k, q);
    return;
  }
  group_small_body<512>(s_ids, s_wts, scales ? s_rs : nullptr, a.T, g.E, g.k, q.offsets, q.mtile, q.einfo, q.rcp,
                        q.rowinfo, q.inv_pos, q.p_offsets, q.p_sorted_tok, q.p_inv, s_ids);
}

hipError_t launch_gate_group(const GateArgs &g, const void *logits, int bf16, const GateOut &o, const StageArgs &a,
                             const GroupArgs &q, hipStream_t s) {
  return with_gate_variant(g, [&](auto per, auto mode, auto whole) {
    hipLaunchKernelGGL((gate_group_kernel<per(), mode(), whole()>), dim3(1), dim3(512), 0, s, g, logits, bf16, o, a, q);
    return hipGetLastError();
  });
}

}  // namespace mq
