// The routing stage of an expert-layer forward under a gate.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gate_select.h"

namespace mq {

// ---------------------------------------------------------------------------
// Routing stage of a gated forward: the gate of the first gate_blocks
// workgroups' tokens, beside it the hidden rows of the others', staged as
// route_kernel stages them (4 rows a wave): FP16 rows and their powers of two
// (1), the powers of two alone (2), FP8 codes and scales (3), NVFP4 values (4),
// nothing (0).  Also clears the saturation flag.  Beside each other in one launch
// the two take the longer one's time: 4096 tokens of 128 experts and 2048 values
// 10.6 us (32 MB of rows: 3.2 TB/s), the layer 429 -> 417 us; 61 tokens 5.4 us,
// the layer 113 -> 106 us.
// ---------------------------------------------------------------------------
struct StageArgs {
  const uint16_t *hidden;
  int T, H, stage_rows, perm_int4, gate_blocks;
  _Float16 *x16;
  float *rowscale;
  uint32_t *flags;
  float act_g;
};
template <int kPer, GateMode kMode>
__global__ __launch_bounds__(256) void gate_stage_kernel(GateArgs g, const void *__restrict__ logits, int bf16,
                                                         GateOut o, StageArgs a) {
  __shared__ GateLds lds[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.flags[0] = 0u;
  if ((int)blockIdx.x < a.gate_blocks) {
    const int64_t t0 = ((int64_t)blockIdx.x * waves + wave) * 4;
    if (t0 < a.T) gate_wave<kPer, kMode>(g, logits, bf16, t0, a.T, lane, &lds[wave], o);
    return;
  }
  const int t0 = (((int)blockIdx.x - a.gate_blocks) * waves + wave) * 4, T = a.T, H = a.H;
  if (t0 >= T) return;
  if (a.stage_rows == 1 && a.perm_int4) rows_to_f16<true>(a.hidden, t0, T, H, lane, a.x16, a.rowscale);
  if (a.stage_rows == 1 && !a.perm_int4) rows_to_f16<false>(a.hidden, t0, T, H, lane, a.x16, a.rowscale);
  if (a.stage_rows == 2) rows_to_f16<false, false>(a.hidden, t0, T, H, lane, a.x16, a.rowscale);
  if (a.stage_rows == 3)
    rows_to_fp8(a.hidden, t0, T, H, lane, (uint8_t *)a.x16, (float *)((uint8_t *)a.x16 + (size_t)T * H));
  if (a.stage_rows == 4) rows_to_nvfp4(a.hidden, t0, T, H, lane, a.act_g, a.x16, a.rowscale);
}

// ---------------------------------------------------------------------------
// Decode batches of up to kFusedT tokens: gate, powers of two of the hidden rows
// and grouping in one workgroup (route_group_kernel's counterpart): waves 0 to 3
// take the gate of 4 tokens each, waves 4 to 7 their rows' powers of two, and
// all of them the grouping on the ids and weights in LDS.  One token of 128
// experts: 5.6 us, bound by the latency of its steps; in three launches the
// layer's step took 23.2 us, with this one 18.6, and with group_few 18.2.
// ---------------------------------------------------------------------------
struct GroupArgs {
  int32_t *offsets, *mtile;
  int4 *einfo;
  int32_t *rcp, *sorted_slots;
  int4 *rowinfo;
  int32_t *inv_pos, *p_offsets, *p_sorted_tok, *p_inv;
};
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
  for (int x = tid; x <= E; x += 512) {
    int rows = 0, experts = 0;
    for (int j = 0; j < R; ++j) {
      const bool lower = __builtin_amdgcn_readlane(e, j) < x;
      rows += lower;
      experts += lower && ((firsts >> j) & 1ull);
    }
    q.offsets[x] = rows;
    if (q.p_offsets) q.p_offsets[x] = rows;
    q.mtile[x] = experts;
  }
  if (tid >= 64) return;
  int rank = 0;  // active experts below this one
  for (int j = 0; j < R; ++j) rank += __builtin_amdgcn_readlane(e, j) < e && ((firsts >> j) & 1ull);
  if (lane < R) {
    const int pos = below + earlier, t = lane / k;
    q.sorted_slots[pos] = lane;
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

template <int kPer, GateMode kMode>
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
      gate_wave<kPer, kMode>(g, logits, bf16, t0, a.T, lane, &lds[wave], in_lds);
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
                        q.sorted_slots, q.rowinfo, q.inv_pos, q.p_offsets, q.p_sorted_tok, q.p_inv, s_ids);
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
  StageArgs a = {P.hidden, P.T, L.H, stage_rows, L.fmt == FMT_INT4, 0, (_Float16 *)(ws + W.x16), (float *)(ws + W.rowscale),
                 P.flags, P.act_g13};
  if (route_groups(L, P, decode)) {
    const GroupArgs q = {(int32_t *)(ws + W.offsets), (int32_t *)(ws + W.mtile), (int4 *)(ws + W.active),
                         (int32_t *)(ws + W.rcpre), (int32_t *)(ws + W.sorted_slots), (int4 *)(ws + W.rowinfo),
                         (int32_t *)(ws + W.inv_pos), P.p_offsets, P.p_sorted_tok, P.p_inv};
    return with_gate_variant<false>(*P.gated, [&](auto per, auto mode) {
      hipLaunchKernelGGL((gate_group_kernel<per(), mode()>), dim3(1), dim3(512), 0, s, *P.gated, logits, bf16, o, a, q);
      return hipGetLastError();
    });
  }
  return with_gate_variant<false>(*P.gated, [&](auto per, auto mode) {
    const int threads = P.T <= 4096 ? 64 : 256, tpb = threads / 16;
    a.gate_blocks = (P.T + tpb - 1) / tpb;
    const unsigned blocks = (unsigned)a.gate_blocks * (stage_rows ? 2u : 1u);
    hipLaunchKernelGGL((gate_stage_kernel<per(), mode()>), dim3(blocks), dim3(threads), 0, s, *P.gated, logits, bf16, o, a);
    return hipGetLastError();
  });
}

}  // namespace mq
