// The routing stage of an expert-layer forward under a gate.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gate_route.h"
#include "gate_select.h"

namespace mq {

// ---------------------------------------------------------------------------
// Routing stage of a gated forward: the gate of the first gate_blocks
// workgroups' tokens, beside it the hidden rows of the others', staged as
// route_kernel stages them (4 rows a wave): FP16 rows and their powers of two
// (1), the powers of two alone (2), FP8 codes and scales (3), NVFP4 values (4),
// nothing (0).  Also clears the saturation flag.  Beside each other in one launch
// the two take the longer one's time: 4096 tokens of 128 experts and 2048 values
// 10.8 us (32 MB of rows: 3.1 TB/s), 61 tokens 5.0 us.  Against two launches, on one
// card: the layer 429 -> 417 us and 113 -> 106 us (424 and 104 on another).
// ---------------------------------------------------------------------------
template <int kPer, GateMode kMode, bool kWhole>
__global__ __launch_bounds__(256) void gate_stage_kernel(GateArgs g, const void *__restrict__ logits, int bf16,
                                                         GateOut o, StageArgs a) {
  __shared__ GateLds lds[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.flags[0] = 0u;
  if ((int)blockIdx.x < a.gate_blocks) {
    const int64_t t0 = ((int64_t)blockIdx.x * waves + wave) * 4;
    if (t0 < a.T) gate_wave<kPer, kMode, kWhole>(g, logits, bf16, t0, a.T, lane, &lds[wave], o);
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
                         (int32_t *)(ws + W.rcpre), (int4 *)(ws + W.rowinfo),
                         (int32_t *)(ws + W.inv_pos), P.p_offsets, P.p_sorted_tok, P.p_inv};
    return launch_gate_group(*P.gated, logits, bf16, o, a, q, s);
  }
  return with_gate_variant(*P.gated, [&](auto per, auto mode, auto whole) {
    const int threads = P.T <= 4096 ? 64 : 256, tpb = threads / 16;
    a.gate_blocks = (P.T + tpb - 1) / tpb;
    const unsigned blocks = (unsigned)a.gate_blocks * (stage_rows ? 2u : 1u);
    hipLaunchKernelGGL((gate_stage_kernel<per(), mode(), whole()>), dim3(blocks), dim3(threads), 0, s, *P.gated, logits, bf16, o, a);
    return hipGetLastError();
  });
}

}  // namespace mq
