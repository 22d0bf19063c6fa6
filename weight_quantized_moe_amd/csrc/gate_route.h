// What the two launches of a gated forward's routing stage take: the gate with
// the staging of the hidden rows (gate_route.hip), and for a few decode tokens
// the gate with the grouping (gate_group.hip).
#pragma once
#include "device.h"
#include "internal.h"

namespace mq {

struct StageArgs {
  const uint16_t *hidden;
  int T, H, stage_rows, perm_int4, gate_blocks;
  _Float16 *x16;
  float *rowscale;
  uint32_t *flags;
  float act_g;
};
struct GroupArgs {
  int32_t *offsets, *mtile;
  int4 *einfo;
  int32_t *rcp;
  int4 *rowinfo;
  int32_t *inv_pos, *p_offsets, *p_sorted_tok, *p_inv;
};

hipError_t launch_gate_group(const GateArgs &g, const void *logits, int bf16, const GateOut &o, const StageArgs &a,
                             const GroupArgs &q, hipStream_t s);

}  // namespace mq
