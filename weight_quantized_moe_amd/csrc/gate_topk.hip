// The gate by itself: ids and weights of a batch of router logits.  Device code
// and its reasons in gate_select.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gate_select.h"

namespace mq {

template <int kPer, GateMode kMode, bool kWhole>
__global__ __launch_bounds__(256) void gate_topk_kernel(GateArgs g, const void *__restrict__ logits, int bf16,
                                                        int64_t T, GateOut o) {
  __shared__ GateLds lds[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t0 = ((int64_t)blockIdx.x * (blockDim.x >> 6) + wave) * 4;
  if (t0 < T) gate_wave<kPer, kMode, kWhole>(g, logits, bf16, t0, T, lane, &lds[wave], o);
}

hipError_t launch_gate_topk(const GateArgs &g, const void *logits, int bf16, int64_t T, const GateOut &o,
                            hipStream_t s) {
  return with_gate_variant(g, [&](auto per, auto mode, auto whole) {
    // One wave a workgroup spreads a small batch over the CUs (3001 tokens of 72
    // experts: 6.0 us, two waves 6.3); a large one is bound by the rate at which
    // workgroups start with it (65536 of 128: 29 us; 2, 4, 8 and 16 waves 21.8,
    // 19.7, 20.6 and 22.4; 16384 of 256: 16.3, then 13.0, 12.7, 13.0 and 12.7).
    const int threads = T <= 4096 ? 64 : 256, tpb = threads / 16;
    hipLaunchKernelGGL((gate_topk_kernel<per(), mode(), whole()>), dim3((unsigned)((T + tpb - 1) / tpb)), dim3(threads), 0, s, g,
                       logits, bf16, T, o);
    return hipGetLastError();
  });
}

}  // namespace mq
