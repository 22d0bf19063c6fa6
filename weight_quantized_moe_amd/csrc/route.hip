// Router top-k + softmax, FP16 staging of the hidden rows, and the stable
// grouping of (token, slot) pairs by expert.
//
// Routing follows the reading documented with the library: the k largest
// logits in descending order, ties to the lower expert id, weights = softmax
// over the selected k.  The router stays an unquantized BF16 layer on the
// model cards ("clef-omni-int4" card, section "Recipe": ignore_layers =
// mlp.gate); its logits arrive as an input.
//
// Top-k runs on a group of 16 lanes per token (4 tokens per wave): every lane
// holds E/16 keys, and each of the k rounds finds the largest key as two
// 32-bit maxima (the logit half, then the id half among the keys that hold
// it), each a local maximum plus a 4-step DPP all-reduce inside the 16-lane
// row.
#include "device.h"
#include "gate.h"
#include "internal.h"
#include "route.h"

namespace mq {

// Test entry: FP32 rows [rows, K] -> NVFP4 codes (packed two per byte, low
// nibble first, [rows, K/2]) and E4M3 block scales [rows, K/16], with the
// group arithmetic of rows_to_nvfp4 and the W4A4 gate/up epilogue.  One wave
// per (row, 512-column pass).
__global__ __launch_bounds__(256) void quant_act_nvfp4_kernel(const float *__restrict__ x, int64_t rows,
                                                              int K, float g, uint8_t *__restrict__ codes,
                                                              uint8_t *__restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int passes = (K + 511) / 512;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wid >= rows * passes) return;  // wave-uniform
  const int64_t row = wid / passes;
  const int c = (int)(wid % passes) * 512 + lane * 8;
  const bool ok = c < K;  // K a multiple of 16: lanes 2i and 2i + 1 agree
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = ok ? x[row * K + c + i] : 0.f;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  m = fmaxf(m, __shfl_xor(m, 1, 64));
  const Nvfp4Scale sc = nvfp4_act_scale(m, g);
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= e2m1_code(f[i], g, sc.s) << (4 * i);
  if (ok) {
    *(uint32_t *)(codes + row * (K / 2) + c / 2) = w;
    if ((lane & 1) == 0) scales[row * (K / 16) + c / 16] = (uint8_t)sc.code;
  }
}

hipError_t launch_quant_act_nvfp4(const float *x, int64_t rows, int K, float g, uint8_t *codes,
                                  uint8_t *scales, hipStream_t s) {
  const int64_t waves = rows * ((K + 511) / 512);
  hipLaunchKernelGGL(quant_act_nvfp4_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, x, rows,
                     K, g, codes, scales);
  return hipGetLastError();
}

// Test entry: FP32 rows [rows, K] -> dynamic 1x128 FP8 codes and scales, with
// the same group arithmetic as rows_to_fp8 and the W8A8 GEMM epilogue.  One
// wave per (row, 512-column pass).
__global__ __launch_bounds__(256) void quant_act_kernel(const float *__restrict__ x, int64_t rows, int K,
                                                        uint8_t *__restrict__ codes,
                                                        float *__restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int passes = (K + 511) / 512;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wid >= rows * passes) return;  // wave-uniform
  const int64_t row = wid / passes;
  const int c = (int)(wid % passes) * 512 + lane * 8;
  const bool ok = c < K;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = ok ? x[row * K + c + i] : 0.f;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  m = max16f(m);
  const float s = fp8_group_scale(m);
  if (ok) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    *(u2 *)(codes + row * K + c) = u2{e4m3x4(f[0], f[1], f[2], f[3], s), e4m3x4(f[4], f[5], f[6], f[7], s)};
    if ((lane & 15) == 0) scales[row * (K / 128) + c / 128] = s;
  }
}

hipError_t launch_quant_act(const float *x, int64_t rows, int K, uint8_t *codes, float *scales,
                            hipStream_t s) {
  const int64_t waves = rows * ((K + 511) / 512);
  hipLaunchKernelGGL(quant_act_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, x, rows, K,
                     codes, scales);
  return hipGetLastError();
}

// General-T routing: 16 lanes per token, 4 tokens per wave, one or four
// waves per block.  Also zeroes the
// flags word and, for the prefill path (stage_rows), stages the hidden rows
// in FP16.
template <int kPer, bool kBf16Logits, bool kPermInt4>
__global__ __launch_bounds__(256) void route_kernel(const void *__restrict__ logits,
                                                    const uint16_t *__restrict__ hidden, int T,
                                                    int E, int H, int k, int32_t *__restrict__ ids,
                                                    float *__restrict__ wts,
                                                    _Float16 *__restrict__ x16,
                                                    float *__restrict__ rowscale,
                                                    uint32_t *__restrict__ flags,
                                                    int32_t *__restrict__ p_ids,
                                                    float *__restrict__ p_w, int stage_rows,
                                                    float act_g) {
  const int lane = threadIdx.x & 63, li = lane & 15;
  const int tpb = blockDim.x >> 4;  // tokens per block: 16 lanes each
  const int t = blockIdx.x * tpb + (threadIdx.x >> 4);
  const int t0 = blockIdx.x * tpb + (threadIdx.x >> 6) * 4;  // first token of this wave
  if (blockIdx.x == 0 && threadIdx.x == 0) flags[0] = 0u;
  if (t0 >= T) return;
  static_assert(kRowRegsMaxH == 4 * 64 * 8, "4 x 16 bytes per lane cover one row");
  if (stage_rows == 3) {  // W8A8: FP8 codes and scales of the hidden rows
    if (t < T) topk16<kPer, kBf16Logits>(logits, t, E, k, li, ids, wts, p_ids, p_w);
    rows_to_fp8(hidden, t0, T, H, lane, (uint8_t *)x16, (float *)((uint8_t *)x16 + (size_t)T * H));
    return;
  }
  if (stage_rows == 4) {  // W4A4: the hidden rows as NVFP4 activations
    if (t < T) topk16<kPer, kBf16Logits>(logits, t, E, k, li, ids, wts, p_ids, p_w);
    rows_to_nvfp4(hidden, t0, T, H, lane, act_g, x16, rowscale);
    return;
  }
  if (stage_rows != 0 && H <= kRowRegsMaxH) {
    // rows of up to 2048 values: the rows' loads and the logits' loads in
    // flight together, each row read once (decode keeps only its scale,
    // prefill also writes the FP16 row)
    uint64_t key[kPer];
    if (t < T) topk16_keys<kPer, kBf16Logits>(logits, t, E, li, key);
    u4 v[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[r][u] = t0 + r < T && lane * 8 + 512 * u < H
                      ? *(const u4 *)(hidden + (size_t)(t0 + r) * H + lane * 8 + 512 * u)
                      : u4{0u, 0u, 0u, 0u};
    float down[4];
    row_scale_regs(v, t0, T, H, lane, rowscale, down);
    if (stage_rows == 1) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (t0 + r < T && lane * 8 + 512 * u < H) {
            const u4 o = bf16x8_to_f16x8(v[r][u], down[r]);
            *(u4 *)(x16 + (size_t)(t0 + r) * H + lane * 8 + 512 * u) = kPermInt4 ? perm_0415(o) : o;
          }
    }
    if (t < T) topk16_select<kPer>(key, t, k, li, ids, wts, p_ids, p_w);
    return;
  }
  if (t < T) topk16<kPer, kBf16Logits>(logits, t, E, k, li, ids, wts, p_ids, p_w);
  if (stage_rows) rows_to_f16<kPermInt4>(hidden, t0, T, H, lane, x16, rowscale);
}

// ---------------------------------------------------------------------------
// Router GEMM fused with the top-k: the logits of the BF16 gate (read as a
// linear layer without bias, logits[t, e] = sum_h x[t, h] w[e, h]; the router
// stays unquantized on every card: "clef-omni-int4" card, section "Recipe";
// "clef-omni-NVFP4" card, section "How it was made") are computed for a block
// of 16 or 32 tokens and all E <= 32 EG experts, kept in LDS, and selected there by
// the same 16-lanes-per-token top-k as route_kernel, while the other half of
// the block stages the tokens' hidden rows as route_kernel does.  The logits
// reach HBM only when the caller asks for them (p_logits).
//   GEMM: 16 waves = EG expert groups of 32 x KS = 16 / EG slices of H; each
//   wave computes a 32x32 partial tile (gate_tile, BF16 MFMA, FP32 sums, the
//   next 64-wide chunk loading while one multiplies) and the KS partials of a tile are
//   added through LDS in wave order, so repeated runs are bit-identical.  The
//   16 waves keep enough loads in flight to stream the whole gate through
//   each block (512 KB at 128 experts x 2048).
// ---------------------------------------------------------------------------
constexpr int kGateWaves = 16;

template <int EG, bool kPermInt4, int TB>
__global__ __launch_bounds__(64 * kGateWaves) void gate_route_kernel(
    const uint16_t *__restrict__ hidden, const uint16_t *__restrict__ gate_w, int T, int E, int H,
    int k, int32_t *__restrict__ ids, float *__restrict__ wts, _Float16 *__restrict__ x16,
    float *__restrict__ rowscale, uint32_t *__restrict__ flags, int32_t *__restrict__ p_ids,
    float *__restrict__ p_w, float *__restrict__ p_logits, int stage_rows) {
  constexpr int KS = kGateWaves / EG, kPer = 2 * EG, EP = 32 * EG + 4, NB = TB / 16;
  static_assert(KS >= 2 && (TB == 16 || TB == 32), "H slices per expert group; 16 or 32 tokens");
  __shared__ f4 red[kGateWaves][4][64];  // partial tiles (16 floats per lane)
  __shared__ float lg[TB][EP];           // the block's logits [token][expert]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int ks = wave % KS, eg = wave / KS;
  const int t0 = blockIdx.x * TB, e0 = eg * 32;
  if (blockIdx.x == 0 && threadIdx.x == 0) flags[0] = 0u;
  const bool live = e0 < E;  // an expert group past E still takes the barriers
  const int nchunk = H / 64;
  const int cb = live ? (ks * nchunk) / KS : 0, ce = live ? ((ks + 1) * nchunk) / KS : 0;
  f4 acc[2][2];
  gate_tile<NB>(hidden, gate_w, T, H, E, t0, e0, cb, ce, lane, acc);
  if (ks > 0) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[wave][2 * a + b][lane] = acc[a][b];
  }
  __syncthreads();
  if (ks == 0 && live) {
#pragma unroll
    for (int p = 1; p < KS; ++p)
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f4 v = red[wave + p][2 * a + b][lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[a][b][i] += v[i];
        }
    // MFMA tile (a, b): token 16 b + l % 16, experts e0 + 16 a + 4 (l / 16) + [0, 4)
    const int r16 = lane & 15, q16 = lane >> 4;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) lg[16 * b + r16][e0 + 16 * a + 4 * q16 + i] = acc[a][b][i];
  }
  __syncthreads();
  if (wave < TB / 4) {
    // top-k of token t0 + tl on the 16 lanes of one DPP row
    const int tl = threadIdx.x >> 4, li = threadIdx.x & 15, t = t0 + tl;
    if (t < T) {
      uint64_t key[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = li + 16 * i;
        key[i] = e < E ? ((uint64_t)ordered_key(lg[tl][e]) << 32) | (uint32_t)(0xFFFFFFFFu - (uint32_t)e) : 0;
      }
      topk16_select<kPer>(key, t, k, li, ids, wts, p_ids, p_w);
      if (p_logits)
        for (int e = li; e < E; e += 16) p_logits[(size_t)t * E + e] = lg[tl][e];
    }
  } else if (wave < TB / 2) {
    // hidden rows of 4 tokens per wave: FP16 rows and their powers of two
    // (prefill), the powers of two alone (decode), or nothing (decode with
    // rows longer than kRowRegsMaxH: the GEMM scans them itself)
    const int tr = t0 + 4 * (wave - TB / 4);
    if (stage_rows == 1)
      rows_to_f16<kPermInt4>(hidden, tr, T, H, lane, x16, rowscale);
    else if (stage_rows == 2)
      rows_to_f16<kPermInt4, false>(hidden, tr, T, H, lane, x16, rowscale);
  }
}

// ---------------------------------------------------------------------------
// T <= kSmallT (and T k <= kSmallRows): grouping in one workgroup of 1024
// threads, after route_kernel's top-k (whose 16-lane-per-token selection is
// VALU work worth spreading over several CUs).  A bit mask of tokens per
// expert (one 64-bit word per 64 tokens) gives the counts (popcounts) and the
// stable rank of every token inside its expert (popcount of the mask bits
// below it).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(1024) void group_small_kernel(
    const int32_t *__restrict__ ids, const float *__restrict__ wts, const float *__restrict__ rowscale,
    int T, int E, int k, int32_t *__restrict__ offsets, int32_t *__restrict__ mtile,
    int4 *__restrict__ einfo, int32_t *__restrict__ rcp, int4 *__restrict__ rowinfo,
    int32_t *__restrict__ inv_pos, int32_t *__restrict__ p_offsets, int32_t *__restrict__ p_sorted_tok,
    int32_t *__restrict__ p_inv) {
  __shared__ int32_t sm_ids[kSmallRows];
  group_small_body<1024>(ids, wts, rowscale, T, E, k, offsets, mtile, einfo, rcp, rowinfo,
                         inv_pos, p_offsets, p_sorted_tok, p_inv, sm_ids);
}

// ---------------------------------------------------------------------------
// Decode batches of up to kFusedT tokens: routing and grouping in one
// workgroup of 4 waves (one launch less on the latency-bound smallest steps).
// Each wave takes 4 tokens as route_kernel does (top-k on 16 lanes per token,
// and with rows of at most kRowRegsMaxH values the rows' powers of two); with
// at most 4 tokens each wave takes one token on all its lanes (topk64) and
// wave 0 finds the rows' powers of two.  The ids, weights and powers of two
// stay in LDS for the grouping, and are also written out for the kernels
// after it.
// ---------------------------------------------------------------------------
template <int kPer, bool kBf16Logits>
__global__ __launch_bounds__(256) void route_group_kernel(
    const void *__restrict__ logits, const uint16_t *__restrict__ hidden, int T, int E, int H, int k,
    int32_t *__restrict__ ids, float *__restrict__ wts, float *__restrict__ rowscale,
    uint32_t *__restrict__ flags, int32_t *__restrict__ p_ids, float *__restrict__ p_w, int with_scales,
    int32_t *__restrict__ offsets, int32_t *__restrict__ mtile, int4 *__restrict__ einfo,
    int32_t *__restrict__ rcp, int4 *__restrict__ rowinfo,
    int32_t *__restrict__ inv_pos, int32_t *__restrict__ p_offsets, int32_t *__restrict__ p_sorted_tok,
    int32_t *__restrict__ p_inv) {
  __shared__ int32_t s_ids[kFusedT * 64];
  __shared__ float s_wts[kFusedT * 64];
  __shared__ float s_rs[kFusedT];
  const int lane = threadIdx.x & 63, li = lane & 15;
  const int t = threadIdx.x >> 4, t0 = (threadIdx.x >> 6) * 4;
  if (threadIdx.x == 0) flags[0] = 0u;
  if (T <= 4) {
    // one token per wave on all its lanes (wave 0 also finds the rows' powers of two)
    const int wave = threadIdx.x >> 6;
    if (wave == 0 && with_scales) {
      u4 v[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[r][u] = r < T && lane * 8 + 512 * u < H ? *(const u4 *)(hidden + (size_t)r * H + lane * 8 + 512 * u)
                                                     : u4{0u, 0u, 0u, 0u};
      row_scale_regs(v, 0, T, H, lane, s_rs);
    }
    if (wave < T) topk64<kPer / 4, kBf16Logits>(logits, wave, E, k, lane, s_ids, s_wts, p_ids, p_w);
  } else if (t0 < T) {
    uint64_t key[kPer];
    if (t < T) topk16_keys<kPer, kBf16Logits>(logits, t, E, li, key);
    if (with_scales) {
      u4 v[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[r][u] = t0 + r < T && lane * 8 + 512 * u < H
                        ? *(const u4 *)(hidden + (size_t)(t0 + r) * H + lane * 8 + 512 * u)
                        : u4{0u, 0u, 0u, 0u};
      row_scale_regs(v, t0, T, H, lane, s_rs);
    }
    if (t < T) topk16_select<kPer>(key, t, k, li, s_ids, s_wts, p_ids, p_w);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * k; i += 256) {
    ids[i] = s_ids[i];
    wts[i] = s_wts[i];
  }
  if (with_scales && threadIdx.x < T) rowscale[threadIdx.x] = s_rs[threadIdx.x];
  group_small_body<256>(s_ids, s_wts, with_scales ? s_rs : nullptr, T, E, k, offsets, mtile, einfo, rcp,
                        rowinfo, inv_pos, p_offsets, p_sorted_tok, p_inv, s_ids);
}

// ---------------------------------------------------------------------------
// Stable grouping by expert for larger batches, in three launches over chunks of
// consecutive tokens (at most kMaxChunks chunks):
//   1. hist_kernel:    per-chunk expert counts cnt[c][e];
//   2. scan_kernel:    one workgroup turns them into the exclusive position of
//                      every chunk's first row of expert e,
//                      base[c][e] = offsets[e] + sum_{c' < c} cnt[c'][e],
//                      plus offsets, M-tile prefix and the active-expert list;
//   3. scatter_kernel: ranks inside a chunk, 256 tokens at a time (4 waves x 64
//                      lanes): per wave and expert the 64-bit mask of lanes
//                      routed there; a row's rank is (rows of earlier waves) +
//                      popcount(mask & lanes below it), which keeps token order
//                      inside every expert.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void hist_kernel(const int32_t *__restrict__ ids, int T, int E,
                                                   int k, int chunk, int32_t *__restrict__ cnt) {
  extern __shared__ int32_t sc[];  // [E]
  const int tid = threadIdx.x;
  for (int e = tid; e < E; e += 256) sc[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * chunk, t1 = min(T, t0 + chunk);
  for (int i = t0 * k + tid; i < t1 * k; i += 256) atomicAdd(&sc[ids[i]], 1);
  __syncthreads();
  for (int e = tid; e < E; e += 256) cnt[(size_t)blockIdx.x * E + e] = sc[e];
}

__global__ __launch_bounds__(1024) void scan_kernel(int32_t *__restrict__ cnt, int nc, int E,
                                                    int32_t *__restrict__ offsets,
                                                    int32_t *__restrict__ mtile,
                                                    int4 *__restrict__ einfo,
                                                    int32_t *__restrict__ rcp,
                                                    int32_t *__restrict__ p_offsets) {
  __shared__ int32_t tot[kMaxExperts];
  __shared__ int32_t off[kMaxExperts];
  __shared__ int32_t subpre[kMaxExperts][8];
  const int tid = threadIdx.x, sub = tid & 7;
  // 8 threads per expert, each over a contiguous range of chunks
  const int per = (nc + 7) / 8, c0 = min(nc, sub * per), c1 = min(nc, c0 + per);
  for (int e0 = 0; e0 < E; e0 += 128) {
    const int e = e0 + (tid >> 3);
    int s = 0;
    if (e < E)
      for (int c = c0; c < c1; ++c) s += cnt[(size_t)c * E + e];
    int incl = s;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      const int v = __shfl_up(incl, d, 8);
      if (sub >= d) incl += v;
    }
    if (e < E) {
      subpre[e][sub] = incl - s;
      if (sub == 7) tot[e] = incl;
    }
  }
  __syncthreads();
  if (tid < 64) scan_experts_wave(tot, E, tid, offsets, mtile, einfo, rcp, p_offsets, off);
  __syncthreads();
  for (int e0 = 0; e0 < E; e0 += 128) {
    const int e = e0 + (tid >> 3);
    if (e >= E) continue;
    int run = off[e] + subpre[e][sub];
    for (int c = c0; c < c1; ++c) {
      const int v = cnt[(size_t)c * E + e];
      cnt[(size_t)c * E + e] = run;
      run += v;
    }
  }
}

__global__ __launch_bounds__(256) void scatter_kernel(
    const int32_t *__restrict__ ids, const float *__restrict__ wts,
    const float *__restrict__ rowscale, int T, int E, int k, int chunk,
    const int32_t *__restrict__ base, int4 *__restrict__ rowinfo, int32_t *__restrict__ inv_pos,
    int32_t *__restrict__ p_sorted_tok, int32_t *__restrict__ p_inv) {
  extern __shared__ __align__(16) unsigned char smem[];
  uint64_t *mask = (uint64_t *)smem;              // [4][E]
  int32_t *wbase = (int32_t *)(mask + 4 * E);     // [4][E]
  int32_t *cursor = wbase + 4 * E;                // [E]
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int e = tid; e < E; e += 256) cursor[e] = base[(size_t)blockIdx.x * E + e];
  const int t0 = blockIdx.x * chunk, t1 = min(T, t0 + chunk);
  const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
  for (int s0 = t0; s0 < t1; s0 += 256) {
    for (int i = tid; i < 4 * E; i += 256) mask[i] = 0ull;
    __syncthreads();
    const int t = s0 + tid;
    const bool valid = t < t1;
    if (valid)
      for (int j = 0; j < k; ++j) atomicOr(&mask[wave * E + ids[(size_t)t * k + j]], 1ull << lane);
    __syncthreads();
    for (int e = tid; e < E; e += 256) {
      int run = cursor[e];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        wbase[w * E + e] = run;
        run += __popcll(mask[w * E + e]);
      }
      cursor[e] = run;
    }
    __syncthreads();
    if (valid) {
      for (int j = 0; j < k; ++j) {
        const int e = ids[(size_t)t * k + j];
        const int pos = wbase[wave * E + e] + __popcll(mask[wave * E + e] & below);
        const int slot = t * k + j;
        const float rs = rowscale ? rowscale[t] : 0.f;
        rowinfo[pos] = int4{slot, t, __builtin_bit_cast(int, rs), __builtin_bit_cast(int, wts[slot])};
        inv_pos[slot] = pos;
        if (p_sorted_tok) p_sorted_tok[pos] = t;
        if (p_inv) p_inv[slot] = pos;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
template <int kPer, bool kBf16, bool kPerm>
static hipError_t route_dispatch(const LayerDims &L, const FwdPtrs &P, const Workspace &W,
                                 int stage_rows, hipStream_t s) {
  char *ws = P.ws;
  // decode batches: one wave (4 tokens) per workgroup spreads the row reads
  // over more CUs; otherwise 16 tokens per workgroup
  const int threads = stage_rows == 2 || P.T <= 256 ? 64 : 256, tpb = threads / 16;
  hipLaunchKernelGGL((route_kernel<kPer, kBf16, kPerm>), dim3((P.T + tpb - 1) / tpb), dim3(threads), 0, s,
                     P.logits, P.hidden, P.T, L.E, L.H, L.k, (int32_t *)(ws + W.topk_ids),
                     (float *)(ws + W.topk_w), (_Float16 *)(ws + W.x16), (float *)(ws + W.rowscale),
                     P.flags, P.p_ids, P.p_w, stage_rows, P.act_g13);
  return hipGetLastError();
}

template <int kPer>
static hipError_t route_dispatch2(const LayerDims &L, const FwdPtrs &P, const Workspace &W,
                                  int stage_rows, hipStream_t s) {
  const bool perm = L.fmt == FMT_INT4;
  if (P.logits_bf16)
    return perm ? route_dispatch<kPer, true, true>(L, P, W, stage_rows, s)
                : route_dispatch<kPer, true, false>(L, P, W, stage_rows, s);
  return perm ? route_dispatch<kPer, false, true>(L, P, W, stage_rows, s)
              : route_dispatch<kPer, false, false>(L, P, W, stage_rows, s);
}

template <int kPer>
static hipError_t route_group_dispatch(const LayerDims &L, const FwdPtrs &P, const Workspace &W,
                                       int stage_rows, hipStream_t s) {
  char *ws = P.ws;
  auto k = P.logits_bf16 ? route_group_kernel<kPer, true> : route_group_kernel<kPer, false>;
  hipLaunchKernelGGL(k, dim3(1), dim3(256), 0, s, P.logits, P.hidden, P.T, L.E, L.H, L.k,
                     (int32_t *)(ws + W.topk_ids), (float *)(ws + W.topk_w), (float *)(ws + W.rowscale),
                     P.flags, P.p_ids, P.p_w, stage_rows == 2 ? 1 : 0, (int32_t *)(ws + W.offsets),
                     (int32_t *)(ws + W.mtile), (int4 *)(ws + W.active), (int32_t *)(ws + W.rcpre),
                     (int4 *)(ws + W.rowinfo), (int32_t *)(ws + W.inv_pos),
                     P.p_offsets, P.p_sorted_tok, P.p_inv);
  return hipGetLastError();
}

template <int EG, bool kPerm>
static hipError_t gate_route_launch(const LayerDims &L, const FwdPtrs &P, const Workspace &W,
                                    int stage_rows, hipStream_t s) {
  char *ws = P.ws;
  // 16 tokens per block up to 8192 tokens (twice the blocks: the batch then
  // spreads over more CUs), 32 above (half the gate reads from L2)
  if (P.T <= 8192) {
    hipLaunchKernelGGL((gate_route_kernel<EG, kPerm, 16>), dim3((P.T + 15) / 16), dim3(64 * kGateWaves), 0, s,
                       P.hidden, P.gate_w, P.T, L.E, L.H, L.k, (int32_t *)(ws + W.topk_ids),
                       (float *)(ws + W.topk_w), (_Float16 *)(ws + W.x16), (float *)(ws + W.rowscale),
                       P.flags, P.p_ids, P.p_w, P.p_logits, stage_rows);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((gate_route_kernel<EG, kPerm, 32>), dim3((P.T + 31) / 32), dim3(64 * kGateWaves), 0, s, P.hidden,
                     P.gate_w, P.T, L.E, L.H, L.k, (int32_t *)(ws + W.topk_ids), (float *)(ws + W.topk_w),
                     (_Float16 *)(ws + W.x16), (float *)(ws + W.rowscale), P.flags, P.p_ids, P.p_w,
                     P.p_logits, stage_rows);
  return hipGetLastError();
}

template <bool kPerm>
static hipError_t gate_route_dispatch(const LayerDims &L, const FwdPtrs &P, const Workspace &W,
                                      int stage_rows, hipStream_t s) {
  if (L.E <= 32) return gate_route_launch<1, kPerm>(L, P, W, stage_rows, s);
  if (L.E <= 64) return gate_route_launch<2, kPerm>(L, P, W, stage_rows, s);
  if (L.E <= 128) return gate_route_launch<4, kPerm>(L, P, W, stage_rows, s);
  return gate_route_launch<8, kPerm>(L, P, W, stage_rows, s);  // E <= kMaxGateExperts
}

hipError_t launch_route(const LayerDims &L, const FwdPtrs &P, const Workspace &W, bool decode,
                        hipStream_t s) {
  // prefill: FP16 rows and their scales (1); decode with H <= 2048: the
  // scales only (2), the decode gate/up GEMM converts the rows it stages;
  // larger decode rows: the GEMM finds the scales too (0); W8A8: FP8 codes
  // and scales (3); W4A4: NVFP4 values and 1 / g (4)
  const int stage_rows = P.w8a8 ? 3 : P.act_g13 > 0.f ? 4 : !decode ? 1 : L.H <= kRowRegsMaxH ? 2 : 0;
  if (P.gated) return launch_route_gated(L, P, W, decode, stage_rows, s);
  if (P.gate_w && P.T >= kGateFusedMinT)  // router GEMM fused with the top-k
    return L.fmt == FMT_INT4 ? gate_route_dispatch<true>(L, P, W, stage_rows, s)
                             : gate_route_dispatch<false>(L, P, W, stage_rows, s);
  if (P.gate_w) {
    // small batch: the router logits kernel, then route_kernel on its logits
    FwdPtrs Q = P;
    float *lg = P.p_logits ? P.p_logits : (float *)(P.ws + W.logits);
    hipError_t e = launch_router_logits(P.hidden, P.gate_w, lg, P.T, L.H, L.E, s);
    if (e != hipSuccess) return e;
    Q.logits = lg;
    Q.logits_bf16 = 0;
    Q.gate_w = nullptr;
    return launch_route(L, Q, W, decode, s);
  }
  if (route_groups(L, P, decode)) {
    if (L.E <= 128) return route_group_dispatch<8>(L, P, W, stage_rows, s);
    if (L.E <= 256) return route_group_dispatch<16>(L, P, W, stage_rows, s);
    return route_group_dispatch<32>(L, P, W, stage_rows, s);
  }
  if (L.E <= 128) return route_dispatch2<8>(L, P, W, stage_rows, s);
  if (L.E <= 256) return route_dispatch2<16>(L, P, W, stage_rows, s);
  return route_dispatch2<32>(L, P, W, stage_rows, s);
}

bool route_groups(const LayerDims &L, const FwdPtrs &P, bool decode) {
  (void)L;
  return decode && !P.w8a8 && P.act_g13 == 0.f && P.T <= kFusedT;
}

hipError_t launch_permute(const LayerDims &L, const FwdPtrs &P, const Workspace &W, bool decode,
                          hipStream_t s) {
  char *ws = P.ws;
  if (route_groups(L, P, decode)) return hipSuccess;  // the routing kernel grouped the rows
  if (P.T <= kSmallT && P.T * L.k <= kSmallRows) {
    hipLaunchKernelGGL(group_small_kernel, dim3(1), dim3(1024), 0, s, (const int32_t *)(ws + W.topk_ids),
                       (const float *)(ws + W.topk_w), decode && L.H > kRowRegsMaxH ? (const float *)nullptr : (const float *)(ws + W.rowscale),
                       P.T, L.E, L.k, (int32_t *)(ws + W.offsets), (int32_t *)(ws + W.mtile),
                       (int4 *)(ws + W.active), (int32_t *)(ws + W.rcpre), (int4 *)(ws + W.rowinfo),
                       (int32_t *)(ws + W.inv_pos), P.p_offsets, P.p_sorted_tok, P.p_inv);
    return hipGetLastError();
  }
  int nc, chunk;
  permute_chunks(P.T, &nc, &chunk);
  int32_t *cnt = (int32_t *)(ws + W.chunks);
  hipLaunchKernelGGL(hist_kernel, dim3(nc), dim3(256), (size_t)L.E * 4, s,
                     (const int32_t *)(ws + W.topk_ids), P.T, L.E, L.k, chunk, cnt);
  hipLaunchKernelGGL(scan_kernel, dim3(1), dim3(1024), 0, s, cnt, nc, L.E,
                     (int32_t *)(ws + W.offsets), (int32_t *)(ws + W.mtile),
                     (int4 *)(ws + W.active), (int32_t *)(ws + W.rcpre), P.p_offsets);
  hipLaunchKernelGGL(scatter_kernel, dim3(nc), dim3(256), (size_t)L.E * (4 * 8 + 4 * 4 + 4), s,
                     (const int32_t *)(ws + W.topk_ids), (const float *)(ws + W.topk_w),
                     decode && L.H > kRowRegsMaxH ? nullptr : (const float *)(ws + W.rowscale), P.T, L.E, L.k, chunk,
                     (const int32_t *)cnt, (int4 *)(ws + W.rowinfo), (int32_t *)(ws + W.inv_pos), P.p_sorted_tok,
                     P.p_inv);
  return hipGetLastError();
}

}  // namespace mq
