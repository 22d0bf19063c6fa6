// The dense E4M3 product: y[t, n] = sum_g sa[t, g] sw[n / 128, g] sum_{k in g} a[t, k] w[n, k].
//
// Both operands are E4M3 codes, so for a BF16 output one 16x16x128 FP8 matrix
// instruction takes the whole inner sum of a block of 128 for 16 weight rows and
// 16 tokens; the block's two scales multiply it in FP32 on the way into the
// accumulator.  That instruction aligns its 128 products to the largest and cuts
// them there: on random codes the sum is off by 2^-14 of the largest product in
// the mean and by 2^-10.8 at most, which a BF16 output does not show (an FP32 one
// does: 3e-5 of its 2-norm).  For an FP32 output the codes become FP16 values
// (exact) and go through four 16x16x32 FP16 instructions, whose sums are FP32
// ones (2^-23.7 of the largest product in the mean), at half the rate.
//
// For many tokens bound by instructions: at 8192^3 the 256 x 256 tiles take 510 us in the
// median (2155 TFLOP/s, the quantization aside; 482 at the least), with the matrix units
// busy 52% of the cycles and the vector units 40%, mostly the four scaling sums per matrix
// instruction (a copy without those ran 13% faster, one without the copies into LDS
// 20%); the library's product of E4M3 tensors with one scale each reaches 2716 TFLOP/s.
// 16384 x 5120 x 2048: 187 to 196 us (1750 to 1840 TFLOP/s; 178 at the least), about a
// tenth of it the tiles' starts and ends, after 24 us for the quantization (100 MB).
// Outputs of N % 8 != 0 are stored value by value (8192 x 5121: 192 us a call, x 5120
// 118).  For few tokens bound by launches and latency.
//
// Three ways through it:
//   few tokens     one launch: every workgroup quantizes the rows itself
//   some           the rows quantized into the workspace, then the weights
//                  streamed from memory to registers, the axis K over the waves
//   many           the rows quantized, then tiles of tokens and weight rows
//                  through LDS
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"

namespace mq {
namespace {

typedef int i8v __attribute__((ext_vector_type(8)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
// 16-byte values at any even address (rows of an odd number of values)
typedef u4 u4_a2 __attribute__((aligned(2)));

// 16 weight rows (a) x 16 tokens (b) x 128 k; E8M0 scale 127 = 2^0 on both.
// Lane l holds row l % 16 of each operand and the same 32 of the 128 k (any,
// as long as both agree); of the result, token l % 16 and weight rows
// 4 (l / 16) + [0, 4).
__device__ __forceinline__ f4 mfma_fp8_16(const i8v &a, const i8v &b, const f4 &c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// A lane's 32 codes of a row and a block of 128, as its products take them.
template <bool kExact>
struct Frag;
template <>
struct Frag<false> {
  i8v v;
  __device__ __forceinline__ void set(u4 x, u4 y) {
    v = i8v{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }
};
template <>
struct Frag<true> {
  h8 v[4];
  __device__ __forceinline__ void set(u4 x, u4 y) {
    v[0] = unpack_fp8(x[0], x[1]);
    v[1] = unpack_fp8(x[2], x[3]);
    v[2] = unpack_fp8(y[0], y[1]);
    v[3] = unpack_fp8(y[2], y[3]);
  }
};
__device__ __forceinline__ f4 block_sum(const Frag<false> &a, const Frag<false> &b) {
  return mfma_fp8_16(a.v, b.v, f4{0.f, 0.f, 0.f, 0.f});
}
__device__ __forceinline__ f4 block_sum(const Frag<true> &a, const Frag<true> &b) {
  f4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = mfma16(a.v[i], b.v[i], p);
  return p;
}

// ---- quantization: 16 lanes take one block of 128 of one token, 8 values each.
// The scale's product and the one division per value are the definition's, so that
// the codes are its codes bit for bit (many quotients of BF16 values lie midway
// between two codes).  The division v / s by one reciprocal per block: with y the
// rounded 1 / s and q the rounded v y, which is within a step of v / s, the
// remainder v - q s is exact in one FMA and q + remainder y rounds to the rounded
// v / s (Markstein's theorem), unless the remainder underflows or the mantissa of s
// is all ones: such blocks, rare ones, divide.  A block with a NaN or an infinity in it
// has a scale of NaN, so its token's results are NaN.
__device__ __forceinline__ u2 quantize8(u4 v, float *scale) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
  }
  // the maximum that keeps NaN
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __builtin_elementwise_maximum(m, fabsf(f[i]));
#pragma unroll
  for (int s = 1; s < 16; s *= 2) m = __builtin_elementwise_maximum(m, __shfl_xor(m, s, 64));
  const float u = m * (1.f / 448.f), s = u == 0.f ? 1.f : u;
  *scale = s;
  if (__any(!(s >= 0x1p-60f && s <= 0x1p120f) || (__float_as_uint(s) & 0x7FFFFFu) == 0x7FFFFFu)) {
    if (s == INFINITY) *scale = __builtin_nanf("");
    return u2{e4m3x4(f[0], f[1], f[2], f[3], s), e4m3x4(f[4], f[5], f[6], f[7], s)};
  }
  const float y = 1.f / s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = f[i] * y;
    f[i] = __builtin_amdgcn_fmed3f(__builtin_fmaf(__builtin_fmaf(-q, s, f[i]), y, q), -448.f, 448.f);
  }
  u2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
    c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], w, true);
  }
  return c;
}

// Workgroups of a launch, of at most 512 lanes: a grid has fewer than 2^32 lanes.
constexpr int64_t kMostGroups = (1 << 23) - 8;
constexpr int64_t kQuantGroups = 1 << 22;   // workgroups at most: 2^30 lanes

__global__ __launch_bounds__(256) void linear_quant_kernel(LinearArgs a) {
  // 16 lanes at a time, so the shuffles stay among live lanes
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < a.T * a.G * 16; id += (int64_t)gridDim.x * 256) {
    const int64_t grp = id >> 4, t = grp / a.G;
    const int g = (int)(grp - t * a.G), at = g * 128 + 8 * (int)(id & 15);
    float s;
    const u2 c = quantize8(at < a.K ? *(const u4 *)(a.x + t * a.K + at) : u4{0u, 0u, 0u, 0u}, &s);
    *(u2 *)(a.codes + t * (a.G * (int64_t)128) + at) = c;
    if ((id & 15) == 0) a.sa[g * a.T + t] = s;
  }
}

// To nearest even by the conversion instruction: a tile's 128 values a lane cost 64 of
// them where the rounding written out takes ten a value, 4 us of a tile of 256 x 256.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  b2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// out[t, n .. n + W) = round(y + residual); fast: all W there and rows 16-byte aligned
template <int W>
__device__ __forceinline__ void store(const LinearArgs &a, int64_t t, int n, const float *y, bool fast) {
  const int64_t at = t * a.N + n;
  if (W >= 8 && fast) {
#pragma unroll
    for (int w = 0; w + 8 <= W; w += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = y[w + i];
      if (a.residual) {
        const u4 r = *(const u4_a2 *)(a.residual + at + w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] += bf16_to_f32(r[i] & 0xFFFFu);
          v[2 * i + 1] += bf16_to_f32(r[i] >> 16);
        }
      }
      if (a.out_bf16) {
        u4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = bf16x2(v[2 * i], v[2 * i + 1]);
        *(u4 *)((uint16_t *)a.out + at + w) = o;
      } else {
        *(f4 *)((float *)a.out + at + w) = f4{v[0], v[1], v[2], v[3]};
        *(f4 *)((float *)a.out + at + w + 4) = f4{v[4], v[5], v[6], v[7]};
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (n + i >= a.N) continue;
    float v = y[i];
    if (a.residual) v += bf16_to_f32(a.residual[at + i]);
    if (a.out_bf16)
      ((uint16_t *)a.out)[at + i] = (uint16_t)bf16x2(v, v);
    else
      ((float *)a.out)[at + i] = v;
  }
}

// ---- few and some tokens: a workgroup of 8 waves takes 16 NT weight rows and 16 MT
// tokens, each wave every 8th block of K, U of its blocks at a time, whose loads are
// all on their way before the first product; the weights go straight from memory to
// registers.  kFused: the workgroup quantizes its (at most 16) tokens' rows into LDS
// while its first weights are on their way; else the codes are read from the
// workspace.
constexpr int kStreamWaves = 8;

template <bool kExact, int NT, int MT, int U, bool kFused>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(LinearArgs a) {
  constexpr int W = kStreamWaves, N = 64 * W;
  // keeps the compiler from asking for the pointers only where the first weights need
  // them, a round trip of 0.3 of one token's 4.6 us
  if constexpr (kFused) asm volatile("" ::"s"(a.x), "s"(a.w), "s"(a.scale));
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ f4 part[W][NT * MT][64];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int tiles = (a.N + 16 * NT - 1) / (16 * NT);
  const int tt = blockIdx.x / tiles, n0 = (blockIdx.x - tt * tiles) * 16 * NT;
  const int64_t t0 = (int64_t)tt * 16 * MT;
  const int G = a.G;
  const int64_t Kp = G * (int64_t)128;
  const uint8_t *wp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) wp[j] = a.w + (int64_t)min(n0 + 16 * j + r, a.N - 1) * a.K;  // rows past the end: never stored
  const float *sw = a.scale + (int64_t)(n0 / 128) * G;
  u4 w[U][NT][2];
  float f[U];
  // blocks g, g + W, ...; those past the last are the last once more, times 0
  auto weights = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(g + u * W, G - 1), k0 = at * 128 + 16 * q, k1 = k0 + 64;
      f[u] = g + u * W < G ? sw[at] : 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        // chunks past K: the codes are 0 there, so any chunk of the same weight row will do
        w[u][j][0] = *(const u4 *)(wp[j] + (k0 < a.K ? k0 : 0));
        w[u][j][1] = *(const u4 *)(wp[j] + (k1 < a.K ? k1 : 0));
      }
    }
  };
  weights(wave);
  const unsigned char *xs = smem;                                   // fused: codes [T][Kp + 16]
  float *ss = (float *)(smem + a.T * (Kp + 16));                    // and scales [T][G]
  if constexpr (kFused) {
    const int chunks = (int)a.T * G * 16;
    for (int id = tid; id < chunks; id += N) {                      // multiples of 16: see the shuffles
      const int t = id / (G * 16), at = (id - t * G * 16) * 8;
      float s;
      const u2 c = quantize8(at < a.K ? *(const u4 *)(a.x + (int64_t)t * a.K + at) : u4{0u, 0u, 0u, 0u}, &s);
      *(u2 *)(smem + t * (Kp + 16) + at) = c;
      if ((id & 15) == 0) ss[t * G + at / 128] = s;
    }
    __syncthreads();
  }
  int64_t tc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) tc[m] = min(t0 + 16 * m + r, a.T - 1);  // tokens past the end: never stored
  f4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[j][m] = f4{0.f, 0.f, 0.f, 0.f};
  for (int g = wave; g < G; g += U * W) {
    if (g != wave) weights(g);
    u4 x[U][MT][2];
    float s[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(g + u * W, G - 1);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint8_t *p = kFused ? xs + tc[m] * (Kp + 16) : a.codes + tc[m] * Kp;
        x[u][m][0] = *(const u4 *)(p + at * 128 + 16 * q);
        x[u][m][1] = *(const u4 *)(p + at * 128 + 16 * q + 64);
        s[u][m] = kFused ? ss[tc[m] * G + at] : a.sa[at * a.T + tc[m]];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Frag<kExact> wf[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) wf[j].set(w[u][j][0], w[u][j][1]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        Frag<kExact> b;
        b.set(x[u][m][0], x[u][m][1]);
        const float sf = s[u][m] * f[u];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const f4 p = block_sum(wf[j], b);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][m][i] = __builtin_fmaf(p[i], sf, acc[j][m][i]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][j * MT + m][lane] = acc[j][m];
  __syncthreads();
  // a wave adds up a result of 16 x 16
  if (wave < NT * MT) {
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const f4 p = part[v][wave][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += p[i];
    }
    const int64_t t = t0 + 16 * (wave % MT) + r;
    if (t < a.T) store<4>(a, t, n0 + 16 * (wave / MT) + 4 * q, y, false);
  }
}

// ---- many tokens: tiles of BM tokens x BN weight rows, WM x WN waves, each with
// TM x 4 results of 16 x 16; KS times as many waves take KS blocks of K at a time,
// and their sums are added at the end.
//
// A k step is one block of 128: BM rows of activation codes, BN of weight codes (128
// bytes each) and BM activation scales, copied from global memory straight into
// one of kStages stages of LDS, kStages - 1 steps ahead; one barrier a step.
//
// A wave's 64 weight rows are dealt to its 4 results so that a lane ends up with 8
// consecutive ones in a pair of results: row rho of result j is weight row 32 (j / 2) +
// 8 (rho / 4) + 4 (j % 2) + rho % 4, so lane group g (rho / 4 in the result's rows) holds
// 8 g + [0, 8) of each half.  A lane then stores 16 bytes of a token's row and four
// lanes 64 that lie side by side.
//
// LDS: chunk c (16 bytes) of row r lies at slot 8 r + (c ^ swz(r)); the 16 rows that
// 16 lanes read at once are consecutive for the tokens (swz = r / 2) and rho's above
// for the weights (swz = 2 (r / 8) + r / 2 % 2), 16 different of 2 x 8 slots either way.
typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ void dma16(const void *g, unsigned char *lds) {
  __builtin_amdgcn_global_load_lds(g, (lds_void *)lds, 16, 0, 0);
}
__device__ __forceinline__ void dma4(const void *g, unsigned char *lds) {
  __builtin_amdgcn_global_load_lds(g, (lds_void *)lds, 4, 0, 0);
}
// s_waitcnt vmcnt(n), other counters left alone
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

template <int WM, int WN, int TM, int STAGES, int KS>
struct Tile {
  static constexpr int kWaves = WM * WN, BM = WM * TM * 16, BN = WN * 64;
  static constexpr int kStages = STAGES;
  static constexpr int kTokenCopies = BM / 8 / kWaves, kWeightCopies = BN / 8 / kWaves;  // per wave and step, 1 KB each
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "waves copy whole groups of 8 rows");
  static constexpr int kScaleRows = BM < 64 ? 64 : BM;             // copied 64 at a time
  static constexpr int kBlockBytes = (BM + BN) * 128 + kScaleRows * 4, kStageBytes = KS * kBlockBytes;
  static constexpr int kBlocks = (BN + 127) / 128;                 // weight blocks that a tile may touch
  static constexpr int lds(int G) { return kStages * kStageBytes + kBlocks * G * 4; }
};

template <bool kExact, int WM, int WN, int TM, int STAGES, int KS>
__global__ __launch_bounds__(64 * WM * WN * KS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void linear_tiles_kernel(LinearArgs a) {
  using L = Tile<WM, WN, TM, STAGES, KS>;
  constexpr int BM = L::BM, BN = L::BN, kStages = L::kStages, CX = L::kTokenCopies, CW = L::kWeightCopies;
  extern __shared__ __align__(16) unsigned char smem[];
  float *sws = (float *)(smem + kStages * L::kStageBytes);
  const int tid = threadIdx.x, all_waves = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int ks = all_waves / L::kWaves, wave = all_waves - ks * L::kWaves;
  const int G = a.G, K = a.K;
  const int64_t Kp = G * (int64_t)128;
  // ---- tile of this workgroup.  The 8 XCDs take contiguous ranges; inside a range
  // tiles go down kDown token tiles before the next column of weight rows, so that
  // the tiles at work at one time share rows of both kinds in their XCD's cache.
  constexpr int kDown = 8;
  const int mt = (int)((a.T + BM - 1) / BM), nt = (a.N + BN - 1) / BN, all = mt * nt;
  const int per = (all + 7) / 8, x = blockIdx.x & 7, s0 = blockIdx.x >> 3;
  const int id = x * per + s0;
  if (s0 >= per || id >= all) return;
  const int band = id / (kDown * nt), first = band * kDown, high = min(kDown, mt - first), in = id - band * kDown * nt;
  const int64_t t0 = (int64_t)(first + in % high) * BM;
  const int n0 = in / high * BN;
  // ---- weight scales of the tile's blocks (0 past the end)
  const int nb = (a.N + 127) / 128;
  for (int i = tid; i < L::kBlocks * G; i += 64 * L::kWaves * KS) {
    const int b = i / G, g = i - b * G, at = n0 / 128 + b;
    sws[i] = at < nb ? a.scale[(int64_t)at * G + g] : 0.f;
  }
  // ---- copies: a wave's number p fills rows 8 (CX wave + p) + [0, 8) of the tokens'
  // part of the stage, CW of the weights'; rows past the end copy the last row,
  // which is never stored
  const uint8_t *xbase = a.codes + t0 * Kp, *wbase = a.w + (int64_t)n0 * K;
  uint32_t xoff[CX], woff[CW];
#pragma unroll
  for (int p = 0; p < CX; ++p) {
    const int row = 8 * (CX * wave + p) + (lane >> 3);
    xoff[p] = (uint32_t)(min((int64_t)row, a.T - 1 - t0) * Kp) + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  auto wchunk = [&](int p) {
    const int row = 8 * (CW * wave + p) + (lane >> 3);
    return 16 * ((lane & 7) ^ (2 * ((row >> 3) & 3) + ((row >> 1) & 1)));
  };
#pragma unroll
  for (int p = 0; p < CW; ++p)
    woff[p] = (uint32_t)min(8 * (CW * wave + p) + (lane >> 3), a.N - 1 - n0) * (uint32_t)K + wchunk(p);
  // activation scales: wave w copies those of tokens 64 (w % (kScaleRows / 64)) + [0, 64)
  const int sg = wave % (L::kScaleRows / 64);
  const float *sbase = a.sa + min(t0 + 64 * sg + lane, a.T - 1);
  // steps of the axis: block KS g + ks, the last one again behind the end (times 0)
  const int steps = (G + KS - 1) / KS;
  auto issue = [&](int step) {
    unsigned char *st = smem + (step % kStages) * L::kStageBytes + ks * L::kBlockBytes;
    const int g = KS == 1 ? step : min(KS * step + ks, G - 1);
    const uint8_t *xg = xbase + g * 128, *wg = wbase + g * 128;
#pragma unroll
    for (int p = 0; p < CX; ++p) dma16(xg + xoff[p], st + 1024 * (CX * wave + p));
    if (g * 128 + 128 <= K) {
#pragma unroll
      for (int p = 0; p < CW; ++p) dma16(wg + woff[p], st + BM * 128 + 1024 * (CW * wave + p));
    } else {
      // chunks past K meet codes of 0: the same row's first one will do
#pragma unroll
      for (int p = 0; p < CW; ++p) {
        const int c = wchunk(p);
        const uint32_t back = g * 128 + c < K ? 0u : (uint32_t)(g * 128 + c);
        dma16(wg + woff[p] - back, st + BM * 128 + 1024 * (CW * wave + p));
      }
    }
    dma4(sbase + (int64_t)g * a.T, st + (BM + BN) * 128 + 256 * sg);
  };
  // ---- the wave's part of the tile
  const int wm = wave / WN, wn = wave - wm * WN;
  const int tok = wm * TM * 16 + r;                                   // + 16 m
  const int wrow = wn * 64 + 8 * (r >> 2) + (r & 3);                  // + 32 (j / 2) + 4 (j % 2)
  const int blk = (wn * 64) / 128;
  f4 acc[TM][4];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f4{0.f, 0.f, 0.f, 0.f};
  // One k step: the next token rows' operand and the sums of the rows before are in
  // work while the matrix units multiply (the barriers keep the compiler from
  // putting each read right in front of its use).
  auto compute = [&](int step) {
    const unsigned char *st = smem + (step % kStages) * L::kStageBytes + ks * L::kBlockBytes, *ws = st + BM * 128;
    const float *ss = (const float *)(st + (BM + BN) * 128);
    const int g = KS * step + ks;
    const float f = KS == 1 || g < G ? sws[blk * G + g] : 0.f;
    auto token = [&](int m, Frag<kExact> &b) {
      const int t = tok + 16 * m, z = (t >> 1) & 7;
      b.set(*(const u4 *)(st + t * 128 + 16 * (q ^ z)), *(const u4 *)(st + t * 128 + 16 * ((q + 4) ^ z)));
    };
    Frag<kExact> w[4], b[2];
    float sa[TM];
    token(0, b[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = wrow + 32 * (j >> 1) + 4 * (j & 1), z = 2 * ((n >> 3) & 3) + ((n >> 1) & 1);
      w[j].set(*(const u4 *)(ws + n * 128 + 16 * (q ^ z)), *(const u4 *)(ws + n * 128 + 16 * ((q + 4) ^ z)));
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) sa[m] = ss[tok + 16 * m] * f;
    f4 p[2][4];
#pragma unroll
    for (int m = 0; m <= TM; ++m) {
      if (m + 1 < TM) token(m + 1, b[(m + 1) & 1]);
      if (m < TM) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[m & 1][j] = block_sum(w[j], b[m & 1]);
      }
      if (m > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[m - 1][j][i] = __builtin_fmaf(p[(m - 1) & 1][j][i], sa[m - 1], acc[m - 1][j][i]);
      }
      // reads for m + 1, then a product of m and four sums of m - 1 in turn
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x8, kExact ? 4 : 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  __syncthreads();   // the weight scales; nothing else is in flight yet
  for (int g = 0; g < kStages - 1 && g < steps; ++g) issue(g);
  for (int g = 0; g < steps; ++g) {
    // step g's copies have landed (later ones stay in flight), for every wave; and
    // every wave is done with step g - 1, whose stage the next copies fill
    if (kStages > 2 && g + kStages - 2 < steps)
      wait_vm<(kStages - 2) * (CX + CW + 1)>();
    else
      wait_vm<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (g + kStages - 1 < steps) issue(g + kStages - 1);
    compute(g);
  }
  // ---- the other blocks' sums, through LDS
  if constexpr (KS > 1) {
    static_assert((KS - 1) * BM * BN * 4 <= kStages * L::kStageBytes, "sums fit the stages");
    f4 *sums = (f4 *)smem;
    __syncthreads();   // every wave is done with the stages
    if (ks > 0) {
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[(((ks - 1) * L::kWaves + wave) * TM * 4 + 4 * m + j) * 64 + lane] = acc[m][j];
    }
    __syncthreads();
    if (ks > 0) return;
#pragma unroll
    for (int o = 0; o < KS - 1; ++o)
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] += sums[((o * L::kWaves + wave) * TM * 4 + 4 * m + j) * 64 + lane];
  }
  // ---- results: token tok + 16 m, weight rows 64 wn + 32 h + 8 q + [0, 8)
  const bool rows16 = a.N % 8 == 0 && ((uintptr_t)a.out & 15) == 0;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int64_t t = t0 + tok + 16 * m;
    if (t >= a.T) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + wn * 64 + 32 * h + 8 * q;
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = acc[m][2 * h][i];
        y[4 + i] = acc[m][2 * h + 1][i];
      }
      store<8>(a, t, n, y, rows16 && n + 8 <= a.N);
    }
  }
}

template <bool kExact, int WM, int WN, int TM, int STAGES, int KS = 1>
hipError_t run_tiles(const LinearArgs &a, hipStream_t s) {
  using L = Tile<WM, WN, TM, STAGES, KS>;
  const int64_t all = ((a.T + L::BM - 1) / L::BM) * ((a.N + L::BN - 1) / L::BN);
  if (all > kMostGroups) return hipErrorInvalidConfiguration;
  raise_lds_limit((const void *)linear_tiles_kernel<kExact, WM, WN, TM, STAGES, KS>);
  linear_tiles_kernel<kExact, WM, WN, TM, STAGES, KS>
      <<<dim3((unsigned)((all + 7) / 8 * 8)), dim3(64 * L::kWaves * KS), L::lds(a.G), s>>>(a);
  return hipGetLastError();
}

template <bool kExact, int NT, int MT, int U, bool kFused>
hipError_t run_stream(const LinearArgs &a, hipStream_t s) {
  const int64_t wgs = (int64_t)((a.N + 16 * NT - 1) / (16 * NT)) * ((a.T + 16 * MT - 1) / (16 * MT));
  if (wgs > kMostGroups) return hipErrorInvalidConfiguration;
  const size_t lds = kFused ? a.T * (a.G * (size_t)128 + 16 + a.G * 4) : 0;
  linear_stream_kernel<kExact, NT, MT, U, kFused><<<dim3((unsigned)wgs), dim3(64 * kStreamWaves), lds, s>>>(a);
  return hipGetLastError();
}

// Which way, by how many workgroups of each form there would be (us of a whole call
// from Python, K = 2048 unless said; one launch from the host takes 2.4, quantizing
// beforehand 2 to 3 more).
template <bool kExact>
hipError_t run_linear(const LinearArgs &a, hipStream_t s) {
  // few tokens: every workgroup quantizes what it needs (1 x 5120: 4.9, quantized
  // beforehand 7.2; 8 x 2048: 5.9 and 6.9), up to 128 blocks (16 x 5120, 256 of them:
  // 10.6 and 8.1)
  if (a.T <= 16 && a.T * a.G <= 128) return run_stream<kExact, 1, 1, 1, true>(a, s);
  const int64_t quant = (a.T * a.G * 16 + 255) / 256;
  linear_quant_kernel<<<dim3((unsigned)(quant < kQuantGroups ? quant : kQuantGroups)), dim3(256), 0, s>>>(a);
  auto cover = [&](int bm, int bn) { return ((a.T + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  // streamed: the largest part of the result that still leaves 150 workgroups (64 x
  // 5120: 11.3 with parts of 64 x 32, 13.1 of 16 x 32, 14.3 of 16 x 16; 32 x 2048, K 4096:
  // 8.6 of 16 x 16, 10.2 of 16 x 32), for up to 64 tokens and up to 128 parts of 64 x 32
  // (128 x 2048: 9.0, tiles 10.5; 256 x 2048: 11.7, tiles 10.9)
  if (a.T <= 64 || cover(64, 32) <= 128) {
    if (a.T > 32 && cover(64, 32) >= 150) return run_stream<kExact, 2, 4, 2, false>(a, s);
    if (a.T > 16 && cover(32, 32) >= 150) return run_stream<kExact, 2, 2, 2, false>(a, s);
    if (cover(16, 32) >= 150) return run_stream<kExact, 2, 1, 2, false>(a, s);
    return run_stream<kExact, 1, 1, 2, false>(a, s);
  }
  // 256 x 256, a workgroup a CU: two rounds of them at least (16384 x 5120: 196, in
  // tiles of 128 x 128 218; 8192 x 5120, 2.5 rounds: 107 and 109; 4096 x 5120, 1.25: 71
  // and 59).  Its registers do not hold the FP16 operands.
  if constexpr (!kExact) {
    if (cover(256, 256) >= 512) return run_tiles<false, 2, 4, 8, 2>(a, s);
  }
  // 128 x 128 and 64 x 128, two a CU (1024 x 5120, 320 and 640 of them: 24.7 and 27.1;
  // 2048 x 2048, 256 and 512: 22.1 and 21.3)
  if (cover(128, 128) >= 320) return run_tiles<kExact, 2, 2, 4, 2>(a, s);
  if (cover(64, 128) >= 512) return run_tiles<kExact, 2, 2, 2, 3>(a, s);
  // 64 x 64: two a CU where there are more than CUs (256 x 5120, 320 of them: 13.7), else
  // one, whose 16 waves take four blocks of K at a time (16.8; 128 x 5120, 160: 10.6,
  // two a CU 11.9; 512 x 2048, K 4096: 16.6 and 20.4)
  if (cover(64, 64) > 256) return run_tiles<kExact, 4, 1, 1, 4>(a, s);
  return run_tiles<kExact, 4, 1, 1, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
  return a.out_bf16 ? run_linear<false>(a, s) : run_linear<true>(a, s);
}

}  // namespace mq
