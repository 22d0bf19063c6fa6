// Attention of one new token of each request over a paged cache.
//
// One pass over the keys and values with the running maximum and sum of the
// softmax.  The query heads that share a key head are the columns of the matrix
// instructions (16 of them; a group of more takes several passes), 32 tokens
// the rows:
//   S^T [32 tokens, 16 heads] = K Q^T       two 16x16x32 products per 32 of D;
//   O^T [D, 16 heads] += V^T P^T            one 16x16x32 product per 16 of D.
// Nothing but the page numbers crosses lanes: lane l = 16 g + r loads the 16 bytes
// of K rows r and 16 + r that its operand holds, its results are head r's scores
// of tokens 4 g + [0, 4) and 16 + the same, and with these eight tokens as the
// lane's part of the sum over tokens, P is the second product's operand as it
// stands.  V's operand holds, for one of D, the lane's eight tokens: the lane loads
// D / 16 consecutive values of each of its eight tokens (the 16 lanes of a group
// the whole row) and transposes them in registers, one byte permute per pair.
//
// The probabilities go into the second product as the sum of two BF16 values,
// p = hi + lo (2^-17 of p is lost): with one BF16 value their rounding (2^-9)
// would be as large an error as the output's own rounding.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"

namespace mq {
namespace {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4 mfma_bf16(u4 a, u4 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// Two E4M3 bytes -> two BF16 values (exact: scale 2^0).
template <bool kHiWord>
__device__ __forceinline__ uint32_t e4m3x2_to_b2(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, kHiWord));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  b2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

constexpr int kTile = 32;    // tokens of one step of a wave
constexpr int kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// One wave's running state: maximum (in base-2 exponents) and sum for head r
// (the sum over this lane's tokens), O^T of head r: register i of o[j] is
// d = (DT / 16) (4 g + i) + j.
template <int DT>
struct Running {
  float m, l;
  f4 o[DT / 16];
};

template <int DT, bool FP8>
struct Attend {
  static constexpr int VJ = DT / 16;                    // values of a token's row per lane
  static constexpr int VW = FP8 ? VJ / 4 : VJ / 2;      // and their 32-bit words
  static constexpr int KS = DT / 32;                    // products of 32 over D
  static constexpr int KL = FP8 ? DT / 64 : DT / 32;    // 16-byte loads of a key row per lane

  // d of the 8 values that operand kk holds on lane group g
  static __device__ __forceinline__ int d_of(int kk, int g) {
    return FP8 ? 64 * (kk >> 1) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
  }

  // One tile of 32 tokens from token j0 on.
  static __device__ __forceinline__ void tile(const AttendArgs &a, const u4 *qf, int kh, const int32_t *table, int j0,
                                              int start, int end, Running<DT> &R) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int ps = 1 << a.page_log2, D = a.D;
    // slot of token j0 + lane % 32, -1 where there is none
    int slot = -1;
    {
      const int j = j0 + (lane & 31);
      if (j >= start && j < end) {
        const int p = table[j >> a.page_log2];
        if (p >= 0 && p < a.num_pages) slot = (p << a.page_log2) + (j & (ps - 1));
      }
    }
    const bool whole = __all(slot >= 0);
    auto row = [&](int s) -> int64_t {
      s = s < 0 ? 0 : s;  // an absent token reads the first row and is masked
      return ((((int64_t)(s >> a.page_log2) * a.Hk + kh) << a.page_log2) + (s & (ps - 1))) * D;
    };
    u4 kw[2][KL];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = row(__shfl(slot, 16 * h + r, 64));
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int d = FP8 ? 64 * i + 16 * g : 32 * i + 8 * g;
        kw[h][i] = u4{0u, 0u, 0u, 0u};
        if (d < D) kw[h][i] = FP8 ? *(const u4 *)((const uint8_t *)a.kc + at + d)
                                  : *(const u4 *)((const uint16_t *)a.kc + at + d);
      }
    }
    uint32_t vw[8][VW];
    bool seen[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = __shfl(slot, (i < 4 ? 4 * g + i : 12 + 4 * g + i), 64);
      seen[i] = s >= 0;
      const int64_t at = row(s) + VJ * r;
#pragma unroll
      for (int w = 0; w < VW; ++w) vw[i][w] = 0u;
      if (VJ * r < D && seen[i]) {  // absent values are 0 whatever the cache holds there
        const uint32_t *p = FP8 ? (const uint32_t *)((const uint8_t *)a.vc + at) : (const uint32_t *)((const uint16_t *)a.vc + at);
        if constexpr (VW == 1) {
          vw[i][0] = p[0];
        } else if constexpr (VW == 2) {
          const u2 v = *(const u2 *)p;
          vw[i][0] = v[0]; vw[i][1] = v[1];
        } else {
#pragma unroll
          for (int w = 0; w < VW; w += 4) {
            const u4 v = *(const u4 *)(p + w);
            vw[i][w] = v[0]; vw[i][w + 1] = v[1]; vw[i][w + 2] = v[2]; vw[i][w + 3] = v[3];
          }
        }
      }
    }
    // ---- scores
    f4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        u4 k;
        if constexpr (FP8) {
          const uint32_t w0 = kw[h][kk >> 1][2 * (kk & 1)], w1 = kw[h][kk >> 1][2 * (kk & 1) + 1];
          k = u4{e4m3x2_to_b2<false>(w0), e4m3x2_to_b2<true>(w0), e4m3x2_to_b2<false>(w1), e4m3x2_to_b2<true>(w1)};
        } else {
          k = kw[h][kk];
        }
        s[h] = mfma_bf16(k, qf[kk], s[h]);
      }
    }
    const float c = a.score_scale * kLog2e;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3] * c;
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = seen[i] ? p[i] : -INFINITY;
    }
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, p[i]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float m = fmaxf(R.m, top), mm = m == -INFINITY ? 0.f : m;
    const float f = __builtin_amdgcn_exp2f(R.m - mm);
    R.m = m;
    if (__any(f != 1.f)) {
      R.l *= f;
#pragma unroll
      for (int j = 0; j < VJ; ++j) R.o[j] *= f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(p[i] - mm);
      R.l += p[i];
    }
    u4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
      lo[i] = pack_bf16(p[2 * i] - bf16_to_f32(hi[i] & 0xFFFFu), p[2 * i + 1] - bf16_to_f32(hi[i] >> 16));
    }
    // ---- values: operand j holds the eight tokens' value VJ r + j
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      u4 v[FP8 ? 4 : 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = vw[2 * i][w], y = vw[2 * i + 1][w];
        if constexpr (FP8) {
          const uint32_t e = __builtin_amdgcn_perm(y, x, 0x05010400u), o = __builtin_amdgcn_perm(y, x, 0x07030602u);
          v[0][i] = e4m3x2_to_b2<false>(e); v[1][i] = e4m3x2_to_b2<true>(e);
          v[2][i] = e4m3x2_to_b2<false>(o); v[3][i] = e4m3x2_to_b2<true>(o);
        } else {
          v[0][i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          v[1][i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
      }
      constexpr int N = FP8 ? 4 : 2;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        R.o[N * w + n] = mfma_bf16(v[n], hi, R.o[N * w + n]);
        R.o[N * w + n] = mfma_bf16(v[n], lo, R.o[N * w + n]);
      }
    }
  }
};

template <int DT, bool FP8>
__global__ __launch_bounds__(64 * kWaves) void attend_kernel(AttendArgs a) {
  using A = Attend<DT, FP8>;
  constexpr int LD = DT + 4;
  __shared__ float sm[kWaves][16], sl[kWaves][16];
  __shared__ __align__(16) float so[kWaves][16][LD];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int G = a.Hq / a.Hk, ht = (G + 15) / 16;
  const int unit = blockIdx.x, b = unit / (a.Hk * ht), kt = unit - b * (a.Hk * ht), kh = kt / ht;
  const int h0 = (kt - kh * ht) * 16, nh = min(16, G - h0);   // heads of the group that this workgroup takes
  const int64_t head = (int64_t)b * a.Hq + kh * G + h0;
  const int end = max(0, min(a.lengths[b], a.max_tokens)), start = a.window ? max(0, end - a.window) : 0;
  u4 qf[A::KS];
#pragma unroll
  for (int kk = 0; kk < A::KS; ++kk) {
    const int d = A::d_of(kk, g);
    qf[kk] = u4{0u, 0u, 0u, 0u};
    if (d < a.D && r < nh) qf[kk] = *(const u4 *)(a.q + (head + r) * a.D + d);
  }
  Running<DT> R;
  R.m = -INFINITY;
  R.l = 0.f;
#pragma unroll
  for (int j = 0; j < A::VJ; ++j) R.o[j] = f4{0.f, 0.f, 0.f, 0.f};
  const int32_t *table = a.table + b * a.table_stride;
  for (int j0 = (start / kTile + wave) * kTile; j0 < end; j0 += kWaves * kTile) A::tile(a, qf, kh, table, j0, start, end, R);
  // ---- the waves' states joined
  R.l += __shfl_xor(R.l, 16, 64);
  R.l += __shfl_xor(R.l, 32, 64);
  if (g == 0) {
    sm[wave][r] = R.m;
    sl[wave][r] = R.l;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < A::VJ; j += 4)
      *(f4 *)&so[wave][r][A::VJ * (4 * g + i) + j] = f4{R.o[j][i], R.o[j + 1][i], R.o[j + 2][i], R.o[j + 3][i]};
  __syncthreads();
  const int D = a.D;
  for (int at = threadIdx.x; at < nh * (D / 2); at += 64 * kWaves) {
    const int n = at / (D / 2), d = 2 * (at - n * (D / 2));
    float m = sm[0][n];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sm[w][n]);
    const float mm = m == -INFINITY ? 0.f : m;
    float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][n] - mm);
      l += f * sl[w][n];
      x += f * so[w][n][d];
      y += f * so[w][n][d + 1];
    }
    const float f = l > 0.f ? a.v_scale / l : 0.f;
    *(uint32_t *)(a.out + (head + n) * D + d) = (uint32_t)f32_to_bf16_rne(x * f) | ((uint32_t)f32_to_bf16_rne(y * f) << 16);
    if (a.lse && d == 0) a.lse[head + n] = l > 0.f ? m * kLn2 + logf(l) : -INFINITY;
  }
}

}  // namespace

size_t attend_workspace(int64_t, int, int, int) { return 256; }

hipError_t launch_attend(const AttendArgs &a, int fp8, hipStream_t s) {
  const int ht = (a.Hq / a.Hk + 15) / 16;
  const dim3 grid((unsigned)a.B * a.Hk * ht), block(64 * kWaves);
  if (a.D <= 64) {
    if (fp8) attend_kernel<64, true><<<grid, block, 0, s>>>(a);
    else attend_kernel<64, false><<<grid, block, 0, s>>>(a);
  } else if (a.D <= 128) {
    if (fp8) attend_kernel<128, true><<<grid, block, 0, s>>>(a);
    else attend_kernel<128, false><<<grid, block, 0, s>>>(a);
  } else {
    if (fp8) attend_kernel<256, true><<<grid, block, 0, s>>>(a);
    else attend_kernel<256, false><<<grid, block, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mq
