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
//
// Bound by the cache's bytes, which are read once (of more than 16 heads per key head once
// for each 16): a call of 64 requests of 1 to 8192 tokens (32 query heads on 4 key heads
// of 128, BF16, 540 MB) takes 107 to 116 us by the lengths drawn, 4.8 to 5.0 TB/s, where a
// large copy moves 5.4; four of 100000 to 131072 in E4M3 (473 MB) 92 us, 5.1 TB/s.  The
// matrix units are busy 4 to 10% of that time and the vector units 20 to 40%, so the
// 16 columns that fewer shared heads leave empty cost nothing that would be missed.  A
// wave has two tiles' loads in flight (16 KB each at D = 128 in BF16) and a CU 8 waves, so
// memory is kept busy without LDS.  D above 128 has no tile ahead: those 64 requests take
// 170 us at 192 (810 MB) and 215 at 256 (1080 MB).
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
// Requests that the pieces' plan goes through; a workgroup takes whole units above it:
// every wave walks the lengths twice, which with 4097 requests of up to 600 tokens and one
// of 20000 costs more than the long one alone on its workgroups (2268 us, whole 763).  At
// 1025 of up to 8192 whole is no slower (1487 us, in pieces 1508), but one of 100000 among
// 1024 of up to 2000 is (1681, in pieces 595).
constexpr int kPlanBatch = 1024;
constexpr float kLn2 = 0.693147180559945309417f;

// Heads of a unit at most, and floats of a part of one: R maxima, R sums, O [R, D].
__host__ __device__ __forceinline__ int rows_of(const AttendArgs &a) { return a.Hq / a.Hk < 16 ? a.Hq / a.Hk : 16; }
__host__ __device__ __forceinline__ int64_t part_size(const AttendArgs &a) { return rows_of(a) * (int64_t)(a.D + 2); }

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
  static constexpr int LD = DT + 4;

  struct Shared {
    float m[kWaves][16], l[kWaves][16];
    __align__(16) float o[kWaves][16][LD];
  };
  // What a tile takes from memory.
  struct Frag {
    u4 k[2][KL];
    uint32_t v[8][VW];
    int seen;    // bit i: the lane's token i is there
  };

  // d of the 8 values that operand kk holds on lane group g
  static __device__ __forceinline__ int d_of(int kk, int g) {
    return FP8 ? 64 * (kk >> 1) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
  }
  // slot of token j0 + lane % 32, -1 where there is none
  static __device__ __forceinline__ int slot_of(const AttendArgs &a, const int32_t *table, int j0, int start, int end) {
    const int j = j0 + (threadIdx.x & 31);
    int slot = -1;
    if (j >= start && j < end) {
      const int p = table[j >> a.page_log2];
      if (p >= 0 && p < a.num_pages) slot = (p << a.page_log2) + (j & ((1 << a.page_log2) - 1));
    }
    return slot;
  }
  // Absent tokens read the first row of the cache, values behind D the row's first
  // ones (their products meet zeros of q, or land in rows of O that are not kept).
  static __device__ __forceinline__ void load(const AttendArgs &a, int kh, int slot, Frag &f) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    auto row = [&](int s) -> int64_t {
      s = s < 0 ? 0 : s;
      return ((((int64_t)(s >> a.page_log2) * a.Hk + kh) << a.page_log2) + (s & ((1 << a.page_log2) - 1))) * a.D;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = row(__shfl(slot, 16 * h + r, 64));
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int d0 = FP8 ? 64 * i + 16 * g : 32 * i + 8 * g, d = d0 < a.D ? d0 : 0;
        f.k[h][i] = FP8 ? *(const u4 *)((const uint8_t *)a.kc + at + d) : *(const u4 *)((const uint16_t *)a.kc + at + d);
      }
    }
    const int dv = VJ * r < a.D ? VJ * r : 0;
    f.seen = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = __shfl(slot, (i < 4 ? 4 * g + i : 12 + 4 * g + i), 64);
      f.seen |= s >= 0 ? 1 << i : 0;
      const int64_t at = row(s) + dv;
      const uint32_t *p = FP8 ? (const uint32_t *)((const uint8_t *)a.vc + at) : (const uint32_t *)((const uint16_t *)a.vc + at);
      if constexpr (VW == 1) {
        f.v[i][0] = p[0];
      } else if constexpr (VW == 2) {
        const u2 v = *(const u2 *)p;
        f.v[i][0] = v[0]; f.v[i][1] = v[1];
      } else {
#pragma unroll
        for (int w = 0; w < VW; w += 4) {
          const u4 v = *(const u4 *)(p + w);
          f.v[i][w] = v[0]; f.v[i][w + 1] = v[1]; f.v[i][w + 2] = v[2]; f.v[i][w + 3] = v[3];
        }
      }
    }
  }

  static __device__ __forceinline__ void compute(float c, const u4 *qf, Frag &f, Running<DT> &R) {
    // ---- scores
    f4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        u4 k;
        if constexpr (FP8) {
          const uint32_t w0 = f.k[h][kk >> 1][2 * (kk & 1)], w1 = f.k[h][kk >> 1][2 * (kk & 1) + 1];
          k = u4{e4m3x2_to_b2<false>(w0), e4m3x2_to_b2<true>(w0), e4m3x2_to_b2<false>(w1), e4m3x2_to_b2<true>(w1)};
        } else {
          k = f.k[h][kk];
        }
        s[h] = mfma_bf16(k, qf[kk], s[h]);
      }
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3] * c;
    if (!__all(f.seen == 255)) {
      // absent tokens: no score, and values of 0 whatever the cache holds there
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool seen = (f.seen >> i) & 1;
        p[i] = seen ? p[i] : -INFINITY;
#pragma unroll
        for (int w = 0; w < VW; ++w) f.v[i][w] = seen ? f.v[i][w] : 0u;
      }
    }
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, p[i]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if (__any(top > R.m)) {
      const float m = fmaxf(R.m, top), e = __builtin_amdgcn_exp2f(R.m - (m == -INFINITY ? 0.f : m));
      R.m = m;
      R.l *= e;
#pragma unroll
      for (int j = 0; j < VJ; ++j) R.o[j] *= e;
    }
    const float mm = R.m == -INFINITY ? 0.f : R.m;
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
        const uint32_t x = f.v[2 * i][w], y = f.v[2 * i + 1][w];
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

  // Tiles t0 to t1 of one unit: a request's tokens [start, end) (tile 0 holds token
  // `start`) and nh query heads from `head` on that share key head kh.  The
  // workgroup's waves take the tiles in turn; the joined state goes to `part` (max,
  // sum, O of 16 heads) if that is given, else the result to out and lse.
  static __device__ __forceinline__ void unit(const AttendArgs &a, Shared &sh, int b, int kh, int64_t head, int nh, int start,
                                              int end, int t0, int t1, float *part) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15,
              g = lane >> 4;
    u4 qf[KS];
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int d = d_of(kk, g);
      qf[kk] = u4{0u, 0u, 0u, 0u};
      if (d < a.D && r < nh) qf[kk] = *(const u4 *)(a.q + (head + r) * a.D + d);
    }
    Running<DT> R;
    R.m = -INFINITY;
    R.l = 0.f;
#pragma unroll
    for (int j = 0; j < VJ; ++j) R.o[j] = f4{0.f, 0.f, 0.f, 0.f};
    const int32_t *table = a.table + b * a.table_stride;
    const float c = a.score_scale;
    // one tile's loads are in flight while the one before is computed, and the page
    // numbers of the tile after that
    const int base = (start / kTile) * kTile, step = kWaves * kTile, stop = base + t1 * kTile;
    int j = base + (t0 + wave) * kTile;
    if constexpr (DT > 128) {
      // registers for one tile only
      for (; j < stop; j += step) {
        Frag f;
        load(a, kh, slot_of(a, table, j, start, end), f);
        compute(c, qf, f, R);
      }
    } else if (j < stop) {
      Frag f;
      int slot = slot_of(a, table, j, start, end);
      load(a, kh, slot, f);
      if (j + step < stop) slot = slot_of(a, table, j + step, start, end);
      for (; j + step < stop; j += step) {
        Frag n;
        load(a, kh, slot, n);
        if (j + 2 * step < stop) slot = slot_of(a, table, j + 2 * step, start, end);
        compute(c, qf, f, R);
        f = n;
      }
      compute(c, qf, f, R);
    }
    // ---- the waves' states joined
    R.l += __shfl_xor(R.l, 16, 64);
    R.l += __shfl_xor(R.l, 32, 64);
    __syncthreads();  // the unit before has been read out
    if (g == 0) {
      sh.m[wave][r] = R.m;
      sh.l[wave][r] = R.l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < VJ; j += 4)
        *(f4 *)&sh.o[wave][r][VJ * (4 * g + i) + j] = f4{R.o[j][i], R.o[j + 1][i], R.o[j + 2][i], R.o[j + 3][i]};
    __syncthreads();
    const int D = a.D, half = D / 2;
    for (int at = threadIdx.x; at < nh * half; at += 64 * kWaves) {
      const int n = at / half, d = 2 * (at - n * half);
      float m = sh.m[0][n];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sh.m[w][n]);
      const float mm = m == -INFINITY ? 0.f : m;
      float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(sh.m[w][n] - mm);
        l += f * sh.l[w][n];
        x += f * sh.o[w][n][d];
        y += f * sh.o[w][n][d + 1];
      }
      if (part) {
        const int R = rows_of(a);
        *(float2 *)(part + 2 * R + n * D + d) = float2{x, y};
        if (d == 0) {
          part[n] = m;
          part[R + n] = l;
        }
      } else {
        write_out(a, head + n, d, m, l, x, y);
      }
    }
  }

  // Two values of head hd's result from its maximum, sum and O.
  static __device__ __forceinline__ void write_out(const AttendArgs &a, int64_t hd, int d, float m, float l, float x, float y) {
    // l: 0 only where no token is there, else 1 at least, or NaN for a query of NaN.
    // (v_scale / l may be subnormal: the scale comes last)
    const float f = l == 0.f ? 0.f : 1.f / l;
    *(uint32_t *)(a.out + hd * a.D + d) = pack_bf16(x * f * a.v_scale, y * f * a.v_scale);
    if (a.lse && d == 0) a.lse[hd] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  }
};

// A request's tokens [start, end) and its tiles.
struct Span {
  int start, end, tiles;
};
__device__ __forceinline__ Span span_of(const AttendArgs &a, int length) {
  Span s;
  s.end = max(0, min(length, a.max_tokens));
  s.start = a.window ? max(0, s.end - a.window) : 0;
  s.tiles = s.end > s.start ? (s.end + kTile - 1) / kTile - s.start / kTile : 0;
  return s;
}
// Query heads of unit kt (of Hk ceil(group / 16)) of a request.
struct Heads {
  int kh, nh;
  int64_t head;
};
__device__ __forceinline__ Heads heads_of(const AttendArgs &a, int b, int kt) {
  const int G = a.Hq / a.Hk, ht = (G + 15) / 16;
  Heads h;
  h.kh = kt / ht;
  const int h0 = (kt - h.kh * ht) * 16;
  h.nh = min(16, G - h0);
  h.head = (int64_t)b * a.Hq + h.kh * G + h0;
  return h;
}

// ---- short requests: a workgroup takes a whole unit
template <int DT, bool FP8>
__global__ __launch_bounds__(64 * kWaves, 2) void attend_units_kernel(AttendArgs a) {
  using A = Attend<DT, FP8>;
  __shared__ typename A::Shared sh;
  const int units = a.Hk * ((a.Hq / a.Hk + 15) / 16);
  const int b = blockIdx.x / units, kt = blockIdx.x - b * units;
  const Heads h = heads_of(a, b, kt);
  const Span s = span_of(a, a.lengths[b]);
  A::unit(a, sh, b, h.kh, h.head, h.nh, s.start, s.end, 0, s.tiles, nullptr);
}

// ---- the others: a unit of n tiles goes to k = ceil(n / share) workgroups in equal
// pieces, share being what a workgroup gets if the tiles of all units are dealt
// evenly to `groups`.  The lengths are known on the device only: every wave of a
// workgroup x goes through them (64 a step) for the piece that is number x, and
// the pieces behind the last one, at most groups + units in all, have nothing to do.
__device__ __forceinline__ uint32_t wave_sum(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}

struct Plan {
  int groups, share_min;   // share: at least share_min tiles
  int *first;              // [B + 1]: number of a request's first piece; of all pieces
  float *parts;            // per piece, if its unit has others: R maxima, R sums, O [R, D]
};

template <int DT, bool FP8>
__global__ __launch_bounds__(64 * kWaves, 2) void attend_pieces_kernel(AttendArgs a, Plan plan) {
  using A = Attend<DT, FP8>;
  __shared__ typename A::Shared sh;
  const int lane = threadIdx.x & 63, units = a.Hk * ((a.Hq / a.Hk + 15) / 16);
  auto tiles_of = [&](int b) { return b < a.B ? span_of(a, a.lengths[b]).tiles : 0; };
  int64_t total = 0;
  for (int b = 0; b < a.B; b += 64) total += wave_sum((uint32_t)tiles_of(b + lane));  // 64 of at most 2^25
  total *= units;
  // (a share above a request's 2^25 tiles is as good as any)
  const int share = (int)min((int64_t)1 << 26, max((int64_t)plan.share_min, (total + plan.groups - 1) / plan.groups));
  int base = 0, found = -1, rel = 0, k = 1;
  for (int b = 0; b < a.B; b += 64) {
    const int n = tiles_of(b + lane), mine = b + lane < a.B ? max(1, (n + share - 1) / share) : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const int from = base + (upto - mine) * units;
    if (blockIdx.x == 0 && threadIdx.x < 64 && b + lane < a.B) plan.first[b + lane] = from;
    const uint64_t here = __ballot(from <= (int)blockIdx.x && (int)blockIdx.x < from + mine * units);
    if (here) {
      const int at = __builtin_ctzll(here);
      found = b + at;
      rel = blockIdx.x - __shfl(from, at, 64);
      k = __shfl(mine, at, 64);
    }
    base += __shfl(upto, 63, 64) * units;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) plan.first[a.B] = base;
  if (found < 0) return;
  const int b = __builtin_amdgcn_readfirstlane(found);
  k = __builtin_amdgcn_readfirstlane(k);
  rel = __builtin_amdgcn_readfirstlane(rel);
  const int kt = rel / k, i = rel - kt * k;
  const Span s = span_of(a, a.lengths[b]);
  const Heads h = heads_of(a, b, kt);
  float *part = plan.parts + blockIdx.x * part_size(a);
  A::unit(a, sh, b, h.kh, h.head, h.nh, s.start, s.end, (int)((int64_t)s.tiles * i / k), (int)((int64_t)s.tiles * (i + 1) / k),
          k == 1 ? nullptr : part);
}

// ---- the pieces of a unit joined: a query head to W of a workgroup's 4 waves, a pair
// of D (or more, in turn) to a lane, every W-th piece to a wave.  W = 4 where there are
// few units, which then have many pieces, else 1.  The first pieces' values are asked
// for together with the maxima and sums.
constexpr int kGroupsMost = 1024;   // of a plan, so no unit has more pieces
constexpr int kAhead = 8;

template <int W>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, Plan plan) {
  __shared__ float sx[4][64], sy[4][64], weight[4 / W][kGroupsMost];
  const int units = a.Hk * ((a.Hq / a.Hk + 15) / 16);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, D = a.D, mine = wave / W, first = wave % W;
  const int b = blockIdx.x / units, kt = blockIdx.x - b * units, r = blockIdx.y * (4 / W) + mine;
  const int f0 = plan.first[b], k = (plan.first[b + 1] - f0) / units;
  const Heads h = heads_of(a, b, kt);
  if (k <= 1) return;
  const bool live = r < h.nh;       // (of W = 1 some of the last workgroup's waves are not)
  if (W == 4 && !live) return;
  const int64_t size = part_size(a);
  const int R = rows_of(a);
  const float *part = plan.parts + (f0 + kt * k) * size;
  auto values = [&](int w, int d) { return *(const float2 *)(part + w * size + 2 * R + r * D + d); };
  float2 ahead[kAhead];
  float m = -INFINITY, l = 0.f;
  if (live) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      ahead[i] = float2{0.f, 0.f};
      if (first + W * i < k && 2 * lane < D) ahead[i] = values(first + W * i, 2 * lane);
    }
    for (int w = lane; w < k; w += 64) m = fmaxf(m, part[w * size + r]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d, 64));
    const float mm = m == -INFINITY ? 0.f : m;
    for (int w = lane; w < k; w += 64) {
      const float f = __builtin_amdgcn_exp2f(part[w * size + r] - mm);
      l += part[w * size + R + r] * f;
      if (first == 0) weight[mine][w] = f;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) l += __shfl_xor(l, d, 64);
  }
  __syncthreads();
  for (int d0 = 0; d0 < D; d0 += 128) {
    const int d = d0 + 2 * lane;
    float x = 0.f, y = 0.f;
    if (live && d < D) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int w = first + W * i;
        if (w < k) {
          const float2 o = d0 ? values(w, d) : ahead[i];
          x += weight[mine][w] * o.x;
          y += weight[mine][w] * o.y;
        }
      }
#pragma unroll 4
      for (int w = first + W * kAhead; w < k; w += W) {
        const float2 o = values(w, d);
        x += weight[mine][w] * o.x;
        y += weight[mine][w] * o.y;
      }
    }
    if constexpr (W == 4) {
      __syncthreads();
      sx[wave][lane] = x;
      sy[wave][lane] = y;
      __syncthreads();
      x = (sx[0][lane] + sx[1][lane]) + (sx[2][lane] + sx[3][lane]);
      y = (sy[0][lane] + sy[1][lane]) + (sy[2][lane] + sy[3][lane]);
    }
    if (first == 0 && live && d < D) Attend<64, false>::write_out(a, h.head + r, d, m, l, x, y);
  }
}

// Workgroups that the tiles are dealt to: two on each CU, and all their pieces at
// once, where units are few; with more units, whose lengths may differ by much,
// smaller pieces so that the last ones end together (512 - units against 1024 -
// units groups: 16 units of 3100 to 4096 tiles 98 and 110 us; 192 units of 1 to 256
// tiles 96 and 89 us).  At least 512 for many units, which need few pieces.
int groups_of(int64_t units) {
  if (units <= 64) return 512 - (int)units;
  return units < 512 ? kGroupsMost - (int)units : 512;
}
// Tiles of a piece at least: with few units one per wave (4 units of 32 tiles:
// 11.4 us, 12.8 with two per wave), with many as much as keeps a unit whole that the
// other units' workgroups hide (396 units of 32 tiles: 24 us whole, 31 in two).  Whole
// calls by this rule and with 4 tiles at least, key heads 4: 32 requests of 500 tokens
// 11.8 and 15.3 us, 64 of 500 17.3 and 27.2, 32 of 1000 22.7 and 27.3, 99 of 1000 42.1 and
// 54.6; 16 of 500 13.1 and 12.1, 48 of 2000 53.7 and 49.4.
int share_min_of(int64_t units) { return units / 8 < 4 ? 4 : units / 8 > 128 ? 128 : (int)(units / 8); }

}  // namespace

// [B + 1] numbers of pieces, then the parts.
static size_t first_bytes(int64_t B) { return ((size_t)(B + 1) * 4 + 255) / 256 * 256; }

size_t attend_workspace_need(int64_t B, int Hq, int Hk, int D) {
  if (B > kPlanBatch) return 256;   // no pieces
  AttendArgs a{};
  a.Hq = Hq; a.Hk = Hk; a.D = D;
  const int64_t units = B * Hk * ((Hq / Hk + 15) / 16);
  return first_bytes(B) + ((size_t)(groups_of(units) + units) * part_size(a) * 4 + 255) / 256 * 256;
}

// What a call of any number of requests up to B needs: groups_of(units) + units and so
// the need grow with B up to kPlanBatch.
size_t attend_workspace(int64_t B, int Hq, int Hk, int D) {
  return attend_workspace_need(B < kPlanBatch ? B : kPlanBatch, Hq, Hk, D);
}

template <int DT, bool FP8>
static hipError_t run_attend(const AttendArgs &a, hipStream_t s) {
  const int G = a.Hq / a.Hk;
  const unsigned units = (unsigned)a.B * a.Hk * ((G + 15) / 16);
  const int share_min = share_min_of(units), groups = groups_of(units);
  // tiles of a unit at most; a window may end inside of one at either end
  const int tokens = a.window && a.window < a.max_tokens ? a.window + kTile - 1 : a.max_tokens, most = (tokens + kTile - 1) / kTile;
  if (most <= share_min || a.B > kPlanBatch) {
    attend_units_kernel<DT, FP8><<<dim3(units), dim3(64 * kWaves), 0, s>>>(a);
    return hipGetLastError();
  }
  const Plan plan = {groups, share_min, (int *)a.ws, (float *)((char *)a.ws + first_bytes(a.B))};
  attend_pieces_kernel<DT, FP8><<<dim3(groups + units), dim3(64 * kWaves), 0, s>>>(a, plan);
  const unsigned heads = G < 16 ? G : 16;
  if (units <= 64)
    attend_join_kernel<4><<<dim3(units, heads), dim3(256), 0, s>>>(a, plan);
  else
    attend_join_kernel<1><<<dim3(units, (heads + 3) / 4), dim3(256), 0, s>>>(a, plan);
  return hipGetLastError();
}

hipError_t launch_attend(const AttendArgs &a, int fp8, hipStream_t s) {
  if (a.D <= 64) return fp8 ? run_attend<64, true>(a, s) : run_attend<64, false>(a, s);
  if (a.D <= 128) return fp8 ? run_attend<128, true>(a, s) : run_attend<128, false>(a, s);
  return fp8 ? run_attend<256, true>(a, s) : run_attend<256, false>(a, s);
}

}  // namespace mq
