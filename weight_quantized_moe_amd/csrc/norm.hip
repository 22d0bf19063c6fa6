// Norms before and after a block, fused with the block's gate, the residual
// scale and the residual add (mq_norm in the C header states the formulas):
//   z  = x  or  x rsqrt(mean x^2 + eps) (offset + w_post)
//   r' = round(residual + scale gate z)
//   n  = bf16(r' rsqrt(mean r'^2 + eps) (offset + w_pre))
// A row is held in the registers of one wave or of one workgroup in 32 bits
// between the steps: every input is read once, every output written once, and
// the kernel is bound by those bytes.  Lane c of NT holds values
// 8 (c + NT j) + [0, 8), j < R, so loads and stores are 16 bytes per lane and
// consecutive over the lanes.  Rows whose length is no multiple of 8 start at
// odd addresses: the same accesses, which the hardware takes at any alignment of
// the element (see Ends for the row's last lane).
//
// Measured: 16384 rows of 2048, both norms, BF16: 50 us (5.4 TB/s, a plain copy
// of that size 5.5); 4096 rows of 8192 with a 32-bit residual 63-67 us (5.0-5.3
// TB/s); 16384 odd rows of 1023 with a 32-bit residual and a full gate 52 us
// (4.5), of 1024 45 us.  With the row in LDS and one value a lane: 158 and 234
// us for the first two.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "internal.h"
#include "route.h"

namespace mq {

typedef u4 u4_a2 __attribute__((aligned(2)));
typedef u4 u4_a4 __attribute__((aligned(4)));
typedef f4 f4_a4 __attribute__((aligned(4)));

struct Row8 {
  float v[8];
};
// 8 values as they lie in memory: 8 BF16 values in a, or 8 floats in a and b.
// Loads keep this form until the values are used, so that none of them is
// waited for at the branch that picked its type.
struct Raw8 {
  u4 a, b;
};

__device__ __forceinline__ Row8 widen(u4 u) {
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_to_f32(u[i] & 0xFFFFu);
    r.v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ Row8 widen(const Raw8 &w, int bf16) {
  if (bf16) return widen(w.a);
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[i] = __builtin_bit_cast(float, (uint32_t)w.a[i]);
    r.v[4 + i] = __builtin_bit_cast(float, (uint32_t)w.b[i]);
  }
  return r;
}

// How a lane reads the 8 values of a row of n from index `at` on.
//   kEven   n is a multiple of 8;
//   kShift  n >= 8: a lane that reaches past the row's end reads the row's last
//           8 values instead and shifts them down when they are used (zeros
//           follow), so no load is waited for one by one;
//   kSmall  n < 8: single values.
enum Ends { kEven, kShift, kSmall };

template <Ends kEnds>
__device__ __forceinline__ Raw8 load8(const void *p, int bf16, int64_t row, int at, int n) {
  Raw8 w = {u4{0u, 0u, 0u, 0u}, u4{0u, 0u, 0u, 0u}};
  if (kEnds == kEven && at >= n) return w;
  if (kEnds == kShift) at = min(at, n - 8);
  if (bf16) {
    const uint16_t *q = (const uint16_t *)p + row + at;
    if (kEnds != kSmall) {
      w.a = *(const u4_a2 *)q;
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (at + i < n) w.a[i >> 1] |= (uint32_t)q[i] << (16 * (i & 1));
    }
  } else {
    const uint32_t *q = (const uint32_t *)p + row + at;
    if (kEnds != kSmall) {
      w.a = *(const u4_a4 *)q;
      w.b = *(const u4_a4 *)(q + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (at + i < n) (i < 4 ? w.a : w.b)[i & 3] = q[i];
    }
  }
  return w;
}
// The values of load8: for kShift, `by` = at - min(at, n - 8) of them lie before
// the lane's first one.
template <Ends kEnds>
__device__ __forceinline__ Row8 values(const Raw8 &w, int bf16, int by) {
  Row8 r = widen(w, bf16);
  if (kEnds == kShift && __any(by > 0)) {
#pragma unroll
    for (int b = 4; b >= 1; b >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = (by & b) ? (i + b < 8 ? r.v[i + b] : 0.f) : r.v[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = by >= 8 ? 0.f : r.v[i];
  }
  return r;
}
template <Ends kEnds>
__device__ __forceinline__ void store_bf16x8(uint16_t *p, int at, int n, u4 u) {
  if (at + 8 <= n) {
    *(u4_a2 *)(p + at) = u;
  } else if (kEnds != kEven) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (at + i < n) p[at + i] = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
  }
}
template <Ends kEnds>
__device__ __forceinline__ void store_f32x8(float *p, int at, int n, const Row8 &r) {
  if (at + 8 <= n) {
    *(f4_a4 *)(p + at) = f4{r.v[0], r.v[1], r.v[2], r.v[3]};
    *(f4_a4 *)(p + at + 4) = f4{r.v[4], r.v[5], r.v[6], r.v[7]};
  } else if (kEnds != kEven) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (at + i < n) p[at + i] = r.v[i];
  }
}
__device__ __forceinline__ u4 narrow(const Row8 &r) {
  u4 u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = (uint32_t)f32_to_bf16_rne(r.v[2 * i]) | ((uint32_t)f32_to_bf16_rne(r.v[2 * i + 1]) << 16);
  return u;
}

// 1 / sqrt(mean + eps) of a row whose lanes hold partial sums ss of squares:
// added over the row's lanes by a fixed tree, over several waves in wave order
// (red: 16 floats of LDS).
template <int kLanes>
__device__ __forceinline__ float inv_rms(float ss, int H, float eps, float *red) {
  if (kLanes == 16 || kLanes == 32) {
    ss = sum16(ss);
    if (kLanes == 32) ss += __shfl_xor(ss, 16, 64);
  } else {
    ss = sum64f(ss);
  }
  if (kLanes == 0) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = red[0];
    for (int w = 1; w < waves; ++w) ss += red[w];
  }
  return 1.f / sqrtf(ss / H + eps);
}

// kLanes: lanes of a row, 256 / kLanes rows per workgroup; 0: a workgroup a row.
template <int R, int kLanes, bool kResBf16, Ends kEnds>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void norm_kernel(NormArgs a, int64_t T) {
  constexpr bool kEarly = R <= 2;  // 4 x 40 values a lane would not fit its registers
  __shared__ float red[2][16];
  const int H = a.H, NT = kLanes ? kLanes : blockDim.x;
  const int c = kLanes ? threadIdx.x % NT : threadIdx.x;
  // rows past the last one repeat it and store nothing: every lane of a wave stays for the sums
  const int64_t row = kLanes ? (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT : blockIdx.x;
  const bool live = row < T;
  const int64_t t = live ? row : T - 1;
  const int64_t o = t * H;
  const bool vec_gate = a.gate_kind == MQ_GATE_CHANNEL || a.gate_kind == MQ_GATE_FULL;
  const int64_t go = a.gate_kind == MQ_GATE_FULL ? o : 0;
  Raw8 x[R] = {}, res[R] = {}, g[R], w_post[R], w_pre[R];
  if (a.x) {
#pragma unroll
    for (int j = 0; j < R; ++j) x[j] = load8<kEnds>(a.x, 1, o, 8 * (c + NT * j), H);
  }
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < R; ++j) res[j] = load8<kEnds>(a.residual, kResBf16, o, 8 * (c + NT * j), H);
  }
  // everything the row needs is on its way before the first sum is taken
  auto load_gate = [&](int j) { g[j] = load8<kEnds>(a.gate, a.gate_bf16, go, 8 * (c + NT * j), H); };
  auto load_post = [&](int j) { w_post[j] = load8<kEnds>(a.post_w, a.w_bf16, 0, 8 * (c + NT * j), H); };
  auto load_pre = [&](int j) { w_pre[j] = load8<kEnds>(a.pre_w, a.w_bf16, 0, 8 * (c + NT * j), H); };
  if (kEarly) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (vec_gate) load_gate(j);
      if (a.post_w) load_post(j);
      if (a.pre_w) load_pre(j);
    }
  }
  float scale = a.x ? a.scale : -0.f;  // no x: r + -0 is r, a zero's sign with it
  if (a.gate_kind == MQ_GATE_TOKEN)
    scale *= a.gate_bf16 ? bf16_to_f32(((const uint16_t *)a.gate)[t]) : ((const float *)a.gate)[t];
  Row8 v[R];
  int by[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    by[j] = max(8 * (c + NT * j) - (H - 8), 0);
    v[j] = values<kEnds>(x[j], 1, by[j]);
  }
  float ss = 0.f;
  if (a.post_w) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += v[j].v[i] * v[j].v[i];
    const float inv = inv_rms<kLanes>(ss, H, a.eps, red[0]);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (!kEarly) load_post(j);
      const Row8 w = values<kEnds>(w_post[j], a.w_bf16, by[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j].v[i] *= inv * (a.offset + w.v[i]);
    }
  }
  if (vec_gate) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (!kEarly) load_gate(j);
      const Row8 w = values<kEnds>(g[j], a.gate_bf16, by[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j].v[i] *= w.v[i];
    }
  }
  ss = 0.f;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const Row8 r = values<kEnds>(res[j], kResBf16, by[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j].v[i] = r.v[i] + scale * v[j].v[i];
    if (kResBf16) {
      const u4 u = narrow(v[j]);
      if (a.residual_out && live) store_bf16x8<kEnds>((uint16_t *)a.residual_out + o, 8 * (c + NT * j), H, u);
      v[j] = widen(u);
    } else if (a.residual_out && live) {
      store_f32x8<kEnds>((float *)a.residual_out + o, 8 * (c + NT * j), H, v[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += v[j].v[i] * v[j].v[i];
  }
  if (!a.norm_out) return;
  const float inv = inv_rms<kLanes>(ss, H, a.eps, red[1]);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (!kEarly) load_pre(j);
    const Row8 w = values<kEnds>(w_pre[j], a.w_bf16, by[j]);
    Row8 n;
#pragma unroll
    for (int i = 0; i < 8; ++i) n.v[i] = v[j].v[i] * inv * (a.offset + w.v[i]);
    if (live) store_bf16x8<kEnds>(a.norm_out + o, 8 * (c + NT * j), H, narrow(n));
  }
}

template <int R, int kLanes>
static void norm_launch(const NormArgs &a, int64_t T, int threads, hipStream_t s) {
  void (*f)(NormArgs, int64_t);
  if (a.H % 8 == 0)
    f = a.r_bf16 ? norm_kernel<R, kLanes, true, kEven> : norm_kernel<R, kLanes, false, kEven>;
  else
    f = a.r_bf16 ? norm_kernel<R, kLanes, true, kShift> : norm_kernel<R, kLanes, false, kShift>;
  if (R == 1 && kLanes == 16 && a.H < 8)
    f = a.r_bf16 ? norm_kernel<1, 16, true, kSmall> : norm_kernel<1, 16, false, kSmall>;
  constexpr int kRows = kLanes ? 256 / (kLanes ? kLanes : 1) : 1;
  hipLaunchKernelGGL(f, dim3((unsigned)((T + kRows - 1) / kRows)), dim3(threads), 0, s, a, T);
}

// Few values a lane and many lanes a row: with 8 a lane everything a row needs is
// in flight at once (16384 rows of 2048: 51 us; 16 a lane 54, 32 a lane, one wave a
// row, 60).  Rows of up to 512 share a workgroup, of up to 256 a wave (50000 rows
// of 128: 25.7 -> 17.0 us).
hipError_t launch_norm(const NormArgs &all, int64_t rows, hipStream_t s) {
  // a grid holds fewer than 2^32 lanes, 2^21 rows at most 2^31
  constexpr int64_t kMostRows = 1 << 21;
  NormArgs a = all;
  for (; rows > kMostRows; rows -= kMostRows) {
    const hipError_t e = launch_norm(a, kMostRows, s);
    if (e != hipSuccess) return e;
    const int64_t n = kMostRows * a.H;
    auto after = [](const void *p, int64_t bytes) { return p ? (const char *)p + bytes : nullptr; };
    if (a.x) a.x += n;
    a.residual = after(a.residual, n * (a.r_bf16 ? 2 : 4));
    if (a.gate_kind != MQ_GATE_CHANNEL)
      a.gate = after(a.gate, (a.gate_kind == MQ_GATE_FULL ? n : kMostRows) * (a.gate_bf16 ? 2 : 4));
    a.residual_out = (void *)after(a.residual_out, n * (a.r_bf16 ? 2 : 4));
    if (a.norm_out) a.norm_out += n;
  }
  const int64_t T = rows;
  const int eights = (a.H + 7) / 8;
  if (eights <= 16)
    norm_launch<1, 16>(a, T, 256, s);
  else if (eights <= 32)
    norm_launch<1, 32>(a, T, 256, s);
  else if (eights <= 64)
    norm_launch<1, 64>(a, T, 256, s);
  else if (eights <= 1024)
    norm_launch<1, 0>(a, T, (eights + 63) / 64 * 64, s);
  else if (eights <= 2048)
    norm_launch<2, 0>(a, T, 1024, s);
  else
    norm_launch<4, 0>(a, T, 1024, s);
  return hipGetLastError();
}

}  // namespace mq
