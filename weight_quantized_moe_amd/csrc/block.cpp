// Host side of the operators in front of the expert layer: the dense E4M3
// product, the paged cache's append and the attention over it.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "internal.h"

using mq::fail;
using mq::kMaxTokens;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}
// Memory that a call reads or writes (p: NULL where it is not given).
struct Bytes {
  const void *p;
  size_t n;
};
bool meets(const Bytes &a, std::initializer_list<Bytes> others) {
  for (const Bytes &b : others)
    if (a.p && b.p && overlap(a.p, a.n, b.p, b.n)) return true;
  return false;
}
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct LinearWs {
  size_t codes, sa, total;
};
LinearWs linear_ws(int64_t T, int K) {
  const size_t G = (size_t)(K + 127) / 128;
  LinearWs w;
  w.codes = 0;
  w.sa = up256((size_t)T * G * 128);
  w.total = w.sa + up256((size_t)T * G * 4);
  return w;
}

mq_status check_linear(const mq_linear *l, const char *who) {
  if (!l) return fail(MQ_E_NULL, "%s: NULL descriptor", who);
  if (l->abi_version != MOE_QUANT_ABI_VERSION)
    return fail(MQ_E_ABI, "%s: descriptor abi_version %u, library %u", who, l->abi_version, MOE_QUANT_ABI_VERSION);
  if (l->n < 1 || l->n > (1 << 20)) return fail(MQ_E_SHAPE, "%s: n %d outside [1, 2^20]", who, l->n);
  if (l->k < 16 || l->k > 65536 || l->k % 16)
    return fail(MQ_E_SHAPE, "%s: k %d must be a multiple of 16 from 16 to 65536", who, l->k);
  if (l->out_dtype != MQ_F32 && l->out_dtype != MQ_BF16)
    return fail(MQ_E_DTYPE, "%s: unknown out dtype %d", who, l->out_dtype);
  if (!l->w || !l->scale) return fail(MQ_E_NULL, "%s: weight and scale must be non-NULL", who);
  if (!aligned(l->w, 16) || !aligned(l->scale, 4))
    return fail(MQ_E_ALIGN, "%s: weight 16-byte, scale 4-byte aligned", who);
  return MQ_OK;
}

mq_status check_tokens(int64_t n, const char *who) {
  if (n < 0 || n > kMaxTokens)
    return fail(MQ_E_SHAPE, "%s: num_tokens %lld outside [0, %lld]", who, (long long)n, (long long)kMaxTokens);
  return MQ_OK;
}

mq_status check_batch(int64_t n, const char *who) {
  if (n < 0 || n > mq::kMaxBatch)
    return fail(MQ_E_SHAPE, "%s: batch %lld outside [0, %lld]", who, (long long)n, (long long)mq::kMaxBatch);
  return MQ_OK;
}

mq_status check_cache(const mq_kv_cache *c, const char *who) {
  if (!c) return fail(MQ_E_NULL, "%s: NULL cache", who);
  if (c->abi_version != MOE_QUANT_ABI_VERSION)
    return fail(MQ_E_ABI, "%s: cache abi_version %u, library %u", who, c->abi_version, MOE_QUANT_ABI_VERSION);
  if (c->dtype != MQ_KV_BF16 && c->dtype != MQ_KV_FP8)
    return fail(MQ_E_DTYPE, "%s: unknown cache dtype %d", who, c->dtype);
  if (c->kv_heads < 1 || c->kv_heads > mq::kMaxHeads)
    return fail(MQ_E_SHAPE, "%s: kv_heads %d outside [1, %d]", who, c->kv_heads, mq::kMaxHeads);
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
    return fail(MQ_E_SHAPE, "%s: head_dim %d must be a multiple of 16 from 16 to 256", who, c->head_dim);
  if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(MQ_E_SHAPE, "%s: page_size %d must be a power of two from 1 to 1024", who, c->page_size);
  if (c->num_pages < 1 || c->num_pages > INT32_MAX / c->page_size)
    return fail(MQ_E_SHAPE, "%s: num_pages %lld must be positive, num_pages * page_size below 2^31", who,
                (long long)c->num_pages);
  for (float s : {c->k_scale, c->v_scale})
    if (!std::isfinite(s) || !(s > 0.f) || (c->dtype == MQ_KV_BF16 && s != 1.f))
      return fail(MQ_E_SHAPE, "%s: k_scale %g and v_scale %g must be finite and positive, 1 for a BF16 cache", who,
                  (double)c->k_scale, (double)c->v_scale);
  if (!c->k || !c->v) return fail(MQ_E_NULL, "%s: the cache's k and v must be non-NULL", who);
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(MQ_E_ALIGN, "%s: the cache's k and v must be 16-byte aligned", who);
  return MQ_OK;
}

size_t cache_bytes(const mq_kv_cache *c) {
  return (size_t)(c->num_pages * c->page_size) * c->kv_heads * c->head_dim * (c->dtype == MQ_KV_BF16 ? 2 : 1);
}

mq_status check_rotary(const mq_rotary *r, const mq_kv_cache *c, const char *who) {
  if (!r) return fail(MQ_E_NULL, "%s: NULL rotary", who);
  if (r->abi_version != MOE_QUANT_ABI_VERSION)
    return fail(MQ_E_ABI, "%s: rotary abi_version %u, library %u", who, r->abi_version, MOE_QUANT_ABI_VERSION);
  if (r->head_dim != c->head_dim)
    return fail(MQ_E_SHAPE, "%s: the rotary's head_dim is %d, the cache's %d", who, r->head_dim, c->head_dim);
  if (r->rot_dim < 0 || r->rot_dim > r->head_dim || r->rot_dim % 16)
    return fail(MQ_E_SHAPE, "%s: rot_dim %d must be a multiple of 16 up to head_dim %d", who, r->rot_dim, r->head_dim);
  if (r->rot_dim && r->max_positions < 1)
    return fail(MQ_E_SHAPE, "%s: max_positions %d must be positive", who, r->max_positions);
  if (!std::isfinite(r->eps) || !(r->eps >= 1e-30f))
    return fail(MQ_E_SHAPE, "%s: eps %g must be finite and at least 1e-30", who, (double)r->eps);
  if ((r->cos_sin != nullptr) != (r->rot_dim != 0))
    return fail(MQ_E_NULL, "%s: cos_sin must be given exactly where rot_dim is not 0", who);
  for (const void *p : {(const void *)r->cos_sin, (const void *)r->q_norm, (const void *)r->k_norm})
    if (p && !aligned(p, 16)) return fail(MQ_E_ALIGN, "%s: cos_sin and norm weights must be 16-byte aligned", who);
  return MQ_OK;
}

mq_status check_heads(const mq_kv_cache *c, int32_t q_heads, const char *who) {
  if (q_heads < 1 || q_heads > mq::kMaxHeads || q_heads % c->kv_heads)
    return fail(MQ_E_SHAPE, "%s: q_heads %d must be a multiple of kv_heads %d and at most %d", who, q_heads,
                c->kv_heads, mq::kMaxHeads);
  return MQ_OK;
}

mq_status check_units(const mq_kv_cache *c, int32_t q_heads, int64_t batch, const char *who) {
  const int64_t units = batch * c->kv_heads * ((q_heads / c->kv_heads + 15) / 16);
  if (units > mq::kMaxUnits)
    return fail(MQ_E_SHAPE, "%s: batch %lld times %lld groups of up to 16 query heads exceed %lld", who, (long long)batch,
                (long long)(units / batch), (long long)mq::kMaxUnits);
  return MQ_OK;
}

}  // namespace

extern "C" {

mq_status moe_quant_linear_workspace_size(const mq_linear *l, int64_t num_tokens, size_t *bytes) {
  mq_status st = check_linear(l, "linear_workspace_size");
  if (st == MQ_OK) st = check_tokens(num_tokens, "linear_workspace_size");
  if (st != MQ_OK) return st;
  if (!bytes) return fail(MQ_E_NULL, "linear_workspace_size: NULL argument");
  *bytes = linear_ws(num_tokens, l->k).total;
  return MQ_OK;
}

mq_status moe_quant_linear(const mq_linear *l, const uint16_t *x_bf16, const uint16_t *residual_bf16,
                           int64_t num_tokens, void *out, void *workspace, size_t workspace_bytes,
                           struct ihipStream_t *stream) {
  mq_status st = check_linear(l, "linear");
  if (st == MQ_OK) st = check_tokens(num_tokens, "linear");
  if (st != MQ_OK) return st;
  if (num_tokens == 0) {
    mq::clear_error();
    return MQ_OK;
  }
  if (!x_bf16 || !out) return fail(MQ_E_NULL, "linear: x and out must be non-NULL");
  const bool bf16 = l->out_dtype == MQ_BF16;
  if (!aligned(x_bf16, 16) || !aligned(out, bf16 ? 2 : 4) || (residual_bf16 && !aligned(residual_bf16, 2)))
    return fail(MQ_E_ALIGN, "linear: x must be 16-byte aligned, out and residual to their element");
  const size_t values = (size_t)num_tokens * l->n;
  if (overlap(out, values * (bf16 ? 2 : 4), x_bf16, (size_t)num_tokens * l->k * 2))
    return fail(MQ_E_SHAPE, "linear: out must not overlap x, which other workgroups still read");
  if (residual_bf16 && (bf16 ? out != residual_bf16 : true) && overlap(out, values * (bf16 ? 2 : 4), residual_bf16, values * 2))
    return fail(MQ_E_SHAPE, "linear: out may overlap the residual only as a BF16 out that is the residual itself");
  if (!workspace) return fail(MQ_E_WORKSPACE, "linear: workspace is NULL");
  if (!aligned(workspace, 256)) return fail(MQ_E_ALIGN, "linear: workspace not 256-byte aligned");
  const LinearWs w = linear_ws(num_tokens, l->k);
  if (workspace_bytes < w.total)
    return fail(MQ_E_WORKSPACE, "linear: workspace %zu bytes, need %zu", workspace_bytes, w.total);
  const Bytes o = {out, values * (bf16 ? 2 : 4)}, ws = {workspace, w.total}, wt = {l->w, (size_t)l->n * l->k},
              sc = {l->scale, (size_t)((l->n + 127) / 128) * ((l->k + 127) / 128) * 4};
  if (meets(o, {ws, wt, sc}) || meets(ws, {{x_bf16, (size_t)num_tokens * l->k * 2}, {residual_bf16, values * 2}, wt, sc}))
    return fail(MQ_E_SHAPE, "linear: out and workspace must not overlap each other, the weight, the scale or an input");
  mq::LinearArgs a;
  a.x = x_bf16; a.residual = residual_bf16; a.w = l->w; a.scale = l->scale; a.out = out;
  a.codes = (uint8_t *)workspace + w.codes;
  a.sa = (float *)((char *)workspace + w.sa);
  a.T = num_tokens; a.N = l->n; a.K = l->k; a.G = (l->k + 127) / 128; a.out_bf16 = bf16;
  const hipError_t e = mq::launch_linear(a, (hipStream_t)stream);
  if (e != hipSuccess) return fail(MQ_E_HIP, "linear: %s", hipGetErrorString(e));
  mq::clear_error();
  return MQ_OK;
}

mq_status moe_quant_kv_append(const mq_kv_cache *c, const mq_rotary *r, int32_t q_heads,
                              const uint16_t *q, int64_t q_stride, const uint16_t *k,
                              int64_t k_stride, const uint16_t *v, int64_t v_stride,
                              const int32_t *positions, const int32_t *slots, int64_t num_tokens,
                              uint16_t *q_out, struct ihipStream_t *stream) {
  mq_status st = check_cache(c, "kv_append");
  if (st == MQ_OK) st = check_rotary(r, c, "kv_append");
  if (st == MQ_OK) st = check_tokens(num_tokens, "kv_append");
  if (st != MQ_OK) return st;
  if (q_heads < 0 || q_heads > mq::kMaxHeads)
    return fail(MQ_E_SHAPE, "kv_append: q_heads %d outside [0, %d]", q_heads, mq::kMaxHeads);
  if (num_tokens == 0) {
    mq::clear_error();
    return MQ_OK;
  }
  if (!k || !v || !slots || (r->rot_dim && !positions))
    return fail(MQ_E_NULL, "kv_append: k, v, slots and (with a rotation) positions must be non-NULL");
  if ((q != nullptr) != (q_heads != 0) || (q_out != nullptr) != (q_heads != 0))
    return fail(MQ_E_NULL, "kv_append: q and q_out must be given exactly where q_heads is not 0");
  for (const void *p : {(const void *)q, (const void *)k, (const void *)v, (const void *)q_out})
    if (p && !aligned(p, 16)) return fail(MQ_E_ALIGN, "kv_append: q, k, v and q_out must be 16-byte aligned");
  if (!aligned(slots, 4) || (positions && !aligned(positions, 4)))
    return fail(MQ_E_ALIGN, "kv_append: positions and slots must be 4-byte aligned");
  const int64_t D = c->head_dim, kv = c->kv_heads * D;
  if ((q && q_stride < q_heads * D) || k_stride < kv || v_stride < kv)
    return fail(MQ_E_SHAPE, "kv_append: token strides %lld, %lld and %lld shorter than a token's heads",
                (long long)q_stride, (long long)k_stride, (long long)v_stride);
  if ((q && q_stride % 8) || k_stride % 8 || v_stride % 8)
    return fail(MQ_E_ALIGN, "kv_append: token strides must be multiples of 8 values");
  if (q && q_out == q && q_stride != q_heads * D)
    return fail(MQ_E_SHAPE, "kv_append: q_out may be q only where q's tokens lie one behind the other");
  auto span = [&](int64_t stride, int64_t row) { return (size_t)((num_tokens - 1) * stride + row) * 2; };
  const size_t out_bytes = (size_t)(num_tokens * q_heads * D) * 2;
  if (q && (overlap(q_out, out_bytes, k, span(k_stride, kv)) || overlap(q_out, out_bytes, v, span(v_stride, kv)) ||
            (q_out != q && overlap(q_out, out_bytes, q, span(q_stride, q_heads * D)))))
    return fail(MQ_E_SHAPE, "kv_append: q_out may be q itself but must not overlap q, k and v otherwise");
  const Bytes kc = {c->k, cache_bytes(c)}, vc = {c->v, cache_bytes(c)}, qo = {q_out, out_bytes},
              at = {slots, (size_t)num_tokens * 4}, pos = {r->rot_dim ? positions : nullptr, (size_t)num_tokens * 4},
              cs = {r->cos_sin, (size_t)r->max_positions * r->rot_dim * 4}, qn = {r->q_norm, (size_t)D * 2},
              kn = {r->k_norm, (size_t)D * 2};
  if (meets(qo, {kc, vc, at, pos, cs, qn, kn}) || meets(kc, {vc}))
    return fail(MQ_E_SHAPE, "kv_append: q_out and the cache's k and v must not overlap each other or what is read");
  for (const Bytes &cache : {kc, vc})
    if (meets(cache, {{q, span(q_stride, q_heads * D)}, {k, span(k_stride, kv)}, {v, span(v_stride, kv)}, at, pos, cs, qn, kn}))
      return fail(MQ_E_SHAPE, "kv_append: the cache's k and v must not overlap what the call reads");
  mq::KvAppendArgs a;
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.positions = positions; a.slots = slots; a.cos_sin = r->cos_sin; a.q_norm = r->q_norm; a.k_norm = r->k_norm;
  a.q_out = q_out; a.kc = c->k; a.vc = c->v;
  a.num_slots = c->num_pages * c->page_size; a.T = num_tokens;
  a.Hq = q_heads; a.Hk = c->kv_heads; a.D = c->head_dim; a.R = r->rot_dim; a.interleaved = r->interleaved != 0;
  a.max_positions = r->max_positions; a.page_log2 = __builtin_ctz(c->page_size); a.fp8 = c->dtype == MQ_KV_FP8;
  a.eps = r->eps; a.k_scale = c->k_scale; a.v_scale = c->v_scale;
  const hipError_t e = mq::launch_kv_append(a, (hipStream_t)stream);
  if (e != hipSuccess) return fail(MQ_E_HIP, "kv_append: %s", hipGetErrorString(e));
  mq::clear_error();
  return MQ_OK;
}

mq_status moe_quant_attend_workspace_size(const mq_kv_cache *c, int32_t q_heads, int64_t batch,
                                          size_t *bytes) {
  mq_status st = check_cache(c, "attend_workspace_size");
  if (st == MQ_OK) st = check_heads(c, q_heads, "attend_workspace_size");
  if (st == MQ_OK) st = check_batch(batch, "attend_workspace_size");
  if (st == MQ_OK) st = check_units(c, q_heads, batch, "attend_workspace_size");
  if (st != MQ_OK) return st;
  if (!bytes) return fail(MQ_E_NULL, "attend_workspace_size: NULL argument");
  *bytes = mq::attend_workspace(batch, q_heads, c->kv_heads, c->head_dim);
  return MQ_OK;
}

mq_status moe_quant_attend(const mq_kv_cache *c, int32_t q_heads, float scale, int32_t window,
                           const uint16_t *q_bf16, const int32_t *block_table, int64_t table_stride,
                           int32_t max_pages, const int32_t *lengths, int64_t batch,
                           uint16_t *out_bf16, float *lse, void *workspace, size_t workspace_bytes,
                           struct ihipStream_t *stream) {
  mq_status st = check_cache(c, "attend");
  if (st == MQ_OK) st = check_heads(c, q_heads, "attend");
  if (st == MQ_OK) st = check_batch(batch, "attend");
  if (st == MQ_OK) st = check_units(c, q_heads, batch, "attend");
  if (st != MQ_OK) return st;
  const float score_scale = scale * c->k_scale * 1.44269504088896340736f;
  if (!std::isfinite(scale) || !std::isfinite(score_scale))
    return fail(MQ_E_SHAPE, "attend: scale %g, and times k_scale %g and log2(e), must be finite", (double)scale,
                (double)c->k_scale);
  if (window < 0) return fail(MQ_E_SHAPE, "attend: window %d must not be negative", window);
  if (max_pages < 0 || max_pages > mq::kMaxRequest / c->page_size || table_stride < max_pages)
    return fail(MQ_E_SHAPE, "attend: max_pages %d times page_size must be at most 2^30, table_stride %lld at least "
                "max_pages", max_pages, (long long)table_stride);
  if (batch == 0) {
    mq::clear_error();
    return MQ_OK;
  }
  if (!q_bf16 || !lengths || !out_bf16 || (!block_table && max_pages))
    return fail(MQ_E_NULL, "attend: q, block_table, lengths and out must be non-NULL");
  if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) ||
      (lse && !aligned(lse, 4)))
    return fail(MQ_E_ALIGN, "attend: q and out must be 16-byte, block_table, lengths and lse 4-byte aligned");
  const size_t q_bytes = (size_t)(batch * q_heads) * c->head_dim * 2;
  if (out_bf16 != q_bf16 && overlap(out_bf16, q_bytes, q_bf16, q_bytes))
    return fail(MQ_E_SHAPE, "attend: out may be q itself but must not overlap it otherwise");
  if (!workspace) return fail(MQ_E_WORKSPACE, "attend: workspace is NULL");
  if (!aligned(workspace, 256)) return fail(MQ_E_ALIGN, "attend: workspace not 256-byte aligned");
  const size_t need = mq::attend_workspace_need(batch, q_heads, c->kv_heads, c->head_dim);
  if (workspace_bytes < need)
    return fail(MQ_E_WORKSPACE, "attend: workspace %zu bytes, need %zu", workspace_bytes, need);
  const Bytes kc = {c->k, cache_bytes(c)}, vc = {c->v, cache_bytes(c)}, o = {out_bf16, q_bytes}, ws = {workspace, need},
              l = {lse, (size_t)(batch * q_heads) * 4}, len = {lengths, (size_t)batch * 4},
              tab = {block_table, ((size_t)(batch - 1) * (size_t)table_stride + max_pages) * 4}, q = {q_bf16, q_bytes};
  if (meets(o, {kc, vc, ws, l, len, tab}) || meets(l, {kc, vc, ws, len, tab, q}) || meets(ws, {kc, vc, len, tab, q}))
    return fail(MQ_E_SHAPE, "attend: out, lse and workspace must not overlap each other, the cache or an input");
  mq::AttendArgs a;
  a.q = q_bf16; a.kc = c->k; a.vc = c->v; a.table = block_table; a.lengths = lengths;
  a.table_stride = table_stride; a.out = out_bf16; a.lse = lse; a.ws = workspace;
  a.B = (int)batch; a.Hq = q_heads; a.Hk = c->kv_heads; a.D = c->head_dim; a.page_log2 = __builtin_ctz(c->page_size);
  a.num_pages = (int)c->num_pages; a.max_tokens = max_pages * c->page_size; a.window = window;
  a.score_scale = score_scale; a.v_scale = c->v_scale;
  const hipError_t e = mq::launch_attend(a, c->dtype == MQ_KV_FP8, (hipStream_t)stream);
  if (e != hipSuccess) return fail(MQ_E_HIP, "attend: %s", hipGetErrorString(e));
  mq::clear_error();
  return MQ_OK;
}

}  // extern "C"
