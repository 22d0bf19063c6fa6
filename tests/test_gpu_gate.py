"""Gated routing on the GPU against the float64 oracle: ids equal, weights to
FP32 accuracy."""
import math

import numpy as np
import pytest
import torch

from oracle import gate as ogate
from weight_quantized_moe_amd import Gate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def as_f64(logits):
    return logits.float().cpu().numpy().astype(np.float64)


def weight_tolerance(lg, bias, ids, kw):
    """Relative error allowed for a weight.  Its exponentials take an argument a
    whose FP32 rounding (relative 2^-24, and as much again for the product with
    log2 e) becomes an error of 2 |a| 2^-24 in the result; with another such term
    for the row's sum that is 4 |a| 2^-24, plus about 24 roundings of 2^-24 (the
    exponential's own, the sum's at most 9 additions, quotients and the scale).
    |a| is a negative logit's size for a sigmoid (renormalised: its distance from
    the largest), the distance from the row's maximum for a softmax, and in the
    softmax's sum over all experts the terms' error is weighted by the terms
    themselves, at most ln E on average."""
    picked = np.take_along_axis(lg, ids.astype(np.int64), 1)
    if kw.get("score", "softmax") == "softmax":
        a = np.nanmax(np.where(np.isfinite(lg), lg, np.nan), 1, keepdims=True, initial=-1e300) - picked
    else:
        a = np.minimum(picked, 0.0)
        if kw.get("renormalize", True):
            a = np.maximum(a, -1e300) - np.maximum(a, -1e300).max(1, keepdims=True)
            a = np.where(a < -1e299, 0.0, a)              # masked: weight 0
    a = np.where(np.isfinite(a), np.abs(a), 0.0)
    if kw.get("renormalize", True):
        a = np.maximum(a, a.max(1, keepdims=True))
    return 2.0 ** -24 * (24 + 4 * np.maximum(a, math.log(lg.shape[1])))


def check(logits, k, bias=None, g=None, **kw):
    t, e = logits.shape
    g = g or Gate(e, k, bias=bias, **{("num_groups" if n == "groups" else n): v for n, v in kw.items()})
    # places behind the last token stay as they were
    ids = torch.full((t + 2, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((t + 2, k), -7.0, device="cuda")
    g.topk(logits, ids=ids[:t], weights=w[:t])
    torch.cuda.synchronize()
    assert torch.all(ids[t:] == -7) and torch.all(w[t:] == -7.0)
    lg = as_f64(logits)
    b = None if bias is None else bias.cpu().numpy().astype(np.float64)
    ref_ids, ref_w = ogate.gate(lg, k, bias=b, **kw)
    got = ids[:t].cpu().numpy()
    bad = np.nonzero((got != ref_ids).any(1))[0]
    assert not len(bad), (len(bad), bad[:3], got[bad[:3]], ref_ids[bad[:3]])
    got_w = w[:t].cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got_w))
    clean = np.where(np.isnan(lg), -np.inf, np.minimum(lg, float(np.finfo(np.float32).max)))
    tol = weight_tolerance(clean, b, ref_ids, kw)
    off = np.abs(got_w - ref_w)
    assert np.all(off <= tol * np.abs(ref_w) + 2.0 ** -126), float((off / np.maximum(np.abs(ref_w), 1e-30)).max())
    return ids[:t], w[:t]


def logits(t, e, seed=0, dtype=torch.float32, spread=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lg = spread * torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
    return lg.to(dtype)


def a_bias(e, seed=1, size=0.1):
    return size * torch.randn(e, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


KINDS = {
    "softmax": dict(score="softmax"),
    "softmax_raw": dict(score="softmax", renormalize=False, scale=16.0),
    "sigmoid": dict(score="sigmoid"),
    "sigmoid_raw": dict(score="sigmoid", renormalize=False, scale=0.5),
}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 128, 8), (2, 7, 7), (5, 16, 4), (17, 65, 3), (64, 127, 16),
                                   (33, 128, 17), (130, 256, 8), (7, 511, 64), (300, 72, 6), (3, 512, 33), (37, 192, 8), (37, 384, 8), (9, 380, 16), (21, 186, 5), (5, 2, 1)])
def test_topk(kind, with_bias, t, e, k):
    check(logits(t, e, seed=t + e), k, bias=a_bias(e) if with_bias else None, **KINDS[kind])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid_raw"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k,groups,topk_groups,group_top", [
    (5, 256, 8, 8, 4, 2), (64, 256, 8, 8, 4, 1), (129, 128, 6, 4, 2, 2), (3, 16, 2, 16, 5, 1), (40, 72, 6, 8, 3, 2),
    (31, 96, 9, 3, 2, 2), (21, 512, 20, 32, 7, 2), (11, 512, 8, 64, 64, 2), (50, 24, 3, 2, 1, 2), (50, 20, 4, 5, 1, 2),
    (77, 160, 6, 16, 8, 2), (9, 8, 2, 4, 1, 2)])
def test_groups(kind, with_bias, dtype, t, e, k, groups, topk_groups, group_top):
    check(logits(t, e, seed=e + k, dtype=dtype), k, bias=a_bias(e) if with_bias else None, groups=groups,
          topk_groups=topk_groups, group_top=group_top, **KINDS[kind])


@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
def test_scores_closer_than_a_32_bit_rounding(groups, topk_groups):
    """Biases that differ by about 2^-30 next to scores that are equal, and by
    1 or 2 units of the last place next to scores that are not: a 32-bit sum
    cannot order them."""
    t, e = 64, 64
    gen = np.random.default_rng(5)
    lg = np.repeat(gen.normal(size=(t, e // 4)), 4, axis=1).astype(np.float32)
    near = lg.copy()
    near[:, 1::4] = np.nextafter(lg[:, 1::4], np.float32(9))
    near[:, 2::4] = np.nextafter(lg[:, 2::4], np.float32(-9))
    bias = (0.25 + gen.integers(-8, 8, e) * 2.0 ** -25).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        check(torch.from_numpy(near).cuda(), 8, bias=torch.from_numpy(bias).cuda(), score=kind, groups=groups,
              topk_groups=topk_groups, group_top=2 if groups > 1 else 1)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_ties(kind, with_bias, groups, topk_groups):
    """Equal scores go to the lower id: rows of one value, few values, +0 and -0,
    and rows of BF16 logits."""
    e, k = 64, 8
    lg = logits(40, e, dtype=torch.bfloat16).float()
    lg[0] = 0.25
    lg[1] = torch.where(torch.arange(e, device="cuda") % 2 == 0, 0.0, -0.0)
    lg[2:12] = lg[2:12].round()
    lg[12, ::3] = lg[12].max()
    b = torch.zeros(e, device="cuda") if with_bias else None
    for x in (lg, lg.bfloat16()):
        check(x, k, bias=b, groups=groups, topk_groups=topk_groups, group_top=2 if groups > 1 else 1, **KINDS[kind])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2), (3, 2)])
def test_masks(kind, dtype, groups, topk_groups):
    """-inf and NaN mask an expert, rows with few or no live experts, +inf, and the
    type's lowest value, which is a number."""
    e, k = 48, 6
    lg = logits(24, e).to(dtype)
    inf, low = math.inf, torch.finfo(dtype).min
    lg[0] = -inf
    lg[1] = math.nan
    lg[2], lg[2, 40] = -inf, -1.0
    lg[3], lg[3, 5], lg[3, 17], lg[3, 18] = -inf, 0.5, 0.5, 3.0
    lg[4, ::2] = -inf
    lg[5, 3] = math.nan
    lg[6, 7] = inf
    lg[7, 9], lg[7, 30], lg[7, 2] = inf, inf, -inf
    lg[8] = low
    lg[9, 1:] = low
    lg[10] = torch.finfo(dtype).max
    lg[11, : e // 3] = -inf
    bias = a_bias(e)
    bias[4], bias[21], bias[33] = -inf, math.nan, inf
    for b in (None, bias):
        check(lg, k, bias=b, groups=groups, topk_groups=topk_groups, group_top=2 if groups > 1 else 1, **KINDS[kind])


@pytest.mark.parametrize("kind", list(KINDS))
def test_far_logits(kind):
    """Sigmoids that underflow or round to 1 and exponentials of every size: the
    renormalised weights of very negative logits keep their digits."""
    for shift in (-3e4, -200.0, -90.0, -60.0, 30.0, 3e4):
        lg = logits(16, 96, seed=3) + shift
        if kind == "sigmoid_raw" and shift < -80:
            continue                                  # weights below the smallest normal number
        check(lg, 8, **KINDS[kind])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid_raw"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("e,k,groups,topk_groups", [(512, 12, 1, 1), (256, 8, 8, 1), (512, 8, 16, 4), (128, 8, 4, 1),
                                                    (256, 16, 8, 2), (160, 16, 1, 1)])
def test_scores_bunched_in_few_lanes(kind, with_bias, e, k, groups, topk_groups):
    """The best experts next to each other, in falling and rising order: many
    candidates in a lane, and groups that keep few lanes."""
    lg = logits(40, e, seed=k)
    lg[:10] = torch.linspace(3, -3, e, device="cuda")
    lg[10:20] = torch.linspace(-3, 3, e, device="cuda")
    lg[20:30, e // 2:e // 2 + 40] += 4
    check(lg, k, bias=a_bias(e, size=0.01) if with_bias else None, groups=groups, topk_groups=topk_groups,
          group_top=2 if groups > 1 else 1, **KINDS[kind])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_closer_than_a_32_bit_rounding(score):
    """Group sums that differ by 2^-26 and less, equal ones, and groups whose
    three best experts lie within 2^-24."""
    t, e, groups = 64, 128, 8
    gen = np.random.default_rng(7)
    lg = np.zeros((t, e), np.float32)
    top = gen.normal(size=(t, 1, 3)).astype(np.float32) + 3
    lg.reshape(t, groups, 16)[:] = gen.normal(size=(t, groups, 16)) - 2
    lg.reshape(t, groups, 16)[:, :, 4:7] = top
    lg.reshape(t, groups, 16)[20:40, :, 9] = top[20:40, :, 0]
    bias = (gen.integers(-4, 4, e) * 2.0 ** -27).astype(np.float32)
    wide = (gen.integers(-4, 4, e) * 2.0 ** -23).astype(np.float32)
    for b in (bias, wide, None):
        for top_n in (1, 2):
            check(torch.from_numpy(lg).cuda(), 6, bias=None if b is None else torch.from_numpy(b).cuda(), score=score,
                  groups=groups, topk_groups=3, group_top=top_n)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 1), (8, 3), (3, 2)])
def test_biases_whose_sums_pass_32_bits(score, groups, topk_groups):
    # the type's lowest value is a number, not a mask: a group that holds nothing
    # else comes before one that is masked, a group of larger numbers before both
    e, k = 96, 6
    per, low = e // groups, torch.finfo(torch.float32).min
    for values in ((-math.inf, low, 0.75 * low), (low, -math.inf, low), (0.75, 1.0, 0.875), (0.0, low, math.inf)):
        size = 1.0 if abs(values[0]) > 1.0 or values[0] == 0.0 else -low
        bias = torch.empty(e, device="cuda")
        for i in range(groups):
            bias[i * per:(i + 1) * per] = values[min(i, 2)] * size
        bias[per // 2] = 0.5 * low
        check(logits(9, e, seed=groups), k, bias=bias, score=score, groups=groups, topk_groups=topk_groups,
              group_top=2 if groups > 1 else 1)


def test_many_tokens_and_limits():
    check(logits(5000, 64, seed=9), 4, bias=a_bias(64), score="sigmoid", groups=8, topk_groups=4, group_top=2, scale=2.5)
    g = Gate(16, 2)
    empty = torch.empty((0, 16), device="cuda")
    ids, w = g.topk(empty)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


def test_offsets_past_32_bits():
    """Rows whose logits lie beyond 2^31 elements of their array."""
    t, e, k = (1 << 22), 513 - 1, 2                     # 2^31 logits in BF16
    lg = torch.zeros((t, e), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, t // 2, t - 2, t - 1], device="cuda")
    lg[rows] = logits(len(rows), e, dtype=torch.bfloat16)
    ids, w = Gate(e, k).topk(lg)
    ref_ids, ref_w = ogate.gate(as_f64(lg[rows]), k)
    assert np.array_equal(ids[rows].cpu().numpy(), ref_ids)
    assert np.allclose(w[rows].cpu().numpy(), ref_w, rtol=1e-5)
    assert torch.equal(ids[5], torch.tensor([0, 1], dtype=torch.int32, device="cuda"))


def test_same_bits_again_on_another_stream_and_in_a_graph():
    lg, b = logits(333, 256), a_bias(256)
    g = Gate(256, 8, score="sigmoid", bias=b, num_groups=8, topk_groups=4, group_top=2)
    ids, w = g.topk(lg)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    i2, w2 = g.topk(lg, stream=s)
    s.synchronize()
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    i3, w3, x = torch.zeros_like(ids), torch.zeros_like(w), lg.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.topk(x, ids=i3, weights=w3)
    for r in range(3):
        x.copy_(logits(333, 256, seed=20 + r))
        graph.replay()
        i4, w4 = g.topk(x)
        torch.cuda.synchronize()
        assert torch.equal(i3, i4) and torch.equal(w3, w4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [6, 17])
def test_raw_weights_keep_their_digits_far_from_zero(score, k):
    """The exponent of a far logit is exact: a sigmoid's is the logit itself, and
    these softmaxes' logits are multiples of 2^-10 below a maximum of 0.  What is
    left, in units of 2^-24: 2 for the power and 2 for the reciprocal (one unit in
    their last place), 1 each for the power's correction, the product, the scale
    and the reference's own cast, the denominator's 1 + exp(-|l|) 2 (a rounding,
    and |l| exp(-|l|) log2 e of the power at most 0.53); a softmax's sum over 24
    experts takes at most 24 additions in place of those 2, and its terms' powers,
    off by |a| exp(-|a|) log2 e + 2, weighted by themselves, at most 3: 10, 36."""
    e, t = 24, 400
    gen = np.random.default_rng(3)
    lg = gen.uniform(-85.0, 20.0, (t, e)).astype(np.float32)
    if score == "softmax":
        lg = np.round(lg * 1024 * 0.8).clip(-81920, 0).astype(np.float32) / 1024
        lg[:, 5] = 0.0
    ids, w = Gate(e, k, score=score, renormalize=False, scale=1.5).topk(torch.from_numpy(lg).cuda())
    torch.cuda.synchronize()
    ref_ids, ref = ogate.gate(lg.astype(np.float64), k, score, renormalize=False, scale=1.5)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    off = np.abs(w.cpu().numpy().astype(np.float64) - ref) / ref
    assert off.max() <= (10 if score == "sigmoid" else 36) * 2.0 ** -24, off.max() * 2.0 ** 24


def test_the_largest_array_in_32_bits():
    """The most tokens and experts there may be: 2^31 logits, the last at element
    2^31 - 1 and past byte 2^33."""
    t, e, k = 1 << 22, 512, 3
    lg = torch.zeros((t, e), device="cuda")
    rows = torch.tensor([0, 1, 5, t // 4, t // 2 + 1, t - 2, t - 1], device="cuda")
    lg[rows] = logits(len(rows), e)
    ids, w = Gate(e, k, score="sigmoid", bias=a_bias(e)).topk(lg)
    ref_ids, ref_w = ogate.gate(as_f64(lg[rows]), k, "sigmoid", bias=as_f64(a_bias(e)))
    assert np.array_equal(ids[rows].cpu().numpy(), ref_ids)
    assert np.allclose(w[rows].cpu().numpy(), ref_w, rtol=1e-5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e,t0", [(128, 3), (65, 8), (511, 16), (48, 5)])
def test_rows_from_the_middle_of_larger_arrays(dtype, e, t0):
    """Logits, ids and weights that begin and end inside larger arrays, as a prompt
    in chunks gives them: what lies around the outputs stays."""
    t, k = 21, 5
    lg, bias = logits(64, e, dtype=dtype), a_bias(e)
    lg[:t0], lg[t0 + t:] = 100.0, 100.0
    g = Gate(e, k, score="sigmoid", bias=bias)
    ids = torch.full((64, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((64, k), -7.0, device="cuda")
    cut = slice(t0, t0 + t)
    g.topk(lg[cut], ids=ids[cut], weights=w[cut])
    torch.cuda.synchronize()
    ref_ids, ref_w = ogate.gate(as_f64(lg[cut]), k, "sigmoid", bias=as_f64(bias))
    assert np.array_equal(ids[cut].cpu().numpy(), ref_ids) and np.allclose(w[cut].cpu().numpy(), ref_w, rtol=1e-5)
    for a in (ids, w):
        assert bool((a[:t0] == -7).all()) and bool((a[t0 + t:] == -7).all())


@pytest.mark.parametrize("e,k,groups,topk_groups", [(12, 4, 1, 1), (64, 4, 1, 1), (64, 17, 1, 1), (64, 8, 8, 3), (48, 6, 3, 2)])
def test_sigmoids_as_small_as_64_bits_hold(e, k, groups, topk_groups):
    """Logits of -735 to -700 half a unit apart: their sigmoids are subnormal numbers
    in 64 bits, in the logits' order."""
    gen = np.random.default_rng(11)
    lg = np.stack([gen.permutation(70)[:e] for _ in range(30)]).astype(np.float32) * 0.5 - 735.0
    for top in (1, 2) if groups > 1 else (1,):
        g = Gate(e, k, score="sigmoid", bias=torch.zeros(e, device="cuda"), num_groups=groups, topk_groups=topk_groups,
                 group_top=top)
        ids, _ = g.topk(torch.from_numpy(lg).cuda())
        ref, _ = ogate.gate(lg.astype(np.float64), k, "sigmoid", bias=np.zeros(e), groups=groups,
                            topk_groups=topk_groups, group_top=top)
        assert np.array_equal(ids.cpu().numpy(), ref)
