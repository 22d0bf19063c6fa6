"""Norms before and after a block on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import norm as onorm
from weight_quantized_moe_amd import ResidualNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def inputs(t, h, rd=BF, wd=BF, gate="none", gd=BF, seed=0, size=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    shape = {"none": None, "channel": (h,), "token": (t, 1), "full": (t, h)}[gate]
    return dict(x=(size * rn(t, h)).to(BF), r=(4 * rn(t, h)).to(rd),
                g=None if shape is None else (1 + 0.5 * rn(*shape)).to(gd),
                post=(1 + 0.1 * rn(h)).to(wd), pre=(1 + 0.1 * rn(h)).to(wd))


def check(t, h, d, post=True, pre=True, rd=BF, eps=1e-6, offset=0.0, scale=1.0, x=True, residual=True, size=None):
    """Elementwise bounds.  The squares' sum takes h / 64 additions in a lane and
    about 16 across lanes and waves at most, halved by the root; a handful of
    products follow: c = 16 + h / 64 roundings of 2^-24 of each term, and half a
    step of the output's type.  The second norm is compared with the oracle's
    norm of the residual that came back, which it is defined on."""
    n = ResidualNorm(h, post_weight=d["post"] if post else None, pre_weight=d["pre"] if pre else None, eps=eps,
                     weight_offset=offset, scale=scale, residual_dtype=rd)
    # rows behind the last one stay as they were
    ro = torch.full((t + 1, h), 7.0, dtype=rd, device="cuda")
    no = torch.full((t + 1, h), 7.0, dtype=BF, device="cuda")
    got_r, got_n = n.forward(d["x"] if x else None, d["r"] if residual else None, gate=d["g"] if x else None,
                             residual_out=ro[:t], norm_out=no[:t] if pre else None)
    torch.cuda.synchronize()
    assert torch.all(ro[t:] == 7.0) and torch.all(no[t:] == 7.0) and (got_n is None) == (not pre)
    c = (16 + h / 64) * 2.0 ** -24
    half = torch.finfo(rd).eps / 2
    r, add = onorm.residual_update(f64(d["x"]) if x else None, f64(d["r"]) if residual else None,
                                   f64(d["g"]) if x else None, f64(d["post"]) if post else None, eps, offset, scale)
    ref = r + add
    off = np.abs(f64(got_r) - ref)
    limit = half * np.abs(ref) * (1 + c) + c * (np.abs(r) + np.abs(add)) + 1e-38
    assert np.all(off <= limit), (float((off / limit).max()), np.unravel_index((off / limit).argmax(), off.shape))
    if pre:
        ref = onorm.rms_norm(f64(got_r), f64(d["pre"]), eps, offset)
        off, limit = np.abs(f64(got_n) - ref), (2.0 ** -8 + c) * np.abs(ref) + 1e-38
        assert np.all(off <= limit), (float((off / limit).max()), np.unravel_index((off / limit).argmax(), off.shape))
    return got_r, got_n


HIDDEN = [1, 2, 7, 8, 64, 129, 256, 520, 1023, 1024, 2048, 2056, 4096, 4100, 5000, 8192, 8200, 16384, 16392, 32760, 32768]


@pytest.mark.parametrize("h", HIDDEN)
@pytest.mark.parametrize("rd", [BF, F32])
def test_sizes(h, rd):
    for t in (1, 3, 37):
        check(t, h, inputs(t, h, rd, gate="full", seed=h), rd=rd, scale=0.5)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("gd", [BF, F32])
@pytest.mark.parametrize("wd", [BF, F32])
@pytest.mark.parametrize("h", [96, 333, 2048])
def test_gates_and_types(gate, gd, wd, h):
    for post, pre in ((True, True), (True, False), (False, True), (False, False)):
        for rd in (BF, F32):
            check(5, h, inputs(5, h, rd, wd, gate, gd), post, pre, rd, offset=1.0, scale=-0.22, eps=1e-5)


def test_without_x_or_residual():
    for h in (64, 77, 4096):
        d = inputs(9, h)
        check(9, h, d, post=False, x=False)
        check(9, h, d, residual=False)
        check(9, h, d, pre=False, residual=False)
        r, _ = check(9, h, d, post=False, pre=False, x=False)
        assert torch.equal(r, d["r"])


@pytest.mark.parametrize("h", [256, 333, 8192])
def test_two_calls_give_the_bits_of_one(h):
    for rd in (BF, F32):
        d = inputs(11, h, rd, gate="channel")
        r, n = check(11, h, d, rd=rd)
        r1, none = ResidualNorm(h, post_weight=d["post"], residual_dtype=rd).forward(d["x"], d["r"], gate=d["g"])
        r2, n2 = ResidualNorm(h, pre_weight=d["pre"], residual_dtype=rd).forward(None, r1)
        assert none is None and torch.equal(r, r1) and torch.equal(r, r2) and torch.equal(n, n2)


@pytest.mark.parametrize("h", [64, 1001, 2048, 16384])
def test_outputs_in_the_inputs_own_buffers(h):
    for rd in (BF, F32):
        d = inputs(13, h, rd, gate="full")
        r, n = check(13, h, d, rd=rd)
        op = ResidualNorm(h, post_weight=d["post"], pre_weight=d["pre"], residual_dtype=rd)
        x, res = d["x"].clone(), d["r"].clone()
        op.forward(x, res, gate=d["g"], residual_out=res, norm_out=x)
        torch.cuda.synchronize()
        assert torch.equal(res, r) and torch.equal(x, n)


def test_zero_rows_and_far_values():
    h = 512
    d = inputs(6, h)
    d["x"][0], d["r"][0] = 0, 0
    d["x"][1] = 2.0 ** 50
    d["r"][2] = -(2.0 ** 50)
    d["x"][3] = 2.0 ** -60
    d["x"][4, 1:], d["x"][4, 0] = 0, 1e30 * 2.0 ** -60
    r, n = check(6, h, d)
    assert torch.all(r[0] == 0) and torch.all(n[0] == 0)


def test_many_rows_and_none():
    d = inputs(20000, 128, gate="token")
    check(20000, 128, d)
    d = inputs(1, 64)
    op = ResidualNorm(64, post_weight=d["post"], pre_weight=d["pre"])
    r, n = op.forward(d["x"][:0], d["r"][:0])
    assert r.shape == (0, 64) and n.shape == (0, 64)


def test_offsets_past_32_bits():
    t, h = 70000, 32768                                 # 2.3e9 values
    x = torch.zeros((t, h), dtype=BF, device="cuda")
    d = inputs(3, h)
    x[-3:] = d["x"]
    op = ResidualNorm(h, post_weight=d["post"])
    r, _ = op.forward(x)
    small, _ = op.forward(d["x"])
    assert torch.equal(r[-3:], small) and torch.all(r[-4] == 0)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("rd", [BF, F32])
def test_more_rows_than_a_launch_takes(gate, rd):
    t, h, k = (1 << 21) + 5, 16, 9
    d = inputs(t, h, rd, gate=gate, gd=F32 if rd == BF else BF)
    op = ResidualNorm(h, post_weight=d["post"], pre_weight=d["pre"], residual_dtype=rd)
    r, n = op.forward(d["x"], d["r"], gate=d["g"])
    for cut in (slice(0, k), slice(t - k, t)):          # the batch's ends, each by itself
        g = d["g"][cut].clone() if gate in ("token", "full") else d["g"]
        r2, n2 = op.forward(d["x"][cut].clone(), d["r"][cut].clone(), gate=g)
        assert torch.equal(r[cut], r2) and torch.equal(n[cut], n2)


def test_same_bits_again_on_another_stream_and_in_a_graph():
    h = 2048
    d = inputs(50, h, gate="channel")
    op = ResidualNorm(h, post_weight=d["post"], pre_weight=d["pre"])
    r, n = op.forward(d["x"], d["r"], gate=d["g"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r2, n2 = op.forward(d["x"], d["r"], gate=d["g"], stream=s)
    s.synchronize()
    assert torch.equal(r, r2) and torch.equal(n, n2)
    r3, n3 = torch.zeros_like(r), torch.zeros_like(n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(d["x"], d["r"], gate=d["g"], residual_out=r3, norm_out=n3)
    for seed in range(3):
        d["x"].copy_(inputs(50, h, seed=30 + seed)["x"])
        graph.replay()
        r4, n4 = op.forward(d["x"], d["r"], gate=d["g"])
        torch.cuda.synchronize()
        assert torch.equal(r3, r4) and torch.equal(n3, n4)


@pytest.mark.parametrize("h", [5, 256, 333, 8192, 16384])
@pytest.mark.parametrize("rd", [BF, F32])
def test_two_calls_give_the_bits_of_one_for_zeros_too(h, rd):
    """Zeros of either sign in the block's output and in the residual: without x
    the residual comes back as it is."""
    d = inputs(8, h, rd)
    d["x"][:4], d["x"][2] = -0.0, 0.0
    d["r"][::2], d["r"][1, ::2] = -0.0, 0.0
    whole = torch.int16 if rd == BF else torch.int32
    for scale in (1.0, -0.5):
        kw = dict(residual_dtype=rd, scale=scale)
        r, n = ResidualNorm(h, post_weight=d["post"], pre_weight=d["pre"], **kw).forward(d["x"], d["r"])
        r1, _ = ResidualNorm(h, post_weight=d["post"], **kw).forward(d["x"], d["r"])
        r2, n2 = ResidualNorm(h, pre_weight=d["pre"], **kw).forward(None, r1)
        torch.cuda.synchronize()
        assert torch.equal(r.view(whole), r1.view(whole)) and torch.equal(r.view(whole), r2.view(whole))
        assert torch.equal(n.view(torch.int16), n2.view(torch.int16))
    assert bool(torch.signbit(r).any())


@pytest.mark.parametrize("gd", [BF, F32])
def test_a_per_token_gate_begins_at_any_of_its_elements(gd):
    """Tokens from the second on: also where a row is one value, so that a factor
    per token and a factor per value have the same shape."""
    for h in (1, 8, 77):
        d = inputs(9, h, gate="token", gd=gd)
        check(8, h, dict(d, x=d["x"][1:].clone(), r=d["r"][1:].clone(), g=d["g"][1:]))


@pytest.mark.parametrize("h,t0", [(2048, 3), (1023, 8), (77, 16), (8, 1), (16392, 2)])
@pytest.mark.parametrize("rd", [BF, F32])
def test_rows_from_the_middle_of_larger_arrays(h, t0, rd):
    """Rows that begin and end inside larger arrays: as from arrays of their own,
    and what lies around the outputs stays."""
    d, t = inputs(40, h, rd, gate="full", seed=h), 13
    cut = slice(t0, t0 + t)
    own = {n: (v[cut].clone() if n in ("x", "r", "g") else v) for n, v in d.items()}
    r, n = check(t, h, own, rd=rd, scale=0.5)
    op = ResidualNorm(h, post_weight=d["post"], pre_weight=d["pre"], residual_dtype=rd, scale=0.5)
    ro = torch.full((40, h), 7.0, dtype=rd, device="cuda")
    no = torch.full((40, h), 7.0, dtype=BF, device="cuda")
    op.forward(d["x"][cut], d["r"][cut], gate=d["g"][cut], residual_out=ro[cut], norm_out=no[cut])
    torch.cuda.synchronize()
    assert torch.equal(ro[cut], r) and torch.equal(no[cut], n)
    for a in (ro, no):
        assert bool((a[:t0] == 7.0).all()) and bool((a[t0 + t:] == 7.0).all())
