"""The expert layer under a gate on the GPU: routing and outputs against the
float64 oracle, in every weight format and activation kind, and the block of
norm, router, gate, experts, shared expert and norm as it is used."""
import numpy as np
import pytest
import torch

from oracle import gate as ogate
from oracle import moe as omoe
from oracle import norm as onorm
from gpu_helpers import ATOL_MAX, RTOL_L2, GpuLayer, random_layer
from weight_quantized_moe_amd import Gate, MoeQuantError, ResidualNorm, router_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


FORMATS = ["int4_g128", "fp8_b128", "nvfp4_g16"]
BF = torch.bfloat16


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def oracle_layer(lay, ids, w, x_bits):
    """The oracle's permute, expert loop and combine under given ids and weights."""
    from oracle import formats
    perm = omoe.permute(ids, lay.layer.num_experts)
    x = omoe.bf16_bits_to_f64(x_bits)
    out = np.empty((ids.size, lay.layer.hidden))
    for e in range(lay.layer.num_experts):
        lo, hi = perm.offsets[e], perm.offsets[e + 1]
        if hi > lo:
            out[lo:hi] = omoe.expert_mlp(x[perm.sorted_token_ids[lo:hi]], formats.dequantize_expert(lay.p13, e),
                                         formats.dequantize_expert(lay.p2, e))
    return omoe.combine(perm, w, out), perm


def make(t, e, h, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    return dict(lg=1.5 * rn(t, e) + 0.5 * rn(e), x=rn(t, h).to(BF), r=rn(t, h).to(BF), bias=0.1 * rn(e))


def probe_for(t, lay):
    k, e = lay.top_k, lay.layer.num_experts
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(topk_ids=torch.empty((t, k), **i32), topk_w=torch.empty((t, k), device="cuda"),
                expert_offsets=torch.empty(e + 1, **i32), sorted_token_ids=torch.empty(t * k, **i32),
                inv_pos=torch.empty(t * k, **i32))


def check(lay, gate, kw, d, residual=True, router_w=None, **call):
    """Ids and grouping equal the oracle's, the output to the layer's tolerance
    (relative to the size of the weights' sum)."""
    t = d["x"].shape[0]
    pr, lg = probe_for(t, lay), d["lg"]
    more = dict(logits=lg)
    if router_w is not None:
        lg = torch.empty((t, gate.num_experts), device="cuda")
        more = dict(router_w=router_w, logits_out=lg)
    out = lay.layer.forward_gated(gate, d["x"], residual=d["r"] if residual else None, probe=pr, **more, **call)
    torch.cuda.synchronize()
    ids, w = ogate.gate(f64(lg), lay.top_k, bias=None if gate.bias is None else f64(gate.bias), **kw)
    assert np.array_equal(pr["topk_ids"].cpu().numpy(), ids)
    assert np.allclose(f64(pr["topk_w"]), w, rtol=1e-5, atol=1e-30)
    y, perm = oracle_layer(lay, ids, w, bits(d["x"]))
    for name in ("sorted_token_ids", "inv_pos"):
        assert np.array_equal(pr[name].cpu().numpy(), getattr(perm, name)), name
    assert np.array_equal(pr["expert_offsets"].cpu().numpy(), perm.offsets)
    if residual:
        y = y + f64(d["r"])
    got, big = f64(out), max(1.0, np.abs(w).sum(1).max())
    rel = np.linalg.norm(got - y) / max(np.linalg.norm(y), 1e-300)
    assert rel <= RTOL_L2 and np.abs(got - y).max() <= ATOL_MAX * big, (rel, np.abs(got - y).max())
    return out


GROUPED = dict(score="sigmoid", groups=4, topk_groups=2, group_top=2, scale=2.5)


def gate_of(e, k, bias=None, **kw):
    return Gate(e, k, bias=bias, **{("num_groups" if n == "groups" else n): v for n, v in kw.items()})


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", [1, 2, 3, 16, 17, 61, 300])
@pytest.mark.parametrize("residual", [False, True])
def test_layer(fmt, t, residual):
    lay = GpuLayer(*random_layer(fmt, 3, 16, 256, 128), 4)
    d = make(t, 16, 256, seed=t)
    check(lay, gate_of(16, 4, d["bias"], **GROUPED), GROUPED, d, residual)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", [1, 40])
def test_long_rows(fmt, t):
    """Hidden rows longer than the routing stage keeps in registers."""
    lay = GpuLayer(*random_layer(fmt, 5, 8, 2304, 128), 2)
    kw = dict(score="softmax", renormalize=False)
    d = make(t, 8, 2304, seed=t)
    check(lay, gate_of(8, 2, **kw), kw, d)


@pytest.mark.parametrize("t", [1, 5, 33, 4100])
def test_from_the_router_weight(t):
    """In-library logits, at every routing size; the gate is checked on the logits it
    decided on."""
    lay = GpuLayer(*random_layer("int4_g128", 3, 16, 256, 128), 4)
    d = make(t, 16, 256, seed=t)
    w = (0.1 * torch.randn(16, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))).to(BF)
    check(lay, gate_of(16, 4, d["bias"], **GROUPED), GROUPED, d, router_w=w)
    # without logits_out the same logits are used
    a = lay.layer.forward_gated(gate_of(16, 4, d["bias"], **GROUPED), d["x"], router_w=w)
    b = lay.layer.forward_gated(gate_of(16, 4, d["bias"], **GROUPED), d["x"], logits=router_logits(d["x"], w))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_more_experts_than_the_fused_router_holds():
    lay = GpuLayer(*random_layer("fp8_b128", 3, 300, 128, 128), 3)
    d = make(20, 300, 128)
    w = (0.1 * torch.randn(300, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))).to(BF)
    check(lay, gate_of(300, 3, d["bias"], score="sigmoid"), dict(score="sigmoid"), d, router_w=w)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t", [1, 2, 16, 65, 300])
def test_the_default_gate_is_the_layers_own_routing(fmt, t):
    lay = GpuLayer(*random_layer(fmt, 7, 16, 256, 128), 4)
    d = make(t, 16, 256, seed=t)
    pr, pg = probe_for(t, lay), probe_for(t, lay)
    a = lay.layer.forward(d["lg"], d["x"], residual=d["r"], probe=pr)
    b = lay.layer.forward_gated(Gate(16, 4), d["x"], logits=d["lg"], residual=d["r"], probe=pg)
    torch.cuda.synchronize()
    for n in ("topk_ids", "expert_offsets", "sorted_token_ids", "inv_pos"):
        assert torch.equal(pr[n], pg[n]), n
    assert np.allclose(f64(pr["topk_w"]), f64(pg["topk_w"]), rtol=2e-6)
    assert np.linalg.norm(f64(a) - f64(b)) <= RTOL_L2 * np.linalg.norm(f64(a))


@pytest.mark.parametrize("t", [1, 2, 50])
def test_weights_of_any_size_keep_their_digits(t):
    """Weights far below what FP16 holds: the output is the scaled output."""
    lay = GpuLayer(*random_layer("int4_g128", 7, 16, 256, 128), 4)
    d = make(t, 16, 256, seed=t)
    kw = dict(score="sigmoid", scale=2.0 ** -40)
    check(lay, gate_of(16, 4, **kw), kw, d, residual=False)
    kw = dict(score="sigmoid", renormalize=False)
    far = dict(d, lg=d["lg"] - 40.0)
    check(lay, gate_of(16, 4, **kw), kw, far, residual=False)


@pytest.mark.parametrize("t", [3, 12, 40])
def test_saturates_no_earlier_than_the_layers_own_routing(t):
    """Expert outputs between 131000 and 262000 times weights of a quarter fit FP16.
    The outputs are linear in the down projection's scales, so a power of two on
    those sets their size."""
    p13, p2 = random_layer("fp8_b128", 7, 16, 256, 128)
    d = make(t, 16, 256, seed=t)
    d["lg"] = torch.zeros_like(d["lg"])
    lay = GpuLayer(p13, p2, 4)
    alone = [oracle_layer(lay, np.full((t, 1), e, np.int32), np.ones((t, 1)), bits(d["x"]))[0] for e in range(4)]
    p2.scale[:] = p2.scale * 2.0 ** np.floor(np.log2(262000 / np.abs(alone).max()))
    lay = GpuLayer(p13, p2, 4)
    ws = lay.layer.workspace(t)
    a = lay.layer.forward(d["lg"], d["x"], workspace=ws)
    assert not lay.layer.check(ws)
    b = lay.layer.forward_gated(Gate(16, 4), d["x"], logits=d["lg"], workspace=ws)
    assert not lay.layer.check(ws)
    assert torch.equal(a, b)          # weights of exactly a quarter in both


def test_masked_rows():
    """A row without live experts gives the residual, and rows with few take
    their live experts alone."""
    lay = GpuLayer(*random_layer("nvfp4_g16", 7, 16, 256, 128), 4)
    for t in (2, 12, 100):
        d = make(t, 16, 256, seed=t)
        d["lg"][0] = -float("inf")
        d["lg"][1, 3:] = -float("inf")
        for kw in (GROUPED, dict(score="softmax")):
            out = check(lay, gate_of(16, 4, **kw), kw, d)
            assert torch.equal(out[0], d["r"][0])


@pytest.mark.parametrize("t", [1, 20, 300])
def test_fp8_and_nvfp4_activations(t):
    """The gate in front of the W8A8 and W4A4 paths: with the default gate they
    give what forward_w8a8 and forward_w4a4 give."""
    d = make(t, 16, 256, seed=t)
    lay = GpuLayer(*random_layer("fp8_b128", 7, 16, 256, 128), 4)
    a = lay.layer.forward_w8a8(d["lg"], d["x"], residual=d["r"])
    b = lay.layer.forward_gated(Gate(16, 4), d["x"], logits=d["lg"], residual=d["r"], activations="fp8")
    lay4 = GpuLayer(*random_layer("nvfp4_g16", 7, 16, 256, 128), 4)
    c = lay4.layer.forward_w4a4(d["lg"], d["x"], 300.0, 900.0, residual=d["r"])
    e = lay4.layer.forward_gated(Gate(16, 4), d["x"], logits=d["lg"], residual=d["r"], activations="nvfp4",
                                 act_gscale13=300.0, act_gscale2=900.0)
    torch.cuda.synchronize()
    for p, q in ((a, b), (c, e)):
        assert np.linalg.norm(f64(p) - f64(q)) <= RTOL_L2 * np.linalg.norm(f64(p))


def test_refusals_and_no_tokens():
    lay = GpuLayer(*random_layer("int4_g128", 7, 16, 256, 128), 4)
    d = make(3, 16, 256)
    with pytest.raises(MoeQuantError, match="picks 2 of 16"):
        lay.layer.forward_gated(Gate(16, 2), d["x"], logits=d["lg"])
    with pytest.raises(ValueError, match="workspace"):
        lay.layer.forward_gated(Gate(16, 4), d["x"], logits=d["lg"], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    out = lay.layer.forward_gated(Gate(16, 4), d["x"][:0], logits=d["lg"][:0])
    assert out.shape == (0, 256)


@pytest.mark.parametrize("t", [1, 9, 200])
def test_two_streams_and_graph_replays(t):
    """Calls on two streams with workspaces of their own, and a captured call
    replayed with other inputs between eager ones on another workspace."""
    lay = GpuLayer(*random_layer("fp8_b128", 7, 16, 256, 128), 4)
    d = make(t, 16, 256, seed=t)
    gate = gate_of(16, 4, d["bias"], **GROUPED)
    ref = lay.layer.forward_gated(gate, d["x"], logits=d["lg"])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [lay.layer.forward_gated(gate, d["x"], logits=d["lg"], stream=s) for s in (s1, s2, s1)]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in outs)
    lg, out, ws = d["lg"].clone(), torch.zeros_like(d["x"]), lay.layer.workspace(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.layer.forward_gated(gate, d["x"], logits=lg, out=out, workspace=ws)
    for r in range(3):
        lg.copy_(make(t, 16, 256, seed=50 + r)["lg"])
        graph.replay()
        eager = lay.layer.forward_gated(gate, d["x"], logits=lg)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("t", [1, 7, 150])
def test_a_block_as_it_is_used(t):
    """norm -> router -> gated experts + shared expert -> norm after the block, gated
    and scaled onto the residual stream -> norm before the next block."""
    e, k, h, i = 16, 4, 256, 128
    lay = GpuLayer(*random_layer("int4_g128", 11, e, h, i), k)
    shared = GpuLayer(*random_layer("fp8_b128", 12, 1, h, i), 1)
    d = make(t, e, h, seed=t)
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = lambda *s: (0.1 * torch.randn(*s, generator=gen, device="cuda")).to(BF)  # noqa: E731
    router, shared_router = w(e, h), w(1, h)
    norms = [1 + w(h).float() for _ in range(3)]
    channel = 1 + w(h).float()
    stream = d["r"].float()
    before = ResidualNorm(h, pre_weight=norms[0], residual_dtype=torch.float32)
    after = ResidualNorm(h, post_weight=norms[1], pre_weight=norms[2], residual_dtype=torch.float32, scale=0.5)
    gate, sgate = gate_of(e, k, d["bias"], **GROUPED), Gate(1, 1, score="sigmoid", renormalize=False)
    stream1, x = before.forward(d["x"], stream)
    y_s = shared.layer.forward_gated(sgate, x, router_w=shared_router)
    y = lay.layer.forward_gated(gate, x, router_w=router, residual=y_s)
    stream2, nxt = after.forward(y, stream1, gate=channel)
    torch.cuda.synchronize()
    # each step against the oracle on the values that the step before it gave
    assert np.allclose(f64(stream1), f64(stream) + f64(d["x"]), rtol=2.0 ** -24, atol=1e-12)
    ref = onorm.rms_norm(f64(stream1), f64(norms[0]), 1e-6, 0.0)
    assert np.all(np.abs(f64(x) - ref) <= (2.0 ** -8 + 1e-5) * np.abs(ref))
    lg = f64(router_logits(x, router))
    ids, wt = ogate.gate(lg, k, bias=f64(d["bias"]), **GROUPED)
    ref, _ = oracle_layer(lay, ids, wt, bits(x))
    sl = f64(router_logits(x, shared_router))
    sref, _ = oracle_layer(shared, np.zeros((t, 1), np.int32), 1 / (1 + np.exp(-sl)), bits(x))
    for got, want in ((y_s, sref), (y, ref + f64(y_s))):
        assert np.linalg.norm(f64(got) - want) <= RTOL_L2 * np.linalg.norm(want)
    r, add = onorm.residual_update(f64(y), f64(stream1), f64(channel), f64(norms[1]), scale=0.5)
    assert np.allclose(f64(stream2), r + add, rtol=0, atol=2e-5 * np.abs(r + add).max())
    ref = onorm.rms_norm(f64(stream2), f64(norms[2]), 1e-6, 0.0)
    assert np.all(np.abs(f64(nxt) - ref) <= (2.0 ** -8 + 1e-5) * np.abs(ref))


@pytest.mark.parametrize("t", [1, 16, 17, 300])
def test_a_block_in_a_graph(t):
    """The whole block captured, and replayed on other inputs between eager runs
    of it on buffers of their own."""
    e, k, h, i = 16, 4, 256, 128
    lay = GpuLayer(*random_layer("nvfp4_g16", 11, e, h, i), k)
    d = make(t, e, h, seed=t)
    router = (0.1 * torch.randn(e, h, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))).to(BF)
    w = torch.ones(h, device="cuda")
    before = ResidualNorm(h, pre_weight=w, residual_dtype=torch.float32)
    after = ResidualNorm(h, post_weight=w, pre_weight=w, residual_dtype=torch.float32, scale=0.5)
    gate = gate_of(e, k, d["bias"], **GROUPED)

    def block(x, stream):
        s1, n = before.forward(x, stream)
        y = lay.layer.forward_gated(gate, n, router_w=router)
        return after.forward(y, s1)

    x, stream = d["x"].clone(), d["r"].float()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        block(x, stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, nxt = block(x, stream)
    for r in range(3):
        x.copy_(make(t, e, h, seed=70 + r)["x"])
        graph.replay()
        eager_out, eager_nxt = block(x, stream)
        torch.cuda.synchronize()
        assert torch.equal(out, eager_out) and torch.equal(nxt, eager_nxt)


def test_two_threads():
    """Host threads with streams and workspaces of their own on one layer and gate."""
    import threading
    lay = GpuLayer(*random_layer("int4_g128", 7, 16, 256, 128), 4)
    gate = Gate(16, 4, score="sigmoid")
    cases = [make(t, 16, 256, seed=t) for t in (5, 40)]
    ref = [lay.layer.forward_gated(gate, d["x"], logits=d["lg"]) for d in cases]
    ids = [gate.topk(d["lg"])[0] for d in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        d, s = cases[n], torch.cuda.Stream()
        ws = lay.layer.workspace(d["x"].shape[0])
        for _ in range(50):
            out = lay.layer.forward_gated(gate, d["x"], logits=d["lg"], workspace=ws, stream=s)
            got, _ = gate.topk(d["lg"], stream=s)
            s.synchronize()
            if not (torch.equal(out, ref[n]) and torch.equal(got, ids[n])):
                wrong.append(n)

    threads = [threading.Thread(target=work, args=(n,)) for n in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


@pytest.mark.parametrize("t", [1, 3, 17, 300])
def test_the_workspace_is_all_it_takes(t):
    """A workspace of exactly the stated size between bytes that stay as they were."""
    lay = GpuLayer(*random_layer("fp8_b128", 7, 16, 256, 128), 4)
    d = make(t, 16, 256, seed=t)
    gate, n = gate_of(16, 4, d["bias"], **GROUPED), lay.layer.workspace_size(t)
    around = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    for call in (lambda **kw: lay.layer.forward_gated(gate, d["x"], logits=d["lg"], **kw),
                 lambda **kw: lay.layer.forward(d["lg"], d["x"], **kw)):
        out, ref = call(workspace=around[4096:4096 + n]), call()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and bool((around[:4096] == 0xA5).all()) and bool((around[4096 + n:] == 0xA5).all())


@pytest.mark.parametrize("e", [2, 63, 64, 65, 300, 511, 512])
@pytest.mark.parametrize("t,k", [(1, 2), (3, 2), (16, 1), (13, 4), (16, 4), (8, 8)])
def test_few_slots_and_any_number_of_experts(e, t, k):
    """Up to 64 slots are grouped beside the gate: tables of E + 1 entries, whose
    last pass over the experts a workgroup takes with few lanes or one."""
    k = min(k, e)
    lay = GpuLayer(*random_layer("nvfp4_g16", 9, e, 128, 128), k)
    d = make(t, e, 128, seed=t + e)
    check(lay, gate_of(e, k, d["bias"], score="sigmoid"), dict(score="sigmoid"), d)


SIGMOID8 = dict(score="sigmoid", groups=8, topk_groups=4, group_top=2, scale=2.5)


@pytest.mark.parametrize("t", [9, 16, 61])
@pytest.mark.parametrize("e,k,kw", [
    (64, 8, dict(score="sigmoid")), (64, 8, SIGMOID8), (128, 8, dict(score="softmax")), (128, 8, SIGMOID8),
    (192, 8, SIGMOID8), (256, 8, dict(score="sigmoid", renormalize=False)), (256, 8, SIGMOID8),
    (384, 8, dict(score="softmax", groups=16, topk_groups=7)), (380, 9, dict(score="softmax", renormalize=False)),
    (512, 8, dict(score="sigmoid")), (512, 16, SIGMOID8),
    (48, 6, dict(score="sigmoid", groups=3, topk_groups=2, group_top=2)),      # no number of groups for four tokens a wave
    (48, 17, dict(score="softmax")), (512, 33, dict(score="sigmoid", groups=32, topk_groups=9, scale=0.25)),
    (96, 64, dict(score="softmax", scale=16.0)),
])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_every_gate_in_front_of_the_experts(t, e, k, kw, dtype):
    """The gate's variants beside the grouping (up to 16 tokens, with more than 64
    slots) and beside the rows' staging."""
    lay = GpuLayer(*random_layer("int4_g128", 9, e, 128, 128), k)
    d = make(t, e, 128, seed=t + e)
    d["lg"] = d["lg"].to(dtype)
    bias = d["bias"] if kw["score"] == "sigmoid" or k == 9 else None
    check(lay, gate_of(e, k, bias, **kw), kw, d)


def check_activations(lay, kw, d, bias, g13=None, g2=None):
    """W8A8, or with global scales W4A4: the intermediate's values against the
    oracle's before it rounds them, and the output against the oracle's from the
    intermediate that came back, to the layer's tolerance.  The output is not held
    to the oracle's own intermediate: a step of E4M3 is up to 2^-3 of the value, so
    where one slot has nearly all of a token's weight the 1 in 100 of its values that
    may differ by a step move the output by up to 2^-3 sqrt(1 / 100) = 1.3e-2, more
    than the layer's tolerance.  E4M3: half a step, 2^-4 of the value or of the least
    normal number 2^-6, and 0.05 (twice 448 times the 5e-5 that the FP8 matrix unit's
    sums are off by).  E2M1: 1 in 100 of n values may differ, a spread of
    sqrt(n / 100), 5 of which are allowed for."""
    from oracle import codecs, formats, w4a4, w8a8
    t, k, i = d["x"].shape[0], lay.top_k, lay.layer.inter
    pr = dict(probe_for(t, lay), h=torch.empty((t * k, i), dtype=torch.float16, device="cuda"))
    act = dict(activations="fp8") if g13 is None else dict(activations="nvfp4", act_gscale13=g13, act_gscale2=g2)
    gate, ws = gate_of(lay.layer.num_experts, k, bias, **kw), lay.layer.workspace(t)
    out = lay.layer.forward_gated(gate, d["x"], logits=d["lg"], probe=pr, workspace=ws, **act)
    torch.cuda.synchronize()
    assert not lay.layer.check(ws)
    ids, w = ogate.gate(f64(d["lg"]), k, bias=None if bias is None else f64(bias), **kw)
    assert np.array_equal(pr["topk_ids"].cpu().numpy(), ids)
    assert np.allclose(f64(pr["topk_w"]), w, rtol=1e-5, atol=1e-30)
    perm = omoe.permute(ids, lay.layer.num_experts)
    assert np.array_equal(pr["inv_pos"].cpu().numpy(), perm.inv_pos)
    x = f64(d["x"])
    if g13 is None:
        hb = pr["h"].cpu().numpy().view(np.uint8).reshape(-1)
        n = t * k * i
        codes, scales = hb[:n].reshape(t * k, i), hb[n:n + n // 32].view(np.float32).reshape(t * k, i // 128)
        h = w8a8.dequantize_act(codes, scales)
        xq = w8a8.dequantize_act(*w8a8.quantize_act(x))
    else:
        h = f64(pr["h"]) / np.float64(np.float32(g2))
        xq = w4a4.quantize_dequantize(x, g13)
    forced, h32 = np.empty((t * k, lay.layer.hidden)), np.empty((t * k, i), np.float32)
    for e in range(lay.layer.num_experts):
        lo, hi = perm.offsets[e], perm.offsets[e + 1]
        if hi > lo:
            w13, w2 = formats.dequantize_expert(lay.p13, e), formats.dequantize_expert(lay.p2, e)
            forced[lo:hi] = h[lo:hi] @ w2.T
            gu = xq[perm.sorted_token_ids[lo:hi]] @ w13.T
            h32[lo:hi] = omoe.silu(gu[:, :i]) * gu[:, i:]
    if g13 is None:
        ref = w8a8.quantize_act(h32)[1]
        assert np.allclose(scales, ref, rtol=2.0 ** -12, atol=0)
        q = h32 / np.repeat(ref, 128, axis=1)
        off = np.abs(codecs.decode_e4m3(codes) - q) - 2.0 ** -4 * np.maximum(np.abs(q), 2.0 ** -6)
        assert off.max() <= 0.05, off.max()
    else:
        differ = (np.abs(h - w4a4.quantize_dequantize(h32, g2)) > 1e-6 * np.abs(h)).sum()
        assert differ <= h.size / 100 + 5 * np.sqrt(h.size / 100), (differ, h.size)
    y = omoe.combine(perm, w, forced)
    rel = np.linalg.norm(f64(out) - y) / np.linalg.norm(y)
    assert rel <= RTOL_L2, rel


WEIGHTS = {
    "above one": (GROUPED, 0.0), "far above one": (dict(GROUPED, scale=300.0), 0.0),
    "small": (dict(score="sigmoid", scale=2.0 ** -40), 0.0),
    "raw and small": (dict(score="sigmoid", renormalize=False), -40.0),
    "raw softmax": (dict(score="softmax", renormalize=False, scale=2.0 ** -9), 0.0),
}


@pytest.mark.parametrize("t", [1, 9, 40, 300])
@pytest.mark.parametrize("weights", list(WEIGHTS))
def test_fp8_and_nvfp4_activations_under_weights_of_any_size(t, weights):
    """Groups, sigmoids and biases in front of the W8A8 and W4A4 paths, with weights
    that a power of two is taken out of."""
    from oracle import w4a4
    kw, shift = WEIGHTS[weights]
    d = make(t, 16, 256, seed=t)
    d["lg"] = d["lg"] + shift
    bias = d["bias"] if kw["score"] == "sigmoid" and shift == 0.0 else None
    check_activations(GpuLayer(*random_layer("fp8_b128", 7, 16, 256, 128), 4), kw, d, bias)
    lay = GpuLayer(*random_layer("nvfp4_g16", 7, 16, 256, 128), 4)
    g13 = 448 * 6 / float(d["x"].float().abs().max())
    g2 = 448 * 6 / float(np.abs(w4a4.intermediate_w4a4(lay.oracle, f64(d["lg"]), bits(d["x"]), g13)).max())
    check_activations(lay, kw, d, bias, g13, g2)


@pytest.mark.parametrize("t", [3, 12, 40, 300])
@pytest.mark.parametrize("scale", [2.5, 2.0 ** -40])
def test_scaled_rows_saturate_where_a_power_of_two_says(t, scale):
    """Renormalised weights of a quarter times a scale: above 1 or far below 2^-7
    their largest is brought to [1/2, 1), so expert outputs of up to 65504 fit and
    twice that times 5/8 does not."""
    p13, p2 = random_layer("fp8_b128", 7, 16, 256, 128)
    d = make(t, 16, 256, seed=t)
    d["lg"] = torch.zeros_like(d["lg"])
    lay = GpuLayer(p13, p2, 4)
    alone = [oracle_layer(lay, np.full((t, 1), e, np.int32), np.ones((t, 1)), bits(d["x"]))[0] for e in range(4)]
    kw, big = dict(score="softmax", scale=4 * scale), np.abs(alone).max()
    scales = p2.scale.copy()
    w = scale * 2.0 ** -np.floor(np.log2(scale) + 1)            # the weight without its power of two
    for factor, saturated in ((0.95 * 65504 / w / big, False), (1.1 * 65504 / w / big, True)):
        p2.scale[:] = scales * factor
        lay = GpuLayer(p13, p2, 4)
        ws = lay.layer.workspace(t)
        out = lay.layer.forward_gated(gate_of(16, 4, **kw), d["x"], logits=d["lg"], workspace=ws)
        assert lay.layer.check(ws) == saturated
        if not saturated:
            ids, wt = ogate.gate(f64(d["lg"]), 4, **kw)
            y, _ = oracle_layer(lay, ids, wt, bits(d["x"]))
            assert np.linalg.norm(f64(out) - y) <= RTOL_L2 * np.linalg.norm(y)
