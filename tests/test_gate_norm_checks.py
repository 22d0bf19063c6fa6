"""The gate's and the norm's argument checks, and their oracles (runs without a
GPU: every call here is refused or has no tokens)."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import gate as ogate
from oracle import moe as omoe
from oracle import norm as onorm
from weight_quantized_moe_amd import Gate, Layer, MoeQuantError, ResidualNorm, binding, build
from weight_quantized_moe_amd.binding import GateDesc, LayerDesc, NormDesc

OK, NULL, SHAPE, ALIGN, FORMAT, DTYPE, WORKSPACE, ABI = range(8)
P = 0x10000            # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        pytest.fail("libmoe_quant.so is not built (run __graft_entry__.build())")
    return binding.load_library()


@pytest.mark.timeout(900)
def test_checks_under_address_sanitizer():
    """This file again, with AddressSanitizer on the library's host code."""
    if os.environ.get("MOE_QUANT_LIB"):
        pytest.skip("runs on another library already")
    from test_abi_asan import _stale
    try:
        runtime = build.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    if _stale(build.ASAN_LIB):
        build.build_asan()
    env = dict(os.environ, MOE_QUANT_LIB=build.ASAN_LIB, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                         env=env, capture_output=True, text=True, timeout=600)
    tail = (res.stdout + res.stderr)[-3000:]
    assert res.returncode == 0 and "AddressSanitizer" not in res.stderr, tail


def test_struct_layouts_match_header():
    assert ctypes.sizeof(GateDesc) == 9 * 4 + 4 + 8 and GateDesc.bias.offset == 40
    assert ctypes.sizeof(NormDesc) == 7 * 4 + 4 + 16 and NormDesc.post_weight.offset == 32


def _gate(**over):
    f = dict(abi=1, e=16, k=4, score=1, groups=4, topk=2, top=2, renorm=1, scale=1.0, bias=None)
    f.update(over)
    return GateDesc(f["abi"], f["e"], f["k"], f["score"], f["groups"], f["topk"], f["top"], f["renorm"], f["scale"],
                    f["bias"])


@pytest.mark.parametrize("over,expect", [
    (dict(abi=2), ABI), (dict(e=0), SHAPE), (dict(e=513, groups=1, topk=1), SHAPE), (dict(k=0), SHAPE),
    (dict(k=9), SHAPE),                                   # two kept groups hold 8 experts
    (dict(e=512, groups=1, topk=1, k=65), SHAPE), (dict(score=2), SHAPE), (dict(score=-1), SHAPE),
    (dict(groups=0), SHAPE), (dict(groups=3), SHAPE), (dict(e=128, groups=128), SHAPE), (dict(topk=0), SHAPE),
    (dict(topk=5), SHAPE), (dict(top=0), SHAPE), (dict(top=3), SHAPE),
    (dict(groups=16, topk=4, top=2), SHAPE),              # groups of one expert have no second
    (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE), (dict(bias=P + 2), ALIGN),
])
def test_gate_refuses_bad_fields(lib, over, expect):
    assert lib.moe_quant_gate_topk(ctypes.byref(_gate(**over)), P, 0, 0, P, P, None) == expect
    assert lib.moe_quant_last_error()


def test_gate_accepts_limits(lib):
    for over in (dict(), dict(e=1, k=1, groups=1, topk=1, top=1), dict(e=512, k=64, groups=64, topk=64),
                 dict(groups=1, topk=1, top=2, k=16), dict(groups=16, topk=4, top=1), dict(scale=-2.0)):
        assert lib.moe_quant_gate_topk(ctypes.byref(_gate(**over)), None, 0, 0, None, None, None) == OK


@pytest.mark.parametrize("args,expect", [
    ((None, P, 0, 1, P, P), NULL), (("g", P, 2, 1, P, P), DTYPE), (("g", P, 0, -1, P, P), SHAPE),
    (("g", P, 0, (1 << 22) + 1, P, P), SHAPE), (("g", None, 0, 1, P, P), NULL), (("g", P, 0, 1, None, P), NULL),
    (("g", P, 0, 1, P, None), NULL), (("g", P + 4, 0, 1, P, P), ALIGN), (("g", P, 0, 1, P + 2, P), ALIGN),
    (("g", P, 0, 1, P, P + 1), ALIGN),
])
def test_gate_refuses_bad_arguments(lib, args, expect):
    g = None if args[0] is None else ctypes.byref(_gate())
    assert lib.moe_quant_gate_topk(g, *args[1:], None) == expect


def _layer(lib, fmt=1, e=16, k=4):
    g = P + 0x4000 if fmt == 3 else None
    d = LayerDesc(1, e, 256, 128, k, fmt, P, P + 0x1000, g, P + 0x2000, P + 0x3000, g)
    h = ctypes.c_void_p()
    assert lib.moe_quant_init(ctypes.byref(d), ctypes.byref(h)) == OK
    return h


@pytest.mark.parametrize("fmt,over,expect", [
    (1, dict(gate=None), NULL), (1, dict(gate=_gate(abi=3)), ABI), (1, dict(gate=_gate(e=8, groups=2)), SHAPE),
    (1, dict(gate=_gate(k=3)), SHAPE), (1, dict(logits=None), NULL), (1, dict(router=P), NULL),
    (1, dict(logits_out=P), NULL), (1, dict(act=3), FORMAT), (1, dict(act=1), FORMAT), (2, dict(act=2), FORMAT),
    (3, dict(act=2, g13=0.0), SHAPE), (3, dict(act=2, g2=math.inf), SHAPE), (1, dict(dtype=5), DTYPE),
    (1, dict(t=-1), SHAPE), (1, dict(hidden=None), NULL), (1, dict(out=P + 8), ALIGN), (1, dict(ws=None), WORKSPACE),
    (1, dict(ws_bytes=64), WORKSPACE), (1, dict(router=P + 8, logits=None), ALIGN),
])
def test_forward_gated_refuses(lib, fmt, over, expect):
    f = dict(gate=_gate(), logits=P, dtype=0, router=None, hidden=P, residual=None, t=4, out=P, ws=P, ws_bytes=1 << 30,
             act=0, g13=1.0, g2=1.0, logits_out=None)
    f.update(over)
    h = _layer(lib, fmt)
    st = lib.moe_quant_forward_gated(h, None if f["gate"] is None else ctypes.byref(f["gate"]), f["logits"], f["dtype"],
                                     f["router"], f["hidden"], f["residual"], f["t"], f["out"], f["ws"], f["ws_bytes"],
                                     f["act"], f["g13"], f["g2"], f["logits_out"], None, None)
    lib.moe_quant_destroy(h)
    assert st == expect, lib.moe_quant_last_error()


def _norm(**over):
    f = dict(abi=1, h=64, rd=1, wd=1, eps=1e-6, off=0.0, scale=1.0, post=P, pre=P)
    f.update(over)
    return NormDesc(f["abi"], f["h"], f["rd"], f["wd"], f["eps"], f["off"], f["scale"], f["post"], f["pre"])


@pytest.mark.parametrize("over,args,expect", [
    (dict(abi=0), {}, ABI), (dict(h=0), {}, SHAPE), (dict(h=32769), {}, SHAPE), (dict(rd=2), {}, DTYPE),
    (dict(wd=-1), {}, DTYPE), (dict(eps=0.0), {}, SHAPE), (dict(eps=1e-31), {}, SHAPE), (dict(eps=-1.0), {}, SHAPE), (dict(eps=math.nan), {}, SHAPE),
    (dict(off=math.inf), {}, SHAPE), (dict(scale=math.nan), {}, SHAPE), ({}, dict(kind=4, gate=P), SHAPE),
    ({}, dict(kind=-1), SHAPE), ({}, dict(kind=1, gate=P, gd=7), DTYPE), ({}, dict(t=-1), SHAPE),
    ({}, dict(t=(1 << 22) + 1), SHAPE), ({}, dict(gate=P), NULL), ({}, dict(kind=2), NULL), ({}, dict(x=None), NULL),
    (dict(post=None), dict(x=None, gate=P, kind=1), NULL), (dict(post=None), dict(x=None, r=None), NULL),
    (dict(pre=None), {}, NULL), ({}, dict(n=None), NULL), (dict(pre=None), dict(n=None, ro=None), NULL),
    ({}, dict(x=P + 2), ALIGN), ({}, dict(r=P + 8), ALIGN), ({}, dict(ro=P + 8), ALIGN), ({}, dict(n=P + 4), ALIGN),
    (dict(post=P + 2), {}, ALIGN), (dict(pre=P + 8), {}, ALIGN), ({}, dict(gate=P + 8, kind=1), ALIGN),
    ({}, dict(gate=P + 2, kind=2, gd=0), ALIGN),
])
def test_norm_refuses(lib, over, args, expect):
    a = dict(x=P, r=P, gate=None, kind=0, gd=1, t=4, ro=P, n=P)
    a.update(args)
    d = _norm(**over)
    assert lib.moe_quant_norm(ctypes.byref(d), a["x"], a["r"], a["gate"], a["kind"], a["gd"], a["t"], a["ro"], a["n"],
                              None) == expect, lib.moe_quant_last_error()
    assert lib.moe_quant_norm(None, P, P, None, 0, 0, 4, P, P, None) == NULL


def test_binding_gate_checks():
    with pytest.raises(ValueError, match="score"):
        Gate(8, 2, score="tanh")
    with pytest.raises(MoeQuantError) as ei:
        Gate(8, 2, num_groups=3)
    assert ei.value.status == SHAPE
    with pytest.raises(ValueError, match="shape"):
        Gate(8, 2, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="dtype"):
        Gate(8, 2, bias=torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU tensor"):
        Gate(8, 2, bias=torch.zeros(8))
    g = Gate(8, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.topk(torch.zeros(3, 8))
    for bad in (torch.zeros(3, 9), torch.zeros(3, 8, dtype=torch.float16), torch.zeros(8, 3).t(), torch.zeros(8)):
        with pytest.raises(ValueError) as ei:
            g.topk(bad)
        assert "GPU tensor" not in str(ei.value)
    with pytest.raises(ValueError, match="shape"):
        g.topk(torch.zeros(3, 8), ids=torch.zeros(3, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="dtype"):
        g.topk(torch.zeros(3, 8), weights=torch.zeros(3, 2, dtype=torch.bfloat16))


def test_binding_forward_gated_checks():
    lay = Layer.__new__(Layer)                 # a layer object without a device handle
    lay._lib, lay._h = binding.load_library(), None
    lay.fmt, lay.num_experts, lay.hidden, lay.inter, lay.top_k = "int4_g128", 8, 256, 128, 2
    lay.device, lay.workspace_size = torch.device("cpu"), lambda t: 256
    g, x = Gate(8, 2), torch.zeros(3, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        lay.forward_gated(g, x, logits=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="exactly one"):
        lay.forward_gated(g, x)
    with pytest.raises(ValueError, match="exactly one"):
        lay.forward_gated(g, x, logits=torch.zeros(3, 8), router_w=torch.zeros(8, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="activations"):
        lay.forward_gated(g, x, logits=torch.zeros(3, 8), activations="int8")
    with pytest.raises(ValueError, match="logits_out"):
        lay.forward_gated(g, x, logits=torch.zeros(3, 8), logits_out=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="shape"):
        lay.forward_gated(g, x, logits=torch.zeros(4, 8))


def test_binding_norm_checks():
    w = torch.ones(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="residual_dtype"):
        ResidualNorm(8, residual_dtype=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        ResidualNorm(9, pre_weight=w)
    with pytest.raises(ValueError, match="one dtype"):
        ResidualNorm(8, post_weight=w, pre_weight=w.float())
    with pytest.raises(ValueError, match="GPU tensor"):
        ResidualNorm(8, pre_weight=w)
    with pytest.raises(MoeQuantError):
        ResidualNorm(8, eps=0.0)
    n = ResidualNorm(8)
    x, r = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        n.forward(x, r)
    with pytest.raises(ValueError, match="need x"):
        n.forward()
    for kw in (dict(x=x.float()), dict(x=x[:, :7]), dict(residual=r.float()), dict(residual=r[:2]),
               dict(gate=torch.zeros(3)), dict(gate=torch.zeros(8, dtype=torch.float16)), dict(gate=torch.zeros(2, 1)),
               dict(norm_out=x), dict(residual_out=r.float()), dict(x=torch.zeros(8, 3, dtype=torch.bfloat16).t())):
        with pytest.raises(ValueError) as ei:
            n.forward(**{**dict(x=x, residual=r), **kw})
        assert "GPU tensor" not in str(ei.value), kw


# ---- the oracles against closed forms and the routing oracle
def test_gate_oracle_is_the_softmax_routing_by_default():
    lg = np.random.default_rng(0).normal(size=(50, 24))
    lg[3, :] = 0.5                                     # all tied
    ids, w = ogate.gate(lg, 5)
    ref_ids, ref_w = omoe.route(lg, 5)
    assert np.array_equal(ids, ref_ids) and np.allclose(w, ref_w, rtol=1e-13)


def test_gate_oracle_by_hand():
    # two groups of three; group sums of two: 0.9 + 0.1 against 0.6 + 0.5
    s = np.array([[0.9, 0.1, 0.05, 0.6, 0.5, 0.2]])
    lg = np.log(s / (1 - s))
    ids, w = ogate.gate(lg, 2, "sigmoid", groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[3, 4]] and np.allclose(w, [[6 / 11, 5 / 11]])
    ids, w = ogate.gate(lg, 2, "sigmoid", groups=2, topk_groups=1, renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1.8, 0.2]])
    # the bias decides the choice and stays out of the weight
    ids, w = ogate.gate(lg, 1, "sigmoid", bias=[0, 0, 1.0, 0, 0, 0], renormalize=False)
    assert ids.tolist() == [[2]] and np.allclose(w, [[0.05]])


def test_gate_oracle_masks():
    lg = np.full((2, 4), -np.inf)
    lg[0, 2] = 1.0
    ids, w = ogate.gate(lg, 3, "sigmoid")
    assert ids.tolist() == [[2, 0, 1], [0, 1, 2]] and w.tolist() == [[1, 0, 0], [0, 0, 0]]
    ids, w = ogate.gate(np.array([[np.nan, np.inf, 0.0]]), 2)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[1, 0]]


def test_norm_oracle():
    x = np.array([[3.0, 4.0]])
    r, add = onorm.residual_update(x, None, post_weight=[1.0, 2.0], eps=1e-12, scale=0.5, gate=[[2.0]])
    assert np.allclose(add, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]) and np.all(r == 0)


@pytest.mark.parametrize("e,h,i,k", [(8, 256, 128, 2), (128, 2048, 768, 8), (512, 128, 128, 1), (16, 256, 128, 16)])
def test_the_gate_takes_no_workspace_of_its_own(lib, e, h, i, k):
    """A workspace of the size that the layer needed before it had a gate is
    enough: its arrays, each rounded up to 256 bytes, are these."""
    d = LayerDesc(1, e, h, i, k, 2, P, P + 0x1000, None, P + 0x2000, P + 0x3000, None)
    handle, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.moe_quant_init(ctypes.byref(d), ctypes.byref(handle)) == OK

    def size(t):
        assert lib.moe_quant_workspace_size(handle, t, ctypes.byref(n)) == OK
        return n.value

    assert size(0) > 0
    chunks = 256 * e * 4
    for t in (1, 2, 17, 64, 65, 300, 4096, 100000):
        r = t * k
        parts = (16, 4 * r, 4 * r, 4 * (e + 1), 16 * (e + 1), 16 * r, 4 * (e + 1), 4 * (e + 1), 4 * r, 4 * r, chunks,
                 2 * t * h, 4 * t, 4 * t * e, 2 * r * i, 2 * r * h)
        assert size(t) <= sum(-(-p // 256) * 256 for p in parts), t
    lib.moe_quant_destroy(handle)


def test_noalloc_takes_as_many_tokens_as_before(lib):
    d = LayerDesc(1, 8, 256, 128, 2, 2, P, P + 0x1000, None, P + 0x2000, P + 0x3000, None)
    handle, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.moe_quant_init(ctypes.byref(d), ctypes.byref(handle)) == OK
    assert lib.moe_quant_workspace_size(handle, 31237, ctypes.byref(n)) == OK
    assert n.value <= 64 << 20
    lib.moe_quant_destroy(handle)
