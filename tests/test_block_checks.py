"""Argument checks of the dense product, the cache's append and the attention
over it, and their oracles (runs without a GPU: every call here is refused or has
no tokens)."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import attention as oattn
from oracle import codecs
from oracle import linear as olin
from oracle import w8a8
from weight_quantized_moe_amd import KVCache, Linear, MoeQuantError, Rotary, binding, build
from weight_quantized_moe_amd.binding import KvCacheDesc, LinearDesc, RotaryDesc

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
    assert ctypes.sizeof(LinearDesc) == 32 and LinearDesc.w.offset == 16
    assert ctypes.sizeof(KvCacheDesc) == 56 and KvCacheDesc.num_pages.offset == 16 and KvCacheDesc.k.offset == 40
    assert ctypes.sizeof(RotaryDesc) == 48 and RotaryDesc.cos_sin.offset == 24


# ---------------------------------------------------------------- the product
def _linear(**over):
    f = dict(abi=1, n=128, k=256, out=1, w=P, scale=P)
    f.update(over)
    return LinearDesc(f["abi"], f["n"], f["k"], f["out"], f["w"], f["scale"])


@pytest.mark.parametrize("over,expect", [
    (dict(abi=2), ABI), (dict(n=0), SHAPE), (dict(n=-1), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(k=0), SHAPE),
    (dict(k=8), SHAPE), (dict(k=24), SHAPE), (dict(k=65552), SHAPE), (dict(out=2), DTYPE), (dict(w=None), NULL),
    (dict(scale=None), NULL), (dict(w=P + 8), ALIGN), (dict(scale=P + 2), ALIGN)])
def test_linear_refuses_bad_fields(lib, over, expect):
    d, b = _linear(**over), ctypes.c_size_t()
    assert lib.moe_quant_linear(ctypes.byref(d), P, None, 0, P, P, 1 << 30, None) == expect
    assert lib.moe_quant_linear_workspace_size(ctypes.byref(d), 1, ctypes.byref(b)) == expect
    assert lib.moe_quant_last_error()


def test_linear_refuses_bad_calls(lib):
    d, b = _linear(), ctypes.c_size_t()
    r = ctypes.byref(d)
    assert lib.moe_quant_linear_workspace_size(r, 3, ctypes.byref(b)) == OK and b.value > 0
    assert lib.moe_quant_linear_workspace_size(r, 3, None) == NULL
    Q = 2 * P                                        # apart from x
    assert lib.moe_quant_linear_workspace_size(r, -1, ctypes.byref(b)) == SHAPE
    assert lib.moe_quant_linear_workspace_size(r, (1 << 22) + 1, ctypes.byref(b)) == SHAPE
    for args, expect in (((P, None, -1, Q, P, b.value), SHAPE), ((P, None, (1 << 22) + 1, Q, P, b.value), SHAPE),
                         ((None, None, 3, Q, P, b.value), NULL), ((P, None, 3, None, P, b.value), NULL),
                         ((P + 8, None, 3, Q, P, b.value), ALIGN), ((P, P + 1, 3, Q, P, b.value), ALIGN),
                         ((P, None, 3, Q + 1, P, b.value), ALIGN), ((P, None, 3, Q, None, b.value), WORKSPACE),
                         ((P, None, 3, Q, P + 16, b.value), ALIGN), ((P, None, 3, Q, P, b.value - 1), WORKSPACE)):
        assert lib.moe_quant_linear(r, *args, None) == expect, args
    # n 128, k 256, 3 rows: x takes 0x600 bytes, a BF16 out and the residual 0x300
    for x, res, out in ((P, None, P), (P, None, P + 0x5FE), (P + 0x2F0, None, P), (P, 9 * P, 9 * P + 2), (P, 9 * P + 0x2FE, 9 * P)):
        assert lib.moe_quant_linear(r, x, res, 3, out, 99 * P, b.value, None) == SHAPE, (x, res, out)
    assert lib.moe_quant_linear(ctypes.byref(_linear(out=0)), P, 9 * P, 3, 9 * P, 99 * P, b.value, None) == SHAPE
    assert lib.moe_quant_linear(None, P, None, 3, P, P, b.value, None) == NULL
    f = _linear(out=0)
    assert lib.moe_quant_linear(ctypes.byref(f), P, None, 3, P + 2, P, b.value, None) == ALIGN
    assert lib.moe_quant_linear(r, None, None, 0, None, None, 0, None) == OK
    assert lib.moe_quant_last_error() == b""


# ---------------------------------------------------------------- the cache
def _cache(**over):
    f = dict(abi=1, heads=4, d=64, page=16, pages=10, dtype=0, ks=1.0, vs=1.0, k=P, v=P)
    f.update(over)
    return KvCacheDesc(f["abi"], f["heads"], f["d"], f["page"], f["pages"], f["dtype"], f["ks"], f["vs"], f["k"], f["v"])


def _rotary(**over):
    f = dict(abi=1, d=64, r=32, inter=0, most=100, eps=1e-6, c=P, qn=None, kn=None)
    f.update(over)
    return RotaryDesc(f["abi"], f["d"], f["r"], f["inter"], f["most"], f["eps"], f["c"], f["qn"], f["kn"])


BAD_CACHES = [
    (dict(abi=0), ABI), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(d=0), SHAPE), (dict(d=24), SHAPE),
    (dict(d=272), SHAPE), (dict(page=0), SHAPE), (dict(page=12), SHAPE), (dict(page=2048), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=-1), SHAPE), (dict(pages=1 << 27), SHAPE), (dict(pages=1 << 40), SHAPE), (dict(dtype=2), DTYPE),
    (dict(ks=0.5), SHAPE), (dict(vs=2.0), SHAPE), (dict(dtype=1, ks=0.0), SHAPE), (dict(dtype=1, vs=-1.0), SHAPE),
    (dict(dtype=1, ks=math.nan), SHAPE), (dict(dtype=1, vs=math.inf), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN)]


@pytest.mark.parametrize("over,expect", BAD_CACHES)
def test_cache_refuses_bad_fields(lib, over, expect):
    c, r, b = ctypes.byref(_cache(**over)), ctypes.byref(_rotary()), ctypes.c_size_t()
    assert lib.moe_quant_kv_append(c, r, 8, P, 512, P, 256, P, 256, P, P, 0, P, None) == expect
    assert lib.moe_quant_attend_workspace_size(c, 8, 1, ctypes.byref(b)) == expect
    assert lib.moe_quant_attend(c, 8, 1.0, 0, P, P, 4, 4, P, 0, P, None, P, 1 << 30, None) == expect


@pytest.mark.parametrize("over,expect", [
    (dict(abi=3), ABI), (dict(d=128), SHAPE), (dict(r=-16), SHAPE), (dict(r=80), SHAPE), (dict(r=24), SHAPE),
    (dict(most=0), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE),
    (dict(c=None), NULL), (dict(r=0), NULL), (dict(c=P + 8), ALIGN), (dict(qn=P + 2), ALIGN), (dict(kn=P + 8), ALIGN)])
def test_rotary_refuses_bad_fields(lib, over, expect):
    c, r = ctypes.byref(_cache()), ctypes.byref(_rotary(**over))
    assert lib.moe_quant_kv_append(c, r, 8, P, 512, P, 256, P, 256, P, P, 0, P, None) == expect


def test_append_refuses_bad_calls(lib):
    c, r = ctypes.byref(_cache()), ctypes.byref(_rotary())
    # q and q_out take 0xC00 bytes, k and v 0x600
    good = dict(hq=8, q=P, qs=512, k=P, ks=256, v=P, vs=256, pos=P, slots=P, t=3, out=2 * P)
    for over, expect in ((dict(t=-1), SHAPE), (dict(t=(1 << 22) + 1), SHAPE), (dict(hq=-1), SHAPE), (dict(hq=1025), SHAPE),
                         (dict(q=None), NULL), (dict(out=None), NULL), (dict(hq=0), NULL), (dict(k=None), NULL),
                         (dict(v=None), NULL), (dict(pos=None), NULL), (dict(slots=None), NULL), (dict(q=P + 8), ALIGN),
                         (dict(k=P + 4), ALIGN), (dict(v=P + 2), ALIGN), (dict(out=P + 8), ALIGN), (dict(pos=P + 2), ALIGN),
                         (dict(slots=P + 1), ALIGN), (dict(qs=504), SHAPE), (dict(ks=248), SHAPE), (dict(vs=0), SHAPE),
                         (dict(vs=-256), SHAPE), (dict(qs=516), ALIGN), (dict(ks=260), ALIGN), (dict(vs=257), ALIGN),
                         (dict(qs=1024, out=P), SHAPE), (dict(out=P), SHAPE), (dict(out=P + 16, k=9 * P, v=9 * P), SHAPE),
                         (dict(k=2 * P + 0xBF0), SHAPE), (dict(v=2 * P - 0x5F0), SHAPE),
                         (dict(q=2 * P, out=2 * P, vs=1 << 16), SHAPE)):
        f = dict(good, **over)
        assert lib.moe_quant_kv_append(c, r, f["hq"], f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["pos"],
                                       f["slots"], f["t"], f["out"], None) == expect, over
    assert lib.moe_quant_kv_append(None, r, 8, P, 512, P, 256, P, 256, P, P, 0, P, None) == NULL
    assert lib.moe_quant_kv_append(c, None, 8, P, 512, P, 256, P, 256, P, P, 0, P, None) == NULL
    assert lib.moe_quant_kv_append(c, r, 0, None, 0, None, 0, None, 0, None, None, 0, None, None) == OK


def test_attend_refuses_bad_calls(lib):
    c, b = ctypes.byref(_cache()), ctypes.c_size_t()
    assert lib.moe_quant_attend_workspace_size(c, 8, 5, ctypes.byref(b)) == OK and b.value > 0
    assert lib.moe_quant_attend_workspace_size(c, 8, 5, None) == NULL
    good = dict(hq=8, scale=0.1, window=0, q=P, table=P, apart=7, pages=7, lengths=P, b=5, out=P, lse=None, ws=P, n=b.value)
    for over, expect in ((dict(hq=0), SHAPE), (dict(hq=6), SHAPE), (dict(hq=2048), SHAPE), (dict(scale=math.nan), SHAPE),
                         (dict(scale=math.inf), SHAPE), (dict(window=-1), SHAPE), (dict(pages=-1), SHAPE),
                         (dict(pages=1 << 28, apart=1 << 28), SHAPE), (dict(apart=6), SHAPE), (dict(b=-1), SHAPE),
                         (dict(b=(1 << 16) + 1), SHAPE), (dict(q=None), NULL), (dict(table=None), NULL),
                         (dict(lengths=None), NULL), (dict(out=None), NULL), (dict(q=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
                         (dict(table=P + 2), ALIGN), (dict(lengths=P + 1), ALIGN), (dict(lse=P + 2), ALIGN),
                         (dict(out=P + 16), SHAPE), (dict(out=P - 16), SHAPE), (dict(ws=None), WORKSPACE),
                         (dict(ws=P + 128), ALIGN), (dict(n=b.value - 1), WORKSPACE)):
        f = dict(good, **over)
        assert lib.moe_quant_attend(c, f["hq"], f["scale"], f["window"], f["q"], f["table"], f["apart"], f["pages"],
                                    f["lengths"], f["b"], f["out"], f["lse"], f["ws"], f["n"], None) == expect, over
    # the most requests, and too many of the most heads
    wide = ctypes.byref(_cache(heads=1024))
    assert lib.moe_quant_attend_workspace_size(wide, 1024, 1 << 13, ctypes.byref(b)) == OK
    assert lib.moe_quant_attend_workspace_size(wide, 1024, (1 << 13) + 1, ctypes.byref(b)) == SHAPE
    assert lib.moe_quant_attend(wide, 1024, 1.0, 0, P, P, 7, 7, P, 1 << 14, P, None, P, 1 << 40, None) == SHAPE
    # a request of 2^30 tokens, and one page more; a scale that only its product with the keys' makes infinite
    for pages, ws, expect in ((1 << 26, 0, WORKSPACE), ((1 << 26) + 1, 1 << 40, SHAPE)):
        assert lib.moe_quant_attend(c, 8, 1.0, 0, P, P, 1 << 27, pages, P, 5, P, None, P, ws, None) == expect
    assert lib.moe_quant_attend(ctypes.byref(_cache(dtype=1, ks=1e10)), 8, 1e30, 0, P, P, 7, 7, P, 5, P, None, P, 1 << 40,
                                None) == SHAPE
    assert lib.moe_quant_attend(c, 8, 1.0, 0, None, None, 0, 0, None, 0, None, None, None, 0, None) == OK


# ---------------------------------------------------------------- the binding
def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refuses_what_is_not_on_a_gpu():
    u8 = torch.zeros(128, 256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        Linear(u8, torch.zeros(1, 2))                      # not on a GPU
    with pytest.raises(ValueError):
        Linear(u8, torch.zeros(2, 2))                      # scales of another shape
    with pytest.raises(ValueError):
        Linear(u8.float(), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        Linear(u8, torch.zeros(1, 2), out_dtype=torch.float16)
    with pytest.raises(ValueError):
        Linear(u8[0], torch.zeros(1, 2))
    for k, v in ((_bf(4, 2, 16, 64), _bf(4, 2, 16, 64)), (_bf(4, 2, 16, 64), _bf(4, 2, 16, 32)),
                 (_bf(4, 2, 16, 64), torch.zeros(4, 2, 16, 64)), (_bf(2, 16, 64), _bf(2, 16, 64)),
                 (_bf(4, 16, 2, 64).transpose(1, 2), _bf(4, 2, 16, 64))):
        with pytest.raises(ValueError):
            KVCache(k, v)
    for over in (dict(cos_sin=torch.zeros(10, 32)), dict(cos_sin=torch.zeros(10, 80)), dict(cos_sin=torch.zeros(10, 24)),
                 dict(cos_sin=torch.zeros(10, 32).double()), dict(cos_sin=torch.zeros(32)), dict(q_norm=_bf(64)),
                 dict(k_norm=_bf(32)), dict(q_norm=torch.zeros(64)), dict(cos_sin=torch.zeros(0, 32)),
                 dict(cos_sin=torch.zeros(10, 0))):
        with pytest.raises(ValueError):
            Rotary(64, **over)
    assert not Rotary(64).rotates


def test_table_of_angles():
    t = Rotary.table(40000, 32, base=1e6, device="cpu")
    assert t.shape == (40000, 32) and t.dtype == torch.float32
    for p in (0, 1, 39999):
        for i in (0, 7, 15):
            a = p * 1e6 ** (-2 * i / 32)
            assert abs(float(t[p, i]) - math.cos(a)) <= 2.0 ** -23 and abs(float(t[p, 16 + i]) - math.sin(a)) <= 2.0 ** -23


# ---------------------------------------------------------------- the oracles
def test_oracle_linear_against_loops():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 144)).astype(np.float32)
    x[1, :128] = 0
    w = codecs.quantize_e4m3(rng.standard_normal((130, 144)))
    s = (1 + rng.random((2, 2))).astype(np.float32)
    y, size, largest = olin.forward(x, w, s)
    codes, sa = olin.quantize_rows(x)
    assert sa[1, 0] == 1 and codes.shape == (3, 256) and not codes[:, 144:].any() and not codes[1, :128].any()
    table = codecs.decode_e4m3(np.arange(256, dtype=np.uint8))
    for t in range(3):
        for n in (0, 127, 129):
            terms = [table[codes[t, k]] * float(sa[t, k // 128]) * table[w[n, k]] * float(s[n // 128, k // 128])
                     for k in range(144)]
            assert abs(y[t, n] - sum(terms)) <= 1e-12 * size[t, n]
            assert np.isclose(largest[t, n], max(map(abs, terms[:128])) + max(map(abs, terms[128:])))
    back = np.repeat(sa, 128, 1)[:, :144] * table[codes[:, :144]]
    assert np.all(np.abs(back - x) <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) + 2.0 ** -10 * np.repeat(sa, 128, 1)[:, :144])


def test_oracle_turn_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 48))
    angle = rng.standard_normal((5, 16)) * 100
    table = np.concatenate((np.cos(angle), np.sin(angle)), 1)
    for inter in (False, True):
        y = oattn.turn(x, None, 1e-6, table, inter)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        one, two = (slice(0, 32, 2), slice(1, 32, 2)) if inter else (slice(0, 16), slice(16, 32))
        z = (x[..., one] + 1j * x[..., two]) * np.exp(1j * angle)[:, None]
        assert np.allclose(y[..., one], z.real) and np.allclose(y[..., two], z.imag)
    n = oattn.turn(x, np.full(48, 2.0), 0.0, None, False)
    assert np.allclose((n * n).mean(2), 4.0)


def test_oracle_attend_on_a_dense_cache():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 4, 16)), rng.standard_normal((6, 2, 4, 16)), rng.standard_normal((6, 2, 4, 16))
    table = np.array([[3, 1, 5], [0, 7, 2]])     # page 7 is not there
    out, lse, _, _ = oattn.attend(q, k, v, table, [10, 12], 0.25, window=0)
    for b, at in ((0, [(3, i) for i in range(4)] + [(1, i) for i in range(4)] + [(5, 0), (5, 1)]),
                  (1, [(0, i) for i in range(4)] + [(2, i) for i in range(4)])):
        for h in range(4):
            e = np.exp([0.25 * q[b, h] @ k[p, h // 2, s] for p, s in at])
            assert np.allclose(out[b, h], (e[:, None] * [v[p, h // 2, s] for p, s in at]).sum(0) / e.sum())
            assert np.isclose(lse[b, h], np.log(e.sum()))
    out, lse, _, _ = oattn.attend(q, k, v, table, [0, -3], 0.25)
    assert not out.any() and np.all(lse == -np.inf)


def test_attend_refuses_scales_whose_base_2_factor_is_infinite(lib):
    """Scores become exponents of 2: scale k_scale log2(e) has to be finite, 2.3586e38 at most."""
    for dtype, ks, scale, expect in ((0, 1.0, 2.36e38, SHAPE), (0, 1.0, -3e38, SHAPE), (0, 1.0, 2.358e38, WORKSPACE),
                                     (1, 1e19, 2.4e19, SHAPE), (1, 1e19, 2.3e19, WORKSPACE), (1, 1e-5, 3e38, WORKSPACE)):
        c = ctypes.byref(_cache(dtype=dtype, ks=ks))
        got = lib.moe_quant_attend(c, 8, scale, 0, P, P, 7, 7, P, 5, P, None, None, 0, None)
        assert got == expect, (dtype, ks, scale)


def test_how_the_rows_codes_relate_to_the_layers():
    """The product's scale is m * fl(1 / 448), the layer's m / 448: the same or the next
    FP32 number, for 71 of a BF16 maximum's 128 mantissas; codes a step apart at most."""
    m = np.zeros((128, 128), np.float32)
    m[:, 0] = 1 + np.arange(128) / 128
    far = olin.quantize_rows(m)[1].view(np.int32) - w8a8.quantize_act(m)[1].view(np.int32)
    assert int((far == 1).sum()) == 71 and int((far == 0).sum()) == 57
    x = torch.randn(1000, 512, generator=torch.Generator().manual_seed(0)).bfloat16().float().numpy()
    (a, sa), (b, sb) = olin.quantize_rows(x), w8a8.quantize_act(x)
    far = sa.view(np.int32) - sb.view(np.int32)
    assert np.all((far == 0) | (far == 1))
    step = (a & 127).astype(int) - (b & 127)
    assert np.all(np.abs(step) <= 1) and np.array_equal(a >> 7, b >> 7)
    # and only in blocks whose scales differ
    assert 1 / 2000 < np.mean(step != 0) < 1 / 400 and not step[np.repeat(far, 128, 1) == 0].any()


def test_attend_workspace_does_not_shrink_with_the_batch(lib):
    """One sized for the largest batch serves every smaller one, across 1024 requests, where
    the plan of pieces ends, too."""
    for heads, hq, d in ((1, 1, 16), (1, 20, 128), (4, 32, 128), (8, 8, 64), (16, 256, 256), (64, 64, 80), (1024, 1024, 64)):
        c, last = ctypes.byref(_cache(heads=heads, d=d)), 0
        for batch in list(range(0, 140)) + [255, 256, 257, 511, 512, 513, 1023, 1024, 1025, 2048, 8192]:
            b = ctypes.c_size_t()
            assert lib.moe_quant_attend_workspace_size(c, hq, batch, ctypes.byref(b)) == OK
            assert b.value >= last, (heads, hq, d, batch)
            last = b.value


# ---------------------------------------------------------------- what must not overlap
BIG = 1 << 40            # addresses far from each other, that no refused call reads


def test_linear_refuses_overlaps_of_what_it_writes(lib):
    # n 128, k 256, 3 rows: x 0x600 bytes, a BF16 out and the residual 0x300, w 0x8000, scale 8
    w, sc, x, res, out, ws = (BIG * i for i in range(1, 7))
    d, b = _linear(w=w, scale=sc), ctypes.c_size_t()
    assert lib.moe_quant_linear_workspace_size(ctypes.byref(d), 3, ctypes.byref(b)) == OK
    n = b.value
    for over in (dict(out=w), dict(out=w + 0x7FFE), dict(out=w - 0x2FE), dict(out=sc + 4), dict(out=ws), dict(out=ws + n - 2),
                 dict(out=ws - 0x2FE), dict(ws=w + 0x7F00), dict(ws=w - 256), dict(ws=sc), dict(ws=x), dict(ws=x + 0x500),
                 dict(ws=res + 0x200), dict(ws=res - 256), dict(ws=out)):
        f = dict(dict(x=x, res=res, out=out, ws=ws), **over)
        assert lib.moe_quant_linear(ctypes.byref(d), f["x"], f["res"], 3, f["out"], f["ws"], n, None) == SHAPE, over


def test_append_refuses_overlaps_of_what_it_writes(lib):
    # a cache of 10 pages of 16 tokens and 4 heads of 64: 0x14000 bytes each of k and v in BF16
    kc, vc, cs, qn, kn, q, k, v, pos, slots, out = (BIG * i for i in range(1, 12))
    for over in (dict(vc=kc), dict(vc=kc + 0x13FF0), dict(vc=kc - 0x13FF0), dict(out=kc), dict(out=kc - 0xBF0),
                 dict(out=vc + 0x13FF0), dict(out=slots - 0xBF0), dict(out=pos), dict(out=cs + 100 * 128 - 16), dict(out=qn),
                 dict(out=kn - 16), dict(q=kc), dict(q=vc + 0x13FF0), dict(k=kc), dict(k=vc - 16), dict(v=vc), dict(v=kc + 16),
                 dict(slots=kc), dict(slots=vc + 0x13FFC), dict(pos=kc - 8), dict(cs=kc + 16), dict(cs=vc - 16), dict(qn=kc),
                 dict(kn=vc + 16)):
        f = dict(dict(kc=kc, vc=vc, cs=cs, qn=qn, kn=kn, q=q, k=k, v=v, pos=pos, slots=slots, out=out), **over)
        c, r = _cache(k=f["kc"], v=f["vc"]), _rotary(c=f["cs"], qn=f["qn"], kn=f["kn"])
        got = lib.moe_quant_kv_append(ctypes.byref(c), ctypes.byref(r), 8, f["q"], 512, f["k"], 256, f["v"], 256, f["pos"],
                                      f["slots"], 3, f["out"], None)
        assert got == SHAPE, over
    # of an E4M3 cache half as many bytes
    c, r = _cache(dtype=1, k=kc, v=kc + 0xA000 - 16), _rotary(c=cs)
    assert lib.moe_quant_kv_append(ctypes.byref(c), ctypes.byref(r), 0, None, 0, k, 256, v, 256, pos, slots, 3, None, None) == SHAPE


def test_attend_refuses_overlaps_of_what_it_writes(lib):
    # 5 requests of 8 heads of 64: q and out 0x1400 bytes, lse 0xA0, 7 pages a request 9 entries apart
    kc, vc, q, table, lengths, out, lse, ws = (BIG * i for i in range(1, 9))
    b = ctypes.c_size_t()
    assert lib.moe_quant_attend_workspace_size(ctypes.byref(_cache()), 8, 5, ctypes.byref(b)) == OK
    n = b.value
    for over in (dict(out=kc), dict(out=vc + 0x13FF0), dict(out=ws), dict(out=ws + n - 16), dict(out=lengths), dict(out=lse - 16),
                 dict(out=table + 160), dict(lse=out + 0x13FC), dict(lse=q), dict(lse=kc + 4), dict(lse=vc - 0x9C),
                 dict(lse=ws + n - 4), dict(lse=lengths + 16), dict(lse=table + 4 * (4 * 9 + 6)), dict(lse=q, out=q),
                 dict(ws=q), dict(ws=kc), dict(ws=vc + 0x13F00), dict(ws=table), dict(ws=lengths)):
        f = dict(dict(kc=kc, vc=vc, q=q, table=table, lengths=lengths, out=out, lse=lse, ws=ws), **over)
        c = ctypes.byref(_cache(k=f["kc"], v=f["vc"]))
        got = lib.moe_quant_attend(c, 8, 0.1, 0, f["q"], f["table"], 9, 7, f["lengths"], 5, f["out"], f["lse"], f["ws"], n, None)
        assert got == SHAPE, over
