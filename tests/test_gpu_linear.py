"""The dense product on E4M3 weights on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import codecs
from oracle import linear as olin
from weight_quantized_moe_amd import Linear, MoeQuantError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(n, k, seed=0, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(0, 255, (n, k), generator=gen, device="cuda").to(torch.uint8)
    w = torch.where((w & 127) == 127, w - 1, w)                      # no NaN codes
    s = torch.exp(spread * torch.randn(-(-n // 128), -(-k // 128), generator=gen, device="cuda")) * 0.01
    return w, s


def rows(t, k, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    x = torch.randn(t, k, generator=gen, device="cuda") * torch.exp(torch.randn(t, 1, generator=gen, device="cuda"))
    x[:, ::61] *= 30.0
    return x.to(BF)


def limit(y, size, largest, k, dtype):
    """FP32 output: products of codes are exact and a block of 128 is added in FP32
    (2^-23 each, should the matrix unit cut off): 128 of 2^-23 of the terms'
    magnitudes; then two products and an addition per block, the joining of at most
    16 partial sums and the residual: G + 24 roundings of 2^-24; then half a step
    of the output's type.  BF16 output: the FP8 units cut each of a block's 128
    products at 2^-16 of the block's largest on top of it, 2^-9 of it in all."""
    c = (128 * 2.0 ** -23 + (-(-k // 128) + 24) * 2.0 ** -24) * size
    if dtype == BF:
        c = c + 2.0 ** -9 * largest
    return c + (torch.finfo(dtype).eps / 2) * (np.abs(y) + c) + 1e-38


def check(t, n, k, dtype=BF, residual=False, seed=0, x=None, ws=None):
    w, s = make(n, k, seed)
    x = rows(t, k, seed) if x is None else x
    r = None
    if residual:
        r = (50.0 * torch.randn(t, n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(BF)
    lin = Linear(w, s, out_dtype=dtype)
    out = torch.full((t + 1, n), 7.0, dtype=dtype, device="cuda")    # the row behind the last stays as it was
    got = lin.forward(x, residual=r, out=out[:t], workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(out[t] == 7.0)
    y, *parts = olin.forward(f64(x), w.cpu().numpy(), s.cpu().numpy(), None if r is None else f64(r))
    off, most = np.abs(f64(got) - y), limit(y, *parts, k, dtype)
    assert np.all(off <= most), (t, n, k, float((off / most).max()), np.unravel_index((off / most).argmax(), off.shape))
    # in the 2-norm: a rounding is evenly spread over its step (2^-8 / sqrt 3 at most for
    # BF16), the FP8 units' 128 cuts are independent: sqrt(128 / 3) 2^-16 of the largest
    far = np.sqrt(np.sum(off ** 2))
    if t * n >= 1000:
        near = torch.finfo(dtype).eps / 2 / np.sqrt(3) * np.sqrt(np.sum(y ** 2))
        near += np.sqrt(128 / 3) * 2.0 ** -16 * np.sqrt(np.sum(parts[1] ** 2)) if dtype == BF else 0
        near += np.sqrt(128 + k / 128) * 2.0 ** -23 * np.sqrt(np.sum(parts[0] ** 2))
        assert far <= 1.2 * near, (far, near)
    return lin, x, got


SIZES = [(1, 1, 16), (1, 128, 128), (1, 129, 144), (3, 130, 272), (15, 64, 2064), (16, 576, 256), (17, 1000, 400),
         (33, 513, 640), (64, 2048, 1024), (65, 257, 1040), (100, 33, 4112), (128, 384, 128), (129, 640, 512),
         (255, 300, 272), (256, 256, 2048), (257, 511, 1136), (300, 5, 48), (511, 1, 256), (513, 1025, 384), (777, 1000, 2064),
         (1030, 768, 896), (2049, 520, 528)]


@pytest.mark.parametrize("t,n,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sizes(t, n, k, dtype):
    check(t, n, k, dtype, residual=(t + n) % 2 == 1, seed=t)
    check(t, n, k, dtype, residual=(t + n) % 2 == 0, seed=t + 1)


@pytest.mark.parametrize("t,n,k", [(10, 4999, 2064), (16, 4900, 1040), (20, 4999, 400), (33, 5000, 272), (64, 4801, 2064),
                                   (130, 1300, 400), (200, 960, 144),       # streamed, 32 weight rows a workgroup
                                   (130, 4000, 144), (333, 2000, 400), (300, 2300, 1040),   # 64 x 64, 4 blocks of K at a time
                                   (70, 9000, 144), (600, 2000, 400),       # tiles of 64 x 64
                                   (2049, 2100, 272),                       # tiles of 64 x 128
                                   (2050, 2570, 144)])                      # tiles of 128 x 128
@pytest.mark.parametrize("dtype", [BF, F32])
def test_each_way(t, n, k, dtype):
    check(t, n, k, dtype, residual=n % 2 == 0, seed=t)


@pytest.mark.parametrize("n", [8200, 8201])
def test_the_largest_tiles(n):
    """256 x 256; the reference in 64 bits on the GPU, a block's largest product bounded
    by its factors' largest."""
    t, k = 8197, 272
    w, s = make(n, k, 1)
    x = rows(t, k, 1)
    r = torch.randn(t, n, device="cuda").to(BF)
    out = torch.full((t + 1, n), 7.0, dtype=BF, device="cuda")
    Linear(w, s).forward(x, residual=r, out=out[:t])
    codes, sa = olin.quantize_rows(f64(x))
    a = torch.from_numpy(codecs.decode_e4m3(codes) * np.repeat(sa.astype(np.float64), 128, 1))[:, :k].cuda()
    v = torch.from_numpy(codecs.decode_e4m3(w.cpu().numpy())).cuda()
    v = v * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    y, size, largest = r.double(), r.double().abs(), torch.zeros(t, n, dtype=torch.float64, device="cuda")
    for at in range(0, k, 128):
        p, q = a[:, at:at + 128], v[:, at:at + 128]
        y, size = y + p @ q.t(), size + p.abs() @ q.abs().t()
        largest += p.abs().amax(1)[:, None] * q.abs().amax(1)
    assert torch.all(out[t] == 7.0)
    off = (out[:t].double() - y).abs()
    c = (128 * 2.0 ** -23 + 27 * 2.0 ** -24) * size + 2.0 ** -9 * largest
    assert bool((off <= c + 2.0 ** -8 * (y.abs() + c)).all())
    near = 2.0 ** -8 / 3 ** 0.5 * float(y.norm()) + (128 / 3) ** 0.5 * 2.0 ** -16 * float(largest.norm())
    assert float(off.norm()) <= 1.2 * near


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 20, 24, 31, 32, 40, 48, 63, 80, 96, 127, 160, 192])
def test_few_tokens(t):
    for n, k in ((512, 2048), (2048, 512), (300, 1552)):
        check(t, n, k, residual=t % 2 == 0, seed=t)


@pytest.mark.parametrize("t,n,k", [(1, 20000, 128), (1, 16, 65536), (40, 16, 65536), (300, 256, 16384), (4096, 2048, 256)])
def test_long_axes(t, n, k):
    check(t, n, k, dtype=F32, seed=n)


def test_more_rows_than_a_launch_has_lanes():
    """2^20 + 5 rows of 64 blocks: more groups of 16 lanes than one pass of the
    quantization holds."""
    t, k = (1 << 20) + 5, 8192
    w, s = make(16, k, 2)
    x = torch.empty(t, k, dtype=BF, device="cuda")
    x[:] = rows(1, k, 3)
    at = [0, 1, 65535, 1 << 19, (1 << 20) - 1, 1 << 20, t - 2, t - 1]
    some = rows(len(at), k, 4)
    x[at] = some
    got = Linear(w, s).forward(x)
    torch.cuda.synchronize()
    y, *parts = olin.forward(f64(some), w.cpu().numpy(), s.cpu().numpy())
    assert np.all(np.abs(f64(got[at]) - y) <= limit(y, *parts, k, BF))
    assert torch.equal(got[2], got[t - 3]) and torch.equal(got[2], got[1 << 18])


def test_rows_of_every_size():
    """Zero rows, rows below the smallest normal number, rows near the largest."""
    for t in (9, 300):
        x = rows(t, 400, 5)
        x[0] = 0
        x[1] = 2.0 ** -133 * torch.sign(x[1].float()).to(BF)         # the smallest there is
        x[2, :128] = 0
        x[3] = (x[3].float() * 2.0 ** -120).to(BF)
        x[4] = torch.finfo(BF).max
        x[5] = -x[4]
        x[6, 5] = torch.finfo(BF).max
        x[7] = 0
        x[7, 399] = 1.0
        w, s = make(200, 400)
        s *= 2.0 ** -20
        lin = Linear(w, s, out_dtype=F32)
        got = lin.forward(x)
        y, *parts = olin.forward(f64(x), w.cpu().numpy(), s.cpu().numpy())
        off, most = np.abs(f64(got) - y), limit(y, *parts, 400, F32)
        # sums of products below 2^-126 may be flushed by the matrix unit
        assert np.all(off <= most + 2.0 ** -120), float((off / most).max())
        assert not f64(got)[0].any()


def test_ties_of_the_codes():
    """x / s lies midway between codes: 448 / 128 = 3.5 = s exactly, so multiples of
    s / 2 above 16 s are ties of the coarser steps."""
    for t in (4, 260):
        x = torch.zeros(t, 256, device="cuda")
        x[:, :128] = (torch.arange(128, device="cuda") - 64) * 7.0
        x[:, 128:] = (torch.arange(128, device="cuda") - 64) * 7.0 + 0.5
        check(t, 192, 256, F32, x=x.to(BF))


def test_codes_are_the_definitions():
    """The quantized rows as they lie in the workspace (codes [T, 128 G], then the scales
    [G, T]), for values of every exponent and for blocks whose largest is any BF16
    mantissa, where many quotients lie midway between two codes."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    t, k = 6000, 400
    bits = torch.randint(0, 1 << 16, (t, k), generator=gen, device="cuda")
    bits = torch.where((bits & 0x7F80) == 0x7F80, bits & 0x7F7F, bits)            # finite
    near = (torch.randint(0, 1 << 7, (t, k), generator=gen, device="cuda")
            | (torch.randint(118, 128, (t, k), generator=gen, device="cuda") << 7)
            | (torch.randint(0, 2, (t, k), generator=gen, device="cuda") << 15))
    bits[t // 3:] = near[t // 3:]
    x = bits.to(torch.int32).to(torch.int16).view(BF)
    lin = Linear(*make(64, k))
    ws = lin.workspace(t)
    lin.forward(x, workspace=ws)
    torch.cuda.synchronize()
    codes, sa = olin.quantize_rows(f64(x))
    got = ws[:t * 512].view(t, 512).cpu().numpy()
    assert np.array_equal(got & 127, codes & 127) and np.array_equal((got >> 7)[codes & 127 > 0], (codes >> 7)[codes & 127 > 0])
    at = -(-t * 512 // 256) * 256
    assert np.array_equal(ws[at:at + 4 * 4 * t].view(F32).view(4, t).cpu().numpy().T, sa)


def test_a_nan_weight_stays_in_its_column():
    for t, k in ((3, 400), (300, 400), (300, 512)):
        w, s = make(300, k)
        w[17, 5] = 127
        w[299, k - 1] = 255
        for c in (Linear(w, s).forward(rows(t, k)), Linear(w, s, out_dtype=F32).forward(rows(t, k))):
            bad = torch.isnan(c)
            assert bad[:, 17].all() and bad[:, 299].all() and int(bad.sum()) == 2 * t


def test_residual_in_the_output():
    for t in (1, 5, 130, 600):
        lin, x, _ = check(t, 320, 512, residual=True)
        r = torch.randn(t, 320, device="cuda").to(BF)
        want = lin.forward(x, residual=r)
        got = lin.forward(x, residual=r, out=r)
        torch.cuda.synchronize()
        assert got is r and torch.equal(got, want)


def test_rows_do_not_see_each_other():
    """A token's result is the same wherever it stands in a batch of the same size."""
    for t in (2, 16, 70, 500):
        w, s = make(384, 1024)
        lin, x = Linear(w, s), rows(t, 1024)
        turned = torch.roll(x, 1, 0)
        a, b = lin.forward(x), lin.forward(turned)
        assert torch.equal(torch.roll(a, 1, 0), b)


def test_workspace_of_any_content_and_repeats():
    for t in (1, 13, 64, 400):
        w, s = make(400, 1040)
        lin, x = Linear(w, s), rows(t, 1040)
        ws = lin.workspace(t)
        outs = []
        for fill in (0, 127, 255):
            ws.fill_(fill)
            outs.append(lin.forward(x, workspace=ws))
        outs.append(lin.forward(x))
        torch.cuda.synchronize()
        assert all(torch.equal(o, outs[0]) for o in outs)


def test_unaligned_output_rows():
    """Outputs that start anywhere an element may start."""
    for t in (3, 300):
        for dtype in (BF, F32):
            w, s = make(257, 528)
            lin, x = Linear(w, s, out_dtype=dtype), rows(t, 528)
            want = lin.forward(x)
            raw = torch.zeros(t * 257 + 3, dtype=dtype, device="cuda")
            out = raw[1:1 + t * 257].view(t, 257)
            lin.forward(x, out=out)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and raw[0] == 0 and not raw[1 + t * 257:].any()


def test_streams_and_two_workspaces():
    w, s = make(512, 2048)
    lin = Linear(w, s)
    xs = [rows(t, 2048, t) for t in (1, 40, 700)]
    want = [lin.forward(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [lin.forward(x, stream=st) for x, st in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_of_one_workspace_and_two_host_threads():
    import threading
    w, s = make(512, 1024)
    lin = Linear(w, s)
    xs = [rows(t, 1024, t) for t in (20, 300)]
    want = [lin.forward(x) for x in xs]
    ws, outs, graphs = lin.workspace(300), [torch.empty_like(o) for o in want], []
    for x, o in zip(xs, outs):
        lin.forward(x, out=o, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            lin.forward(x, out=o, workspace=ws)
    for rep in range(3):
        for o in outs:
            o.zero_()
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = lin.forward(xs[i])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(got, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    [x.start() for x in threads], [x.join() for x in threads]
    assert not bad


@pytest.mark.parametrize("t", [1, 48, 600])
def test_graph_replays_match_eager(t):
    w, s = make(512, 1024)
    lin, x = Linear(w, s), rows(t, 1024)
    ws, out = lin.workspace(t), torch.empty(t, 512, dtype=BF, device="cuda")
    lin.forward(x, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out=out, workspace=ws)
    for rep in range(4):
        x.copy_(rows(t, 1024, 50 + rep))
        want = lin.forward(x)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


def test_no_tokens_and_refusals():
    w, s = make(128, 256)
    lin = Linear(w, s)
    assert lin.forward(rows(1, 256)[:0]).shape == (0, 128)
    x = rows(4, 256)
    for bad in (x.float(), x[:, :128], x.t(), x.cpu(), x[None]):
        with pytest.raises(ValueError):
            lin.forward(bad)
    for over in (dict(out=torch.empty(4, 128, device="cuda")), dict(out=torch.empty(3, 128, dtype=BF, device="cuda")),
                 dict(residual=torch.empty(4, 128, device="cuda")), dict(residual=x),
                 dict(out=torch.empty(4, 256, dtype=BF, device="cuda")[:, ::2]),
                 dict(workspace=torch.empty(1 << 16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            lin.forward(x, **over)
    square = Linear(*make(256, 256))
    with pytest.raises(MoeQuantError):
        square.forward(x, out=x)
    with pytest.raises(MoeQuantError):
        lin.forward(x, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(MoeQuantError):
        Linear(*make(128, 264))                                      # no multiple of 16


@pytest.mark.parametrize("t,n,k", [(1, 128, 256), (5, 300, 400), (16, 512, 2064), (40, 256, 1040), (64, 4801, 528),
                                   (130, 4000, 144), (300, 1000, 400), (600, 2000, 400), (2049, 2100, 272), (2050, 2570, 144),
                                   (8197, 8200, 144)])
def test_activations_that_are_not_finite_show_in_their_rows(t, n, k):
    w, s = make(n, k, 3)
    w[n // 2] = 0                                                    # and where the weights are zero
    x = rows(t, k, 3)
    for dtype in (BF, F32):
        lin = Linear(w, s, out_dtype=dtype)
        want = lin.forward(x)
        bad = x.clone()
        at = sorted({0, t // 2, t - 1})
        for i, value in zip(at, (float("nan"), float("inf"), -float("inf"))):
            bad[i, (5, k - 1, 100)[at.index(i)]] = value
        got = lin.forward(bad)
        torch.cuda.synchronize()
        assert torch.isnan(got[at]).all()
        got[at] = want[at]
        assert torch.equal(got, want)
        if t > 3000:
            break
