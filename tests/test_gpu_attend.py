"""Attention of one new token over a paged cache on the GPU against the float64
oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oattn
from weight_quantized_moe_amd import KVCache, MoeQuantError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = {BF: 0x7FC0, E4: 0x7F}


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """Requests of these lengths on pages in no order; what no token of a request
    fills holds NaN, and table entries behind a request's pages hold anything."""

    def __init__(self, lengths, hq=4, hk=2, d=64, page=16, dtype=BF, seed=0, size=1.5, ks=1.0, vs=1.0, wide=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        b = len(lengths)
        counts = [max(0, -(-n // page)) for n in lengths]
        pages, most = max(1, sum(counts)) + 2, max([1] + counts) + wide
        order = rng.permutation(pages)
        table = rng.integers(-2 ** 31, 2 ** 31, (b, most)).astype(np.int32)
        self.k, self.v = (torch.empty(pages, hk, page, d, dtype=dtype, device="cuda") for _ in range(2))
        for c in (self.k, self.v):
            c.view(torch.uint8 if dtype == E4 else torch.int16).fill_(NAN[dtype])
        at = 0
        for i, n in enumerate(lengths):
            for p in range(counts[i]):
                page_id, m = int(order[at]), min(page, n - p * page)
                table[i, p], at = page_id, at + 1
                for c in (self.k, self.v):
                    c[page_id, :, :m] = torch.randn(hk, m, d, generator=gen, device="cuda").to(dtype)
        self.table = torch.from_numpy(table).cuda()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.q = (size * torch.randn(b, hq, d, generator=gen, device="cuda")).to(BF)
        self.cache, self.ks, self.vs = KVCache(self.k, self.v, k_scale=ks, v_scale=vs), ks, vs

    def check(self, scale=None, window=0, **over):
        """A score's D products are added in FP32 by the matrix unit (2^-23 each, of
        scale sum |q k| = reach) and meet two factors and the base-2 exponential (8
        roundings of 2^-24 of |score| <= reach, and 2^-22); a probability loses 2^-16 in
        its two BF16 parts; the sums over the tokens take n / 16 + 64 additions at most,
        and joining 16.  Those errors reach the quotient twice; then half a step."""
        b, hq, d = self.q.shape
        out = torch.full((b + 1, hq, d), 7.0, dtype=BF, device="cuda")
        lse = torch.full((b + 1, hq), 7.0, device="cuda")
        used = d ** -0.5 if scale is None else scale
        self.cache.attend(self.q, self.table, self.lengths, scale=scale, window=window, out=out[:b], lse=lse[:b], **over)
        torch.cuda.synchronize()
        assert torch.all(out[b] == 7.0) and torch.all(lse[b] == 7.0)
        k, v = f64(self.k) * self.ks, f64(self.v) * self.vs
        ref, l, spread, reach = oattn.attend(f64(self.q), k, v, self.table.cpu().numpy(), self.lengths.cpu().numpy(), used,
                                             window)
        n = float(self.lengths.max()) if b else 0.0
        e = reach * (d * 2.0 ** -23 + 8 * 2.0 ** -24) + 2.0 ** -22 + 2.0 ** -16 + (n / 16 + 96) * 2.0 ** -23
        off = np.abs(f64(out[:b]) - ref)
        lim = 2 * e[..., None] * spread
        lim = lim + 2.0 ** -8 * (np.abs(ref) + lim) + 1e-38
        assert np.all(off <= lim), (float((off / lim).max()), np.unravel_index((off / lim).argmax(), off.shape))
        got, empty = f64(lse[:b]), np.isinf(l)
        assert np.array_equal(np.isinf(got) & (got < 0), empty)
        off = np.abs(got - l)[~empty]
        assert np.all(off <= (e + 4 * 2.0 ** -24 * np.abs(l))[~empty] + 1e-30)
        return out[:b], lse[:b]


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 257, 511, 700]


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_head_sizes(d, dtype):
    Case(LENGTHS[::2], d=d, dtype=dtype, seed=d).check()


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 1024])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_pages(page, dtype):
    for d in (64, 128):
        Case(LENGTHS, d=d, page=page, dtype=dtype, seed=page, wide=3).check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (3, 1), (7, 1), (8, 1), (15, 1), (16, 1), (17, 1), (33, 1), (64, 1), (5, 5),
                                   (12, 4), (32, 4), (48, 2), (40, 2), (256, 8)])
def test_shared_heads(hq, hk):
    for dtype in (BF, E4):
        Case([0, 1, 40, 333], hq, hk, 128, dtype=dtype, seed=hq).check()


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 128, 256, 500, 10 ** 6, 2 ** 31 - 1])
def test_windows(window):
    for page in (1, 16, 64):
        Case(LENGTHS, page=page, seed=window % 97).check(window=window)


@pytest.mark.parametrize("batch", [1, 2, 5, 64, 257, 700, 1024, 1100])
def test_batches(batch):
    rng = np.random.default_rng(batch)
    lengths = [int(n) for n in rng.integers(0, 200 if batch > 100 else 900, batch)]
    lengths[batch // 2] = 3000
    Case(lengths, 8, 2, 64, seed=batch).check()


@pytest.mark.parametrize("lengths", [[5000], [40000], [3, 20000, 0, 1], [33000, 31, 32768], [1] * 30 + [9000]])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_long_ones_among_short_ones(lengths, dtype):
    for hq, hk, d in ((8, 1, 128), (2, 2, 64), (20, 1, 256)):
        Case(lengths, hq, hk, d, page=64, dtype=dtype, seed=len(lengths)).check()


def test_scales_and_sizes_of_scores():
    for scale in (0.0, -0.3, 1.0, 1e-20):
        Case(LENGTHS, seed=1).check(scale=scale)
    Case(LENGTHS, size=1e-30, seed=2).check()
    Case(LENGTHS, size=300.0, seed=3).check()             # the maximum takes it all
    Case(LENGTHS, dtype=E4, ks=1e-3, vs=1e4, seed=4).check(scale=100.0)
    # scores that rise, and that fall, from one end of the request to the other
    for sign in (1.0, -1.0):
        c = Case([600, 77], 4, 2, 64, seed=5)
        c.q[:] = 1.0
        for i, n in enumerate((600, 77)):
            for j in range(n):
                c.k[c.table[i, j // 16].long(), :, j % 16] = sign * 0.02 * j
        c.check(scale=1.0)


def test_lengths_out_of_range_and_empty_tables():
    c = Case([50, 20, 70, 10], seed=6)
    most = c.table.shape[1] * 16
    c.lengths.copy_(torch.tensor([-1, -2 ** 31, 70, 0], dtype=torch.int32))
    out, lse = c.check()
    assert not out[0].any() and torch.isinf(lse[1]).all() and not out[3].any()
    c.lengths.copy_(torch.tensor([50, 2 ** 31 - 1, most + 1, 10], dtype=torch.int32))
    c.table.clamp_(0, c.k.shape[0] - 1)
    c.k.nan_to_num_(0.25), c.v.nan_to_num_(0.25)
    c.check()
    none = c.cache.attend(c.q, c.table[:, :0], c.lengths)
    torch.cuda.synchronize()
    assert not none.any()


@pytest.mark.parametrize("page", [1, 16, 128])
def test_pages_that_are_not_there(page):
    """Their tokens are absent, at the ends and in the middle, and where all are."""
    c = Case([300, 300, 300, 300, 5000], 8, 2, 128, page=page, seed=7)
    n, hole = c.k.shape[0], max(1, 40 // page)
    c.table[0, :hole] = -1
    c.table[1, hole:2 * hole] = n
    c.table[2, :] = -2 ** 31
    c.table[3, -(-300 // page) - 1] = 2 ** 31 - 1
    c.table[4, 5000 // page // 2:] = n + 5
    out, lse = c.check()
    assert not out[2].any() and torch.isinf(lse[2]).all()


def test_nan_behind_the_last_token_at_every_length():
    for dtype in (BF, E4):
        for d in (64, 80, 256):
            c = Case(list(range(0, 70)), 2, 1, d, page=32, dtype=dtype, seed=8)
            out, _ = c.check()
            assert torch.isfinite(out.float()).all()


def test_table_rows_apart_and_output_in_the_query():
    c = Case([100, 300, 50], 8, 2, 128, seed=9)
    want, _ = c.check()
    wide = torch.full((3, 64), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + c.table.shape[1]] = c.table
    view = wide[:, 5:5 + c.table.shape[1]]
    q = c.q.clone()
    got = c.cache.attend(q, view, c.lengths, out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(got, want)
    for n in (1, 9000):                                   # one workgroup a request, and many
        c = Case([n], 8, 2, 128, seed=10)
        want, _ = c.check()
        q = c.q.clone()
        assert torch.equal(c.cache.attend(q, c.table, c.lengths, out=q), want)


def test_requests_that_share_pages():
    c = Case([400], 8, 2, 64, seed=11)
    one, _ = c.check()
    table, lengths, q = c.table.repeat(5, 1), c.lengths.repeat(5), c.q.repeat(5, 1, 1)
    out = c.cache.attend(q, table, lengths)
    ref = f64(one[0])
    torch.cuda.synchronize()
    # another number of requests may split the request elsewhere: each half a step off
    assert np.all(np.abs(f64(out) - ref[None]) <= 2.0 ** -6 * np.abs(ref) + 1e-4)
    assert all(torch.equal(out[0], o) for o in out[1:]) or torch.allclose(out[0].float(), out[4].float(), rtol=2 ** -6)


def test_workspace_of_any_content_and_repeats():
    for lengths in ([700], [20000, 5], LENGTHS):
        c = Case(lengths, 8, 2, 128, seed=12)
        want, lse = (x.clone() for x in c.check())
        ws = c.cache.attend_workspace(len(lengths), 8)
        for fill in (0, 127, 255):
            ws.fill_(fill)
            got, l2 = c.check(workspace=ws)
            assert torch.equal(got, want) and torch.equal(l2, lse)


def test_streams():
    cases = [Case(n, 8, 2, 128, seed=i) for i, n in enumerate(([900] * 3, [10], [30000], LENGTHS))]
    want = [c.cache.attend(c.q, c.table, c.lengths) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = [c.cache.attend(c.q, c.table, c.lengths, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays_follow_the_lengths():
    """One captured call serves requests as they grow."""
    c = Case([1000, 30, 4000], 8, 2, 128, seed=13, wide=2)
    full = c.lengths.clone()
    out, lse = torch.empty_like(c.q), torch.empty(3, 8, device="cuda")
    ws = c.cache.attend_workspace(3, 8)
    c.cache.attend(c.q, c.table, c.lengths, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.cache.attend(c.q, c.table, c.lengths, out=out, lse=lse, workspace=ws)
    for lengths in ([1000, 30, 4000], [1, 0, 3999], [0, 0, 0], [999, 29, 33], [64, 1, 4000]):
        c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        l2 = torch.empty_like(lse)
        want = c.cache.attend(c.q, c.table, c.lengths, lse=l2)
        out.fill_(9), lse.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, l2), lengths
    c.lengths.copy_(full)


def test_two_graphs_of_one_workspace_and_two_host_threads():
    import threading
    cases = [Case([9000, 3], 8, 2, 128, seed=16), Case([700, 50, 2000, 0, 40], 8, 2, 128, seed=17)]
    want = [c.cache.attend(c.q, c.table, c.lengths) for c in cases]
    ws = cases[1].cache.attend_workspace(5, 8)
    ws = ws if ws.numel() >= cases[0].cache.attend_workspace_size(2, 8) else cases[0].cache.attend_workspace(2, 8)
    outs, graphs = [torch.empty_like(o) for o in want], []
    for c, o in zip(cases, outs):
        c.cache.attend(c.q, c.table, c.lengths, out=o, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.cache.attend(c.q, c.table, c.lengths, out=o, workspace=ws)
    for rep in range(3):
        for o in outs:
            o.zero_()
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    bad = []

    def work(i):
        c = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = c.cache.attend(c.q, c.table, c.lengths)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(got, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i % 2,)) for i in range(4)]
    [x.start() for x in threads], [x.join() for x in threads]
    assert not bad


def test_join_by_lse():
    """Two parts of a request, joined by their lse, are the whole."""
    c = Case([600], 4, 2, 64, page=32, seed=14)
    whole, _ = c.check()
    parts = []
    for table, n in ((c.table[:, :9].contiguous(), 288), (c.table[:, 9:].contiguous(), 600 - 288)):
        lse = torch.empty(1, 4, device="cuda")
        out = c.cache.attend(c.q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), lse=lse)
        parts.append((out.double(), lse.double()))
    w = torch.softmax(torch.stack([p[1] for p in parts]), 0)
    joined = sum(wi[..., None] * p[0] for wi, p in zip(w, parts))
    size = sum(wi[..., None] * p[0].abs() for wi, p in zip(w, parts))
    assert torch.all((joined - whole.double()).abs() <= 2.0 ** -7 * size + 2.0 ** -8 * whole.double().abs() + 1e-6)


def test_no_requests_and_refusals():
    c = Case([100, 50], 8, 2, 64, seed=15)
    assert c.cache.attend(c.q[:0], c.table[:0], c.lengths[:0]).shape == (0, 8, 64)
    good = dict(q=c.q, block_table=c.table, lengths=c.lengths)
    for over in (dict(q=c.q.float()), dict(q=c.q[:1]), dict(q=c.q[..., :32]), dict(q=c.q[0]), dict(q=c.q.transpose(0, 1)),
                 dict(block_table=c.table.long()), dict(block_table=c.table[:1]), dict(block_table=c.table.cpu()),
                 dict(block_table=c.table[:, ::2]), dict(block_table=c.table[:1].expand(2, -1)),
                 dict(lengths=c.lengths.long()), dict(lengths=c.lengths[:1]), dict(out=torch.empty(2, 8, 64, device="cuda")),
                 dict(lse=torch.empty(2, 7, device="cuda")), dict(lse=torch.empty(2, 8, dtype=BF, device="cuda")),
                 dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            c.cache.attend(**dict(good, **over))
    for over in (dict(window=-1), dict(scale=math.nan), dict(q=c.q[:, :7].contiguous())):
        with pytest.raises(MoeQuantError):
            c.cache.attend(**dict(good, **over))


@pytest.mark.parametrize("n,scale", [(300, 1e-42), (300, 1e-39), (1 << 18, 1e-39), (1 << 18, 1e-38), (1 << 18, 2.0 ** -100),
                                     (1 << 18, 1e35)])
def test_value_scales_of_every_size(n, scale):
    """Every token the same value, so that is the result, however many there are: the
    sums of equal terms are off by (n / 16 + 96) 2^-24 at most and mostly exact, the
    quotient and the scale's product by a rounding each; then half a step."""
    gen = torch.Generator(device="cuda").manual_seed(18)
    pages = -(-n // 1024)
    k, v = (torch.zeros(pages, 1, 1024, 64, dtype=E4, device="cuda") for _ in range(2))
    row = (200.0 * torch.randn(64, generator=gen, device="cuda")).clamp(-448, 448).to(E4)
    v[:] = row
    q = torch.randn(1, 3, 64, generator=gen, device="cuda").to(BF)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = KVCache(k, v, v_scale=scale).attend(q, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    ref = f64(row) * float(np.float32(scale))
    lim = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6) + 2.0 ** -134
    assert np.all(np.abs(f64(out[0]) - ref) <= lim), float((np.abs(f64(out[0]) - ref) / lim).max())


def test_a_nan_query_shows_in_both_results():
    """In its own head alone, in one launch and in two."""
    for lengths in ([40, 20, 3], [700, 9000, 3]):
        c = Case(lengths, 8, 2, 128, seed=19)
        want, lse = (x.clone() for x in c.check())
        for b, h in ((0, 1), (1, 6)):
            q = c.q.clone()
            q[b, h, 17] = math.nan
            l2 = torch.empty_like(lse)
            got = c.cache.attend(q, c.table, c.lengths, lse=l2)
            torch.cuda.synchronize()
            assert torch.isnan(got[b, h]).all() and torch.isnan(l2[b, h])
            got[b, h], l2[b, h] = want[b, h], lse[b, h]
            assert torch.equal(got, want) and torch.equal(l2, lse)


def test_one_workspace_for_every_batch():
    """Sized for the largest; more than 1024 requests go whole and need 256 bytes of it."""
    c = Case([100, 9000] + [5] * 1098, 8, 2, 64, seed=21)
    want, _ = c.check(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    ws = c.cache.attend_workspace(1100, 8)
    for b in (1100, 1024, 300, 2, 1):
        got = c.cache.attend(c.q[:b], c.table[:b], c.lengths[:b], workspace=ws)
        torch.cuda.synchronize()
        # cut elsewhere: half a step each
        assert torch.allclose(got.float(), want[:b].float(), rtol=2.0 ** -6, atol=1e-4), b


def _way(c, window=0):
    """(units, whether the call splits them): a plan of pieces for up to 1024 requests whose
    pages hold more tiles of 32 tokens than the least of a piece."""
    b, hq, _ = c.q.shape
    hk, page = c.k.shape[1:3]
    units = b * hk * -(-(hq // hk) // 16)
    tokens = c.table.shape[1] * page
    tokens = min(window + 31, tokens) if window else tokens
    return units, b <= 1024 and -(-tokens // 32) > min(128, max(4, units // 8))


@pytest.mark.parametrize("hq", [1, 3, 5, 7, 20])
@pytest.mark.parametrize("d", [64, 96, 128, 208, 256])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_many_units_in_pieces(hq, d, dtype):
    """Above 64 units a wave joins a head: any number of heads, one and two passes over D,
    pieces beyond the ones asked for ahead."""
    rng = np.random.default_rng(hq + d)
    lengths = [int(n) for n in rng.integers(0, 150, 70)]
    lengths[11], lengths[40] = 3000, 5000
    c = Case(lengths, hq, 1, d, page=32, dtype=dtype, seed=hq)
    units, split = _way(c)
    assert units > 64 and split
    c.check()


@pytest.mark.parametrize("batch", [65, 257, 300, 700, 1023, 1024])
def test_plans_of_many_requests(batch):
    rng = np.random.default_rng(batch)
    lengths = [int(n) for n in rng.integers(0, 40, batch)]
    lengths[batch // 3], lengths[-1] = 4500, 6000
    for window in (0, 5000):
        c = Case(lengths, 6, 2, 64, page=64, seed=batch)
        units, split = _way(c, window)
        assert units == 2 * batch and split
        c.check(window=window)


@pytest.mark.parametrize("batch,n,hq,hk", [(5, 400, 8, 2), (5, 9000, 8, 2), (70, 700, 4, 1), (70, 3000, 20, 1), (1100, 100, 4, 2)])
def test_equal_requests_have_equal_bits(batch, n, hq, hk):
    c = Case([n], hq, hk, 64, seed=20)
    table, lengths, q = c.table.repeat(batch, 1), c.lengths.repeat(batch), c.q.repeat(batch, 1, 1)
    lse = torch.empty(batch, hq, device="cuda")
    out = c.cache.attend(q, table, lengths, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    ref = f64(c.check()[0][0])
    # the request alone may be cut elsewhere: each half a step off, and both within the sums' errors
    assert np.all(np.abs(f64(out[0]) - ref) <= 2.0 ** -6 * np.abs(ref) + 1e-4)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 + 5, 2 ** 64 + 1])
def test_windows_beyond_32_bits(window):
    """As large as any request, and no window of the low 32 bits; the negative ones are refused."""
    c = Case([300, 70, 0], seed=22)
    want = c.cache.attend(c.q, c.table, c.lengths)
    got = c.cache.attend(c.q, c.table, c.lengths, window=window)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(MoeQuantError):
        c.cache.attend(c.q, c.table, c.lengths, window=-window)


def test_a_table_beyond_32_bits_of_pages():
    c = Case([300], seed=23)
    wide = torch.empty(1, 2 ** 32 + c.table.shape[1], dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    with pytest.raises(MoeQuantError):
        c.cache.attend(c.q, wide, c.lengths)
