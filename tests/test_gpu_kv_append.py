"""Queries, keys and values on their way into a paged cache, on the GPU against the
float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import attention as oattn
from oracle import codecs
from weight_quantized_moe_amd import KVCache, MoeQuantError, Rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
P = 5000


def f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


class Case:
    def __init__(self, t, hq, hk, d, r, page, dtype=BF, inter=False, norm=True, fused=True, seed=0, size=1.0, ks=1.0, vs=1.0,
                 extra=3, eps=1e-6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.t, self.hq, self.hk, self.d, self.r, self.page, self.inter, self.eps = t, hq, hk, d, r, page, inter, eps
        if fused:
            qkv = (size * randn(gen, t, (hq + 2 * hk) * d)).to(BF)
            a, b = hq * d, (hq + hk) * d
            self.q, self.k, self.v = (x.view(t, -1, d) for x in (qkv[:, :a], qkv[:, a:b], qkv[:, b:]))
        else:
            self.q, self.k, self.v = ((size * randn(gen, t, h, d)).to(BF) for h in (hq, hk, hk))
        self.qn = (1 + 0.3 * randn(gen, d)).to(BF) if norm else None
        self.kn = (1 + 0.3 * randn(gen, d)).to(BF) if norm else None
        self.table = Rotary.table(P, r, base=1e5) if r else None
        self.rotary = Rotary(d, self.table, interleaved=inter, q_norm=self.qn, k_norm=self.kn, eps=eps)
        pages = -(-t // page) + extra
        self.kc, self.vc = (randn(gen, pages, hk, page, d).to(dtype) for _ in range(2))
        self.cache = KVCache(self.kc, self.vc, k_scale=ks, v_scale=vs)
        self.ks, self.vs = ks, vs
        self.slots = torch.randperm(pages * page, generator=gen, device="cuda")[:t].to(torch.int32)
        self.positions = torch.randint(0, P, (t,), generator=gen, device="cuda").to(torch.int32)

    def row_limits(self, x, weight, ref, angles):
        """The norm: D products and sums of squares halved by the root, the quotient and
        two products; the rotation: two products and a sum of magnitudes |a| + |b|:
        (D / 32 + 12) roundings of 2^-24 of |row value| + |its partner|."""
        c = (self.d / 32 + 12) * 2.0 ** -24
        plain = np.abs(oattn.turn(x, weight, self.eps, None, False))
        both = plain.copy()
        if angles is not None:
            h = self.r // 2
            one, two = (slice(0, self.r, 2), slice(1, self.r, 2)) if self.inter else (slice(0, h), slice(h, self.r))
            both[..., one], both[..., two] = plain[..., one] + plain[..., two], plain[..., one] + plain[..., two]
        return c * both

    def check(self, q=True, q_out=None, stream=None):
        kc, vc = self.kc.clone(), self.vc.clone()
        t, hq = self.t, self.hq
        out = torch.full((t + 1, hq, self.d), 7.0, dtype=BF, device="cuda")
        before = out.clone()
        got = self.cache.append(self.rotary, self.q if q else None, self.k, self.v, self.positions, self.slots,
                                q_out=out[:t] if q else None)
        torch.cuda.synchronize()
        slots, pos = self.slots.cpu().numpy(), self.positions.cpu().numpy()
        total = self.kc.shape[0] * self.page
        live = (slots >= 0) & (slots < total)
        if self.r:
            live &= (pos >= 0) & (pos < P)
        angles = None if self.table is None else self.table.cpu().numpy().astype(np.float64)[np.clip(pos, 0, P - 1)]
        if q:
            x = f64(self.q)
            ref = oattn.turn(x, f64(self.qn), self.eps, angles, self.inter)
            most = self.row_limits(x, f64(self.qn), ref, angles)
            off = np.abs(f64(out[:t]) - ref)
            lim = most + 2.0 ** -8 * (np.abs(ref) + most) + 1e-38
            assert np.all(off[live] <= lim[live]), float((off / lim)[live].max())
            dead = torch.from_numpy(np.append(~live, True)).cuda()
            assert torch.equal(bits(out)[dead], bits(before)[dead])
        else:
            assert got is None
        # every row of the cache that no token names stays as it was, bit for bit
        at = torch.from_numpy(slots[live]).long().cuda()
        for cache, old, x, weight, scale, turn in ((self.kc, kc, self.k, self.kn, self.ks, True),
                                                   (self.vc, vc, self.v, None, self.vs, False)):
            rows, olds = (bits(c).transpose(1, 2).reshape(total, self.hk, self.d) for c in (cache, old))
            keep = torch.ones(total, dtype=torch.bool, device="cuda")
            keep[at] = False
            assert torch.equal(rows[keep], olds[keep])
            xs = f64(x)
            ref = oattn.turn(xs, f64(weight), self.eps, angles if turn else None, self.inter)[live]
            most = self.row_limits(xs, f64(weight), ref, angles if turn else None)[live]
            new = f64(rows[at].view(cache.dtype))
            if cache.dtype == BF:
                lim = most + 2.0 ** -8 * (np.abs(ref) + most) + 1e-38
            else:
                # the quotient's rounding; half a step of E4M3: 2^-4 of the value, 2^-10 at least
                ref, most = ref / scale, most / scale + 2.0 ** -24 * np.abs(ref) / scale
                cut = np.clip(ref, -448, 448)
                lim = most + np.maximum(2.0 ** -4 * (np.abs(cut) + most), 2.0 ** -10)
                ref = cut
            off = np.abs(new - ref)
            assert np.all(off <= lim), float((off / lim).max())
        return out[:t]


@pytest.mark.parametrize("d,r", [(16, 16), (16, 0), (32, 16), (48, 48), (64, 64), (64, 32), (80, 32), (96, 64), (112, 112),
                                 (128, 128), (128, 64), (128, 16), (160, 96), (192, 192), (192, 64), (240, 240), (256, 256),
                                 (256, 64)])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_head_sizes(d, r, dtype):
    for inter in (False, True):
        for norm in (False, True):
            kw = dict(ks=0.5, vs=1.5) if dtype == E4 else {}
            Case(37, 6, 3, d, r, 8, dtype, inter, norm, seed=d + r, **kw).check()


@pytest.mark.parametrize("t", [1, 2, 3, 17, 64, 301, 2000])
@pytest.mark.parametrize("page", [1, 2, 16, 64, 1024])
def test_tokens_and_pages(t, page):
    for dtype in (BF, E4):
        Case(t, 8, 2, 128, 128, page, dtype, fused=t % 2 == 1, seed=t).check()


@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 4), (12, 12), (40, 8), (7, 7), (64, 1), (5, 1), (1024, 1024)])
def test_heads(hq, hk):
    for q in (True, False):
        Case(5, hq, hk, 64, 64, 16, seed=hq).check(q=q)


def test_far_values_and_scales():
    for dtype, ks, vs in ((BF, 1.0, 1.0), (E4, 0.01, 0.003), (E4, 100.0, 1e-6), (E4, 1e10, 1e-3)):
        for size in (1e-4, 1.0, 1000.0):
            Case(40, 4, 2, 128, 128, 16, dtype, norm=False, size=size, ks=ks, vs=vs).check()
    c = Case(9, 4, 2, 64, 64, 16, norm=True)
    c.k[3] = 0
    c.q[3] = 0
    c.check()
    c = Case(9, 4, 2, 64, 64, 16, E4, norm=False)
    c.v[2, 1, 5], c.v[4, 0, 3] = float("nan"), float("inf")
    c.cache.append(c.rotary, c.q, c.k, c.v, c.positions, c.slots)
    torch.cuda.synchronize()
    rows = c.vc.float().transpose(1, 2).reshape(-1, 2, 64)
    assert torch.isnan(rows[c.slots[2].long(), 1, 5]) and rows[c.slots[4].long(), 0, 3] == 448


@pytest.mark.parametrize("dtype", [BF, E4])
def test_padding_and_what_is_out_of_range(dtype):
    c = Case(60, 4, 2, 96, 64, 16, dtype, seed=3)
    total = c.kc.shape[0] * 16
    c.slots[::7] = -1
    c.slots[3] = total
    c.slots[4] = 2 ** 31 - 1
    c.slots[5] = -2 ** 31
    c.positions[10] = -1
    c.positions[11] = P
    c.positions[12] = 2 ** 31 - 1
    c.positions[13] = -2 ** 31
    c.check()
    c = Case(20, 4, 2, 96, 64, 16, dtype, seed=3)
    c.slots[:] = -1
    c.check()


def test_a_slot_named_twice_holds_one_or_the_other():
    c = Case(64, 2, 2, 64, 64, 16, seed=4)
    c.slots[:] = 5
    c.cache.append(c.rotary, c.q, c.k, c.v, c.positions, c.slots)
    torch.cuda.synchronize()
    row = c.vc[0, :, 5]
    for part in range(0, 64, 8):
        for h in range(2):
            assert (c.v[:, h, part:part + 8] == row[h, part:part + 8]).all(1).any()


def test_queries_in_their_own_buffer():
    for d, r, inter in ((128, 128, False), (96, 64, False), (64, 64, True)):
        c = Case(33, 8, 2, d, r, 16, inter=inter, fused=False)
        want = c.check().clone()
        q = c.q.clone()
        got = c.cache.append(c.rotary, q, c.k, c.v, c.positions, c.slots, q_out=q)
        torch.cuda.synchronize()
        assert got is q and torch.equal(q, want)


def test_one_token_of_a_strided_view():
    c = Case(1, 8, 2, 64, 64, 16)
    c.check()
    c = Case(10, 8, 2, 64, 64, 16)
    c.q, c.k, c.v = (x[3:4] for x in (c.q, c.k, c.v))
    c.t, c.slots, c.positions = 1, c.slots[:1], c.positions[:1]
    c.check()


def test_a_cache_beyond_32_bits_of_offsets():
    """Rows whose element offsets pass 2^31 and 2^32."""
    pages, hk, page, d = 70000, 4, 64, 256                # 4.6e9 values, 9.2 GB each
    kc, vc = (torch.zeros(pages, hk, page, d, dtype=BF, device="cuda") for _ in range(2))
    cache, rot = KVCache(kc, vc), Rotary(d)
    k, v = (torch.randn(4, hk, d, device="cuda").to(BF) for _ in range(2))
    slots = torch.tensor([0, 32767 * page + 63, 65536 * page + 1, pages * page - 1], dtype=torch.int32, device="cuda")
    cache.append(rot, None, k, v, None, slots)
    torch.cuda.synchronize()
    s = slots.long()
    assert torch.equal(kc[s // page, :, s % page], k) and torch.equal(vc[s // page, :, s % page], v)
    # only those rows: counted without a copy of the cache
    assert int(kc.count_nonzero()) == int(k.count_nonzero())
    table = (s // page).to(torch.int32)[:, None].contiguous()
    q = torch.randn(4, hk, d, device="cuda").to(BF)
    out = cache.attend(q, table, torch.tensor([1, 64, 2, 64], dtype=torch.int32, device="cuda"), scale=0.01)
    torch.cuda.synchronize()
    want = []
    for i in range(4):
        n = (1, 64, 2, 64)[i]
        kk, vv = kc[s[i] // page, :, :n].double(), vc[s[i] // page, :, :n].double()
        p = torch.softmax((q[i].double()[:, None] * kk).sum(2) * 0.01, 1)
        want.append((p[..., None] * vv).sum(1))
    assert torch.allclose(out.double(), torch.stack(want), rtol=2.0 ** -7, atol=1e-3)


def test_streams_and_graph():
    c = Case(50, 8, 2, 128, 128, 16)
    want = c.check().clone()
    k, v = c.kc.clone(), c.vc.clone()
    c.kc.zero_(), c.vc.zero_()
    torch.cuda.synchronize()
    got = c.cache.append(c.rotary, c.q, c.k, c.v, c.positions, c.slots, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    at = c.slots.long()
    assert torch.equal(got, want) and torch.equal(c.kc[at // 16, :, at % 16], k[at // 16, :, at % 16])
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        c.cache.append(c.rotary, c.q, c.k, c.v, c.positions, c.slots, q_out=out)
    for rep in range(3):
        c.slots.copy_(torch.randperm(c.kc.shape[0] * 16, device="cuda")[:50])
        c.kc.zero_(), out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = c.slots.long()
        assert torch.equal(out, want) and torch.equal(c.kc[now // 16, :, now % 16], k[at // 16, :, at % 16])
        assert int(c.kc.count_nonzero()) == int(k[at // 16, :, at % 16].count_nonzero())


def test_no_tokens_and_refusals():
    c = Case(8, 4, 2, 64, 64, 16)
    none = c.cache.append(c.rotary, c.q[:0], c.k[:0], c.v[:0], c.positions[:0], c.slots[:0])
    assert none.shape == (0, 4, 64)
    good = dict(q=c.q, k=c.k, v=c.v, positions=c.positions, slots=c.slots)
    for over in (dict(q=c.q.float()), dict(q=c.q[:7]), dict(k=c.k[:, :1]), dict(k=c.k[..., :32]), dict(v=c.v.cpu()),
                 dict(positions=None), dict(positions=c.positions.long()), dict(slots=c.slots.long()), dict(slots=c.slots[:7]),
                 dict(slots=c.slots.cpu()), dict(q_out=torch.empty(8, 4, 64, device="cuda")), dict(q=None, q_out=c.q),
                 dict(k=c.k.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=c.q[0])):
        with pytest.raises(ValueError):
            c.cache.append(c.rotary, **dict(good, **over))
    with pytest.raises(MoeQuantError):
        c.cache.append(Rotary(128), **good)
    odd = torch.zeros(8, 4 * 64 + 4, dtype=BF, device="cuda")[:, :256].view(8, 4, 64)
    with pytest.raises(MoeQuantError):                    # tokens no multiple of 8 values apart
        c.cache.append(c.rotary, **dict(good, q=odd))
    with pytest.raises(MoeQuantError):                    # in place, but tokens apart
        _in_place(c)
    for k, v, over in ((c.kc, c.vc, dict(k_scale=0.5)), (c.kc[:, :, :12].contiguous(), c.vc[:, :, :12].contiguous(), {})):
        with pytest.raises(MoeQuantError):
            KVCache(k, v, **over)


def _in_place(c):
    from weight_quantized_moe_amd import binding
    st = c.cache._lib.moe_quant_kv_append(c.cache._ref, c.rotary._ref, 4, c.q.data_ptr(), c.q.stride(0), c.k.data_ptr(),
                                          c.k.stride(0), c.v.data_ptr(), c.v.stride(0), c.positions.data_ptr(),
                                          c.slots.data_ptr(), 8, c.q.data_ptr(), None)
    binding._check(c.cache._lib, st)


@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-42, 1e-40, 2.0 ** -128, 3e-39, 2.0 ** -126, 1e-36, 1e-27, 2.0 ** -9, 0.7,
                                   1.9999999, 1e20, 2.0 ** 126, 2.0 ** 127, 3.4e38])
def test_codes_of_scales_of_every_size(scale):
    """RNE-to-E4M3 of one FP32 division, bit for bit: zeros, values of every code, ties and
    what saturates, also where the scale's reciprocal is infinite or subnormal."""
    gen, s = torch.Generator().manual_seed(11), np.float32(scale)
    steps = torch.randn(40, 4, 64, generator=gen) * torch.exp2(torch.randint(-12, 10, (40, 4, 64), generator=gen))
    steps[10:25] = torch.randint(-470, 471, (15, 4, 64), generator=gen).float()
    steps[30:33] = 0
    x = (steps.double() * float(s)).clamp(-3e38, 3e38).float().to(BF)
    c = Case(40, 2, 2, 64, 0, 16, E4, norm=False, ks=scale, vs=scale)
    c.k, c.v = x[:, :2].contiguous().cuda(), x[:, 2:].contiguous().cuda()
    c.cache.append(c.rotary, None, c.k, c.v, None, c.slots)
    torch.cuda.synchronize()
    at = c.slots.long().cpu()
    for cache, new in ((c.kc, x[:, :2]), (c.vc, x[:, 2:])):
        got = bits(cache).cpu()[at // 16, :, at % 16].numpy()
        with np.errstate(over="ignore"):
            want = codecs.quantize_e4m3((new.float().numpy() / s).astype(np.float64))
        assert np.array_equal(got & 127, want & 127), np.argwhere((got ^ want) & 127)[:4]
        assert np.array_equal((got >> 7)[want & 127 > 0], (want >> 7)[want & 127 > 0])


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("d,r", [(16, 16), (64, 64), (96, 0), (128, 64), (256, 256)])
def test_norms_of_large_heads(d, r, dtype):
    """Heads whose squares add up beyond FP32's range, beside ordinary ones and zeros."""
    for size in (2.0 ** 59, 1e19, 1e25, 5e37):
        for inter in (False, True):
            c = Case(21, 5, 3, d, r, 16, dtype, inter, fused=False, seed=d, size=size)
            gen = torch.Generator(device="cuda").manual_seed(1)
            for x in (c.q, c.k):
                x[3] = randn(gen, *x[3].shape).to(BF)
                x[4, 0] = 0
                x[5, 1] = torch.finfo(BF).max
                x[6, :, 1:] = 0
                x[7, 0] *= 2.0 ** -60
            c.check()
