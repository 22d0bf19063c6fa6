"""A decoder block's decode step through the framework alone: norm, the fused
projection, append with rotation, attention over the pages, the projection back,
norm, and the gated expert layer, eager and captured."""
import numpy as np
import pytest
import torch

from oracle import attention as oattn
from oracle import formats
from oracle import linear as olin
from weight_quantized_moe_amd import Gate, KVCache, Linear, ResidualNorm, Rotary

from gpu_helpers import GpuLayer, random_layer

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H, HQ, HK, D, PAGE, PAGES = 256, 8, 2, 64, 16, 40


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _weight(n, k, gen):
    w = 0.05 * torch.randn(n // 128, 128, k // 128, 128, generator=gen, device="cuda")
    s = w.abs().amax((1, 3)) / 448
    codes = (w / s[:, None, :, None]).to(E4).view(torch.uint8).view(n, k)
    return codes.contiguous(), s.contiguous()


class Block:
    def __init__(self, dtype):
        gen = torch.Generator(device="cuda").manual_seed(3)

        def rn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.wqkv, self.wo = _weight((HQ + 2 * HK) * D, H, gen), _weight(H, HQ * D, gen)
        self.qkv, self.o = Linear(*self.wqkv), Linear(*self.wo)
        self.before = ResidualNorm(H, pre_weight=(1 + 0.1 * rn(H)).to(BF))
        self.after = ResidualNorm(H, pre_weight=(1 + 0.1 * rn(H)).to(BF))
        self.qn, self.kn = ((1 + 0.1 * rn(D)).to(BF) for _ in range(2))
        self.table = Rotary.table(1000, D)
        self.rotary = Rotary(D, self.table, q_norm=self.qn, k_norm=self.kn)
        self.k, self.v = (torch.zeros(PAGES, HK, PAGE, D, dtype=dtype, device="cuda") for _ in range(2))
        self.cache = KVCache(self.k, self.v, **(dict(k_scale=0.05, v_scale=0.02) if dtype == E4 else {}))
        self.layer = GpuLayer(*random_layer(formats.FP8, 5, 8, H, 128), 2).layer
        self.gate = Gate(8, 2, score="sigmoid")
        self.router = (0.1 * rn(8, H)).to(BF)

    def step(self, stream, positions, slots, table, lengths, keep=None):
        _, x = self.before.forward(None, stream)
        qkv = self.qkv.forward(x)
        t = len(qkv)
        q, k, v = (p.view(t, -1, D) for p in qkv.split([HQ * D, HK * D, HK * D], 1))
        q = self.cache.append(self.rotary, q, k, v, positions, slots)
        a = self.cache.attend(q, table, lengths)
        y = self.o.forward(a.view(t, HQ * D))
        stream, n = self.after.forward(y, stream)
        out = self.layer.forward_gated(self.gate, n, router_w=self.router, residual=stream)
        if keep is not None:
            keep.update(x=x, qkv=qkv, q=q, a=a, y=y, n=n, out=out)
        return out


def _inputs(i, batch, table, gen):
    """Step i of requests of different ages."""
    age = torch.arange(batch, device="cuda") * 7 + i
    slots = table.gather(1, (age // PAGE)[:, None])[:, 0] * PAGE + age % PAGE
    return (torch.randn(batch, H, generator=gen, device="cuda").to(BF), age.to(torch.int32), slots.to(torch.int32),
            (age + 1).to(torch.int32))


@pytest.mark.parametrize("dtype", [BF, E4])
def test_decode_steps_of_a_block(dtype):
    batch, blk = 5, Block(dtype)
    gen = torch.Generator(device="cuda").manual_seed(4)
    table = torch.randperm(PAGES, generator=gen, device="cuda")[:batch * 8].view(batch, 8)
    t32 = table.to(torch.int32).contiguous()
    # prompts first: what is older than a request's first step, appended in one call
    age0 = torch.arange(batch, device="cuda") * 7
    req = torch.repeat_interleave(torch.arange(batch, device="cuda"), age0)
    pos = torch.cat([torch.arange(int(a), device="cuda") for a in age0])
    rows = torch.randn(len(req), (HQ + 2 * HK) * D, generator=gen, device="cuda").to(BF)
    q, k, v = (p.view(len(req), -1, D) for p in rows.split([HQ * D, HK * D, HK * D], 1))
    blk.cache.append(blk.rotary, None, k, v, pos.to(torch.int32),
                     (table[req, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32))
    for i in range(20):
        x, p, s, n = _inputs(i, batch, table, gen)
        keep = {}
        blk.step(x, p, s, t32, n, keep)
        torch.cuda.synchronize()
        # each stage on what the one before gave: its output's rounding and some FP32 ones
        y, size, largest = olin.forward(f64(keep["x"]), blk.wqkv[0].cpu().numpy(), blk.wqkv[1].cpu().numpy())
        assert np.all(np.abs(f64(keep["qkv"]) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -14 * size + 2.0 ** -9 * largest)
        qkv = f64(keep["qkv"])[:, :HQ * D].reshape(batch, HQ, D)
        angles = blk.table.cpu().numpy().astype(np.float64)[p.cpu().numpy()]
        q = oattn.turn(qkv, f64(blk.qn), 1e-6, angles, False)
        assert np.all(np.abs(f64(keep["q"]) - q) <= 2.0 ** -8 * np.abs(q) + 1e-5)
        a, _, spread, _ = oattn.attend(f64(keep["q"]), f64(blk.k) * blk.cache.desc.k_scale,
                                       f64(blk.v) * blk.cache.desc.v_scale, t32.cpu().numpy(), n.cpu().numpy(), D ** -0.5)
        assert np.all(np.abs(f64(keep["a"]) - a) <= 2.0 ** -8 * np.abs(a) + 2.0 ** -14 * spread)
        y, size, largest = olin.forward(f64(keep["a"]).reshape(batch, -1), blk.wo[0].cpu().numpy(),
                                        blk.wo[1].cpu().numpy())
        assert np.all(np.abs(f64(keep["y"]) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -14 * size + 2.0 ** -9 * largest)
        assert torch.isfinite(keep["out"].float()).all()


def test_a_captured_step_replays_as_the_eager_one():
    batch, blk, ref = 4, Block(BF), Block(BF)
    gen = torch.Generator(device="cuda").manual_seed(6)
    table = torch.randperm(PAGES, generator=gen, device="cuda")[:batch * 8].view(batch, 8)
    t32 = table.to(torch.int32).contiguous()
    steps = [_inputs(i, batch, table, gen) for i in range(6)]
    # what lies before each request's first step is whatever the pages hold (zeros)
    x, p, s, n = (a.clone() for a in steps[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk.step(x, p, s, t32, n)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = blk.step(x, p, s, t32, n)
    for step in steps:
        for mine, new in zip((x, p, s, n), step):
            mine.copy_(new)
        want = ref.step(*step[:3], t32, step[3])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(blk.k, ref.k) and torch.equal(blk.v, ref.v)
