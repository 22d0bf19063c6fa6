"""Cases of the operators of a decoder block in front of the expert layer: the
matrix product on E4M3 weights with a scale for each block of 128, keys and
values appended to a paged cache with the per-head norm and the position
rotation on the way, and the attention of one new token over that cache.

``run`` computes a case in its plain form (elementary torch operations) where
``own`` is false, and through the package's entry points where it is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
POSITIONS = 40960        # rows of the rotation's table


def _linear(name, tokens, n, k, **over):
    case = dict(op="linear", tokens=tokens, n=n, k=k, out="bfloat16", residual=False)
    return dict(case, **({"name": name} if name else {}), **over)


def _append(name, tokens, **over):
    case = dict(op="append", tokens=tokens, q_heads=32, kv_heads=4, head_dim=128, rotary=128, interleaved=False,
                norm=True, page=16, cache="bfloat16", prompt=False, padded=False)
    case.update(over)
    return dict(case, **({"name": name} if name else {}))


def _attend(name, batch, longest, **over):
    case = dict(op="attend", batch=batch, shortest=longest, longest=longest, q_heads=32, kv_heads=4, head_dim=128,
                page=16, cache="bfloat16", window=0)
    case.update(over)
    return dict(case, **({"name": name} if name else {}))


def listed():
    return [
        # one token of one request through a fused q, k and v projection
        _linear("linear one token", 1, 5120, 2048),
        # a decode step of 64 requests: the projection behind the attention, onto the residual stream
        _linear("linear decode 64", 64, 2048, 4096, residual=True),
        # a ragged chunk of a prompt on sizes that fill no block of 128, in 32 bits
        _linear("linear ragged chunk", 777, 1000, 2064, out="float32"),
        # prompts of a batch through the q, k and v projection
        _linear("linear prefill", 16384, 5120, 2048),
        # a decode step of 64 requests at far positions
        _append("append decode 64", 64),
        # a padded chunk, heads of 96 of which 64 turn in neighbouring pairs, pages of 64 tokens in 8 bits
        _append("append ragged chunk", 3001, q_heads=24, kv_heads=24, head_dim=96, rotary=64, interleaved=True,
                norm=False, page=64, cache="float8_e4m3fn", prompt=True, padded=True),
        # prompts of a batch
        _append("append prefill", 16384, prompt=True),
        # one request of ordinary length: latency
        _attend("attend one request", 1, 1000),
        # a batch of requests of every length
        _attend("attend decode 64", 64, 8192, shortest=1),
        # heads of 96 without sharing, a sliding window, an odd number of requests
        _attend("attend window", 33, 3000, shortest=0, q_heads=12, kv_heads=12, head_dim=96, page=8, window=1000),
        # a few requests over long documents, the cache in 8 bits
        _attend("attend long", 4, 131072, shortest=100000, page=64, cache="float8_e4m3fn"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_heads(rng):
    kv = rng.choice((1, 2, 4, 8, 16))
    return dict(q_heads=kv * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16, 24) if kv * g <= 64]), kv_heads=kv,
                head_dim=rng.choice((64, 64, 80, 96, 128, 128, 128, 192, 256)), page=rng.choice((1, 8, 16, 32, 64, 128)),
                cache=rng.choice(("bfloat16", "float8_e4m3fn")))


def draw(rng):
    op = rng.choice(("linear", "append", "attend"))
    if op == "linear":
        n, k = _log_int(rng, 64, 16384), 16 * _log_int(rng, 4, 1024)
        n, k = rng.choice((n, -(-n // 128) * 128)), rng.choice((k, -(-k // 128) * 128))
        most = 16384 * 5120 * 2048 // (n * k)
        return _linear("", _log_int(rng, 1, min(16384, most)), n, k, out=rng.choice(("bfloat16", "bfloat16", "float32")),
                       residual=rng.random() < 0.4)
    heads = _draw_heads(rng)
    d, kv = heads["head_dim"], heads["kv_heads"]
    if op == "append":
        most = 16384 * 40 * 128 // ((heads["q_heads"] + 2 * kv) * d)
        return _append("", _log_int(rng, 1, min(65536, most)), rotary=rng.choice((d, d, d // 32 * 16, 0)),
                       interleaved=rng.random() < 0.3, norm=rng.random() < 0.5, prompt=rng.random() < 0.7,
                       padded=rng.random() < 0.3, **heads)
    # tokens of all requests: at most half a gigabyte of keys and values in 16 bits
    most = min(1 << 18, (1 << 29) // (4 * kv * d))
    batch = _log_int(rng, 1, min(256, most))
    longest = _log_int(rng, 1, most // batch)
    return _attend("", batch, longest, shortest=rng.choice((longest, longest // 2, 0)),
                   window=rng.choice((0, 0, 0, _log_int(rng, 1, 4096))), **heads)


def _dtype(name):
    return getattr(torch, name)


def _sequences(lengths, page, gen, dev):
    """A table of pages [requests, most pages] for requests of these lengths, in no order, and the number of
    pages of the cache; entries that no token needs are -1."""
    counts = [-(-n // page) for n in lengths]
    total, most = max(1, sum(counts)), max(1, max(counts))
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lengths), most), -1, dtype=torch.int32, device=dev)
    row = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(counts)).to(dev)
    col = torch.cat([torch.arange(c) for c in counts] or [torch.arange(0)]).to(dev)
    table[row, col] = order[:sum(counts)]
    return table, total


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        nb, kb = -(-n // 128), -(-k // 128)
        # rows of different sizes with a few channels far above the others, as hidden states have them
        x = randn(t, k) * torch.exp(0.5 * randn(t, 1))
        x[:, torch.randint(0, k, (max(1, k // 256),), generator=gen, device=dev)] *= 20.0
        s["x"] = x.bfloat16()
        w = 0.02 * randn(nb * 128, kb * 128)
        w[n:], w[:, k:] = 0, 0
        blocks = w.view(nb, 128, kb, 128)
        scale = blocks.abs().amax((1, 3)) / E4M3_MAX
        codes = (blocks / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(nb * 128, kb * 128)
        s["w"], s["scale"] = codes[:n, :k].contiguous(), scale.contiguous()
        s["r"] = (4.0 * randn(t, n)).bfloat16() if case["residual"] else None
        if own:
            from weight_quantized_moe_amd import Linear
            s["linear"] = Linear(s["w"], s["scale"], out_dtype=_dtype(case["out"]))
            s["ws"] = s["linear"].workspace(t)
            s["y"] = torch.empty((t, n), dtype=_dtype(case["out"]), device=dev)
        return s

    hq, hk, d, page, kind = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"], _dtype(case["cache"])
    if case["op"] == "append":
        t, r = case["tokens"], case["rotary"]
        requests = -(-t // 4096) if case["prompt"] else t
        at = torch.randint(0, POSITIONS - 4096, (requests,), generator=host)
        # prompts: runs of consecutive positions; decoding: one token of each request
        lengths = [min(4096, t - 4096 * i) for i in range(requests)] if case["prompt"] else [1] * t
        position = torch.cat([at[i] + torch.arange(m) for i, m in enumerate(lengths)])
        table, pages = _sequences([-(-m // page) * page + page for m in lengths], page, gen, dev)
        first = at % page
        col = torch.cat([(first[i] + torch.arange(m)) for i, m in enumerate(lengths)]).to(dev)
        row = torch.repeat_interleave(torch.arange(requests), torch.tensor(lengths)).to(dev)
        slots = table[row, col // page] * page + col % page
        if case["padded"]:
            slots[torch.rand(t, generator=gen, device=dev) < 0.1] = -1
        s["slots"], s["positions"] = slots.to(torch.int32), position.to(dev, torch.int32)
        qkv = randn(t, (hq + 2 * hk) * d).bfloat16()
        cut = (hq * d, (hq + hk) * d)
        s["q"] = qkv[:, :cut[0]].view(t, hq, d)
        s["k"] = qkv[:, cut[0]:cut[1]].view(t, hk, d)
        s["v"] = qkv[:, cut[1]:].view(t, hk, d)
        s["qn"] = (1.0 + 0.2 * randn(d)).bfloat16() if case["norm"] else None
        s["kn"] = (1.0 + 0.2 * randn(d)).bfloat16() if case["norm"] else None
        s["table"] = None
        if r:
            rate = 1e6 ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r)
            angle = torch.arange(POSITIONS, device=dev, dtype=torch.float64)[:, None] * rate
            s["table"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["kc"] = randn(pages, hk, page, d).to(kind)
        s["vc"] = randn(pages, hk, page, d).to(kind)
        s["q_out"] = torch.zeros((t, hq, d), dtype=torch.bfloat16, device=dev)
        if own:
            from weight_quantized_moe_amd import KVCache, Rotary
            s["rotary"] = Rotary(d, s["table"], interleaved=case["interleaved"], q_norm=s["qn"], k_norm=s["kn"])
            s["cache"] = KVCache(s["kc"], s["vc"])
        return s

    b = case["batch"]
    lengths = torch.randint(case["shortest"], case["longest"] + 1, (b,), generator=host).tolist()
    table, pages = _sequences(lengths, page, gen, dev)
    s["block_table"], s["lengths"] = table, torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["q"] = (1.5 * randn(b, hq, d)).bfloat16()
    s["kc"] = torch.empty((pages, hk, page, d), dtype=kind, device=dev)
    s["vc"] = torch.empty_like(s["kc"])
    step = max(1, (1 << 26) // (hk * page * d))
    for c in (s["kc"], s["vc"]):
        for i in range(0, pages, step):
            c[i:i + step] = randn(*c[i:i + step].shape).to(kind)
    s["scales"] = (0.75, 1.25) if kind is not torch.bfloat16 else (1.0, 1.0)
    if own:
        from weight_quantized_moe_amd import KVCache
        s["cache"] = KVCache(s["kc"], s["vc"], k_scale=s["scales"][0], v_scale=s["scales"][1])
        s["ws"] = s["cache"].attend_workspace(b, hq)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, hq), dtype=torch.float32, device=dev)
    return s


def _plain_linear(s):
    n, k = s["w"].shape
    t, kb = s["x"].shape[0], -(-k // 128)
    x = torch.zeros((t, kb * 128), dtype=torch.float32, device=s["x"].device)
    x[:, :k] = s["x"].float()
    x = x.view(t, kb, 128)
    top = x.abs().amax(2, keepdim=True)
    size = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    a = torch.clamp(x / size, -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float() * size
    scale = s["scale"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    w = s["w"].view(torch.float8_e4m3fn).float() * scale
    y = a.view(t, kb * 128)[:, :k] @ w.t()
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(_dtype(s["case"]["out"]))


def _plain_turn(case, x, weight, c, eps=1e-6):
    """Heads x [T, H, D] normed and turned, in float32; c: the table's rows [T, R] or None."""
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps) * weight.float()
    if c is None:
        return x
    r = case["rotary"]
    cos, sin = c[:, None, :r // 2], c[:, None, r // 2:]
    y = x.clone()
    one, two = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    return y


def _plain_append(case, s):
    c = None if s["table"] is None else s["table"][s["positions"].long()]
    q, k = _plain_turn(case, s["q"], s["qn"], c), _plain_turn(case, s["k"], s["kn"], c)
    valid = s["slots"] >= 0
    s["q_out"].copy_(torch.where(valid[:, None, None], q.bfloat16(), s["q_out"]))
    # a padded token writes what the first real one writes
    first = valid.int().argmax()
    slot = torch.where(valid, s["slots"], s["slots"][first]).long()
    for cache, rows in ((s["kc"], k), (s["vc"], s["v"].float())):
        if cache.dtype is not torch.bfloat16:
            rows = torch.clamp(rows, -E4M3_MAX, E4M3_MAX)
        rows = rows.to(cache.dtype).view(torch.int8 if cache.element_size() == 1 else torch.int16)
        rows = torch.where(valid[:, None, None], rows, rows[first])
        raw = cache.view(rows.dtype)
        raw[slot // case["page"], :, slot % case["page"]] = rows
    return s["q_out"], s["kc"], s["vc"]


def _gather(cache, table, most):
    """float32 [B, heads, most, D] of the first tokens of each request."""
    rows = cache[table.clamp(min=0).long()].float()
    b, p, h, n, d = rows.shape
    return rows.permute(0, 2, 1, 3, 4).reshape(b, h, p * n, d)[:, :, :most]


def _plain_attend(case, s):
    b, hq, d = s["q"].shape
    hk, most = case["kv_heads"], max(1, s["block_table"].shape[1] * case["page"])
    at = torch.arange(most, device=s["q"].device)
    length = s["lengths"][:, None]
    seen = at < length
    if case["window"]:
        seen = seen & (at >= length - case["window"])
    outs, lses = [], []
    # some requests at a time, so that their gathered keys and values stay below a gigabyte each
    step = max(1, (1 << 28) // (hk * most * d))
    for i in range(0, b, step):
        part = slice(i, i + step)
        k = _gather(s["kc"], s["block_table"][part], most)
        q = s["q"][part].float().view(-1, hk, hq // hk, d)
        score = q @ k.transpose(2, 3).contiguous() * (s["scales"][0] / math.sqrt(d))
        score = torch.where(seen[part, None, None], score, torch.full_like(score, -math.inf))
        top = score.amax(3, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        p = torch.exp(score - top)
        total = p.sum(3, keepdim=True)
        v = _gather(s["vc"], s["block_table"][part], most)
        o = p @ v * (s["scales"][1] / torch.where(total > 0, total, torch.ones_like(total)))
        outs.append(o.reshape(-1, hq, d).bfloat16())
        lses.append((top + torch.log(total)).reshape(-1, hq))
    return torch.cat(outs), torch.cat(lses)


def run(state):
    s = state
    case = s["case"]
    if case["op"] == "linear":
        if own:
            return s["linear"].forward(s["x"], residual=s["r"], out=s["y"], workspace=s["ws"])
        return _plain_linear(s)
    if case["op"] == "append":
        if own:
            s["cache"].append(s["rotary"], s["q"], s["k"], s["v"], s["positions"], s["slots"], q_out=s["q_out"])
            return s["q_out"], s["kc"], s["vc"]
        return _plain_append(case, s)
    if own:
        out = s["cache"].attend(s["q"], s["block_table"], s["lengths"], window=case["window"], out=s["out"],
                                lse=s["lse"], workspace=s["ws"])
        return out, s["lse"]
    return _plain_attend(case, s)


def work(case):
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        out = 4 if case["out"] == "float32" else 2
        return {"bytes": n * k + 4 * (-(-n // 128)) * (-(-k // 128)) + t * (2 * k + n * (out + 2 * case["residual"])),
                "flops": 2.0 * t * n * k}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    size = 2 if case["cache"] == "bfloat16" else 1
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * (2 * (2 * hq + 2 * hk) * d + 2 * size * hk * d + 4 * case["rotary"] + 8),
                "flops": t * (hq + hk) * (3 * case["rotary"] + 4 * d * case["norm"])}
    mean = 0.5 * (case["shortest"] + case["longest"])
    if case["window"]:
        # lengths spread evenly: the mean of what of each the window leaves
        lo, hi, w = case["shortest"], case["longest"], case["window"]
        mean = sum(min(lo + (hi - lo) * (i + 0.5) / 64, w) for i in range(64)) / 64
    b = case["batch"]
    return {"bytes": b * (mean * (2 * size * hk * d + 4 / case["page"]) + hq * (4 * d + 4)),
            "flops": 4.0 * b * mean * hq * d}


def _exact_linear(case, s):
    t, (n, k) = case["tokens"], s["w"].shape
    y = torch.zeros((t, n), dtype=torch.float64, device=s["x"].device)
    for g, at in enumerate(range(0, k, 128)):
        x = s["x"][:, at:at + 128].float()
        # the scale and the code are defined by one 32-bit division each
        m = x.abs().max(1, keepdim=True).values
        size = torch.where(m == 0, 1.0, m / E4M3_MAX)
        code = torch.div(x, size).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
        w = s["w"][:, at:at + 128].contiguous().view(torch.float8_e4m3fn).double()
        w *= s["scale"][torch.arange(n, device=w.device) // 128, g].double()[:, None]
        y.addmm_(code * size.double(), w.t())
    return y if s["r"] is None else y + s["r"].double()


def _exact_heads(case, x, weight, table, positions):
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.square().sum(2, keepdim=True) / case["head_dim"] + 1e-6) * weight.double()
    if table is None:
        return x
    r = case["rotary"]
    row = table.double()[positions.long()]
    turn = torch.complex(row[:, :r // 2], row[:, r // 2:])[:, None]
    if case["interleaved"]:
        turned = torch.view_as_real(torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2)) * turn)
        return torch.cat((turned.flatten(2), x[..., r:]), 2)
    turned = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
    return torch.cat((turned.real, turned.imag, x[..., r:]), 2)


def _exact_append(case, s):
    q = _exact_heads(case, s["q"], s["qn"], s["table"], s["positions"])
    k = _exact_heads(case, s["k"], s["kn"], s["table"], s["positions"])
    real = torch.nonzero(s["slots"] >= 0)[:, 0]
    q_out = torch.zeros_like(q)
    q_out[real] = q[real]
    caches = []
    for cache, rows in ((s["kc"], k), (s["vc"], s["v"].double())):
        new = cache.double()
        lane = new.transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])
        lane[s["slots"][real].long()] = rows[real]
        caches.append(lane.view(new.shape[0], case["page"], *lane.shape[1:]).transpose(1, 2).contiguous())
    return q_out, caches[0], caches[1]


def _exact_attend(case, s):
    b, hq, d = s["q"].shape
    hk = case["kv_heads"]
    out = torch.zeros((b, hq, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["lengths"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == lo:
            continue
        at = torch.arange(lo, n, device=s["q"].device)
        page = s["block_table"][i, at // case["page"]].long()
        for h in range(hk):
            k, v = (c[page, h, at % case["page"]].double() for c in (s["kc"], s["vc"]))
            mine = slice(h * (hq // hk), (h + 1) * (hq // hk))
            score = (s["q"][i, mine].double() / math.sqrt(d)) @ (k * s["scales"][0]).t()
            lse[i, mine] = torch.logsumexp(score, 1)
            out[i, mine] = torch.softmax(score, 1) @ (v * s["scales"][1])
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)
