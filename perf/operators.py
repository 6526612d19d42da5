"""Timing cases of the attention-side operators: head norms with rotary positions, the 4-bit key/value cache, and
attention over that cache.

Each case is a dict of sizes; ``prepare`` makes what a program holds before the call, ``run`` makes one pass.  With
``own`` false, ``run`` computes the operators from elementary torch operations in 32 bits (64 for angles); with ``own``
true it calls the library.  ``exact`` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decoding step of 16 sequences: latency.  Keys are rotated by the head's Hadamard for the 4-bit cache.
        dict(name="norm_rope_decode", op="norm_rope", tokens=16, q_heads=32, k_heads=8, dim=128, dtype="bf16",
             pairs="64", restart=True, interleaved=False, norm=True, hadamard=True),
        # A diffusion transformer's image tokens: (index, row, column) positions on adjacent pairs, norms, no rotation.
        dict(name="norm_rope_image", op="norm_rope", tokens=4096, q_heads=32, k_heads=32, dim=128, dtype="bf16",
             pairs="8,28,28", restart=True, interleaved=True, norm=True, hadamard=False),
        # A vision-language prompt: one spectrum in (time, height, width) sections over half-split pairs, grouped heads.
        dict(name="norm_rope_sections", op="norm_rope", tokens=9973, q_heads=28, k_heads=4, dim=128, dtype="bf16",
             pairs="16,24,24", restart=False, interleaved=False, norm=True, hadamard=True),
        # Video latents with 64-wide heads in half precision, part of the head without positions.
        dict(name="norm_rope_video", op="norm_rope", tokens=29991, q_heads=20, k_heads=20, dim=64, dtype="fp16",
             pairs="4,10,10", restart=True, interleaved=True, norm=True, hadamard=False),
        # The new token of each of 61 running sequences (three of 64 rows are padding) goes into the cache.
        dict(name="cache_write_decode", op="cache_write", tokens=64, kv_heads=8, dim=128, page=16, padding=3,
             dtype="bf16"),
        # A long prompt's keys and values go into the cache, read out of the packed projection output.
        dict(name="cache_write_prompt", op="cache_write", tokens=16411, kv_heads=8, dim=128, page=64, padding=0,
             dtype="bf16"),
        # One token of one sequence: latency.
        dict(name="attend_one", op="attention", requests=1, new=1, context=1021, q_heads=32, kv_heads=8, dim=128,
             page=16, causal=True, dtype="bf16", lse=False),
        # One token of each of 64 sequences of unequal length.
        dict(name="attend_batch", op="attention", requests=64, new=1, context=8192, q_heads=32, kv_heads=8, dim=128,
             page=64, causal=True, dtype="bf16", lse=False),
        # One token of two very long sequences: the long axis has to be split.
        dict(name="attend_long", op="attention", requests=2, new=1, context=131059, q_heads=32, kv_heads=4, dim=128,
             page=128, causal=True, dtype="bf16", lse=False),
        # Up to five drafted tokens of each of 16 sequences are checked at once, 64-wide heads.
        dict(name="attend_draft", op="attention", requests=16, new=5, context=3001, q_heads=32, kv_heads=8, dim=64,
             page=16, causal=True, dtype="fp16", lse=False),
        # A chunk of a long prompt behind what the cache holds already.
        dict(name="attend_prompt", op="attention", requests=2, new=1024, context=8203, q_heads=32, kv_heads=8, dim=128,
             page=64, causal=True, dtype="bf16", lse=False),
        # Image tokens read an encoder's states (no order): with the log sums, to be joined with another part.
        dict(name="attend_states", op="attention", requests=1, new=4096, context=4333, q_heads=32, kv_heads=32,
             dim=128, page=64, causal=False, dtype="bf16", lse=True),
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "norm_rope", "cache_write", "attention", "attention", "attention"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    dim = rng.choice((64, 128, 128))
    if op == "norm_rope":
        k_heads = rng.randint(1, 16)
        q_heads = k_heads * rng.choice((1, 1, 2, 4))
        tokens = _between(rng, 1, 32 * 4096 * 128 // ((q_heads + k_heads) * dim))
        p = dim // 2
        a = 2 * rng.randint(1, p // 8 - 1)
        pairs = rng.choice(("%d" % p, "%d,%d,%d" % (p - 4 * a, 2 * a, 2 * a), "%d" % (p // 2)))
        return dict(op=op, tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, dtype=dtype, pairs=pairs,
                    restart=rng.random() < 0.5, interleaved=rng.random() < 0.5, norm=rng.random() < 0.8,
                    hadamard=rng.random() < 0.5)
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "cache_write":
        kv_heads = rng.randint(1, 16)
        tokens = _between(rng, 1, 16384 * 8 * 128 // (kv_heads * dim))
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, page=page,
                    padding=rng.randint(0, 3) if tokens > 4 else 0, dtype=dtype)
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16))
    q_heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
    kind = rng.choice(("decode", "decode", "draft", "prompt"))
    causal = rng.random() < 0.7
    if kind == "prompt":
        new = _between(rng, 16, 2048)
        requests = rng.randint(1, 3)
        most = min(16384, 4096 * 4333 * 32 // (new * requests * q_heads))
        context = max(_between(rng, 64, max(64, most)), new if causal else 1)
    else:
        new = 1 if kind == "decode" else rng.randint(2, 8)
        requests = _between(rng, 1, 64)
        context = max(new, _between(rng, 16, min(131072, 64 * 6144 * 8 // (kv_heads * requests))))
    return dict(op=op, requests=requests, new=new, context=context, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                page=page, causal=causal, dtype=dtype, lse=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _pairs(case):
    return [int(n) for n in case["pairs"].split(",")]


def _lengths(case):
    """(new tokens, keys) of each request: unequal where there are several, the last one the longest."""
    r = random.Random(case["requests"] * 1000003 + case["context"] * 31 + case["new"])
    new, keys = [], []
    for i in range(case["requests"]):
        last = i == case["requests"] - 1
        n = case["new"] if last else r.randint(max(1, case["new"] // 2), case["new"])
        new.append(n)
        keys.append(case["context"] if last else r.randint(max(1, n if case["causal"] else 1, case["context"] // 2),
                                                           max(n, case["context"])))
    return new, keys


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _heads(g, tokens, heads, dim, dtype, out=None):
    """Projected heads: normal values, a few channels of each head ten times as large."""
    x = torch.randn(tokens, heads, dim, device="cuda", generator=g)
    x *= torch.where(torch.rand(heads, dim, device="cuda", generator=g) < 0.02, 10.0, 1.0)
    return x.to(TYPES[dtype])


def _hadamard(n):
    """The Sylvester matrix: -1 where the two indexes share an odd number of bits."""
    i = torch.arange(n, device="cuda")
    both = (i[:, None] & i[None, :])[..., None] >> torch.arange(n.bit_length(), device="cuda")
    return 1.0 - 2.0 * ((both & 1).sum(-1) % 2).float()


def _pack(x):
    """NVFP4 of the last axis: (codes, two to a byte, low half first; e4m3 scale bytes, one for 16 values)."""
    x = x.float().unflatten(-1, (-1, 16))
    s = (x.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()
    a = torch.where(f > 0, x.abs() / f, 0.0)
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c |= torch.where((x < 0) & (f > 0), 8, 0).to(torch.uint8)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.squeeze(-1).view(torch.uint8)


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case, "grid": torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")}
    if case["op"] == "norm_rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        packed = _heads(g, t, hq + 2 * hk, d, case["dtype"])       # the projection's output: q, k and v of a token
        st["q"], st["k"] = packed[:, :hq], packed[:, hq:hq + hk]
        if case["norm"]:
            st["qw"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(TYPES[case["dtype"]])
            st["kw"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(TYPES[case["dtype"]])
        else:
            st["qw"] = st["kw"] = None
        pairs = _pairs(case)
        n = torch.arange(t, device="cuda")
        if len(pairs) == 1:      # far positions of a long context
            pos = (n + torch.randint(0, 1 << 17, (1,), device="cuda", generator=g))[:, None]
        else:                    # rows and columns of frames
            w = max(1, int(math.sqrt(min(t, 4096))))
            pos = torch.stack((n // (w * w), n // w % w, n % w), 1)
        st["pos"] = pos.to(torch.int32)
        total = sum(pairs)
        f, axis = [], []
        for a, p in enumerate(pairs):
            start = 0 if case["restart"] else len(f)
            f += [10000.0 ** (-(start + j) / (p if case["restart"] else total)) for j in range(p)]
            axis += [a] * p
        st["freq"] = torch.tensor(f, dtype=torch.float32, device="cuda")
        st["axis"] = torch.tensor(axis, dtype=torch.uint8, device="cuda")
        st["rotation"] = _hadamard(d) / math.sqrt(d) if case["hadamard"] else None
        return st
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "cache_write":
        t = case["tokens"]
        packed = _heads(g, t, 4 * h, d, case["dtype"])             # grouped heads: two of q, one of k, one of v
        st["k"], st["v"] = packed[:, 2 * h:3 * h], packed[:, 3 * h:]
        pages = -(-t // page) + 3
        slots = torch.randperm(pages, device="cuda", generator=g)[:, None] * page + torch.arange(page, device="cuda")
        slots = slots.flatten()[:t].clone()
        if t <= 256:             # decoding: each token has a page of its own sequence
            slots = torch.randperm(pages * page, device="cuda", generator=g)[:t].clone()
        if case["padding"]:
            slots[t - case["padding"]:] = -1
        st["slots"] = slots
        st["cache"] = tuple(torch.zeros(pages, h, page, n, dtype=torch.uint8, device="cuda")
                            for n in (d // 2, d // 16, d // 2, d // 16))
        return st
    new, keys = _lengths(case)
    need = [-(-n // page) for n in keys]
    pages = sum(need) + 1
    order = torch.randperm(pages, device="cuda", generator=g)[:sum(need)].to(torch.int32)
    table = torch.full((len(keys), max(need)), -1, dtype=torch.int32)
    at = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
    table[at] = order.cpu()
    st["table"] = table.cuda()
    cache = []
    for _ in range(2):
        parts = [_pack(_heads(g, n * h, page, d, "bf16").reshape(n, h, page, d))
                 for n in [min(2048, pages - i) for i in range(0, pages, 2048)]]
        cache += [torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])]
    st["cache"] = tuple(cache)
    st["lengths"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
    st["start"] = None
    if case["new"] > 1:
        st["start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    st["most"] = (max(new), max(keys))
    st["q"] = torch.randn(sum(new), case["q_heads"], d, device="cuda", generator=g).to(TYPES[case["dtype"]])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        import bit_quantized_linear_svdq_b200 as S
        if case["op"] == "norm_rope":
            return S.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], positions=st["pos"], inv_freq=st["freq"],
                                  pair_axis=st["axis"], interleaved=case["interleaved"], hadamard=case["hadamard"])
        if case["op"] == "cache_write":
            S.kv4_append(st["cache"], st["k"], st["v"], st["slots"])
            return S.kv4_read(st["cache"], st["slots"], dtype=TYPES[case["dtype"]])
        return S.kv4_attention(st["q"], st["cache"], st["lengths"], st["table"], q_start=st["start"],
                               causal=case["causal"], max_kv_len=st["most"][1], return_lse=case["lse"])
    if case["op"] == "norm_rope":
        return _norm_rope(st, st["q"], st["qw"]), _norm_rope(st, st["k"], st["kw"])
    if case["op"] == "cache_write":
        return _kept(st, st["k"]), _kept(st, st["v"])
    return _attend(st)


def _norm_rope(st, x, w):
    case, y = st["case"], x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    p = st["freq"].numel()
    turn = st["pos"].double()[:, st["axis"].long()] * st["freq"].double()
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]
    if case["interleaved"]:
        a, b = y[..., 0:2 * p:2], y[..., 1:2 * p:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = y[..., :p], y[..., p:2 * p]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    y = torch.cat((turned, y[..., 2 * p:]), -1)
    if case["hadamard"]:
        y = y @ st["rotation"]
    return y.to(x.dtype)


def _kept(st, x):
    codes, scales = _pack(x)
    y = _values(st, codes, scales)
    return torch.where(st["slots"][:, None, None] >= 0, y, 0.0).to(x.dtype)


def _values(st, codes, scales):
    v = torch.stack((st["grid"][(codes & 15).int()], st["grid"][(codes >> 4).int()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _attend(st):
    case, q = st["case"], st["q"]
    n_req, h, d, page = case["requests"], case["kv_heads"], case["dim"], case["page"]
    group, tokens = case["q_heads"] // h, q.shape[0]
    most_q, most_k = st["most"]
    start = st["start"]
    if start is None:
        start = torch.arange(n_req + 1, device="cuda", dtype=torch.int32)
    token = torch.arange(tokens, device="cuda", dtype=torch.int32)
    owner = torch.searchsorted(start[1:], token, right=True)
    place = (token - start[owner]).long()
    rows = torch.zeros(n_req, most_q, h, group, d, device="cuda")
    rows[owner, place] = q.float().unflatten(1, (h, group))
    rows = rows.permute(0, 2, 1, 3, 4).reshape(n_req, h, most_q * group, d)
    table = st["table"].long().clamp(min=0)

    def gathered(codes, scales):      # (requests, heads, keys, dim)
        v = _values(st, codes[table], scales[table])
        return v.transpose(1, 2).reshape(n_req, h, -1, d)[:, :, :most_k]

    s = rows @ gathered(st["cache"][0], st["cache"][1]).transpose(-1, -2) / math.sqrt(d)
    key = torch.arange(most_k, device="cuda")
    last = st["lengths"][:, None].long().expand(n_req, most_q)
    if case["causal"]:
        last = last - (start[1:] - start[:-1])[:, None] + torch.arange(most_q, device="cuda") + 1
    last = last.repeat_interleave(group, 1)[:, None, :, None]
    s = s.masked_fill_(key >= last, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ gathered(st["cache"][2], st["cache"][3]) / total
    o = o.unflatten(2, (most_q, group)).permute(0, 2, 1, 3, 4)[owner, place].flatten(1, 2).to(q.dtype)
    if not case["lse"]:
        return o
    lse = (m + total.log()).unflatten(2, (most_q, group))[..., 0].permute(0, 2, 1, 3)[owner, place]
    return o, lse.flatten(1, 2)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    d = case["dim"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * d
        axes = len(_pairs(case))
        flops = n * ((4 if case["norm"] else 0) + 3 + (math.log2(d) + 1 if case["hadamard"] else 0))
        return {"bytes": 4 * n + 4 * axes * case["tokens"] + 5 * sum(_pairs(case)) + (4 * d if case["norm"] else 0),
                "flops": flops}
    h = case["kv_heads"]
    kept = 2 * (d // 2 + d // 16)                               # bytes of one key and its value in the cache
    if case["op"] == "cache_write":                             # values in, cache written and read, values out
        n = case["tokens"] * h
        return {"bytes": n * (8 * d + 2 * kept) + 16 * case["tokens"], "flops": 8 * n * d}
    new, keys = _lengths(case)
    hq = case["q_heads"]
    seen = sum(n * k - (n * (n - 1) // 2 if case["causal"] else 0) for n, k in zip(new, keys))
    moved = sum(keys) * h * kept + 4 * sum(new) * hq * d + (4 * sum(new) * hq if case["lse"] else 0)
    moved += 4 * sum(-(-k // case["page"]) for k in keys) + 8 * len(keys)
    return {"bytes": moved, "flops": 4.0 * d * hq * seen}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_exact_heads(case, st, st[n], st[n + "w"]) for n in ("q", "k"))
    if case["op"] == "cache_write":
        live = (st["slots"] >= 0).double()[:, None, None]
        return tuple(_exact_nearest(st[n].double()) * live for n in ("k", "v"))
    return _exact_attention(case, st)


def _exact_heads(case, st, x, w):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + 1e-6) * w.double()
    y = y.clone()
    p = st["freq"].numel()
    for i in range(p):           # one pair of channels at a time
        phi = st["pos"][:, int(st["axis"][i])].double() * st["freq"][i].double()
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + p)
        z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(phi), phi)[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    if case["hadamard"]:
        h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
        while h.shape[0] < case["dim"]:
            h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0) / math.sqrt(2.0)
        y = y @ h
    return y


def _nearest(a, grid):
    """The value of the ascending grid nearest to each a >= 0; the even place of two equally near ones."""
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), grid[lo], grid[hi])


def _exact_nearest(x):
    e4m3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    scale_grid = torch.tensor(e4m3[:-1], dtype=torch.float64, device="cuda")
    x = x.unflatten(-1, (-1, 16))
    s = _nearest(x.abs().amax(-1, keepdim=True) / 6, scale_grid)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    return (torch.sign(x) * _nearest(x.abs() / s.clamp(min=2.0 ** -20), grid) * s).flatten(-2)


def _exact_attention(case, st):
    new, keys = _lengths(case)
    h, d, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def unpacked(codes, scales, pages, n):       # (heads, n, dim)
        c = codes[pages].transpose(0, 1).reshape(h, -1, d // 2)[:, :n].long()
        s = scales[pages].transpose(0, 1).reshape(h, -1, d // 16)[:, :n].long()
        v = torch.empty(h, n, d, dtype=torch.float64, device="cuda")
        for half in (0, 1):
            nib = (c >> (4 * half)) & 15
            v[..., half::2] = grid[nib & 7] * torch.where(nib > 7, -1.0, 1.0)
        e, m = (s >> 3) & 15, (s & 7).double()
        size = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
        return v * size.repeat_interleave(16, -1)

    outs, sums, at = [], [], 0
    for b, (n, k) in enumerate(zip(new, keys)):
        pages = st["table"][b, :-(-k // case["page"])].long()
        q = st["q"][at:at + n].double().reshape(n, h, group, d).permute(1, 2, 0, 3)      # (heads, group, n, dim)
        at += n
        s = torch.matmul(q, unpacked(st["cache"][0], st["cache"][1], pages, k).transpose(1, 2)[:, None]) * d ** -0.5
        if case["causal"]:
            seen = torch.ones(n, k, dtype=torch.bool, device="cuda").tril(k - n)
            s = torch.where(seen, s, -math.inf)
        lse = torch.logsumexp(s, -1)
        v = unpacked(st["cache"][2], st["cache"][3], pages, k)[:, None]
        outs.append(torch.matmul(torch.exp(s - lse[..., None]), v).permute(2, 0, 1, 3).reshape(n, h * group, d))
        sums.append(lse.permute(2, 0, 1).reshape(n, h * group))
    return (torch.cat(outs), torch.cat(sums)) if case["lse"] else torch.cat(outs)
