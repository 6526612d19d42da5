"""GPU tests of the attention-side operators against plain 64-bit definitions: head norms with rotary positions, the
4-bit cache (bit-exact against the oracle's quantizer) and attention over it."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_svdq_b200 as S
from bit_quantized_linear_svdq_b200 import attention, synthetic
from oracle import svdq_oracle as O

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}          # half a step of the type, relative
TINY = {BF: 2.0 ** -134, FP: 2.0 ** -25}        # half a step below the normal range


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bit_quantized_linear_svdq_b200 import build
    build.build()
    S.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def heads(g, t, h, d, dtype, scale=1.0):
    x = torch.randn(t, h, d, device="cuda", generator=g) * scale
    return (x * torch.where(torch.rand(h, d, device="cuda", generator=g) < 0.03, 8.0, 1.0)).to(dtype)


# ------------------------------------------------------------------ norm, positions, rotation

def rope_reference(x, w, eps, pos, freq, axis, interleaved, hadamard):
    """(y, bound of the fp32 error) in 64 bits.  Bound: the norm's factor is off by at most 16 units of 2^-24 (sums of
    20 terms a lane and tree halved by the root, rsqrt 2 ulp, two products), cosine and sine by 7 (reduced angle to
    2^-25 turns, sincospi 2 ulp), the pair's products and sum by 3: 26 < 32 = 2^-19 / 2^-24 of |a| + |b|.  The Hadamard
    adds log2 D + 2 units of the sum of magnitudes over sqrt(D): within 2^-18."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.double()
    bound = 2.0 ** -19 * y.abs()
    d, p = x.shape[-1], 0 if freq is None else freq.numel()
    if p:
        phi = torch.stack([pos[:, int(axis[i])].double() * freq[i].double() for i in range(p)], 1)[:, None]
        ia = torch.arange(p, device="cuda") * 2 if interleaved else torch.arange(p, device="cuda")
        ib = ia + (1 if interleaved else p)
        a, b = y[..., ia], y[..., ib]
        y = y.clone()
        y[..., ia], y[..., ib] = a * phi.cos() - b * phi.sin(), a * phi.sin() + b * phi.cos()
        bound[..., ia] = bound[..., ib] = 2.0 ** -19 * (a.abs() + b.abs())
    if hadamard:
        h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
        while h.shape[0] < d:
            h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
        bound = 2.0 ** -18 * 2 * y.abs().sum(-1, keepdim=True).expand(y.shape) / math.sqrt(d)
        y = y @ h / math.sqrt(d)
    return y, bound


def assert_rounded(got, want, bound, dtype):
    err = (got.double() - want).abs()
    tol = bound + HALF[dtype] * (want.abs() + bound) + TINY[dtype]
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {(err / tol).max():.3g} of the tolerance"


ROPE_CASES = [
    # tokens, q heads, k heads, dim, dtype, pairs, restart, interleaved, norm, hadamard
    (1, 1, 1, 64, BF, (32,), True, False, True, False),
    (1, 32, 8, 128, BF, (64,), True, False, True, True),
    (7, 5, 1, 128, FP, (16, 24, 24), False, False, True, True),
    (33, 24, 24, 128, BF, (8, 28, 28), True, True, True, False),
    (130, 3, 2, 64, FP, (4, 10, 10), True, True, True, True),
    (65, 4, 4, 128, BF, (32,), True, False, True, False),         # part of the head has no position
    (65, 4, 4, 128, BF, (8,), True, False, False, False),
    (9, 2, 2, 256, BF, (128,), True, False, True, True),
    (9, 2, 2, 256, FP, (24, 24, 16), True, False, True, False),
    (11, 3, 1, 80, BF, (40,), True, False, True, False),          # 80 and 96: no power of two
    (11, 3, 1, 96, FP, (17, 3), True, True, True, False),
    (5, 2, 2, 8, BF, (4,), True, True, True, True),
    (5, 2, 2, 16, FP, (8,), True, False, True, True),
    (5, 2, 2, 32, BF, (5, 3), True, False, False, True),
    (6, 7, 3, 40, BF, (), True, False, True, False),              # norm alone
    (6, 7, 3, 128, BF, (), True, False, False, True),             # rotation alone
    (3000, 8, 2, 128, BF, (64,), True, False, True, False),       # many tokens a CTA
    (2500, 1, 1, 256, BF, (128,), True, True, True, True),
    (70, 3, 1, 128, FP, (32,), True, False, True, True),          # half-split pairs of a quarter of the head, rotated
    (1700, 2, 1, 64, BF, (8,), True, False, True, True),
    (300, 2, 2, 40, FP, (13,), True, True, True, False),          # adjacent pairs that end inside a chunk
    (4500, 1, 1, 64, BF, (3, 2), True, True, True, True),
    (21, 2, 2, 32, FP, (5, 5, 5), True, True, False, False),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_qk_norm_rope(case):
    t, hq, hk, d, dtype, pairs, restart, inter, norm, had = case
    g = gen(hash(case[:4]) & 0xFFFF)
    packed = heads(g, t, hq + 2 * hk, d, dtype, 3.0)             # q, k, v of a token side by side
    q, k = packed[:, :hq], packed[:, hq:hq + hk]
    w = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dtype) if norm else None for _ in range(2)]
    kw = dict(interleaved=inter, hadamard=had)
    pos = freq = axis = None
    if pairs:
        freq, axis = S.rope_frequencies(pairs, restart=restart)
        pos = torch.randint(-200000, 200000, (t, len(pairs)), device="cuda", generator=g, dtype=torch.int32)
        kw.update(positions=pos, inv_freq=freq, pair_axis=axis)
    before = packed.clone()
    qo, ko = S.qk_norm_rope(q, k, *w, **kw)
    torch.cuda.synchronize()
    assert torch.equal(packed, before)
    for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
        want, bound = rope_reference(x, wt, 1e-6, pos, freq, axis, inter, had)
        assert_rounded(got, want, bound, dtype)
    # In place, in the packed buffer: the same values, and v untouched.
    S.qk_norm_rope(q, k, *w, inplace=True, **kw)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(packed[:, hq + hk:], before[:, hq + hk:])
    # Queries alone.
    assert torch.equal(S.qk_norm_rope(before[:, :hq], None, w[0], **kw)[0], qo)


def test_qk_norm_rope_one_side_normed_and_layouts():
    g = gen(3)
    x = heads(g, 17, 6, 128, BF)
    q, k = x.transpose(0, 1).contiguous().transpose(0, 1)[:, :4], x[:, 4:]   # heads outermost in memory
    w = torch.full((128,), 2.0, dtype=BF, device="cuda")
    qo, ko = S.qk_norm_rope(q, k, w)                                        # no positions, keys pass
    assert torch.equal(ko, k)
    want, bound = rope_reference(q, w, 1e-6, None, None, None, False, False)
    assert_rounded(qo, want, bound, BF)
    # One position per token (a vector, and a strided column); an axis past the last counts as the last.
    f, axis = S.rope_frequencies((64,))
    pos = torch.randint(0, 9000, (17, 3), device="cuda", generator=g, dtype=torch.int32)
    a = S.qk_norm_rope(q, k, positions=pos[:, 1], inv_freq=f)[0]
    b = S.qk_norm_rope(q, k, positions=pos[:, 1:2].contiguous(), inv_freq=f, pair_axis=axis + 9)[0]
    assert torch.equal(a, b)
    # One token's heads stretched over all tokens: allowed as an input, not as an output.
    e = x[:1].expand(17, 6, 128)
    assert torch.equal(S.qk_norm_rope(e, None, w)[0], S.qk_norm_rope(e.contiguous(), None, w)[0])
    with pytest.raises(ValueError, match="overlap"):
        S.qk_norm_rope(e, None, w, inplace=True)


def test_qk_norm_rope_empty_and_special_values():
    w = torch.ones(128, dtype=BF, device="cuda")
    q = torch.zeros(0, 4, 128, dtype=BF, device="cuda")
    assert S.qk_norm_rope(q, q, w, w)[1].shape == (0, 4, 128)
    x = torch.zeros(4, 2, 128, dtype=BF, device="cuda")
    x[1, 0, 5], x[2, 1, 7] = float("nan"), float("inf")
    x[3] = 1e-20
    y = S.qk_norm_rope(x, None, w, eps=1e-6)[0].float()
    assert (y[0] == 0).all() and y[1, 0].isnan().all() and (y[1, 1] == 0).all()
    assert y[2, 1].isnan().any() and (y[2, 0] == 0).all()
    want, bound = rope_reference(x[3:], w, 1e-6, None, None, None, False, False)
    assert_rounded(y[3:].to(BF), want, bound, BF)


def test_qk_norm_rope_refusals():
    q = torch.zeros(4, 2, 128, dtype=BF, device="cuda")
    f, axis = S.rope_frequencies((64,))
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(128, dtype=BF, device="cuda")
    for err, call in [
        (TypeError, lambda: S.qk_norm_rope(q.float())),
        (TypeError, lambda: S.qk_norm_rope(q, q.half())),
        (ValueError, lambda: S.qk_norm_rope(q[0])),
        (ValueError, lambda: S.qk_norm_rope(q, q[:3])),
        (ValueError, lambda: S.qk_norm_rope(q, q[..., :64])),
        (ValueError, lambda: S.qk_norm_rope(q.transpose(1, 2))),
        (ValueError, lambda: S.qk_norm_rope(q[..., 4:68])),                    # not 16-byte aligned
        (TypeError, lambda: S.qk_norm_rope(q, None, w.half())),
        (ValueError, lambda: S.qk_norm_rope(q, None, w[:64])),
        (ValueError, lambda: S.qk_norm_rope(q, None, None, w)),
        (ValueError, lambda: S.qk_norm_rope(q, inv_freq=f)),
        (ValueError, lambda: S.qk_norm_rope(q, positions=pos)),
        (TypeError, lambda: S.qk_norm_rope(q, positions=pos.long(), inv_freq=f)),
        (ValueError, lambda: S.qk_norm_rope(q, positions=pos[:3], inv_freq=f)),
        (TypeError, lambda: S.qk_norm_rope(q, positions=pos, inv_freq=f.double())),
        (ValueError, lambda: S.qk_norm_rope(q, positions=pos.cpu(), inv_freq=f)),
        (S.SvdqError, lambda: S.qk_norm_rope(q, positions=pos, inv_freq=f[:20])),
        (S.SvdqError, lambda: S.qk_norm_rope(q[..., :96].contiguous(), hadamard=True)),
        (S.SvdqError, lambda: S.qk_norm_rope(q, eps=-1.0)),
    ]:
        with pytest.raises(err):
            call()


# ------------------------------------------------------------------ the cache

def quantized(x):
    """The oracle's codes and scale bytes of rows of 16-value blocks (bf16 and fp16 are exact in fp32)."""
    v = x.float().cpu().numpy()
    c, s = O.quantize_nvfp4_rows(np.ascontiguousarray(v.reshape(-1, v.shape[-1])))
    return (torch.from_numpy(np.ascontiguousarray(c)).reshape(*v.shape[:-1], -1),
            torch.from_numpy(np.ascontiguousarray(s)).reshape(*v.shape[:-1], -1))


@pytest.mark.parametrize("t,h,d,page,dtype", [(1, 1, 64, 16, BF), (5, 3, 128, 16, FP), (100, 2, 64, 32, FP),
                                              (333, 5, 128, 64, BF), (70, 1, 128, 128, BF), (300, 8, 64, 256, BF)])
def test_append_and_read(t, h, d, page, dtype):
    g = gen(t)
    pages = -(-t // page) + 2
    cache = S.kv4_cache(pages, page, h, d)
    for c in cache:
        c.copy_(torch.randint(0, 126, c.shape, device="cuda", generator=g, dtype=torch.uint8))
    before = [c.clone() for c in cache]
    packed = heads(g, t, 3 * h, d, dtype)
    k, v = packed[:, h:2 * h], packed[:, 2 * h:]
    if t > 4:     # zeros, a value too small for a scale, the type's ends, infinity and NaN
        k[0, 0, :16] = 0
        k[1, 0, :16] = 2.0 ** -13
        v[2, 0, :3] = torch.tensor([torch.finfo(dtype).max, -torch.finfo(dtype).max, 1.0])
        k[3, 0, 4], v[3, 0, 20] = float("inf"), float("nan")
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:t]
    skipped = torch.zeros(t, dtype=torch.bool)
    if t > 20:
        skipped[[2, 9, 11]] = True
        slots[2], slots[9], slots[11] = -1, pages * page, 1 << 40
    S.kv4_append(cache, k, v, slots)
    live = slots.cpu()[~skipped]
    for i, x in ((0, k), (2, v)):
        codes, scales = quantized(x)
        want_c, want_s = before[i].cpu(), before[i + 1].cpu()
        p, o = live // page, live % page
        want_c[p, :, o], want_s[p, :, o] = codes[~skipped], scales[~skipped]
        assert torch.equal(cache[i].cpu(), want_c) and torch.equal(cache[i + 1].cpu(), want_s)
        got = S.kv4_read(cache, slots, dtype=dtype)[i // 2].cpu()
        rows = want_c[p, :, o].numpy().reshape(-1, d // 2), want_s[p, :, o].numpy().reshape(-1, d // 16)
        want = torch.from_numpy(np.asarray(O.dequantize_nvfp4(*rows))).reshape(-1, h, d)
        assert torch.equal(got[~skipped].double().nan_to_num(nan=7e4), want.double().nan_to_num(nan=7e4))
        assert (got[skipped] == 0).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_any_16_bytes(d, dtype):
    """Rows that start at odd multiples of 16 bytes, read by append and written by the C entry point of read."""
    g = gen(17)
    t, h = 45, 3
    wide = torch.randn(2, t, h, d + 8, device="cuda", generator=g).to(dtype)
    k, v = wide[0, ..., 8:], wide[1, ..., :d]
    slots = torch.randperm(64, device="cuda", generator=g)[:t]
    a, b = S.kv4_cache(4, 16, h, d), S.kv4_cache(4, 16, h, d)
    S.kv4_append(a, k, v, slots)
    S.kv4_append(b, k.contiguous(), v.contiguous(), slots)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and a.k_codes.any()
    want = S.kv4_read(a, slots, dtype)
    out = torch.full_like(wide, 7.0)
    side = [attention.svdq_heads(o.data_ptr(), o.stride(0), o.stride(1)) for o in (out[0, ..., 8:], out[1, ..., :d])]
    c = attention.svdq_kv4_cache(*(x.data_ptr() for x in a), 4, h, 16, d)
    attention.svdq_kv4_read(c, *side, t, 0 if dtype is BF else 1, slots.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out[0, ..., 8:], want[0]) and torch.equal(out[1, ..., :d], want[1])
    assert (out[0, ..., :8] == 7).all() and (out[1, ..., d:] == 7).all()


def test_append_matches_the_weight_quantizer():
    g = gen(5)
    x = heads(g, 64, 2, 128, BF)
    cache = S.kv4_cache(4, 16, 2, 128)
    S.kv4_append(cache, x, x, torch.arange(64, device="cuda"))
    qw, ws = S.quantize_weight(x.reshape(128, 128))
    assert torch.equal(cache.k_codes.transpose(1, 2).reshape(128, 64), qw)
    assert torch.equal(cache.k_scales.transpose(1, 2).reshape(128, 8), ws.t())
    assert torch.equal(cache.v_codes, cache.k_codes) and torch.equal(cache.v_scales, cache.k_scales)
    S.kv4_append(cache, x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device="cuda"))
    a, b = S.kv4_read(cache, torch.tensor([3, 3, -5], device="cuda"))       # repeated, outside
    assert torch.equal(a[0], a[1]) and (a[2] == 0).all() and b.shape == (3, 2, 128)
    # e4m3 tensors in place of bytes
    typed = (cache[0], cache[1].view(torch.float8_e4m3fn), cache[2], cache[3].view(torch.float8_e4m3fn))
    assert torch.equal(S.kv4_read(typed, torch.tensor([3], device="cuda"))[0][0], a[0])


def test_cache_refusals():
    x = torch.zeros(4, 2, 128, dtype=BF, device="cuda")
    cache = S.kv4_cache(2, 16, 2, 128)
    slots = torch.arange(4, device="cuda")
    small = S.kv4_cache(2, 16, 2, 64)
    for err, call in [
        (TypeError, lambda: S.kv4_append(cache, x.float(), x.float(), slots)),
        (TypeError, lambda: S.kv4_append(cache, x, x.half(), slots)),
        (TypeError, lambda: S.kv4_append(cache, x, x, slots.int())),
        (ValueError, lambda: S.kv4_append(cache, x, x, slots[:3])),
        (ValueError, lambda: S.kv4_append(cache, x, x, slots[:, None])),
        (ValueError, lambda: S.kv4_append(small, x, x, slots)),
        (ValueError, lambda: S.kv4_append((cache[0][:1],) + tuple(cache[1:]), x, x, slots)),
        (ValueError, lambda: S.kv4_append((cache[0].transpose(0, 1),) + tuple(cache[1:]), x, x, slots)),
        (TypeError, lambda: S.kv4_append((cache[0].int(),) + tuple(cache[1:]), x, x, slots)),
        (TypeError, lambda: S.kv4_read(cache, slots, dtype=torch.float32)),
        (ValueError, lambda: S.kv4_read(cache, slots.cpu())),
    ]:
        with pytest.raises(err):
            call()


# ------------------------------------------------------------------ attention

def filled_cache(g, pages, page, h, d):
    cache = S.kv4_cache(pages, page, h, d)
    n = pages * page
    S.kv4_append(cache, heads(g, n, h, d, BF), heads(g, n, h, d, BF), torch.arange(n, device="cuda"))
    return cache


def values(cache, i):
    """The cache's keys (0) or values (2) in 64 bits, (pages, page, heads, dim)."""
    c, s = cache[i].cpu().numpy(), cache[i + 1].cpu().numpy()
    v = O.dequantize_nvfp4(c.reshape(-1, c.shape[-1]), s.reshape(-1, s.shape[-1]))
    return torch.from_numpy(np.asarray(v, dtype=np.float64)).reshape(*c.shape[:3], -1).transpose(1, 2).cuda()


def attend_reference(q, cache, lens, table, start, causal, scale):
    """(out, lse, error bounds of both) in 64 bits; rows of no request are NaN in all.  Bounds, before the output's own
    rounding: a score is off by (D + 4) adds of 2^-23 of scale sum|q k| (tensor-core sums may truncate) and 2^-22 of
    itself (two products, ex2), a weight by that, 2^-11 (fp16) or 2^-25 absolutely (below fp16's normal range, where
    the sum of weights is at least 1), sums over n keys by n 2^-24."""
    kk, vv = values(cache, 0), values(cache, 2)
    page, h, d = kk.shape[1:]
    hq = q.shape[1]
    nan = float("nan")
    out = torch.full(q.shape, nan, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], nan, dtype=torch.float64, device="cuda")
    eo, el = out.clone(), lse.clone()
    for b, n_keys in enumerate(lens):
        s0, s1 = start[b], start[b + 1]
        n = s1 - s0
        j = torch.arange(n_keys, device="cuda")
        pages = table[b].long()[j // page]
        exists = (pages >= 0) & (pages < kk.shape[0])
        pages = pages.clamp(0, kk.shape[0] - 1)
        kb, vb = (x[pages, j % page].repeat_interleave(hq // h, 1) for x in (kk, vv))
        for i in range(n):
            see = exists & (j <= n_keys - n + i) if causal else exists
            ks, vs, qi = kb[see], vb[see], q[s0 + i].double()
            sc = (ks * qi).sum(-1) * scale                           # (keys, heads)
            if not see.any():
                out[s0 + i], lse[s0 + i], eo[s0 + i], el[s0 + i] = 0, -math.inf, 0, 0
                continue
            l = torch.logsumexp(sc, 0)
            p = torch.exp(sc - l)
            ds = (2.0 ** -23 * (d + 4) * (ks * qi).abs().sum(-1) * abs(scale) + 2.0 ** -22 * (sc.abs() + 1)).amax(0)
            m = ks.shape[0]
            out[s0 + i], lse[s0 + i] = torch.einsum("kh,khd->hd", p, vs), l
            mag = torch.einsum("kh,khd->hd", p, vs.abs())
            eo[s0 + i] = (2.0 ** -11 + 2 * ds[:, None] + 2 * m * 2.0 ** -24) * mag + 2.0 ** -25 * vs.abs().sum(0)
            el[s0 + i] = ds + m * 2.0 ** -24 + 2.0 ** -22 * (1 + l.abs())
    return out, lse, eo, el


def check(q, cache, lens, table, start, causal, scale=None, **kw):
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    start_t = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    n = len(lens)
    full = start or [i * (q.shape[0] // n) for i in range(n + 1)]
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device="cuda")
    got, lse = S.kv4_attention(q, cache, lens_t, table, q_start=start_t, causal=causal, softmax_scale=scale, out=out,
                               return_lse=True, **kw)
    assert got is out
    sc = 1 / math.sqrt(q.shape[2]) if scale is None else float(np.float32(scale))
    want, wl, eo, el = attend_reference(q, cache, lens, table, full, causal, sc)
    none = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    none[full[0]:full[-1]] = False
    assert (out[none] == 77.0).all()                                 # rows of no request are left alone
    live = ~none
    assert_rounded(out[live], want[live], eo[live], q.dtype)
    inf = wl[live] == -math.inf
    assert torch.equal(lse[live] == -math.inf, inf)
    assert ((lse[live].double() - wl[live]).abs() <= el[live])[~inf].all()
    return out, lse.masked_fill(none[:, None], 0.0)                  # (a new tensor: unspecified there)


def tables(g, lens, page, pages, extra=0):
    need = [-(-max(n, 0) // page) for n in lens]
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    t = torch.full((len(lens), max(max(need) + extra, 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


ATTEND = [
    # lens, new per request (or q_start), q heads, kv heads, dim, page, causal, dtype
    ([1], 1, 1, 1, 64, 16, True, BF),
    ([1, 0, 17], 1, 4, 2, 128, 16, True, BF),
    ([15, 16, 31, 33, 64, 65], 1, 8, 2, 128, 16, True, FP),
    ([300, 1, 0, 129], 1, 6, 2, 64, 32, False, FP),
    ([1000], 1, 32, 8, 128, 64, True, BF),                         # the key axis is split
    ([4097, 2], 1, 7, 1, 128, 256, True, BF),                      # one key head, seven query heads
    ([2050], 1, 40, 2, 64, 128, True, BF),                         # 20 rows a tile of 32
    ([77, 5, 40], [0, 3, 4, 9], 8, 2, 128, 16, True, BF),          # unequal new tokens
    ([77, 5, 40], [2, 3, 3, 9], 3, 3, 64, 16, True, FP),           # tokens before, none in the middle, one behind
    ([3, 10], [0, 8, 10], 4, 4, 128, 16, True, BF),                # more queries than keys: the first see none
    ([0, 0], [0, 3, 5], 2, 1, 128, 16, True, BF),
    ([500, 33], [0, 70, 103], 4, 2, 128, 64, True, BF),            # many row tiles
    ([500, 33], [0, 70, 103], 4, 2, 64, 64, False, FP),
    ([140], 200, 2, 1, 128, 32, False, BF),                        # more queries than keys, no order
    ([1500], 130, 9, 3, 128, 64, True, FP),
    ([513], 300, 8, 1, 64, 16, True, BF),
    ([900, 31, 400, 65], [0, 200, 201, 401, 402], 6, 2, 128, 32, True, BF),   # prompts beside single tokens
    ([900, 31, 400, 65], [3, 300, 301, 310, 311], 4, 2, 64, 16, False, FP),
    ([260, 0, 129], [0, 129, 400, 700], 2, 1, 128, 16, True, FP),  # a prompt without keys; more queries than keys
    ([300, 450, 40], 1, 7, 1, 128, 16, True, BF),                  # two to four parts a segment, an odd number of rows
    ([400, 300], 33, 15, 5, 128, 64, True, FP),
    ([511, 260], 41, 9, 3, 64, 32, False, BF),
]


def make(case, seed):
    lens, new, hq, h, d, page, causal, dtype = case
    g = gen(seed)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = filled_cache(g, pages, page, h, d)
    start = None if isinstance(new, int) else new
    tokens = new * len(lens) if start is None else new[-1] + 1
    q = heads(g, tokens, hq, d, dtype)
    return q, cache, lens, tables(g, lens, page, pages, extra=1), start, causal


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-{c[1]}-{c[2:7]}".replace(" ", ""))
def test_attention(case):
    q, cache, lens, table, start, causal = make(case, 11)
    a = check(q, cache, lens, table, start, causal)
    # The same bits again; a bound of the lengths that is too small changes the split, not the result.
    b = check(q, cache, lens, table, start, causal)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].nan_to_num(), b[1].nan_to_num())
    check(q, cache, lens, table, start, causal, max_kv_len=max(1, max(lens) // 3))
    check(q, cache, lens, table, start, causal, scale=0.31, max_kv_len=max(1, max(lens)))
    check(q, cache, lens, table, start, causal, scale=-0.2)
    assert S.svdq_kv4_attention_status() == 0


@pytest.mark.parametrize("d,keys", [(64, 50), (128, 50), (128, 300)])
def test_many_row_tiles_a_block(d, keys):
    """More (row tile, head) pairs than resident blocks, each over few keys: blocks go from one to the next, whole and
    cut ones.  Without an order all queries see all keys, so the reference is one softmax."""
    tokens, h = 6000, 16
    g = gen(d + keys)
    cache = filled_cache(g, -(-keys // 16) + 1, 16, h, d)
    table = tables(g, [keys], 16, cache[0].shape[0])
    q = heads(g, tokens, h, d, BF)
    lens = torch.tensor([keys], dtype=torch.int32, device="cuda")
    j = torch.arange(keys, device="cuda")
    kb, vb = (values(cache, i)[table[0, j // 16].long(), j % 16].transpose(0, 1) for i in (0, 2))     # (heads, keys, dim)
    sc = q.double().transpose(0, 1) @ kb.transpose(1, 2) / math.sqrt(d)
    p, want_lse = torch.softmax(sc, -1), torch.logsumexp(sc, -1).t()
    # (The bounds of attend_reference, with the largest score's for all.)
    ds = 2.0 ** -23 * (d + 4) * float((q.double().abs().transpose(0, 1) @ kb.abs().transpose(1, 2)).max()) / math.sqrt(d) \
        + 2.0 ** -22 * (float(sc.abs().max()) + 1)
    want = (p @ vb).transpose(0, 1)
    bound = (2.0 ** -11 + 2 * ds + 2 * keys * 2.0 ** -24) * (p @ vb.abs()).transpose(0, 1) + 2.0 ** -25 * vb.abs().sum(1)
    for _ in range(5):
        out, lse = S.kv4_attention(q, cache, lens, table, causal=False, return_lse=True)
        assert_rounded(out, want, bound, BF)
        assert ((lse.double() - want_lse).abs() <= ds + keys * 2.0 ** -24 + 2.0 ** -22 * (1 + want_lse.abs())).all()


def test_attention_strided_arguments():
    g = gen(21)
    case = ([90, 31], [0, 2, 5], 4, 2, 128, 16, True, BF)
    _, cache, lens, table, start, causal = make(case, 21)
    packed = heads(g, 5, 8, 128, BF)
    wide = torch.full((2, table.shape[1] + 5), 99, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    buf = torch.full((5, 12, 128), 3.0, dtype=BF, device="cuda")
    args = dict(q_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = S.kv4_attention(packed[:, :4].contiguous(), cache, lens_t, table, **args)
    S.kv4_attention(packed[:, :4], cache, lens_t, wide[:, :table.shape[1]], out=buf[:, 4:8], **args)
    assert torch.equal(buf[:, 4:8], want)
    assert (buf[:, :4] == 3).all() and (buf[:, 8:] == 3).all()
    by_head = packed[:, :4].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(S.kv4_attention(by_head, cache, lens_t, table, **args), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [(1, [40, 100]), (6, [40, 100]), (150, [170, 400])])
def test_masked_places_may_hold_anything(d, new, lens):
    """NaN in rows behind the keys, and in keys that some of the queries do not see."""
    page, h, hq = 16, 2, 4
    case = (lens, new, hq, h, d, page, True, BF)
    q, cache, lens, table, _, _ = make(case, 31)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean, clean_lse = S.kv4_attention(q, cache, lens_t, table, return_lse=True)
    for b, n in enumerate(lens):                       # all that is no key: rest of the last page, unused pages
        last = int(table[b, (n - 1) // page])
        if n % page:
            for c in (1, 3):
                cache[c][last, :, n % page:] = 0x7F
    used = set(table[table >= 0].tolist())
    for p in range(cache[0].shape[0]):
        if p not in used:
            cache[1][p] = cache[3][p] = 0xFF
    out, lse = S.kv4_attention(q, cache, lens_t, table, return_lse=True)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    if new == 1:
        return
    # A NaN value in one 16-channel block of head 1 at key j of request 0: queries from that key's position on get NaN
    # in that block, earlier ones nothing.  A NaN key makes whole rows NaN.
    n = lens[0]
    j, blk = n - 3, d // 16 - 1
    at = int(table[0, j // page]), 1, j % page, blk
    keep = cache[3][at].clone()
    cache[3][at] = 0x7F
    got = S.kv4_attention(q, cache, lens_t, table).float()
    want = clean.float()
    seeing = torch.zeros_like(want, dtype=torch.bool)
    seeing[new - 3:new, hq // h:, 16 * blk:] = True    # queries at positions n-3 .. n-1 of request 0
    assert got[seeing].isnan().all() and torch.equal(got[~seeing], want[~seeing])
    cache[3][at] = keep
    cache[1][at] = 0x7F
    got = S.kv4_attention(q, cache, lens_t, table).float()
    seeing[new - 3:new, hq // h:] = True
    assert got[seeing].isnan().all() and torch.equal(got[~seeing], want[~seeing])


def test_special_queries():
    case = ([50], 4, 2, 1, 128, 16, True, BF)
    q, cache, lens, table, start, causal = make(case, 41)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = S.kv4_attention(q, cache, lens_t, table).float()
    q[1, 0, 3], q[2, 1, 4] = float("nan"), float("inf")
    got = S.kv4_attention(q, cache, lens_t, table).float()
    bad = torch.zeros(4, 2, dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])
    # The ends of bf16: tiny queries weigh all keys alike, large ones pick one; neither overflows on the way.
    q2 = torch.zeros_like(q)
    q2[0], q2[1] = 1e-38, 3e38
    q2[2, :, 0], q2[2, :, 1] = 1e30, 1.0
    check(q2[:1], cache, lens, table, None, True)
    assert S.kv4_attention(q2[:3], cache, lens_t, table, softmax_scale=1e-38).isfinite().all()
    check(q, cache, lens, table, None, True, scale=0.0) if not q.isnan().any() else None


def test_pages_outside_the_cache_have_no_keys():
    """(After the same content has passed the host check of the index arithmetic.)"""
    case = ([100, 70, 33], 1, 4, 2, 128, 16, True, BF)
    q, cache, lens, table, start, causal = make(case, 51)
    table[0, 2], table[0, 4], table[1, :], table[2, 0] = -7, 1 << 30, -1, cache[0].shape[0]
    out, lse = check(q, cache, lens, table, start, causal)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_lengths_beyond_the_table_are_clamped():
    case = ([64, 32], 2, 4, 2, 64, 16, True, BF)
    q, cache, lens, table, start, causal = make(case, 61)
    table = table[:, :4].contiguous()
    lens_t = torch.tensor([64, -9], dtype=torch.int32, device="cuda")
    want = S.kv4_attention(q, cache, lens_t, table)
    got = S.kv4_attention(q, cache, torch.tensor([1 << 30, 0], dtype=torch.int32, device="cuda"), table)
    assert torch.equal(got, want) and (want[2:] == 0).all()
    empty = S.kv4_attention(q, cache, lens_t, table[:, :0])
    assert (empty == 0).all()
    assert S.kv4_attention(q[:0], cache, lens_t, table).shape == (0, 4, 64)


def test_offsets_beyond_32_bits():
    """Pages behind 2^31 codes and 2^32 bytes of the cache."""
    page, h, d = 256, 8, 128
    pages = (1 << 32) // (page * h * d // 2) + 3
    cache = S.kv4_cache(pages, page, h, d)
    g = gen(71)
    n = 500
    slots = torch.cat((torch.arange((pages - 1) * page, pages * page), torch.arange(n - page) + (pages // 2) * page)).cuda()
    k, v = heads(g, n, h, d, BF), heads(g, n, h, d, BF)
    S.kv4_append(cache, k, v, slots)
    small = S.kv4_cache(2, page, h, d)
    S.kv4_append(small, k, v, torch.arange(n, device="cuda"))
    for a, b in zip(S.kv4_read(cache, slots), S.kv4_read(small, torch.arange(n, device="cuda"))):
        assert torch.equal(a, b)
    q = heads(g, 1, 16, d, BF)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    far = torch.tensor([[pages - 1, pages // 2]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    assert torch.equal(S.kv4_attention(q, cache, lens, far), S.kv4_attention(q, small, lens, near))
    q = heads(g, 200, 16, d, BF)
    assert torch.equal(S.kv4_attention(q, cache, lens, far), S.kv4_attention(q, small, lens, near))


def test_attention_refusals():
    case = ([64, 32], 2, 4, 2, 64, 16, True, BF)
    q, cache, lens, table, start, causal = make(case, 61)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for err, call in [
        (TypeError, lambda: S.kv4_attention(q.float(), cache, n, table)),
        (ValueError, lambda: S.kv4_attention(q[0], cache, n, table)),
        (ValueError, lambda: S.kv4_attention(q[..., :32], cache, n, table)),
        (S.SvdqError, lambda: S.kv4_attention(q[:, :3], cache, n, table)),
        (S.SvdqError, lambda: S.kv4_attention(q[:3], cache, n, table)),
        (TypeError, lambda: S.kv4_attention(q, cache, n.long(), table)),
        (ValueError, lambda: S.kv4_attention(q, cache, n[:1], table)),
        (TypeError, lambda: S.kv4_attention(q, cache, n, table.long())),
        (ValueError, lambda: S.kv4_attention(q, cache, n, table[:1])),
        (ValueError, lambda: S.kv4_attention(q, cache, n, table.t().contiguous().t())),
        (ValueError, lambda: S.kv4_attention(q, cache, n, table, q_start=qs[:2])),
        (TypeError, lambda: S.kv4_attention(q, cache, n, table, q_start=qs.long())),
        (ValueError, lambda: S.kv4_attention(q, cache, n, table, out=q[:2])),
        (ValueError, lambda: S.kv4_attention(q, cache, n, table, out=q[:1].expand(4, 4, 64))),
        (TypeError, lambda: S.kv4_attention(q, cache, n, table, out=q.half())),
        (ValueError, lambda: S.kv4_attention(q, cache, n.cpu(), table)),
        (S.SvdqError, lambda: S.kv4_attention(q, cache, n, table, softmax_scale=float("inf"))),
        (S.SvdqError, lambda: S.kv4_attention(q, cache, n, table, max_kv_len=-1)),
        (ValueError, lambda: S.kv4_attention(q, cache[:3], n, table)),
    ]:
        with pytest.raises((err, IndexError) if err is ValueError else err):
            call()


def test_outputs_over_inputs_are_refused():
    case = ([64, 32], 2, 4, 2, 64, 16, True, BF)
    q, cache, lens, table, start, causal = make(case, 62)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = S.kv4_attention(q, cache, n, table)
    room = torch.zeros(6, 4, 64, dtype=BF, device="cuda")
    room[:4] = q
    for out in (room[:4], room[1:5], room[2:]):
        with pytest.raises(ValueError, match="overlap"):
            S.kv4_attention(room[:4], cache, n, table, out=out)
    both = torch.cat((q, torch.zeros_like(q)), 1)                # heads of one buffer, side by side
    assert S.kv4_attention(both[:, :4], cache, n, table, out=both[:, 4:]).data_ptr() == both[:, 4:].data_ptr()
    assert torch.equal(both[:, 4:], want) and torch.equal(both[:, :4], q)
    with pytest.raises(ValueError, match="overlap"):
        S.qk_norm_rope(q, q, torch.ones(64, dtype=BF, device="cuda"), inplace=True)


# ------------------------------------------------------------------ streams, graphs, and a run of them together

def test_calls_at_once_on_two_streams():
    calls = []
    for i, case in enumerate([([900, 1500], 256, 8, 2, 128, 64, True, BF), ([3000, 40], 1, 8, 2, 128, 64, True, BF),
                              ([700], 300, 4, 4, 64, 32, True, FP)]):
        q, cache, lens, table, start, causal = make(case, 90 + i)
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        calls.append((q, cache, n, table))
    want = [S.kv4_attention(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [S.kv4_attention(*calls[(i + j) % 3], stream=streams[j]) for i in range(12) for j in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(got[2 * i + j], want[(i + j) % 3]) for i in range(12) for j in range(2))


def test_streams_and_graphs():
    case = ([900, 40], 1, 8, 2, 128, 64, True, BF)
    q, cache, lens, table, start, causal = make(case, 81)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    f, axis = S.rope_frequencies((64,))
    pos = (n - 1)[:, None].contiguous()
    kn, vn = heads(gen(1), 2, 2, 128, BF), heads(gen(2), 2, 2, 128, BF)
    slots = torch.stack([table[b, (lens[b] - 1) // 64].long() * 64 + (lens[b] - 1) % 64 for b in range(2)])

    def step(**kw):
        a, b = S.qk_norm_rope(q, kn, positions=pos, inv_freq=f, hadamard=True, **kw)
        S.kv4_append(cache, b, vn, slots, **kw)
        return S.kv4_attention(a, cache, n, table, **kw)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(stream=side)
    also = step(stream=torch.cuda.Stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(also, want)
    graphs, outs = [], []
    for _ in range(2):                                 # two graphs: each has its own workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    # New inputs in the captured buffers: replays follow them, with the graphs side by side on two streams.
    q.copy_(heads(gen(3), 2, 8, 128, BF))
    n.copy_(torch.tensor([733, 21], dtype=torch.int32))
    pos.copy_((n - 1)[:, None])
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("rotate", [False, True])
def test_attention_block_from_projection_to_projection(rotate):
    """Packed W4A4 projection -> head norms, positions (and the Hadamard) -> 4-bit cache -> attention -> W4A4 output
    projection: a prompt, then a decoding step, each stage against its definition on the stage's actual input."""
    ck = synthetic.load("tiny_16x256x256_r32")

    def bf16(b):
        return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(BF).cuda()

    def u8(b):
        return torch.from_numpy(np.ascontiguousarray(b).view(np.uint8)).cuda()

    layer = S.SVDQLinear(u8(ck.qweight), u8(ck.wscales), bf16(ck.proj_down), bf16(ck.proj_up), bf16(ck.smooth_factor),
                         bf16(ck.wcscales), bf16(ck.wtscale))
    cache = S.kv4_cache(4, 16, 1, 64)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    f, axis = S.rope_frequencies((8, 12, 12))
    w = torch.linspace(0.5, 1.5, 64, device="cuda").to(BF)
    x = bf16(ck.x)
    seen = 0
    for rows in (x[:15], x[15:]):
        t = rows.shape[0]
        qkv = layer(rows.contiguous()).reshape(t, 4, 64)            # two query heads, one key head, one value head
        q, k, v = qkv[:, :2], qkv[:, 2:3], qkv[:, 3:]
        pos = (torch.arange(t, device="cuda", dtype=torch.int32) + seen)[:, None].repeat(1, 3)
        qr, kr = S.qk_norm_rope(q, k, w, w, positions=pos, inv_freq=f, pair_axis=axis, hadamard=rotate)
        for got, src in ((qr, q), (kr, k)):
            assert_rounded(got, *rope_reference(src, w, 1e-6, pos, f, axis, False, rotate), BF)
        at = torch.arange(seen, seen + t, device="cuda")
        slots = table[0, at // 16].long() * 16 + at % 16
        S.kv4_append(cache, kr, v, slots)
        codes, scales = quantized(kr)
        assert torch.equal(cache.k_codes[slots // 16, :, slots % 16].cpu(), codes)
        seen += t
        out, _ = check(qr, cache, [seen], table, None, True)
        y = layer(torch.cat((out, out), 1).reshape(t, 256))
        assert y.shape == (t, 256) and y.isfinite().all()
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    layer.close()


# ------------------------------------------------------------------ every size of a ragged call reaches a kernel

@pytest.mark.parametrize("start,group,dim", [([0, r], 1, 64) for r in (64, 65, 255, 256, 257, 511, 512, 513)] +
                         [([0, 64], 4, 128), ([0, 75], 4, 128), ([0, 128], 4, 128), ([0, 100, 512], 1, 128),
                          ([0, 256, 512], 1, 64), ([0, 1, 512], 1, 64), ([0, 0, 511, 512], 1, 64), ([130, 150], 2, 128)])
def test_ragged_calls_of_any_size_are_answered(start, group, dim):
    """(check fills the output with another value first; [130, 150] is one request in the middle of a padded batch.)"""
    n = len(start) - 1
    case = ([690, 300, 61][:n], start, group, 1, dim, 32, True, BF)
    q, cache, lens, table, start, causal = make(case, 101)
    q = q[:-1] if start[0] == 0 else torch.cat((q, q))          # as many rows as the requests have; or rows behind them
    check(q, cache, lens, table, start, causal)
    check(q, cache, lens, table, start, False, max_kv_len=max(lens))


# ------------------------------------------------------------------ the ends of the softmax scale and of the queries

@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-30, -1e-40])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-{c[1]}-{c[2:7]}".replace(" ", ""))
def test_scales_of_zero_and_next_to_it(case, scale):
    """All keys that a query sees weigh alike; masked ones nothing."""
    q, cache, lens, table, start, causal = make(case, 111)
    check(q, cache, lens, table, start, causal, scale=scale)


@pytest.mark.parametrize("causal", [False, True])
def test_tiny_queries_and_scales_of_many_rows(causal):
    """The factor of a row's exponents falls below fp32's range; rows without keys among them."""
    case = ([100, 70, 0], [0, 120, 190, 260], 2, 1, 128, 16, causal, BF)
    q, cache, lens, table, start, _ = make(case, 112)
    check(q * 1e-37, cache, lens, table, start, causal, scale=1e-5)
    check(q * 1e-37, cache, lens, table, start, causal)
    check(torch.zeros_like(q), cache, lens, table, start, causal)
    table[0, 1] = -1                                             # 16 keys in no page
    check(q, cache, lens, table, start, causal, scale=0.0)


@pytest.mark.parametrize("dim,dtype", [(64, FP), (128, BF)])
@pytest.mark.parametrize("new", [4, 150])
def test_special_queries_of_few_and_many_rows(new, dim, dtype):
    case = ([200], new, 2, 1, dim, 16, True, dtype)
    q, cache, lens, table, start, causal = make(case, 113)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for scale in (None, 0.0):
        clean = S.kv4_attention(q, cache, lens_t, table, softmax_scale=scale).float()
        x = q.clone()
        x[1, 0, 3], x[new - 1, 1, 4], x[new // 2, 1] = float("nan"), float("inf"), float("-inf")
        got = S.kv4_attention(x, cache, lens_t, table, softmax_scale=scale).float()
        bad = torch.zeros(new, 2, dtype=torch.bool)
        bad[1, 0] = bad[new - 1, 1] = bad[new // 2, 1] = True
        assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])
    # The type's ends: tiny queries weigh all keys alike, the largest ones are scaled back into range.
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    check(torch.full_like(q, tiny), cache, lens, table, None, True)
    check((torch.sign(q) * big).to(dtype), cache, lens, table, None, True, scale=0.5 / big)


# ------------------------------------------------------------------ many small weights beside a large one

@pytest.mark.parametrize("new,dim,dtype", [(1, 128, BF), (1, 64, FP), (20, 128, FP), (80, 128, BF), (80, 64, FP), (300, 64, BF)])
def test_many_small_weights_beside_a_large_one(new, dim, dtype):
    """Every 32nd key weighs 2^26 times the others and has values of zero: the output is what the others leave.  The
    bound is attend_reference's with the weights' absolute rounding where it has to lie: a weight is rounded to fp16
    after a factor of at least 2^7, so to 2^-25 / 2^7 of the largest one (below fp16's normal range), and to 2^-11 of
    itself above it; the sum of weights divides both."""
    keys, page = 3000, 64
    pages = -(-keys // page)
    cache = S.kv4_cache(pages, page, 1, dim)
    n = pages * page
    large = torch.arange(n, device="cuda") % 32 == 0
    k = torch.zeros(n, 1, dim, dtype=dtype, device="cuda")
    k[:, 0, 0] = torch.where(large, 6.0, -6.0).to(dtype)
    v = torch.rand(n, 1, dim, device="cuda", generator=gen(121)) + 0.5
    v[large] = 0
    S.kv4_append(cache, k, v.to(dtype), torch.arange(n, device="cuda"))
    q = torch.zeros(new, 1, dim, dtype=dtype, device="cuda")
    q[..., 0] = 1
    scale = float(np.float32(26 * math.log(2) / 12))
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    out, lse = S.kv4_attention(q, cache, torch.tensor([keys], dtype=torch.int32, device="cuda"), table, causal=False,
                               softmax_scale=scale, return_lse=True)
    kk, vv = (values(cache, i).reshape(n, dim)[:keys] for i in (0, 2))
    s = kk[:, 0] * scale
    l = torch.logsumexp(s, 0)
    want = torch.exp(s - l) @ vv
    ds = 2.0 ** -23 * (dim + 4) * 6 * scale + 2.0 ** -22 * (6 * scale + 1)
    bound = (2.0 ** -11 + 2 * ds + 2 * keys * 2.0 ** -24) * want + 2.0 ** -32 * vv.sum(0) / torch.exp(l - s.max())
    assert (bound < 0.02 * want).all()                          # (a bound that would notice their absence)
    assert_rounded(out[:, 0], want.expand(new, dim), bound.expand(new, dim), dtype)
    assert ((lse.double() - l).abs() <= ds + keys * 2.0 ** -24 + 2.0 ** -22 * (1 + l.abs())).all()


# ------------------------------------------------------------------ outputs that lie over inputs, in packed buffers

def test_outputs_over_inputs_of_a_packed_buffer_are_refused():
    q, cache, lens, table, start, causal = make(([64, 32], 2, 4, 2, 64, 16, True, BF), 131)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = S.kv4_attention(q, cache, n, table)
    packed = torch.zeros(6, 12, 64, dtype=BF, device="cuda")
    by_head = torch.zeros(12, 6, 64, dtype=BF, device="cuda").transpose(0, 1)
    for buf in (packed, by_head):
        buf[:4, :4] = q
        for out in (buf[:4, 1:5], buf[:4, 3:7], buf[1:5, :4], buf[2:6, 2:6], buf[:4, 0:8:2], buf[1:5, 3:12:2][:, :4]):
            with pytest.raises(ValueError, match="overlap"):
                S.kv4_attention(buf[:4, :4], cache, n, table, out=out)
        for out in (buf[:4, 4:8], buf[:4, 4:12:2]):
            S.kv4_attention(buf[:4, :4], cache, n, table, out=out)
            assert torch.equal(out, want) and torch.equal(buf[:4, :4], q)
        buf.zero_()
        buf[:4, 0:8:2] = q                                       # heads of queries and outputs in turn
        S.kv4_attention(buf[:4, 0:8:2], cache, n, table, out=buf[:4, 1:9:2])
        assert torch.equal(buf[:4, 1:9:2], want) and torch.equal(buf[:4, 0:8:2], q)
        w = torch.ones(64, dtype=BF, device="cuda")
        before = buf.clone()
        for k in (buf[:, 3:5], buf[:, 2:8:2], buf[:, :4]):
            with pytest.raises(ValueError, match="overlap"):
                S.qk_norm_rope(buf[:, :4], k, w, inplace=True)
        assert torch.equal(buf, before)
        S.qk_norm_rope(buf[:, :4], buf[:, 4:6], w, w, inplace=True)


def test_outputs_over_the_cache_and_the_cache_over_inputs_are_refused():
    page, h, d = 16, 2, 64
    rows = 4 * h * page
    arena = torch.zeros(rows * (d + d // 8) + 4 * 2 * h * d * 2, dtype=torch.uint8, device="cuda")
    sizes, cache, at = (d // 2, d // 16, d // 2, d // 16), [], 0
    for n in sizes:
        cache.append(arena[at:at + rows * n].view(4, h, page, n))
        at += rows * n
    k, v = (arena[at + i * 4 * h * d * 2:][:4 * h * d * 2].view(BF).view(4, h, d) for i in range(2))
    k.copy_(heads(gen(132), 4, h, d, BF))
    v.copy_(heads(gen(133), 4, h, d, BF))
    slots = torch.tensor([0, 17, 40, 63], device="cuda")
    S.kv4_append(cache, k, v, slots)                             # side by side in one buffer
    other = S.kv4_cache(4, page, h, d)
    S.kv4_append(other, k, v, slots)
    assert all(torch.equal(a, b) for a, b in zip(cache, other)) and cache[0].any()
    over = arena[at - 512:][:4 * h * d * 2].view(BF).view(4, h, d)
    for call in (lambda: S.kv4_append(cache, over, v, slots), lambda: S.kv4_append(cache, k, over, slots),
                 lambda: S.kv4_append(cache, k, v, cache[2].view(-1)[:32].view(torch.int64)),
                 lambda: S.kv4_append((cache[0], cache[1], cache[0], cache[3]), k, v, slots),
                 lambda: S.kv4_append((cache[0], cache[1], cache[2], cache[1]), k, v, slots)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    n = torch.tensor([60], dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for out in (over, cache[0].view(-1)[:4 * h * d * 2].view(BF).view(4, h, d)):
        with pytest.raises(ValueError, match="overlap"):
            S.kv4_attention(k, cache, n, table, out=out)
    assert all(torch.equal(a, b) for a, b in zip(cache, other))
    # Reading is free to share: keys that serve as values too.
    both = (cache[0], cache[1], cache[0], cache[1])
    a, b = S.kv4_read(both, slots)
    assert torch.equal(a, b)
    assert torch.equal(S.kv4_attention(k, both, n, table, out=v), S.kv4_attention(k, both, n, table))


# ------------------------------------------------------------------ autograd: no backward pass, and no silence about it

def test_gradients_are_refused_not_lost():
    q, cache, lens, table, _, _ = make(([64, 32], 2, 4, 2, 64, 16, True, BF), 141)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    f, _ = S.rope_frequencies((32,))
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    k = heads(gen(142), 4, 2, 64, BF)

    def norm(x=q, y=k, a=w, b=w, g=f, **kw):
        return S.qk_norm_rope(x, y, a, b, positions=pos, inv_freq=g, **kw)

    def grad(t):
        return t.clone().requires_grad_()

    def attend(x, **kw):
        return S.kv4_attention(x, cache, n, table, return_lse=True, **kw)

    plain, seen = norm(), attend(q)
    assert not any(t.requires_grad for t in plain + seen)
    for name, want, got in [("qk_norm_rope", plain, norm(x=grad(q))), ("qk_norm_rope", plain, norm(y=grad(k))),
                            ("qk_norm_rope", plain, norm(a=grad(w))), ("qk_norm_rope", plain, norm(b=grad(w))),
                            ("qk_norm_rope", plain, norm(g=grad(f))), ("kv4_attention", seen, attend(grad(q))),
                            ("qk_norm_rope", plain, norm(x=grad(q) * 1.0, y=k.expand(4, 2, 64)))]:
        for a, b in zip(want, got):
            assert torch.equal(a, b) and b.requires_grad
            with pytest.raises(RuntimeError, match=name + " is not implemented"):
                b.float().sum().backward()
    assert not S.qk_norm_rope(grad(q).detach())[0].requires_grad
    with torch.no_grad():
        assert not any(t.requires_grad for t in norm(x=grad(q)) + attend(grad(q)))
    for call in (lambda: norm(x=grad(q), inplace=True), lambda: norm(x=q.clone(), y=grad(k), inplace=True),
                 lambda: norm(x=q.clone(), y=k.clone(), a=grad(w), inplace=True),
                 lambda: attend(q, out=grad(q)), lambda: attend(grad(q), out=torch.empty_like(q))):
        with pytest.raises(RuntimeError, match="no backward pass"):
            call()
    with torch.no_grad():
        x = grad(q)
        assert torch.equal(norm(x=x, y=k.clone(), inplace=True)[0], plain[0])
        out = torch.empty_like(q)
        assert torch.equal(attend(grad(q), out=out)[0], seen[0])


def test_written_tensors_change_their_version():
    q, cache, lens, table, _, _ = make(([64, 32], 2, 4, 2, 64, 16, True, BF), 143)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k = heads(gen(144), 4, 2, 64, BF)
    out = torch.empty_like(q)

    def versions():
        return [t._version for t in (q, k, out, *cache)]

    v = versions()
    S.kv4_append(cache, k, k, torch.arange(4, device="cuda"))
    assert versions() == v[:3] + [x + 1 for x in v[3:]]
    v = versions()
    S.kv4_attention(q, cache, n, table, out=out)
    assert versions() == v[:2] + [v[2] + 1] + v[3:]
    v = versions()
    S.kv4_read(cache, torch.arange(4, device="cuda"))
    S.qk_norm_rope(q, k)
    assert versions() == v
    w = torch.ones(4, 1, 1, device="cuda", dtype=BF, requires_grad=True)
    y = (w * q).sum()                                            # keeps q for w's gradient
    S.qk_norm_rope(q, k, inplace=True)
    assert versions() == [v[0] + 1, v[1] + 1] + v[2:]
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()
    with torch.inference_mode():                                 # tensors that have no version
        c, a = S.kv4_cache(4, 16, 2, 64), k.clone()
        S.kv4_append(c, a, a, torch.arange(4, device="cuda"))
        S.qk_norm_rope(a, inplace=True)
    S.kv4_append(c, k, k, torch.arange(4, device="cuda"))
    assert S.kv4_read(c, torch.arange(4, device="cuda"))[0].any()


@pytest.mark.parametrize("new", [3, 150])
def test_largest_scales(new):
    """Scores of zero stay zero under any scale; tiny queries under a large one have scores of ordinary size."""
    q, cache, lens, table, start, causal = make(([200], new, 2, 1, 128, 16, True, BF), 151)
    top = float(torch.finfo(torch.float32).max)
    for scale in (top, -top, 2.0 ** 127):
        check(torch.zeros_like(q), cache, lens, table, None, True, scale=scale)
    for scale in (1e36, -3e36):
        check(q * 1e-37, cache, lens, table, None, True, scale=scale)


# ------------------------------------------------------------------ every instance of the few-row kernel, and both kernels in one call

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [3, 8, 9, 16, 17, 23, 24, 25, 32, 33, 64, 65])
def test_group_sizes(group, dim, dtype):
    """Rows a request of each tile of the few-row kernel (8, 16, 24 and 32 rows), one past it, and past that kernel."""
    q, cache, lens, table, start, causal = make(([300, 37], 1, 2 * group, 2, dim, 16, True, dtype), 161)
    check(q, cache, lens, table, start, causal)
    case = ([300, 37], [0, 3, 4], 2 * group, 2, dim, 32, True, dtype)
    q, cache, lens, table, start, causal = make(case, 162)
    check(q, cache, lens, table, start, causal)


@pytest.mark.parametrize("dim,dtype,causal", [(128, BF, True), (128, FP, True), (64, BF, True), (128, BF, False)])
def test_prompts_beside_single_and_drafted_tokens(dim, dtype, causal):
    lens = [650, 1, 300, 129, 0, 280, 90, 33, 512]
    start = [0, 1, 2, 180, 181, 182, 190, 191, 195, 400]
    q, cache, lens, table, start, _ = make((lens, start, 8, 2, dim, 32, causal, dtype), 163)
    a = check(q, cache, lens, table, start, causal)
    b = check(q, cache, lens, table, start, causal)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].nan_to_num(), b[1].nan_to_num())
    check(q, cache, lens, table, start, causal, scale=-0.15, max_kv_len=700)


# ------------------------------------------------------------------ the C entry points by their descriptions

def test_calls_by_description():
    """The ctypes mirrors of the header against the calls with tensors."""
    t, hq, h, d, page = 5, 4, 2, 128, 16
    g = gen(164)
    packed = heads(g, t, hq + 2 * h, d, FP)
    q, k, v = packed[:, :hq], packed[:, hq:hq + h], packed[:, hq + h:]
    w = torch.rand(d, device="cuda", generator=g).to(FP)
    f, axis = S.rope_frequencies((16, 24))
    pos = torch.randint(0, 999, (t, 2), device="cuda", generator=g, dtype=torch.int32)
    stream = torch.cuda.current_stream().cuda_stream

    def side(x):
        return attention.svdq_heads(x.data_ptr(), x.stride(0), x.stride(1))

    want = S.qk_norm_rope(q, k, w, w, positions=pos, inv_freq=f, pair_axis=axis, hadamard=True)
    qo, ko = torch.empty(t, hq, d, dtype=FP, device="cuda"), torch.empty(t, h, d, dtype=FP, device="cuda")
    attention.svdq_qk_norm_rope(attention.svdq_qk_norm_rope_desc(
        t, hq, h, d, 1, side(q), side(k), side(qo), side(ko), w.data_ptr(), w.data_ptr(), 1e-6, pos.data_ptr(), 2, 2,
        f.data_ptr(), axis.data_ptr(), 40, 0, 1), stream)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    caches = [S.kv4_cache(3, page, h, d) for _ in range(2)]
    slots = torch.tensor([40, 3, -1, 17, 16], device="cuda")
    S.kv4_append(caches[0], ko, v, slots)
    c = attention.svdq_kv4_cache(*(x.data_ptr() for x in caches[1]), 3, h, page, d)
    attention.svdq_kv4_append(c, side(ko), side(v), t, 1, slots.data_ptr(), stream)
    assert all(torch.equal(a, b) for a, b in zip(*caches)) and caches[1][0].any()
    lens, table = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([9], [[1, 2]]))
    want = S.kv4_attention(qo, caches[0], lens, table, return_lse=True)
    out, lse = torch.empty_like(qo), torch.empty(t, hq, device="cuda")
    desc = attention.svdq_kv4_attention_desc(c, t, 1, hq, 1, side(qo), side(out), lse.data_ptr(), lens.data_ptr(), None,
                                             table.data_ptr(), 2, 2, 0, 1, d ** -0.5)
    size = attention.svdq_kv4_attention_workspace_bytes(desc)
    work = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    attention.svdq_kv4_attention(desc, work.data_ptr(), size, stream)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("new", [3, 150])
def test_largest_scales_of_smallest_queries(new):
    q, cache, lens, table, start, causal = make(([200], new, 2, 1, 128, 16, True, BF), 171)
    for scale in (3e38, -3.4e38):
        check(q * 1e-38, cache, lens, table, None, True, scale=scale)
