"""Attention over a prefix shared by a batch and per-request caches
(swa_attn_fwd_shared) against the definition in 64 bits.

Tolerances.  P is rounded to bf16 (half a step, 2^-8 of each term) for the
product with v, and o once more (2^-8 of the value); scores carry
2^-18 * scale * sum |q k| at most (fp32 accumulation over D <= 512 products of
exact bf16 factors), which shifts a term by that much again, and the sums
2^-14 at most.  So |o - ref| <= (2^-8 + s + 2^-14) sum p |v| + 2^-8 |ref| with
s = 2^-17 * scale * max sum |q k| (numerator and normaliser), and
|lse - ref| <= s + 2^-18 (1 + |ref|).
"""
import math

import pytest
import torch

BF = torch.bfloat16


def make(B, Hq, Hkv, Lq, D, P, rows, seed, sinks=False, prefix_rows=None):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g).to(BF)

    q, ko, vo = r(B, Hq, Lq, D), r(B, Hkv, rows, D), r(B, Hkv, rows, D)
    pr = P if prefix_rows is None else prefix_rows
    return dict(q=q, kp=r(Hkv, pr, D), vp=r(Hkv, pr, D), ko=ko, vo=vo,
                sinks=torch.randn(Hq, generator=g) if sinks else None)


def reference(a, lens, P, window, scale):
    """(o, lse, sum p |v|, max scale sum |q k|) in fp64; NaN rows for empty places."""
    q = a["q"]
    B, Hq, Lq, D = q.shape
    G = Hq // a["ko"].shape[1]
    rows = a["ko"].shape[2]
    o, mag = torch.full((2, B, Hq, Lq, D), math.nan, dtype=torch.float64)
    lse, s = torch.full((2, B, Hq, Lq), math.nan, dtype=torch.float64)
    for b in range(B):
        n = min(int(lens[b]), rows)
        if n < 0:
            continue
        k = torch.cat((a["kp"][:, :P], a["ko"][b, :, :n]), 1).double().repeat_interleave(G, 0)
        v = torch.cat((a["vp"][:, :P], a["vo"][b, :, :n]), 1).double().repeat_interleave(G, 0)
        x = q[b].double() @ k.transpose(1, 2) * scale
        pos = P + n - Lq + torch.arange(Lq)[:, None]
        j = torch.arange(P + n)[None]
        see = j <= pos
        if window:
            see &= pos - j < window
        x = x.masked_fill(~see, -math.inf)
        if a["sinks"] is not None:
            x = torch.cat((x, a["sinks"].double()[:, None, None].expand(Hq, Lq, 1)), 2)
        m = x.amax(2, keepdim=True) if x.shape[2] else torch.full((Hq, Lq, 1), -math.inf, dtype=torch.float64)
        m = torch.where(m == -math.inf, 0.0, m)
        e = torch.exp(x - m)
        z = e.sum(2, keepdim=True)
        p = torch.where(z > 0, e / z, 0.0)[..., :P + n]
        o[b], mag[b] = p @ v, p @ v.abs()
        lse[b] = (m + torch.log(z))[..., 0]
        big = (q[b].double().abs() @ k.abs().transpose(1, 2) * abs(scale)).masked_fill(~see, 0.0)
        s[b] = big.amax(2) if big.shape[2] else 0.0
    return o, lse, mag, s


def run(a, lens, P, window, scale, **kw):
    import sliding_window_attention_gb300 as swa

    d = {n: None if t is None else t.cuda() for n, t in a.items()}
    lens = torch.as_tensor(lens, dtype=torch.int32).cuda()
    o, lse = swa.forward_shared(d["q"], d["kp"], d["vp"], d["ko"], d["vo"], lens, window, scale, prefix_len=P,
                                sinks=d["sinks"], **kw)
    torch.cuda.synchronize()
    assert swa.swa_attn_get_status() == 0
    return o, lse


def check(got, ref):
    o, lse = (t.double().cpu() for t in got)
    ro, rl, mag, s = ref
    live = ~torch.isnan(rl)
    s = 2.0 ** -17 * s
    tol = (2.0 ** -8 + s[..., None] + 2.0 ** -14) * mag + 2.0 ** -8 * ro.abs()
    err = (o - ro).abs()
    assert torch.isfinite(o[live]).all()
    bad = (err > tol)[live]
    assert not bad.any(), f"o: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol.clamp_min(1e-30))[live].max()):.2f} of the tolerance"
    empty = live & (rl == -math.inf)
    assert torch.equal(lse[empty], rl[empty]) and not o[empty].any()
    some = live & ~empty
    e = (lse - rl).abs()[some]
    t = (s + 2.0 ** -18 * (1 + rl.abs()))[some]
    assert (e <= t).all(), f"lse: worst {float((e / t).max()):.2f} of the tolerance"


CASES = [
    # B, Hq, Hkv, Lq, D, P, own rows, lengths, window, sinks
    (1, 1, 1, 1, 64, 1, 1, [1], 0, False),
    (1, 2, 1, 1, 128, 128, 1, [0], 0, False),            # the prefix alone, one tile
    (2, 2, 1, 1, 64, 0, 130, [130, 1], 0, False),        # no prefix
    (3, 4, 2, 1, 128, 129, 40, [40, 1, 17], 0, False),
    (4, 8, 4, 1, 128, 1000, 300, [300, 129, 128, 127], 0, False),
    (2, 8, 1, 2, 256, 500, 64, [64, 2], 0, False),       # 16 rows a request: one block of 16 each way
    (5, 8, 2, 1, 512, 333, 200, [1, 200, 0, 131, 77], 0, False),
    (9, 8, 1, 1, 64, 700, 30, list(range(9)), 0, True),  # 72 rows: two prefix blocks, the second part full
    (17, 4, 1, 1, 256, 260, 10, [10] * 17, 0, False),
    (40, 4, 2, 1, 128, 640, 20, [i % 21 for i in range(40)], 0, False),
    (3, 6, 2, 5, 64, 300, 50, [50, 5, 20], 0, True),     # 15 rows a request, 3 heads a group
    (2, 16, 1, 2, 128, 200, 40, [40, 2], 0, False),      # 32 rows a request: two own blocks
    (2, 16, 1, 5, 64, 333, 300, [300, 150], 0, False),   # 80 rows a request: two prefix blocks each
    (1, 32, 1, 6, 256, 130, 140, [139], 100, True),      # 192 rows a request
    (6, 8, 1, 3, 512, 257, 129, [129, 3, 60, 128, 4, 100], 0, False),
    (4, 4, 2, 1, 256, 900, 400, [400, 10, 1, 0], 200, False),   # the window leaves some rows no prefix
    (4, 2, 1, 3, 128, 300, 500, [500, 400, 499, 450], 128, False),  # and here none of it to anyone
    (3, 2, 1, 4, 64, 50, 60, [60, 7, 33], 1, False),     # each row sees its own key alone
    (2, 4, 4, 1, 64, 5000, 3000, [3000, 12], 0, False),
    (3, 4, 2, 4, 128, 2, 10, [1, 0, 4], 0, False),       # sequences shorter than the queries: rows without a key
    (3, 4, 2, 4, 128, 2, 10, [1, 0, 4], 0, True),
    (6, 4, 2, 1, 128, 200, 90, [-1, 30, -7, 0, 95, 90], 0, False),  # empty places, a length past the cache
    (70, 2, 1, 1, 64, 100, 5, [(-1 if i % 3 else 5) for i in range(70)], 0, False),
    (200, 2, 2, 1, 64, 64, 3, [i % 4 for i in range(200)], 0, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,P,rows,lens,window,sinks", CASES)
def test_matches_definition(B, Hq, Hkv, Lq, D, P, rows, lens, window, sinks):
    a = make(B, Hq, Hkv, Lq, D, P, rows, 7 * B + D + P, sinks)
    scale = D ** -0.5
    got = run(a, lens, P, window, scale)
    check(got, reference(a, lens, P, window, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("B", [3, 12])
def test_what_lies_behind_the_lengths_is_never_read(D, B):
    """NaN and infinities behind the prefix's and every cache's length change no bit."""
    Hq, Hkv, P, rows = 4, 1, 150, 260
    a = make(B, Hq, Hkv, 1, D, P, rows, 5, prefix_rows=200)
    lens = [(37 * b + 1) % rows for b in range(B)]
    clean = run(a, lens, P, 0, 0.1)
    check(clean, reference(a, lens, P, 0, 0.1))
    for n in ("kp", "vp"):
        a[n][:, P:] = math.nan
    for b, n in enumerate(lens):
        a["ko"][b, :, n:] = math.inf
        a["vo"][b, :, n:] = math.nan
    for x, y in zip(clean, run(a, lens, P, 0, 0.1)):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales_and_growing_maxima(scale):
    """A scale of 0 and a negative one; scores whose maximum keeps growing along the keys, so that references move
    at many tiles (in blocks of 64 rows and of 16)."""
    for B, D in ((20, 64), (20, 256), (2, 128)):
        a = make(B, 4, 1, 1, D, 700, 300, 11)
        ramp = torch.linspace(0.0, 3.0, 700)[None, :, None]
        a["kp"] = (a["kp"].float() * ramp).to(BF)
        a["ko"] = (a["ko"].float() * 4).to(BF)
        lens = [300 - 7 * b for b in range(B)]
        check(run(a, lens, 700, 0, scale), reference(a, lens, 700, 0, scale))


@pytest.mark.gpu
def test_extreme_values():
    """One key far above all others (weights of exactly 0 elsewhere), and a request whose queries are NaN:
    only its own rows are."""
    a = make(6, 2, 1, 1, 128, 256, 100, 13)
    a["kp"][0, 17] = (a["q"][0, 0, 0].float() * 40).to(BF)
    lens = [100, 50, 3, 99, 1, 64]
    ref = reference(a, lens, 256, 0, 1.0)
    base = run(a, lens, 256, 0, 1.0)
    check(base, ref)
    a["q"][2] = math.nan
    o, lse = run(a, lens, 256, 0, 1.0)
    keep = torch.tensor([0, 1, 3, 4, 5], device="cuda")
    assert torch.isnan(o[2]).all() and torch.equal(o[keep], base[0][keep]) and torch.equal(lse[keep], base[1][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("B,D", [(2, 64), (30, 64), (70, 64), (2, 128), (2, 256), (2, 512)])
def test_large_values_behind_scores_that_grow(B, D):
    """Every second tile's scores are 2^28.9 above those of the tile before it, and v is of the order of 2^100: the
    products with v must not leave fp32's range where the definition does not (128 such keys' sum is below 2^110)."""
    H, P, rows = 64, 1024, 256
    a = make(B, H, H, 1, D, P, rows, 12)
    a["q"] = torch.ones_like(a["q"])
    high = torch.arange(P) // 128 % 2 * (20.0 / D)  # scores of 20 / D rounded to bf16, D times
    a["kp"] = high[None, :, None].to(BF).expand(H, P, D).contiguous()
    a["ko"] = high[None, None, :rows, None].to(BF).expand(B, H, rows, D).contiguous()
    a["vp"], a["vo"] = a["vp"] * 2.0 ** 100, a["vo"] * 2.0 ** 100
    lens = [256 if b % 3 else 128 for b in range(B)]
    check(run(a, lens, P, 0, 1.0), reference(a, lens, P, 0, 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,P,rows,window", [
    (700, 64, 8, 1, 64, 70, 3, 0),      # more prefix segments than pieces, more requests than a CTA's threads
    (1500, 2, 1, 1, 128, 129, 130, 0),  # rounds of 128 rows over three times a CTA's threads
    (650, 1, 1, 1, 512, 65, 140, 50),
    (330, 1, 1, 3, 256, 1, 2, 0),
])
def test_many_requests(B, Hq, Hkv, Lq, D, P, rows, window):
    a = make(B, Hq, Hkv, Lq, D, P, rows, 3)
    lens = [(i * 37) % (rows + 2) - 1 for i in range(B)]  # empty places and lengths of zero among them
    got = run(a, lens, P, window, 0.2)
    ref = reference(a, lens, P, window, 0.2)
    check(got, ref)


@pytest.mark.gpu
def test_only_empty_places():
    import sliding_window_attention_gb300 as swa

    a = {n: None if t is None else t.cuda() for n, t in make(5, 4, 2, 2, 128, 300, 40, 1).items()}
    lens = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(a["q"], 7), torch.full((5, 4, 2), 7.0, device="cuda")
    ws = torch.empty(swa.fwd_workspace_bytes_shared(5, 4, 2, 2, 300, 40, 128, 0), dtype=torch.uint8, device="cuda")
    swa.swa_attn_fwd_shared(a["q"], a["kp"], a["vp"], a["ko"], a["vo"], lens, None, o, lse, 0, 0.1, workspace=ws)
    torch.cuda.synchronize()
    assert swa.swa_attn_get_status() == 0 and (o == 7).all() and (lse == 7).all()


@pytest.mark.gpu
def test_steps_back_to_back():
    """Appends, attention and growing lengths with nothing between them on the stream, against the same steps one by
    one: a kernel that starts before its predecessor has ended must not read what that one still writes."""
    import sliding_window_attention_gb300 as swa

    B, Hq, Hkv, D, P, rows, steps = 6, 8, 2, 128, 200, 64, 40
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((steps, B, 1, Hq + 2 * Hkv, D), device="cuda", generator=g).to(BF)
    kp, vp = (torch.randn((Hkv, P, D), device="cuda", generator=g).to(BF) for _ in range(2))
    f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
    w = torch.ones(D, device="cuda")

    def chain(wait):
        kc, vc = (torch.zeros((B, Hkv, rows, D), dtype=BF, device="cuda") for _ in range(2))
        n = torch.tensor([1, 5, 9, 13, 17, 21], dtype=torch.int32, device="cuda")
        outs = []
        torch.cuda.synchronize()
        for i in range(steps):
            q, k, v = x[i].split((Hq, Hkv, Hkv), 2)
            q = swa.qk_rope_append(q, k, v, w, w, f, kc, vc, n, 1e-6, pos0=P)
            outs.append(swa.forward_shared(q, kp, vp, kc, vc, n, 0, 0.1))
            n += 1
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, kc, vc

    (outs, kc, vc), (want, kw, vw) = chain(False), chain(True)
    assert torch.equal(kc, kw) and torch.equal(vc, vw)
    for (o, lse), (po, pl) in zip(outs, want):
        assert torch.equal(o, po) and torch.equal(lse, pl)


@pytest.mark.gpu
def test_two_threads_on_two_streams():
    """Calls of two threads at once, each on its own stream: each call's own bits."""
    import threading

    import sliding_window_attention_gb300 as swa

    cases = []
    for lens, shape in (([90, 1, 37], (8, 2, 1, 128, 300, 90)), ([130] * 20, (4, 2, 2, 64, 513, 200))):
        a = make(len(lens), *shape, seed=5)
        cases.append([a[n].cuda() for n in ("q", "kp", "vp", "ko", "vo")] + [torch.tensor(lens, dtype=torch.int32).cuda()])
    alone = [swa.forward_shared(*x, 0, 0.2) for x in cases]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in cases]

    def calls(i):
        for _ in range(50):
            got[i].append(swa.forward_shared(*cases[i], 0, 0.2, stream=streams[i]))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for want, outs in zip(alone, got):
        assert len(outs) == 50
        for o, lse in outs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_a_cache_beyond_32_bits():
    """Caches of more than 2^32 bytes and 2^31 elements, against 64 bits on the GPU in parts."""
    import sliding_window_attention_gb300 as swa

    B, Hq, D, rows = 2, 2, 128, (1 << 30) // 128 + 777
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((B, Hq, 1, D), device="cuda", generator=g).to(BF)
    ko, vo = (torch.randn((B, 1, rows, D), device="cuda", generator=g, dtype=BF) for _ in range(2))
    kp, vp = (torch.randn((1, 200, D), device="cuda", generator=g).to(BF) for _ in range(2))
    lens = [rows, rows - 1000]
    o, lse = swa.forward_shared(q, kp, vp, ko, vo, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0, 0.3)
    for b, n in enumerate(lens):
        z, num, mag = (torch.zeros((Hq, c), dtype=torch.float64, device="cuda") for c in (1, D, D))
        for i in range(0, n, 1 << 20):
            e = torch.exp(q[b, :, 0].double() @ ko[b, 0, i:min(n, i + (1 << 20))].double().T * 0.3)
            v = vo[b, 0, i:min(n, i + (1 << 20))].double()
            z += e.sum(1, keepdim=True)
            num += e @ v
            mag += e @ v.abs()
        e = torch.exp(q[b, :, 0].double() @ kp[0].double().T * 0.3)
        z, num, mag = z + e.sum(1, keepdim=True), num + e @ vp[0].double(), mag + e @ vp[0].double().abs()
        ref = num / z
        assert ((o[b, :, 0].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -11) * mag / z + 2.0 ** -8 * ref.abs()).all()
        assert ((lse[b, :, 0].double() - z[:, 0].log()).abs() <= 2.0 ** -12).all()


@pytest.mark.gpu
def test_empty_places_keep_their_rows():
    import sliding_window_attention_gb300 as swa

    a = {n: None if t is None else t.cuda() for n, t in make(4, 4, 2, 2, 64, 100, 20, 3).items()}
    o = torch.full_like(a["q"], 7.0)
    lse = torch.full((4, 4, 2), 9.0, device="cuda")
    ws = torch.full((swa.fwd_workspace_bytes_shared(4, 4, 2, 2, 100, 20, 64, 0),), 255, dtype=torch.uint8, device="cuda")
    for lens in ([5, -1, 20, -2 ** 31], [-1, -1, -1, -1]):
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        swa.swa_attn_fwd_shared(a["q"], a["kp"], a["vp"], a["ko"], a["vo"], n, None, o, lse, 0, 0.1, workspace=ws)
        for b, x in enumerate(lens):
            assert (x >= 0) != (bool((o[b] == 7.0).all()) and bool((lse[b] == 9.0).all()))
        o.fill_(7.0)
        lse.fill_(9.0)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,P,n,window", [(3, 8, 4, 1, 128, 600, 77, 0), (2, 16, 2, 2, 256, 300, 200, 150)])
def test_equals_the_decode_step_on_the_joined_cache(B, Hq, Hkv, Lq, D, P, n, window):
    """Equal lengths: the same numbers as swa_attn_fwd_ex on [prefix; own] of each request, up to both
    calls' roundings of P and the bf16 of o."""
    import sliding_window_attention_gb300 as swa

    a = make(B, Hq, Hkv, Lq, D, P, n, 23)
    o, lse = run(a, [n] * B, P, window, D ** -0.5)
    k, v = (torch.cat((a[p][None].expand(B, -1, -1, -1), a[w]), 2).contiguous().cuda() for p, w in (("kp", "ko"), ("vp", "vo")))
    ro, rl = swa.forward(a["q"].cuda(), k, v, window, D ** -0.5)
    mag = reference(a, [n] * B, P, window, D ** -0.5)[2].cuda()
    assert ((o.double() - ro.double()).abs() <= (2 * 2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * ro.abs()).all()
    assert (lse - rl).abs().max() <= 2.0 ** -14


@pytest.mark.gpu
def test_repeats_streams_and_workspaces():
    """Equal calls give equal bits; two calls overlap on two streams with their own workspaces."""
    a, b = make(24, 8, 2, 1, 128, 2000, 200, 1), make(5, 4, 4, 2, 256, 900, 150, 2)
    la, lb = [(13 * i) % 201 for i in range(24)], [150, 2, 60, 4, 130]
    ra, rb = run(a, la, 2000, 0, 0.1), run(b, lb, 900, 0, 0.1)
    import sliding_window_attention_gb300 as swa

    def args(x, lens):
        d = {n: None if t is None else t.cuda() for n, t in x.items()}
        return d["q"], d["kp"], d["vp"], d["ko"], d["vo"], torch.tensor(lens, dtype=torch.int32, device="cuda"), 0, 0.1

    xa, xb = args(a, la), args(b, lb)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, x in ((s1, xa), (s2, xb)):
            with torch.cuda.stream(s):
                got.append(swa.forward_shared(*x))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        r = rb if i % 2 else ra
        assert torch.equal(o, r[0]) and torch.equal(lse, r[1])


@pytest.mark.gpu
@pytest.mark.parametrize("sinks", [False, True])
def test_both_marshalling_paths_give_the_same(sinks):
    """With numpy scalars (marshalled in Python), others (in C++), and on a stream of the call's own: equal bits."""
    import numpy as np

    import sliding_window_attention_gb300 as swa

    a = {n: None if t is None else t.cuda() for n, t in make(3, 4, 2, 2, 128, 90, 20, 9, sinks, prefix_rows=100).items()}
    n = torch.tensor([20, 3, 11], dtype=torch.int32, device="cuda")
    x = (a["q"], a["kp"], a["vp"], a["ko"], a["vo"], n)
    for kw in (dict(), dict(prefix_len=90), dict(prefix_len=0)):
        got = [swa.forward_shared(*x, w, 0.1, sinks=a["sinks"], **kw, **s)
               for w, s in ((17, dict()), (17, dict(stream=torch.cuda.Stream())), (np.int64(17), dict()))]
        torch.cuda.synchronize()
        for o, lse in got[1:]:
            assert torch.equal(got[0][0], o) and torch.equal(got[0][1], lse)


@pytest.mark.gpu
def test_captured_step_follows_the_lengths():
    """Append and attend, captured once: every replay takes the lengths and tokens of its moment."""
    import sliding_window_attention_gb300 as swa

    B, Hq, Hkv, D, P, rows, steps = 5, 8, 2, 128, 300, 140, 6
    g = torch.Generator().manual_seed(4)
    a = make(B, Hq, Hkv, 1, D, P, rows, 6)
    d = {n: None if t is None else t.cuda() for n, t in a.items()}
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
    lens = torch.tensor([1, 126, 0, 128, 50], dtype=torch.int32, device="cuda")
    qkv = torch.empty((B, 1, Hq + 2 * Hkv, D), dtype=BF, device="cuda")
    q, k, v = qkv.split((Hq, Hkv, Hkv), 2)
    tokens = torch.randn((steps,) + tuple(qkv.shape), generator=g).to(BF).cuda()

    def step(kc, vc, n):
        qr = swa.qk_rope_append(q, k, v, w, w, f, kc, vc, n, 1e-6, pos0=P)
        return qr, swa.forward_shared(qr, d["kp"], d["vp"], kc, vc, n, 0, D ** -0.5)

    s = torch.cuda.Stream()
    kc, vc = d["ko"].clone(), d["vo"].clone()
    qkv.copy_(tokens[0])
    with torch.cuda.stream(s):
        step(kc.clone(), vc.clone(), lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    n = lens.clone()
    with torch.cuda.graph(graph):
        qr, out = step(kc, vc, n)
    kc.copy_(d["ko"])
    vc.copy_(d["vo"])
    kc2, vc2, n2 = d["ko"].clone(), d["vo"].clone(), lens.clone()
    for i in range(steps):
        qkv.copy_(tokens[i])
        n += 1
        graph.replay()
        n2 += 1
        _, ref = step(kc2, vc2, n2)
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]) and torch.equal(kc, kc2)
        x = dict(a, q=qr.cpu(), ko=kc.cpu(), vo=vc.cpu())
        check(out, reference(x, n.tolist(), P, 0, D ** -0.5))


# --------------------------------------------------------------------------- refusals (no GPU)


def test_c_abi_refuses_bad_arguments():
    import sliding_window_attention_gb300 as swa
    from sliding_window_attention_gb300 import build

    build.build()
    lib = swa.load()
    ok = dict(q=0x1000, kp=0x2000, vp=0x3000, ko=0x4000, vo=0x5000, n=0x6000, sinks=None, o=0x7000, lse=0x8000, B=2,
              Hq=4, Hkv=2, Lq=1, P=10, pr=12, rows=8, D=64, W=0, scale=0.1, ws=0x10000, wsb=1 << 30, stream=None)

    def fwd(**kw):
        return lib.swa_attn_fwd_shared(*{**ok, **kw}.values())

    for name in ("q", "kp", "vp", "ko", "vo", "n", "o", "lse"):
        assert fwd(**{name: None}) == -1, name
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Lq=0)):
        assert fwd(**kw) == -2, kw
    assert fwd(Hkv=3) == -3 and fwd(D=96) == -4 and fwd(W=-1) == -5 and fwd(scale=float("nan")) == -6
    for kw in (dict(P=-1), dict(P=13), dict(rows=0)):
        assert fwd(**kw) == -18, kw
    assert fwd(rows=2 ** 31 - 1, pr=2 ** 31 - 1) == -10 and fwd(B=60000, rows=2 ** 30) == -10
    for name in ("q", "kp", "vp", "ko", "vo", "o"):
        assert fwd(**{name: 0x1008}) == -7, name
    assert fwd(n=0x6002) == -7 and fwd(sinks=0x6001) == -7 and fwd(lse=0x8002) == -7 and fwd(ws=0x10080) == -7
    need = lib.swa_attn_fwd_workspace_bytes_shared(2, 4, 2, 1, 10, 8, 64, 0)
    assert need > 0 and need % 256 == 0 and fwd(wsb=need - 1) == -8 and fwd(ws=None) == -8
    assert lib.swa_attn_fwd_workspace_bytes_shared(2, 4, 2, 1, -1, 8, 64, 0) == 0
    assert lib.swa_attn_fwd_workspace_bytes_shared(2, 4, 3, 1, 10, 8, 64, 0) == 0
    # partials grow with the requests' rows, not with the caches' lengths
    assert lib.swa_attn_fwd_workspace_bytes_shared(64, 32, 4, 1, 16384, 1024, 512, 0) == \
        lib.swa_attn_fwd_workspace_bytes_shared(64, 32, 4, 1, 100, 10, 512, 0) < 128 << 20


def test_binding_refuses_host_tensors():
    import sliding_window_attention_gb300 as swa

    a = make(2, 4, 2, 1, 64, 10, 8, 1)
    n = torch.tensor([1, 2], dtype=torch.int32)
    lse = torch.empty(2, 4, 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        swa.swa_attn_fwd_shared(a["q"], a["kp"], a["vp"], a["ko"], a["vo"], n, None, a["q"].clone(), lse, 0, 0.1)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    import sliding_window_attention_gb300 as swa

    a = {n: None if t is None else t.cuda() for n, t in make(2, 4, 2, 1, 64, 10, 8, 1).items()}
    ok = dict(q=a["q"], kp=a["kp"], vp=a["vp"], ko=a["ko"], vo=a["vo"],
              n=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    for bad in (dict(q=a["q"].float()), dict(kp=a["kp"].transpose(0, 1)), dict(vp=a["vp"][:, :9]), dict(ko=a["ko"][:1]),
                dict(vo=a["vo"].cpu()), dict(n=ok["n"].long()), dict(n=ok["n"][:1]), dict(kp=a["kp"][:1])):
        x = {**ok, **bad}
        with pytest.raises(ValueError):
            swa.forward_shared(x["q"], x["kp"], x["vp"], x["ko"], x["vo"], x["n"], 0, 0.1)
    with pytest.raises(ValueError):
        swa.forward_shared(*ok.values(), 0, 0.1, sinks=torch.zeros(2, device="cuda"))
    with pytest.raises(swa.SwaError):
        swa.forward_shared(*ok.values(), 0, 0.1, prefix_len=11)
    for kw in (dict(prefix_len=2 ** 32), dict(window=-2 ** 40)):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            swa.forward_shared(*ok.values(), **{**dict(window=0, scale=0.1), **kw})


def test_a_workspace_has_its_bytes_on_the_device():
    """Host memory, or a tensor whose elements share bytes, has not what its size says."""
    from sliding_window_attention_gb300 import _native

    assert _native._scratch_bytes(None, 0) == 0
    for ws in (torch.empty(4096, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8).expand(1 << 30)):
        with pytest.raises(ValueError, match="workspace"):
            _native._scratch_bytes(ws, 0)
    assert _native._scratch_bytes(torch.empty(16, dtype=torch.float32), -1) == 64  # (-1: the host's index)
    with pytest.raises(ValueError, match="workspace"):
        _native._scratch_bytes(torch.empty(1, dtype=torch.uint8).expand(1 << 30), -1)


@pytest.mark.gpu
def test_binding_refuses_such_workspaces():
    import sliding_window_attention_gb300 as swa

    a = {n: None if t is None else t.cuda() for n, t in make(2, 4, 2, 1, 64, 10, 8, 1).items()}
    n = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(a["q"]), torch.empty((2, 4, 1), device="cuda")
    need = swa.fwd_workspace_bytes_shared(2, 4, 2, 1, 10, 8, 64, 0)
    x = torch.zeros((1, 3, 2, 64), dtype=BF, device="cuda")
    dy, dw = torch.zeros((1, 2, 3, 64), device="cuda"), torch.ones(64, device="cuda")
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(need)):
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_attn_fwd_shared(a["q"], a["kp"], a["vp"], a["ko"], a["vo"], n, None, o, lse, 0, 0.1, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_attn_qk_rope_bwd(x, None, dw, None, None, dy, None, None, x.clone(), None, None, dw.clone(), None,
                                     1e-6, workspace=ws)


@pytest.mark.gpu
def test_no_prefix_at_all():
    """None for the prefix (a NULL of the C call) is a prefix of no rows, on either marshalling path; one of k and v
    alone is refused, and so is a length of a prefix that is not there."""
    import numpy as np

    import sliding_window_attention_gb300 as swa

    a = {n: None if t is None else t.cuda() for n, t in make(3, 4, 2, 1, 128, 0, 40, 2).items()}
    n = torch.tensor([40, 0, 7], dtype=torch.int32, device="cuda")
    rest = (a["ko"], a["vo"], n)
    want = swa.forward_shared(a["q"], a["kp"], a["vp"], *rest, 0, 0.1)
    check(want, reference(make(3, 4, 2, 1, 128, 0, 40, 2), [40, 0, 7], 0, 0, 0.1))
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(swa.fwd_workspace_bytes_shared(3, 4, 2, 1, 0, 40, 128, 0), dtype=torch.uint8, device="cuda")
    swa.swa_attn_fwd_shared(a["q"], None, None, *rest, None, o, lse, 0, 0.1, workspace=ws)
    for got in ((o, lse), *(swa.forward_shared(a["q"], None, None, *rest, w, 0.1) for w in (0, np.int64(0)))):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for w in (0, np.int64(0)):
        for prefix in ((a["kp"], None), (None, a["vp"])):
            with pytest.raises(ValueError, match="together"):
                swa.forward_shared(a["q"], *prefix, *rest, w, 0.1)
        with pytest.raises(swa.SwaError):
            swa.forward_shared(a["q"], None, None, *rest, w, 0.1, prefix_len=1)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,P,rows", [(6, 8, 4, 1, 128, 900, 64), (40, 8, 2, 1, 128, 2000, 100),
                                                  (16, 16, 2, 4, 64, 700, 200), (12, 32, 4, 1, 512, 600, 150)])
def test_adjacent_calls_take_turns_in_one_workspace(B, Hq, Hkv, Lq, D, P, rows):
    """Calls on two inputs in turn, captured so that nothing lies between them on the stream and no host time keeps
    them apart, with one workspace: a call that wrote partials or the split before the merge of the one before had
    read its own would change that one's result.  Against calls that are waited for."""
    import sliding_window_attention_gb300 as swa

    calls = 12
    x = []
    for i in range(2):
        a = {n: None if t is None else t.cuda() for n, t in make(B, Hq, Hkv, Lq, D, P, rows, 50 + i).items()}
        n = torch.tensor([(29 * b + 31 * i) % rows + 1 for b in range(B)], dtype=torch.int32, device="cuda")
        x.append((a["q"], a["kp"], a["vp"], a["ko"], a["vo"], n, None))
    ws = torch.empty(swa.fwd_workspace_bytes_shared(B, Hq, Hkv, Lq, P, rows, D, 0), dtype=torch.uint8, device="cuda")
    outs = [(torch.full_like(x[0][0], math.nan), torch.full((B, Hq, Lq), math.nan, device="cuda")) for _ in range(calls)]

    def run_all(wait):
        for i in range(calls):
            swa.swa_attn_fwd_shared(*x[i % 2], *outs[i], 0, 0.1, workspace=ws)
            if wait:
                torch.cuda.synchronize()

    run_all(True)
    want = [(o.clone(), lse.clone()) for o, lse in outs[:2]]
    assert not torch.equal(want[0][0], want[1][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(False)
    for _ in range(5):
        for o, lse in outs:
            o.fill_(math.nan)
            lse.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, lse) in enumerate(outs):
            assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1]), i


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,D,P,rows", [(6, 8, 2, 128, 300, 90), (30, 4, 2, 64, 1000, 200), (8, 32, 4, 512, 400, 140)])
def test_layers_back_to_back(B, Hq, Hkv, D, P, rows):
    """Append, attention, append, attention, ... with nothing between them, captured: each append writes the rows that
    the attention before it has read last, as a model's layers do that share a cache, and takes its queries' buffer
    again.  Against the same steps waited for one by one."""
    import sliding_window_attention_gb300 as swa

    steps = 12
    g = torch.Generator(device="cuda").manual_seed(14)
    x = torch.randn((steps, B, 1, Hq + 2 * Hkv, D), device="cuda", generator=g).to(BF)
    kp, vp = (torch.randn((Hkv, P, D), device="cuda", generator=g).to(BF) for _ in range(2))
    kc, vc = (torch.randn((B, Hkv, rows, D), device="cuda", generator=g).to(BF) for _ in range(2))
    n = torch.tensor([(37 * b) % rows + 1 for b in range(B)], dtype=torch.int32, device="cuda")
    f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
    q = torch.empty((B, Hq, 1, D), dtype=BF, device="cuda")
    ws = torch.empty(swa.fwd_workspace_bytes_shared(B, Hq, Hkv, 1, P, rows, D, 0), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")) for _ in range(steps)]

    def run_all(wait):
        for i in range(steps):
            xq, xk, xv = x[i].split((Hq, Hkv, Hkv), 2)
            swa.swa_attn_qk_rope_fwd(xq, xk, xv, None, None, f, q, kc, vc, 1e-6, None, n, P)
            if wait:
                torch.cuda.synchronize()
            swa.swa_attn_fwd_shared(q, kp, vp, kc, vc, n, None, *outs[i], 0, 0.1, workspace=ws)
            if wait:
                torch.cuda.synchronize()

    run_all(True)
    want = [(o.clone(), lse.clone()) for o, lse in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(False)
    for _ in range(5):
        for o, lse in outs:
            o.fill_(math.nan)
            lse.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, lse) in enumerate(outs):
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]), i
