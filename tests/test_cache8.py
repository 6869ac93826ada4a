"""A cache held in 8 bits (swa_attn_cache8_append, swa_attn_cache8_read,
swa_attn_fwd_cache8) against the definitions in 64 bits.

Appends and reads are exact: codes and scales are compared bit for bit with a
quantiser written out here, read-back values with code * scale rounded once.

Tolerances of the attention.  A weight (p times its value's scale) is rounded to
fp16 (half a step, 2^-11 of each term) and written as three e5m2 numbers, which
hold it exactly but for what lies below 2^-17 when the row's largest weight is
2^10 or more: 2^-27 of the largest weight for each key.  o is rounded once more
(2^-8 of the value).  Scores carry 2^-18 * scale * sum |q k| (fp32 accumulation
over D <= 512 products of exact factors) and, from q's two parts, 2^-22 of q's
largest element times scale * sum |k|; that shifts a term by as much, and the
sums by 2^-14 at most.  So with s twice those two (numerator and normaliser)
  |o - ref| <= (2^-11 + s + 2^-14) sum p |v| + 2^-27 max(p vs) sum |cv| + 2^-8 |ref|
  |lse - ref| <= s + 2^-18 (1 + |ref|).
"""
import math

import pytest
import torch

BF = torch.bfloat16
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the quantiser, element by element


def two_to(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    s = 2.0 ** -64
    while amax > 448 * s:
        s *= 2
    return s


def e4m3(y):
    """fp64 values to the nearest e4m3 number, ties to even, 448 at most."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def ref_append(x, codes, scales, lens, block):
    """x [B, H, L, D] into fp64 codes [B, H, rows, D] and scales [B, H, NB], in place."""
    B, H, L, _ = x.shape
    rows = codes.shape[2]
    for b in range(B):
        n = L if lens is None else int(lens[b])
        first = max(0, n - L)
        for h in range(H):
            for j in range(first // block, -(-min(n, rows) // block)):
                lo, hi = j * block, min((j + 1) * block, n, rows)
                a = max(lo, first)
                if hi <= a:
                    continue
                new = x[b, h, a - (n - L):hi - (n - L)].double()
                top, was = float(new.abs().max()), float(scales[b, h, j])
                now = was if a > lo and top <= 448 * was else two_to(top)
                if a > lo:
                    codes[b, h, lo:a] = e4m3(codes[b, h, lo:a] * (was / now))
                codes[b, h, a:hi] = e4m3(new / now)
                scales[b, h, j] = now


def filled(B, H, rows, D, block, seed, spread=1.0):
    """A cache of random values: (codes F8, scales fp32) and what was quantised."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, rows, D, generator=g) * torch.exp(spread * torch.randn(B, H, rows, 1, generator=g))
    codes = torch.zeros(B, H, rows, D, dtype=torch.float64)
    scales = torch.zeros(B, H, -(-rows // block), dtype=torch.float64)
    ref_append(x.to(BF), codes, scales, None, block)
    return codes.float().to(F8), scales.float()


def status_ok():
    import sliding_window_attention_gb300 as swa

    torch.cuda.synchronize()
    assert swa.swa_attn_get_status() == 0


# ---------------------------------------------------------------- append


def check_append(k, v, cache, lens, block):
    import sliding_window_attention_gb300 as swa

    k8, v8, ks, vs = cache
    want = []
    for x, c, s in ((k, k8, ks), (v, v8, vs)):
        codes, scales = c.double(), s.double()
        ref_append(x, codes, scales, lens, block)
        want.append((codes, scales))
    d = [t.cuda() for t in cache]
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    swa.cache8_append(k.cuda(), v.cuda(), *d, n, block)
    status_ok()
    for got_c, got_s, (c, s) in ((d[0], d[2], want[0]), (d[1], d[3], want[1])):
        assert torch.equal(got_s.cpu().double(), s)
        assert torch.equal(got_c.cpu().double(), c)
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,L,D,rows,block,lens", [
    (3, 2, 1, 64, 50, 16, [1, 17, 50]),             # first of a block, second block's first, the last row
    (4, 1, 1, 512, 130, 128, [1, 2, 128, 130]),
    (3, 2, 3, 128, 70, 32, [3, 33, 35]),            # across a block's border
    (2, 3, 7, 256, 100, 16, [20, 100]),
    (2, 2, 33, 64, 64, 64, [33, 64]),
    (1, 2, 300, 128, 301, 64, [301]),               # a long ragged one behind older tokens
    (1, 1, 1000, 512, 1001, 128, [1000]),
    (2, 1, 200, 256, 203, 128, [201, 203]),
    (2, 2, 100, 64, 120, 16, None),                 # tokens at rows 0 ..
])
def test_append_is_the_quantiser(B, H, L, D, rows, block, lens):
    g = torch.Generator().manual_seed(L + D)
    k = torch.randn(B, H, L, D, generator=g).to(BF)
    v = (4 * torch.randn(B, H, L, D, generator=g)).to(BF)
    kc, vc = filled(B, H, rows, D, block, 1), filled(B, H, rows, D, block, 2)
    check_append(k, v, (kc[0], vc[0], kc[1], vc[1]), lens, block)


@pytest.mark.gpu
def test_append_outside_the_cache_and_empty_places():
    """Rows outside [0, rows) are not written; a length of 0 or below writes nothing; rows behind stay."""
    k = torch.randn(6, 2, 5, 64).to(BF)
    kc, vc = filled(6, 2, 40, 64, 16, 3), filled(6, 2, 40, 64, 16, 4)
    check_append(k, (2 * k.float()).to(BF), (kc[0], vc[0], kc[1], vc[1]), [-1, 0, 3, 42, 45, -2 ** 31], 16)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [16, 128])
def test_append_scales(block):
    """Borders of the scale's powers of two, zeros, tiny and huge tokens, step after step in one block."""
    steps = [0.0, 448.0, 449.0, 2.0 ** -140, 448.0 * 2 ** -20, 3.0e38, 1.0, 0.4375, 2.0 ** 100, 450.0]
    kc, vc = filled(1, 1, 16, 64, block, 5), filled(1, 1, 16, 64, block, 6)
    cache = [kc[0], vc[0], kc[1], vc[1]]
    for i, x in enumerate(steps):
        k = torch.full((1, 1, 1, 64), x).to(BF)
        k[..., 1::2] *= -0.37
        d = check_append(k, k.flip(3), cache, [i + 1], block)
        cache = [t.cpu() for t in d]
    # a block that starts again takes a new scale whatever it held
    check_append(torch.full((1, 1, 1, 64), 0.1).to(BF), torch.full((1, 1, 1, 64), 0.2).to(BF), cache, [1], block)


@pytest.mark.gpu
def test_append_with_scales_that_are_no_powers_of_two():
    """A cache that another quantiser wrote: codes are x / s for a scale that stays."""
    kc, vc = filled(2, 2, 64, 128, 32, 7), filled(2, 2, 64, 128, 32, 8)
    g = torch.Generator().manual_seed(9)
    ks, vs = kc[1] * 1.2734375, vc[1] * 1.9921875
    k = torch.randn(2, 2, 2, 128, generator=g).to(BF)
    check_append((k.float() * 0.1).to(BF), k, (kc[0], vc[0], ks, vs), [20, 45], 32)


@pytest.mark.gpu
def test_append_strides_and_one_tensor():
    """Slices of a projection's rows, and k alone."""
    import sliding_window_attention_gb300 as swa

    g = torch.Generator().manual_seed(11)
    B, H, L, D, rows = 2, 3, 21, 64, 40
    x = torch.randn(B, L, 2 + 2 * H, D, generator=g).to(BF)
    k, v = x[:, :, 2:2 + H].transpose(1, 2), x[:, :, 2 + H:].transpose(1, 2)
    kc, vc = filled(B, H, rows, D, 32, 12), filled(B, H, rows, D, 32, 13)
    check_append(k, v, (kc[0], vc[0], kc[1], vc[1]), [21, 39], 32)
    dx = x.cuda()
    d = [t.cuda() for t in (kc[0], kc[1])]
    codes, scales = kc[0].double(), kc[1].double()
    ref_append(k, codes, scales, [30, 22], 32)
    swa.swa_attn_cache8_append(dx[:, :, 2:2 + H].transpose(1, 2), None, d[0], None, d[1], None,
                               torch.tensor([30, 22], dtype=torch.int32).cuda(), 32)
    status_ok()
    assert torch.equal(d[0].cpu().double(), codes) and torch.equal(d[1].cpu().double(), scales)


# ---------------------------------------------------------------- read


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,D,rows,block,lens,row0,n", [
    (3, 2, 64, 100, 16, [0, 57, 100], 0, None),
    (2, 1, 512, 33, 128, [33, -5], 0, None),
    (2, 3, 128, 777, 64, [700, 1000], 513, 264),
    (1, 2, 256, 300, 32, None, 7, 1),
])
def test_read_is_code_times_scale(B, H, D, rows, block, lens, row0, n):
    import sliding_window_attention_gb300 as swa

    kc, vc = filled(B, H, rows, D, block, 21), filled(B, H, rows, D, block, 22)
    vs = vc[1] * 1.37  # another quantiser's
    length = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    got = swa.cache8_read(kc[0].cuda(), vc[0].cuda(), kc[1].cuda(), vs.cuda(),
                          None if lens is None else length.cuda(), block, row0, n)
    status_ok()
    for g, c, s in ((got[0], kc[0], kc[1]), (got[1], vc[0], vs)):
        per = s.repeat_interleave(block, 2)[:, :, :rows, None]
        want = (c.float() * per).to(BF)  # one fp32 product of 4 and 24 bits, rounded, then bf16: not always the nearest
        if lens is not None:
            want *= (torch.arange(rows) < length[:, None])[:, None, :, None]
        assert torch.equal(g.cpu(), want[:, :, row0:rows if n is None else row0 + n])


# ---------------------------------------------------------------- attention


def attention(q, kc, vc, ks, vs, sinks, lens, window, scale, block):
    """(o, tolerance of o, lse, tolerance of lse) in fp64; NaN for empty places."""
    B, Hq, Lq, D = q.shape
    _, Hkv, rows, _ = kc.shape
    G = Hq // Hkv
    o, tol = torch.full((2, B, Hq, Lq, D), math.nan, dtype=torch.float64)
    lse, ltol = torch.full((2, B, Hq, Lq), math.nan, dtype=torch.float64)
    for b in range(B):
        n = min(int(lens[b]), rows)
        if n < 0:
            continue
        per = torch.arange(n) // block
        for h in range(Hq):
            x = q[b, h].double()
            ck, cv = kc[b, h // G, :n].double(), vc[b, h // G, :n].double()
            sk, sv = ks[b, h // G].double()[per], vs[b, h // G].double()[per]
            k = ck * sk[:, None]
            y = x @ k.T * scale
            i = n - Lq + torch.arange(Lq)[:, None]
            j = torch.arange(n)[None]
            see = j <= i
            if window:
                see &= i - j < window
            y = y.masked_fill(~see, -math.inf)
            c = float(sinks[h]) if sinks is not None else -math.inf
            m = torch.cat((y, torch.full((Lq, 1), c, dtype=torch.float64)), 1).amax(1, keepdim=True)
            m0 = torch.where(m == -math.inf, 0.0, m)
            e = torch.exp(y - m0)
            z = e.sum(1, keepdim=True) + math.exp(c - 0.0) * torch.exp(-m0) if c > -math.inf else e.sum(1, keepdim=True)
            p = torch.where(z > 0, e / z, 0.0)
            w = p * sv
            s = 2 * abs(scale) * (2.0 ** -18 * (x.abs() @ k.abs().T).masked_fill(~see, 0) +
                                  2.0 ** -22 * x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] * see)
            s = s.amax(1, keepdim=True) if n else torch.zeros(Lq, 1, dtype=torch.float64)
            o[b, h] = w @ cv
            big = w.amax(1, keepdim=True) if n else 0.0
            tol[b, h] = (2.0 ** -11 + s + 2.0 ** -14) * (w @ cv.abs()) + 2.0 ** -27 * big * (see.double() @ cv.abs()) + \
                2.0 ** -8 * o[b, h].abs()
            lse[b, h] = (m0 + torch.log(z))[:, 0]
            ltol[b, h] = s[:, 0] + 2.0 ** -18 * (1 + torch.where(lse[b, h].isfinite(), lse[b, h].abs(), 0.0))
    return o, tol, lse, ltol


def attend(q, kc, vc, sinks, lens, window, scale, block, **kw):
    import sliding_window_attention_gb300 as swa

    n = torch.tensor(lens, dtype=torch.int32).cuda()
    got = swa.forward_cache8(q.cuda(), kc[0].cuda(), vc[0].cuda(), kc[1].cuda(), vc[1].cuda(), n, block, window, scale,
                             sinks=None if sinks is None else sinks.cuda(), **kw)
    status_ok()
    return [t.double().cpu() for t in got]


def check_attention(q, kc, vc, sinks, lens, window, scale, block):
    got_o, got_lse = attend(q, kc, vc, sinks, lens, window, scale, block)
    o, tol, lse, ltol = attention(q, kc[0], vc[0], kc[1], vc[1], sinks, lens, window, scale, block)
    live = torch.tensor(lens) >= 0
    for got, ref, t, name in ((got_o, o, tol, "o"), (got_lse, lse, ltol, "lse")):
        got, ref, t = got[live], ref[live], t[live]
        inf = ref == -math.inf
        assert torch.equal(got == -math.inf, inf), name
        d = (got - ref).masked_fill(inf, 0.0).abs()
        assert bool((d <= t.masked_fill(inf, 1.0)).all()), \
            f"{name}: {float((d / t.clamp(min=1e-300)).masked_fill(inf, 0).max()):.2f} of its tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("B,Hq,Hkv,Lq,rows,window,sinks,block,lens", [
    (1, 2, 1, 1, 1, 0, False, 16, [1]),                               # one key
    (2, 4, 2, 1, 300, 0, False, 16, [300, 129]),
    (3, 8, 2, 2, 520, 0, True, 64, [1, 2, 513]),                      # a row without a key
    (4, 16, 1, 1, 200, 0, False, 128, [0, 128, -1, 127]),             # an empty cache, an empty place
    (2, 6, 2, 3, 700, 100, False, 32, [700, 99]),                     # a window
    (2, 8, 1, 5, 260, 0, True, 32, [260, 3]),                         # 40 rows: three blocks
    (1, 4, 4, 1, 5001, 333, True, 16, [4999]),
])
def test_attention(D, B, Hq, Hkv, Lq, rows, window, sinks, block, lens):
    g = torch.Generator().manual_seed(D + rows)
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    kc, vc = filled(B, Hkv, rows, D, block, 31, 0.3), filled(B, Hkv, rows, D, block, 32)
    s = torch.randn(Hq, generator=g) if sinks else None
    check_attention(q, kc, vc, s, lens, window, 1.0 / math.sqrt(D), block)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,rows,window,block,spread", [
    (16, 4, 4, 1, 64, 8192, 0, 64, 1),      # equal lengths: every run in several waves
    (40, 8, 4, 1, 128, 5000, 0, 128, 0),    # ragged ones
    (3, 16, 8, 3, 256, 20000, 0, 16, 0),    # long segments, cut by many runs
    (33, 12, 4, 4, 512, 4000, 2500, 32, 0),  # 12 rows, a window
    (9, 16, 2, 4, 64, 9000, 0, 16, 0),      # 32 rows
    (6, 16, 2, 3, 128, 12000, 3000, 64, 0),  # 24 rows, a window
    (5, 20, 2, 5, 256, 7000, 0, 128, 0),    # 50 rows: a block of 32 and one of 18
])
def test_attention_of_many_tiles(B, Hq, Hkv, Lq, D, rows, window, block, spread):
    """More tiles than five a CTA: runs that CTAs take over, and their merge."""
    g = torch.Generator().manual_seed(rows)
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    x = torch.randint(0, 256, (2, B, Hkv, rows, D), generator=g, dtype=torch.uint8)
    x &= 0xDF  # no NaN, 30 at most
    kc, vc = (t.view(F8) for t in x)
    s = torch.exp2(torch.randint(-6, -2, (2, B, Hkv, -(-rows // block)), generator=g).float())
    lens = [rows] * B if spread else torch.randint(1, rows + 1, (B,), generator=g).tolist()
    some = sorted({0, B // 2, B - 1})  # (the whole batch in 64 bits on the host would take minutes)
    got_o, got_lse = attend(q, (kc, s[0]), (vc, s[1]), None, lens, window, 0.25 / math.sqrt(D), block)
    o, tol, lse, ltol = attention(q[some], x[0][some].view(F8), x[1][some].view(F8), s[0][some], s[1][some], None,
                                  [lens[b] for b in some], window, 0.25 / math.sqrt(D), block)
    assert bool(((got_o[some] - o).abs() <= tol).all()) and bool(((got_lse[some] - lse).abs() <= ltol).all())
    again = attend(q, (kc, s[0]), (vc, s[1]), None, lens, window, 0.25 / math.sqrt(D), block)
    assert torch.equal(again[0], got_o) and torch.equal(again[1], got_lse)
