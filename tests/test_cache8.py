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


# L, D, block: one for each of the append's groups of threads and vectors a thread, in their order, by the min(L, block)
# * D / 8 vectors that a block can get: up to 64, 128, 256, 512, 1,024, 2,048, 4,096 and more
GROUPS = [(1, 512, 64), (4, 256, 64), (7, 256, 16), (70, 64, 64), (100, 256, 32), (300, 128, 128), (200, 256, 64),
          (100, 512, 32), (300, 256, 128), (200, 512, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("L,D,block", GROUPS)
@pytest.mark.parametrize("times", [1.0, 1.2734375, 1.9921875])
@pytest.mark.parametrize("size", [0.01, 1.0, 40.0])
def test_append_behind_older_tokens(L, D, block, times, size):
    """Each group's kernel behind a partial block of older tokens that fits the new ones, or has to grow for them; with
    scales that are powers of two and another quantiser's.  A value that is written again changes by what the header
    says: 2^-10 s of a power of two, and 2^-4 of itself where that is more with other scales."""
    g = torch.Generator().manual_seed(L + D + block)
    B, H = 2, 2
    rows = L + block + 5
    k, v = (size * torch.randn(B, H, L, D, generator=g)).to(BF), (3 * size * torch.randn(B, H, L, D, generator=g)).to(BF)
    kc, vc = filled(B, H, rows, D, block, 71, 0.3), filled(B, H, rows, D, block, 72, 0.3)
    ks, vs = kc[1] * times, vc[1] * times
    lens = [L + 3, rows - 1]
    d = check_append(k, v, (kc[0], vc[0], ks, vs), lens, block)
    for was_c, was_s, now_c, now_s in ((kc[0], ks, d[0], d[2]), (vc[0], vs, d[1], d[3])):
        for b, n in enumerate(lens):
            j = torch.arange(n - L) // block
            was = was_c[b, :, :n - L].double() * was_s[b][:, j, None].double()
            s = now_s.cpu()[b][:, j, None].double()
            change = (now_c.cpu()[b, :, :n - L].double() * s - was).abs()
            most = s * 2.0 ** -10 if times == 1.0 else torch.maximum(s * 2.0 ** -10, was.abs() * 2.0 ** -4)
            assert bool((change <= most).all())


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


ROWS_MAIN = """
#include <cstdio>
#include "cache8_rows.h"
int main() {
  int n, L, rows, lb, j;
  while (std::scanf("%d %d %d %d %d", &n, &L, &rows, &lb, &j) == 5) {
    const swa::Cache8Rows r = swa::cache8_rows(n, L, rows, lb, j);
    std::printf("%d %d %d %d %d %d\\n", (int)r.any, r.blk, r.lo, r.a, r.hi, r.token);
  }
}
"""


def test_rows_that_an_append_writes(tmp_path):
    """The kernel's own arithmetic, compiled for the host: lengths over the whole range of an int, its ends among them."""
    import random
    import subprocess

    from sliding_window_attention_gb300 import build

    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(ROWS_MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", build.CSRC,
                    str(src), "-o", str(exe)], check=True)
    rng = random.Random(1)
    top = 2 ** 31 - 1
    cases = [(top, 2, 64, 4, 1), (top, 2, 64, 4, 0), (top, 40, 2_000_000_000, 4, 2), (-top - 1, 5, 64, 4, 0)]
    for _ in range(4000):
        lb, L = rng.choice((4, 5, 6, 7)), rng.choice((1, 2, 7, 64, 300, 5000, 2_000_000_000))
        rows = rng.choice((1, 50, 64, 1000, 2_000_000_000))
        n = rng.choice((rng.randint(-5, 400), rng.randint(rows - 200, rows + 400), rng.randint(top - 300, top),
                        rng.randint(-top - 1, top), -top - 1 + rng.randint(0, 300)))
        meets = min((L + 2 ** lb - 2) // 2 ** lb + 1, -(-rows // 2 ** lb))
        cases.append((max(min(n, top), -top - 1), L, rows, lb, rng.randrange(meets)))
    out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, check=True,
                         capture_output=True).stdout.splitlines()
    assert len(out) == len(cases)
    for c, line in zip(cases, out):
        n, L, rows, lb, j = c
        row0 = max(n - L, 0)
        blk = (row0 >> lb) + j
        a, hi = max(blk << lb, row0), min(n, rows, (blk + 1) << lb)
        want = [1, blk, blk << lb, a, hi, a - (n - L)] if a < hi else [0] * 6
        assert [int(x) for x in line.split()] == want, c


@pytest.mark.gpu
def test_append_at_the_largest_lengths():
    """Lengths up to 2^31 - 1 lie behind the cache: nothing is written, by calls that meet several blocks too."""
    top = 2 ** 31 - 1
    for L, D, block in ((5, 64, 16), (40, 128, 16), (300, 64, 128)):
        k = torch.randn(6, 2, L, D).to(BF)
        kc, vc = filled(6, 2, 64, D, block, 14), filled(6, 2, 64, D, block, 15)
        check_append(k, (2 * k.float()).to(BF), (kc[0], vc[0], kc[1], vc[1]), [top, top - 1, top - 15, 64 + L, -top - 1, 63],
                     block)


@pytest.mark.gpu
def test_what_a_call_does_not_use_is_not_checked():
    """With k or v alone the other's strides, codes and scales are anything (here: the middle of a tensor, oddly placed)."""
    import sliding_window_attention_gb300 as swa

    lib = swa.load()
    B, H, L, D, rows, block = 2, 2, 3, 64, 40, 16
    g = torch.Generator().manual_seed(17)
    x = torch.randn(B, H, L, D, generator=g).to(BF)
    n = torch.tensor([3, 20], dtype=torch.int32)
    c0, s0 = filled(B, H, rows, D, block, 18)
    want_c, want_s = c0.double(), s0.double()
    ref_append(x, want_c, want_s, n, block)
    dx, dn, rest = x.cuda(), n.cuda(), torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    strides, odd = x.stride()[:3], rest.data_ptr() + 2049
    for first in (True, False):
        for other in (0, odd):
            c, s = c0.cuda(), s0.cuda()
            out = torch.empty(B, H, rows, D, dtype=BF, device="cuda")

            def pair(mine, none=other):  # (k's, v's)
                return (mine, none) if first else (none, mine)

            sk, sv = pair(strides, (-1, 3, 5))
            assert lib.swa_attn_cache8_append(*pair(dx.data_ptr(), None), *sk, *sv, dn.data_ptr(), *pair(c.data_ptr()),
                                              *pair(s.data_ptr()), B, H, L, D, rows, block, None) == 0
            assert lib.swa_attn_cache8_read(*pair(c.data_ptr()), *pair(s.data_ptr()), None, *pair(out.data_ptr(), None),
                                            B, H, D, rows, block, 0, rows, None) == 0
            status_ok()
            assert torch.equal(c.cpu().double(), want_c) and torch.equal(s.cpu().double(), want_s)
            per = want_s.float().repeat_interleave(block, 2)[:, :, :rows, None]
            assert torch.equal(out.cpu(), (want_c.float() * per).to(BF))
    assert bool((rest == 7).all())


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


def rows_of_a_block(B, Hq, Hkv, Lq, rows, D, block, window):
    """Query rows of a block, by the partials that the workspace holds (D + 2 floats a row, two slots for each of 304 CTAs)."""
    import sliding_window_attention_gb300 as swa

    return swa.fwd_workspace_bytes_cache8(B, Hq, Hkv, Lq, rows, D, block, window) // (608 * 4 * (D + 2))


# B, Hq, Hkv, Lq, D, rows, window, sinks, block: more than 16 rows a kv head at D <= 128, over caches of more than 1,824
# tiles, which are what blocks of 32 rows are taken for
BLOCKS_OF_32 = [
    (40, 16, 2, 4, 64, 4000, 3500, True, 16),     # a window and sinks
    (40, 16, 2, 4, 128, 4000, 3500, True, 64),
    (24, 20, 2, 4, 128, 3000, 0, True, 128),      # 40 rows: a block of 32 and one of 8
    (24, 20, 2, 5, 64, 3000, 0, False, 16),       # 50: one of 32 and one of 18
    (100, 16, 2, 3, 128, 2000, 1500, True, 32),   # 24 of 32
    (1900, 17, 1, 1, 64, 300, 100, True, 64),     # 17; a window within a tile or two: many visits of one tile
    (256, 32, 4, 4, 64, 400, 0, False, 32),       # many short requests
    (256, 32, 4, 4, 128, 400, 130, True, 128),
    (20, 32, 1, 4, 128, 4000, 0, True, 64),       # 128 rows: four whole blocks
    (30, 25, 1, 4, 64, 8000, 2000, False, 128),   # 100: three and one of 4, over a long window
]


def test_which_blocks_are_tested(lib):
    """The cases above are of blocks of 32 rows, their likes with fewer tiles, few rows or longer heads of 16 or 8."""
    for B, Hq, Hkv, Lq, D, rows, window, _, block in BLOCKS_OF_32:
        assert rows_of_a_block(B, Hq, Hkv, Lq, rows, D, block, window) == (32 if Hq // Hkv * Lq > 32 else Hq // Hkv * Lq)
        units = B * Hkv * -(-Hq // Hkv * Lq // 32) * -(-min(rows, window + Lq - 1 if window else rows) // 128)
        assert units >= 1.02 * 6 * 304
    assert rows_of_a_block(40, 20, 2, 4, 4000, 256, 16, 0) == 16 and rows_of_a_block(40, 20, 2, 4, 4000, 512, 16, 0) == 16
    assert rows_of_a_block(2, 20, 2, 4, 4000, 64, 16, 0) == 16 and rows_of_a_block(40, 8, 2, 4, 4000, 64, 16, 0) == 16
    assert rows_of_a_block(40, 8, 2, 2, 4000, 64, 16, 0) == 8


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,rows,window,sinks,block", BLOCKS_OF_32)
@pytest.mark.parametrize("equal", [False, True])
def test_attention_in_blocks_of_32_rows(B, Hq, Hkv, Lq, D, rows, window, sinks, block, equal):
    g = torch.Generator().manual_seed(rows + D + equal)
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    x = torch.randint(0, 256, (2, B, Hkv, rows, D), generator=g, dtype=torch.uint8)
    x &= 0xDF  # no NaN, 30 at most
    kc, vc = (t.view(F8) for t in x)
    sc = torch.exp2(torch.randint(-6, -2, (2, B, Hkv, -(-rows // block)), generator=g).float())
    s = torch.randn(Hq, generator=g) if sinks else None
    lens = [rows] * B if equal else torch.randint(0, rows + 1, (B,), generator=g).tolist()
    if not equal:
        lens[1:5] = [0, -1, 1, 2]  # no key, an empty place, rows without a key among others
    some = [0, 1, 3, 4, B // 2, B - 1]
    got_o, got_lse = attend(q, (kc, sc[0]), (vc, sc[1]), s, lens, window, 0.25 / math.sqrt(D), block)
    o, tol, lse, ltol = attention(q[some], x[0][some].view(F8), x[1][some].view(F8), sc[0][some], sc[1][some], s,
                                  [lens[b] for b in some], window, 0.25 / math.sqrt(D), block)
    inf = lse == -math.inf
    assert torch.equal(got_lse[some] == -math.inf, inf)
    assert bool(((got_o[some] - o).abs() <= tol).all())
    assert bool(((got_lse[some] - lse).masked_fill(inf, 0).abs() <= ltol).all())
    again = attend(q, (kc, sc[0]), (vc, sc[1]), s, lens, window, 0.25 / math.sqrt(D), block)
    live = torch.tensor(lens) >= 0
    assert torch.equal(again[0][live], got_o[live]) and torch.equal(again[1][live], got_lse[live])


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq,rising", [(64, 2, True), (128, 8, True), (256, 20, True), (512, 3, False)])
def test_references_that_move(D, Hq, rising):
    """Scores that rise (or fall) by some 200 along the cache: references move often, sums and outputs with them."""
    g = torch.Generator().manual_seed(D)
    rows, block = 1500, 16
    q = torch.randn(2, Hq, 1, D, generator=g).to(BF)
    q[..., 0] = 4.0
    k = 0.2 * torch.randn(2, 1, rows, D, generator=g)
    ramp = torch.linspace(-25, 25, rows)
    k[..., 0] = ramp if rising else -ramp
    codes = torch.zeros(2, 1, rows, D, dtype=torch.float64)
    scales = torch.zeros(2, 1, -(-rows // block), dtype=torch.float64)
    ref_append(k.to(BF), codes, scales, None, block)
    vc = filled(2, 1, rows, D, block, 41)
    check_attention(q, (codes.float().to(F8), scales.float()), vc, None, [rows, 1111], 0, 1.0, block)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_references_that_move_apart(D):
    """28 rows of one block, of which some rise and some fall along a long cache."""
    g = torch.Generator().manual_seed(D + 5)
    B, Hq, Hkv, Lq, rows, block = 8, 16, 4, 7, 7300, 64
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    q[..., 0] = torch.tensor([4.0, -4.0, 0.5, 3.0, -1.0, 0.0, 2.0])[(torch.arange(Hq)[:, None] + torch.arange(Lq)) % 7]
    k = 0.2 * torch.randn(B, Hkv, rows, D, generator=g)
    k[..., 0] = torch.linspace(-25, 25, rows)
    codes = torch.zeros(B, Hkv, rows, D, dtype=torch.float64)
    scales = torch.zeros(B, Hkv, -(-rows // block), dtype=torch.float64)
    ref_append(k.to(BF), codes, scales, None, block)
    kc, vc = (codes.float().to(F8), scales.float()), filled(B, Hkv, rows, D, block, 46)
    lens = torch.randint(rows // 2, rows + 1, (B,), generator=g).tolist()
    some = [0, B - 1]
    got_o, got_lse = attend(q, kc, vc, None, lens, 0, 1.0, block)
    o, tol, lse, ltol = attention(q[some], *(t.view(torch.uint8)[some].view(F8) for t in (kc[0], vc[0])), kc[1][some],
                                  vc[1][some], None, [lens[b] for b in some], 0, 1.0, block)
    assert bool(((got_o[some] - o).abs() <= tol).all()) and bool(((got_lse[some] - lse).abs() <= ltol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,rows,window,sinks,block,lens", [
    (1, 8, 1, 700, 64, 900, 0, True, 16, [800]),           # 350 blocks: more than CTAs
    (1, 8, 1, 400, 256, 700, 200, False, 64, [650]),       # 200: one CTA each
    (2, 4, 1, 1000, 128, 1500, 0, False, 128, [1500, 990]),  # 125 of 32 rows; rows without a key
])
def test_attention_of_many_row_blocks(B, Hq, Hkv, Lq, D, rows, window, sinks, block, lens):
    g = torch.Generator().manual_seed(rows + 1)
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    kc, vc = filled(B, Hkv, rows, D, block, 47, 0.3), filled(B, Hkv, rows, D, block, 48)
    s = torch.randn(Hq, generator=g) if sinks else None
    check_attention(q, kc, vc, s, lens, window, 1.0 / math.sqrt(D), block)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 512])
def test_scales_far_apart(D):
    """Blocks of values and keys whose scales lie 2^60 apart, zeros among them, and the least scale."""
    g = torch.Generator().manual_seed(D + 1)
    B, Hkv, rows, block = 2, 2, 400, 32
    nb = -(-rows // block)
    q = torch.randn(B, 4, 2, D, generator=g).to(BF)
    kc, vc = filled(B, Hkv, rows, D, block, 42, 0.2), filled(B, Hkv, rows, D, block, 43, 0.2)
    vs = vc[1] * torch.exp2(torch.randint(-30, 31, (B, Hkv, nb), generator=g).float())
    vs[0, 0, :] = 2.0 ** -64
    ks = kc[1] * torch.exp2(torch.randint(-8, 1, (B, Hkv, nb), generator=g).float())
    codes = vc[0].float()
    codes[1, 1, 64:128] = 0
    check_attention(q, (kc[0], ks), (codes.to(F8), vs), None, [rows, 333], 0, 1.0 / math.sqrt(D), block)


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq,Lq,sinks", [(64, 8, 1, False), (128, 8, 4, True), (256, 2, 5, False), (512, 4, 1, True)])
@pytest.mark.parametrize("apart", [20, 100])
def test_scales_as_far_apart_as_the_header_allows(D, Hq, Lq, sinks, apart):
    """Values' scales 2^100 apart, the largest ones over codes of 0 (an outlier's block): lse keeps its
    precision, and o is off by 2^-27 of the largest weight for each key, which at 2^20 leaves the small scales' values 6 bits."""
    g = torch.Generator().manual_seed(D + apart)
    B, Hkv, rows, block = 2, 2, 700, 32
    nb = -(-rows // block)
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    kc, vc = filled(B, Hkv, rows, D, block, 65, 0.2), filled(B, Hkv, rows, D, block, 66, 0.2)
    low = torch.rand(B, Hkv, nb, generator=g) < 0.5
    vs = torch.where(low, 2.0 ** -(apart // 2), 2.0 ** (apart - apart // 2))
    codes = vc[0].float() * low.repeat_interleave(block, 2)[:, :, :rows, None]
    s = torch.randn(Hq, generator=g) if sinks else None
    check_attention(q, kc, (codes.to(F8), vs), s, [rows, 333], 0, 1.0 / math.sqrt(D), block)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_scales_of_the_softmax(scale):
    g = torch.Generator().manual_seed(7)
    q = torch.randn(2, 4, 1, 64, generator=g).to(BF)
    q[0, 0] = 0
    q[1, 1] *= 2.0 ** 40  # a row far larger than the others
    q[1, 2] *= 2.0 ** -40
    kc, vc = filled(2, 2, 200, 64, 64, 44, 0.2), filled(2, 2, 200, 64, 64, 45, 0.2)
    check_attention(q, kc, vc, None, [200, 77], 0, scale, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("sinks", [False, True])
def test_queries_that_are_not_finite(D, bad, sinks):
    """One such element makes its row's o and lse NaN, whole or cut, unless the row sees no key; the other rows' bits stay."""
    g = torch.Generator().manual_seed(D)
    B, Hq, Hkv, Lq, rows, block = 3, 8, 2, 3, 900, 32
    lens = [900, 2, 130]  # the second request's first row sees no key
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF)
    kc, vc = filled(B, Hkv, rows, D, block, 61, 0.3), filled(B, Hkv, rows, D, block, 62)
    s = torch.randn(Hq, generator=g) if sinks else None
    hit = [(0, 1, 2), (0, 6, 0), (1, 3, 0), (1, 4, 1), (2, 7, 1)]
    dirty, clean = q.clone(), q.clone()
    for i, (b, h, l) in enumerate(hit):
        dirty[b, h, l, (37 * i) % D] = bad
        clean[b, h, l] = 0
    got, want = attend(dirty, kc, vc, s, lens, 0, 0.1, block), attend(clean, kc, vc, s, lens, 0, 0.1, block)
    live = torch.ones(B, Hq, Lq, dtype=torch.bool)
    for b, h, l in hit:
        if lens[b] - Lq + l >= 0:
            live[b, h, l] = False
    assert int((~live).sum()) == 4
    assert bool(got[0][~live].isnan().all()) and bool(got[1][~live].isnan().all())
    assert torch.equal(got[0][live], want[0][live]) and torch.equal(got[1][live], want[1][live])


@pytest.mark.gpu
@pytest.mark.parametrize("D,Lq,window", [(64, 4, 0), (128, 1, 100), (256, 5, 0), (512, 1, 0)])
def test_what_stands_behind_the_lengths(D, Lq, window):
    """NaN codes and scales behind the lengths, and in empty places, change nothing; rows of empty places stay."""
    import sliding_window_attention_gb300 as swa

    g = torch.Generator().manual_seed(D)
    B, Hq, Hkv, rows, block = 5, 8, 2, 333, 32
    lens = [0, 1, -7, 200, 1000]
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF).cuda()
    kc, vc = filled(B, Hkv, rows, D, block, 51), filled(B, Hkv, rows, D, block, 52)
    clean = [kc[0].cuda(), vc[0].cuda(), kc[1].cuda(), vc[1].cuda()]
    dirty = [t.clone() for t in clean]
    for b, n in enumerate(lens):
        n = max(n, 0)
        for c, s in ((dirty[0], dirty[2]), (dirty[1], dirty[3])):
            c.view(torch.uint8)[b, :, n:] = 0x7F
            s[b, :, -(-n // block):] = math.nan
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    got = []
    for cache in (clean, dirty):
        o = torch.full((B, Hq, Lq, D), 7.0, dtype=BF, device="cuda")
        lse = torch.full((B, Hq, Lq), 7.0, device="cuda")
        ws = torch.full((swa.fwd_workspace_bytes_cache8(B, Hq, Hkv, Lq, rows, D, block, window),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        swa.swa_attn_fwd_cache8(q, *cache, n, None, o, lse, block, window, 0.1, ws)
        status_ok()
        got.append((o, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool((got[0][0][2] == 7).all()) and bool((got[0][1][2] == 7).all())
    assert bool((got[0][0][0] == 0).all()) and bool((got[0][1][0] == -math.inf).all())
    assert bool(got[0][0][[1, 3, 4]].isfinite().all())
    read = swa.cache8_read(*dirty, n, block)
    assert bool(read[0].isfinite().all()) and bool(read[1].isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("D,Lq,window", [(64, 1, 0), (128, 3, 200), (512, 9, 37)])
def test_attention_at_the_ends_of_the_lengths(D, Lq, window):
    """-2^31 is an empty place like -1, 2^31 - 1 a full cache like its number of rows."""
    import sliding_window_attention_gb300 as swa

    g = torch.Generator().manual_seed(D)
    B, Hq, Hkv, rows, block = 5, 4, 2, 300, 64
    q = torch.randn(B, Hq, Lq, D, generator=g).to(BF).cuda()
    kc, vc = filled(B, Hkv, rows, D, block, 63), filled(B, Hkv, rows, D, block, 64)
    cache = [t.cuda() for t in (kc[0], vc[0], kc[1], vc[1])]
    ws = torch.empty(swa.fwd_workspace_bytes_cache8(B, Hq, Hkv, Lq, rows, D, block, window), dtype=torch.uint8, device="cuda")
    got = []
    for lens in ([-2 ** 31, 200, 2 ** 31 - 1, -2 ** 31 + 5, 2 ** 31 - 200], [-1, 200, rows, -1, rows]):
        o, lse = torch.full_like(q, 3), torch.full((B, Hq, Lq), 3.0, device="cuda")
        n = torch.tensor(lens, dtype=torch.int32).cuda()
        swa.swa_attn_fwd_cache8(q, *cache, n, None, o, lse, block, window, 0.1, ws)
        kb, vb = swa.cache8_read(*cache, n, block)
        status_ok()
        got.append((o, lse, kb, vb))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert bool((got[0][0][[0, 3]] == 3).all()) and bool((got[0][1][[0, 3]] == 3).all())


@pytest.mark.gpu
def test_a_step_with_the_calls_around_it():
    """Rotation, append and attention, step after step, a request ending and a place reused: like
    forward_shared over bf16 caches that hold what the 8-bit cache's reads give."""
    import sliding_window_attention_gb300 as swa

    torch.manual_seed(3)
    B, Hq, Hkv, D, rows, block = 3, 8, 2, 128, 160, 16
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    w = torch.ones(D, device="cuda")
    cache = swa.make_cache8(B, Hkv, rows, D, block)
    lens = torch.tensor([100, 0, -1], dtype=torch.int32, device="cuda")
    for step, L in enumerate((1, 3, 1, 2, 1)):
        if step == 3:
            lens[1], lens[2] = -1, 0  # the second request ends, a third begins
        n = torch.where(lens >= 0, lens + L, lens).to(torch.int32)
        x = torch.randn(B, L, Hq + 2 * Hkv, D, device="cuda").to(BF)
        xq, xk, xv = x.split((Hq, Hkv, Hkv), 2)
        pos = ((n - L).clamp(min=0)[:, None] + torch.arange(L, device="cuda")).to(torch.int32).contiguous()
        q, k, _ = swa.qk_rope(xq, xk, None, w, w, inv, 1e-6, positions=pos)
        swa.cache8_append(k, xv.transpose(1, 2), *cache, n, block)
        o, lse = swa.forward_cache8(q, *cache, n, block, 64, 0.09)
        kb, vb = swa.cache8_read(*cache, n, block)
        live = n >= 0
        o2, lse2 = swa.forward_shared(q, None, None, kb, vb, n, 64, 0.09)
        # both round o (2^-8), one its weights to 2^-8, the other to 2^-11: of sum p |v| at most; scores to 2^-16 of 12
        assert float((o.float() - o2.float())[live].abs().max()) <= 3.25 * 2.0 ** -8 * float(vb.float().abs().max())
        assert float((lse - lse2)[live].abs().max()) <= 2.0 ** -9
        # what was appended reads back within half a step of e4m3, of the block's scale below
        for got, want, s in ((kb, k, cache[2]), (vb, xv.transpose(1, 2), cache[3])):
            for b in range(B):
                if live[b]:
                    m = int(n[b])
                    y, z = got[b, :, m - L:m].float(), want[b].float()
                    step_ = s[b, :, torch.arange(m - L, m, device="cuda") // block][..., None]
                    assert bool(((y - z).abs() <= torch.maximum(z.abs() * 2.0 ** -4, step_ * 2.0 ** -10)).all())
        lens = n
    status_ok()


@pytest.mark.gpu
def test_a_prompt_in_chunks():
    """A prompt's chunks appended, read back and attended by the training forward: the same as one append of all."""
    import sliding_window_attention_gb300 as swa

    torch.manual_seed(4)
    B, Hkv, D, L, block = 1, 2, 64, 300, 64
    k, v = (torch.randn(B, Hkv, L, D, device="cuda").to(BF) for _ in range(2))
    one, parts = swa.make_cache8(B, Hkv, L, D, block), swa.make_cache8(B, Hkv, L, D, block)
    swa.cache8_append(k, v, *one, None, block)
    for a, b in ((0, 128), (128, 192), (192, 300)):  # at the blocks' borders: no scale has to grow
        swa.cache8_append(k[:, :, a:b], v[:, :, a:b], *parts, torch.tensor([b], dtype=torch.int32, device="cuda"), block)
    for x, y in zip(one, parts):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    kb, vb = swa.cache8_read(*parts, None, block)
    q = torch.randn(B, 4, 108, D, device="cuda").to(BF)
    o, lse = swa.forward(q, kb, vb, 0, 0.125)  # 108 rows behind 192 keys
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    o8, lse8 = swa.forward_cache8(q, *parts, n, block, 0, 0.125)
    status_ok()
    # o is rounded once (2^-8), weights to 2^-11 on either side, scores to 2^-14 with the sums
    assert float((o - o8.float()).abs().max()) <= (2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -12) * float(vb.float().abs().max())
    assert float((lse - lse8).abs().max()) <= 2.0 ** -10


@pytest.mark.gpu
def test_captured_and_replayed():
    """A captured step replays with the lengths and tokens of then; two graphs share a workspace one after the other."""
    import sliding_window_attention_gb300 as swa

    torch.manual_seed(5)
    B, Hq, Hkv, D, rows, block = 4, 8, 4, 128, 700, 64
    cache = swa.make_cache8(B, Hkv, rows, D, block)
    k, v = (torch.randn(B, Hkv, 1, D, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(B, Hq, 1, D, device="cuda").to(BF)
    big = torch.randn(2, B, Hkv, rows, D, device="cuda").to(BF)
    swa.cache8_append(big[0], big[1], *cache, None, block)
    n = torch.tensor([5, 700, -1, 300], dtype=torch.int32, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(B, Hq, 1, device="cuda")
    ws = torch.empty(swa.fwd_workspace_bytes_cache8(B, Hq, Hkv, 1, rows, D, block, 0), dtype=torch.uint8, device="cuda")

    def step(out, l):
        swa.cache8_append(k, v, *cache, n, block)
        swa.swa_attn_fwd_cache8(q, *cache, n, None, out, l, block, 0, 0.1, ws)

    step(o, lse)
    o2, lse2 = torch.zeros_like(q), torch.zeros_like(lse)
    graphs = []
    for out, l in ((o, lse), (o2, lse2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(out, l)
        graphs.append(g)
    for lens in ([6, 700, 1, 299], [640, -1, 2, 1]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        for t in (k, v, q):
            t.copy_(torch.randn_like(t))
        o.fill_(3)
        o2.fill_(3)
        for g in graphs:
            g.replay()
        want = swa.forward_cache8(q, *cache, n, block, 0, 0.1)  # (the append again changes nothing)
        torch.cuda.synchronize()
        live = n >= 0
        assert torch.equal(o[live], want[0][live]) and torch.equal(o2[live], want[0][live])
        assert torch.equal(lse[live], want[1][live]) and bool((o[~live] == 3).all())
    status_ok()


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls of different shapes on two streams, like their results one after the other."""
    import sliding_window_attention_gb300 as swa

    torch.manual_seed(6)
    jobs = []
    for B, Hq, Hkv, Lq, D, rows, block in ((8, 8, 4, 1, 128, 4000, 64), (3, 32, 4, 4, 256, 3000, 32)):
        cache = swa.make_cache8(B, Hkv, rows, D, block)
        x = torch.randn(2, B, Hkv, rows, D, device="cuda").to(BF)
        n = torch.randint(1, rows, (B,), device="cuda", dtype=torch.int32)
        q = torch.randn(B, Hq, Lq, D, device="cuda").to(BF)
        swa.cache8_append(x[0], x[1], *cache, None, block)
        jobs.append((q, cache, n, block, swa.forward_cache8(q, *cache, n, block, 0, 0.1)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [[], []]
    for _ in range(20):
        for i, (q, cache, n, block, _w) in enumerate(jobs):
            out[i].append(swa.forward_cache8(q, *cache, n, block, 0, 0.1, stream=streams[i]))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for got in out[i]:
            assert torch.equal(got[0], job[4][0]) and torch.equal(got[1], job[4][1])
    status_ok()


@pytest.mark.gpu
def test_beyond_four_gigabytes():
    """Codes behind 2^32 bytes: an append at the end, the read of it, and the attention's window there."""
    import sliding_window_attention_gb300 as swa

    B, Hkv, D, rows, block, L = 1, 2, 512, 4_400_000, 128, 200
    assert Hkv * rows * D > 2 ** 32
    codes = [torch.zeros((B, Hkv, rows, D), dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
    scales = [torch.ones((B, Hkv, -(-rows // block)), device="cuda") for _ in range(2)]
    torch.manual_seed(8)
    k, v = (torch.randn(B, Hkv, L, D, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(B, 4, 1, D, device="cuda").to(BF)
    end = rows - 3
    n = torch.tensor([end], dtype=torch.int32, device="cuda")
    swa.cache8_append(k, v, *codes, *scales, n, block)
    kb, vb = swa.cache8_read(*codes, *scales, n, block, end - L, L)
    o, lse = swa.forward_cache8(q, *codes, *scales, n, block, 150, 0.05)
    # the same tokens at the same places of their blocks in a small cache
    first = (end - L) % block
    small = swa.make_cache8(B, Hkv, first + L, D, block)
    m = torch.tensor([first + L], dtype=torch.int32, device="cuda")
    swa.cache8_append(k, v, *small, m, block)
    nb, j0 = small[2].shape[2], (end - L) // block
    assert torch.equal(scales[0][:, :, j0:j0 + nb], small[2]) and torch.equal(scales[1][:, :, j0:j0 + nb], small[3])
    k2, v2 = swa.cache8_read(*small, m, block, first, L)
    o2, lse2 = swa.forward_cache8(q, *small, m, block, 150, 0.05)
    status_ok()
    assert torch.equal(kb, k2) and torch.equal(vb, v2) and torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def lib():
    from sliding_window_attention_gb300 import build as b
    from sliding_window_attention_gb300 import _native

    b.build()
    return _native.load()


def codes_of(lib):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "swa_attn.h")).read()
    return {m.group(1): int(m.group(2)) for m in re.finditer(r"#define (SWA_\w+) (-?\d+)", text)}


def test_append_refuses_before_any_cuda_call(lib):
    c = codes_of(lib)

    def call(k=0x1000, v=0x2000, sb=4096, sh=1024, st=64, n=0x3000, kc=0x4000, vc=0x5000, ks=0x6000, vs=0x7000, B=2,
             Hkv=2, L=3, D=64, rows=32, block=16):
        return lib.swa_attn_cache8_append(k, v, sb, sh, st, sb, sh, st, n, kc, vc, ks, vs, B, Hkv, L, D, rows, block, None)

    assert call(k=0, v=0) == c["SWA_ERR_NULL_POINTER"]
    assert call(kc=0) == c["SWA_ERR_NULL_POINTER"] and call(vs=0) == c["SWA_ERR_NULL_POINTER"]
    assert call(B=0) == c["SWA_ERR_BAD_SHAPE"] and call(L=0) == c["SWA_ERR_BAD_SHAPE"]
    assert call(D=96) == c["SWA_ERR_BAD_HEAD_DIM"]
    assert call(rows=0) == c["SWA_ERR_BAD_CACHE"] and call(block=48) == c["SWA_ERR_BAD_CACHE"]
    assert call(n=0, L=33) == c["SWA_ERR_BAD_CACHE"]
    assert call(st=65) == c["SWA_ERR_BAD_STRIDE"] and call(st=0) == c["SWA_ERR_BAD_STRIDE"]
    assert call(sh=-64) == c["SWA_ERR_BAD_STRIDE"]
    for name in ("k", "v", "kc", "vc"):
        assert call(**{name: 0x8008}) == c["SWA_ERR_MISALIGNED"], name
    assert call(n=0x3002) == c["SWA_ERR_MISALIGNED"] and call(ks=0x6001) == c["SWA_ERR_MISALIGNED"]
    assert call(B=60000, Hkv=60000) == c["SWA_ERR_TOO_LARGE"]


def test_read_refuses_before_any_cuda_call(lib):
    c = codes_of(lib)

    def call(kc=0x1000, vc=0x2000, ks=0x3000, vs=0x4000, n=0x5000, ko=0x6000, vo=0x7000, B=2, Hkv=2, D=64, rows=32,
             block=16, row0=0, count=32):
        return lib.swa_attn_cache8_read(kc, vc, ks, vs, n, ko, vo, B, Hkv, D, rows, block, row0, count, None)

    assert call(ko=0, vo=0) == c["SWA_ERR_NULL_POINTER"] and call(kc=0) == c["SWA_ERR_NULL_POINTER"]
    assert call(Hkv=0) == c["SWA_ERR_BAD_SHAPE"] and call(D=1024) == c["SWA_ERR_BAD_HEAD_DIM"]
    assert call(row0=-1) == c["SWA_ERR_BAD_CACHE"] and call(row0=1) == c["SWA_ERR_BAD_CACHE"]
    assert call(count=0) == c["SWA_ERR_BAD_CACHE"] and call(block=0) == c["SWA_ERR_BAD_CACHE"]
    assert call(row0=2 ** 31 - 1, count=2 ** 31 - 1) == c["SWA_ERR_BAD_CACHE"]
    assert call(vo=0x7008) == c["SWA_ERR_MISALIGNED"]


def test_attention_refuses_before_any_cuda_call(lib):
    import ctypes

    c = codes_of(lib)

    def call(q=0x1000, kc=0x2000, vc=0x3000, ks=0x4000, vs=0x5000, n=0x6000, sinks=0, o=0x7000, lse=0x8000, B=2, Hq=4,
             Hkv=2, Lq=1, rows=64, D=64, block=16, window=0, scale=0.1, ws=0x100000, nbytes=None):
        if nbytes is None:
            nbytes = lib.swa_attn_fwd_workspace_bytes_cache8(B, Hq, Hkv, Lq, rows, D, block, window)
        return lib.swa_attn_fwd_cache8(q, kc, vc, ks, vs, n, sinks, o, lse, B, Hq, Hkv, Lq, rows, D, block, window,
                                       ctypes.c_float(scale), ws, nbytes, None)

    for name in ("q", "kc", "vc", "ks", "vs", "n", "o", "lse"):
        assert call(**{name: 0}) == c["SWA_ERR_NULL_POINTER"], name
    assert call(Hq=3) == c["SWA_ERR_BAD_GROUPS"] and call(Lq=0) == c["SWA_ERR_BAD_SHAPE"]
    assert call(D=32) == c["SWA_ERR_BAD_HEAD_DIM"] and call(window=-1) == c["SWA_ERR_BAD_WINDOW"]
    assert call(scale=math.inf) == c["SWA_ERR_BAD_SCALE"] and call(scale=math.nan) == c["SWA_ERR_BAD_SCALE"]
    assert call(rows=0) == c["SWA_ERR_BAD_CACHE"] and call(block=24) == c["SWA_ERR_BAD_CACHE"]
    assert call(ws=0) == c["SWA_ERR_WORKSPACE"] and call(nbytes=1000) == c["SWA_ERR_WORKSPACE"]
    assert call(ws=0x100010) == c["SWA_ERR_MISALIGNED"] and call(sinks=0x9002) == c["SWA_ERR_MISALIGNED"]
    assert call(kc=0x2004) == c["SWA_ERR_MISALIGNED"] and call(lse=0x8002) == c["SWA_ERR_MISALIGNED"]
    assert call(B=60000, rows=10 ** 6) == c["SWA_ERR_TOO_LARGE"]
    assert lib.swa_attn_fwd_workspace_bytes_cache8(2, 3, 2, 1, 64, 64, 16, 0) == 0
    assert lib.swa_attn_fwd_workspace_bytes_cache8(2, 4, 2, 1, 64, 64, 16, 0) % 256 == 0


def test_binding_refuses_host_tensors(lib):
    import sliding_window_attention_gb300 as swa

    cache = swa.make_cache8(1, 2, 32, 64, 16, device="cpu")
    k = torch.zeros(1, 2, 1, 64, dtype=BF)
    n = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.cache8_append(k, k, *cache, n, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.cache8_read(*cache, n, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.forward_cache8(torch.zeros(1, 4, 1, 64, dtype=BF), *cache, n, 16, 0, 0.1)


def test_a_cache_that_no_call_takes_is_not_made():
    import sliding_window_attention_gb300 as swa

    for shape in ((1, 2, 32, 64, 0), (1, 2, 32, 64, 24), (1, 2, 32, 64, -16), (1, 2, 32, 96, 16), (0, 2, 32, 64, 16),
                  (1, 0, 32, 64, 16), (1, 2, 0, 64, 16), (1, 2, -1, 64, 16)):
        with pytest.raises(ValueError, match="block must be|a cache has"):
            swa.make_cache8(*shape, device="cpu")
    k8, v8, ks, vs = swa.make_cache8(2, 3, 33, 64, 16, device="cpu")
    assert k8.shape == v8.shape == (2, 3, 33, 64) and ks.shape == vs.shape == (2, 3, 3) and k8.dtype is F8


@pytest.mark.gpu
def test_a_read_refuses_outputs_of_other_dimensions():
    import sliding_window_attention_gb300 as swa

    k8, v8, ks, vs = swa.make_cache8(2, 2, 48, 64, 16)
    out = torch.zeros(2, 2, 48, 64, dtype=BF, device="cuda")
    for k_out, v_out in ((out[0, 0], out), (out[0], None), (None, out[0, 0]), (out[None], out)):
        with pytest.raises(ValueError):
            swa.swa_attn_cache8_read(k8, v8, ks, vs, None, k_out, v_out, 16)
    status_ok()


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    import sliding_window_attention_gb300 as swa

    k8, v8, ks, vs = swa.make_cache8(2, 2, 48, 64, 16)
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 2, 1, 64, dtype=BF, device="cuda")
    q = torch.zeros(2, 4, 1, 64, dtype=BF, device="cuda")
    bad = [lambda: swa.cache8_append(k.float(), k, k8, v8, ks, vs, n, 16),
           lambda: swa.cache8_append(k[:, :1], k, k8, v8, ks, vs, n, 16),
           lambda: swa.cache8_append(k, k, k8.view(torch.uint8), v8, ks, vs, n, 16),
           lambda: swa.cache8_append(k, k, k8, v8, ks[..., :2], vs, n, 16),
           lambda: swa.cache8_append(k, k, k8, v8, ks, vs, n.long(), 16),
           lambda: swa.cache8_append(k, k, k8, v8, ks, vs, n, 32),
           lambda: swa.cache8_append(torch.zeros(2, 2, 1, 128, dtype=BF, device="cuda")[..., ::2], k, k8, v8, ks, vs, n,
                                     16),
           lambda: swa.cache8_append(None, None, k8, v8, ks, vs, n, 16),
           lambda: swa.cache8_append(k, k, None, v8, ks, vs, n, 16),
           lambda: swa.cache8_read(k8, v8, ks, vs.double(), n, 16),
           lambda: swa.cache8_read(k8, v8, ks, vs, n, 16, 40, 9),
           lambda: swa.cache8_read(k8, v8, ks, vs, n, 16, -1),
           lambda: swa.forward_cache8(q.float(), k8, v8, ks, vs, n, 16, 0, 0.1),
           lambda: swa.forward_cache8(q[:1], k8, v8, ks, vs, n, 16, 0, 0.1),
           lambda: swa.forward_cache8(q[0], k8, v8, ks, vs, n, 16, 0, 0.1),
           lambda: swa.forward_cache8(q, k8, v8, ks, vs, None, 16, 0, 0.1),
           lambda: swa.forward_cache8(q, k8, v8, ks, vs, n, 16, 2 ** 40, 0.1),
           lambda: swa.forward_cache8(q, k8, v8, ks, vs, n, 16, 0, 0.1, sinks=torch.zeros(3, device="cuda")),
           lambda: swa.forward_cache8(q.transpose(1, 3).contiguous().transpose(1, 3), k8, v8, ks, vs, n, 16, 0, 0.1)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    wide = torch.zeros(2, 2, 1, 68, dtype=BF, device="cuda")[..., :64]  # heads 68 elements apart
    for f in (lambda: swa.cache8_append(wide, k, k8, v8, ks, vs, n, 16),
              lambda: swa.cache8_append(k[:, :1].expand(2, 2, 1, 64), k, k8, v8, ks, vs, n, 16),
              lambda: swa.forward_cache8(q, k8, v8, ks, vs, n, 16, -3, 0.1),
              lambda: swa.forward_cache8(q[:, :3].contiguous(), k8, v8, ks, vs, n, 16, 0, 0.1)):
        with pytest.raises(swa.SwaError):
            f()
    status_ok()
