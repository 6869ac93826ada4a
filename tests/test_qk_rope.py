"""Per-head norm, scale and rotation of q and k (swa_attn_qk_rope_fwd / _bwd)
against the definition in 64 bits, on the same bf16 inputs.

Tolerances, from the kernel's roundings (eps = 2^-24 for one fp32 rounding).
A value u = x r w carries at most 2^-18 relative error before the rotation:
the sum of D squares is 8 or 16 sequential and 5 or fewer pairwise additions
(21 eps), rsqrtf and the products a few eps more; cos and sin add their ulps
and a phase error below 2^-22 of a radian.  A rotated element is a difference
of two products, so its error before the last rounding is at most
2^-18 (|u_a| + |u_b|); rounding to bf16 adds half a step, 2^-8 of the value.
"""
import math

import pytest
import torch

BF = torch.bfloat16
HALF_STEP = 2.0 ** -8  # bf16
F32 = 2.0 ** -18
EPS = 1e-6


def freqs(pairs, theta=10000.0):
    return theta ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))


def fused(B, L, Hq, Hkv, D, seed, pad=0):
    """q, k, v as slices of one projection output, `pad` elements between tokens."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn((B, L, (Hq + 2 * Hkv) * D + pad), generator=g).to(BF)
    rows = buf[:, :, :(Hq + 2 * Hkv) * D].unflatten(2, (Hq + 2 * Hkv, D))
    return rows.split((Hq, Hkv, Hkv), dim=2), g


def turn(x, pos, inv_freq, interleaved, sign=1.0):
    """fp64 x [B, L, H, D] turned by sign * pos [B, L] * inv_freq."""
    n = inv_freq.numel()
    a = sign * pos.double()[:, :, None, None] * inv_freq
    c, s = torch.cos(a), torch.sin(a)
    y = x.clone()
    if interleaved:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = u * c - v * s, v * c + u * s
    else:
        u, v = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = u * c - v * s, v * c + u * s
    return y


def pair_size(x, n, interleaved):
    """|x_a| + |x_b| of each element's pair (|x| beyond the rotated part)."""
    y = x.abs()
    z = y.clone()
    if interleaved:
        s = y[..., 0:2 * n:2] + y[..., 1:2 * n:2]
        z[..., 0:2 * n:2] = z[..., 1:2 * n:2] = s
    else:
        s = y[..., :n] + y[..., n:2 * n]
        z[..., :n] = z[..., n:2 * n] = s
    return z


def norm_ref(x, w, off):
    x = x.double()
    n = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    return n, (torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double() + off)


def forward_ref(x, w, off, pos, inv_freq, interleaved):
    """(y, size) [B, H, L, D]: the definition, and |u_a| + |u_b| of each element."""
    n, we = norm_ref(x, w, off)
    u = n * we
    return turn(u, pos, inv_freq, interleaved).transpose(1, 2), pair_size(u, inv_freq.numel(), interleaved).transpose(1, 2)


def check_rows(name, got, ref, size):
    d = (got.double().cpu() - ref).abs()
    tol = HALF_STEP * ref.abs() + F32 * (1 + HALF_STEP) * size
    bad = d > tol
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst by {float((d - tol).max()):.3e}"


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def dev_rows(ts, pad):
    """The same slices on the GPU, with the same strides between tokens."""
    B, L, _, D = ts[0].shape
    H = sum(t.shape[2] for t in ts)
    buf = torch.full((B, L, H * D + pad), float("nan"), dtype=BF, device="cuda")
    rows = buf[:, :, :H * D].unflatten(2, (H, D))
    rows.copy_(torch.cat(ts, 2))
    return rows.split([t.shape[2] for t in ts], dim=2)


CASES = [
    # B, L, Hq, Hkv, D, rot, interleaved, weights, off, pos0, pad
    (1, 1, 1, 1, 64, 64, False, True, 0.0, 0, 0),
    (2, 37, 2, 1, 64, 32, False, True, 1.0, 5, 8),
    (1, 129, 8, 4, 128, 128, False, True, 0.0, 0, 0),
    (3, 50, 5, 5, 128, 96, False, False, 0.0, 999983, 0),
    (1, 200, 6, 3, 256, 256, False, True, 0.0, 2147480000, 16),
    (1, 77, 3, 1, 256, 16, True, True, 1.0, 30553, 0),
    (2, 33, 4, 2, 512, 512, False, True, 0.0, 0, 0),
    (1, 40, 2, 1, 512, 384, False, True, 0.5, 100, 0),
    (1, 40, 2, 1, 512, 256, False, False, 0.0, 100, 0),
    (1, 19, 3, 1, 512, 512, True, True, 0.0, 7, 8),
    (1, 21, 9, 3, 64, 64, True, True, 0.0, 16384, 0),
    (1, 10, 2, 2, 128, 0, False, True, 0.0, 0, 0),  # norm alone
    (600, 7, 3, 1, 64, 64, False, True, 0.0, 0, 0),   # many tokens, short sequences
    # long sequences (staged through shared memory): heads that leave a stage part empty, odd lengths
    (1, 4100, 3, 1, 64, 64, False, True, 0.0, 0, 0),
    (3, 401, 9, 1, 64, 32, True, True, 1.0, 3, 8),
    (2, 705, 5, 3, 128, 128, False, True, 0.0, 70000, 0),
    (1, 1024, 4, 4, 128, 96, False, False, 0.0, 0, 16),
    (1, 1100, 5, 3, 256, 256, True, True, 0.5, 0, 0),
    (2, 515, 2, 1, 256, 32, False, True, 0.0, 999983, 0),
    (1, 1030, 3, 2, 512, 512, False, True, 0.0, 0, 8),
    (1, 1025, 2, 1, 512, 384, False, True, 0.0, 5, 0),
    (5, 210, 1, 1, 512, 0, False, True, 0.0, 0, 0),
    # many tokens of few heads (several tokens a warp)
    (1, 7001, 2, 1, 64, 64, False, True, 0.0, 0, 0),
    (3, 2403, 2, 1, 64, 32, True, True, 1.0, 3, 8),
    (2, 5003, 1, 1, 128, 128, False, True, 0.0, 999983, 0),
    (1, 9005, 2, 1, 128, 96, False, False, 0.5, 0, 16),
    (5, 1301, 8, 4, 64, 64, False, True, 0.0, 30553, 0),
    (700, 33, 2, 1, 64, 48, False, True, 0.0, 0, 0),
    (1, 12000, 1, 1, 128, 128, True, True, 0.0, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,Hq,Hkv,D,rot,inter,weights,off,pos0,pad", CASES)
def test_forward(B, L, Hq, Hkv, D, rot, inter, weights, off, pos0, pad):
    import sliding_window_attention_gb300 as swa

    (q, k, v), g = fused(B, L, Hq, Hkv, D, 100 + L + D, pad)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g) - off) if weights else None for _ in range(2))
    f = freqs(rot // 2)
    pos = torch.arange(L)[None].expand(B, L) + pos0
    qd, kd, vd = dev_rows((q, k, v), pad)
    got = swa.qk_rope(qd, kd, vd, *cuda(wq, wk, f if rot else None), EPS, pos0=pos0, weight_offset=off,
                      interleaved=inter)
    for name, x, w, y in (("q", q, wq, got[0]), ("k", k, wk, got[1])):
        check_rows(name, y, *forward_ref(x, w, off, pos, f, inter))
    assert torch.equal(got[2].cpu(), v.transpose(1, 2).contiguous())


@pytest.mark.gpu
def test_forward_positions_and_missing_k_and_v():
    """Positions in any order, negative ones too; queries alone, and keys without values."""
    import sliding_window_attention_gb300 as swa

    B, L, Hq, Hkv, D = 2, 30, 3, 1, 128
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 3)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    pos = torch.randint(-5000, 5000, (B, L), generator=g, dtype=torch.int32)
    pos[0, 0], pos[1, 3] = 2 ** 31 - 1, -2 ** 31
    f = freqs(64)
    qd, kd, vd, wd, fd, pd = cuda(q, k, v, w, f, pos)
    qd, kd = qd.contiguous(), kd.contiguous()
    a = swa.qk_rope(qd, kd, None, wd, wd, fd, EPS, positions=pd)
    assert a[2] is None
    check_rows("q", a[0], *forward_ref(q, w, 0.0, pos, f, False))
    check_rows("k", a[1], *forward_ref(k, w, 0.0, pos, f, False))
    b = swa.qk_rope(qd, None, None, wd, None, fd, EPS, positions=pd)
    assert b[1] is None and b[2] is None and torch.equal(a[0], b[0])


@pytest.mark.gpu
def test_extreme_rows():
    """A row of zeros stays zero; rows at the ends of bf16's range of squares keep the formula's value."""
    import sliding_window_attention_gb300 as swa

    (q, _, _), _ = fused(1, 6, 2, 1, 128, 9)
    q = q.contiguous()
    q[0, 1] = 0
    q[0, 2] *= 2.0 ** 60   # squares to 2^120 and a sum below fp32's largest
    q[0, 3] *= 2.0 ** -60  # far below eps: x / sqrt(eps)
    f = freqs(64)
    got = swa.qk_rope(q.cuda(), None, None, None, None, f.cuda(), EPS)[0]
    check_rows("q", got, *forward_ref(q, None, 0.0, torch.arange(6)[None], f, False))
    assert torch.count_nonzero(got[0, :, 1]) == 0
    q[0, 4, 0, 5] = float("nan")  # stays within its row
    again = swa.qk_rope(q.cuda(), None, None, None, None, f.cuda(), EPS)[0]
    assert torch.isnan(again[0, 0, 4]).all()
    keep = torch.ones(2, 6, dtype=torch.bool)
    keep[0, 4] = False
    assert torch.equal(again[0][keep.cuda()], got[0][keep.cuda()])


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,D,inter", [(5, 1, 128, False), (3, 4, 512, True), (70, 2, 64, False), (5, 260, 128, False),
                                         (3, 600, 64, True)])
def test_append(B, L, D, inter):
    """Keys and values land in each request's rows, positions follow them, and nothing else is written."""
    import sliding_window_attention_gb300 as swa

    Hq, Hkv, rows, pos0 = 4, 2, L + 7, 1000
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 17 + B)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    n = torch.randint(L, rows + 1, (B,), generator=g, dtype=torch.int32)
    n[0] = L - 1       # the first token would go in front of the cache
    n[1] = rows + 1    # the last one behind it
    n[2] = -1          # an empty place
    f = freqs(D // 2)
    kc, vc = (torch.full((B, Hkv, rows, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    qd, kd, vd = dev_rows((q, k, v), 0)
    got = swa.qk_rope_append(qd, kd, vd, w.cuda(), w.cuda(), f.cuda(), kc, vc, n.cuda(), EPS, pos0=pos0,
                             interleaved=inter)
    pos = pos0 + n[:, None] - L + torch.arange(L)
    check_rows("q", got, *forward_ref(q, w, 0.0, pos, f, inter))
    ref, size = forward_ref(k, w, 0.0, pos, f, inter)
    written = torch.zeros(B, rows, dtype=torch.bool)
    for b in range(B):
        l = torch.arange(L)
        r = int(n[b]) - L + l
        l, r = l[(r >= 0) & (r < rows)], r[(r >= 0) & (r < rows)]
        written[b, r] = True
        check_rows("k", kc[b][:, r.cuda()], ref[b][:, l], size[b][:, l])
        assert torch.equal(vc[b][:, r.cuda()].cpu(), v[b, l].transpose(0, 1))
    for c in (kc, vc):
        assert torch.isnan(c).all(-1).all(1).cpu().logical_xor(written).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,Hq,Hkv,D,rot,inter,weights,off,pos0,pad", CASES)
def test_backward(B, L, Hq, Hkv, D, rot, inter, weights, off, pos0, pad):
    """dx = r (h - n mean(h n)) with g = R^T dy, h = g w: g carries 2^-18 of its
    pair's size like the forward, the mean's term 2^-18 of mean |h n|, and the
    result is rounded to bf16 once.  dw sums g n over the rows: each term
    carries 2^-18 of its size, the sums their chains' roundings (a lane's rows,
    then at most 64 more additions)."""
    import sliding_window_attention_gb300 as swa

    (q, k, v), g = fused(B, L, Hq, Hkv, D, 200 + L + D, pad)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g) - off) if weights else None for _ in range(2))
    dq, dk, dv = (0.3 * torch.randn((B, h, L, D), generator=g) for h in (Hq, Hkv, Hkv))
    f = freqs(rot // 2)
    pos = torch.arange(L)[None].expand(B, L) + pos0
    qd, kd, _ = dev_rows((q, k, v), pad)
    d, dwq, dwk = swa.qk_rope_backward(qd, kd, *cuda(wq, wk, f if rot else None, dq, dk, dv), EPS, pos0=pos0,
                                       weight_offset=off, interleaved=inter)
    gq, gk, gv = d.split((Hq, Hkv, Hkv), 2)
    assert torch.equal(gv.cpu(), dv.transpose(1, 2).to(BF))
    chain = math.ceil(B * math.ceil(L / 8) * max(Hq, Hkv) / 152) + 8 + 64
    for name, x, w, dy, got, dw in (("q", q, wq, dq, gq, dwq), ("k", k, wk, dk, gk, dwk)):
        n, we = norm_ref(x, w, off)
        r = 1 / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt()
        gr = turn(dy.double().transpose(1, 2), pos, f, inter, -1.0)
        size = pair_size(dy.double().transpose(1, 2), rot // 2, inter)
        h = gr * we
        ref = r * (h - n * (h * n).mean(-1, keepdim=True))
        part = r * (size * we.abs() + n.abs() * (size * we.abs() * n.abs()).mean(-1, keepdim=True))
        check_rows("d" + name, got, ref, part)
        if w is None:
            assert dw is None
            continue
        terms = (size * n.abs()).sum((0, 1, 2))
        err = (dw.double().cpu() - (gr * n).sum((0, 1, 2))).abs()
        tol = (F32 + chain * 2.0 ** -24) * terms
        assert (err <= tol).all(), f"dw{name}: worst {float((err / tol).max()):.2f} of the tolerance"


@pytest.mark.gpu
def test_backward_matches_differences():
    """The gradient against central differences of the definition's loss, one input and one scale at a time.
    With a step of 1e-4 and third derivatives of order one in these units the differences are exact to
    about 1e-8.  dx is a bf16 rounding of it; 1e-4 covers 2^-18 of terms that add up to at most 25."""
    import sliding_window_attention_gb300 as swa

    B, L, Hq, Hkv, D = 1, 3, 2, 1, 64
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 5)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    dq, dk, dv = (torch.randn((B, h, L, D), generator=g) for h in (Hq, Hkv, Hkv))
    f = freqs(32)
    pos = torch.arange(L)[None] + 11
    qd, kd, _ = dev_rows((q, k, v), 0)
    d, dwq, _ = swa.qk_rope_backward(qd, kd, *cuda(w, w, f, dq, dk, dv), EPS, pos0=11)

    def loss(x, ww):
        n = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * ww
        return float((turn(n, pos, f, False).transpose(1, 2) * dq.double()).sum())

    x, ww = q.double().contiguous(), w.double()
    for l, h, e in ((0, 0, 0), (1, 1, 33), (2, 0, 63), (2, 1, 31)):
        a, b = x.clone(), x.clone()
        a[0, l, h, e] += 1e-4
        b[0, l, h, e] -= 1e-4
        num = (loss(a, ww) - loss(b, ww)) / 2e-4
        assert abs(float(d[0, l, h, e]) - num) <= HALF_STEP * abs(num) + 1e-4
    for e in (0, 17, 32, 63):
        a, b = ww.clone(), ww.clone()
        a[e] += 1e-4
        b[e] -= 1e-4
        assert abs(float(dwq[e]) - (loss(x, a) - loss(x, b)) / 2e-4) <= 1e-4


@pytest.mark.gpu
def test_backward_without_k_or_v_and_repeats():
    """Two runs give equal bits; queries alone give the same rows, and dwq but for the order of its sum
    (which follows the launch's list of heads): two sums of the same fp32 terms in chains of at most 80
    additions are at most 160 eps of the terms' sizes apart."""
    import sliding_window_attention_gb300 as swa

    B, L, Hq, Hkv, D = 2, 600, 4, 2, 128
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 8)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    dq, dk, dv = (torch.randn((B, h, L, D), generator=g) for h in (Hq, Hkv, Hkv))
    qd, kd, wd, fd, dqd, dkd, dvd = cuda(q, k, w, freqs(64), dq, dk, dv)
    qd, kd = qd.contiguous(), kd.contiguous()
    full = swa.qk_rope_backward(qd, kd, wd, wd, fd, dqd, dkd, dvd, EPS)
    twice = swa.qk_rope_backward(qd, kd, wd, wd, fd, dqd, dkd, dvd, EPS)
    for a, b in zip(full, twice):
        assert torch.equal(a, b)
    alone = swa.qk_rope_backward(qd, None, wd, None, fd, dqd, None, None, EPS)
    assert alone[0].shape == (B, L, Hq, D) and alone[2] is None
    assert torch.equal(alone[0], full[0][:, :, :Hq].contiguous())
    n, _ = norm_ref(q, None, 0.0)
    terms = (pair_size(dq.double().transpose(1, 2), 64, False) * n.abs()).sum((0, 1, 2))
    assert ((alone[1] - full[1]).abs().cpu() <= 160 * 2.0 ** -24 * terms).all()


@pytest.mark.gpu
def test_side_stream_and_graph():
    """On a stream of its own, and captured and replayed on new inputs in the same buffers."""
    import sliding_window_attention_gb300 as swa

    B, L, Hq, Hkv, D = 4, 1, 4, 2, 128
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 21)
    w, f = cuda(1 + 0.2 * torch.randn(D, generator=g), freqs(64))
    qd, kd, vd = dev_rows((q, k, v), 0)
    n = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((B, Hkv, 8, D), dtype=BF, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = swa.qk_rope_append(qd, kd, vd, w, w, f, kc, vc, n, EPS)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = swa.qk_rope_append(qd, kd, vd, w, w, f, kc, vc, n, EPS)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    n += 1
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, swa.qk_rope_append(qd, kd, vd, w, w, f, kc, vc, n, EPS))
    for b in range(B):
        assert torch.equal(vc[b, :, b], vc[b, :, b + 1]) and not torch.equal(kc[b, :, b], kc[b, :, b + 1])


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """More than 2^32 bytes and 2^31 elements on both sides: the last tokens' rows, and rows far inside a cache."""
    import sliding_window_attention_gb300 as swa

    H, D, L = 4, 512, (1 << 31) // (4 * 512) + 1003
    g = torch.Generator().manual_seed(2)
    x = torch.empty((1, L, H, D), dtype=BF, device="cuda")
    x[:, -9:] = torch.randn((9, H, D), generator=g).to(BF)
    f = freqs(64)
    tail = torch.arange(L - 9, L)[None]
    y = swa.qk_rope(x, None, None, None, None, f.cuda(), EPS)[0]
    check_rows("q", y[:, :, -9:], *forward_ref(x[:, -9:].cpu(), None, 0.0, tail, f, False))
    dy = torch.zeros((1, H, L, D), dtype=torch.float32, device="cuda")
    dy[:, :, -9:] = torch.randn((H, 9, D), generator=g)
    d, _, _ = swa.qk_rope_backward(x, None, None, None, f.cuda(), dy, None, None, EPS)
    xr, gr = x[:, -9:].cpu().double(), turn(dy[:, :, -9:].cpu().double().transpose(1, 2), tail, f, False, -1.0)
    r = 1 / (xr.square().mean(-1, keepdim=True) + EPS).sqrt()
    n = xr * r
    size = pair_size(dy[:, :, -9:].cpu().double().transpose(1, 2), 64, False)
    ref = r * (gr - n * (gr * n).mean(-1, keepdim=True))
    check_rows("dq", d[:, -9:], ref, r * (size + n.abs() * (size * n.abs()).mean(-1, keepdim=True)))
    del d, dy
    k = x[:, -2:, :1].contiguous()
    kc = y.view(1, 1, H * L, D)  # a cache of 2^31 elements and more
    at = H * L - 5
    swa.qk_rope_append(x[:, -2:].contiguous(), k, k, None, None, f.cuda(), kc, kc.clone(),
                       torch.tensor([at], dtype=torch.int32, device="cuda"), EPS)
    check_rows("k", kc[:, :, at - 2:at], *forward_ref(k.cpu(), None, 0.0, torch.tensor([[at - 2, at - 1]]), f, False))


@pytest.mark.gpu
def test_training_chain_matches_64_bits():
    """Projection output -> rotation -> shared-prefix attention -> its backward -> rotation's backward,
    against 64-bit autograd of the whole; the attention's bar (1e-2 in relative Frobenius norm) covers the
    bf16 roundings on the way."""
    import sliding_window_attention_gb300 as swa

    B, L, Hq, Hkv, D, W, prompt, chosen = 1, 300, 4, 2, 128, 90, 120, 100
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 31)
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    dO = torch.randn((B, Hq, L, D), generator=g).to(BF)
    f, scale = freqs(64), D ** -0.5
    pos = swa.prefix_positions(B, L, prompt, chosen, "cpu")
    assert pos[0, prompt + chosen] == prompt and pos[0, prompt + chosen - 1] == prompt + chosen - 1
    qd, kd, vd = dev_rows((q, k, v), 0)
    wqd, wkd, fd, pd, gd = cuda(wq, wk, f, pos, dO)
    qr, kr, vr = swa.qk_rope(qd, kd, vd, wqd, wkd, fd, EPS, positions=pd)
    o, lse = swa.forward(qr, kr, vr, W, scale, prefix=(prompt, chosen))
    dq, dk, dv = swa.backward(qr, kr, vr, o, lse, gd, W, scale, prefix=(prompt, chosen))
    d, dwq, dwk = swa.qk_rope_backward(qd, kd, wqd, wkd, fd, dq, dk, dv, EPS, positions=pd)

    x = [t.double().contiguous().requires_grad_() for t in (q, k, v, wq, wk)]

    def prep(t, w):
        n = t / (t.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        a = pos.double()[:, :, None, None] * f
        u, s = n[..., :64], n[..., 64:]
        return torch.cat((u * a.cos() - s * a.sin(), s * a.cos() + u * a.sin()), -1).transpose(1, 2)

    qq, kk = prep(x[0], x[3]), prep(x[1], x[4]).repeat_interleave(Hq // Hkv, 1)
    vv = x[2].transpose(1, 2).repeat_interleave(Hq // Hkv, 1)
    i, j = torch.arange(L)[:, None], torch.arange(L)[None]
    lp = pos[0].long()
    see = (j <= i) & ~((i >= prompt + chosen) & (j >= prompt) & (j < prompt + chosen)) & (lp[:, None] - lp[None] < W)
    ref = torch.softmax((qq @ kk.transpose(2, 3) * scale).masked_fill(~see, -math.inf), -1) @ vv
    ref.backward(dO.double())
    want = torch.cat([t.grad for t in x[:3]], 2)
    for name, a, b in (("o", o, ref.detach()), ("d", d, want), ("dwq", dwq, x[3].grad), ("dwk", dwk, x[4].grad)):
        rel = float((a.double().cpu() - b).norm() / b.norm())
        assert rel <= 1e-2, f"{name}: {rel:.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("has_k,has_v", [(True, True), (True, False), (False, True), (False, False)])
def test_both_marshalling_paths_give_the_same(has_k, has_v):
    """A call with numpy scalars is marshalled in Python, others in C++; a call with a stream runs there: equal
    bits, equal outputs left out."""
    import numpy as np

    import sliding_window_attention_gb300 as swa

    B, L, Hq, Hkv, D = 3, 5, 4, 2, 64
    (q, k, v), g = fused(B, L, Hq, Hkv, D, 41, 8)
    w, f, dq, dk, dv = cuda(1 + 0.2 * torch.randn(D, generator=g), freqs(16),
                            *(torch.randn((B, h, L, D), generator=g) for h in (Hq, Hkv, Hkv)))
    q, k, v = dev_rows((q, k, v), 8)
    k, v = k if has_k else None, v if has_v else None
    s = torch.cuda.Stream()
    n = torch.tensor([5, 9, 7], dtype=torch.int32, device="cuda")
    for kw in (dict(pos0=7, weight_offset=0.5, interleaved=True), dict(), dict(positions=torch.arange(
            15, dtype=torch.int32, device="cuda").view(3, 5))):
        kc = [torch.zeros((B, Hkv, 9, D), dtype=BF, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        ways = (kw, dict(kw, stream=s), dict(kw, pos0=np.int64(kw.get("pos0", 0))))
        calls = [swa.qk_rope(q, k, v, w, w, f, EPS, **x) for x in ways]
        appends = [swa.qk_rope_append(q, k, v, w, w, f, kc[2 * i] if has_k else None, kc[2 * i + 1] if has_v else None,
                                      n, EPS, **x) for i, x in enumerate(ways)]
        grads = [swa.qk_rope_backward(q, k, w, w, f, dq, dk if has_k else None, dv if has_v else None, EPS, **x)
                 for x in ways]
        torch.cuda.synchronize()
        for outs in (calls, grads):
            for other in outs[1:]:
                for a, b in zip(outs[0], other):
                    assert (a is None and b is None) or torch.equal(a, b)
        for i in (1, 2):
            assert torch.equal(appends[0], appends[i])
            assert torch.equal(kc[0], kc[2 * i]) and torch.equal(kc[1], kc[2 * i + 1])
        assert (calls[0][1] is not None) == has_k and (calls[0][2] is not None) == has_v


# --------------------------------------------------------------------------- refusals (no GPU)


def test_c_abi_refuses_bad_arguments():
    import ctypes

    import sliding_window_attention_gb300 as swa
    from sliding_window_attention_gb300 import build

    build.build()
    lib = swa.load()
    ok = dict(q=0x1000, k=0x2000, v=0x3000, qs=64, ks=64, vs=64, wq=0x4000, wk=0x5000, f=0x6000, pos=None, kv=None,
              qo=0x7000, ko=0x8000, vo=0x9000, B=1, Hq=1, Hkv=1, L=4, D=64, rows=4, rot=64, inter=0, pos0=0,
              eps=1e-6, off=0.0, stream=None)

    def fwd(**kw):
        return lib.swa_attn_qk_rope_fwd(*{**ok, **kw}.values())

    for name in ("q", "qo", "ko", "vo", "f"):
        assert fwd(**{name: None}) == -1, name
    for name in ("B", "Hq", "Hkv", "L"):
        assert fwd(**{name: 0}) == -2, name
    assert fwd(D=96) == -4
    for kw in (dict(rot=80), dict(rot=8), dict(rot=-16), dict(eps=0.0), dict(eps=float("nan")),
               dict(off=float("inf")), dict(qs=56), dict(ks=68), dict(vs=-64), dict(Hq=2)):
        assert fwd(**kw) == -17, kw
    assert fwd(rows=3) == -18 and fwd(rows=0, kv=0x4000) == -18
    assert fwd(B=2 ** 30, L=4) == -10
    for name in ("q", "k", "v", "qo", "ko", "vo"):
        assert fwd(**{name: 0x1008}) == -7, name
    assert fwd(wq=0x4002) == -7 and fwd(f=0x6004) == -7 and fwd(pos=0x6002) == -7 and fwd(kv=0x6001) == -7

    okb = dict(q=0x1000, k=0x2000, qs=64, ks=64, wq=0x4000, wk=0x5000, f=0x6000, pos=None, dq=0x7000, dk=0x8000,
               dv=0x9000, gq=0xa000, gk=0xb000, gv=0xc000, gqs=64, gks=64, gvs=64, dwq=0xd000, dwk=0xe000, B=1, Hq=1,
               Hkv=1, L=4, D=64, rot=64, inter=0, pos0=0, eps=1e-6, off=0.0, ws=0x10000, wsb=1 << 20, stream=None)

    def bwd(**kw):
        return lib.swa_attn_qk_rope_bwd(*{**okb, **kw}.values())

    for name in ("q", "dq", "gq", "dk", "gk", "gv", "f", "k"):
        assert bwd(**{name: None}) == -1, name
    assert bwd(gks=8) == -17 and bwd(rot=24) == -17 and bwd(D=32) == -4 and bwd(L=0) == -2
    assert bwd(B=2 ** 29, L=1) == -10  # 2^32 tokens once counted in groups of 8
    assert bwd(dq=0x7008) == -7 and bwd(ws=0x10010) == -7 and bwd(dwk=0xe001) == -7
    need = lib.swa_attn_qk_rope_bwd_workspace_bytes(1, 4, 64)
    assert need == 304 * 2 * 64 * 4 and bwd(wsb=need - 1) == -8 and bwd(ws=None) == -8
    assert lib.swa_attn_qk_rope_bwd_workspace_bytes(0, 4, 64) == 0
    assert lib.swa_attn_qk_rope_bwd_workspace_bytes(1, 1 << 20, 512) == 304 * 2 * 512 * 4
    assert ctypes.string_at(lib.swa_attn_strerror(-17)) != b"unknown error code"


def test_binding_refuses_host_tensors():
    import sliding_window_attention_gb300 as swa

    (q, k, v), _ = fused(1, 4, 2, 1, 64, 1)
    w, f = torch.ones(64), freqs(32)
    with pytest.raises(ValueError, match="current CUDA device"):
        swa.qk_rope(q, k, v, w, w, f, EPS)
    with pytest.raises(ValueError, match="current CUDA device"):
        swa.swa_attn_qk_rope_bwd(q, k, w, w, f, None, None, None, q, k, v, w, w, EPS)


@pytest.mark.gpu
def test_binding_refuses_wrong_layouts():
    import numpy as np

    import sliding_window_attention_gb300 as swa

    (q, k, v), _ = fused(2, 4, 2, 1, 64, 1)
    q, k, v = dev_rows((q, k, v), 0)
    w, f = torch.ones(64, device="cuda"), freqs(32).cuda()
    swa.qk_rope(q, k, v, w, w, f, EPS)
    for bad in (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=q.float()), dict(k=k[:, :2]),
                dict(q=q.expand(2, 4, 2, 64)[:, ::2]), dict(wq=w.double()), dict(wk=w[:32]), dict(f=f.float()),
                dict(f=f.cpu()), dict(v=v[..., :32]), dict(v=torch.cat((v, v), 2)),
                dict(positions=torch.zeros(2, 4, dtype=torch.int64, device="cuda")),
                dict(positions=torch.zeros(4, dtype=torch.int32, device="cuda"))):
        a = {**dict(q=q, k=k, v=v, wq=w, wk=w, f=f, positions=None), **bad}
        with pytest.raises(ValueError):
            swa.qk_rope(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["f"], EPS, positions=a["positions"])
    for kw in (dict(), dict(pos0=np.int64(0))):
        with pytest.raises(swa.SwaError):
            swa.qk_rope(q, k, v, w, w, freqs(36).cuda(), EPS, **kw)  # rot_dim 72 > D
        with pytest.raises(swa.SwaError):
            swa.qk_rope(q, k, v, w, w, f, 0.0, **kw)
        with pytest.raises(ValueError):
            swa.qk_rope_append(q, k, v, w, w, f, None, None, torch.ones(2, dtype=torch.int32, device="cuda"), EPS, **kw)
    for pos0 in (2 ** 31, -2 ** 31 - 1, 2 ** 80):
        with pytest.raises(ValueError, match="pos0 does not fit"):
            swa.qk_rope(q, k, v, w, w, f, EPS, pos0=pos0)
        with pytest.raises(ValueError, match="pos0 does not fit"):
            swa.qk_rope_backward(q, k, w, w, f, q.float().transpose(1, 2).contiguous(),
                                 k.float().transpose(1, 2).contiguous(), None, EPS, pos0=pos0)
    with pytest.raises(RuntimeError):  # a truth value that there is none of
        swa.qk_rope(q, k, v, w, w, f, EPS, interleaved=torch.zeros(2))


def test_append_refuses_missing_lengths():
    """Without lengths there are no rows to append to: refused on either marshalling path, before anything is looked at."""
    import numpy as np

    import sliding_window_attention_gb300 as swa

    (q, k, v), _ = fused(2, 1, 2, 1, 64, 1)
    c = torch.zeros((2, 1, 4, 64), dtype=BF)
    for pos0 in (0, np.int64(0)):
        with pytest.raises(ValueError, match="kv_len"):
            swa.qk_rope_append(q, k, v, None, None, freqs(32), c, c.clone(), None, EPS, pos0=pos0)


@pytest.mark.gpu
def test_append_without_lengths_leaves_the_caches():
    import numpy as np

    import sliding_window_attention_gb300 as swa

    (q, k, v), _ = fused(2, 1, 2, 1, 64, 1)
    q, k, v = dev_rows((q, k, v), 0)
    kc, vc = (torch.zeros((2, 1, 4, 64), dtype=BF, device="cuda") for _ in range(2))
    for kw in (dict(), dict(pos0=np.int64(0)), dict(stream=torch.cuda.Stream())):
        with pytest.raises(ValueError, match="kv_len"):
            swa.qk_rope_append(q, k, v, None, None, freqs(32).cuda(), kc, vc, None, EPS, **kw)
    torch.cuda.synchronize()
    assert not kc.any() and not vc.any()


@pytest.mark.gpu
def test_running_out_of_memory_keeps_its_type():
    """A call whose outputs do not fit raises what PyTorch's own allocations raise, on either marshalling path.  The
    allocator's limit for this process is what runs out, not the device's memory."""
    import numpy as np

    import sliding_window_attention_gb300 as swa

    q = torch.randn((1, 400000, 2, 64), device="cuda").to(BF)  # 102 MB, more than any piece that the allocator keeps
    dy = torch.zeros((1, 2, 400000, 64), device="cuda")
    f = freqs(32).cuda()
    many, cache = (torch.zeros((400000, 1, 1, 64), dtype=BF, device="cuda") for _ in range(2))
    n, prefix = torch.zeros(400000, dtype=torch.int32, device="cuda"), cache[:5].view(1, 5, 64)
    calls = [lambda **kw: swa.qk_rope(q, None, None, None, None, f, EPS, **kw),
             lambda **kw: swa.qk_rope_backward(q, None, None, None, f, dy, None, None, EPS, **kw),
             lambda pos0=0: swa.forward_shared(many, prefix, prefix, cache, cache, n, type(pos0)(0), 0.1)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(torch.cuda.current_device()).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    held = []
    try:
        with pytest.raises(torch.OutOfMemoryError):  # what earlier tests left in the allocator's pool
            while True:
                held.append(torch.empty(16 << 20, dtype=torch.uint8, device="cuda"))
        for call in calls:
            for pos0 in (0, np.int64(0)):
                with pytest.raises(torch.OutOfMemoryError):
                    call(pos0=pos0)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
        held.clear()
    assert calls[0]()[0].shape == (1, 2, 400000, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,Hq,Hkv,D", [(1, 2000, 8, 4, 128), (2, 500, 4, 2, 512), (1, 9000, 2, 1, 64)])
def test_adjacent_backwards_take_turns_in_one_workspace(B, L, Hq, Hkv, D):
    """Backwards of two inputs in turn, captured so that nothing lies between them, with one workspace: partial sums
    that were overwritten before they had been read would change the scales' gradients."""
    import sliding_window_attention_gb300 as swa

    calls, x = 12, []
    for i in range(2):
        (q, k, v), g = fused(B, L, Hq, Hkv, D, 60 + i)
        w = 1 + 0.2 * torch.randn(D, generator=g)
        dy = [torch.randn((B, h, L, D), generator=g) for h in (Hq, Hkv, Hkv)]
        q, k, _ = dev_rows((q, k, v), 0)
        x.append((q, k, *cuda(w, w, freqs(D // 2), *dy)))
    ws = torch.empty(swa.qk_rope_bwd_workspace_bytes(B, L, D), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((B, L, Hq + 2 * Hkv, D), dtype=BF, device="cuda").split((Hq, Hkv, Hkv), 2) +
            tuple(torch.empty((2, D), device="cuda")) for _ in range(calls)]

    def run_all(wait):
        for i in range(calls):
            swa.swa_attn_qk_rope_bwd(*x[i % 2], *outs[i], EPS, workspace=ws)
            if wait:
                torch.cuda.synchronize()

    run_all(True)
    want = [[t.clone() for t in o] for o in outs[:2]]
    assert not torch.equal(want[0][3], want[1][3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(False)
    for _ in range(5):
        for o in outs:
            for t in o:
                t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            for a, b in zip(o, want[i % 2]):
                assert torch.equal(a, b), i


@pytest.mark.gpu
@pytest.mark.parametrize("L,Hq,Hkv,D,W", [(1000, 8, 4, 512, 0), (1500, 4, 2, 256, 300), (2000, 8, 4, 128, 0)])
def test_attention_backward_then_rotation_backward(L, Hq, Hkv, D, W):
    """The rotation's backward right behind the attention's, whose dK/dV and dQ passes run side by side: it may read
    none of dq, dk, dv before both have ended.  Two inputs in turn, captured, in the same gradient buffers, so that
    what is read too early is the other input's.  Against the same calls waited for."""
    import sliding_window_attention_gb300 as swa

    calls, x, scale = 6, [], D ** -0.5
    f = freqs(D // 2).cuda()
    for i in range(2):
        (q, k, v), g = fused(1, L, Hq, Hkv, D, 70 + i)
        rows = dev_rows((q, k, v), 0)
        qr, kr, vr = swa.qk_rope(*rows, None, None, f, EPS)
        o, lse = swa.forward(qr, kr, vr, W, scale)
        x.append((rows, qr, kr, vr, o, lse, torch.randn((1, Hq, L, D), generator=g).to(BF).cuda()))
    w = torch.ones(D, device="cuda")
    dq, dk, dv = (torch.empty((1, h, L, D), device="cuda") for h in (Hq, Hkv, Hkv))
    ws = torch.empty(swa.bwd_workspace_bytes(1, Hq, Hkv, L, D, W), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(swa.qk_rope_bwd_workspace_bytes(1, L, D), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((1, L, Hq + 2 * Hkv, D), dtype=BF, device="cuda").split((Hq, Hkv, Hkv), 2) +
            tuple(torch.empty((2, D), device="cuda")) for _ in range(calls)]

    def run_all(wait):
        for i in range(calls):
            rows, *attn = x[i % 2]
            swa.swa_attn_bwd(*attn, dq, dk, dv, W, scale, workspace=ws)
            if wait:
                torch.cuda.synchronize()
            swa.swa_attn_qk_rope_bwd(rows[0], rows[1], w, w, f, dq, dk, dv, *outs[i], EPS, workspace=ws2)
            if wait:
                torch.cuda.synchronize()

    run_all(True)
    assert swa.swa_attn_get_status() == 0
    want = [[t.clone() for t in o] for o in outs[:2]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(False)
    for _ in range(4):
        for t in (dq, dk, dv):
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            for a, b in zip(o, want[i % 2]):
                assert torch.equal(a, b), i


@pytest.mark.gpu
@pytest.mark.parametrize("p", [1, 16384, 999983, 2 ** 31 - 1, -2 ** 31])
def test_angles_are_as_close_as_documented(p):
    """An angle is within 2^-25 of a turn and 2^-52 of the turns made.  Where the cosine crosses zero, bf16 shows it:
    for pairs (1, 0) turned to a quarter turn and at most 2^-22 more, the first element is r cos of at most 2^-19,
    whose half step is 2^-28 r.  (The reference's turns are exact fractions of the fp64 frequencies, with 2 pi to 60
    digits.)  r carries 2^-18 as elsewhere, and r (0.5 + eps)^(1/2) is 1 but for that."""
    from fractions import Fraction

    import sliding_window_attention_gb300 as swa

    D, pairs = 512, 256
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889")
    whole = [abs(p) * i // (8 * pairs) for i in range(pairs)]  # turns made, frequencies up to 2 pi / 8
    f = [float(two_pi * (m + Fraction(1, 4) + Fraction(i % 16, 1 << 26)) / abs(p)) for i, m in enumerate(whole)]
    x = torch.zeros((1, 1, 1, D), dtype=BF, device="cuda")
    x[..., :pairs] = 1
    y = swa.qk_rope(x, None, None, None, None, torch.tensor(f, dtype=torch.float64, device="cuda"), EPS,
                    positions=torch.tensor([[p]], dtype=torch.int32, device="cuda"))[0][0, 0, 0].double().cpu()
    r = (0.5 + EPS) ** -0.5
    for i in range(pairs):
        turns = p * Fraction(f[i]) / two_pi
        frac = turns - math.floor(turns)
        quarter = Fraction(1, 4) if p > 0 else Fraction(3, 4)
        ref = -r * math.sin(float(two_pi * (frac - quarter))) * (1 if p > 0 else -1)
        off = 2 * math.pi * (2.0 ** -25 + 2.0 ** -52 * abs(float(turns)))
        assert abs(ref) <= 2.0 ** -18 and abs(float(y[i]) - ref) <= (HALF_STEP + F32) * abs(ref) + 1.01 * r * off, i


def test_prefix_positions():
    """The rejected response starts behind the prompt again; what swa_attn_fwd_prefix refuses is refused."""
    import sliding_window_attention_gb300 as swa

    assert swa.prefix_positions(2, 7, 2, 3, "cpu").tolist() == [[0, 1, 2, 3, 4, 2, 3]] * 2
    assert swa.prefix_positions(1, 4, 0, 0, "cpu").tolist() == [[0, 1, 2, 3]]
    assert swa.prefix_positions(1, 4, 1, 3, "cpu").tolist() == [[0, 1, 2, 3]]
    for prompt, chosen in ((-5, 3), (2, -1), (5, 3)):
        with pytest.raises(ValueError, match="shared-prefix"):
            swa.prefix_positions(1, 7, prompt, chosen, "cpu")


@pytest.mark.gpu
def test_missing_gradients_are_named():
    """Keys without dk, or no dq: a ValueError, like every other refusal of the binding."""
    import sliding_window_attention_gb300 as swa

    (q, k, v), _ = fused(2, 4, 2, 1, 64, 1)
    q, k, _ = dev_rows((q, k, v), 0)
    dq = torch.zeros((2, 2, 4, 64), device="cuda")
    for grads, name in (((dq, None, None), "dk"), ((None, None, None), "dq")):
        with pytest.raises(ValueError, match=name + " is missing"):
            swa.qk_rope_backward(q, k, None, None, None, *grads, EPS)


def test_a_missing_tensor_is_named():
    from sliding_window_attention_gb300 import _native

    with pytest.raises(ValueError, match="dk is missing"):
        _native._check(-1, (("dk", None, torch.float32, (2, 3)),))
