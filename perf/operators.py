"""What is measured of the operators beside the attention kernels, and their plain forms.

Three operators:

  rope      queries and keys of one projection normalised per head (RMS, learned scale), rotated by
            position and laid out [B, H, L, D] for the attention, values laid out with them; with
            "append" the keys and values of a generation step go into each request's cache instead
  rope_bwd  its backward: the attention's fp32 dq, dk, dv to the projection's bf16 gradient and the
            gradients of the two scales
  shared    attention of a generation step over a prefix that a whole batch shares (read once for
            all requests) and each request's own cache of its own length

`own` false: elementary torch operations in 32 bits (angles in 64).  `own` true: the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
THETA = 10000.0

# (Hq, Hkv) pairs and head dims of this repository's workloads, and two generic groupings
HEADS = ((2, 1), (8, 4), (32, 16), (32, 4), (8, 8), (16, 2))
MOST_ROPE = 30553 * 64 * 256      # elements of the largest listed forward
MOST_BWD = 16384 * 40 * 512       # of the largest listed backward
MOST_SHARED = 16384 * 4 * 512 + 64 * 4 * 1024 * 512  # cache elements of the largest listed shared case
MOST_PAIRS = 64 * 32 * 17408 * 512                   # and its products


def listed():
    return [
        # a training step's causal layer, 8,192 tokens, the whole head rotated
        {"name": "rope_l8192_d128", "op": "rope", "B": 1, "L": 8192, "Hq": 8, "Hkv": 4, "D": 128, "rot": 128,
         "interleaved": False, "pos0": 0, "rows": 0},
        # the long ragged step of the sliding layers, 30,553 tokens (no multiple of any tile)
        {"name": "rope_l30553_d256", "op": "rope", "B": 1, "L": 30553, "Hq": 32, "Hkv": 16, "D": 256, "rot": 256,
         "interleaved": False, "pos0": 0, "rows": 0},
        # one generation step of the global layer for a batch of 64: a quarter of the head rotated, far positions
        {"name": "append_b64_d512", "op": "rope", "B": 64, "L": 1, "Hq": 32, "Hkv": 4, "D": 512, "rot": 128,
         "interleaved": False, "pos0": 16384, "rows": 256},
        # the smallest step: four requests, latency alone
        {"name": "append_b4_d128", "op": "rope", "B": 4, "L": 1, "Hq": 8, "Hkv": 4, "D": 128, "rot": 128,
         "interleaved": True, "pos0": 1024, "rows": 64},
        # backward of the causal layer's training step
        {"name": "rope_bwd_l8192_d128", "op": "rope_bwd", "B": 1, "L": 8192, "Hq": 8, "Hkv": 4, "D": 128, "rot": 128,
         "interleaved": False, "pos0": 0},
        # backward of the global layer's training step
        {"name": "rope_bwd_l16384_d512", "op": "rope_bwd", "B": 1, "L": 16384, "Hq": 32, "Hkv": 4, "D": 512,
         "rot": 512, "interleaved": False, "pos0": 0},
        # backward of a small batch of odd length, neighbouring pairs rotated
        {"name": "rope_bwd_b2_l1001_d64", "op": "rope_bwd", "B": 2, "L": 1001, "Hq": 2, "Hkv": 1, "D": 64, "rot": 64,
         "interleaved": True, "pos0": 0},
        # four requests behind a short system prompt: latency
        {"name": "shared_b4_p1024_d128", "op": "shared", "B": 4, "Hq": 8, "Hkv": 4, "Lq": 1, "D": 128, "P": 1024,
         "rows": 64, "window": 0, "sinks": False},
        # a batch of 32 behind an 8,192-token document
        {"name": "shared_b32_p8192_d128", "op": "shared", "B": 32, "Hq": 8, "Hkv": 4, "Lq": 1, "D": 128, "P": 8192,
         "rows": 512, "window": 0, "sinks": False},
        # the global layer, 64 requests behind 16,384 tokens: 512 query rows for each kv head
        {"name": "shared_b64_p16384_d512", "op": "shared", "B": 64, "Hq": 32, "Hkv": 4, "Lq": 1, "D": 512, "P": 16384,
         "rows": 1024, "window": 0, "sinks": False},
        # the sliding layer: the window leaves each request the prefix's end and its own cache
        {"name": "shared_b32_p4096_d256_w1024", "op": "shared", "B": 32, "Hq": 32, "Hkv": 16, "Lq": 1, "D": 256,
         "P": 4096, "rows": 1024, "window": 1024, "sinks": False},
        # four drafted tokens a request checked at once, attention sinks, an odd prefix
        {"name": "shared_b16_q4_p5001_d64_sinks", "op": "shared", "B": 16, "Hq": 16, "Hkv": 2, "Lq": 4, "D": 64,
         "P": 5001, "rows": 300, "window": 0, "sinks": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope_bwd", "shared"))
    while True:
        hq, hkv = rng.choice(HEADS)
        d = rng.choice((64, 128, 256, 512))
        if op == "shared":
            c = {"op": op, "B": _log(rng, 1, 64), "Hq": hq, "Hkv": hkv, "Lq": rng.choice((1, 1, 1, 2, 4)), "D": d,
                 "P": _log(rng, 64, 32768), "rows": _log(rng, 8, 2048), "window": rng.choice((0, 0, 0, 1024, 333)),
                 "sinks": rng.random() < 0.25}
            kv = hkv * d * (c["P"] + c["B"] * c["rows"])
            pairs = c["B"] * hq * c["Lq"] * (c["P"] + c["rows"]) * d
            if kv <= MOST_SHARED and pairs <= MOST_PAIRS:
                return c
            continue
        step = op == "rope" and rng.random() < 0.3
        c = {"op": op, "B": _log(rng, 1, 64) if step else rng.choice((1, 1, 2, 3)),
             "L": rng.choice((1, 1, 2, 4)) if step else _log(rng, 16, 30553), "Hq": hq, "Hkv": hkv, "D": d,
             "rot": rng.choice([r for r in (32, 64, 96, 128, 256, 512) if r <= d]),
             "interleaved": rng.random() < 0.3, "pos0": _log(rng, 1, 1000000) - 1}
        if op == "rope":
            c["rows"] = rng.randrange(8, 200) if step else 0
        if c["B"] * c["L"] * (hq + 2 * hkv) * d <= (MOST_ROPE if op == "rope" else MOST_BWD):
            return c


def _lens(c):
    """Own lengths of a shared case's requests, spread evenly over Lq .. rows."""
    lo, hi = min(c["Lq"], c["rows"]), c["rows"]
    return [lo + (hi - lo) * (2 * b + 1) // (2 * c["B"]) for b in range(c["B"])]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape, mul=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, device=DEV, generator=gen, dtype=torch.float32).mul_(mul).to(dtype)

    c = case
    s = dict(c)
    if c["op"] == "shared":
        s["q"] = randn(c["B"], c["Hq"], c["Lq"], c["D"])
        s["kp"], s["vp"] = (randn(c["Hkv"], c["P"], c["D"]) for _ in range(2))
        s["ko"], s["vo"] = (randn(c["B"], c["Hkv"], c["rows"], c["D"]) for _ in range(2))
        order = torch.randperm(c["B"], device=DEV, generator=gen)
        s["len"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)[order].contiguous()
        s["sink"] = randn(c["Hq"], dtype=torch.float32) if c["sinks"] else None
        s["scale"] = 1.0 / math.sqrt(c["D"])
        return s
    B, L, hq, hkv, D = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"]
    qkv = randn(B, L, hq + 2 * hkv, D)  # one projection's output
    s["q"], s["k"], s["v"] = qkv.split((hq, hkv, hkv), dim=2)
    s["wq"], s["wk"] = (1.0 + randn(D, mul=0.1, dtype=torch.float32) for _ in range(2))
    n = c["rot"] // 2
    s["inv_freq"] = THETA ** (-torch.arange(n, device=DEV, dtype=torch.float64) / n)  # radians a position
    if c["op"] == "rope_bwd":
        s["dq"] = randn(B, hq, L, D, mul=0.1, dtype=torch.float32)
        s["dk"], s["dv"] = (randn(B, hkv, L, D, mul=0.1, dtype=torch.float32) for _ in range(2))
    elif c["rows"]:
        s["kc"], s["vc"] = (randn(B, hkv, c["rows"], D) for _ in range(2))
        s["len"] = torch.randint(L, c["rows"] + 1, (B,), device=DEV, generator=gen, dtype=torch.int32)
    return s


# --------------------------------------------------------------------------- plain forms


def _angles(s):
    """cos, sin fp32 [B or 1, L, 1, rot / 2] of the step's positions."""
    pos = torch.arange(s["L"], device=DEV, dtype=torch.float64)[None]
    pos = pos + s["pos0"]
    if s.get("rows"):
        pos = pos + (s["len"].double() - s["L"])[:, None]
    a = (pos[..., None] * s["inv_freq"])[:, :, None, :]
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, rot, interleaved):
    """Rotates the first rot of the last dimension's elements in pairs (i, i + rot / 2) or (2 i, 2 i + 1)."""
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2] = a * cos - b * sin
        out[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2] = a * cos - b * sin
        out[..., rot // 2:rot] = b * cos + a * sin
    return out


def _rope_plain(s):
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        return _rotate(x, cos, sin, s["rot"], s["interleaved"]).to(torch.bfloat16).transpose(1, 2).contiguous()

    qr, kr, vr = one(s["q"], s["wq"]), one(s["k"], s["wk"]), s["v"].transpose(1, 2).contiguous()
    if not s["rows"]:
        return qr, kr, vr
    b = torch.arange(s["B"], device=DEV)[:, None]
    row = (s["len"].long() - s["L"])[:, None] + torch.arange(s["L"], device=DEV)
    s["kc"][b, :, row] = kr.transpose(1, 2)
    s["vc"][b, :, row] = vr.transpose(1, 2)
    return qr, s["kc"], s["vc"]


def _rope_bwd_plain(s):
    cos, sin = _angles(s)

    def one(dy, x, w):
        dn = _rotate(dy.transpose(1, 2), cos, -sin, s["rot"], s["interleaved"])  # the rotation's transpose
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        dw = (dn * n).sum((0, 1, 2))
        dn = dn * w
        return r * (dn - n * (dn * n).mean(-1, keepdim=True)), dw

    dq, dwq = one(s["dq"], s["q"], s["wq"])
    dk, dwk = one(s["dk"], s["k"], s["wk"])
    return torch.cat((dq, dk, s["dv"].transpose(1, 2)), 2).to(torch.bfloat16), dwq, dwk


def _shared_plain(s):
    B, hq, Lq, D, P = s["B"], s["Hq"], s["Lq"], s["D"], s["P"]
    hkv, rows = s["Hkv"], s["rows"]
    M = hq // hkv * Lq  # query rows of one request and kv head
    q = s["q"].float().view(B, hkv, M, D)
    sp = q.transpose(0, 1).reshape(hkv, B * M, D) @ s["kp"].float().transpose(1, 2)
    sp = sp.view(hkv, B, M, P).transpose(0, 1) * s["scale"]
    so = q @ s["ko"].float().transpose(2, 3) * s["scale"]
    # row i of a request sits behind its own cache's last Lq keys
    pos = (P + s["len"].long() - Lq)[:, None] + torch.arange(Lq, device=DEV)  # [B, Lq]
    pos = pos.repeat(1, hq // hkv)[:, None, :, None]
    key = torch.arange(P + rows, device=DEV)
    see = key <= pos
    if s["window"]:
        see = see & (pos - key < s["window"])
    x = torch.cat((sp, so), 3).masked_fill(~see, -math.inf)
    m = x.amax(3, keepdim=True)
    if s["sink"] is not None:
        c = s["sink"].view(1, hkv, hq // hkv, 1).expand(B, hkv, hq // hkv, Lq).reshape(B, hkv, M, 1)
        m = torch.maximum(m, c)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    if s["sink"] is not None:
        l = l + torch.exp(c - m)
    o = (p[..., :P].transpose(0, 1).reshape(hkv, B * M, P) @ s["vp"].float()).view(hkv, B, M, D).transpose(0, 1)
    o = o + p[..., P:] @ s["vo"].float()
    return (o / l).to(torch.bfloat16).reshape(B, hq, Lq, D), (m + torch.log(l)).reshape(B, hq, Lq)


def run(state):
    s = state
    if own:
        import sliding_window_attention_gb300 as swa

        if s["op"] == "shared":
            return swa.forward_shared(s["q"], s["kp"], s["vp"], s["ko"], s["vo"], s["len"], s["window"], s["scale"],
                                      sinks=s["sink"])
        how = {"pos0": s["pos0"], "interleaved": s["interleaved"]}
        if s["op"] == "rope_bwd":
            return swa.qk_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["dq"], s["dk"], s["dv"],
                                        EPS, **how)
        if s["rows"]:
            qr = swa.qk_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["inv_freq"], s["kc"], s["vc"],
                                    s["len"], EPS, **how)
            return qr, s["kc"], s["vc"]
        return swa.qk_rope(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["inv_freq"], EPS, **how)
    return {"rope": _rope_plain, "rope_bwd": _rope_bwd_plain, "shared": _shared_plain}[s["op"]](s)


def work(case):
    c = case
    hq, hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] != "shared":
        rows = c["B"] * c["L"]
        if c["op"] == "rope":  # bf16 in, bf16 out
            return {"bytes": rows * (hq + 2 * hkv) * D * 4, "flops": rows * (hq + hkv) * D * 8}
        # fp32 dq, dk, dv and bf16 q, k in; bf16 out
        return {"bytes": rows * D * ((hq + 2 * hkv) * 6 + (hq + hkv) * 2), "flops": rows * (hq + hkv) * D * 14}
    W, P, Lq = c["window"], c["P"], c["Lq"]
    first, own_keys, pairs = P, 0, 0
    for n in _lens(c):
        for i in range(Lq):
            a = P + n - Lq + i
            pairs += max(0, a + 1 - (max(0, a - W + 1) if W else 0))
        lo = max(0, P + n - Lq - W + 1) if W else 0
        first = min(first, lo)
        own_keys += n - max(0, lo - P)
    keys = (P - first) + own_keys  # K and V rows, each kv head's read once
    io = c["B"] * hq * Lq * (4 * D + 4)
    return {"bytes": keys * hkv * D * 4 + io, "flops": 4 * D * hq * pairs}


# --------------------------------------------------------------------------- 64 bits, from the definitions


def _turned(x, s, sign):
    """Complex rotation of fp64 x [B, L, H, D] by sign * position * frequency."""
    B, L, H, D = x.shape
    n = s["rot"] // 2
    start = s["len"].double() - L if s.get("rows") else torch.zeros(B, dtype=torch.float64, device=x.device)
    pos = start[:, None] + s["pos0"] + torch.arange(L, device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(B, L, 1, n),
                       (sign * pos[:, :, None] * s["inv_freq"])[:, :, None, :])
    head, rest = x[..., :2 * n], x[..., 2 * n:]
    if s["interleaved"]:
        z = torch.view_as_complex(head.reshape(B, L, H, n, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(B, L, H, 2 * n)
    else:
        z = torch.complex(head[..., :n].contiguous(), head[..., n:].contiguous()) * turn
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, rest), -1)


def _exact_rope(s):
    def one(x, w):
        x = x.double()
        return _turned(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double(), s, 1.0).transpose(1, 2)

    qr, kr, vr = one(s["q"], s["wq"]), one(s["k"], s["wk"]), s["v"].double().transpose(1, 2)
    if not s["rows"]:
        return qr.contiguous(), kr.contiguous(), vr.contiguous()
    kc, vc = s["kc"].double(), s["vc"].double()
    for b, n in enumerate(s["len"].tolist()):
        kc[b, :, n - s["L"]:n] = kr[b]
        vc[b, :, n - s["L"]:n] = vr[b]
    return qr.contiguous(), kc, vc


def _exact_rope_bwd(s):
    def one(dy, x, w):
        x, w = x.double(), w.double()
        dn = _turned(dy.double().transpose(1, 2), s, -1.0)
        inv = 1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        dw = torch.einsum("blhd,blhd->d", dn, x * inv)
        dn = dn * w
        along = (dn * x).sum(-1, keepdim=True) * inv ** 3 / x.shape[-1]
        return dn * inv - x * along, dw

    dq, dwq = one(s["dq"], s["q"], s["wq"])
    dk, dwk = one(s["dk"], s["k"], s["wk"])
    return torch.cat((dq, dk, s["dv"].double().transpose(1, 2)), 2), dwq, dwk


def _exact_shared(s):
    B, hq, Lq, D, P = s["B"], s["Hq"], s["Lq"], s["D"], s["P"]
    G = hq // s["Hkv"]
    o = torch.zeros(B, hq, Lq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, hq, Lq, dtype=torch.float64, device=DEV)
    kp, vp = s["kp"].double(), s["vp"].double()
    for b, n in enumerate(s["len"].tolist()):
        k = torch.cat((kp, s["ko"][b, :, :n].double()), 1).repeat_interleave(G, 0)  # [Hq, P + n, D]
        v = torch.cat((vp, s["vo"][b, :, :n].double()), 1).repeat_interleave(G, 0)
        x = torch.einsum("hid,hjd->hij", s["q"][b].double(), k) * s["scale"]
        i = torch.arange(P + n - Lq, P + n, device=DEV)[:, None]
        j = torch.arange(P + n, device=DEV)[None]
        hide = (j > i) | ((i - j >= s["window"]) if s["window"] else torch.zeros_like(j > i))
        x[:, hide] = -math.inf
        if s["sink"] is not None:  # one more logit, which carries no value
            x = torch.cat((x, s["sink"].double().view(hq, 1, 1).expand(hq, Lq, 1)), 2)
        lse[b] = torch.logsumexp(x, 2)
        o[b] = torch.exp(x[..., :P + n] - lse[b][..., None]) @ v
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "rope_bwd": _exact_rope_bwd, "shared": _exact_shared}[s["op"]](s)
