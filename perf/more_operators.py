"""What is measured of the operators around a cache held in 8 bits, and their plain forms.

A cache keeps the keys and values of B requests as e4m3 codes [B, Hkv, rows, D] with one fp32 scale
for each block of 16, 32, 64 or 128 tokens of a head, [B, Hkv, ceil(rows / block)]: a value is its
code times its block's scale.  Scales are powers of two, so a block's scale can grow as tokens come
in and the codes that it has already only move their exponents.

  append  the keys and values of a step, or of a whole prompt, quantised and written behind what a
          request has; a block whose scale has to grow for them has its older codes written again
  read    rows of the cache as bf16, zeros behind each request's length
  attend  attention of a generation step over the 8-bit cache, each request with a length of its own

`own` false: elementary torch operations in 32 bits.  `own` true: the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
F8 = torch.float8_e4m3fn
TOP = 448.0      # the largest e4m3 value
LEAST = -64      # the smallest scale is 2^-64

# (Hq, Hkv) pairs and head dims of this repository's workloads, and two generic groupings
HEADS = ((2, 1), (8, 4), (32, 16), (32, 4), (8, 8), (16, 2))
MOST_APPEND = 30553 * 16 * 256          # elements of the largest listed append, of k alone
MOST_READ = 2 * 16384 * 4 * 512         # of the largest listed read
MOST_ATTEND = 32 * 4 * 16384 * 512      # of the largest listed cache
MOST_PAIRS = 32 * 32 * 16384 * 512      # and its products


def listed():
    return [
        # a prompt of the causal layer, 8,192 tokens into an empty cache
        {"name": "append_l8192_d128", "op": "append", "B": 1, "L": 8192, "Hkv": 4, "D": 128, "rows": 8192,
         "block": 64, "older": False},
        # the long ragged prompt of the sliding layers, behind what earlier turns left in the cache
        {"name": "append_l30553_d256", "op": "append", "B": 1, "L": 30553, "Hkv": 16, "D": 256, "rows": 30900,
         "block": 32, "older": True},
        # one generation step of the global layer for a batch of 64
        {"name": "append_b64_d512", "op": "append", "B": 64, "L": 1, "Hkv": 4, "D": 512, "rows": 256, "block": 64,
         "older": True},
        # four drafted tokens for each of 16 requests: latency alone
        {"name": "append_b16_q4_d64", "op": "append", "B": 16, "L": 4, "Hkv": 2, "D": 64, "rows": 300, "block": 16,
         "older": True},
        # a cache read back for a chunk of two long prompts of the global layer
        {"name": "read_b2_l16384_d512", "op": "read", "B": 2, "Hkv": 4, "D": 512, "rows": 16384, "block": 128},
        # eight short requests of odd length
        {"name": "read_b8_l1001_d128", "op": "read", "B": 8, "Hkv": 4, "D": 128, "rows": 1001, "block": 64},
        # the smallest step: four requests of up to 1,024 tokens, latency alone
        {"name": "attend_b4_l1024_d128", "op": "attend", "B": 4, "Hq": 8, "Hkv": 4, "Lq": 1, "D": 128, "rows": 1024,
         "window": 0, "sinks": False, "block": 64},
        # one long conversation: the cache split along its length over the whole GPU
        {"name": "attend_b1_l131072_d128", "op": "attend", "B": 1, "Hq": 8, "Hkv": 4, "Lq": 1, "D": 128,
         "rows": 131072, "window": 0, "sinks": False, "block": 128},
        # a full batch of the causal layer
        {"name": "attend_b64_l8192_d128", "op": "attend", "B": 64, "Hq": 8, "Hkv": 4, "Lq": 1, "D": 128,
         "rows": 8192, "window": 0, "sinks": False, "block": 64},
        # the global layer, 32 requests of up to 16,384 tokens
        {"name": "attend_b32_l16384_d512", "op": "attend", "B": 32, "Hq": 32, "Hkv": 4, "Lq": 1, "D": 512,
         "rows": 16384, "window": 0, "sinks": False, "block": 128},
        # the sliding layer: the window leaves the last 1,024 tokens of each request
        {"name": "attend_b32_d256_w1024", "op": "attend", "B": 32, "Hq": 32, "Hkv": 16, "Lq": 1, "D": 256,
         "rows": 4096, "window": 1024, "sinks": False, "block": 32},
        # four drafted tokens a request checked at once, attention sinks, an odd length: 32 query rows a kv head
        {"name": "attend_b16_q4_l5001_d64_sinks", "op": "attend", "B": 16, "Hq": 16, "Hkv": 2, "Lq": 4, "D": 64,
         "rows": 5001, "window": 0, "sinks": True, "block": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend"))
    while True:
        hq, hkv = rng.choice(HEADS)
        c = {"op": op, "Hkv": hkv, "D": rng.choice((64, 128, 256, 512)), "block": rng.choice((16, 32, 64, 128))}
        if op == "append":
            step = rng.random() < 0.5
            c["B"] = _log(rng, 1, 64) if step else rng.choice((1, 1, 2, 3))
            c["L"] = rng.choice((1, 1, 2, 4, 7)) if step else _log(rng, 16, 30553)
            c["older"] = step or rng.random() < 0.5
            c["rows"] = c["L"] + (rng.randrange(8, 400) if c["older"] else 0)
            if c["B"] * c["Hkv"] * c["rows"] * c["D"] <= MOST_APPEND:
                return c
        elif op == "read":
            c["B"], c["rows"] = _log(rng, 1, 32), _log(rng, 16, 32768)
            if c["B"] * hkv * c["rows"] * c["D"] <= MOST_READ:
                return c
        else:
            c.update(B=_log(rng, 1, 64), Hq=hq, Lq=rng.choice((1, 1, 1, 2, 4)), rows=_log(rng, 64, 131072),
                     window=rng.choice((0, 0, 0, 1024, 333)), sinks=rng.random() < 0.25)
            kv = c["B"] * hkv * c["rows"] * c["D"]
            if kv <= MOST_ATTEND and kv * (hq // hkv) * c["Lq"] <= MOST_PAIRS:
                return c


def _lens(c):
    """The requests' lengths, spread evenly over the cache's rows (an append's include its tokens)."""
    if c["op"] == "append":
        lo = c["L"] if c["older"] else c["rows"]
    else:
        lo = min(c.get("Lq", 1), c["rows"]) if c["B"] > 1 else c["rows"]
    hi = c["rows"]
    return [lo + (hi - lo) * (2 * b + 1) // (2 * c["B"]) for b in range(c["B"])]


def _two_to(amax):
    """The smallest power of two s >= 2^LEAST with amax <= 448 s, of fp32 or fp64 values, exactly."""
    m, e = torch.frexp(amax)  # amax = m 2^e, and 448 = 0.875 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), LEAST).clamp(min=LEAST)
    return torch.ldexp(torch.ones_like(amax), e)


def _filled(x, block):
    """Codes and scales of bf16 x [B, H, rows, D], quantised whole."""
    B, H, rows, D = x.shape
    nb = -(-rows // block)
    codes = torch.empty(B, H, rows, D, dtype=F8, device=DEV)
    scales = torch.empty(B, H, nb, dtype=torch.float32, device=DEV)
    for b in range(B):  # a request at a time: the fp32 copy stays small
        y = torch.zeros(H, nb * block, D, dtype=torch.float32, device=DEV)
        y[:, :rows] = x[b]
        s = _two_to(y.view(H, nb, block * D).abs().amax(2))
        codes[b] = (y.view(H, nb, block, D) / s[..., None, None]).view(H, nb * block, D)[:, :rows].to(F8)
        scales[b] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c = case
    s = dict(c)
    B, H, D, rows = c["B"], c["Hkv"], c["D"], c["rows"]

    def randn(*shape):
        return torch.randn(shape, device=DEV, generator=gen, dtype=torch.float32)

    # keys have channels that are larger throughout, values tokens that are
    channel = torch.exp(0.5 * randn(H, 1, D))

    def keys(n):
        return (randn(H, n, D) * channel).to(torch.bfloat16)

    def values(n):
        return (randn(H, n, D) * torch.exp(0.5 * randn(H, n, 1))).to(torch.bfloat16)

    s["k8"], s["ks"], s["v8"], s["vs"] = [], [], [], []
    for _ in range(B):
        for make, codes, scales in ((keys, "k8", "ks"), (values, "v8", "vs")):
            x, y = _filled(make(rows)[None], c["block"])
            s[codes].append(x)
            s[scales].append(y)
    for name in ("k8", "ks", "v8", "vs"):
        s[name] = torch.cat(s[name]) if B > 1 else s[name][0]
    order = torch.randperm(B, device=DEV, generator=gen)
    s["len"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)[order].contiguous()
    if c["op"] == "append":
        s["k"] = torch.stack([keys(c["L"]) for _ in range(B)])                               # [B, H, L, D]
        s["v"] = torch.stack([values(c["L"]) for _ in range(B)]).transpose(1, 2).contiguous()  # a projection's rows
        s["v"] = s["v"].transpose(1, 2)
    elif c["op"] == "attend":
        s["q"] = randn(B, c["Hq"], c["Lq"], D).to(torch.bfloat16)
        s["sink"] = randn(c["Hq"]) if c["sinks"] else None
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# --------------------------------------------------------------------------- plain forms


def _append_one(s, x, codes, scales):
    B, H, L, D = x.shape
    rows, block = s["rows"], s["block"]
    n = s["len"].long()
    first = (n - L) // block                   # the first block that gets a token
    nb = (L + block - 2) // block + 1          # blocks that may get one
    start = first * block
    # the blocks' tokens, old and new, beside one another: local row r is row start + r
    r = torch.arange(nb * block, device=x.device)
    row = start[:, None] + r                                        # [B, nb * block]
    new = (row >= (n - L)[:, None]) & (row < n[:, None]) & (row < rows)
    old = row < (n - L)[:, None]
    at = (row - (n - L)[:, None]).clamp(0, L - 1)[:, None, :, None].expand(B, H, nb * block, D)
    y = torch.gather(x, 2, at).float() * new[:, None, :, None]
    inside = row.clamp(max=rows - 1)[:, None, :, None].expand(B, H, nb * block, D)
    was = torch.gather(codes.view(torch.uint8), 2, inside).view(F8).float()
    blk = (first[:, None] + torch.arange(nb, device=x.device)).clamp(max=scales.shape[2] - 1)
    s_old = torch.gather(scales, 2, blk[:, None].expand(B, H, nb))
    has_old = old.view(B, 1, nb, block).any(3)
    amax = y.view(B, H, nb, block * D).abs().amax(3)
    sc = torch.where(has_old & (amax <= TOP * s_old), s_old, _two_to(amax))
    per = sc.repeat_interleave(block, 2)[..., None]
    z = torch.where(old[:, None, :, None], was * s_old.repeat_interleave(block, 2)[..., None], y) / per
    z = z.clamp(-TOP, TOP).to(F8).view(torch.uint8)
    # into the cache: row -> local row, where the call writes it
    all_rows = torch.arange(rows, device=x.device)
    local = all_rows - start[:, None]
    written = (local >= 0) & (all_rows < n[:, None])
    local = local.clamp(0, nb * block - 1)[:, None, :, None].expand(B, H, rows, D)
    c8 = codes.view(torch.uint8)
    c8.copy_(torch.where(written[:, None, :, None], torch.gather(z, 2, local), c8))
    every = torch.arange(scales.shape[2], device=x.device)
    lb = every - first[:, None]
    hit = (lb >= 0) & (every * block < n[:, None])
    scales.copy_(torch.where(hit[:, None], torch.gather(sc, 2, lb.clamp(0, nb - 1)[:, None].expand(B, H, -1)), scales))


def _append_plain(s):
    _append_one(s, s["k"], s["k8"], s["ks"])
    _append_one(s, s["v"], s["v8"], s["vs"])
    return s["k8"], s["v8"], s["ks"], s["vs"]


def _values(s, codes, scales):
    return codes.float() * scales.repeat_interleave(s["block"], 2)[:, :, :s["rows"], None]


def _read_plain(s):
    there = (torch.arange(s["rows"], device=DEV) < s["len"][:, None])[:, None, :, None]
    return tuple(torch.where(there, _values(s, s[c], s[x]), 0.0).to(torch.bfloat16)
                 for c, x in (("k8", "ks"), ("v8", "vs")))


def _attend_plain(s):
    B, hq, Lq, D = s["q"].shape
    hkv, rows = s["Hkv"], s["rows"]
    G = hq // hkv
    q = s["q"].float().view(B, hkv, G * Lq, D)
    x = q @ _values(s, s["k8"], s["ks"]).transpose(2, 3) * s["scale"]
    # row i of a request sits behind its cache's last Lq keys
    pos = (s["len"].long() - Lq)[:, None] + torch.arange(Lq, device=DEV)
    pos = pos.repeat(1, G)[:, None, :, None]
    key = torch.arange(rows, device=DEV)
    see = key <= pos
    if s["window"]:
        see = see & (pos - key < s["window"])
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(3, keepdim=True)
    if s["sink"] is not None:
        c = s["sink"].view(1, hkv, G, 1).expand(B, hkv, G, Lq).reshape(B, hkv, G * Lq, 1)
        m = torch.maximum(m, c)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    if s["sink"] is not None:
        l = l + torch.exp(c - m)
    o = p @ _values(s, s["v8"], s["vs"])
    return (o / l).to(torch.bfloat16).reshape(B, hq, Lq, D), (m + torch.log(l)).reshape(B, hq, Lq)


def run(state):
    s = state
    if own:
        import sliding_window_attention_gb300 as swa

        if s["op"] == "append":
            swa.cache8_append(s["k"], s["v"], s["k8"], s["v8"], s["ks"], s["vs"], s["len"], s["block"])
            return s["k8"], s["v8"], s["ks"], s["vs"]
        if s["op"] == "read":
            return swa.cache8_read(s["k8"], s["v8"], s["ks"], s["vs"], s["len"], s["block"])
        return swa.forward_cache8(s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["len"], s["block"], s["window"],
                                  s["scale"], sinks=s["sink"])
    return {"append": _append_plain, "read": _read_plain, "attend": _attend_plain}[s["op"]](s)


def work(case):
    c = case
    H, D, block = c["Hkv"], c["D"], c["block"]
    if c["op"] == "append":  # k and v: bf16 in, codes and their blocks' scales out
        n = c["B"] * c["L"]
        return {"bytes": 2 * n * H * D * 3 + 2 * 4 * c["B"] * H * -(-c["L"] // block), "flops": 2 * n * H * D * 3}
    if c["op"] == "read":  # k and v: codes and scales up to the lengths in, bf16 out
        keys, out = sum(_lens(c)), c["B"] * c["rows"]
        return {"bytes": 2 * H * (keys * D + 4 * keys // block + 2 * out * D), "flops": 2 * H * keys * D}
    W, Lq = c["window"], c["Lq"]
    keys, pairs = 0, 0
    for n in _lens(c):
        for i in range(Lq):
            a = n - Lq + i
            pairs += max(0, a + 1 - (max(0, a - W + 1) if W else 0))
        keys += n - (max(0, n - Lq - W + 1) if W else 0)
    io = c["B"] * c["Hq"] * Lq * (4 * D + 4)
    return {"bytes": 2 * H * (keys * D + 4 * keys // block) + io, "flops": 4 * D * c["Hq"] * pairs}


# --------------------------------------------------------------------------- 64 bits, from the definitions


def _round_e4m3(y):
    """fp64 values at most 448 in size to the nearest of 0, n 2^-9 (n < 8) and (8 + n) 2^(e - 3), e >= -6; ties to even."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _exact_append(s):
    outs = []
    for x, codes, scales in (("k", "k8", "ks"), ("v", "v8", "vs")):
        x, codes, scales = s[x].double(), s[codes].double(), s[scales].double()
        L, block, rows = x.shape[2], s["block"], s["rows"]
        for b, n in enumerate(s["len"].tolist()):
            for j in range((n - L) // block, -(-min(n, rows) // block)):
                lo, hi = j * block, min((j + 1) * block, n, rows)
                a = max(lo, n - L)  # the block's older tokens are rows lo .. a, its new ones a .. hi
                new = x[b, :, a - (n - L):hi - (n - L)]
                top = new.abs().amax((1, 2))
                was = scales[b, :, j].clone()
                now = torch.full_like(top, 2.0 ** LEAST)
                for _ in range(200):  # the least power of two that reaches
                    now = torch.where(top > TOP * now, now * 2, now)
                if a > lo:
                    now = torch.where(top <= TOP * was, was, now)
                    codes[b, :, lo:a] = _round_e4m3(codes[b, :, lo:a] * (was / now)[:, None, None])
                codes[b, :, a:hi] = _round_e4m3(new / now[:, None, None])
                scales[b, :, j] = now
        outs.append((codes, scales))
    (k, ks), (v, vs) = outs
    return k, v, ks, vs


def _exact_read(s):
    outs = []
    for codes, scales in (("k8", "ks"), ("v8", "vs")):
        y = torch.zeros(s[codes].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["len"].tolist()):
            block_of = torch.arange(n, device=DEV) // s["block"]
            y[b, :, :n] = s[codes][b, :, :n].double() * s[scales][b].double()[:, block_of, None]
        outs.append(y)
    return tuple(outs)


def _exact_attend(s):
    B, hq, Lq, D = s["q"].shape
    hkv, W = s["Hkv"], s["window"]
    G = hq // hkv
    o = torch.zeros(B, hq, Lq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, hq, Lq, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["len"].tolist()):
        block_of = torch.arange(n, device=DEV) // s["block"]
        i = torch.arange(n - Lq, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hide = (j > i) | (i - j >= W) if W else j > i
        for h in range(hkv):
            k = s["k8"][b, h, :n].double() * s["ks"][b, h].double()[block_of, None]
            v = s["v8"][b, h, :n].double() * s["vs"][b, h].double()[block_of, None]
            heads = slice(h * G, (h + 1) * G)
            x = torch.einsum("gid,jd->gij", s["q"][b, heads].double(), k) * s["scale"]
            x[:, hide] = -math.inf
            if s["sink"] is not None:  # one more logit, which carries no value
                x = torch.cat((x, s["sink"][heads].double().view(G, 1, 1).expand(G, Lq, 1)), 2)
            lse[b, heads] = torch.logsumexp(x, 2)
            o[b, heads] = torch.einsum("gij,jd->gid", torch.exp(x[..., :n] - lse[b, heads][..., None]), v)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[s["op"]](s)
