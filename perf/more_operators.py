"""What is measured of the operators of a transformer block that stand beside the
embedding, dropout and the linear map: layer and RMS normalisation (forward,
gradient, per-sample norms of its parameters' gradients), rotary positions with
one or several axes, and attention with capped scores, a bias by distance,
document and prefix masks (forward, gradient, few tokens over a cache).

`run` computes an operator in its plain form (elementary torch operations in 32
bits, in 64 for the angles of far positions, rounded once at the end) or, with
`own` set, through the library's public entry points.  `exact` computes the same
from the definition in 64 bits.

Activations and gradients are Gaussian; lengths of documents, prefixes and
caches are uneven and fixed by the case, their order is drawn.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # fp32 at sizes that are multiples of nothing
        {"name": "layernorm f32 3x1000x321", "op": "norm", "dtype": "f32", "B": 3, "T": 1000,
         "d": 321, "center": True, "bias": True},
        # one new token of each of four sequences, as a decoding step normalises them
        {"name": "rms norm 4 tokens", "op": "norm", "dtype": "bf16", "B": 4, "T": 1, "d": 2048,
         "center": False, "bias": False},
        # a training batch of the 112-layer model: input gradient, parameter gradients and
        # their per-sample norms
        {"name": "layernorm_grad 4x4096x2048", "op": "norm_grad", "dtype": "bf16", "B": 4,
         "T": 4096, "d": 2048, "center": True, "bias": True},
        # queries and keys of that batch, in place in the product's [q | k | v] rows
        {"name": "rotary 4x4096 40 heads", "op": "rotary", "dtype": "bf16", "B": 4, "T": 4096,
         "H": 40, "D": 64, "R": 64, "axes": 1, "interleaved": False, "inverse": False,
         "far": 100000},
        # the gradient's way back through positions of three axes (time, height, width)
        {"name": "rotary f32 3 axes inverse", "op": "rotary", "dtype": "f32", "B": 2, "T": 777,
         "H": 5, "D": 44, "R": 42, "axes": 3, "interleaved": True, "inverse": True, "far": 500},
        # four sequences that have just begun, one new token each
        {"name": "attention 4 tokens over 128", "op": "attend", "dtype": "bf16", "B": 4, "Tq": 1,
         "T": 128, "H": 32, "Hkv": 8, "D": 64, "mask": "cache", "cap": 0.0, "slopes": False},
        # one new token for each of eight long sequences (the long-context length)
        {"name": "attention 8 tokens over 32768", "op": "attend", "dtype": "bf16", "B": 8,
         "Tq": 1, "T": 32768, "H": 32, "Hkv": 8, "D": 64, "mask": "cache", "cap": 0.0,
         "slopes": False},
        # fp32, odd sizes, a bias by distance, packed documents with padding
        {"name": "attention f32 2x257 documents", "op": "attend", "dtype": "f32", "B": 2,
         "Tq": 257, "T": 257, "H": 6, "Hkv": 2, "D": 40, "mask": "documents", "cap": 0.0,
         "slopes": True},
        # a training batch of the 112-layer model (32 heads of 64, 8 of keys)
        {"name": "attention 4x4096", "op": "attend", "dtype": "bf16", "B": 4, "Tq": 4096,
         "T": 4096, "H": 32, "Hkv": 8, "D": 64, "mask": "causal", "cap": 0.0, "slopes": False},
        # a long sequence, the first third read as a prefix, capped scores, wide heads
        {"name": "attention 16384 capped prefix", "op": "attend", "dtype": "bf16", "B": 1,
         "Tq": 16384, "T": 16384, "H": 16, "Hkv": 4, "D": 128, "mask": "prefix", "cap": 20.0,
         "slopes": False},
        # the gradient in fp32 at odd sizes
        {"name": "attention_grad f32 2x300", "op": "attend_grad", "dtype": "f32", "B": 2,
         "Tq": 300, "T": 300, "H": 4, "Hkv": 2, "D": 33, "mask": "prefix", "cap": 10.0,
         "slopes": False},
        # the gradient of the training batch, packed documents, a bias by distance
        {"name": "attention_grad 4x4096 documents", "op": "attend_grad", "dtype": "bf16", "B": 4,
         "Tq": 4096, "T": 4096, "H": 32, "Hkv": 8, "D": 64, "mask": "documents", "cap": 0.0,
         "slopes": True},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "rotary", "attend", "attend", "attend_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        d = _spread(rng, 8, 16384)
        d = d if rng.random() < 0.4 else max(8, d // 8 * 8)
        rows = _spread(rng, 1, max(1, (1 << 25) // d))
        B = min(rows, _spread(rng, 1, 16))
        return {"op": op, "dtype": dtype, "B": B, "T": max(1, rows // B), "d": d,
                "center": rng.random() < 0.5, "bias": rng.random() < 0.5}
    if op == "rotary":
        D = rng.choice([16, 40, 64, 80, 96, 128, 2 * rng.randint(3, 64)])
        H = _spread(rng, 1, 48)
        rows = _spread(rng, 1, max(1, (1 << 25) // (D * H)))
        B = min(rows, _spread(rng, 1, 8))
        R = D if rng.random() < 0.6 else 2 * rng.randint(max(1, D // 8), D // 2)
        return {"op": op, "dtype": dtype, "B": B, "T": max(1, rows // B), "H": H, "D": D, "R": R,
                "axes": rng.choice([1, 1, 2, 3]) if R >= 6 else 1,
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.3,
                "far": _spread(rng, 1, 1 << 20)}
    while True:
        group = rng.choice([1, 2, 3, 4, 4, 7, 8])
        Hkv, B = _spread(rng, 1, 8), _spread(rng, 1, 8)
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 8 * rng.randint(2, 16)])
        if dtype == "f32" and rng.random() < 0.5:
            D = rng.randint(16, 128)
        mask = rng.choice(["causal", "documents", "documents", "prefix", "full", "cache"])
        if mask == "cache" and op == "attend_grad":
            continue
        T = _spread(rng, 16, 32768 if mask == "cache" else 8192)
        Tq = min(T, _spread(rng, 1, 16)) if mask == "cache" else T
        case = {"op": op, "dtype": dtype, "B": B, "Tq": Tq, "T": T, "H": Hkv * group,
                "Hkv": Hkv, "D": D, "mask": mask, "cap": rng.choice([0.0, 0.0, 15.0, 40.0]),
                "slopes": rng.random() < 0.3}
        # bounded by the largest listed cases (fp32: by a sixteenth of them)
        most = 4 * 32 * 4096 ** 2 if op == "attend_grad" else 16 * 16384 ** 2
        if B * Hkv * group * Tq * T <= most // (16 if dtype == "f32" else 1):
            return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + k)
    return g


def _normal(shape, dtype, seed, k, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed, k), device="cuda") * scale).to(dtype)


def _shares(total, parts):
    """`parts` uneven positive whole numbers that add up to total."""
    w = [1.0 + 3.0 * ((0.618034 * (i + 1)) % 1.0) for i in range(parts)]
    cut = [int(round(sum(w[:i]) / sum(w) * total)) for i in range(parts + 1)]
    return [b - a for a, b in zip(cut, cut[1:])]


def _documents(case):
    """(lengths of the documents of a sample, positions of padding behind them)."""
    T = case["T"]
    pad = T // 16
    return [n for n in _shares(T - pad, max(1, min(6, T // 8))) if n > 0], pad


def _lengths(case):
    """Keys in each sample's cache: from all of T down to near half of it."""
    B, T, Tq = case["B"], case["T"], case["Tq"]
    return [max(Tq, T - (T * i) // (2 * B)) for i in range(B)]


def _prefixes(case):
    B, T = case["B"], case["T"]
    return [(T * (i + 1)) // (B + 2) for i in range(B)]


def _cuda_i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _mask_inputs(case, seed):
    """docs [B][T], prefix [B], lengths [B], first [B], causal of a case."""
    rng = random.Random(seed * 7919 + 1)
    m = dict(docs=None, prefix=None, lengths=None, first=None, causal=case["mask"] != "full")
    if case["mask"] == "documents":
        rows = []
        for _ in range(case["B"]):
            lens, pad = _documents(case)
            rng.shuffle(lens)
            rows.append([i for i, n in enumerate(lens) for _ in range(n)] + [-1] * pad)
        m["docs"] = _cuda_i32(rows)
    elif case["mask"] == "prefix":
        p = _prefixes(case)
        rng.shuffle(p)
        m["prefix"] = _cuda_i32(p)
    elif case["mask"] == "cache":
        n = _lengths(case)
        rng.shuffle(n)
        m["lengths"] = _cuda_i32(n)
        m["first"] = _cuda_i32([x - case["Tq"] for x in n])
    return m


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        B, T, d = case["B"], case["T"], case["d"]
        s["X"] = _normal((B, T, d), dt, seed, 1, 1.5) + (0.5 if case["center"] else 0.0)
        s["w"] = (1.0 + _normal((d,), torch.float32, seed, 2, 0.2)).to(dt)
        s["b"] = _normal((d,), dt, seed, 3, 0.2) if case["bias"] else None
        if op == "norm_grad":
            s["dY"] = _normal((B, T, d), dt, seed, 4, 0.01)
            x = s["X"].double()
            mean = x.mean(-1, keepdim=True) if case["center"] else torch.zeros_like(x[..., :1])
            rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS).rsqrt()
            s["stats"] = torch.cat((mean, rstd), -1).float()  # what the forward pass left
        return s
    if op == "rotary":
        B, T, H, D = case["B"], case["T"], case["H"], case["D"]
        # [q | k | v] rows of a fused product; the values' heads behind are not turned
        s["qkv"] = _normal((B, T, H + 2, D), dt, seed, 1)
        a, P = case["axes"], case["R"] // 2
        off = torch.randint(0, case["far"], (B, 1, a), generator=_gen(seed, 2), device="cuda")
        pos = torch.arange(T, device="cuda").view(1, T, 1)
        if a > 1:  # frames of rows of cells
            w = max(1, int(math.sqrt(T)) // 2)
            pos = torch.cat((pos // (w * w), pos // w % w, pos % w), -1)[..., :a]
        s["pos"] = (pos + off).contiguous()
        s["sections"] = _shares(P, a)
        s["freqs"] = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
                                for n in s["sections"]]).cuda()
        return s
    B, Tq, T, H, Hkv, D = (case[k] for k in ("B", "Tq", "T", "H", "Hkv", "D"))
    gain = 2.0 if case["cap"] else 1.0  # (scores that the cap bends)
    if Tq == T:  # views of the rows [q | k | v] of one product
        rows = _normal((B, T, H + 2 * Hkv, D), dt, seed, 1, gain)
        s["Q"], s["K"], s["V"] = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
    else:
        s["Q"] = _normal((B, Tq, H, D), dt, seed, 1, gain)
        s["K"] = _normal((B, T, Hkv, D), dt, seed, 2)
        s["V"] = _normal((B, T, Hkv, D), dt, seed, 3)
    s["mask"] = _mask_inputs(case, seed)
    s["slopes"] = None
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    if op == "attend_grad":
        s["dO"] = _normal((B, Tq, H, D), dt, seed, 4, 0.01)
        o, s["lse"] = _plain_attention(s)  # what the forward pass left
        s["O"] = o.to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    x = s["X"].float()
    if case["center"]:
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return {"y": y.to(dt)}


def _plain_norm_grad(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    rstd = s["stats"][..., 1:]
    xh = (s["X"].float() - s["stats"][..., :1]) * rstd
    dy = s["dY"].float()
    g = dy * s["w"].float()
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - g.mean(-1, keepdim=True)
    dw, db = (dy * xh).sum(1), dy.sum(1)  # of each sample
    n = (dw * dw).sum(-1)
    if case["bias"]:
        n = n + (db * db).sum(-1)
    return {"dX": (dx * rstd).to(dt), "dW": dw.sum(0).to(dt),
            "db": db.sum(0).to(dt) if case["bias"] else None, "n": n}


def _plain_rotary(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    H, D, P = case["H"], case["D"], case["R"] // 2
    x = s["qkv"][:, :, :H].float()
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    angle = (s["pos"][..., axis].double() * s["freqs"])[:, :, None]
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()
    if case["inverse"]:
        sn = -sn
    if case["interleaved"]:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        turned = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return {"out": torch.cat((turned, x[..., 2 * P:]), -1).to(dt)}


def _scores(s):
    """The masked scores [B][key heads][heads of each][Tq][T], the tanh of the cap (or
    None), and the queries and keys they are made of."""
    case, mask = s["case"], s["mask"]
    B, Tq, T, H, Hkv, D = (case[k] for k in ("B", "Tq", "T", "H", "Hkv", "D"))
    q = s["Q"].float().view(B, Tq, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    k = s["K"].float().permute(0, 2, 1, 3)[:, :, None]
    z = q @ k.transpose(-1, -2) / math.sqrt(D)
    t = None
    if case["cap"]:
        t = torch.tanh(z / case["cap"])
        z = t * case["cap"]
    j = torch.arange(T, device="cuda")
    first = torch.full((B, 1), T - Tq, device="cuda")
    if mask["first"] is not None:
        first = mask["first"].long()[:, None]
    i = first + torch.arange(Tq, device="cuda")  # positions of the queries
    if s["slopes"] is not None:
        far = (i[:, :, None] - j).abs().float()
        z = z - s["slopes"].view(1, Hkv, -1, 1, 1) * far[:, None, None]
    see = (j <= i[:, :, None]) if mask["causal"] else torch.ones_like(j <= i[:, :, None])
    if mask["prefix"] is not None:
        see = see | (j < mask["prefix"].view(B, 1, 1))
    if mask["lengths"] is not None:
        see = see & (j < mask["lengths"].view(B, 1, 1))
    if mask["docs"] is not None:
        d = mask["docs"]
        see = see & (torch.gather(d, 1, i)[:, :, None] == d[:, None]) & (d[:, None] >= 0)
    return torch.where(see[:, None, None], z, -math.inf), t, q, k


def _plain_attention(s):
    case = s["case"]
    z = _scores(s)[0]
    m = z.amax(-1, keepdim=True)
    z = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    l = z.sum(-1, keepdim=True)
    o = z @ s["V"].float().permute(0, 2, 1, 3)[:, :, None] / torch.where(l == 0.0, 1.0, l)
    lse = (m + torch.log(l)).reshape(case["B"], case["H"], case["Tq"])
    return o.permute(0, 3, 1, 2, 4).reshape(s["Q"].shape), lse


def _plain_attention_grad(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    z, t, q, k = _scores(s)
    lse = s["lse"].view(*z.shape[:-1], 1)
    p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse))
    do, o = (s[x].float().view(q.shape[0], q.shape[3], *q.shape[1:3], -1).permute(0, 2, 3, 1, 4)
             for x in ("dO", "O"))
    dp = do @ s["V"].float().permute(0, 2, 3, 1)[:, :, None]
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) / math.sqrt(case["D"])
    if t is not None:
        ds = ds * (1.0 - t * t)
    dQ = (ds @ k).permute(0, 3, 1, 2, 4).reshape(s["Q"].shape)
    dK = (ds.transpose(-1, -2) @ q).sum(2).transpose(1, 2)
    dV = (p.transpose(-1, -2) @ do).sum(2).transpose(1, 2)
    return {"dQ": dQ.to(dt), "dK": dK.to(dt), "dV": dV.to(dt)}


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "rotary":
        return _plain_rotary(s)
    if op == "attend":
        return {"out": _plain_attention(s)[0].to(DTYPES[s["case"]["dtype"]])}
    return _plain_attention_grad(s)


def _own(s):
    import randomized_norm_clipping_gb300 as rnc

    case = s["case"]
    op = case["op"]
    if op == "norm":
        return {"y": rnc.dprc_layernorm(s["X"], s["w"], s["b"], eps=EPS, center=case["center"])}
    if op == "norm_grad":
        dX, dW = torch.empty_like(s["X"]), torch.empty_like(s["w"])
        db = torch.empty_like(s["b"]) if case["bias"] else None
        n = torch.empty(case["B"], device="cuda")
        rnc.dprc_layernorm_grad(s["dY"], s["X"], s["stats"], s["w"], center=case["center"], dX=dX,
                                dW=dW, db=db, n=n, norm_of_bias=case["bias"])
        return {"dX": dX, "dW": dW, "db": db, "n": n}
    if op == "rotary":
        return {"out": rnc.dprc_rotary(s["qkv"][:, :, :case["H"]], s["pos"], s["freqs"],
                                       sections=s["sections"], interleaved=case["interleaved"],
                                       inverse=case["inverse"])}
    kw = dict(cap=case["cap"], slopes=s["slopes"], **s["mask"])
    if op == "attend":
        return {"out": rnc.dprc_attention(s["Q"], s["K"], s["V"], **kw)}
    dQ, dK, dV = (torch.empty(s[k].shape, dtype=s[k].dtype, device="cuda") for k in "QKV")
    rnc.dprc_attention_grad(s["dO"], s["Q"], s["K"], s["V"], s["O"], s["lse"], dQ=dQ, dK=dK, dV=dV,
                            **kw)
    return {"dQ": dQ, "dK": dK, "dV": dV}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_norm(s, grad):
    case = s["case"]
    X, w = s["X"].double(), s["w"].double()
    mu = X.mean(2) if case["center"] else X.new_zeros(X.shape[:2])
    sd = torch.sqrt(((X - mu[..., None]) ** 2).sum(2) / case["d"] + EPS)
    hat = (X - mu[..., None]) / sd[..., None]
    if not grad:
        y = hat * w
        return {"y": y if s["b"] is None else y + s["b"].double()}
    dY = s["dY"].double()
    g = dY * w
    along = torch.einsum("btd,btd->bt", g, hat) / case["d"]
    rest = g.sum(2) / case["d"] if case["center"] else torch.zeros_like(along)
    each_w = torch.einsum("btd,btd->bd", dY, hat)
    each_b = dY.sum(1)
    n = each_w.square().sum(1) + (each_b.square().sum(1) if case["bias"] else 0.0)
    return {"dX": (g - rest[..., None] - hat * along[..., None]) / sd[..., None],
            "dW": each_w.sum(0), "db": each_b.sum(0) if case["bias"] else None, "n": n}


def _exact_rotary(s):
    """A pair as a complex number, turned by exp(i angle)."""
    case = s["case"]
    P = case["R"] // 2
    x = s["qkv"][:, :, :case["H"]].double()
    first = 0
    out = x.clone()
    for a, n in enumerate(s["sections"]):
        angle = s["pos"][..., a, None].double() * s["freqs"][first:first + n]
        turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, :, None]
        at = torch.arange(first, first + n, device="cuda")
        re, im = (2 * at, 2 * at + 1) if case["interleaved"] else (at, P + at)
        z = torch.complex(x[..., re], x[..., im]) * turn
        out[..., re], out[..., im] = z.real, z.imag
        first += n
    return {"out": out}


def _exact_attention(s, grad):
    case, m = s["case"], s["mask"]
    B, Tq, T, H, D = (case[k] for k in ("B", "Tq", "T", "H", "D"))
    G = H // case["Hkv"]
    out = torch.zeros(s["Q"].shape, device="cuda", dtype=torch.float64)
    dQ, dK, dV = ((torch.zeros(s[k].shape, device="cuda", dtype=torch.float64) for k in "QKV")
                  if grad else (None, None, None))
    cols = torch.arange(T, device="cuda")
    for b in range(B):
        start = int(m["first"][b]) if m["first"] is not None else T - Tq
        pos = torch.arange(start, start + Tq, device="cuda").view(-1, 1)
        hidden = cols > pos if m["causal"] else torch.zeros((Tq, T), dtype=torch.bool, device="cuda")
        if m["prefix"] is not None:
            hidden[:, :int(m["prefix"][b])] = False
        if m["lengths"] is not None:
            hidden[:, int(m["lengths"][b]):] = True
        if m["docs"] is not None:
            doc = m["docs"][b].long()
            hidden |= (doc[pos] != doc.view(1, -1)) | (doc.view(1, -1) < 0)
        some = ~hidden.all(1, keepdim=True)
        for h in range(H):
            q, k, v = s["Q"][b, :, h].double(), s["K"][b, :, h // G].double(), s["V"][b, :, h // G].double()
            score = torch.mm(q, k.t()).mul_(D ** -0.5)
            slope = None
            if case["cap"]:
                score = torch.tanh(score.div_(case["cap"]))
                slope = 1.0 - score.square() if grad else None
                score.mul_(case["cap"])
            if s["slopes"] is not None:
                score -= float(s["slopes"][h]) * (pos - cols).abs()
            score.masked_fill_(hidden, -math.inf)
            # rows that see nothing have weights of zero
            w = torch.nan_to_num_(torch.softmax(score, 1), nan=0.0) * some
            o = w @ v
            out[b, :, h] = o
            if grad:
                do = s["dO"][b, :, h].double()
                dw = do @ v.t()
                dz = w * (dw - (do * o).sum(1, keepdim=True)) * D ** -0.5
                if slope is not None:
                    dz *= slope
                dQ[b, :, h] = dz @ k
                dK[b, :, h // G] += dz.t() @ q
                dV[b, :, h // G] += w.t() @ do
    return {"dQ": dQ, "dK": dK, "dV": dV} if grad else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, op == "norm_grad")
    if op == "rotary":
        return _exact_rotary(s)
    return _exact_attention(s, op == "attend_grad")


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _pairs(case):
    """Pairs of a query and a key that it sees, over the batch, of one head."""
    B, Tq, T = case["B"], case["Tq"], case["T"]
    if case["mask"] == "full":
        return B * T * T
    if case["mask"] == "causal":
        return B * T * (T + 1) // 2
    if case["mask"] == "documents":
        return B * sum(n * (n + 1) // 2 for n in _documents(case)[0])
    if case["mask"] == "prefix":
        return sum(p * p + (T * (T + 1) - p * (p + 1)) // 2 for p in _prefixes(case))
    return sum(Tq * n - Tq * (Tq - 1) // 2 for n in _lengths(case))


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        N, d = case["B"] * case["T"] * case["d"], case["d"]
        if op == "norm":
            return {"bytes": (2 * N + d * (1 + case["bias"])) * e, "flops": 6 * N}
        return {"bytes": (3 * N + d * (2 + case["bias"])) * e + 8 * case["B"] * case["T"]
                + 4 * case["B"], "flops": 12 * N}
    if op == "rotary":
        N = case["B"] * case["T"]
        return {"bytes": 2 * N * case["H"] * case["D"] * e + 8 * N * case["axes"]
                + 8 * case["R"] // 2, "flops": 3 * N * case["H"] * case["R"]}
    B, Tq, T, H, Hkv, D = (case[k] for k in ("B", "Tq", "T", "H", "Hkv", "D"))
    keys = sum(_lengths(case)) if case["mask"] == "cache" else B * T
    q, kv = B * Tq * H * D, keys * Hkv * D
    flops = 4 * _pairs(case) * H * D
    if op == "attend":
        return {"bytes": (2 * q + 2 * kv) * e, "flops": flops}
    return {"bytes": (4 * q + 4 * kv) * e + 4 * B * H * Tq, "flops": flops * 5 // 2}
