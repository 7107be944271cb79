"""What is measured of the operators that stand around the norm path in a
DP-SGD-RC step: the embedding (lookup, per-sample norm of its gradient, its
clipped gradient), dropout from the library's Philox stream, and the linear map
with bias, activation, dropout and residual in its epilogue, with its gradient.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, with `own` set, through the library's
public entry points.  `exact` computes the same from the definition in 64 bits.

Tokens are drawn log-uniformly over the vocabulary (a token of rank r has a
probability near 1 / r, as words have), the trailing part of each sample is
padding (-1), and activations and gradients are Gaussian.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one new token for each of four sequences, as a decoding step looks them up
        {"name": "lookup 4 tokens", "op": "lookup", "dtype": "bf16", "B": 4, "T": 1, "V": 128256,
         "d": 2048, "pad": 0.0, "ids": "i64"},
        # a training batch of the 112-layer model: 4 samples of 4096 tokens
        {"name": "lookup 4x4096", "op": "lookup", "dtype": "bf16", "B": 4, "T": 4096,
         "V": 128256, "d": 2048, "pad": 0.05, "ids": "i64"},
        # the fp32 single-layer batch (4 samples of 128 tokens, width 64)
        {"name": "norm f32 4x128", "op": "norm", "dtype": "f32", "B": 4, "T": 128, "V": 1000,
         "d": 64, "pad": 0.1, "ids": "i64"},
        # per-sample norms of the embedding's gradient in the 112-layer model's step
        {"name": "norm 4x4096", "op": "norm", "dtype": "bf16", "B": 4, "T": 4096, "V": 128256,
         "d": 2048, "pad": 0.05, "ids": "i64"},
        # a small vocabulary and odd sizes in fp32, clipped
        {"name": "grad f32 3x1000 odd", "op": "grad", "dtype": "f32", "B": 3, "T": 1000,
         "V": 5003, "d": 321, "pad": 0.1, "ids": "i32", "clip": True},
        # the long-context batch (2 samples of 32768 tokens), clipped, all rows written
        {"name": "grad 2x32768", "op": "grad", "dtype": "bf16", "B": 2, "T": 32768, "V": 128256,
         "d": 2048, "pad": 0.05, "ids": "i64", "clip": True},
        # one piece of a tensor at an odd offset of the stream
        {"name": "dropout f32 odd piece", "op": "dropout", "dtype": "f32", "N": 100003,
         "first": 5, "p": 0.1, "residual": False},
        # a block's output of the q_proj batch (8 x 4096 tokens, width 2048) onto its residual
        {"name": "dropout 8x4096x2048", "op": "dropout", "dtype": "bf16", "N": 8 * 4096 * 2048,
         "first": 0, "p": 0.1, "residual": True},
        # single tokens of eight sequences through an up map
        {"name": "linear 8 tokens", "op": "linear", "dtype": "bf16", "M": 8, "K": 2048,
         "N": 8192, "act": "silu", "bias": False, "residual": False, "p": 0.0},
        # the down map of a training batch, dropped out onto the residual
        {"name": "linear 16384 down", "op": "linear", "dtype": "bf16", "M": 16384, "K": 8192,
         "N": 2048, "act": "none", "bias": True, "residual": True, "p": 0.1},
        # fp32, sizes that are multiples of no tile
        {"name": "linear_grad f32 odd", "op": "linear_grad", "dtype": "f32", "M": 1001, "K": 517,
         "N": 263, "act": "gelu", "bias": True, "p": 0.1},
        # the gradient of an up map with its activation for a training batch
        {"name": "linear_grad 16384 up", "op": "linear_grad", "dtype": "bf16", "M": 16384,
         "K": 2048, "N": 8192, "act": "silu", "bias": False, "p": 0.0},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["lookup", "norm", "grad", "dropout", "linear", "linear_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("lookup", "norm", "grad"):
        d = _spread(rng, 8, 8192)
        d = d if rng.random() < 0.4 else max(8, d // 8 * 8)
        V = _spread(rng, 16, 150000)
        V = max(16, min(V, (1 << 28) // d))
        N = _spread(rng, 1, max(1, min(65536, (1 << 27) // d)))
        B = min(N, _spread(rng, 1, 16))
        case = {"op": op, "dtype": dtype, "B": B, "T": max(1, N // B), "V": V, "d": d,
                "pad": round(rng.uniform(0.0, 0.3), 3), "ids": rng.choice(["i32", "i64"])}
        if op == "grad":
            case["clip"] = rng.random() < 0.7
        return case
    if op == "dropout":
        return {"op": op, "dtype": dtype, "N": _spread(rng, 1000, 1 << 26),
                "first": rng.choice([0, 0, _spread(rng, 1, 1 << 40)]),
                "p": round(rng.uniform(0.02, 0.6), 3), "residual": rng.random() < 0.5}
    # the product's cost is bounded by the largest listed case (fp32: by a sixteenth of it)
    most = 16384 * 8192 * 2048 // (16 if dtype == "f32" else 1)
    while True:
        M, K, N = _spread(rng, 1, 32768), _spread(rng, 16, 8192), _spread(rng, 16, 8192)
        if rng.random() < 0.6:
            K, N = max(16, K // 8 * 8), max(16, N // 8 * 8)
        if M * K * N <= most:
            break
    case = {"op": op, "dtype": dtype, "M": M, "K": K, "N": N,
            "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.6,
            "p": rng.choice([0.0, 0.0, round(rng.uniform(0.02, 0.5), 3)])}
    if op == "linear":
        case["residual"] = rng.random() < 0.5
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


def _tokens(case, seed):
    """[B][T] token ids, log-uniform over [0, V); the last `pad` of each sample is -1."""
    B, T, V = case["B"], case["T"], case["V"]
    u = torch.rand((B, T), generator=_gen(seed, 1), device="cuda", dtype=torch.float64)
    r = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    # ranks are scattered over the ids by an odd multiplier coprime to V
    mul = next(m for m in range(7919, 7919 + 2 * V + 2, 2) if math.gcd(m, V) == 1)
    t = (r * mul + 3) % V
    t[:, T - int(T * case["pad"]):] = -1
    return t.to(torch.int32 if case["ids"] == "i32" else torch.int64).contiguous()


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case, "seed": 1000003 * seed + 17, "step": seed % 1000}
    if op in ("lookup", "norm", "grad"):
        s["tokens"] = _tokens(case, seed)
        s["scale"] = math.sqrt(case["d"])
        if op == "lookup":
            s["W"] = _normal((case["V"], case["d"]), dt, seed, 2, 0.02)
        else:
            s["G"] = _normal((case["B"], case["T"], case["d"]), dt, seed, 2, 0.01)
        s["c"] = None
        if case.get("clip"):
            s["c"] = torch.rand(case["B"], generator=_gen(seed, 3), device="cuda").clamp_(0.05, 1.0)
    elif op == "dropout":
        s["x"] = _normal((case["N"],), dt, seed, 2)
        s["residual"] = _normal((case["N"],), dt, seed, 3) if case["residual"] else None
    else:
        M, K, N = case["M"], case["K"], case["N"]
        s["X"] = _normal((M, K), dt, seed, 2)
        s["W"] = _normal((N, K), dt, seed, 3, 1.0 / math.sqrt(K))
        if op == "linear":
            s["bias"] = _normal((N,), dt, seed, 4, 0.1) if case["bias"] else None
            s["residual"] = _normal((M, N), dt, seed, 5) if case["residual"] else None
        else:
            s["dY"] = _normal((M, N), dt, seed, 6, 0.01)
            s["Z"] = _normal((M, N), dt, seed, 7) if case["act"] != "none" else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _philox(j, step, seed):
    """Philox4x32-10 (Salmon et al., SC'11) of the counters (j, step) under the key seed:
    the four words of each block as int64."""
    m = 0xFFFFFFFF
    x0, x1 = j & m, (j >> 32) & m
    x2 = torch.full_like(j, step & m)
    x3 = torch.full_like(j, (step >> 32) & m)
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):
        p0, p1 = x0 * 0xD2511F53, x2 * 0xCD9E8D57  # low 64 bits of the products
        x0, x1, x2, x3 = ((p1 >> 32) & m) ^ x1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ x3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return x0, x1, x2, x3


def _threshold(p):
    return min(65536, int(math.floor(p * 65536.0 + 0.5)))


def _dropped(x, p, seed, step, first=0):
    """x (fp32) with element e zeroed where half (e & 7) of block e >> 3 is below
    p 2^16, and the rest scaled so that the mean is kept."""
    thr = _threshold(p)
    if thr == 0:
        return x
    n = x.numel()
    b0 = first >> 3
    j = torch.arange(b0, ((first + n - 1) >> 3) + 1, device=x.device, dtype=torch.int64)
    w = torch.stack(_philox(j, step, seed), 1)
    halves = torch.stack((w & 0xFFFF, w >> 16), 2).reshape(-1)
    keep = halves[first - 8 * b0: first - 8 * b0 + n] >= thr
    return torch.where(keep.view(x.shape), x * (65536.0 / max(1, 65536 - thr)), 0.0)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (
            1.0 + 3.0 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "lookup":
        t = s["tokens"].long()
        rows = s["W"][t.clamp(min=0)].float() * s["scale"]
        return {"out": torch.where((t >= 0)[..., None], rows, 0.0).to(dt)}
    if op in ("norm", "grad"):
        t, B, d, V = s["tokens"].long(), case["B"], case["d"], case["V"]
        g = torch.where((t >= 0)[..., None], s["G"].float() * s["scale"], 0.0)
        if op == "grad":
            if s["c"] is not None:
                g = g * s["c"].view(B, 1, 1)
            dW = torch.zeros((V, d), device=g.device)
            dW.index_add_(0, t.clamp(min=0).reshape(-1), g.reshape(-1, d))
            return {"dW": dW.to(dt)}
        # the rows of equal (sample, token) pairs are summed, then squared
        key, order = torch.sort((torch.arange(B, device=t.device)[:, None] * V
                                 + t.clamp(min=0)).reshape(-1))
        first = torch.cat([torch.ones_like(key[:1]), (key[1:] != key[:-1]).long()])
        run_of = torch.cumsum(first, 0) - 1
        sums = torch.zeros((key.numel(), d), device=g.device)
        sums.index_add_(0, run_of, g.reshape(-1, d)[order])
        sample = torch.zeros_like(key).scatter_(0, run_of, key // V)
        n = torch.zeros(B, device=g.device)
        n.index_add_(0, sample, (sums * sums).sum(1))
        return {"n": n}
    if op == "dropout":
        y = _dropped(s["x"].float(), case["p"], s["seed"], s["step"], case["first"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt)}
    if op == "linear":
        z = s["X"].float() @ s["W"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _dropped(_act(z, case["act"]), case["p"], s["seed"], s["step"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "z": z.to(dt) if case["act"] != "none" else None}
    dz = _dropped(s["dY"].float(), case["p"], s["seed"], s["step"])
    if case["act"] != "none":
        dz = dz * _act_slope(s["Z"].float(), case["act"])
    return {"dX": (dz @ s["W"].float()).to(dt), "dW": (dz.t() @ s["X"].float()).to(dt),
            "db": dz.sum(0).to(dt) if case["bias"] else None}


def _own(s):
    import randomized_norm_clipping_gb300 as rnc

    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "lookup":
        return {"out": rnc.dprc_embed_lookup(s["W"], s["tokens"], scale=s["scale"])}
    if op == "norm":
        plan = rnc.dprc_embed_plan(s["tokens"], case["V"])
        n = torch.empty(case["B"], device="cuda")
        return {"n": rnc.dprc_embed_norm(s["G"], plan, n, scale=s["scale"])}
    if op == "grad":
        plan = rnc.dprc_embed_plan(s["tokens"], case["V"])
        dW = torch.empty((case["V"], case["d"]), device="cuda", dtype=dt)
        return {"dW": rnc.dprc_embed_grad(s["G"], plan, dW, c=s["c"], scale=s["scale"])}
    if op == "dropout":
        return {"y": rnc.dprc_dropout(s["x"], case["p"], s["seed"], s["step"],
                                      residual=s["residual"], first_element=case["first"])}
    if op == "linear":
        z = (torch.empty((case["M"], case["N"]), device="cuda", dtype=dt)
             if case["act"] != "none" else None)
        y = rnc.dprc_linear(s["X"], s["W"], bias=s["bias"], act=case["act"], p=case["p"],
                            seed=s["seed"], step=s["step"], residual=s["residual"], Z=z)
        return {"y": y, "z": z}
    dX, dW = torch.empty_like(s["X"]), torch.empty_like(s["W"])
    db = torch.empty(case["N"], device="cuda", dtype=dt) if case["bias"] else None
    rnc.dprc_linear_grad(s["dY"], s["X"], s["W"], Z=s["Z"], act=case["act"], p=case["p"],
                         seed=s["seed"], step=s["step"], dX=dX, dW=dW, db=db)
    return {"dX": dX, "dW": dW, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _keep_exact(n, p, seed, step, first):
    """The factor of each element (0 or 1 / (1 - p)), from unsigned 64-bit words."""
    thr = _threshold(p)
    u = np.uint64
    m32, s32 = u(0xFFFFFFFF), u(32)
    j = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    ctr = [j & m32, j >> s32, np.full_like(j, step & 0xFFFFFFFF),
           np.full_like(j, (step >> 32) & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for r in range(10):
        a, b = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
        ka = u((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF)
        kb = u((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        ctr = [(b >> s32) ^ ctr[1] ^ ka, b & m32, (a >> s32) ^ ctr[3] ^ kb, a & m32]
    words = np.stack(ctr, axis=1).astype("<u4")
    halves = words.view("<u2").reshape(-1)[first % 8: first % 8 + n]
    f = np.where(halves < thr, 0.0, 65536.0 / max(1, 65536 - thr))
    return torch.from_numpy(f).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        t = s["tokens"].long().reshape(-1)
        out = torch.zeros((t.numel(), case["d"]), device="cuda", dtype=torch.float64)
        at = torch.nonzero(t >= 0).reshape(-1)
        out[at] = s["W"].index_select(0, t[at]).double().mul_(s["scale"])
        return {"out": out.view(case["B"], case["T"], case["d"])}
    if op in ("norm", "grad"):
        B, T, d, V = case["B"], case["T"], case["d"], case["V"]
        n = torch.zeros(B, device="cuda", dtype=torch.float64)
        dW = torch.zeros((V, d), device="cuda", dtype=torch.float64) if op == "grad" else None
        for i in range(B):
            t = s["tokens"][i].long()
            at = torch.nonzero(t >= 0).reshape(-1)
            ids, which = torch.unique(t[at], return_inverse=True)
            rows = torch.zeros((ids.numel(), d), device="cuda", dtype=torch.float64)
            rows.index_add_(0, which, s["G"][i, at].double())
            n[i] = rows.square().sum() * s["scale"] ** 2
            if dW is not None:
                dW[ids] += rows * (s["scale"] * (float(s["c"][i]) if s["c"] is not None else 1.0))
        return {"dW": dW} if op == "grad" else {"n": n}
    if op == "dropout":
        y = s["x"].double() * _keep_exact(case["N"], case["p"], s["seed"], s["step"], case["first"])
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    M, N = case["M"], case["N"]
    keep = None
    if case["p"] > 0:
        keep = _keep_exact(M * N, case["p"], s["seed"], s["step"], 0).view(M, N)
    W, X, act = s["W"].double(), s["X"].double(), case["act"]
    z = X @ W.t() if op == "linear" else (s["Z"].double() if act != "none" else None)
    if op == "linear" and s["bias"] is not None:
        z += s["bias"].double()
    cdf = slope = None
    if act == "relu":
        cdf, slope = (z > 0).double(), (z > 0).double()
    elif act == "gelu":  # 0.5 (1 + tanh u) = sigmoid(2 u)
        a = 2.0 * math.sqrt(2.0 / math.pi)
        cdf = torch.sigmoid(a * (z + 0.044715 * z ** 3))
        slope = cdf + z * cdf * (1.0 - cdf) * a * (1.0 + 0.134145 * z ** 2)
    elif act == "silu":
        cdf = torch.sigmoid(z)
        slope = cdf + z * cdf * (1.0 - cdf)
    if op == "linear":
        y = z if cdf is None else z * cdf
        y = y if keep is None else y * keep
        y = y if s["residual"] is None else y + s["residual"].double()
        return {"y": y, "z": z if act != "none" else None}
    dz = s["dY"].double()
    dz = dz if keep is None else dz * keep
    dz = dz if slope is None else dz * slope
    return {"dX": dz @ W, "dW": dz.t() @ X, "db": dz.sum(0) if case["bias"] else None}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _distinct(case, draws):
    """Expected number of distinct ids among `draws` log-uniform ones."""
    v = np.arange(case["V"], dtype=np.float64)
    q = np.log1p(1.0 / (v + 1.0)) / math.log(case["V"] + 1.0)
    return float(np.sum(-np.expm1(draws * np.log1p(-np.minimum(q, 1.0 - 1e-12)))))


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("lookup", "norm", "grad"):
        N, d = case["B"] * case["T"], case["d"]
        used = case["B"] * (case["T"] - int(case["T"] * case["pad"]))
        ids = N * (4 if case["ids"] == "i32" else 8)
        if op == "lookup":
            return {"bytes": ids + (_distinct(case, used) + N) * d * e, "flops": used * d}
        if op == "norm":
            return {"bytes": ids + used * d * e + 4 * case["B"], "flops": 3 * used * d}
        return {"bytes": ids + used * d * e + case["V"] * d * e, "flops": 2 * used * d}
    if op == "dropout":
        return {"bytes": case["N"] * e * (3 if case["residual"] else 2), "flops": 2 * case["N"]}
    M, K, N = case["M"], case["K"], case["N"]
    if op == "linear":
        outs = 1 + (case["act"] != "none")
        b = M * K + N * K + M * N * (outs + case["residual"]) + N * case["bias"]
        return {"bytes": b * e, "flops": 2 * M * K * N}
    b = 2 * M * K + 2 * N * K + M * N * (1 + (case["act"] != "none")) + N * case["bias"]
    return {"bytes": b * e, "flops": 4 * M * K * N}
