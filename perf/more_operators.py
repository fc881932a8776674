"""Cases of what lies between the products of a fine-tuning step: the norm of
a layer's input (forward, backward with the gains' gradients), rotary
positions, and the log probabilities of given tokens with entropy, top
alternatives and their gradient.

``run`` computes a case with elementary torch operations, or with the
library's calls where ``own`` is set.  Widths are those of the 7B-shaped
layer (4096; 32 heads of 128; 32000 tokens), or generic ones.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
BASE = 10000.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "bf16": 2}


def listed():
    return [
        # a generated token: residual addition and norm before a layer
        _norm("norm one token", 1, 4096, "rms", "bf16", res=True),
        # a training step: residual addition and layer norm with bias
        _norm("norm training", 4096, 4096, "layer", "bf16", res=True, bias=True),
        # its backward pass, the gradient of the residual path added
        _norm("norm grad training", 4096, 4096, "rms", "bf16", grad=True, res=True),
        # a short batch of an odd width, everything in fp32
        _norm("norm grad ragged", 517, 1375, "layer", "f32", grad=True, bias=True),
        # a generated token's queries and keys, far into a long context
        _rotary("rotary one token", 1, 1, 32, 8, 128, 128, "half", "bf16", far=True),
        # queries and keys of a training step
        _rotary("rotary training", 2, 2048, 32, 32, 128, 128, "half", "bf16"),
        # gradients through a rotation of part of the head, out of a wider buffer
        _rotary("rotary grad ragged", 3, 171, 12, 4, 80, 20, "pairs", "f32", grad=True, packed=True, far=True),
        # one new token of each of 8 answers, with its 20 likeliest alternatives
        _logprob("logprob one token", 8, 32000, "bf16", top=20, entropy=True),
        # the loss of a training step
        _logprob("logprob training", 4096, 32000, "bf16", entropy=True, skip=0.1),
        # scoring of a short batch: a masked vocabulary of odd size, five alternatives each
        _logprob("logprob alternatives", 1003, 50001, "f32", top=5, entropy=True, masked=0.4, scale=1.25),
        # the gradient of a training step's loss
        _logprob("logprob grad training", 4096, 32000, "bf16", grad=True, skip=0.1),
        # the gradient of a loss with an entropy term
        _logprob("logprob grad ragged", 517, 33001, "f32", grad=True, entropy=True, masked=0.2, scale=0.8),
    ]


def _named(name, c):
    return {**c, "name": name} if name else c


def _norm(name, tokens, cols, kind, dtype, grad=False, res=False, bias=False, gain="f32", pad=0):
    return _named(name, {"op": "norm grad" if grad else "norm", "tokens": tokens, "cols": cols, "kind": kind,
                         "dtype": dtype, "res": res, "bias": bias, "gain": gain, "pad": pad})


def _rotary(name, batch, tokens, heads, kv, dim, rot, layout, dtype, grad=False, packed=False, far=False):
    return _named(name, {"op": "rotary", "batch": batch, "tokens": tokens, "heads": heads, "kv": kv, "dim": dim,
                         "rot": rot, "layout": layout, "dtype": dtype, "grad": grad, "packed": packed, "far": far})


def _logprob(name, tokens, vocab, dtype, grad=False, top=0, entropy=False, skip=0.0, masked=0.0, scale=1.0, pad=0):
    return _named(name, {"op": "logprob grad" if grad else "logprob", "tokens": tokens, "vocab": vocab,
                         "dtype": dtype, "top": top, "entropy": entropy, "skip": skip, "masked": masked,
                         "scale": scale, "pad": pad})


def draw(rng):
    def size(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    def flag(p=0.5):
        return rng.random() < p

    op = rng.choice(["norm", "norm grad", "rotary", "logprob", "logprob grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm grad"):
        cols = size(1, 2048) * 8 if flag() else size(1, 16384)
        tokens = min(size(1, 16384), max(1, (1 << 25) // (cols * WIDTH[dtype])))
        return _norm(None, tokens, cols, rng.choice(["rms", "layer"]), dtype, op == "norm grad", flag(), flag(),
                     rng.choice(["f32", "bf16"]), rng.choice([0, 0, 8, 5]))
    if op == "rotary":
        dim = rng.choice([32, 64, 80, 96, 128, 256, 2 * rng.randint(4, 128)])
        rot = dim if flag() else 2 * rng.randint(1, dim // 2)
        kv = size(1, 32)
        heads = kv * rng.choice([1, 2, 4, 8])
        batch, most = size(1, 16), (1 << 26) // (WIDTH[dtype] * (heads + kv) * dim)
        tokens = min(size(1, 4096), max(1, most // batch))
        return _rotary(None, batch, tokens, heads, kv, dim, rot, rng.choice(["half", "pairs"]), dtype, flag(), flag(),
                       flag())
    vocab = size(100, 150000)
    top = 0 if op == "logprob grad" or flag() else rng.randint(1, 32)
    most = (1 << 26) // (WIDTH[dtype] * (4 if top else 1))
    tokens = min(size(1, 8192), max(1, most // vocab))
    return _logprob(None, tokens, vocab, dtype, op == "logprob grad", top, flag(), rng.choice([0.0, 0.3]),
                    rng.choice([0.0, 0.5]), rng.choice([1.0, round(0.5 + rng.random(), 3)]), rng.choice([0, 0, 7]))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(mean, std, generator=gen).to(dtype)

    def uniform(shape):
        return torch.rand(shape, generator=gen, device=DEV)

    s = {"case": case}
    if case["op"] in ("norm", "norm grad"):
        T, C, pad = case["tokens"], case["cols"], case["pad"]

        def rows(std, mean=0.0):
            return normal((T, C + pad), std, mean, dtype)[:, :C]

        s["X"] = rows(1.5, 0.3)
        s["gain"] = normal((C,), 0.2, 1.0, DTYPES[case["gain"]])
        s["bias"] = normal((C,), 0.2, 0.0, DTYPES[case["gain"]]) if case["bias"] else None
        if case["op"] == "norm":
            s["res"] = rows(2.0) if case["res"] else None
            s["H"] = torch.empty((T, C), dtype=dtype, device=DEV) if case["res"] else None
            s["Y"] = torch.empty((T, C), dtype=dtype, device=DEV)
            s["mean"] = torch.empty(T, device=DEV) if case["kind"] == "layer" else None
            s["rstd"] = torch.empty(T, device=DEV)
            return s
        # what the forward pass left
        x = s["X"].double()
        mean = x.mean(1) if case["kind"] == "layer" else torch.zeros(T, dtype=torch.float64, device=DEV)
        s["mean"] = mean.float() if case["kind"] == "layer" else None
        s["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["dY"] = rows(0.01)
        s["dH"] = rows(0.01) if case["res"] else None
        s["dX"] = torch.empty((T, C), dtype=dtype, device=DEV)
        s["dgain"] = torch.empty(C, device=DEV)
        s["dbias"] = torch.empty(C, device=DEV) if case["bias"] else None
        return s
    if case["op"] == "rotary":
        B, T, H, K, D = case["batch"], case["tokens"], case["heads"], case["kv"], case["dim"]
        if case["packed"]:       # queries, keys and values of a token beside one another
            whole = normal((B, T, H + 2 * K, D), 1.0, 0.0, dtype)
            s["q"], s["k"] = whole[:, :, :H], whole[:, :, H:H + K]
        else:
            s["q"], s["k"] = normal((B, T, H, D), 1.0, 0.0, dtype), normal((B, T, K, D), 1.0, 0.0, dtype)
        s["q_out"], s["k_out"] = (torch.empty(x.shape, dtype=dtype, device=DEV) for x in (s["q"], s["k"]))
        start = torch.randint(0, 200_000 if case["far"] else 1, (B, 1), generator=gen, device=DEV)
        s["pos"] = (start + torch.arange(T, device=DEV)).int()
        freq = BASE ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"])
        if case["far"]:          # a context 32 times the one trained on: slow turns are slowed, fast ones kept
            keep = np.clip((8192 * freq / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
            freq = freq * (keep + (1.0 - keep) / 32.0)
        s["freq"] = torch.from_numpy(freq).to(DEV)
        s["amplitude"] = 1.25 if case["far"] else 1.0
        return s
    N, V, pad = case["tokens"], case["vocab"], case["pad"]
    target = torch.randint(0, V, (N,), generator=gen, device=DEV)
    z = normal((N, V + pad), 2.5)[:, :V]
    if case["masked"]:
        z.masked_fill_(uniform((N, V)) < case["masked"], -math.inf)
    row = torch.arange(N, device=DEV)
    z[row, target] = 6.0 + 3.0 * normal((N,))
    s["Z"] = z.to(dtype) if dtype != torch.float32 else z
    if pad and dtype != torch.float32:
        s["Z"] = torch.nn.functional.pad(s["Z"], (0, pad))[:, :V]
    s["target"] = torch.where(uniform((N,)) < case["skip"], -1, target).int()
    if case["op"] == "logprob":
        s["logp"] = torch.empty(N, device=DEV)
        s["stats"] = torch.empty((N, 2), device=DEV)
        s["entropy"] = torch.empty(N, device=DEV) if case["entropy"] else None
        s["top_logp"] = torch.empty((N, case["top"]), device=DEV) if case["top"] else None
        s["top_index"] = torch.empty((N, case["top"]), dtype=torch.int32, device=DEV) if case["top"] else None
        return s
    # what the forward pass left
    s["stats"], s["entropy"] = torch.empty((N, 2), device=DEV), torch.empty(N, device=DEV)
    for at in range(0, N, 512):
        d = s["Z"][at:at + 512].double()
        top = d.amax(1)
        d = (d - top[:, None]) * case["scale"]
        e = d.exp()
        total = e.sum(1)
        s["stats"][at:at + 512] = torch.stack([top, total.log()], 1)
        s["entropy"][at:at + 512] = total.log() - (e * d.clamp_min(-1000.0)).sum(1) / total
    s["dlogp"] = -(0.5 + uniform((N,))) / N
    s["dentropy"] = 0.3 * uniform((N,)) / N if case["entropy"] else None
    s["dZ"] = torch.empty((N, V), dtype=dtype, device=DEV)
    return s


# ---- the plain forms
def _plain_norm(s):
    case = s["case"]
    x = s["X"].float()
    if case["res"]:
        s["H"].copy_(x + s["res"].float())
        x = s["H"].float()
    mean = x.mean(1, keepdim=True) if case["kind"] == "layer" else 0.0
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd * s["gain"].float()
    if case["bias"]:
        y = y + s["bias"].float()
    s["Y"].copy_(y)
    s["rstd"].copy_(rstd[:, 0])
    if case["kind"] == "layer":
        s["mean"].copy_(mean[:, 0])
    return _normed(s)


def _normed(s):
    return {k: s[k] for k in ("Y", "H", "mean", "rstd")}


def _plain_norm_grad(s):
    case = s["case"]
    x, dy, rstd = s["X"].float(), s["dY"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None] if case["kind"] == "layer" else x) * rstd
    g = dy * s["gain"].float()
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if case["res"]:
        dx = dx + s["dH"].float()
    s["dX"].copy_(dx)
    s["dgain"].copy_((dy * xhat).sum(0))
    if case["bias"]:
        s["dbias"].copy_(dy.sum(0))
    return _norm_grads(s)


def _norm_grads(s):
    return {k: s[k] for k in ("dX", "dgain", "dbias")}


def _plain_rotary(s):
    case, rot = s["case"], s["case"]["rot"]
    angle = s["pos"].double()[..., None] * s["freq"]
    if case["grad"]:
        angle = -angle
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, :, None] for f in (torch.cos, torch.sin))
    for name in ("q", "k"):
        x, y = s[name].float(), s[name + "_out"]
        if case["layout"] == "half":
            a, b = slice(0, rot // 2), slice(rot // 2, rot)
        else:
            a, b = slice(0, rot, 2), slice(1, rot, 2)
        y[..., a] = (x[..., a] * cos - x[..., b] * sin).to(y.dtype)
        y[..., b] = (x[..., a] * sin + x[..., b] * cos).to(y.dtype)
        if rot < case["dim"]:
            y[..., rot:] = s[name][..., rot:]
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_logprob(s):
    case, scale = s["case"], s["case"]["scale"]
    z = s["Z"].float()
    top = z.amax(1, keepdim=True)
    d = (z - top) * scale
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    s["stats"].copy_(torch.cat([top, log_total], 1))
    at = s["target"].long()
    s["logp"].copy_(torch.where(at >= 0, (torch.gather(d, 1, at.clamp_min(0)[:, None]) - log_total)[:, 0], 0.0))
    if case["entropy"]:
        s["entropy"].copy_((log_total - (e * d.clamp_min(-1000.0)).sum(1, keepdim=True) / total)[:, 0])
    if case["top"]:
        # one number for value and place: the larger value, then the lower place
        bits = (z + 0.0).view(torch.int32)      # the two zeros are one value
        order = torch.where(bits >= 0, bits, bits ^ 0x7fffffff).long()
        key = order * 2 ** 32 + (2 ** 32 - 1 - torch.arange(z.shape[1], device=DEV))
        best = (2 ** 32 - 1 - torch.topk(key, min(case["top"], z.shape[1]), 1).values % 2 ** 32)
        logp = torch.gather(d, 1, best) - log_total
        s["top_logp"].fill_(-math.inf)[:, :best.shape[1]] = logp
        s["top_index"].fill_(-1)[:, :best.shape[1]] = torch.where(logp > -math.inf, best, -1)
    return _logprobs(s)


def _logprobs(s):
    return {k: s[k] for k in ("logp", "stats", "entropy", "top_logp", "top_index")}


def _plain_logprob_grad(s):
    case, scale = s["case"], s["case"]["scale"]
    z = s["Z"].float()
    logp = (z - s["stats"][:, :1]) * scale - s["stats"][:, 1:]
    at = s["target"].long()
    given = torch.where(at >= 0, s["dlogp"], 0.0)[:, None]
    weight = given
    if case["entropy"]:
        weight = weight + s["dentropy"][:, None] * (logp.clamp_min(-1000.0) + s["entropy"][:, None])
    dz = -torch.exp(logp) * weight
    dz.scatter_add_(1, at.clamp_min(0)[:, None], given)
    s["dZ"].copy_(dz * scale)
    return s["dZ"]


# ---- the library's calls, their arguments built once as a training loop keeps them
def _call(s):
    from sparse_full_weight_amd import _lib
    case = s["case"]
    if case["op"] == "norm":
        return _lib.prepare_norm_forward(s["X"], s["gain"], s["Y"], kind=case["kind"], eps=EPS, bias=s["bias"],
                                         res=s["res"], H=s["H"], mean=s["mean"], rstd=s["rstd"])
    if case["op"] == "norm grad":
        nbytes = _lib.sft_norm_backward_workspace(case["tokens"], case["cols"], bias=case["bias"])
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        return _lib.prepare_norm_backward(s["X"], s["gain"], s["rstd"], s["dY"], s["dX"], s["dgain"],
                                          kind=case["kind"], mean=s["mean"], dbias=s["dbias"], dH=s["dH"], ws=ws)
    if case["op"] == "rotary":
        return _lib.prepare_rotary([(s["q"], s["q_out"]), (s["k"], s["k_out"])], s["pos"], s["freq"], case["rot"],
                                   layout=case["layout"], inverse=case["grad"], amplitude=s["amplitude"])
    if case["op"] == "logprob":
        return _lib.prepare_logprob(s["Z"], s["target"], s["logp"], scale=case["scale"], stats=s["stats"],
                                    entropy=s["entropy"], top_logp=s["top_logp"], top_index=s["top_index"])
    return _lib.prepare_logprob_grad(s["Z"], s["target"], s["stats"], s["dlogp"], s["dZ"], scale=case["scale"],
                                     entropy=s["entropy"] if case["entropy"] else None, dentropy=s["dentropy"])


_PLAIN = {"norm": _plain_norm, "norm grad": _plain_norm_grad, "rotary": _plain_rotary, "logprob": _plain_logprob,
          "logprob grad": _plain_logprob_grad}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    if "call" not in s:
        s["call"] = _call(s)
    s["call"]()
    if op == "norm":
        return _normed(s)
    if op == "norm grad":
        return _norm_grads(s)
    if op == "rotary":
        return {"q": s["q_out"], "k": s["k_out"]}
    return _logprobs(s) if op == "logprob" else s["dZ"]


def exact(case, seed):
    """The same from the definitions, in 64 bits; the gradients by differentiating them."""
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm grad"):
        x = s["X"].double()
        if case["op"] == "norm" and case["res"]:
            x = (x + s["res"].double()).to(s["X"].dtype).double()
        h = x.clone().requires_grad_(case["op"] == "norm grad")
        gain = s["gain"].double().requires_grad_(h.requires_grad)
        bias = torch.zeros(case["cols"], dtype=torch.float64, device=DEV) if s["bias"] is None else s["bias"].double()
        bias.requires_grad_(h.requires_grad)
        if case["kind"] == "layer":
            mean, var = h.mean(1), h.var(1, correction=0)
        else:
            mean, var = torch.zeros_like(h[:, 0]), h.pow(2).mean(1)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(bias, (h - mean[:, None]) * rstd[:, None], gain)
        if case["op"] == "norm":
            return {"Y": y, "H": None if s["H"] is None else x, "mean": mean if case["kind"] == "layer" else None,
                    "rstd": rstd}
        y.backward(s["dY"].double())
        dx = h.grad if s["dH"] is None else h.grad + s["dH"].double()
        return {"dX": dx, "dgain": gain.grad, "dbias": bias.grad if case["bias"] else None}
    if case["op"] == "rotary":
        rot = case["rot"]
        turn = s["amplitude"] * torch.exp((-1j if case["grad"] else 1j) * (s["pos"].double()[..., None] * s["freq"]))

        def turned(x):
            x = x.double().clone()
            half = case["layout"] == "half"
            pairs = x[..., :rot].unflatten(-1, (2, rot // 2) if half else (rot // 2, 2))
            if half:
                pairs = pairs.transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, :, None])
            x[..., :rot] = (y.transpose(-1, -2) if half else y).flatten(-2)
            return x

        return {"q": turned(s["q"]), "k": turned(s["k"])}
    out = {k: [] for k in ("logp", "stats", "entropy", "top_logp", "top_index", "dZ")}
    N, V, scale, K = case["tokens"], case["vocab"], case["scale"], case["top"]
    for at in range(0, N, 256):
        part = slice(at, at + 256)
        raw = s["Z"][part].double()
        z = raw.clamp_min(-1e6)          # as good as none: exp() of it is 0
        z.requires_grad_(case["op"] == "logprob grad")
        lp = torch.log_softmax(z * scale, 1)
        entropy = -(lp.exp() * lp).sum(1)
        t = s["target"][part].long()
        logp = torch.where(t >= 0, lp[torch.arange(len(t), device=DEV), t.clamp_min(0)], 0.0)
        if case["op"] == "logprob grad":
            loss = (logp * s["dlogp"][part].double()).sum()
            if case["entropy"]:
                loss = loss + (entropy * s["dentropy"][part].double()).sum()
            out["dZ"].append(torch.autograd.grad(loss, z)[0])
            continue
        out["logp"].append(logp)
        out["entropy"].append(entropy)
        top = raw.amax(1)
        out["stats"].append(torch.stack([top, torch.logsumexp(z * scale, 1) - scale * top], 1))
        if K:
            value, index = torch.sort(raw, dim=1, descending=True, stable=True)
            value, index = (torch.nn.functional.pad(x[:, :K], (0, K - min(K, V))) for x in (value, index))
            real = (torch.arange(K, device=DEV) < V) & (value > -math.inf)
            out["top_index"].append(torch.where(real, index, -1).int())
            out["top_logp"].append(torch.where(real, lp.gather(1, index), -math.inf))
    out = {k: torch.cat(v) if v else None for k, v in out.items()}
    if case["op"] == "logprob grad":
        return out["dZ"]
    if not case["entropy"]:
        out["entropy"] = None
    del out["dZ"]
    return out


def work(case):
    size = WIDTH[case["dtype"]]
    if case["op"] in ("norm", "norm grad"):
        T, C = case["tokens"], case["cols"]
        arrays = (2 + 2 * case["res"]) if case["op"] == "norm" else (3 + case["res"])
        stats = T * (8 if case["kind"] == "layer" else 4)
        vectors = C * (1 + case["bias"]) * WIDTH[case["gain"]]
        if case["op"] == "norm grad":
            vectors = C * (WIDTH[case["gain"]] + 4 * (1 + case["bias"]))
        return {"bytes": arrays * T * C * size + stats + vectors, "flops": (7 if case["op"] == "norm" else 14) * T * C}
    if case["op"] == "rotary":
        rows = case["batch"] * case["tokens"]
        n = rows * (case["heads"] + case["kv"])
        return {"bytes": 2 * n * case["dim"] * size + 4 * rows + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    N, V = case["tokens"], case["vocab"]
    if case["op"] == "logprob":
        return {"bytes": N * V * size + N * (16 + 4 * case["entropy"] + 8 * case["top"]), "flops": 5 * N * V}
    return {"bytes": 2 * N * V * size + N * (16 + 8 * case["entropy"]), "flops": 5 * N * V}
