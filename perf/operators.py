"""Cases of the dense half of a fine-tuning step: products grouped by expert
(forward, input gradient, weight gradient), the norm and clip factor of many
gradients, and the AdamW step over many tensors with states in 32 or 8 bits.

``run`` computes a case with elementary torch operations, or with the
library's calls where ``own`` is set.  The rows of every expert matrix are
its output features, as everywhere in this package; widths are those of the
7B-shaped layer (4096, 11008), an eighth of it (1376), or generic ones.
"""
import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 256                    # elements that share one exponent of the 8-bit states
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.1
T_MAX = 64
MAX_NORM = 1.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LAYER = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]


def listed():
    return [
        # one token of a generated answer, sent to 8 of 64 small experts
        _expert("forward", "forward one token", 8, 64, 1376, 4096, "bf16", 0.0),
        # a training step: 4096 tokens, two wide experts each
        _expert("forward", "forward training", 8192, 8, 11008, 4096, "bf16", 0.5),
        # a short odd batch on small experts, fp32 results, some experts without rows
        _expert("forward", "forward ragged", 1003, 12, 1000, 520, "f32", 2.0),
        # input gradients of a training step, many small experts
        _expert("dx", "dx training", 16384, 64, 1376, 4096, "bf16", 0.5),
        # input gradients of a short batch
        _expert("dx", "dx ragged", 517, 16, 1376, 1000, "bf16", 1.0),
        # weight gradients of a training step, fp32 as the sparse path's
        _expert("dw", "dw training", 8192, 8, 11008, 4096, "f32", 0.5),
        # weight gradients of a short batch on many experts: mostly the write
        _expert("dw", "dw short batch", 4099, 64, 1376, 4096, "bf16", 0.5),
        # the norm gains of 32 layers and the last one
        _many("adamw", "adamw gains", "even", 65, 4096, "f32", "f32", 32, False, False),
        # the seven matrices of a layer, trained densely: fp32 master, bf16 live copy, clipped
        _many("adamw", "adamw layer 32 bit", "layer", 7, 0, "f32", "f32", 32, True, True),
        # the same with bf16 weights and gradients and 8-bit states
        _many("adamw", "adamw layer 8 bit", "layer", 7, 0, "bf16", "bf16", 8, False, True),
        # the norm of the gains' gradients
        _many("clip", "clip gains", "even", 65, 4096, "", "f32", 0, False, False),
        # the norm of a layer's bf16 gradients
        _many("clip", "clip layer", "layer", 7, 0, "", "bf16", 0, False, False),
    ]


def _expert(op, name, tokens, experts, rows, cols, out, skew, add=False):
    c = {"op": op, "tokens": tokens, "experts": experts, "rows": rows, "cols": cols, "out": out, "skew": skew,
         "add": add}
    return {**c, "name": name} if name else c


def _many(op, name, kind, count, elems, p, g, bits, live, clip):
    c = {"op": op, "kind": kind, "count": count, "elems": elems, "p": p, "g": g, "bits": bits, "live": live,
         "clip": clip}
    return {**c, "name": name} if name else c


def draw(rng):
    def size(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["forward", "dx", "dw", "adamw", "clip", "forward", "dx", "dw", "adamw"])
    if op in ("forward", "dx", "dw"):
        experts = size(1, 96)
        rows, cols = 8 * size(8, 1376), 8 * size(8, 512)
        while experts * rows * cols > 8 * 11008 * 4096:
            experts = max(1, experts // 2)
        tokens = size(1, 16384)
        tokens = max(1, min(tokens, 8192 * 11008 * 4096 // (rows * cols)))
        out = rng.choice(["bf16", "f32"])
        return _expert(op, None, tokens, experts, rows, cols, out, round(2 * rng.random(), 2),
                       op == "dw" and out == "f32" and rng.random() < 0.5)
    count, elems = size(1, 200), size(100, 40_000_000)
    while count * elems > 150_000_000:
        count = max(1, count // 2)
    p = "" if op == "clip" else rng.choice(["f32", "bf16"])
    bits = 0 if op == "clip" else rng.choice([32, 8])
    return _many(op, None, "spread", count, elems, p, rng.choice(["f32", "bf16"]), bits,
                 p == "f32" and rng.random() < 0.5, op == "adamw" and rng.random() < 0.5)


def _sizes(case):
    n = case["count"]
    if case["kind"] == "layer":
        return [r * c for r, c in LAYER]
    if case["kind"] == "even":
        return [case["elems"]] * n
    return [max(1, case["elems"] // (1 + i % 13) - 3 * i) for i in range(n)]


def _counts(case, rs):
    """Rows of each expert: a draw of `tokens` choices of uneven likelihood."""
    return rs.multinomial(case["tokens"], rs.permutation(_likes(case)))


def _likes(case):
    like = (1.0 + np.arange(case["experts"])) ** -case["skew"]
    return like / like.sum()


def prepare(case, seed):
    rs = np.random.RandomState(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(shape, std, dtype):
        return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=gen).to(dtype)

    s = {"case": case}
    if case["op"] in ("forward", "dx", "dw"):
        T, E, R, C = case["tokens"], case["experts"], case["rows"], case["cols"]
        counts = _counts(case, rs)
        s["first"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
        s["used"] = torch.from_numpy(np.flatnonzero(counts).astype(np.int64)).to(DEV)
        s["most"] = int(counts.max())
        out = DTYPES[case["out"]]
        if case["op"] != "dx":
            s["X"] = normal((T, C), 1.0, torch.bfloat16)
        if case["op"] != "forward":
            s["dY"] = normal((T, R), 0.01, torch.bfloat16)
        if case["op"] != "dw":
            s["W"] = normal((E, R, C), 0.02, torch.bfloat16)
        shape = {"forward": (T, R), "dx": (T, C), "dw": (E, R, C)}[case["op"]]
        s["out"] = normal(shape, 0.1, out) if case["add"] else torch.empty(shape, dtype=out, device=DEV)
        return s

    sizes = _sizes(case)
    # one flat buffer of each kind, as a training program keeps them; every tensor starts on a block
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    start = np.concatenate([[0], np.cumsum(room)])
    total = int(start[-1])
    s["sizes"], s["start"] = sizes, [int(x) for x in start[:-1]]
    s["within"] = torch.from_numpy(np.stack([start[:-1], room])).to(DEV)
    real = torch.cat([torch.arange(r, device=DEV) < n for n, r in zip(sizes, room)])
    std = torch.from_numpy(0.01 * (0.3 + rs.rand(len(sizes))).astype(np.float32)).to(DEV)
    std = std.repeat_interleave(s["within"][1], output_size=total) * real
    s["g"] = (normal((total,), 1.0, torch.float32) * std).to(DTYPES[case["g"]])
    if case["op"] == "clip":
        s["clip"], s["norm"] = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        return s
    s["p"] = (normal((total,), 0.02, torch.float32) * real).to(DTYPES[case["p"]])
    s["live"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV) if case["live"] else None
    s["clip"] = torch.full((1,), 0.25 + rs.rand() / 2, device=DEV) if case["clip"] else None
    s["step"] = int(rs.randint(2, T_MAX))
    t = torch.arange(T_MAX + 1, dtype=torch.float64)
    s["bc1"], s["bc2"] = ((1.0 - float(np.float32(b)) ** t).float().to(DEV) for b in (BETA1, BETA2))
    m = normal((total,), 0.3, torch.float32) * std
    root = (0.2 + normal((total,), 0.6, torch.float32).abs()) * std
    s["scale"] = None
    if case["bits"] == 32:
        s["m"], s["v"] = m, root * root
    else:
        shift = torch.stack([_shift(m), _shift(root)], 1)
        s["m"], s["v"] = ((x.view(-1, BLOCK) * torch.exp2(-shift[:, i, None].float())).view(-1).to(
            torch.float8_e4m3fn) for i, x in enumerate((m, root)))
        s["scale"] = torch.exp2(shift.float()).to(torch.float8_e8m0fnu)
    return s


# ---- the 8-bit states: each block of 256 elements has a scale 2^k that brings
# its largest magnitude into [128, 256), and holds value / 2^k in e4m3.  Of v
# its square root is held.
def _shift(x):
    top = x.abs().view(-1, BLOCK).amax(1)
    return torch.where(top > 0, (top.view(torch.int32) >> 23) - 134, 0)


def _held(x, u, least):
    """Plain form of holding x >= 0 in 8 bits: the scaled values, and k of each block.

    u in [0, 1): a value goes to the next code below it, or above it where u
    exceeds the rest of its step; at least `least` where it is not zero."""
    k = _shift(x)
    y = x.double().view(-1, BLOCK) * torch.exp2(-k.double())[:, None]
    step = torch.exp2(torch.clamp((y.view(torch.int64) >> 52) - 1023, min=-6).double() - 3)
    y = torch.floor(y / step + u) * step
    return torch.where(x.view(-1, BLOCK) > 0, y.clamp_min(least), y).view(-1), k


def _dither(at, step, turn):
    """u in [0, 1), of 20 bits: fills [0, 1) evenly over the steps of each element."""
    return (((at * 0xC2B2AE35 + step * 0x9E3779B9 + turn) & 0xFFFFFFFF) >> 12).double() / 2 ** 20


def _plain_adamw(s):
    case, t, total = s["case"], s["step"], s["p"].numel()
    b1, b2 = float(np.float32(BETA1)), float(np.float32(BETA2))
    c1, c2 = (float(np.float32(1) - np.float32(b)) for b in (BETA1, BETA2))
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        scale = s["scale"].float()
        m = (s["m"].float().view(-1, BLOCK) * scale[:, :1]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * scale[:, 1:]).square().view(-1)
    m = m * b1 + g * c1
    v = v * b2 + g * g * c2
    root = torch.sqrt(v)
    p = s["p"].float()
    p = p * (1.0 - LR * DECAY) - (m * (LR / s["bc1"][t])) / (root / torch.sqrt(s["bc2"][t]) + EPS)
    s["p"].copy_(p)
    if s["live"] is not None:
        s["live"].copy_(p)
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        blocks = s["within"] // BLOCK
        at = torch.arange(total // BLOCK, device=DEV) - blocks[0].repeat_interleave(blocks[1], output_size=total // BLOCK)
        at = BLOCK * at[:, None] + torch.arange(BLOCK, device=DEV)
        y, km = _held(m.abs(), _dither(at, t, 0x55555555), 0.0)
        z, kr = _held(root, _dither(at, t, 0), 2.0 ** -9)
        s["m"].copy_(torch.copysign(y, m))
        s["v"].copy_(z)
        s["scale"].copy_(torch.exp2(torch.stack([km, kr], 1).float()))
    return _updated(s)


def _updated(s):
    return {k: s[k] for k in ("p", "live", "m", "v", "scale")}


def _views(s, name):
    x = s[name]
    return [None if x is None else x[o:o + n] for o, n in zip(s["start"], s["sizes"])]


def _plain_expert(s):
    case, first, used = s["case"], s["first"].long(), s["used"]
    T = case["tokens"]
    n = (first[1:] - first[:-1])[used]
    # every used expert's rows, padded to the longest with a row of zeros
    at = torch.arange(s["most"], device=DEV)
    at = torch.where(at < n[:, None], first[used][:, None] + at, T)

    def padded(x):
        return torch.cat([x.float(), torch.zeros(1, x.shape[1], device=DEV)])[at]

    if case["op"] == "dw":
        d = torch.bmm(padded(s["dY"]).transpose(1, 2).contiguous(), padded(s["X"]))
        if case["add"]:
            s["out"].index_add_(0, used, d)
        else:
            s["out"].zero_().index_copy_(0, used, d.to(s["out"].dtype))
        return s["out"]
    W = s["W"][used].float()
    if case["op"] == "forward":
        y = torch.bmm(padded(s["X"]), W.transpose(1, 2).contiguous())
    else:
        y = torch.bmm(padded(s["dY"]), W)
    s["out"].copy_(y[at < T])
    return s["out"]


def _plain_clip(s):
    norm = s["g"].double().square().sum().sqrt()
    s["norm"].copy_(norm)
    s["clip"].copy_(torch.clamp(MAX_NORM / norm, max=1.0))
    return {"clip": s["clip"], "norm": s["norm"]}


def _call(s):
    """The library call of a state, its arguments built once as a training loop keeps them."""
    from sparse_full_weight_amd import _lib
    op = s["case"]["op"]
    if op == "forward":
        return _lib.prepare_expert_forward(s["first"], s["X"], s["W"], s["out"])
    if op == "dx":
        return _lib.prepare_expert_dx(s["first"], s["dY"], s["W"], s["out"])
    if op == "dw":
        return _lib.prepare_expert_dw(s["first"], s["dY"], s["X"], s["out"], accumulate=s["case"]["add"])
    grads = _views(s, "g")
    if op == "clip":
        ws = torch.empty(_lib.sft_grad_clip_workspace(grads), dtype=torch.uint8, device=DEV)
        return _lib.prepare_grad_clip(grads, MAX_NORM, s["clip"], s["norm"], ws)
    hp = _lib.Adam(LR, BETA1, BETA2, EPS, s["bc1"], s["bc2"], DECAY)
    scale = [None if s["scale"] is None else s["scale"][o // BLOCK:(o + n + BLOCK - 1) // BLOCK]
             for o, n in zip(s["start"], s["sizes"])]
    vecs = [_lib.AdamwVec(*a) for a in zip(_views(s, "p"), grads, _views(s, "m"), _views(s, "v"), scale,
                                           _views(s, "live"))]
    return _lib.prepare_adamw(vecs, s["step"], hp, clip=s["clip"])


def run(s):
    op = s["case"]["op"]
    if own:
        if "call" not in s:
            s["call"] = _call(s)
        s["call"]()
        if op == "adamw":
            return _updated(s)
        return {"clip": s["clip"], "norm": s["norm"]} if op == "clip" else s["out"]
    return _plain_adamw(s) if op == "adamw" else _plain_clip(s) if op == "clip" else _plain_expert(s)


def exact(case, seed):
    """The same from the definitions, in 64 bits: expert by expert, tensor by tensor."""
    s = prepare(case, seed)
    if case["op"] in ("forward", "dx", "dw"):
        first = s["first"].tolist()
        out = s["out"].double() if case["add"] else torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e, (lo, hi) in enumerate(zip(first, first[1:])):
            if lo == hi:
                continue
            if case["op"] == "forward":
                out[lo:hi] = s["X"][lo:hi].double() @ s["W"][e].double().t()
            elif case["op"] == "dx":
                out[lo:hi] = s["dY"][lo:hi].double() @ s["W"][e].double()
            else:
                out[e] += s["dY"][lo:hi].double().t() @ s["X"][lo:hi].double()
        return out
    if case["op"] == "clip":
        norm = sum(float(g.double().pow(2).sum()) for g in _views(s, "g")) ** 0.5
        return {"clip": np.array([min(1.0, MAX_NORM / norm)]), "norm": np.array([norm])}
    new = {k: None if s[k] is None else s[k].double() for k in ("p", "live", "m", "v", "scale")}
    t, f32 = s["step"], lambda x: float(np.float32(x))  # noqa: E731
    for o, n in zip(s["start"], s["sizes"]):
        at = slice(o, o + n)
        blocks = slice(o // BLOCK, (o + n + BLOCK - 1) // BLOCK)
        g = s["g"][at].double() * (1.0 if s["clip"] is None else float(s["clip"]))
        m, v = new["m"][at], new["v"][at]
        if case["bits"] == 8:
            per = new["scale"][blocks].repeat_interleave(BLOCK, 0)[:n]
            m, v = m * per[:, 0], (v * per[:, 1]) ** 2
        m = f32(BETA1) * m + (1 - f32(BETA1)) * g
        v = f32(BETA2) * v + (1 - f32(BETA2)) * g * g
        step = f32(LR) * (m / float(s["bc1"][t])) / ((v / float(s["bc2"][t])).sqrt() + f32(EPS))
        new["p"][at] = new["p"][at] * (1 - f32(LR) * f32(DECAY)) - step
        if new["live"] is not None:
            new["live"][at] = new["p"][at]
        if case["bits"] == 32:
            new["m"][at], new["v"][at] = m, v
            continue
        i = torch.arange(n, dtype=torch.int64, device=DEV)
        for column, (x, name, turn) in enumerate(((m, "m", 0x55555555), (v.sqrt(), "v", 0))):
            u = ((i * 0xC2B2AE35 + t * 0x9E3779B9 + turn) % 2 ** 32 // 2 ** 12) / 2.0 ** 20
            size = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).view(-1, BLOCK)
            k = torch.floor(torch.log2(size.amax(1).clamp_min(2.0 ** -126))) - 7
            k = torch.where(size.amax(1) > 0, k, 0.0)
            new["scale"][blocks, column] = 2.0 ** k
            y = x.abs() * 2.0 ** -k.repeat_interleave(BLOCK)[:n]
            unit = 2.0 ** (torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
            y = (y / unit + u).floor() * unit
            if name == "v":
                y = torch.where((x > 0) & (y == 0), 2.0 ** -9, y)
            new[name][at] = torch.copysign(y, x)
    return new


def work(case):
    if case["op"] in ("forward", "dx", "dw"):
        T, E, R, C = case["tokens"], case["experts"], case["rows"], case["cols"]
        size = 4 if case["out"] == "f32" else 2
        used = float((1 - (1 - _likes(case)) ** T).sum())     # experts that get a row
        moved = {"forward": 2 * T * C + 2 * used * R * C + size * T * R,
                 "dx": 2 * T * R + 2 * used * R * C + size * T * C,
                 "dw": 2 * T * (R + C) + size * E * R * C * (2 if case["add"] else 1)}[case["op"]]
        return {"bytes": moved + 4 * (E + 1), "flops": 2 * T * R * C}
    n, width = sum(_sizes(case)), {"f32": 4, "bf16": 2, "": 0}
    if case["op"] == "clip":
        return {"bytes": n * width[case["g"]] + 8, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK     # read and written
    return {"bytes": n * (2 * width[case["p"]] + width[case["g"]] + state + (2 if case["live"] else 0)),
            "flops": 14 * n}
