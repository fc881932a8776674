"""GPU tests of the dense optimizer calls: the norm of many gradients with its
clip factor (sft_grad_clip) against fp64 sums, and AdamW over many tensors
(sft_adamw) against its formula in fp64, with states in 32 and in 8 bits."""
import numpy as np
import pytest
import torch

from sparse_full_weight_amd import _lib
from tests.gpu_helpers import adam_dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24                     # half a step of fp32
HALF = {F32: U, BF16: 2.0 ** -8}   # half a step, relative
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(n, std, seed, dtype=F32):
    return (torch.randn(n, generator=_gen(seed)) * std).to(dtype)


def _on_gpu(x, shift=0):
    """On the GPU, as a view that starts `shift` elements behind an aligned address, between marked neighbours."""
    whole = torch.full((x.numel() + shift + 8,), 7.0, device="cuda").to(x.dtype)
    whole[shift:shift + x.numel()] = x.to("cuda")
    return whole[shift:shift + x.numel()], whole


def _untouched(whole, shift, n):
    w = whole.float().cpu()
    return bool((w[:shift] == 7.0).all() and (w[shift + n:] == 7.0).all())


def _decode(m, v, scale):
    """What 8-bit states stand for: m and sqrt(v), fp64 on the host."""
    n = m.numel()
    s = scale.float().cpu().double().repeat_interleave(256, 0)[:n]
    return m.float().cpu().double() * s[:, 0], v.float().cpu().double() * s[:, 1]


def _formula(p, g, m, v, step, hp, clip=1.0):
    """AdamW in fp64, with how far fp32 arithmetic may be from it: U for each
    rounding, sums by the size of their terms.  Returns (p, m, v) and their
    bounds."""
    b1, b2 = float(np.float32(hp["beta1"])), float(np.float32(hp["beta2"]))
    c1, c2 = float(np.float32(1) - np.float32(b1)), float(np.float32(1) - np.float32(b2))
    bc1, bc2 = (float(np.float32(1 - b ** step)) for b in (b1, b2))
    lr, eps, decay = (float(np.float32(hp[k])) for k in ("lr", "eps", "weight_decay"))
    g = g * clip
    m1, v1 = b1 * m + c1 * g, b2 * v + c2 * g * g
    em = 3 * U * ((b1 * m).abs() + (c1 * g).abs())     # clip, the products and the sum
    ev = 5 * U * v1                                      # clip twice, square, products, sum: all terms positive
    den = (v1 / bc2).sqrt() + eps
    u = lr / bc1 * m1 / den
    # k1 and its product: 2; k2 (root, quotient), its product, the sum, the root of v and half of v's 5: 7.5; the
    # quotient 1, or as a product with a reciprocal off by one unit in the last place (2 U) 3
    eu = 12.5 * U * u.abs() + lr / bc1 / den * em
    p1 = p * (1 - lr * decay) - u
    ep = 3 * U * p.abs() + eu + U * p1.abs()           # lr*decay, 1 - it, the product; the difference
    return (p1, m1, v1), (1.01 * ep + 1e-45, 1.01 * em + 1e-45, 1.01 * ev + 1e-45)


def _close(got, want, bound, what, dtype=F32):
    got = got.float().cpu().double()
    if dtype != F32:
        bound = bound + HALF[dtype] * (want.abs() + bound)
    worst = ((got - want).abs() - bound).max().item() if got.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} beyond the bound"


@pytest.mark.parametrize("p_type", [F32, BF16])
@pytest.mark.parametrize("g_type", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1])
def test_adamw_32_bit_states(gpu_lib, p_type, g_type, shift):
    step, clip = 7, 0.375
    sizes = [1, 3, 255, 256, 257, 2047, 2048, 2049, 4096, 10007, 0]
    vecs, host, wholes = [], [], []
    for i, n in enumerate(sizes):
        p, g = _normal(n, 0.5, 10 + i, p_type), _normal(n, 0.1, 50 + i, g_type)
        m, v = _normal(n, 0.05, 90 + i), _normal(n, 0.1, 130 + i).square()
        live = _normal(n, 0.0, 1, BF16)
        host.append([x.double() for x in (p, g, m, v)])
        on = [_on_gpu(x, shift) for x in (p, g, m, v, live)]
        wholes.append([w for _, w in on])
        p, g, m, v, live = (x for x, _ in on)
        vecs.append(_lib.AdamwVec(p, g, m, v, None, live if i % 2 else None))
    _lib.sft_adamw(vecs, step, adam_dev(**HP), clip=torch.full((1,), clip, device="cuda"))
    for i, (vec, h) in enumerate(zip(vecs, host)):
        want, bound = _formula(*h, step, HP, clip)
        _close(vec.p, want[0], bound[0], f"p of {sizes[i]}", p_type)
        _close(vec.m, want[1], bound[1], f"m of {sizes[i]}")
        _close(vec.v, want[2], bound[2], f"v of {sizes[i]}")
        if vec.p_live is not None:
            _close(vec.p_live, want[0], bound[0], f"live of {sizes[i]}", BF16)
        assert torch.equal(vec.grad.cpu().double(), h[1])
        assert all(_untouched(w, shift, sizes[i]) for w in wholes[i])


def _codes(x, step, turn, least):
    """The documented way of holding x >= 0 (fp32) in 8 bits, in fp64: values, exponents, and whether a value
    is so near a border that the last bits of its scaled form decide."""
    n = x.numel()
    blocks = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
    top = blocks.amax(1).double().numpy()
    k = torch.from_numpy(np.where(top > 0, np.maximum(np.frexp(top)[1] - 8, -127), 0).astype(np.float64))
    y = x.double() / torch.exp2(k).repeat_interleave(256)[:n]
    e = torch.from_numpy(np.frexp(y.numpy())[1].astype(np.float64)) - 1
    unit = torch.exp2(e.clamp_min(-6) - 3)
    i = torch.arange(n, dtype=torch.int64)
    u = ((i * 0xC2B2AE35 + step * 0x9E3779B9 + turn) % 2 ** 32 // 2 ** 12).double() / 2 ** 20
    t = y / unit + u
    near = (t - t.round()).abs() < 2.0 ** -19
    y = t.floor() * unit
    if least:
        y = torch.where((x > 0) & (y == 0), 2.0 ** -9, y)
    return y, k, unit, near


@pytest.mark.parametrize("p_type", [F32, BF16])
@pytest.mark.parametrize("g_type", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1])
def test_adamw_8_bit_states(gpu_lib, p_type, g_type, shift):
    sizes = [1, 3, 255, 256, 257, 4095, 4096, 4097, 20011, 0]
    vecs, host, wholes = [], [], []
    for i, n in enumerate(sizes):
        p, g = _normal(n, 0.5, 10 + i, p_type), _normal(n, 0.1, 50 + i, g_type)
        vec = [p, g, torch.zeros(n), torch.zeros(n), _normal(n, 0.0, 1, BF16)]
        host.append([p.double(), g.double()])
        vec[2], vec[3] = vec[2].to(torch.float8_e4m3fn), vec[3].to(torch.float8_e4m3fn)
        on = [_on_gpu(x, shift) for x in vec]
        wholes.append([w for _, w in on])
        scale = torch.ones(((n + 255) // 256, 2), device="cuda").to(torch.float8_e8m0fnu)
        vecs.append(_lib.AdamwVec(*(x for x, _ in on[:4]), scale, on[4][0] if i % 2 else None))
    hp = adam_dev(**HP)
    for step in (1, 2, 3):
        before = [(v.p.double().cpu(), *_decode(v.m, v.v, v.scale)) for v in vecs]
        _lib.sft_adamw(vecs, step, hp)
        for i, (vec, h) in enumerate(zip(vecs, host)):
            what = f"of {sizes[i]} at step {step}"
            p, m, root = before[i]
            want, bound = _formula(p, h[1], m, root * root, step, HP)
            _close(vec.p, want[0], bound[0], "p " + what, p_type)
            if vec.p_live is not None:
                _close(vec.p_live, want[0], bound[0], "live " + what, BF16)
            assert all(_untouched(w, shift, sizes[i]) for w in wholes[i])
            # the states: the same fp32 arithmetic on the host gives the same scales and codes
            f = np.float32
            g32, m32, r32 = (x.float().numpy() for x in (h[1], m, root))
            m1 = f(HP["beta1"]) * m32 + (f(1) - f(HP["beta1"])) * g32
            r1 = np.sqrt(f(HP["beta2"]) * (r32 * r32) + (f(1) - f(HP["beta2"])) * (g32 * g32))
            for x, code, turn, least, col in ((m1, vec.m, 0x55555555, False, 0), (r1, vec.v, 0, True, 1)):
                y, k, unit, near = _codes(torch.from_numpy(np.abs(x)), step, turn, least)
                assert torch.equal(vec.scale[:, col].float().cpu().double(), torch.exp2(k)), what
                got = code.float().cpu().double()
                off = (got.abs() - y).abs()
                assert bool(((off == 0) | (near & (off <= 2 * unit))).all()), what
                assert int(near.sum()) <= 1 + g32.size // 100
                assert bool(((got == 0) | (torch.signbit(got) == torch.from_numpy(np.signbit(x)))).all()), what


def test_adamw_8_bit_follows_32_bit_over_many_steps(gpu_lib):
    # gradients of constant spread, then a tenth of it: the held sqrt(v) must follow down as well.  A held value is
    # off by up to a code's width (1/8) up or down at every step, and the even sequence keeps the sum of these
    # deviations over v's memory within a few codes: 0.15 is the simulated rms deviation of the sequence
    # at a spread of e^1.5 within the blocks; half again as much is allowed, and a bias of a third of it.
    n, steps = 4096, 1500
    gen = torch.Generator(device="cuda").manual_seed(5)
    size = torch.exp(1.5 * torch.randn(n, generator=gen, device="cuda")) * 1e-3
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    held = _lib.AdamwVec.alloc8(p.clone(), g)
    full = _lib.AdamwVec(p.clone(), g, torch.zeros_like(p), torch.zeros_like(p))
    hp = adam_dev(lr=1e-3, beta1=0.9, beta2=0.99)
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = _lib.prepare_adamw([held], step, hp), _lib.prepare_adamw([full], step, hp)
    for t in range(steps):
        step += 1
        g.copy_(torch.randn(n, generator=gen, device="cuda") * size * (1.0 if t < steps // 2 else 0.1))
        for c in call:
            c()
    _, root = _decode(held.m, held.v, held.scale)
    ratio = root / full.v.sqrt().cpu().double() - 1
    assert ratio.square().mean().sqrt().item() < 0.225
    assert abs(ratio.mean().item()) < 0.075


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("clip", [0.0, -1.0, float("nan"), float("inf")])
def test_adamw_leaves_a_step_out(gpu_lib, held, clip):
    p, g = _normal(700, 1.0, 1).cuda(), _normal(700, 1.0, 2).cuda()
    vec = _lib.AdamwVec.alloc8(p, g) if held else _lib.AdamwVec(p, g, p * 0.1, p * p)
    hp = adam_dev(**HP)
    _lib.sft_adamw([vec], 1, hp)
    keep = [x.clone().view(torch.uint8) for x in (vec.p, vec.m, vec.v) + ((vec.scale,) if held else ())]
    _lib.sft_adamw([vec], 2, hp, clip=torch.full((1,), clip, device="cuda"))
    for a, b in zip(keep, (vec.p, vec.m, vec.v) + ((vec.scale,) if held else ())):
        assert torch.equal(a, b.view(torch.uint8))


@pytest.mark.parametrize("size", [1e-40, 1e-30, 1e-12, 1e12, 1e18])
def test_adamw_8_bit_extreme_gradients(gpu_lib, size):
    # the first step from zero moments is lr * sign(g) where eps is small against sqrt(v); where v = g^2 (1-beta2)
    # falls below fp32's range the step is m / eps, tiny
    g = (torch.sign(_normal(512, 1.0, 3)) * size).cuda()
    vec = _lib.AdamwVec.alloc8(torch.zeros(512, device="cuda"), g)
    _lib.sft_adamw([vec], 1, adam_dev(lr=1e-2, eps=1e-30))
    m, root = _decode(vec.m, vec.v, vec.scale)
    want = 0.1 * g.cpu().double()
    assert bool(((m - want).abs() <= want.abs() / 8 + 2.0 ** -136).all())
    p = vec.p.cpu().double()
    assert torch.isfinite(p).all() and bool((p.abs() <= 1.001e-2).all())
    if size >= 1e-12:
        assert bool(((p + 1e-2 * torch.sign(g.cpu().double())).abs() <= 1e-6).all())
        assert bool(((root / (size * 1e-3 ** 0.5) - 1).abs() <= 1 / 8 + 1e-3).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_adamw_8_bit_marks_blocks_that_are_not_finite(gpu_lib, bad):
    g = _normal(1000, 0.1, 4).cuda()
    g[300] = bad
    vec = _lib.AdamwVec.alloc8(_normal(1000, 1.0, 5).cuda(), g)
    _lib.sft_adamw([vec], 1, adam_dev(**HP))
    scale = vec.scale.float().cpu()
    assert torch.isnan(scale[1]).all() and torch.isfinite(scale[[0, 2, 3]]).all()
    m, root = _decode(vec.m, vec.v, vec.scale)
    inside = torch.zeros(1000, dtype=torch.bool)
    inside[256:512] = True
    assert torch.equal(torch.isnan(m), inside) and torch.equal(torch.isnan(root), inside)
    assert torch.equal(torch.isnan(vec.p.cpu()), torch.arange(1000) == 300)


def test_adamw_zero_gradient_and_zero_states(gpu_lib):
    p = _normal(600, 1.0, 6).cuda()
    vecs = [_lib.AdamwVec.alloc8(p.clone(), torch.zeros_like(p)),
            _lib.AdamwVec(p.clone(), torch.zeros_like(p), torch.zeros_like(p), torch.zeros_like(p))]
    _lib.sft_adamw(vecs, 3, adam_dev(lr=1e-2))
    for v in vecs:
        assert torch.equal(v.p, p) and not v.m.float().any() and not v.v.float().any()
    assert bool((vecs[0].scale.float() == 1).all())


def test_adamw_many_tensors_of_every_kind(gpu_lib):
    # more tensors of each kind than one launch holds, in mixed order: the same as one call a tensor
    def make():
        out = []
        for i in range(330):
            n = 1 + 37 * i % 5000
            p, g = _normal(n, 1.0, i, (F32, BF16)[i & 1]).cuda(), _normal(n, 0.1, 900 + i, (F32, BF16)[i >> 1 & 1]).cuda()
            held = i % 3 == 0
            out.append(_lib.AdamwVec.alloc8(p, g) if held else
                       _lib.AdamwVec(p, g, torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")))
        return out

    a, b, hp = make(), make(), adam_dev(**HP)
    for step in (1, 2):
        _lib.sft_adamw(a, step, hp)
        for v in b:
            _lib.sft_adamw([v], step, hp)
    for x, y in zip(a, b):
        assert torch.equal(x.p, y.p) and torch.equal(x.m.view(torch.uint8), y.m.view(torch.uint8))
        assert torch.equal(x.v.view(torch.uint8), y.v.view(torch.uint8))
        assert x.scale is None or torch.equal(x.scale.view(torch.uint8), y.scale.view(torch.uint8))


def test_adamw_past_2_31_elements(gpu_lib):
    # the last elements of a tensor whose offsets pass 32 bits, in bytes and in elements
    n, tail = (1 << 31) + 1029, 3000
    p, g = (torch.zeros(n, dtype=BF16, device="cuda") for _ in range(2))
    g[-tail:] = _normal(tail, 0.1, 8, BF16).cuda()
    p[-tail:] = _normal(tail, 1.0, 9, BF16).cuda()
    want = _lib.AdamwVec(p[-tail:].clone(), g[-tail:].clone(), *(torch.zeros(tail, device="cuda") for _ in range(2)))
    vec = _lib.AdamwVec(p, g, torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"))
    hp = adam_dev(**HP)
    _lib.sft_adamw([vec], 4, hp)
    _lib.sft_adamw([want], 4, hp)
    assert torch.equal(p[-tail:], want.p) and torch.equal(vec.m[-tail:], want.m) and torch.equal(vec.v[-tail:], want.v)
    assert not p[:-tail].any()
    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(_lib.sft_grad_clip_workspace([g]), dtype=torch.uint8, device="cuda")
    _lib.sft_grad_clip([g], 1.0, torch.zeros(1, device="cuda"), norm, ws)
    true = g[-tail:].double().square().sum().sqrt().item()
    assert abs(norm.item() - true) <= 2 * U * true


def _clip(grads, max_norm=1.0):
    clip, norm = torch.full((1,), 9.0, device="cuda"), torch.full((1,), 9.0, device="cuda")
    ws = torch.full((_lib.sft_grad_clip_workspace(grads),), 255, dtype=torch.uint8, device="cuda")
    _lib.sft_grad_clip(grads, max_norm, clip, norm, ws)
    return clip.item(), norm.item()


@pytest.mark.parametrize("sizes", [[1], [8192], [8191, 8193], [3, 0, 70001, 5], [4096] * 65, [17] * 450, [3_000_017]])
@pytest.mark.parametrize("max_norm", [0.01, 1e9])
def test_grad_clip(gpu_lib, sizes, max_norm):
    host = [_normal(n, 0.1, i, (F32, BF16)[i & 1]) for i, n in enumerate(sizes)]
    grads = [_on_gpu(x, i % 3)[0] for i, x in enumerate(host)]
    clip, norm = _clip(grads, max_norm)
    # every square is exact in fp64, its sums off by at most 2^-53 each: what is left is the rounding to fp32
    true = float(sum(x.double().square().sum() for x in host)) ** 0.5
    assert abs(norm - true) <= 1.01 * U * true
    factor = min(1.0, float(np.float32(max_norm)) / true)
    assert abs(clip - factor) <= 1.01 * U * factor
    assert (clip, norm) == _clip(grads, max_norm)


@pytest.mark.parametrize("value,clip,norm", [(float("nan"), 0.0, float("nan")), (float("inf"), 0.0, float("inf")),
                                             (3e38, 1 / 3e38, 3e38), (1e-40, 1.0, 1e-40), (0.0, 1.0, 0.0)])
def test_grad_clip_range(gpu_lib, value, clip, norm):
    g = torch.zeros(20000, device="cuda")
    g[12345] = value
    got = _clip([g])
    assert got[1] == pytest.approx(float(np.float32(norm)), rel=2 * U, nan_ok=True)
    assert got[0] == pytest.approx(clip, rel=2 * U, abs=2.0 ** -149)


def test_grad_clip_of_nothing(gpu_lib):
    assert _clip([]) == (1.0, 0.0)
    assert _clip([torch.zeros(0, device="cuda")]) == (1.0, 0.0)
    assert _clip([torch.full((4,), 2.0, device="cuda")], float("inf")) == (1.0, 4.0)


def test_clipped_steps_captured_and_replayed(gpu_lib):
    # the norm, its factor and the step in one graph, with the step number on the device: four replays, with other
    # gradients and eager work between them, against the same calls run eagerly on another stream
    def make():
        vecs = []
        for i in range(6):
            n = 500 + 777 * i
            p, g = _normal(n, 1.0, i).cuda(), torch.zeros(n, device="cuda")
            vecs.append(_lib.AdamwVec.alloc8(p, g) if i % 2 else
                        _lib.AdamwVec(p, g, torch.zeros_like(p), torch.zeros_like(p)))
        grads = [v.grad for v in vecs]
        clip, norm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        ws = torch.empty(_lib.sft_grad_clip_workspace(grads), dtype=torch.uint8, device="cuda")
        step = torch.zeros(1, dtype=torch.int32, device="cuda")
        return vecs, step, norm, (_lib.prepare_grad_clip(grads, 0.5, clip, norm, ws),
                                  _lib.prepare_adamw(vecs, step, hp, clip))

    hp = adam_dev(**HP)
    (a, step_a, norm_a, calls_a), (b, step_b, norm_b, calls_b) = make(), make()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step_a += 1
        for c in calls_a:
            c()
    other = torch.cuda.Stream()
    for t in range(4):
        for i, (x, y) in enumerate(zip(a, b)):
            x.grad.copy_(_normal(x.grad.numel(), 0.1, 100 * t + i))
            y.grad.copy_(x.grad)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            step_b += 1
            for c in calls_b:
                c()
        torch.cuda.synchronize()
        assert step_a.item() == t + 1 and torch.equal(norm_a, norm_b) and norm_a.item() > 0.5
        for x, y in zip(a, b):
            assert torch.equal(x.p, y.p) and torch.equal(x.m.view(torch.uint8), y.m.view(torch.uint8))
            assert torch.equal(x.v.view(torch.uint8), y.v.view(torch.uint8))


def test_grad_clip_feeds_the_coupled_update(gpu_lib):
    # the pair's two factors, each written by a call of its own
    clip = torch.zeros(2, device="cuda")
    grads = [_normal(5000, 1.0, i).cuda() for i in range(2)]
    ws = torch.empty(_lib.sft_grad_clip_workspace(grads), dtype=torch.uint8, device="cuda")
    for i in range(2):
        _lib.sft_grad_clip([grads[i]], 1.0, clip[i:i + 1], None, ws)
    want = [1.0 / g.double().norm().item() for g in grads]
    assert clip.tolist() == pytest.approx(want, rel=2 * U)


@pytest.mark.parametrize("wrong", ["strided", "host", "type", "size", "scale", "state type", "clip size"])
def test_adamw_python_refuses(gpu_lib, wrong):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    m, v, scale, clip = torch.zeros_like(p), torch.zeros_like(p), None, None
    if wrong == "strided":
        g = torch.zeros(128, device="cuda")[::2]
    elif wrong == "host":
        g = torch.zeros(64)
    elif wrong == "type":
        g = torch.zeros(64, dtype=torch.float16, device="cuda")
    elif wrong == "size":
        m = torch.zeros(63, device="cuda")
    elif wrong == "scale":
        held = _lib.AdamwVec.alloc8(p, g)
        m, v, scale = held.m, held.v, torch.ones((2, 2), device="cuda").to(torch.float8_e8m0fnu)
    elif wrong == "state type":
        scale = torch.ones((1, 2), device="cuda").to(torch.float8_e8m0fnu)
    else:
        clip = torch.ones(2, device="cuda")
    with pytest.raises((TypeError, ValueError)):
        _lib.sft_adamw([_lib.AdamwVec(p, g, m, v, scale)], 1, adam_dev(), clip=clip)


def check_8_bit_step(vec, before, g, step, hp, clip, what):
    """One step of 8-bit states against the formula: before = (p, m, sqrt(v)) in fp64 on the host, g the gradient (fp32
    values, fp64), clip as the kernel read it (an fp32 number)."""
    p, m, root = (x.reshape(-1) for x in before)
    g = g.reshape(-1)
    want, bound = _formula(p, g, m, root * root, step, hp, clip)
    _close(vec.p.view(-1), want[0], bound[0], "p " + what, vec.p.dtype)
    if vec.p_live is not None:
        _close(vec.p_live.view(-1), want[0], bound[0], "live " + what, BF16)
    # the same fp32 arithmetic on the host gives the same scales and codes
    f = np.float32
    g32, m32, r32 = (x.float().numpy() for x in (g, m, root))
    g32 = g32 * f(clip)
    m1 = f(hp["beta1"]) * m32 + (f(1) - f(hp["beta1"])) * g32
    r1 = np.sqrt(f(hp["beta2"]) * (r32 * r32) + (f(1) - f(hp["beta2"])) * (g32 * g32))
    for x, code, turn, least, col in ((m1, vec.m, 0x55555555, False, 0), (r1, vec.v, 0, True, 1)):
        y, k, unit, near = _codes(torch.from_numpy(np.abs(x)), step, turn, least)
        assert torch.equal(vec.scale[:, col].float().cpu().double(), torch.exp2(k)), what
        got = code.view(-1).float().cpu().double()
        off = (got.abs() - y).abs()
        assert bool(((off == 0) | (near & (off <= 2 * unit))).all()), what
        assert int(near.sum()) <= 1 + g32.size // 100
        assert bool(((got == 0) | (torch.signbit(got) == torch.from_numpy(np.signbit(x)))).all()), what


def before_8_bit_step(vec):
    return (vec.p.double().cpu(), *_decode(vec.m.view(-1), vec.v.view(-1), vec.scale))


@pytest.mark.parametrize("p_type,g_type", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("clip", [1.0, 0.375, 0.1, 2.0 ** -30])
def test_adamw_8_bit_states_with_a_clip_factor(gpu_lib, p_type, g_type, on_device, clip):
    sizes = [1, 257, 4096, 9003]
    vecs = []
    for i, n in enumerate(sizes):
        p, g = _normal(n, 0.5, 10 + i, p_type).cuda(), _normal(n, 0.1, 50 + i, g_type).cuda()
        vecs.append(_lib.AdamwVec.alloc8(p, g, torch.zeros(n, dtype=BF16, device="cuda") if i % 2 else None))
    hp, factor = adam_dev(**HP), torch.full((1,), clip, device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in (1, 2, 6):
        before = [before_8_bit_step(v) for v in vecs]
        step.fill_(t)
        _lib.sft_adamw(vecs, step if on_device else t, hp, clip=factor)
        for n, vec, b in zip(sizes, vecs, before):
            check_8_bit_step(vec, b, vec.grad.double().cpu(), t, HP, factor.item(), f"of {n} at step {t}")


@pytest.mark.parametrize("held", [False, True])
def test_arrays_behind_one_another_are_not_refused(gpu_lib, held):
    # parameters, gradients and states of two tensors in turn in one buffer, not a byte apart, with the factor and
    # the step number between them, and the norm's workspace behind a gradient: as in buffers of their own
    n = [512, 1280]
    size = dict(p=4, g=4, m=1 if held else 4, v=1 if held else 4)
    order = [("p", 0), ("g", 0), ("m", 0), ("clip", 0), ("v", 0), ("g", 1), ("ws", 0), ("v", 1), ("step", 0), ("m", 1), ("p", 1)]
    grads = [_normal(k, 0.1, 40 + i).cuda() for i, k in enumerate(n)]
    ws = _lib.sft_grad_clip_workspace(grads)
    at, where = 0, {}
    for name, i in order:
        at = -(-at // 16) * 16 if name == "ws" else at
        where[name, i] = at
        at += {"clip": 16, "step": 16, "ws": ws}.get(name) or size[name] * n[i]
    whole = torch.zeros(at, dtype=torch.uint8, device="cuda")
    state = torch.float8_e4m3fn if held else F32

    def part(name, i, count, dtype):
        lo = where[name, i]
        return whole[lo:lo + count * dtype.itemsize].view(dtype)

    def make(inside):
        vecs = []
        for i, k in enumerate(n):
            own = [torch.zeros(k, dtype=t, device="cuda") for t in (F32, F32, state, state)]
            p, g, m, v = [part(c, i, k, t) for c, t in zip("pgmv", (F32, F32, state, state))] if inside else own
            p.copy_(_normal(k, 1.0, 30 + i).cuda())
            g.copy_(grads[i])
            vecs.append(_lib.AdamwVec(p, g, m, v, _lib.AdamwVec.alloc8(p, g).scale if held else None))
        return vecs

    a, b, hp = make(True), make(False), adam_dev(**HP)
    clip, step = part("clip", 0, 1, F32), part("step", 0, 1, torch.int32)
    step.fill_(3)
    _lib.sft_grad_clip([v.grad for v in a], 1.0, clip, None, part("ws", 0, ws, torch.uint8))
    other = torch.zeros(1, device="cuda")
    _lib.sft_grad_clip([v.grad for v in b], 1.0, other, None, torch.empty(ws, dtype=torch.uint8, device="cuda"))
    assert 0.0 < clip.item() < 1.0 and torch.equal(clip, other)
    _lib.sft_adamw(a, step, hp, clip=clip)
    _lib.sft_adamw(b, 3, hp, clip=other)
    for x, y, g in zip(a, b, grads):
        assert torch.equal(x.grad, g) and torch.equal(x.p, y.p)
        assert torch.equal(x.m.view(torch.uint8), y.m.view(torch.uint8))
        assert torch.equal(x.v.view(torch.uint8), y.v.view(torch.uint8))
