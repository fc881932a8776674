"""GPU tests of the row-wise calls together, as a fine-tuning step uses them:
norms, rotary positions and the loss between the products of a small layer,
their backward passes up to the weight gradients, the clip factor and the
update of the gains; eager, captured, and on two streams at once."""
import numpy as np
import pytest
import torch

from sparse_full_weight_amd import _lib
from tests.gpu_helpers import adam_dev
from tests.rowwise import BF16, F32, normal

pytestmark = pytest.mark.gpu

B, S, C, H, K, D, V = 2, 48, 256, 4, 2, 64, 1000
T = B * S
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


class Step:
    """The buffers of a step and its calls, prepared once."""

    def __init__(self, seed):
        def gpu(x):
            return x.cuda()

        def empty(*shape, dtype=BF16):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        self.X = gpu(normal((T, C), 1.0, seed, BF16))
        self.W = {n: gpu(normal((1, r, c), 0.06, seed + i, BF16)) for i, (n, r, c) in enumerate(
            (("q", H * D, C), ("k", K * D, C), ("o", C, H * D), ("v", V, C)), 1)}
        self.gains = {n: gpu(normal((C,), 0.2, seed + 10 + i, F32, m)) for i, (n, m) in enumerate(
            (("g1", 1.0), ("g2", 1.0), ("b2", 0.0)))}
        self.target = gpu(torch.randint(-1, V, (T,), generator=torch.Generator().manual_seed(seed)).int())
        self.dlogp = gpu(-(torch.rand(T, generator=torch.Generator().manual_seed(seed + 1)) + 0.5) / T)
        self.dent = gpu(0.2 * torch.rand(T, generator=torch.Generator().manual_seed(seed + 2)) / T)
        self.pos = gpu((torch.arange(S) + torch.tensor([[0], [4000]])).int())
        self.freq = gpu(torch.from_numpy(_lib.sft_rotary_table(D, 10000.0, scaling="bands", factor=8.0, context=2048.0)))
        first = gpu(torch.tensor([0, T]).int())
        mask = np.zeros(H * D, np.uint8)
        mask[[3, 5, 40, 130, 255]] = 1
        self.rows = torch.from_numpy(np.flatnonzero(mask))
        plan = _lib.sft_plan_rows(mask)
        f32 = F32
        self.Y1, self.rstd1 = empty(T, C), empty(T, dtype=f32)
        self.q, self.k, self.a, self.o = empty(T, H * D), empty(T, K * D), empty(T, H * D), empty(T, C)
        self.Hs, self.Y2, self.mean2, self.rstd2 = empty(T, C), empty(T, C), empty(T, dtype=f32), empty(T, dtype=f32)
        self.Z, self.dZ = empty(T, V, dtype=f32), empty(T, V)
        self.logp, self.stats, self.ent = empty(T, dtype=f32), empty(T, 2, dtype=f32), empty(T, dtype=f32)
        self.top = empty(T, 4, dtype=torch.int32)
        self.dY2, self.dX2, self.dA, self.dk = empty(T, C), empty(T, C), empty(T, H * D), empty(T, K * D)
        self.dYq, self.dYk, self.dY1, self.dX = (empty(T, C, dtype=t) for t in (f32, f32, BF16, BF16))
        self.dW = {n: empty(*w.shape, dtype=f32) for n, w in self.W.items() if n != "q"}
        self.dWq = empty(len(self.rows), C, dtype=f32)
        self.grads = {n: empty(C, dtype=f32) for n in self.gains}
        self.clip, self.norm, self.step = empty(1, dtype=f32), empty(1, dtype=f32), empty(1, dtype=torch.int32)
        self.states = [_lib.AdamwVec(p, self.grads[n], empty(C, dtype=f32), empty(C, dtype=f32)) for n, p in
                       self.gains.items()]

        def ws(n):
            return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

        def heads(x, n):
            return x.view(B, S, n, D)

        qk = [(heads(self.q, H),) * 2, (heads(self.k, K),) * 2]
        dqk = [(heads(self.dA, H),) * 2, (heads(self.dk, K),) * 2]
        group = [_lib.DwGroup(self.Y1, [_lib.DwMat(self.dA, plan.to_device("cuda"), self.dWq)])]
        grads = list(self.grads.values())
        nws = _lib.sft_norm_backward_workspace(T, C, bias=True)
        P = _lib
        self.forward = [
            P.prepare_norm_forward(self.X, self.gains["g1"], self.Y1, kind="rms", rstd=self.rstd1),
            P.prepare_expert_forward(first, self.Y1, self.W["q"], self.q),
            P.prepare_expert_forward(first, self.Y1, self.W["k"], self.k),
            P.prepare_rotary(qk, self.pos, self.freq, D),
            lambda stream=None: self.a.copy_(self.q.float().view(T, K, H // K, D).add(self.k.float().view(T, K, 1, D)).view(T, -1)),
            P.prepare_expert_forward(first, self.a, self.W["o"], self.o),
            P.prepare_norm_forward(self.o, self.gains["g2"], self.Y2, kind="layer", bias=self.gains["b2"], res=self.X,
                                   H=self.Hs, mean=self.mean2, rstd=self.rstd2),
            P.prepare_expert_forward(first, self.Y2, self.W["v"], self.Z),
            P.prepare_logprob(self.Z, self.target, self.logp, scale=1.25, stats=self.stats, entropy=self.ent,
                              top_index=self.top),
        ]
        self.backward = [
            P.prepare_logprob_grad(self.Z, self.target, self.stats, self.dlogp, self.dZ, scale=1.25, entropy=self.ent,
                                   dentropy=self.dent),
            P.prepare_expert_dx(first, self.dZ, self.W["v"], self.dY2),
            P.prepare_expert_dw(first, self.dZ, self.Y2, self.dW["v"]),
            P.prepare_norm_backward(self.Hs, self.gains["g2"], self.rstd2, self.dY2, self.dX2, self.grads["g2"],
                                    kind="layer", mean=self.mean2, dbias=self.grads["b2"], ws=ws(nws)),
            P.prepare_expert_dx(first, self.dX2, self.W["o"], self.dA),
            P.prepare_expert_dw(first, self.dX2, self.a, self.dW["o"]),
            lambda stream=None: self.dk.copy_(self.dA.float().view(T, K, H // K, D).sum(2).view(T, -1)),
            P.prepare_rotary(dqk, self.pos, self.freq, D, inverse=True),
            P.prepare_expert_dx(first, self.dA, self.W["q"], self.dYq),
            P.prepare_expert_dx(first, self.dk, self.W["k"], self.dYk),
            lambda stream=None: self.dY1.copy_(self.dYq + self.dYk),
            P.prepare_expert_dw(first, self.dk, self.Y1, self.dW["k"]),
            P.prepare_masked_dw(group, ws(_lib.sft_masked_dw_workspace(group))),
            P.prepare_norm_backward(self.X, self.gains["g1"], self.rstd1, self.dY1, self.dX, self.grads["g1"], kind="rms",
                                    dH=self.dX2, ws=ws(nws)),
            P.prepare_grad_clip(grads, 0.05, self.clip, self.norm, ws(_lib.sft_grad_clip_workspace(grads))),
            lambda stream=None: self.step.add_(1),
            P.prepare_adamw(self.states, self.step, adam_dev(**HP), clip=self.clip),
        ]

    def __call__(self):
        for c in self.forward + self.backward:
            c()

    def results(self):
        out = dict(logp=self.logp, ent=self.ent, top=self.top, dX=self.dX, dWq=self.dWq, clip=self.clip, norm=self.norm,
                   **{"d" + n: g for n, g in self.grads.items()}, **{"dW" + n: w for n, w in self.dW.items()},
                   **{n: g for n, g in self.gains.items()})
        return {n: x.clone() for n, x in out.items()}


def _held(x):
    return x.to(BF16).double()


def _norm64(h, gain, bias, layer, eps=1e-5):
    mean = h.mean(1, keepdim=True) if layer else torch.zeros(T, 1, dtype=torch.float64)
    rstd = ((h - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    return (h - mean) * rstd * gain + bias, (h - mean) * rstd, rstd


def _norm_back64(xhat, rstd, gain, dy, layer):
    g = dy * gain
    dx = g - xhat * (g * xhat).mean(1, keepdim=True) - (g.mean(1, keepdim=True) if layer else 0.0)
    return dx * rstd, (dy * xhat).sum(0), dy.sum(0)


def _turn64(x, heads, angle, inverse):
    x = x.view(B, S, heads, D)
    c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None] * (-1.0 if inverse else 1.0)
    u, v = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([u * c - v * s, u * s + v * c], -1).reshape(T, -1)


def _oracle(st):
    """The step in fp64, rounded to bf16 where the program holds bf16."""
    X, W = st.X.cpu().double(), {n: w[0].cpu().double() for n, w in st.W.items()}
    g1, g2, b2 = (st.gains[n].cpu().double() for n in ("g1", "g2", "b2"))
    angle = st.pos.cpu().double()[..., None] * st.freq.cpu()
    y1, xhat1, rstd1 = _norm64(X, g1, 0.0, False)
    Y1 = _held(y1)
    q, k = _held(_turn64(_held(Y1 @ W["q"].t()), H, angle, False)), _held(_turn64(_held(Y1 @ W["k"].t()), K, angle, False))
    a = _held((q.view(T, K, H // K, D) + k.view(T, K, 1, D)).view(T, -1))
    hs = _held(_held(a @ W["o"].t()) + X)
    y2, xhat2, rstd2 = _norm64(hs, g2, b2, True)
    Y2 = _held(y2)
    Z = Y2 @ W["v"].t()
    lp = torch.log_softmax(1.25 * Z, 1)
    p, ent = lp.exp(), -(lp.exp() * lp).sum(1)
    t = st.target.cpu().long()
    given = t >= 0
    at = t.clamp_min(0)[:, None]
    own = torch.where(given, st.dlogp.cpu().double(), 0.0)[:, None]
    dent = st.dent.cpu().double()[:, None]
    dZ = -p * (own + dent * (lp + ent[:, None]))
    dZ = _held(1.25 * dZ.scatter_add(1, at, own))
    dY2 = _held(dZ @ W["v"])
    dx2, dg2, db2 = _norm_back64(xhat2, rstd2, g2, dY2, True)
    dX2 = _held(dx2)
    dA = _held(dX2 @ W["o"])
    dk = _held(_turn64(_held(dA.view(T, K, H // K, D).sum(2).view(T, -1)), K, angle, True))
    dq = _held(_turn64(dA, H, angle, True))
    dY1 = _held(dq @ W["q"] + dk @ W["k"])
    dx, dg1, _ = _norm_back64(xhat1, rstd1, g1, dY1, False)
    norm = torch.cat([dg1, dg2, db2]).norm()
    return dict(logp=torch.where(given, lp.gather(1, at)[:, 0], 0.0), ent=ent, dX=dx + dX2, dWq=(dq.t() @ Y1)[st.rows],
                dWk=(dk.t() @ Y1)[None], dWo=(dX2.t() @ a)[None], dWv=(dZ.t() @ Y2)[None], dg1=dg1, dg2=dg2, db2=db2,
                norm=norm[None], clip=(0.05 / norm).clamp_max(1.0)[None])


def test_step_against_its_formulas(gpu_lib):
    st = Step(1)
    want = _oracle(st)
    before = {n: g.cpu().double() for n, g in st.gains.items()}
    st()
    got = st.results()
    for n, w in want.items():
        off = float((got[n].cpu().double() - w).norm() / w.norm())
        # the same values are rounded to bf16 at the same places; an error e before a rounding turns it the other way for
        # a share e / 2^-8 of the values, by 2^-7 each: with e = 2^-17 (fp32 sums of 1000 terms) and 14 roundings behind
        # one another at most sqrt(14 * 2^-9) * 2^-7 = 2^-9.6, and half a step of the result itself where that is bf16
        assert off <= 2.0 ** -9 + (2.0 ** -8 if got[n].dtype == BF16 else 0.0), f"{n}: {off:.3g}"
    assert 0.0 < got["clip"].item() < 1.0 and st.step.item() == 1
    for n, p in before.items():
        g = want["d" + n] * want["clip"]
        # the first step of AdamW: the gradient's sign, lr wide, wherever the gradient is not tiny
        new = p * (1 - 1e-3) - 1e-2 * torch.sign(g)
        big = g.abs() > 1e-2 * g.abs().max()
        assert (got[n].cpu().double() - new)[big].abs().max() <= 1e-4, n
    top = torch.sort(st.Z, dim=1, descending=True, stable=True)[1][:, :4].int()
    assert torch.equal(got["top"], top)


def test_captured_step_equals_eager_ones(gpu_lib):
    # one graph of the whole step, replayed on new inputs; the same step run eagerly on a second set of buffers
    one, two = Step(3), Step(3)
    one()
    two()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one()
    for turn in range(4):
        x = normal((T, C), 1.0, 50 + turn, BF16).cuda()
        target = torch.randint(-1, V, (T,), generator=torch.Generator().manual_seed(turn)).int().cuda()
        for st in (one, two):
            st.X.copy_(x)
            st.target.copy_(target)
        graph.replay()
        two()
        torch.cuda.synchronize()
        a, b = one.results(), two.results()
        for n in a:
            assert torch.equal(a[n], b[n]), f"{n} at replay {turn}"


def test_two_steps_at_once_on_two_streams(gpu_lib):
    # different inputs, interleaved call by call: the results are those of either alone
    alone = []
    for seed in (5, 6):
        st = Step(seed)
        st()
        torch.cuda.synchronize()
        alone.append(st.results())
    both = [Step(5), Step(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for a, b in zip(*((st.forward + st.backward) for st in both)):
        for c, s in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(s):
                c()
    torch.cuda.synchronize()
    for st, want in zip(both, alone):
        got = st.results()
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_calls_on_a_given_stream(gpu_lib):
    # the stream argument, with work before and behind it on that stream and none on the current one
    s = torch.cuda.Stream()
    x = normal((300, 500), 1.0, 1).cuda()
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    rstd = torch.zeros(300, device="cuda")
    target, logp = torch.arange(300, device="cuda").int(), torch.zeros(300, device="cuda")
    stats = torch.zeros(300, 2, device="cuda")
    heads, turned = x.view(300, 5, 100), torch.zeros(300, 5, 100, device="cuda")
    freq = torch.from_numpy(_lib.sft_rotary_table(100)).cuda()
    ws = torch.empty(_lib.sft_norm_backward_workspace(300, 500), dtype=torch.uint8, device="cuda")
    dgain = torch.zeros(500, device="cuda")

    def run(stream):
        _lib.sft_norm_forward(x, None, y, kind="rms", rstd=rstd, stream=stream)
        _lib.sft_norm_backward(x, None, rstd, y, z, dgain, kind="rms", ws=ws, stream=stream)
        _lib.sft_rotary([(heads, turned)], target, freq, 100, stream=stream)
        _lib.sft_logprob(y, target, logp, stats=stats, stream=stream)
        _lib.sft_logprob_grad(y, target, stats, logp, y, stream=stream)

    run(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in (rstd, z, dgain, turned, logp, stats, y)]
    for t in (rstd, z, dgain, turned, logp, stats, y):
        t.zero_()
    torch.cuda.synchronize()
    run(s)
    s.synchronize()
    for a, b in zip((rstd, z, dgain, turned, logp, stats, y), want):
        assert torch.equal(a, b)


def test_what_the_binding_refuses(gpu_lib):
    x = torch.zeros(4, 8, device="cuda")
    g = torch.ones(8, device="cuda")
    r = torch.ones(4, device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    freq = torch.zeros(4, dtype=torch.float64, device="cuda")
    h = torch.zeros(4, 2, 8, device="cuda")
    for error, call in (
        (TypeError, lambda: _lib.sft_norm_forward(x.cpu(), g, x)),
        (TypeError, lambda: _lib.sft_norm_forward(x.double(), g, x)),
        (ValueError, lambda: _lib.sft_norm_forward(x.t(), g[:4], x)),
        (ValueError, lambda: _lib.sft_norm_forward(x, g[:7], x.clone())),
        (ValueError, lambda: _lib.sft_norm_forward(x, g, x[:3])),
        (ValueError, lambda: _lib.sft_norm_forward(x, g, x.clone(), kind="batch")),
        (TypeError, lambda: _lib.sft_norm_forward(x, g, x.clone(), bias=g.bfloat16())),
        (TypeError, lambda: _lib.sft_norm_forward(x, g, x.clone(), res=x.bfloat16(), H=x.clone())),
        (_lib.SftError, lambda: _lib.sft_norm_forward(x, g, x)),
        (_lib.SftError, lambda: _lib.sft_norm_forward(x, g, x.clone(), res=x.clone())),
        (_lib.SftError, lambda: _lib.sft_norm_backward(x, g, r, x.clone(), x.clone(), g.clone())),       # no workspace
        (_lib.SftError, lambda: _lib.sft_norm_backward(x, g, r, x.clone(), x.clone(), None, kind="layer")),   # no mean
        (TypeError, lambda: _lib.sft_norm_backward(x, g, r.double(), x.clone(), x.clone(), None)),
        (ValueError, lambda: _lib.sft_rotary([], i, freq, 8)),
        (ValueError, lambda: _lib.sft_rotary([(h, h)], i[:3], freq, 8)),
        (ValueError, lambda: _lib.sft_rotary([(h, h)], i, freq[:3], 8)),
        (TypeError, lambda: _lib.sft_rotary([(h, h)], i, freq.float(), 8)),
        (TypeError, lambda: _lib.sft_rotary([(h, h)], i.long(), freq, 8)),
        (ValueError, lambda: _lib.sft_rotary([(h, h.bfloat16())], i, freq, 8)),
        (ValueError, lambda: _lib.sft_rotary([(h, h), (h[:3].clone(), h[:3])], i, freq, 8)),
        (ValueError, lambda: _lib.sft_rotary([(h.transpose(1, 2), h.transpose(1, 2))], i, freq[:1], 2)),
        (ValueError, lambda: _lib.sft_rotary([(h, h)], i, freq, 8, layout="thirds")),
        (ValueError, lambda: _lib.sft_rotary_table(8, scaling="some")),
        (_lib.SftError, lambda: _lib.sft_rotary_table(7)),
        (TypeError, lambda: _lib.sft_logprob(x, i.long(), r)),
        (ValueError, lambda: _lib.sft_logprob(x, i[:3], r)),
        (ValueError, lambda: _lib.sft_logprob(x, i, r, top_logp=x)),
        (ValueError, lambda: _lib.sft_logprob(x, i, r, stats=r)),
        (_lib.SftError, lambda: _lib.sft_logprob(x, i, None)),
        (_lib.SftError, lambda: _lib.sft_logprob(x, i, r, scale=0.0)),
        (ValueError, lambda: _lib.sft_logprob_grad(x, i, r, r, x)),
        (_lib.SftError, lambda: _lib.sft_logprob_grad(x, i, x[:, :2].contiguous(), r, x, dentropy=r)),
    ):
        with pytest.raises(error):
            call()
