"""GPU tests of the products grouped by expert (sft_expert_forward, _dx, _dw)
against fp64 products of the same inputs, at ragged groups, odd sizes and
sizes around the kernels' tiles."""
import numpy as np
import pytest
import torch

from sparse_full_weight_amd import _lib
from tests import expert_shapes
from tests.gpu_helpers import adam_dev
from tests.test_gpu_dense import before_8_bit_step, check_8_bit_step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24                     # half a step of fp32


def _normal(shape, std, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def _first(counts, start=0):
    return torch.from_numpy(np.concatenate([[start], start + np.cumsum(counts)]).astype(np.int32)).cuda()


def _check(got, a, b, what):
    """got = a @ b in fp32 sums of exact products: each of the K additions and the joining of partial sums rounds
    by U of a partial sum, which the sum of magnitudes bounds; (K + 4) U of it in all, and half a step of the
    output's type."""
    want = a.double() @ b.double()
    bound = (a.shape[1] + 4) * U * (a.double().abs() @ b.double().abs())
    if got.dtype == BF16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    off = ((got.double() - want).abs() - bound)
    assert off.numel() == 0 or off.max().item() <= 0, f"{what}: {off.max().item()} beyond the bound"


MARK = -77.0


def _run(op, counts, R, C, out, seed=0, start=0, behind=0, integer=False, add=False):
    """One call with the inputs' and outputs' rows that belong to no expert marked; checks all of it."""
    E, T = len(counts), start + int(sum(counts)) + behind
    first = _first(counts, start)
    X, dY, W = _normal((T, C), 1.0, seed), _normal((T, R), 0.1, seed + 1), _normal((E, R, C), 0.1, seed + 2)
    if integer:
        X, dY, W = ((x * s).round().clamp(-3, 3) for x, s in ((X, 1.0), (dY, 10.0), (W, 10.0)))
    for x in (X, dY):                       # rows of no expert must not reach any result
        x[:start] = float("nan")
        x[T - behind:] = float("nan")
    bounds = first.tolist()
    if op == "dw":
        D = torch.full((E, R, C), MARK, dtype=out, device="cuda")
        if add:
            D = torch.randn((E, R, C), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 3))
        before = D.clone()
        _lib.sft_expert_dw(first, dY, X, D, accumulate=add)
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            a, b = dY[lo:hi].t(), X[lo:hi]
            if add:                         # the old value is one more term of the sum
                a = torch.cat([a.double(), before[e].double()], 1)
                b = torch.cat([b.double(), torch.eye(C, device="cuda", dtype=torch.float64)])
            elif integer:
                assert torch.equal(D[e].double(), a.double() @ b.double())
            _check(D[e], a, b, f"dW of expert {e}, {hi - lo} rows")
        return D
    N = R if op == "forward" else C
    Y = torch.full((T, N), MARK, dtype=out, device="cuda")
    if op == "forward":
        _lib.sft_expert_forward(first, X, W, Y)
    else:
        _lib.sft_expert_dx(first, dY, W, Y)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        a, b = (X[lo:hi], W[e].t()) if op == "forward" else (dY[lo:hi], W[e])
        if integer and out == F32:
            assert torch.equal(Y[lo:hi].double(), a.double() @ b.double())
        _check(Y[lo:hi], a, b, f"{op} of expert {e}, {hi - lo} rows")
    assert bool((Y[:start] == MARK).all()) and bool((Y[T - behind:] == MARK).all())
    return Y


OPS = ["forward", "dx", "dw"]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [3, 0, 5, 1, 0], [15, 16, 17, 0, 33], [63, 64, 65], [127, 1, 130],
                                    [255, 0, 257], [300, 0, 0, 511]])
def test_ragged_groups(gpu_lib, op, out, counts):
    _run(op, counts, 72, 136, out, start=2, behind=3)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("R,C", [(8, 8), (8, 4096), (4096, 8), (56, 64), (64, 72), (120, 248), (128, 128), (136, 264),
                                 (256, 256), (264, 520), (1000, 520), (512, 1032)])
def test_odd_sizes(gpu_lib, op, R, C):
    _run(op, [70, 0, 5, 201], R, C, F32)
    _run(op, [2, 1, 0, 7], R, C, BF16, behind=1)


@pytest.mark.parametrize("op", OPS)
def test_integer_inputs_are_exact(gpu_lib, op):
    # lanes, tiles and steps that were mixed up would show: every product and sum of these is exact in fp32
    _run(op, [300, 17, 0, 140], 328, 392, F32, integer=True)
    _run(op, [9, 16, 1, 2], 328, 392, F32, integer=True)


@pytest.mark.parametrize("integer", [False, True])
@pytest.mark.parametrize("op,counts,R,C", [
    ("forward", [8192 - 3, 70], 8000, 72), ("forward", [7700, 0, 530], 8192, 40),        # 256 x 256
    ("dx", [8192 - 3, 70], 4104, 1032), ("dx", [7700, 0, 530], 4096, 1024), ("dx", [3, 1, 0] * 11, 4160, 1288),
    ("forward", [90, 200, 0, 129] * 10, 1160, 72),                                             # 128 x 128
    ("forward", [5000, 61, 131, 3000], 2056, 136), ("dx", [5000, 61, 131, 3000], 136, 2056),   # 128 x 192
    ("dx", [1, 0, 2, 0, 1] * 12, 72, 1160), ("dx", [200, 130] * 8, 200, 584),
    ("forward", [2000, 129, 65], 1032, 72), ("dx", [2000, 129, 65], 72, 1032),                   # 64 x 128
    ("forward", [2, 0, 1, 70], 520, 328), ("dx", [2, 0, 1, 70], 328, 520),                     # 64 x 64
    ("dw", [300, 0, 65, 1], 1096, 2056), ("dw", [33, 31, 97, 0], 1096, 1032), ("dw", [70, 0, 129], 328, 264),
])
def test_every_shape_of_tiles(gpu_lib, op, counts, R, C, integer):
    # sizes that take each of the kernels' tiles, with rows and columns that end inside them; the last launch round of
    # the 256 x 256 tiles is cut in halves in one of the two cases
    _run(op, counts, R, C, F32, start=1, behind=2, integer=integer)
    if not integer:
        _run(op, counts, R, C, BF16)


@pytest.mark.parametrize("integer", [False, True])
@pytest.mark.parametrize("op,counts,R,C", [
    ("forward", [50, 48, 0, 129] * 12, 2056, 72), ("dx", [4, 0, 70, 9] * 12, 136, 2056),     # 128 x 128, short groups
    ("forward", [3, 1, 0] * 11, 520, 72), ("forward", [3, 65, 0] * 11, 520, 200),            # 64 x 128, three stages
    ("forward", [30, 1, 0] * 11, 584, 328), ("dx", [3, 1, 0] * 11, 56, 520), ("dx", [3, 65, 0] * 11, 200, 520),
    ("dx", [30, 1, 0] * 11, 328, 584),
])
def test_shapes_of_tiles_of_short_groups(gpu_lib, op, counts, R, C, integer):
    _run(op, counts, R, C, F32, start=1, behind=2, integer=integer)
    if not integer:
        _run(op, counts, R, C, BF16)


@pytest.mark.parametrize("C", [2040, 2048, 2104, 2176, 2240, 2248, 2304, 4096])
def test_few_tokens_with_long_sums(gpu_lib, C):
    # sums that end in each place of the five stages of the forward's ring; integers are exact below 2^24
    _run("forward", [2, 0, 1, 66], 328, C, F32, start=1, behind=2, integer=True)
    _run("forward", [1], 136, C, BF16)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("E", [1, 63, 64, 65, 200])
def test_numbers_of_experts(gpu_lib, op, E):
    rs = np.random.RandomState(E)
    _run(op, list(rs.randint(0, 6, E) * (rs.rand(E) < 0.7)), 40, 72, F32, seed=E)


@pytest.mark.parametrize("op", OPS)
def test_wide_training_shape(gpu_lib, op):
    _run(op, [700, 129, 0, 1219], 1376, 4096, BF16)


@pytest.mark.parametrize("counts", [[5, 0, 300], [0, 0, 0], [1, 1, 1]])
def test_dw_accumulates(gpu_lib, counts):
    _run("dw", counts, 136, 264, F32, add=True)


@pytest.mark.parametrize("op", OPS)
def test_no_rows_at_all(gpu_lib, op):
    _run(op, [0, 0], 16, 24, F32, behind=4)
    _run(op, [0, 0], 16, 24, BF16)


def test_empty_sums_are_zero(gpu_lib):
    first = _first([2, 3])
    Y = torch.full((5, 16), MARK, device="cuda")
    _lib.sft_expert_forward(first, torch.empty((5, 0), dtype=BF16, device="cuda"),
                            torch.empty((2, 16, 0), dtype=BF16, device="cuda"), Y)
    assert not Y.any()
    dX = torch.full((5, 24), MARK, device="cuda")
    _lib.sft_expert_dx(first, torch.empty((5, 0), dtype=BF16, device="cuda"),
                       torch.empty((2, 0, 24), dtype=BF16, device="cuda"), dX)
    assert not dX.any()


@pytest.mark.parametrize("op", OPS)
def test_values_outside_a_group_do_not_reach_it(gpu_lib, op):
    # infinities and NaN in one expert's tokens and weights, at tile and stage ends that its neighbours share
    counts, R, C = [37, 21, 100], 200, 136
    first, T = _first(counts), sum(counts)
    X, dY, W = _normal((T, C), 1.0, 1), _normal((T, R), 0.1, 2), _normal((3, R, C), 0.1, 3)
    X[37:58], dY[37:58], W[1] = float("nan"), float("inf"), float("nan")
    shape = {"forward": (T, R), "dx": (T, C), "dw": (3, R, C)}[op]
    Y = torch.zeros(shape, device="cuda")
    {"forward": lambda: _lib.sft_expert_forward(first, X, W, Y), "dx": lambda: _lib.sft_expert_dx(first, dY, W, Y),
     "dw": lambda: _lib.sft_expert_dw(first, dY, X, Y)}[op]()
    bad = torch.isnan(Y)
    part = bad[1] if op == "dw" else bad[37:58]
    assert bool(part.all())
    assert int(bad.sum()) == part.numel()


@pytest.mark.parametrize("op", ["forward", "dx"])
def test_a_token_does_not_depend_on_its_group(gpu_lib, op):
    # the same row alone, in a short group and in a long one, at the same launch sizes
    R, C, T = 264, 200, 320
    W = _normal((2, R, C), 0.1, 1)
    row = _normal((1, C if op == "forward" else R), 1.0, 2)
    seen = []
    for at, counts in ((0, [1, 319]), (130, [200, 120]), (40, [41, 279])):
        x = _normal((T, row.shape[1]), 1.0, 3 + at)
        x[at] = row
        Y = torch.zeros((T, R if op == "forward" else C), device="cuda")
        (_lib.sft_expert_forward if op == "forward" else _lib.sft_expert_dx)(_first(counts), x, W, Y)
        seen.append(Y[at].clone())
    assert torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[2])


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("first", [[5, 2, 9], [-3, 4, 4], [0, 99, 7], [50, 60, 70], [2**31 - 1, -2**31, 6]])
def test_first_out_of_range_stays_inside(gpu_lib, op, first):
    # clipped into [0, T]; a group that ends before it starts is empty
    T, R, C = 8, 16, 24
    f = torch.tensor(first, dtype=torch.int64).to(torch.int32).cuda()
    X, dY, W = _normal((T, C), 1.0, 1), _normal((T, R), 0.1, 2), _normal((2, R, C), 0.1, 3)
    n = {"forward": T * R, "dx": T * C, "dw": 2 * R * C}[op]
    whole = torch.full((n + 1024,), MARK, device="cuda")
    Y = whole[512:512 + n].view({"forward": (T, R), "dx": (T, C), "dw": (2, R, C)}[op])
    {"forward": lambda: _lib.sft_expert_forward(f, X, W, Y), "dx": lambda: _lib.sft_expert_dx(f, dY, W, Y),
     "dw": lambda: _lib.sft_expert_dw(f, dY, X, Y)}[op]()
    assert bool((whole[:512] == MARK).all()) and bool((whole[512 + n:] == MARK).all())
    for e in range(2):
        lo = min(max(first[e], 0), T)
        hi = min(max(first[e + 1], lo), T)
        if op == "dw":
            _check(Y[e], dY[lo:hi].t(), X[lo:hi], "dW")
        elif e == 1 or first[2] >= first[1]:
            a, b = (X, W[e].t()) if op == "forward" else (dY, W[e])
            _check(Y[lo:hi], a[lo:hi], b, op)


def test_weights_past_32_bits(gpu_lib):
    # the last of the experts starts beyond 2^32 bytes into W and dW
    E, R, C, T = 9, 16384, 16384, 40
    counts = [0] * 7 + [3, 37]
    W = torch.zeros((E, R, C), dtype=BF16, device="cuda")
    W[7], W[8] = _normal((R, C), 0.1, 1), _normal((R, C), 0.1, 2)
    X, dY, first = _normal((T, C), 1.0, 3), _normal((T, R), 0.1, 4), _first(counts)
    Y, dX = torch.zeros((T, R), device="cuda"), torch.zeros((T, C), device="cuda")
    _lib.sft_expert_forward(first, X, W, Y)
    _lib.sft_expert_dx(first, dY, W, dX)
    for e, lo, hi in ((7, 0, 3), (8, 3, 40)):
        _check(Y[lo:hi], X[lo:hi], W[e].t(), "forward")
        _check(dX[lo:hi], dY[lo:hi], W[e], "dx")
    _lib.sft_expert_dw(first, dY, X, W)
    for e, lo, hi in ((6, 0, 0), (7, 0, 3), (8, 3, 40)):
        _check(W[e][-300:], dY[lo:hi, -300:].t(), X[lo:hi], "dw")


def test_tokens_past_32_bits(gpu_lib):
    # a token array of more than 2^32 bytes, groups at its end
    T, R, C = 1_100_000, 2048, 64
    counts = [1_099_000, 700, 300]
    first, W = _first(counts), _normal((3, R, C), 0.1, 2)
    X, Y = _normal((T, C), 1.0, 3), torch.zeros((T, R), dtype=BF16, device="cuda")
    _lib.sft_expert_forward(first, X, W, Y)
    for e, lo, hi in ((0, 1_098_900, 1_099_000), (1, 1_099_000, 1_099_700), (2, 1_099_700, T)):
        _check(Y[lo:hi], X[lo:hi], W[e].t(), "forward")
    dX = torch.zeros((T, C), device="cuda")
    _lib.sft_expert_dx(first, Y, W, dX)
    for e, lo, hi in ((0, 1_098_900, 1_099_000), (1, 1_099_000, 1_099_700), (2, 1_099_700, T)):
        _check(dX[lo:hi], Y[lo:hi], W[e], "dx")
    dW = torch.zeros((3, R, C), device="cuda")
    _lib.sft_expert_dw(first, Y, X, dW)
    for e, lo, hi in ((1, 1_099_000, 1_099_700), (2, 1_099_700, T)):
        _check(dW[e], Y[lo:hi].t(), X[lo:hi], "dw")


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("wrong", ["first", "T", "R", "strided", "out", "in type", "host"])
def test_python_refuses(gpu_lib, op, wrong):
    E, T, R, C = 2, 6, 16, 24
    first, X, dY, W = _first([3, 3]), _normal((T, C), 1.0, 1), _normal((T, R), 1.0, 2), _normal((E, R, C), 1.0, 3)
    a, b, call = {"forward": (X, W, _lib.sft_expert_forward), "dx": (dY, W, _lib.sft_expert_dx),
                  "dw": (dY, X, _lib.sft_expert_dw)}[op]
    out = torch.zeros({"forward": (T, R), "dx": (T, C), "dw": (E, R, C)}[op], device="cuda")
    if wrong == "first":
        first = first[:-1]
    elif wrong == "T":
        if op == "dw":
            b = b[:-1]
        else:
            out = out[:-1]
    elif wrong == "R":
        a = a[:, :8].contiguous()
    elif wrong == "strided":
        a = torch.cat([a, a], 1)[:, :a.shape[1]]
    elif wrong == "out":
        out = out.half()
    elif wrong == "in type":
        a = a.float()
    else:
        b = b.cpu()
    with pytest.raises((TypeError, ValueError)):
        call(first, a, b, out)


def _layer_step(first, X, W, dY, p, vec, hp, ws, clip, norm, Y, dX, dW, step):
    return [_lib.prepare_expert_forward(first, X, W, Y), _lib.prepare_expert_dx(first, dY, W, dX),
            _lib.prepare_expert_dw(first, dY, X, dW), _lib.prepare_grad_clip([dW], 0.5, clip, norm, ws),
            _lib.prepare_adamw([vec], step, hp, clip)]


@pytest.mark.parametrize("held", [False, True])
def test_training_steps_of_an_expert_layer(gpu_lib, held):
    # forward, gradients, clip and update as a training step uses them, captured once and replayed with other routings and
    # tokens, against the formulas step by step
    E, T, R, C = 5, 300, 136, 200
    X, dY, W = _normal((T, C), 1.0, 1), _normal((T, R), 0.1, 2), _normal((E, R, C), 0.1, 3)
    p = W.float()
    first = _first([0] * E)
    Y, dX, dW = (torch.zeros(s, dtype=t, device="cuda") for s, t in (((T, R), BF16), ((T, C), BF16), ((E, R, C), F32)))
    vec = _lib.AdamwVec.alloc8(p, dW, W) if held else _lib.AdamwVec(p, dW, torch.zeros_like(p), torch.zeros_like(p),
                                                                    None, W)
    hp = adam_dev(lr=1e-2, weight_decay=0.1)
    clip, norm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.empty(_lib.sft_grad_clip_workspace([dW]), dtype=torch.uint8, device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = _layer_step(first, X, W, dY, p, vec, hp, ws, clip, norm, Y, dX, dW, step)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step += 1
        for c in calls:
            c()
    rs = np.random.RandomState(0)
    m = v = torch.zeros((E, R, C), dtype=torch.float64, device="cuda")
    for t in range(1, 5):
        counts = rs.multinomial(T - 7, rs.dirichlet(np.ones(E)))
        first.copy_(_first(counts))
        X.copy_(_normal((T, C), 1.0, 10 * t))
        dY.copy_(_normal((T, R), 0.1, 10 * t + 1))
        W0, p0 = W.clone(), p.double()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        bounds = first.tolist()
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            _check(Y[lo:hi], X[lo:hi], W0[e].t(), "forward")
            _check(dX[lo:hi], dY[lo:hi], W0[e], "dx")
            _check(dW[e], dY[lo:hi].t(), X[lo:hi], "dw")
        true = dW.double().square().sum().sqrt().item()
        assert norm.item() == pytest.approx(true, rel=2 * U) and clip.item() == pytest.approx(0.5 / true, rel=2 * U)
        if not held:
            g = dW.double() * clip.double()
            m, v = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
            u = 1e-2 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
            want = p0 * (1 - 1e-3) - u
            # betas and rates are fp32 numbers and the moments' cancellations stay small against the step's size 1e-2
            assert (p.double() - want).abs().max().item() <= 1e-2 * 1e-4
        else:
            assert (p.double() - p0).abs().max().item() <= 1.2e-2
        assert torch.equal(W, p.bfloat16())


def test_two_streams_at_once(gpu_lib):
    # the calls share nothing: layers stepped on two streams at a time end as they do one after the other
    def layer(seed):
        counts, R, C = [300, 0, 129, 71], 264, 392
        T = sum(counts)
        first, W = _first(counts), _normal((4, R, C), 0.1, seed)
        X, dY = _normal((T, C), 1.0, seed + 1), _normal((T, R), 0.1, seed + 2)
        Y, dX = torch.zeros((T, R), dtype=BF16, device="cuda"), torch.zeros((T, C), dtype=BF16, device="cuda")
        dW, p = torch.zeros((4, R, C), device="cuda"), W.float()
        vec = _lib.AdamwVec.alloc8(p, dW, W)
        clip = torch.zeros(1, device="cuda")
        ws = torch.empty(_lib.sft_grad_clip_workspace([dW]), dtype=torch.uint8, device="cuda")
        hp = adam_dev(lr=1e-2)
        return (Y, dX, p, W), [_lib.prepare_expert_forward(first, X, W, Y), _lib.prepare_expert_dx(first, dY, W, dX),
                               _lib.prepare_expert_dw(first, dY, X, dW), _lib.prepare_grad_clip([dW], 0.1, clip, None, ws),
                               _lib.prepare_adamw([vec], 3, hp, clip)]

    alone, together = [layer(s) for s in (1, 50)], [layer(s) for s in (1, 50)]
    streams = [torch.cuda.Stream() for _ in alone]
    torch.cuda.synchronize()
    for _ in range(5):
        for _, calls in alone:
            for c in calls:
                c()
        torch.cuda.synchronize()
        for i in range(5):
            for s, (_, calls) in zip(streams, together):
                calls[i](s)
    torch.cuda.synchronize()
    for (a, _), (b, _) in zip(alone, together):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("op", ["forward", "dw"])
def test_gradients_agree_with_differences(gpu_lib, op):
    # <dY, Y> is linear in X and in W: a change of one of them changes it by exactly <gradient, change>
    counts, R, C = [40, 0, 25], 72, 56
    T = sum(counts)
    first = _first(counts)
    X, dY, W = _normal((T, C), 1.0, 1), _normal((T, R), 1.0, 2), _normal((3, R, C), 1.0, 3)

    def loss(x, w):
        Y = torch.zeros((T, R), device="cuda")
        _lib.sft_expert_forward(first, x, w, Y)
        return (Y.double() * dY.double()).sum().item()

    if op == "forward":
        other, grad = _normal((T, C), 1.0, 4), torch.zeros((T, C), device="cuda")
        _lib.sft_expert_dx(first, dY, W, grad)
        change, got = loss(other, W) - loss(X, W), (grad.double() * (other.double() - X.double())).sum().item()
    else:
        other, grad = _normal((3, R, C), 1.0, 4), torch.zeros((3, R, C), device="cuda")
        _lib.sft_expert_dw(first, dY, X, grad)
        change, got = loss(X, other) - loss(X, W), (grad.double() * (other.double() - W.double())).sum().item()
    # both sides are sums of T*R*C products in fp32 pieces of at most 72 terms
    assert abs(change - got) <= 4 * (72 + 4) * U * T * R * C ** 0.5 * 4


@pytest.mark.parametrize("op", OPS)
def test_arrays_behind_one_another(gpu_lib, op):
    # the results between the inputs of one buffer, not a byte apart
    counts, R, C = [3, 0, 9, 2, 2], 24, 40
    E, T = len(counts), sum(counts)
    X, dY, W = _normal((T, C), 1.0, 1), _normal((T, R), 0.1, 2), _normal((E, R, C), 0.1, 3)
    first = torch.cat([_first(counts), torch.zeros(2, dtype=torch.int32, device="cuda")])     # 32 bytes
    a, b = {"forward": (X, W), "dx": (dY, W), "dw": (dY, X)}[op]
    shape = {"forward": (T, R), "dx": (T, C), "dw": (E, R, C)}[op]
    out = torch.full(shape, MARK, device="cuda")
    parts = [x.reshape(-1).view(torch.uint8) for x in (first, a, out, b)]
    whole = torch.cat(parts)
    at = np.cumsum([0] + [p.numel() for p in parts])
    f, a1, o, b1 = (whole[at[i]:at[i + 1]].view(t).view(s) for i, (t, s) in enumerate(
        ((torch.int32, (E + 3,)), (BF16, a.shape), (F32, shape), (BF16, b.shape))))
    {"forward": _lib.sft_expert_forward, "dx": _lib.sft_expert_dx, "dw": _lib.sft_expert_dw}[op](f[:E + 1], a1, b1, o)
    assert torch.equal(a1, a) and torch.equal(b1, b)
    bounds = first.tolist()
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if op == "dw":
            _check(o[e], dY[lo:hi].t(), X[lo:hi], "dW")
        else:
            _check(o[lo:hi], a[lo:hi], W[e].t() if op == "forward" else W[e], op)


@pytest.mark.parametrize("op,counts,R,C,shape", expert_shapes.CASES)
def test_the_shape_that_the_sizes_name(gpu_lib, op, counts, R, C, shape):
    for more in (0, expert_shapes.AROUND):
        assert _lib.sft_probe_expert_tiles(op, len(counts), sum(counts) + more, R, C) == shape
    _run(op, counts, R, C, F32, start=1, behind=expert_shapes.AROUND - 1)
    _run(op, counts, R, C, F32, integer=True, seed=10)
    _run(op, counts, R, C, BF16, start=2, behind=expert_shapes.AROUND - 2, seed=20)


@pytest.mark.parametrize("counts,R,C,shape", [c[1:] for c in expert_shapes.DW])
@pytest.mark.parametrize("shift", [0, 4])
def test_dw_accumulates_on_every_shape(gpu_lib, counts, R, C, shape, shift):
    # whole numbers throughout, so that every sum is exact whatever its order: old values that were read from another
    # place, late or twice would show.  Rows of whole cache lines (old values read ahead, results past L2) and others;
    # with the array 16 bytes behind a line no row starts on one.  Rows of experts without tokens stay as they were.
    E, T = len(counts), sum(counts)
    assert _lib.sft_probe_expert_tiles("dw", E, T, R, C) == shape
    first = _first(counts)
    X, dY = ((_normal((T, n), 1.0, i) * 2).round().clamp(-3, 3) for i, n in ((1, C), (2, R)))
    gen = torch.Generator(device="cuda").manual_seed(3)
    whole = torch.randint(-100000, 100000, (E * R * C + 64,), generator=gen, device="cuda").float()
    before = whole.clone()
    D, old = (x[shift:shift + E * R * C].view(E, R, C) for x in (whole, before))
    assert D.data_ptr() % 128 == 4 * shift
    for turn in (1, 2):                                          # and once more onto the sums
        _lib.sft_expert_dw(first, dY, X, D, accumulate=True)
        for e, (lo, hi) in enumerate(zip(first.tolist(), first.tolist()[1:])):
            assert torch.equal(D[e].double(), old[e].double() + turn * (dY[lo:hi].double().t() @ X[lo:hi].double()))
    assert torch.equal(whole[:shift], before[:shift])
    assert torch.equal(whole[shift + E * R * C:], before[shift + E * R * C:])


@pytest.mark.parametrize("counts,R,C,shape", [c[1:] for c in expert_shapes.DW])
def test_dw_accumulates_ordinary_values(gpu_lib, counts, R, C, shape):
    # fp32 sums of exact products, then one addition to the old value, rounded: (rows + 5) U of the magnitudes
    T = sum(counts)
    first, X, dY = _first(counts), _normal((T, C), 1.0, 1), _normal((T, R), 0.1, 2)
    D = torch.randn((len(counts), R, C), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    old = D.clone()
    _lib.sft_expert_dw(first, dY, X, D, accumulate=True)
    for e, (lo, hi) in enumerate(zip(first.tolist(), first.tolist()[1:])):
        a, b = dY[lo:hi].t().double(), X[lo:hi].double()
        bound = (hi - lo + 5) * U * (a.abs() @ b.abs() + old[e].abs().double())
        assert bool(((D[e].double() - (old[e].double() + a @ b)).abs() <= bound).all())
        assert hi > lo or torch.equal(D[e], old[e])


def test_captured_8_bit_steps_of_an_expert_layer(gpu_lib):
    # the clipped 8-bit update behind an expert layer's gradients, captured once: every replay's weights, scales and
    # codes against the formula at that step's number, factor and gradient
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
    E, T, R, C = 5, 300, 136, 200
    X, dY, W = _normal((T, C), 1.0, 1), _normal((T, R), 0.1, 2), _normal((E, R, C), 0.1, 3)
    first, p = _first([0] * E), W.float()
    Y, dX, dW = (torch.zeros(s, dtype=t, device="cuda") for s, t in (((T, R), BF16), ((T, C), BF16), ((E, R, C), F32)))
    vec = _lib.AdamwVec.alloc8(p, dW, W)
    clip, norm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.empty(_lib.sft_grad_clip_workspace([dW]), dtype=torch.uint8, device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = _layer_step(first, X, W, dY, p, vec, adam_dev(**hp), ws, clip, norm, Y, dX, dW, step)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step += 1
        for c in calls:
            c()
    rs = np.random.RandomState(0)
    for t in range(1, 6):
        first.copy_(_first(rs.multinomial(T - 7, rs.dirichlet(np.ones(E)))))
        X.copy_(_normal((T, C), 1.0, 10 * t))
        dY.copy_(_normal((T, R), 0.1, 10 * t + 1))
        before = before_8_bit_step(vec)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert step.item() == t and 0.0 < clip.item() < 1.0
        check_8_bit_step(vec, before, dW.double().cpu(), t, hp, clip.item(), f"at step {t}")
        assert not torch.equal(p.double().cpu(), before[0])


def test_more_short_groups_than_a_launch_has_small_tiles(gpu_lib):
    # one row on each of 16384 experts of 65536 x 8: 17 million tiles of 64 x 64, more than a launch has workgroups
    E, R, C = 16384, 65536, 8
    first = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    X, W = _normal((E, C), 1.0, 1), torch.empty((E, R, C), dtype=BF16, device="cuda")
    W.normal_(0.0, 0.1, generator=torch.Generator(device="cuda").manual_seed(2))
    Y = torch.full((E, R), float("nan"), dtype=BF16, device="cuda")
    _lib.sft_expert_forward(first, X, W, Y)
    assert not torch.isnan(Y).any()
    for e in (0, 1, 63, 64, 8191, 16320, 16383):
        _check(Y[e:e + 1], X[e:e + 1], W[e].t(), f"expert {e}")
