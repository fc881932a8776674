"""GPU tests of the norms (sft_norm_forward, sft_norm_backward) against their
formulas in fp64."""
import pytest
import torch

from sparse_full_weight_amd import _lib
from tests.rowwise import BF16, F32, U, Placed, close, normal

pytestmark = pytest.mark.gpu

EPS = 1e-5
# a row's sum: at most 64 terms in a lane, 6 steps over a wave, the waves, and the quotient
SUM = 80 * U
TYPES = [(F32, F32), (BF16, BF16), (F32, BF16)]
# one below, at and above every width that a team of lanes serves, and odd ones
WIDTHS = [1, 2, 7, 8, 9, 120, 127, 128, 129, 255, 256, 257, 504, 511, 513, 1000, 1024, 1025, 1375, 2047, 2048, 2050,
          4095, 4096, 4104, 8191, 8192, 8193, 11008, 16383, 16384]


def forward64(h, gain, bias, kind, eps):
    """Y, mean, rstd in fp64, and how far fp32 arithmetic may be from them."""
    C = h.shape[1]
    mean = h.mean(1) if kind == "layer" else torch.zeros(h.shape[0], dtype=torch.float64)
    e_mean = SUM * h.abs().mean(1) if kind == "layer" else torch.zeros_like(mean)
    d = h - mean[:, None]
    var = d.square().mean(1)
    rstd = (var + eps) ** -0.5
    # the squares: twice a value's own rounding, products, sum and quotient; the mean's error counts by its square, as
    # the centred values add up to nothing; the sum with eps, root and reciprocal.  Half of a relative error of the sum
    e_rstd = rstd * (0.5 * ((2 * U + SUM + 2 * U) + rstd ** 2 * (e_mean ** 2 + 2 * e_mean * U * d.abs().mean(1))) + 3 * U)
    xhat = d * rstd[:, None]
    w = gain if gain is not None else torch.ones(C, dtype=torch.float64)
    b = bias if bias is not None else torch.zeros(C, dtype=torch.float64)
    e_xhat = rstd[:, None] * (e_mean[:, None] + U * d.abs()) + d.abs() * e_rstd[:, None] + U * xhat.abs()
    y = xhat * w + b
    e_y = w.abs() * e_xhat + U * (xhat * w).abs() + U * y.abs()
    return (y, mean, rstd), (1.01 * e_y + 1e-37, 1.01 * e_mean + U * mean.abs(), 1.01 * e_rstd)


def run_forward(T, C, kind, x_type, y_type, w_type=F32, res=False, bias=True, gain=True, pad=0, shift=0, inplace=None,
                seed=0, x=None, eps=EPS):
    x = normal((T, C), 1.5, seed, x_type, 0.4) if x is None else x
    r = normal((T, C), 2.0, seed + 1, x_type) if res else None
    w = normal((C,), 0.2, seed + 2, w_type, 1.0) if gain else None
    b = normal((C,), 0.2, seed + 3, w_type) if bias else None
    h = (x.float() + r.float()).to(x_type) if res else x
    on_x = Placed(x, pad, shift)
    on_r = Placed(r, pad + 3, shift) if res else None
    on_y = Placed(torch.zeros(T, C, dtype=y_type), 2 * pad, shift)
    on_h = {None: None, "x": on_x, "res": on_r}[inplace] if res else None
    if res and inplace is None:
        on_h = Placed(torch.zeros(T, C, dtype=x_type), pad, shift)
    mean, rstd = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    _lib.sft_norm_forward(on_x.view, None if w is None else w.cuda(), on_y.view, kind=kind, eps=eps,
                          bias=None if b is None else b.cuda(), res=on_r.view if res else None,
                          H=on_h.view if res else None, mean=mean, rstd=rstd)
    (y64, m64, r64), (ey, em, er) = forward64(h.double(), None if w is None else w.double(),
                                              None if b is None else b.double(), kind, eps)
    what = f"{T} x {C}"
    close(on_y.view, y64, ey, "Y of " + what)
    close(mean, m64, em, "mean of " + what)
    close(rstd, r64, er, "rstd of " + what)
    if res:
        assert torch.equal(on_h.view.cpu(), h), "H of " + what
    if on_x is not on_h:
        assert torch.equal(on_x.view.cpu(), x)
    if res and on_r is not on_h:
        assert torch.equal(on_r.view.cpu(), r)
    assert all(p.untouched() for p in (on_x, on_y, on_r, on_h) if p is not None)


@pytest.mark.parametrize("x_type,y_type", TYPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_of_every_width(gpu_lib, kind, x_type, y_type):
    for i, C in enumerate(WIDTHS):
        run_forward([1, 2, 3, 5, 33][i % 5], C, kind, x_type, y_type, seed=i, res=i % 2 == 0, bias=i % 3 != 0,
                    gain=i % 4 != 3, w_type=BF16 if i % 5 < 2 else F32, pad=[0, 0, 1, 8][i % 4], shift=[0, 1, 8][i % 3])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("inplace", ["x", "res"])
def test_forward_into_its_inputs(gpu_lib, inplace, dtype):
    for T, C in ((1, 4096), (70, 1001), (33, 130)):
        run_forward(T, C, "rms", dtype, BF16 if C == 130 else dtype, res=True, inplace=inplace,
                    pad=3 if inplace == "x" else 0)


def test_forward_without_what_is_optional(gpu_lib):
    x = normal((5, 200), 1.0, 1)
    y = torch.empty(5, 200, device="cuda")
    _lib.sft_norm_forward(x.cuda(), None, y, kind="layer", eps=EPS)
    (y64, _, _), (ey, _, _) = forward64(x.double(), None, None, "layer", EPS)
    close(y, y64, ey, "Y")


def test_forward_of_far_and_small_rows(gpu_lib):
    # a mean far above the spread: the squares are of centred values; tiny and huge rows; rows of equal values
    base = normal((6, 777), 1.0, 3)
    scale = torch.tensor([1.0, 1e-15, 1e15, 1.0, 1e-3, 0.0])[:, None]
    x = base * scale + torch.tensor([1000.0, 0.0, 0.0, -300.0, 5.0, 0.7])[:, None]
    run_forward(6, 777, "layer", F32, F32, x=x)
    run_forward(6, 777, "rms", F32, F32, x=x)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_of_values_that_are_not_finite(gpu_lib, kind):
    # such a row is NaN, and the rows that share its wave or workgroup are not
    for C in (9, 100, 200, 400, 1000, 4096, 16384):
        x = normal((9, C), 1.0, C)
        x[3, C // 2] = float("inf")
        x[6, 0] = float("nan")
        y = torch.empty(9, C, device="cuda")
        rstd = torch.empty(9, device="cuda")
        _lib.sft_norm_forward(x.cuda(), None, y, kind=kind, eps=EPS, rstd=rstd)
        ok = torch.tensor([i not in (3, 6) for i in range(9)])
        (y64, _, r64), (ey, _, er) = forward64(x[ok].double(), None, None, kind, EPS)
        close(y.cpu()[ok], y64, ey, "Y")
        close(rstd.cpu()[ok], r64, er, "rstd")
        assert y[6].isnan().all()
        # infinity: its own place is NaN, and all of the row where the mean is taken off; else 0
        assert y[3, C // 2].isnan() and (y[3].isnan().all() if kind == "layer" else (y[3].isnan().sum() == 1))


def test_forward_of_equal_values_without_eps(gpu_lib):
    x = torch.full((2, 300), 0.75, device="cuda")
    x[1] = 0.0
    y = torch.empty_like(x)
    _lib.sft_norm_forward(x, None, y, kind="layer", eps=0.0)
    assert y.isnan().all()
    _lib.sft_norm_forward(x, None, y, kind="rms", eps=0.0)
    assert torch.equal(y[0].cpu(), torch.ones(300)) and y[1].isnan().all()


# ------------------------------------------------------------------ backward
def backward64(h, gain, mean, rstd, dy, dh, kind, rows_depth):
    """dX, dgain, dbias in fp64 from the forward pass's statistics as they are, and bounds."""
    C = h.shape[1]
    w = gain if gain is not None else torch.ones(C, dtype=torch.float64)
    xhat = (h - mean[:, None]) * rstd[:, None]
    e_xhat = 2 * U * xhat.abs()
    g = dy * w
    along, flat = (g * xhat).mean(1, keepdim=True), g.mean(1, keepdim=True)
    # (a product with 1/C in place of the quotient: one rounding more)
    e_along = (SUM + 5 * U) * (g * xhat).abs().mean(1, keepdim=True)
    e_flat = (SUM + 3 * U) * g.abs().mean(1, keepdim=True)
    if kind != "layer":
        flat, e_flat = flat * 0, e_flat * 0
    dx = rstd[:, None] * (g - flat - xhat * along)
    e_dx = rstd[:, None] * (U * g.abs() + e_flat + xhat.abs() * e_along + along.abs() * e_xhat + U * (xhat * along).abs()
                            + 3 * U * (g.abs() + flat.abs() + (xhat * along).abs()))
    if dh is not None:
        dx = dx + dh
        e_dx = e_dx + U * dx.abs()
    dgain, dbias = (dy * xhat).sum(0), dy.sum(0)
    e_dgain = (rows_depth + 4) * U * (dy * xhat).abs().sum(0)
    e_dbias = rows_depth * U * dy.abs().sum(0)
    return (dx, dgain, dbias), (1.01 * e_dx + 1e-37, 1.01 * e_dgain + 1e-37, 1.01 * e_dbias + 1e-37)


def depth(T):
    """Additions behind one another in the sums over T <= 2048 rows: a team's rows, 32 teams, 64 workgroups a share, 8
    shares, the accumulation; never more than T - 1 and the last.  (Narrow rows, T <= 20000: at most 32 of a share, or 4
    of a team of 64 and 8 workgroups a share, and 30 to join them.)"""
    return min(T, 4 + 32 + 64 + 8) + 1


def run_backward(T, C, kind, x_type, y_type, w_type=F32, g_type=F32, dh=True, gain=True, dbias=True, dgain=True,
                 accumulate=False, pad=0, shift=0, inplace=None, seed=0):
    h = normal((T, C), 1.5, seed, x_type, 0.4)
    w = normal((C,), 0.2, seed + 2, w_type, 1.0) if gain else None
    dy = normal((T, C), 0.1, seed + 4, y_type)
    r = normal((T, C), 0.1, seed + 5, x_type) if dh else None
    (_, mean, rstd), _ = forward64(h.double(), None, None, kind, EPS)
    mean, rstd = mean.float(), rstd.float()
    on_h, on_dy = Placed(h, pad, shift), Placed(dy, 2 * pad, shift)
    on_r = Placed(r, pad + 3, shift) if dh else None
    on_dx = {None: None, "dY": on_dy, "dH": on_r}[inplace] or Placed(torch.zeros(T, C, dtype=x_type), pad, shift)
    old = normal((C,), 0.5, seed + 6) if accumulate else torch.full((C,), 3.0)
    sums = [old.cuda().to(g_type) if want else None for want in (dgain, dbias)]
    nbytes = _lib.sft_norm_backward_workspace(T, C, bias=dbias)
    ws = torch.full((nbytes // 4 + 4,), 5.0, device="cuda")[:nbytes // 4] if dgain or dbias else None
    _lib.sft_norm_backward(on_h.view, None if w is None else w.cuda(), rstd.cuda(), on_dy.view, on_dx.view, sums[0],
                           kind=kind, mean=mean.cuda() if kind == "layer" else None, dbias=sums[1],
                           dH=on_r.view if dh else None, accumulate=accumulate, ws=ws)
    want, bound = backward64(h.double(), None if w is None else w.double(), mean.double(), rstd.double(), dy.double(),
                             None if r is None else r.double(), kind, depth(T))
    what = f"{T} x {C}"
    close(on_dx.view, want[0], bound[0], "dX of " + what)
    for got, x, e, name in zip(sums, want[1:], bound[1:], ("dgain", "dbias")):
        if got is not None:
            if accumulate:
                x = x + old.double()
                e = e + U * x.abs()
            close(got, x, e, f"{name} of {what}")
    assert torch.equal(on_h.view.cpu(), h)
    assert on_dx is on_dy or torch.equal(on_dy.view.cpu(), dy)
    assert all(p.untouched() for p in (on_h, on_dy, on_dx, on_r) if p is not None)


@pytest.mark.parametrize("x_type,y_type", TYPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_of_every_width(gpu_lib, kind, x_type, y_type):
    for i, C in enumerate(WIDTHS):
        run_backward([1, 2, 37, 3, 70][i % 5], C, kind, x_type, y_type, seed=i, dh=i % 2 == 0, gain=i % 4 != 3,
                     w_type=BF16 if i % 5 < 2 else F32, dbias=i % 3 != 0, pad=[0, 0, 1, 8][i % 4], shift=[0, 1, 8][i % 3])


@pytest.mark.parametrize("T,C", [(2048, 64), (2047, 136), (1500, 500), (2048, 1024), (1021, 4096), (600, 8200)])
def test_backward_of_many_rows(gpu_lib, T, C):
    for kind in ("layer", "rms"):
        run_backward(T, C, kind, BF16, BF16, seed=T)


@pytest.mark.parametrize("T,C", [(1025, 7), (4096, 64), (4097, 64), (2048, 128), (2049, 128), (9000, 20), (20000, 96)])
def test_backward_of_thousands_of_narrow_rows(gpu_lib, T, C):
    run_backward(T, C, "layer", BF16, BF16, seed=T)
    run_backward(T, C, "rms", F32, F32, seed=T, pad=1)


@pytest.mark.parametrize("dgain,dbias", [(True, False), (False, True), (False, False)])
def test_backward_with_frozen_gains_or_biases(gpu_lib, dgain, dbias):
    for C in (100, 1000, 4096, 16000):
        run_backward(41, C, "layer", F32, F32, dgain=dgain, dbias=dbias)


def test_backward_adds_to_gradients(gpu_lib):
    for C in (9, 2000):
        run_backward(300, C, "layer", BF16, BF16, accumulate=True)
        run_backward(300, C, "rms", F32, F32, accumulate=True, dbias=False)


def test_backward_with_bf16_gradients(gpu_lib):
    run_backward(64, 4096, "layer", BF16, BF16, g_type=BF16)


@pytest.mark.parametrize("inplace", ["dY", "dH"])
def test_backward_into_its_inputs(gpu_lib, inplace):
    for T, C in ((1, 4096), (700, 1001), (33, 130)):
        run_backward(T, C, "layer", BF16, BF16, inplace=inplace, pad=3)
        run_backward(T, C, "rms", F32, F32, inplace=inplace)


def test_backward_is_the_derivative(gpu_lib):
    # central differences of a weighted sum of the fp64 forward pass, along random directions
    T, C = 6, 300
    for kind in ("layer", "rms"):
        h, w, b, dy = (normal(s, 1.0, 9 + i).double() for i, s in enumerate(((T, C), (C,), (C,), (T, C))))
        (_, mean, rstd), _ = forward64(h, w, b, kind, EPS)
        dx, dgain, dbias = (torch.zeros(s, device="cuda") for s in ((T, C), (C,), (C,)))
        ws = torch.empty(_lib.sft_norm_backward_workspace(T, C, bias=True), dtype=torch.uint8, device="cuda")
        _lib.sft_norm_backward(h.float().cuda(), w.float().cuda(), rstd.float().cuda(), dy.float().cuda(), dx, dgain,
                               kind=kind, mean=mean.float().cuda() if kind == "layer" else None, dbias=dbias, ws=ws)
        for grad, at in ((dx, 0), (dgain, 1), (dbias, 2)):
            v = normal(grad.shape, 1.0, 77 + at).double()

            def loss(t):
                moved = [x + t * v if i == at else x for i, x in enumerate((h, w, b))]
                return float((forward64(*moved, kind, EPS)[0][0] * dy).sum())

            slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
            got = float((grad.cpu().double() * v).sum())
            size = float((grad.cpu().double() * v).abs().sum())
            # the difference's own error is of the order of 1e-10, fp32 values and statistics count a few U each
            assert abs(got - slope) <= 1e-6 * size + 1e-7


def test_no_rows(gpu_lib):
    empty = torch.empty(0, 100, device="cuda")
    g = torch.ones(100, device="cuda")
    none = torch.empty(0, device="cuda")
    _lib.sft_norm_forward(empty, g, empty, kind="rms")
    assert _lib.sft_norm_backward_workspace(0, 100) == 0
    dgain, dbias = torch.full((100,), 3.0, device="cuda"), torch.full((100,), 3.0, device="cuda")
    _lib.sft_norm_backward(empty, g, none, empty, empty, dgain, kind="rms", dbias=dbias, accumulate=True)
    assert (dgain == 3.0).all() and (dbias == 3.0).all()
    _lib.sft_norm_backward(empty, g, none, empty, empty, dgain, kind="rms", dbias=dbias)
    assert (dgain == 0.0).all() and (dbias == 0.0).all()


def test_more_rows_than_a_launch_has_workgroups(gpu_lib):
    T = 16 * (1 << 21) + 21          # 16 rows a workgroup
    x = torch.randn(T, 2, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    y = torch.zeros_like(x)
    _lib.sft_norm_forward(x, None, y, kind="rms", eps=0.0)
    for at in (0, 1 << 24, T - 40):
        rows = x[at:at + 40].cpu()
        (y64, _, _), (ey, _, _) = forward64(rows.double(), None, None, "rms", 0.0)
        close(y[at:at + 40], y64, ey, f"rows from {at}")
    dx, dgain, rstd = torch.zeros_like(x), torch.zeros(2, device="cuda"), x.double().square().mean(1).rsqrt().float()
    ws = torch.empty(_lib.sft_norm_backward_workspace(T, 2), dtype=torch.uint8, device="cuda")
    _lib.sft_norm_backward(x, None, rstd, y, dx, dgain, kind="rms", ws=ws)
    # dY = xhat: their product's sum over the rows; at least 128 teams of rows side by side
    want = (y.double() * x.double() * rstd.double()[:, None]).sum(0).cpu()
    assert ((dgain.cpu().double() - want).abs() <= (T / 128 + 200) * U * want).all()


def test_offsets_past_32_bits(gpu_lib):
    # rows 1.2 GB apart
    T, C, ld = 5, 100, 300_000_001
    big = [torch.empty(T * ld, device="cuda").view(T, ld)[:, :C] for _ in range(2)]
    x = normal((T, C), 1.0, 4)
    big[0].copy_(x)
    _lib.sft_norm_forward(big[0], None, big[1], kind="layer", eps=EPS)
    (y64, mean, rstd), (ey, _, _) = forward64(x.double(), None, None, "layer", EPS)
    close(big[1].cpu(), y64, ey, "Y")
    dx = torch.empty(T, C, device="cuda")
    mean, rstd = mean.float(), rstd.float()
    _lib.sft_norm_backward(big[0], None, rstd.cuda(), big[1], dx, None, kind="layer", mean=mean.cuda())
    y = big[1].cpu().double()
    want, bound = backward64(x.double(), None, mean.double(), rstd.double(), y, None, "layer", 1)
    close(dx, want[0], bound[0], "dX")


def test_the_same_results_every_time(gpu_lib):
    x, dy = (normal((1000, 4096), 1.0, s, BF16).cuda() for s in (1, 2))
    rstd = torch.ones(1000, device="cuda")
    ws = torch.empty(_lib.sft_norm_backward_workspace(1000, 4096), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(3):
        dx, dgain = torch.empty_like(x), torch.empty(4096, device="cuda")
        _lib.sft_norm_backward(x, None, rstd, dy, dx, dgain, kind="rms", ws=ws)
        first = first or (dx, dgain)
        assert torch.equal(dx, first[0]) and torch.equal(dgain, first[1])
    # a row's results do not depend on the other rows
    one = torch.empty(1, 4096, dtype=BF16, device="cuda")
    _lib.sft_norm_backward(x[77:78], None, rstd[:1], dy[77:78], one, None, kind="rms")
    assert torch.equal(one[0], first[0][77])


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_of_rows_whose_squares_leave_fp32(gpu_lib, kind):
    # among ordinary rows some whose squares or sums overflow (as bf16 can hold them, too), and, without eps, some whose
    # squares underflow; every kind of team, and rows of H that replaced the ones of X
    for i, C in enumerate((9, 100, 200, 400, 1000, 1024, 2000, 4096, 12000, 16384)):
        scale = torch.ones(9)
        scale[2], scale[3], scale[4], scale[7] = 1e19, 3e25, 1e37, 4e18
        for x_type, y_type in TYPES:
            x = (normal((9, C), 1.0, C) * scale[:, None]).to(x_type)
            run_forward(9, C, kind, x_type, y_type, x=x, pad=i % 3)
            run_forward(9, C, kind, x_type, y_type, x=x, res=True, inplace=[None, "x", "res"][i % 3])
        scale[2], scale[3], scale[4], scale[7] = 1e-20, 1e-26, 1e-33, 1e12
        for x_type, y_type in TYPES:
            x = (normal((9, C), 1.0, C) * scale[:, None]).to(x_type)
            run_forward(9, C, kind, x_type, y_type, x=x, pad=i % 3, eps=0.0)


def test_backward_of_rows_whose_squares_leave_fp32(gpu_lib):
    # the statistics of the forward pass serve the backward pass, at such rows as well
    T, C = 9, 1000
    for kind in ("layer", "rms"):
        scale = torch.ones(9)
        scale[2], scale[3], scale[7] = 1e19, 3e25, 1e30
        h = normal((T, C), 1.0, 3) * scale[:, None]
        dy = normal((T, C), 0.1, 4)
        y, mean, rstd = torch.empty(T, C, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        _lib.sft_norm_forward(h.cuda(), None, y, kind=kind, eps=EPS, mean=mean, rstd=rstd)
        dx, dgain = torch.empty(T, C, device="cuda"), torch.empty(C, device="cuda")
        ws = torch.empty(_lib.sft_norm_backward_workspace(T, C), dtype=torch.uint8, device="cuda")
        _lib.sft_norm_backward(h.cuda(), None, rstd, dy.cuda(), dx, dgain, kind=kind, mean=mean, ws=ws)
        want, bound = backward64(h.double(), None, mean.cpu().double(), rstd.cpu().double(), dy.double(), None, kind, depth(T))
        close(dx, want[0], bound[0], "dX")
        close(dgain, want[1], bound[1], "dgain")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_gradients_are_those_of_a_separate_array(gpu_lib, dtype):
    # dX bit by bit; the sums over the rows the same on every call, and within their bound of one another
    for T, C in ((37, 1375), (700, 300), (1024, 2048), (3000, 64), (2000, 3000)):
        h, dy, dh = (normal((T, C), 1.0, s, dtype).cuda() for s in (1, 2, 3))
        mean, rstd = h.float().mean(1), torch.ones(T, device="cuda")
        ws = torch.empty(_lib.sft_norm_backward_workspace(T, C, bias=True), dtype=torch.uint8, device="cuda")

        def call(place):
            g, r = dy.clone(), dh.clone()
            dx = {"apart": torch.empty_like(h), "dY": g, "dH": r}[place]
            sums = [torch.empty(C, device="cuda") for _ in range(2)]
            _lib.sft_norm_backward(h, None, rstd, g, dx, sums[0], kind="layer", mean=mean, dbias=sums[1], dH=r, ws=ws)
            return [dx, *sums]

        apart = call("apart")
        size = [(dy.double() * (h.double() - mean.double()[:, None])).abs().sum(0), dy.double().abs().sum(0)]
        for place in ("dY", "dH"):
            first = call(place)
            assert all(torch.equal(a, b) for a, b in zip(first, call(place))), (T, C, place)
            assert torch.equal(first[0], apart[0]), (T, C, place)
            for a, b, s in zip(first[1:], apart[1:], size):
                # at most T additions each, and two roundings of a product
                assert ((a.double() - b.double()).abs() <= 2 * (min(T, 200) + 4) * U * s).all(), (T, C, place)
                assert place != "dH" or torch.equal(a, b)


@pytest.mark.parametrize("T,C,dtype", [(8300, 1100, BF16), (8300, 600, F32), (4200, 2050, BF16), (4200, 2048, F32),
                                       (4130, 4100, BF16)])
def test_forward_of_more_rows_than_workgroups_that_share_sums(gpu_lib, T, C, dtype):
    # teams of several waves, past the 16 workgroups a CU of a launch: the places of their sums by turns
    run_forward(T, C, "layer", dtype, dtype, seed=T)
    run_forward(T, C, "rms", dtype, BF16, seed=C, res=True)


@pytest.mark.parametrize("T,C", [(16 * (1 << 21) + 21, 2), (600_007, 40), (100_003, 200), (70_001, 505), (40_001, 1000),
                                 (20_011, 2050), (9001, 4096), (3001, 8192), (2001, 12000), (1100, 16384)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_row_counts_once_in_the_gradients(gpu_lib, T, C, dtype):
    # small whole numbers, so that the sums over the rows are exact in any order: a row left out or taken twice, of a last
    # turn that not all teams have, shows
    g = torch.Generator("cuda").manual_seed(T)
    h = torch.randint(-2, 3, (T, C), device="cuda", generator=g, dtype=torch.int8)
    dy = torch.randint(-1, 2, (T, C), device="cuda", generator=g, dtype=torch.int8)
    dy[-3:] = 1                              # the last rows count for certain
    want_gain, want_bias = torch.zeros(2, C, dtype=torch.int64, device="cuda")
    for at in range(0, T, 1 << 20):
        a, b = h[at:at + (1 << 20)].long(), dy[at:at + (1 << 20)].long()
        want_gain, want_bias = want_gain + (a * b).sum(0), want_bias + b.sum(0)
    h, dy = h.to(dtype), dy.to(dtype)
    dx, rstd, mean = torch.empty_like(h), torch.ones(T, device="cuda"), torch.zeros(T, device="cuda")
    dgain, dbias = torch.empty(2, C, device="cuda")
    ws = torch.empty(_lib.sft_norm_backward_workspace(T, C, bias=True), dtype=torch.uint8, device="cuda")
    for kind in ("rms", "layer"):
        _lib.sft_norm_backward(h, None, rstd, dy, dx, dgain, kind=kind, mean=mean if kind == "layer" else None,
                               dbias=dbias, ws=ws)
        assert torch.equal(dgain.long(), want_gain) and torch.equal(dgain, dgain.round())
        assert torch.equal(dbias.long(), want_bias) and torch.equal(dbias, dbias.round())
        for at in range(0, T, 1 << 18):
            x, d, got = (t[at:at + (1 << 18)].double() for t in (h, dy, dx))
            along, flat = (x * d).mean(1, keepdim=True), d.mean(1, keepdim=True) * (kind == "layer")
            want = d - x * along - flat
            # exact sums; the quotients' two roundings each, a product, two differences
            bound = 4 * U * ((x * along).abs() + flat.abs()) + 3 * U * (d.abs() + (x * along).abs() + flat.abs())
            if dtype == BF16:
                bound = bound + 2.0 ** -8 * (want.abs() + bound)
            assert ((got - want).abs() <= bound).all(), (kind, at)
    # frozen biases take the other instance
    _lib.sft_norm_backward(h, None, rstd, dy, dx, dgain, kind="rms", ws=ws)
    assert torch.equal(dgain.long(), want_gain)
