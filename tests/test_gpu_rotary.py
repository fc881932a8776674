"""GPU tests of rotary positions (sft_rotary) against the rotation in fp64 with
angles in extended precision."""
import numpy as np
import pytest
import torch

from sparse_full_weight_amd import _lib
from tests.rowwise import BF16, F32, MARK, U, close, normal

pytestmark = pytest.mark.gpu

SIZES = [(2, 2), (3, 2), (4, 2), (8, 8), (10, 6), (16, 16), (18, 14), (33, 32), (50, 20), (64, 64), (80, 20), (96, 96),
         (128, 128), (128, 64), (256, 64), (257, 100), (512, 512)]


def rotate64(x, pos, freq, rot, layout, inverse, amplitude):
    """The rotation of x [B, T, heads, D] (fp64), with what fp32 arithmetic may differ by."""
    angle = pos.numpy().astype(np.longdouble)[..., None] * freq.astype(np.longdouble)
    if inverse:
        angle = -angle
    c, s = (torch.from_numpy(f(angle).astype(np.float64))[:, :, None] for f in (np.cos, np.sin))
    # three roundings in fp64 on the way to the turns; the reduced turns in fp32 (half a turn at most: pi * U), 2 units in
    # the last place for each function, amplitude
    e = (np.pi + 4 + 1) * U + 3 * 2.0 ** -53 * torch.from_numpy(np.abs(angle).astype(np.float64))[:, :, None]
    half = rot // 2
    at = (slice(0, half), slice(half, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x[..., at[0]], x[..., at[1]]
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., at[0]] = amplitude * (u * c - v * s)
    y[..., at[1]] = amplitude * (u * s + v * c)
    size = abs(amplitude) * (u.abs() + v.abs())
    bound[..., at[0]] = bound[..., at[1]] = 1.01 * size * (e + 2 * U) + 1e-37
    return y, bound


def check(y, x, pos, freq, rot, layout, inverse=False, amplitude=1.0, what=""):
    want, bound = rotate64(x.double(), pos, freq, rot, layout, inverse, amplitude)
    close(y, want, bound, what)
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:]), what + ": elements behind the turned part"


def table(rot, **kw):
    freq = _lib.sft_rotary_table(rot, **kw)
    return freq, torch.from_numpy(freq).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_sizes(gpu_lib, layout, dtype):
    for i, (D, rot) in enumerate(SIZES):
        B, T, H, K = [(1, 1, 1, 1), (2, 3, 4, 1), (1, 7, 5, 3), (3, 5, 12, 4), (2, 40, 3, 1)][i % 5]
        freq, on_freq = table(rot)
        pos = torch.randint(0, 5000, (B, T), generator=torch.Generator().manual_seed(i), dtype=torch.int32)
        q, k = normal((B, T, H, D), 1.0, i, dtype), normal((B, T, K, D), 1.0, i + 50, dtype)
        out = [torch.full(x.shape, MARK, dtype=dtype, device="cuda") for x in (q, k)]
        _lib.sft_rotary([(q.cuda(), out[0]), (k.cuda(), out[1])], pos.cuda(), on_freq, rot, layout=layout,
                        inverse=i % 2 == 1, amplitude=[1.0, 1.25][i % 2])
        for x, y in zip((q, k), out):
            check(y, x, pos, freq, rot, layout, i % 2 == 1, [1.0, 1.25][i % 2], f"D = {D}, rot = {rot}")


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("inplace", [True, False])
def test_heads_side_by_side(gpu_lib, inplace, dtype, layout):
    # queries, keys and values of a token in one row of a wider buffer, in place or out of it
    B, T, H, K, D, rot = 2, 9, 6, 2, 36, 20
    whole = normal((B, T, (H + 2 * K) * D + 5), 1.0, 3, dtype)
    on = whole.cuda()

    def heads(w):
        rows = w[:, :, :(H + 2 * K) * D].unflatten(-1, (H + 2 * K, D))
        return rows[:, :, :H], rows[:, :, H:H + K]

    freq, on_freq = table(rot)
    pos = torch.arange(B * T, dtype=torch.int32).view(B, T) * 3
    out = heads(on) if inplace else [torch.empty(x.shape, dtype=dtype, device="cuda") for x in heads(on)]
    _lib.sft_rotary(list(zip(heads(on), out)), pos.cuda(), on_freq, rot, layout=layout)
    for x, y in zip(heads(whole), out):
        check(y, x, pos, freq, rot, layout)
    left = on.cpu()
    if inplace:
        assert torch.equal(left[:, :, (H + K) * D:], whole[:, :, (H + K) * D:])
    else:
        assert torch.equal(left, whole)


def test_heads_before_tokens(gpu_lib):
    # [B, heads, T, D] tensors, seen as [B, T, heads, D]; a 3-D call without sequences
    B, T, H, D = 2, 11, 3, 64
    x = normal((B, H, T, D), 1.0, 5, BF16)
    freq, on_freq = table(D)
    pos = torch.arange(T, dtype=torch.int32) + 1000
    on = x.cuda()
    y = torch.empty_like(on)
    _lib.sft_rotary([(on.transpose(1, 2), y.transpose(1, 2))], pos.cuda(), on_freq, D)
    check(y.transpose(1, 2), x.transpose(1, 2), pos.expand(B, T), freq, D, "half")
    y3 = torch.empty(T, H, D, dtype=BF16, device="cuda")
    _lib.sft_rotary([(on[1].transpose(0, 1), y3)], pos.cuda(), on_freq, D)
    assert torch.equal(y3, y[1].transpose(0, 1))
    # in place, too
    _lib.sft_rotary([(on.transpose(1, 2), on.transpose(1, 2))], pos.cuda(), on_freq, D)
    assert torch.equal(on, y)


def test_positions_of_each_sequence_and_far_ones(gpu_lib):
    B, T, H, D = 3, 4, 2, 128
    freq, on_freq = table(D, base=500000.0, scaling="bands", factor=32.0, context=8192.0)
    pos = torch.tensor([[0, 1, 2, 3], [131071, 1 << 20, -5, (1 << 24) + 1], [2 ** 31 - 1, -2 ** 31, 123456789, 7]],
                       dtype=torch.int32)
    x = normal((B, T, H, D), 1.0, 8)
    y = torch.empty(B, T, H, D, device="cuda")
    rows = torch.zeros(B, 9, dtype=torch.int32, device="cuda")
    rows[:, :T] = pos.cuda()
    _lib.sft_rotary([(x.cuda(), y)], rows[:, :T], on_freq, D, amplitude=1.1)     # rows of pos lie apart
    check(y, x, pos, freq, D, "half", amplitude=float(np.float32(1.1)))


def test_inverse_undoes_and_is_the_gradient(gpu_lib):
    T, H, D, rot = 33, 3, 40, 24
    freq, on_freq = table(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 77
    for layout in ("half", "pairs"):
        x, g = normal((T, H, D), 1.0, 1).cuda(), normal((T, H, D), 1.0, 2).cuda()
        y, back, gx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        _lib.sft_rotary([(x, y)], pos, on_freq, rot, layout=layout)
        _lib.sft_rotary([(y, back)], pos, on_freq, rot, layout=layout, inverse=True)
        # either way each value is off by the bound of one call, on values of at most |u| + |v|
        assert (back - x).abs().max() <= 2 * (np.pi + 8) * U * 2 * x.abs().max()
        # <g, R x> = <R^T g, x>
        _lib.sft_rotary([(g, gx)], pos, on_freq, rot, layout=layout, inverse=True, amplitude=1.5)
        left, right = 1.5 * (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
        tail = (g[..., rot:].double() * x[..., rot:].double()).sum()          # not scaled
        left = left - 0.5 * tail
        size = (g.double().norm() * x.double().norm())
        assert abs(float(left - right)) <= 20 * U * float(size)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_tokens_and_heads(gpu_lib, dtype):
    # several tokens a workgroup with a last short one, and more items of a token than a workgroup's threads
    for T, H, K, D, rot in ((1000, 1, 1, 16, 16), (77, 2, 1, 64, 32), (3, 200, 7, 128, 128), (2, 3, 1, 4096, 4096),
                            (2, 3, 1, 4095, 2)):
        freq, on_freq = table(rot)
        pos = torch.arange(T, dtype=torch.int32)[None]
        q, k = normal((1, T, H, D), 1.0, T, dtype), normal((1, T, K, D), 1.0, T + 1, dtype)
        out = [torch.empty(x.shape, dtype=dtype, device="cuda") for x in (q, k)]
        _lib.sft_rotary([(q.cuda(), out[0]), (k.cuda(), out[1])], pos[0].cuda(), on_freq, rot, layout="pairs")
        for x, y in zip((q, k), out):
            check(y, x, pos, freq, rot, "pairs", what=f"{T} x {H} x {D}")


def test_unaligned_and_eight_arrays(gpu_lib):
    freq, on_freq = table(6)
    pos = torch.arange(5, dtype=torch.int32)[None]
    arrays, xs = [], []
    for i in range(8):
        x = normal((1, 5, i + 1, 10), 1.0, i, BF16)
        xs.append(x)
        room = torch.full((x.numel() + 9,), MARK, dtype=BF16, device="cuda")
        on = torch.empty(x.numel() + 1, dtype=BF16, device="cuda")[1:].view(x.shape)
        on.copy_(x)
        arrays.append((on, room[i:i + x.numel()].view(x.shape)))
    _lib.sft_rotary(arrays, pos.cuda(), on_freq, 6)
    for x, (_, y) in zip(xs, arrays):
        check(y, x, pos, freq, 6, "half")
        room = y._base
        i = y.storage_offset()
        assert (room[:i] == MARK).all() and (room[i + x.numel():] == MARK).all()


def test_nothing_to_turn(gpu_lib):
    _, on_freq = table(8)
    empty = torch.empty(0, 3, 8, device="cuda")
    _lib.sft_rotary([(empty, empty)], torch.empty(0, dtype=torch.int32, device="cuda"), on_freq, 8)
    x = torch.ones(2, 3, 8, device="cuda")
    y = torch.zeros_like(x)
    none = torch.empty(2, 0, 8, device="cuda")
    _lib.sft_rotary([(none, none), (x, y)], torch.zeros(2, dtype=torch.int32, device="cuda"), on_freq, 8)
    assert torch.equal(x, y)          # position 0


def test_offsets_past_32_bits(gpu_lib):
    D, far = 64, 1_200_000_001        # 2.4 GB between the tokens
    freq, on_freq = table(D)
    big = torch.empty(2 * far + 2 * D, dtype=BF16, device="cuda")
    view = torch.as_strided(big, (1, 3, 2, D), (0, far, D, 1))
    x = normal((1, 3, 2, D), 1.0, 6, BF16)
    view.copy_(x)
    pos = torch.tensor([[5, 6, 7]], dtype=torch.int32)
    y = torch.empty(1, 3, 2, D, dtype=BF16, device="cuda")
    _lib.sft_rotary([(view, y)], pos.cuda(), on_freq, D)
    check(y, x, pos, freq, D, "half")
    _lib.sft_rotary([(view, view)], pos.cuda(), on_freq, D)
    assert torch.equal(view, y)


@pytest.mark.parametrize("inverse", [False, True])
def test_far_positions_are_as_good_as_near_ones(gpu_lib, inverse):
    # positions over the whole range of int32 whose angle is close to a whole number of half turns: there a sine is as small
    # as the distance, and shows what the angle is off by
    cand = np.random.default_rng(5).integers(-2 ** 31, 2 ** 31, 2_000_000)
    sine = np.sin(cand.astype(np.longdouble))
    pos = cand[np.abs(sine) < 5e-4]
    assert len(pos) > 300 and np.abs(pos).max() > 2 ** 30
    T = len(pos)
    freq, on_freq = table(2)          # one radian a position
    x = torch.zeros(T, 1, 2, device="cuda")
    x[..., 0] = 1.0
    y = torch.empty_like(x)
    _lib.sft_rotary([(x, y)], torch.from_numpy(pos.astype(np.int32)).cuda(), on_freq, 2, inverse=inverse)
    want = np.sin(pos.astype(np.longdouble)).astype(np.float64) * (-1 if inverse else 1)
    # relative: the reduced turns in fp32, 2 units in the last place of the sine, the product; 2 ** -33 of the angle here.
    # Close to half a turn, where the cosine is negative, twice the turns are a number in [1/2, 1], which fp32 holds to
    # 2 ** -25: pi times that of the angle, whatever the distance
    far_side = np.cos(pos.astype(np.longdouble)) < 0
    bound = 8 * U * np.abs(want) + 1e-9 + 1.01 * np.pi * U / 2 * far_side
    assert (np.abs(y[:, 0, 1].cpu().double().numpy() - want) <= bound).all()


def test_more_workgroups_than_a_launch_has(gpu_lib):
    # tokens of 16 elements, 64 of them a workgroup: more than 2^23 workgroups, in place (17 GB)
    B, T, D = 1 << 10, (1 << 19) + 3, 16
    freq, on_freq = table(D)
    x = torch.empty(B, T, 1, D, dtype=BF16, device="cuda")
    row = torch.arange(T, device="cuda", dtype=torch.int32)
    for b in range(0, B, 64):
        x[b:b + 64] = torch.randn(64, T, 1, D, dtype=BF16, device="cuda",
                                  generator=torch.Generator("cuda").manual_seed(b))
    at = [(0, 0), (0, 70), (511, 12345), (B - 1, T - 70), (B - 1, T - 3)]
    at += [(b, (t * 7919) % (T - 3)) for b, t in zip(range(0, B, 8), range(128))]
    before = torch.stack([x[b, t:t + 3] for b, t in at]).cpu()
    _lib.sft_rotary([(x, x)], row, on_freq, D)
    after = torch.stack([x[b, t:t + 3] for b, t in at])
    pos = torch.stack([row[t:t + 3] for _, t in at]).cpu()
    check(after, before, pos, freq, D, "half")
