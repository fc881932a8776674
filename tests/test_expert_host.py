"""CPU tests of the products grouped by expert (sft_expert_forward, _dx, _dw):
what they refuse, before anything is launched."""
import numpy as np
import pytest

from sparse_full_weight_amd import _lib
from tests import expert_shapes

BUF = np.zeros(1 << 12, np.uint8)
BASE = (BUF.ctypes.data + 255) // 256 * 256
GOOD = dict(E=2, T=3, R=8, C=16, first=BASE, a=BASE + 256, b=BASE + 512, out=BASE + 1024, type=0)


def _call(op, **kw):
    k = {**GOOD, **kw}
    args = [k["E"], k["T"], k["R"], k["C"], k["first"], k["a"], k["b"], k["out"], k["type"]]
    if op == "dw":
        args.append(k.get("accumulate", 0))
    return getattr(_lib.lib(), "sft_expert_" + op)(*args, None)


@pytest.mark.parametrize("op", ["forward", "dx", "dw"])
@pytest.mark.parametrize("kw,code", [
    (dict(E=-1), _lib.SFT_EINVAL), (dict(T=-1), _lib.SFT_EINVAL), (dict(R=-8), _lib.SFT_EINVAL),
    (dict(C=-8), _lib.SFT_EINVAL), (dict(type=2), _lib.SFT_EINVAL), (dict(type=-1), _lib.SFT_EINVAL),
    (dict(R=12), _lib.SFT_ESHAPE), (dict(C=4), _lib.SFT_ESHAPE),
    (dict(T=1 << 30), _lib.SFT_ENOTSUP), (dict(E=65537), _lib.SFT_ENOTSUP),
    (dict(R=(1 << 20) + 8), _lib.SFT_ENOTSUP), (dict(C=(1 << 20) + 8), _lib.SFT_ENOTSUP),
    (dict(first=None), _lib.SFT_EINVAL), (dict(a=None), _lib.SFT_EINVAL), (dict(b=None), _lib.SFT_EINVAL),
    (dict(out=None), _lib.SFT_EINVAL), (dict(first=BASE + 2), _lib.SFT_EALIGN), (dict(a=BASE + 8), _lib.SFT_EALIGN),
    (dict(b=BASE + 2), _lib.SFT_EALIGN), (dict(out=BASE + 4), _lib.SFT_EALIGN),
    (dict(E=65536, T=(1 << 30) - 1, R=1 << 20, C=1 << 20), _lib.SFT_ENOTSUP),     # 2^31 tiles
])
def test_refuses(op, kw, code):
    assert _call(op, **kw) == code
    assert _lib.lib().sft_last_error()


@pytest.mark.parametrize("kw", [dict(E=65536, R=8, C=65536), dict(E=65536, R=1 << 20, C=8, accumulate=1)])
def test_weight_gradients_in_too_many_tiles(kw):
    assert _call("dw", **kw) == _lib.SFT_ENOTSUP


def test_dw_accumulates_only_fp32():
    assert _call("dw", type=1, accumulate=1) == _lib.SFT_EINVAL


@pytest.mark.parametrize("op,empty", [("forward", "ETR"), ("dx", "ETC"), ("dw", "ERC")])
def test_nothing_to_write_is_nothing(op, empty):
    for name in empty:
        assert _call(op, **{name: 0}, first=None, a=None, b=None, out=None) == _lib.SFT_OK


# bytes of the arrays at E = 2, T = 4, R = 8, C = 16 with fp32 results
BYTES = {"forward": dict(first=12, a=128, b=512, out=128), "dx": dict(first=12, a=64, b=512, out=256),
         "dw": dict(first=12, a=64, b=128, out=1024)}


@pytest.mark.parametrize("op", ["forward", "dx", "dw"])
@pytest.mark.parametrize("which", ["first", "a", "b"])
@pytest.mark.parametrize("end", ["the results' first bytes", "the results' last bytes"])
def test_refuses_results_over_an_input(op, which, end):
    size = BYTES[op]
    k = dict(T=4, first=BASE + 256, a=BASE + 512, b=BASE + 1024, out=BASE + 2048)
    k[which] = k["out"] + (16 - (size[which] + 15) // 16 * 16 if "first" in end else size["out"] - 16)
    assert k[which] < k["out"] + size["out"] and k["out"] < k[which] + size[which]
    assert _call(op, **k) == _lib.SFT_EINVAL
    assert b"overlap" in _lib.lib().sft_last_error()


@pytest.mark.parametrize("op,counts,R,C,shape", expert_shapes.CASES)
def test_sizes_of_the_gpu_tests_take_the_shapes_they_name(op, counts, R, C, shape):
    for more in (0, expert_shapes.AROUND):
        assert _lib.sft_probe_expert_tiles(op, len(counts), sum(counts) + more, R, C, 256) == shape


def test_every_shape_has_a_size():
    for op, shapes in expert_shapes.SHAPES.items():
        assert {c[4] for c in expert_shapes.CASES if c[0] == op} == shapes
    # and the last launch round of the largest tiles comes whole and in halves
    for cases in (expert_shapes.FORWARD, expert_shapes.DX):
        assert {expert_shapes.halved(*c) for c in cases if c[4][0] == 256} == {True, False}


def test_no_size_takes_a_shape_without_a_kernel():
    # the choice over many sizes stays within the shapes that are tested
    rs = np.random.RandomState(0)
    seen = {op: set() for op in expert_shapes.SHAPES}
    for _ in range(6000):
        E, T = int(2 ** rs.uniform(0, 10)), int(2 ** rs.uniform(0, 18))
        R, C = (8 * int(2 ** rs.uniform(0, 12)) for _ in range(2))
        for op in seen:
            try:
                seen[op].add(_lib.sft_probe_expert_tiles(op, E, T, R, C, int(rs.choice([64, 256, 304]))))
            except _lib.SftError as e:
                assert e.code == _lib.SFT_ENOTSUP
    assert seen == expert_shapes.SHAPES


@pytest.mark.parametrize("args,code", [
    ((3, 1, 1, 8, 8, 0), _lib.SFT_EINVAL), ((-1, 1, 1, 8, 8, 0), _lib.SFT_EINVAL), ((0, 1, 1, 8, 8, -1), _lib.SFT_EINVAL),
    ((0, 0, 1, 8, 8, 0), _lib.SFT_EINVAL), ((1, 1, 0, 8, 8, 0), _lib.SFT_EINVAL), ((0, 1, 1, 12, 8, 0), _lib.SFT_ESHAPE),
    ((0, 1, 1 << 30, 8, 8, 0), _lib.SFT_ENOTSUP)])
def test_probe_of_the_tiles_refuses(args, code):
    out = np.zeros(4, np.int32)
    assert _lib.lib().sft_probe_expert_tiles(*args, out.ctypes.data) == code
    assert _lib.lib().sft_probe_expert_tiles(0, 1, 1, 8, 8, 0, None) == _lib.SFT_EINVAL


@pytest.mark.parametrize("op,E,T,R,C,shape", [
    # 2^24 tiles or more of the shape that the number of rows asks for, fewer of a larger one
    ("forward", 16384, 16384, 65536, 8, (128, 192, 64, 2)), ("forward", 65536, 1 << 20, 16384, 8, (128, 192, 64, 2)),
    ("forward", 8192, 1 << 20, 1 << 17, 8, (128, 192, 64, 2)),              # 128 x 128 for 128 rows on average
    # fewer than 2^24 anyway
    ("forward", 16384, 16384, 64000, 8, (64, 64, 64, 4)), ("dx", 16384, 16384, 8, 65536, (128, 192, 64, 2)),
])
def test_many_tiles_take_a_shape_that_fits_a_launch(op, E, T, R, C, shape):
    assert _lib.sft_probe_expert_tiles(op, E, T, R, C, 256) == shape


@pytest.mark.parametrize("op,E,T,R,C", [
    ("forward", 65536, 1 << 20, 1 << 18, 8), ("dx", 65536, 1 << 20, 8, 1 << 18), ("dw", 65536, 1, 8, 65536)])
def test_more_tiles_than_a_launch_has_workgroups(op, E, T, R, C):
    with pytest.raises(_lib.SftError) as e:
        _lib.sft_probe_expert_tiles(op, E, T, R, C, 256)
    assert e.value.code == _lib.SFT_ENOTSUP
    assert _call(op, E=E, T=T, R=R, C=C) == _lib.SFT_ENOTSUP
