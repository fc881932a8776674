"""CPU tests of the dense optimizer calls (sft_grad_clip, sft_adamw): what
they refuse, before anything is launched."""
import ctypes as C

import numpy as np
import pytest

from sparse_full_weight_amd import _lib

BUF = np.zeros(1 << 14, np.uint8)
BASE = (BUF.ctypes.data + 255) // 256 * 256
HP = (0.1, 0.9, 0.999, 1e-8, 0.0, BASE + 8192, BASE + 8192, 4)


def _vec(n=16, at=BASE, scale=None, live=None, p_type=0, g_type=0):
    return _lib.CAdamwVec(n, at, at + 1024, at + 2048, at + 3328, scale, live, p_type, g_type)


def _adamw(vecs, step=1, hp=HP, clip=None, step_dev=None):
    arr = (_lib.CAdamwVec * max(len(vecs), 1))(*vecs)
    h = _lib.CAdam(*hp)
    return _lib.lib().sft_adamw(arr, len(vecs), step, step_dev, clip, C.byref(h), None)


def _hp(**kw):
    names = ("lr", "beta1", "beta2", "eps", "weight_decay", "bc1", "bc2", "t_max")
    return tuple(kw.get(k, v) for k, v in zip(names, HP))


@pytest.mark.parametrize("what,code", [
    (dict(vecs=[_vec(n=-1)]), _lib.SFT_EINVAL),
    (dict(vecs=[_vec(n=1 << 42)]), _lib.SFT_ENOTSUP),
    (dict(vecs=[_vec(n=(2048 << 24) - 2047)]), _lib.SFT_ENOTSUP),                # 2^24 chunks
    (dict(vecs=[_vec(n=4096 << 23, scale=BASE), _vec(n=2048 << 23)]), _lib.SFT_ENOTSUP),
    (dict(vecs=[_vec(p_type=2)]), _lib.SFT_EINVAL),
    (dict(vecs=[_vec(g_type=-1)]), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CAdamwVec(16, BASE, None, BASE + 2048, BASE + 3328, None, None, 0, 0)]), _lib.SFT_EINVAL),
    (dict(vecs=[_vec(at=BASE + 2)]), _lib.SFT_EALIGN),
    (dict(vecs=[_vec(live=BASE + 4097)]), _lib.SFT_EALIGN),
    (dict(vecs=[_vec(), _vec()]), _lib.SFT_EINVAL),                              # the same tensor twice
    (dict(vecs=[_vec(n=300), _vec(n=16, at=BASE + 4 * 296)]), _lib.SFT_EINVAL),  # p of one inside p of another
    (dict(vecs=[_vec(live=BASE + 60)]), _lib.SFT_EINVAL),                        # the copy over the master
    (dict(vecs=[_vec(scale=BASE + 2050)]), _lib.SFT_EINVAL),                     # the scales inside m
    (dict(vecs=[_vec()], step=0), _lib.SFT_EINVAL),
    (dict(vecs=[_vec()], step_dev=BASE + 2), _lib.SFT_EALIGN),
    (dict(vecs=[_vec()], clip=BASE + 2), _lib.SFT_EALIGN),
    (dict(vecs=[_vec()], hp=_hp(beta1=1.0)), _lib.SFT_EINVAL),
    (dict(vecs=[_vec()], hp=_hp(beta2=float("nan"))), _lib.SFT_EINVAL),
    (dict(vecs=[_vec()], hp=_hp(eps=-1.0)), _lib.SFT_EINVAL),
    (dict(vecs=[_vec()], hp=_hp(eps=1e-40)), _lib.SFT_EINVAL),
    (dict(vecs=[_vec()], hp=_hp(t_max=0)), _lib.SFT_EINVAL),
    (dict(vecs=[_vec()], hp=_hp(bc1=None)), _lib.SFT_EINVAL),
])
def test_adamw_refuses(what, code):
    assert _adamw(**what) == code
    assert _lib.lib().sft_last_error()


def test_adamw_of_nothing_is_nothing():
    assert _adamw([]) == _lib.SFT_OK
    assert _adamw([_lib.CAdamwVec(0, None, None, None, None, None, None, 0, 1)]) == _lib.SFT_OK


def _clip(vecs, max_norm=1.0, clip=BASE + 8192, norm=None, ws=BASE + 4096, ws_bytes=4096):
    arr = (_lib.CGradVec * max(len(vecs), 1))(*vecs)
    return _lib.lib().sft_grad_clip(arr, len(vecs), max_norm, clip, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("what,code", [
    (dict(vecs=[_lib.CGradVec(-1, BASE, 0)]), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(1 << 42, BASE, 0)]), _lib.SFT_ENOTSUP),
    (dict(vecs=[_lib.CGradVec((1 << 42) - 1, BASE, 0)] * 5), _lib.SFT_ENOTSUP),
    (dict(vecs=[_lib.CGradVec(8, None, 0)]), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(8, BASE, 7)]), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(8, BASE + 2, 0)]), _lib.SFT_EALIGN),
    (dict(vecs=[_lib.CGradVec(8, BASE + 1, 1)]), _lib.SFT_EALIGN),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], max_norm=0.0), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], max_norm=float("nan")), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], clip=None), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], norm=BASE + 1), _lib.SFT_EALIGN),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], ws_bytes=7), _lib.SFT_ECAPACITY),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], ws=None), _lib.SFT_EINVAL),
    (dict(vecs=[_lib.CGradVec(8, BASE, 0)], ws=BASE + 8), _lib.SFT_EALIGN),
])
def test_grad_clip_refuses(what, code):
    assert _clip(**what) == code
    assert _lib.lib().sft_last_error()


def test_grad_clip_workspace():
    def need(vecs):
        return _lib.lib().sft_grad_clip_workspace((_lib.CGradVec * max(len(vecs), 1))(*vecs), len(vecs))

    assert need([]) == 0
    assert need([_lib.CGradVec(0, None, 1)]) == 0
    assert need([_lib.CGradVec(1, BASE, 1)]) == 8
    assert need([_lib.CGradVec(8193, BASE, 1)]) == 16
    assert need([_lib.CGradVec(1 << 40, BASE, 1)]) == 8 * 2048
    assert need([_lib.CGradVec(1, BASE, 1)] * 201) == 8 * 201
    assert need([_lib.CGradVec(-1, BASE, 1)]) == C.c_size_t(-1).value


@pytest.mark.parametrize("bc1,bc2,error", [
    ((5, "float32"), (4, "float32"), ValueError), ((4, "float32"), (5, "float32"), ValueError),
    ((1, "float32"), (1, "float32"), ValueError), ((0, "float32"), (0, "float32"), ValueError),
    ((5, "float64"), (5, "float64"), TypeError), ((5, "float32"), (5, "float64"), TypeError),
    ((5, "float16"), (5, "float32"), TypeError),
])
def test_adam_refuses_bias_tables_that_do_not_fit(bc1, bc2, error):
    # a kernel reads both tables up to entry numel - 1 of the first, as fp32: whatever the call, these are refused
    # before it is looked where the tables are
    torch = pytest.importorskip("torch")
    tables = [torch.zeros(n, dtype=getattr(torch, t)) for n, t in (bc1, bc2)]
    with pytest.raises(error, match="bias table"):
        _lib.Adam(0.1, 0.9, 0.999, 1e-8, *tables).c()


@pytest.mark.parametrize("what", [
    dict(vecs=[_lib.CAdamwVec(16, BASE, BASE, BASE + 2048, BASE + 3328, None, None, 0, 0)]),          # p itself
    dict(vecs=[_lib.CAdamwVec(16, BASE, BASE + 60, BASE + 2048, BASE + 3328, None, None, 0, 0)]),     # p's last value
    dict(vecs=[_lib.CAdamwVec(16, BASE, BASE + 2048 - 60, BASE + 2048, BASE + 3328, None, None, 0, 0)]),
    dict(vecs=[_lib.CAdamwVec(16, BASE, BASE + 3328 + 32, BASE + 2048, BASE + 3328, None, None, 0, 1)]),
    dict(vecs=[_lib.CAdamwVec(16, BASE, BASE + 1024, BASE + 2048, BASE + 3328, None, BASE + 1024, 0, 1)]),
    dict(vecs=[_lib.CAdamwVec(16, BASE, BASE + 1024, BASE + 2048, BASE + 3328, BASE + 1084, None, 0, 0)]),
    # a gradient longer than the gap to another tensor's p, both lists out of order
    dict(vecs=[_vec(at=BASE + 4608), _lib.CAdamwVec(64, BASE, BASE + 4400, BASE + 2048, BASE + 3328, None, None, 0, 0)]),
    # two gradients with a short one behind a long one's start: the long one reaches p
    dict(vecs=[_lib.CAdamwVec(300, BASE + 4096, BASE, BASE + 6144, BASE + 9600, None, None, 0, 0),
               _lib.CAdamwVec(4, BASE + 1100, BASE + 16, BASE + 1536, BASE + 1792, None, None, 0, 0)]),
    dict(vecs=[_vec()], clip=BASE + 2048 + 60),
    dict(vecs=[_vec()], step_dev=BASE + 4),
    dict(vecs=[_vec(n=1)], hp=_hp(bc1=BASE + 2048 - 16)),      # entry t_max of a table is the first of m
    dict(vecs=[_vec(n=1)], hp=_hp(bc2=BASE + 3328)),
])
def test_adamw_refuses_inputs_inside_what_it_writes(what):
    assert _adamw(**what) == _lib.SFT_EINVAL
    assert b"overlap" in _lib.lib().sft_last_error()


@pytest.mark.parametrize("what", [
    dict(vecs=[_lib.CGradVec(8, BASE, 0)], norm=BASE + 8192),                 # the factor's own place
    dict(vecs=[_lib.CGradVec(8, BASE + 4096, 0)]),                             # the gradient where the sums go
    dict(vecs=[_lib.CGradVec(8, BASE, 0), _lib.CGradVec(8, BASE + 4096 + 8, 1)]),
    dict(vecs=[_lib.CGradVec(1 + 1024, BASE, 0)]),
    dict(vecs=[]) | dict(norm=BASE + 8192),
])
def test_grad_clip_refuses_arrays_that_overlap(what):
    assert _clip(**what) == _lib.SFT_EINVAL
    assert b"overlap" in _lib.lib().sft_last_error()


def test_grad_clip_workspace_may_follow_a_gradient():
    # no byte shared: not refused for it (a workspace too small is looked at first)
    assert _clip([_lib.CGradVec(1024, BASE, 0)], ws_bytes=0) == _lib.SFT_ECAPACITY
    assert _clip([_lib.CGradVec(8, BASE, 0)], ws=BASE + 32, norm=BASE + 8194) == _lib.SFT_EALIGN
