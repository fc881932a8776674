"""CPU tests of the row-wise calls (norms, rotary positions, log
probabilities): what they refuse before anything is launched, and the table of
rotary angles."""
import ctypes as C
import math

import numpy as np
import pytest

from sparse_full_weight_amd import _lib

BUF = np.zeros(1 << 16, np.uint8)
BASE = (BUF.ctypes.data + 255) // 256 * 256
EINVAL, ESHAPE, EALIGN, ECAPACITY, ENOTSUP = (_lib.SFT_EINVAL, _lib.SFT_ESHAPE, _lib.SFT_EALIGN, _lib.SFT_ECAPACITY,
                                              _lib.SFT_ENOTSUP)
NAN, INF = math.nan, math.inf


def _struct(cls, base, **kw):
    s = cls()
    for k, v in {**base, **kw}.items():
        assert any(k == name for name, *_ in cls._fields_)
        setattr(s, k, v)
    return s


def _refused(rc, code, word=b""):
    assert rc == code, (rc, _lib.lib().sft_last_error())
    assert word in _lib.lib().sft_last_error() and _lib.lib().sft_last_error()


# 4 rows of 8 floats (128 bytes), every array 1024 bytes from the next
NORM = dict(T=4, C=8, X=BASE, res=BASE + 1024, H=BASE + 2048, gain=BASE + 3 * 1024, bias=BASE + 4096, Y=BASE + 5120,
            mean=BASE + 6144, rstd=BASE + 7168, ldx=8, ldr=8, ldh=8, ldy=8, eps=1e-5, kind=0, x_type=0, w_type=0, y_type=0)


def _norm(**kw):
    return _lib.lib().sft_norm_forward(C.byref(_struct(_lib.CNormArgs, NORM, **kw)), None)


@pytest.mark.parametrize("what,code", [
    (dict(T=-1), EINVAL), (dict(C=-8), EINVAL), (dict(C=0), ESHAPE), (dict(C=16385, ldx=16385), ENOTSUP),
    (dict(T=1 << 31), ENOTSUP), (dict(kind=2), EINVAL), (dict(kind=-1), EINVAL), (dict(x_type=2), EINVAL),
    (dict(w_type=7), EINVAL), (dict(x_type=1, y_type=0), EINVAL), (dict(eps=-1e-5), EINVAL), (dict(eps=NAN), EINVAL),
    (dict(eps=INF), EINVAL), (dict(X=None), EINVAL), (dict(Y=None), EINVAL), (dict(res=None), EINVAL),
    (dict(H=None), EINVAL), (dict(ldx=7), ESHAPE), (dict(ldr=0), ESHAPE), (dict(ldh=7), ESHAPE), (dict(ldy=-8), ESHAPE),
    (dict(ldx=1 << 40), ENOTSUP), (dict(T=1 << 30, ldx=1 << 20), ENOTSUP),
    (dict(X=BASE + 2), EALIGN), (dict(Y=BASE + 5121), EALIGN), (dict(gain=BASE + 3074), EALIGN),
    (dict(bias=BASE + 4098), EALIGN), (dict(mean=BASE + 6145), EALIGN), (dict(rstd=BASE + 7170), EALIGN),
])
def test_norm_forward_refuses(what, code):
    _refused(_norm(**what), code)


@pytest.mark.parametrize("what", [
    dict(Y=BASE), dict(Y=BASE + 124), dict(Y=BASE + 1024), dict(Y=BASE + 2048), dict(Y=BASE + 3100),
    dict(Y=BASE + 4096 - 100), dict(mean=BASE + 5120), dict(rstd=BASE + 124), dict(mean=BASE + 7168),
    dict(H=BASE + 4), dict(H=BASE, ldh=9), dict(H=BASE + 1024 + 32), dict(H=BASE + 3 * 1024), dict(H=BASE + 5120),
    dict(H=BASE, ldx=16, ldh=12),                                         # the same address, another distance
    dict(Y=BASE + 28, ldx=16, ldy=16),                                    # side by side, but one element of each row
    dict(Y=BASE + 32, ldx=16, ldy=17),                                    # side by side at first only
])
def test_norm_forward_refuses_arrays_that_overlap(what):
    _refused(_norm(**what), EINVAL, b"overlap")


def test_rows_side_by_side_are_apart():
    # the right halves of the rows whose left halves are read: no byte is shared, so another check is what refuses
    _refused(_norm(Y=BASE + 32, ldx=16, ldy=16, H=BASE + 4096), EINVAL, b"overlap")
    assert b"input" in _lib.lib().sft_last_error()           # of H and bias
    assert _norm(T=0, Y=BASE + 32, ldx=16, ldy=16) == _lib.SFT_OK


GRAD = dict(T=4, C=8, H=BASE, gain=BASE + 1024, mean=BASE + 2048, rstd=BASE + 3 * 1024, dY=BASE + 4096, dH=BASE + 5120,
            dX=BASE + 6144, dgain=BASE + 7168, dbias=BASE + 8192, ldh=8, ldy=8, ldr=8, ldx=8, kind=0, x_type=0, w_type=0,
            y_type=0, g_type=0, accumulate=0)
NEED = 4 * 8 * 4 * 2             # at most 4 partial sums of 8 gains and 8 biases


def _norm_grad(ws=BASE + 16384, ws_bytes=1 << 14, **kw):
    return _lib.lib().sft_norm_backward(C.byref(_struct(_lib.CNormGradArgs, GRAD, **kw)), ws, ws_bytes, None)


@pytest.mark.parametrize("what,code", [
    (dict(T=-1), EINVAL), (dict(C=0), ESHAPE), (dict(C=16385), ENOTSUP), (dict(T=1 << 31), ENOTSUP), (dict(kind=2), EINVAL),
    (dict(g_type=2), EINVAL), (dict(g_type=1, accumulate=1), EINVAL), (dict(x_type=1, y_type=0), EINVAL),
    (dict(H=None), EINVAL), (dict(dY=None), EINVAL), (dict(dX=None), EINVAL), (dict(rstd=None), EINVAL),
    (dict(mean=None), EINVAL), (dict(ldh=7), ESHAPE), (dict(ldy=7), ESHAPE), (dict(ldr=7), ESHAPE), (dict(ldx=7), ESHAPE),
    (dict(H=BASE + 1), EALIGN), (dict(dgain=BASE + 7170), EALIGN), (dict(mean=BASE + 2049), EALIGN),
    (dict(ws=None), EINVAL), (dict(ws=BASE + 16384 + 8), EALIGN), (dict(ws_bytes=0), ECAPACITY),
])
def test_norm_backward_refuses(what, code):
    _refused(_norm_grad(**what), code)


@pytest.mark.parametrize("what", [
    dict(dX=BASE), dict(dX=BASE + 4096, ldx=9), dict(dX=BASE + 4100), dict(dX=BASE + 5120, ldx=12, ldr=16),
    dict(dX=BASE + 1024), dict(dX=BASE + 3 * 1024 - 100), dict(dgain=BASE), dict(dgain=BASE + 8192), dict(dbias=BASE + 6144),
    dict(dgain=BASE + 1024), dict(dbias=BASE + 3 * 1024), dict(ws=BASE), dict(ws=BASE + 6144), dict(ws=BASE + 7168),
    dict(dX=BASE + 4096, x_type=0, y_type=1, ldx=8, ldy=16),              # dY's place, another type
])
def test_norm_backward_refuses_arrays_that_overlap(what):
    _refused(_norm_grad(**what), EINVAL, b"overlap")


def test_norm_backward_workspace():
    need = _lib.lib().sft_norm_backward_workspace
    assert need(0, 100, 1) == 0
    assert need(1, 100, 0) == 400 and need(1, 100, 1) == 800
    assert 0 < need(4, 8, 1) <= NEED
    for T, cols in ((-1, 8), (4, 0), (4, -1), (4, 16385), (1 << 31, 8)):
        assert need(T, cols, 0) == C.c_size_t(-1).value
    # enough rows: a bound that does not grow with them
    assert need(1 << 20, 4096, 0) == need(1 << 24, 4096, 0) < 1 << 26


# 2 sequences of 3 tokens of 2 heads of 8 floats
HEADS = dict(X=BASE, Y=BASE + 4096, heads=2, x_batch=48, x_row=16, x_head=8, y_batch=48, y_row=16, y_head=8)


def _rotary(mats=(HEADS,), B=2, T=3, D=8, rot=8, freq=BASE + 8192, pos=BASE + 12288, pos_batch=3, amplitude=1.0, layout=0,
            type=0):
    arr = (_lib.CRotaryMat * max(len(mats), 1))(*[_struct(_lib.CRotaryMat, m) for m in mats])
    args = _lib.CRotaryArgs(arr, B, T, D, rot, freq, pos, pos_batch, amplitude, len(mats), layout, 0, type)
    return _lib.lib().sft_rotary(C.byref(args), None)


def _one(**kw):
    return ({**HEADS, **kw},)


@pytest.mark.parametrize("what,code", [
    (dict(B=-1), EINVAL), (dict(T=-1), EINVAL), (dict(D=-1), EINVAL), (dict(pos_batch=-1), EINVAL),
    (dict(D=4097), ENOTSUP), (dict(B=1 << 30), ENOTSUP), (dict(B=1 << 15, T=1 << 15), ENOTSUP),
    (dict(rot=7), ESHAPE), (dict(rot=0), ESHAPE), (dict(rot=10), ESHAPE), (dict(type=2), EINVAL), (dict(layout=2), EINVAL),
    (dict(amplitude=NAN), EINVAL), (dict(amplitude=INF), EINVAL), (dict(freq=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(freq=BASE + 8196), EALIGN), (dict(pos=BASE + 2), EALIGN), (dict(pos_batch=1 << 40), ENOTSUP),
    (dict(mats=[HEADS] * 9), ENOTSUP), (dict(mats=_one(X=None)), EINVAL), (dict(mats=_one(Y=None)), EINVAL),
    (dict(mats=_one(heads=-1)), EINVAL), (dict(mats=_one(heads=1 << 16)), ENOTSUP), (dict(mats=_one(x_row=-16)), EINVAL),
    (dict(mats=_one(y_batch=1 << 40)), ENOTSUP), (dict(mats=_one(x_batch=1 << 39), B=1 << 20), ENOTSUP),
    (dict(mats=_one(X=BASE + 2)), EALIGN), (dict(mats=_one(Y=BASE + 4097)), EALIGN),
])
def test_rotary_refuses(what, code):
    _refused(_rotary(**what), code)


@pytest.mark.parametrize("what", [
    dict(mats=_one(Y=BASE + 4)), dict(mats=_one(Y=BASE, y_row=24, y_batch=72)), dict(mats=_one(Y=BASE + 4 * 95)),
    dict(mats=_one(y_head=0)), dict(mats=_one(y_head=7)), dict(mats=_one(y_row=8)), dict(mats=_one(y_batch=0)),
    dict(mats=_one(y_row=8, y_head=8)), dict(mats=_one(y_batch=47)),
    dict(mats=_one(Y=BASE + 8192)), dict(mats=_one(Y=BASE + 12288 - 8)),
    dict(mats=[HEADS, {**HEADS, "X": BASE + 2048}]),                          # one Y for two arrays
    dict(mats=[HEADS, {**HEADS, "Y": BASE + 1020}], B=20),                    # Y of one in X of both
    # queries and keys of one buffer in place, the keys one element into the queries
    dict(mats=[{**HEADS, "Y": BASE, "x_row": 24, "y_row": 24, "x_batch": 72, "y_batch": 72},
               {**HEADS, "X": BASE + 60, "Y": BASE + 60, "heads": 1, "x_row": 24, "y_row": 24, "x_batch": 72, "y_batch": 72}]),
])
def test_rotary_refuses_arrays_that_overlap(what):
    _refused(_rotary(**what), EINVAL, b"overlap")


def test_rotary_of_nothing_is_nothing():
    assert _rotary(mats=()) == _lib.SFT_OK
    assert _rotary(T=0, freq=None, pos=None) == _lib.SFT_OK
    assert _rotary(mats=_one(heads=0, X=None, Y=None)) == _lib.SFT_OK



@pytest.mark.parametrize("kind,args,want", [
    ("plain", {}, lambda f, n: f), ("linear", dict(factor=4.0), lambda f, n: f / 4),
    ("base", dict(factor=8.0), None), ("bands", dict(factor=8.0, context=2048.0, low=1.0, high=4.0), None),
])
@pytest.mark.parametrize("rot,base", [(2, 10000.0), (20, 10000.0), (128, 500000.0)])
def test_rotary_table(kind, args, want, rot, base):
    j = np.arange(rot // 2)
    f = base ** (-2.0 * j / rot)
    got = _lib.sft_rotary_table(rot, base, scaling=kind, **args)
    if want:
        ref = want(f, rot)
    elif kind == "base":
        ref = (base * 8.0 ** (rot / (rot - 2)) if rot > 2 else base) ** (-2.0 * j / rot)
        assert rot == 2 or abs(got[-1] * 8.0 / f[-1] - 1) < 1e-13 and got[0] == 1.0
    else:
        turns = 2048 * f / (2 * np.pi)
        w = np.clip((turns - 1.0) / 3.0, 0, 1)
        ref = f * w + f / 8.0 * (1 - w)
        assert (ref[turns > 4] == f[turns > 4]).all()
    assert np.abs(got / ref - 1).max() < 1e-13


@pytest.mark.parametrize("args,code", [
    (dict(rot=3), ESHAPE), (dict(rot=0), ESHAPE), (dict(rot=-2), ESHAPE), (dict(base=0.0), EINVAL), (dict(base=NAN), EINVAL),
    (dict(kind=4), EINVAL), (dict(kind=-1), EINVAL), (dict(factor=0.5), EINVAL), (dict(factor=INF), EINVAL),
    (dict(kind=3, context=0.0), EINVAL), (dict(kind=3, low=4.0), EINVAL), (dict(kind=3, high=NAN), EINVAL),
    (dict(kind=2, rot=4, factor=1e200), EINVAL), (dict(freq=None), EINVAL),
])
def test_rotary_table_refuses(args, code):
    a = {**dict(rot=8, base=10000.0, kind=0, factor=1.0, context=100.0, low=1.0, high=4.0, freq=BASE), **args}
    _refused(_lib.lib().sft_rotary_table(*[a[k] for k in ("rot", "base", "kind", "factor", "context", "low", "high", "freq")]),
             code)


# 4 rows of 8 floats
LOGP = dict(N=4, V=8, ldz=8, Z=BASE, target=BASE + 1024, logp=BASE + 2048, stats=BASE + 4096, entropy=BASE + 5120,
            top_logp=BASE + 6144, top_index=BASE + 7168, z_type=0, top_k=3, scale=1.0)


def _logprob(**kw):
    return _lib.lib().sft_logprob(C.byref(_struct(_lib.CLogprobArgs, LOGP, **kw)), None)


@pytest.mark.parametrize("what,code", [
    (dict(N=-1), EINVAL), (dict(V=-1), EINVAL), (dict(V=0), ESHAPE), (dict(V=1 << 30, ldz=1 << 30), ENOTSUP),
    (dict(N=1 << 31), ENOTSUP), (dict(ldz=7), ESHAPE), (dict(ldz=1 << 40), ENOTSUP), (dict(z_type=2), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=NAN), EINVAL), (dict(scale=INF), EINVAL),
    (dict(scale=3e38), EINVAL), (dict(top_k=-1), EINVAL), (dict(top_k=65), EINVAL), (dict(Z=None), EINVAL),
    (dict(target=None), EINVAL), (dict(logp=None), EINVAL), (dict(top_index=None), EINVAL), (dict(Z=BASE + 2), EALIGN),
    (dict(target=BASE + 1026), EALIGN), (dict(stats=BASE + 4097), EALIGN), (dict(top_index=BASE + 7169), EALIGN),
])
def test_logprob_refuses(what, code):
    _refused(_logprob(**what), code)


@pytest.mark.parametrize("what", [
    dict(logp=BASE), dict(stats=BASE + 1024), dict(entropy=BASE + 2048), dict(top_logp=BASE + 7168 + 44),
    dict(top_index=BASE + 4096), dict(entropy=BASE + 124),
])
def test_logprob_refuses_arrays_that_overlap(what):
    _refused(_logprob(**what), EINVAL, b"overlap")


DZ = dict(N=4, V=8, ldz=8, lddz=8, Z=BASE, target=BASE + 1024, stats=BASE + 2048, entropy=BASE + 4096, dlogp=BASE + 5120,
          dentropy=BASE + 6144, dZ=BASE + 7168, z_type=0, dz_type=0, scale=1.0)


def _logprob_grad(**kw):
    return _lib.lib().sft_logprob_grad(C.byref(_struct(_lib.CLogprobGradArgs, DZ, **kw)), None)


@pytest.mark.parametrize("what,code", [
    (dict(N=-1), EINVAL), (dict(V=0), ESHAPE), (dict(lddz=7), ESHAPE), (dict(ldz=7), ESHAPE), (dict(z_type=3), EINVAL),
    (dict(z_type=1, dz_type=0), EINVAL), (dict(scale=0.0), EINVAL), (dict(dZ=None), EINVAL), (dict(stats=None), EINVAL),
    (dict(target=None), EINVAL), (dict(dlogp=None), EINVAL), (dict(entropy=None), EINVAL), (dict(dentropy=None), EINVAL),
    (dict(dZ=BASE + 7170), EALIGN), (dict(dlogp=BASE + 5121), EALIGN), (dict(lddz=1 << 40), ENOTSUP),
])
def test_logprob_grad_refuses(what, code):
    _refused(_logprob_grad(**what), code)


@pytest.mark.parametrize("what", [
    dict(dZ=BASE + 4), dict(dZ=BASE, lddz=9), dict(dZ=BASE, dz_type=1), dict(dZ=BASE, dz_type=1, lddz=16),
    dict(dZ=BASE + 1024), dict(dZ=BASE + 2048), dict(dZ=BASE + 4096 - 64), dict(dZ=BASE + 5120), dict(dZ=BASE + 6144),
])
def test_logprob_grad_refuses_arrays_that_overlap(what):
    _refused(_logprob_grad(**what), EINVAL, b"overlap")


def test_no_rows_ask_for_nothing():
    none = dict(N=0, Z=None, target=None, logp=None, stats=None, entropy=None, top_logp=None, top_index=None)
    assert _logprob(**none) == _lib.SFT_OK
    assert _logprob_grad(N=0, Z=None, dZ=None, target=None, stats=None, entropy=None, dlogp=None, dentropy=None) == _lib.SFT_OK


# ------------------------------------------------------------------ the bound of the alternatives
def _values(rs, n, kind):
    x = rs.standard_normal(n).astype(np.float32) * 3
    if kind == "bf16":
        x = (x.view(np.uint32) & 0xffff0000).view(np.float32)
    elif kind == "few":
        x = np.round(x)
    elif kind == "equal":
        x[:] = x[0]
    elif kind == "two":
        x = np.where(rs.random(n) < rs.random(), x[0], x[-1])
    elif kind == "near":
        x = (np.float32(rs.choice([1.0, -1.0, 1e30, -1e-40])).view(np.uint32) + rs.integers(0, 3, n).astype(np.uint32)).view(
            np.float32)
    elif kind == "bits":
        x = rs.integers(0, 1 << 32, n, dtype=np.uint64).astype(np.uint32).view(np.float32)
        x = np.where(np.isnan(x), np.float32(0), x)
    elif kind == "masked":
        x = np.where(rs.random(n) < rs.random(), np.float32(rs.choice([-np.inf, -1e30, -3.4028235e38])), x)
    elif kind == "zeros":
        x = rs.choice(np.array([0.0, -0.0, 1e-45, -1e-45], np.float32), n)
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["any", "bf16", "few", "equal", "two", "near", "bits", "masked", "zeros"])
def test_bound_of_the_alternatives(kind):
    # the search ends, and at least `want` values reach what it finds; where many more do, they are equal to the want-th
    rs = np.random.default_rng(len(kind))
    for n in (64, 128, 1, 2, 3, 63):
        for want in sorted({1, 2, 5, 20, 32, 33, 51, 63, 64, n} & set(range(1, n + 1))):
            for _ in range(40):
                x = _values(rs, n, kind)
                with np.errstate(invalid="ignore"):
                    bound = _lib.sft_probe_logprob_bound(x, want)
                wanted = np.sort(x)[::-1][want - 1]
                if math.isnan(bound):      # below minus infinity: all of them
                    assert wanted == -INF
                    continue
                reach = int((x >= bound).sum())
                assert reach >= want
                assert reach <= want + want // 4 or reach == int((x >= wanted).sum())


def test_bound_of_the_alternatives_refuses():
    x, out = np.ones(128, np.float32), np.zeros(1, np.float32)
    probe = _lib.lib().sft_probe_logprob_bound
    for values, n, want, bound in ((None, 64, 1, out), (x, 64, 1, None), (x, 0, 1, out), (x, 129, 1, out), (x, 64, 0, out),
                                   (x, 64, 65, out)):
        assert probe(None if values is None else values.ctypes.data, n, want,
                     None if bound is None else bound.ctypes.data) == EINVAL
    x[3] = NAN
    _refused(probe(x.ctypes.data, 64, 1, out.ctypes.data), EINVAL, b"NaN")
