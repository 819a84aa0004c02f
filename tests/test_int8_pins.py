"""Pins of the 8-bit oracle (oracle/int8.py) to exact arithmetic, and the host
checks of the 8-bit calls.  No GPU: no kernel is launched."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import rotation_int4_weight_b200 as paro
from synth import bf16_round

OK, INVALID, UNSUPPORTED = 0, 1, 2


def _nearest_even(f: Fraction) -> int:
    return round(f)  # Python rounds a Fraction half to even


def test_row_codes_against_fractions():
    rng = np.random.default_rng(1)
    v = bf16_round((rng.standard_normal((6, 300)) * 4).astype(np.float32)).astype(np.float64)
    v[1] = 0.0
    v[2, :4] = [254.0, 1.0, 3.0, -5.0]    # 127 v / a = v / 2: ties at 0.5, 1.5, -2.5
    v[2, 4:] = 0.0
    q, s = oracle.row_codes(v)
    assert q[2, :4].tolist() == [127, 0, 2, -2]
    for m in range(v.shape[0]):
        a = max(abs(Fraction(float(x))) for x in v[m])
        if a == 0:
            assert s[m] == 1.0 and not q[m].any()
            continue
        assert s[m] == pytest.approx(float(a / 127), rel=1e-15)
        assert [int(c) for c in q[m]] == [_nearest_even(127 * Fraction(float(x)) / a) for x in v[m]]


def test_row_codes_of_rows_that_are_not_finite():
    v = np.ones((3, 16))
    v[0, 3], v[2, 5] = np.nan, -np.inf
    q, s = oracle.row_codes(v)
    assert np.isnan(s[[0, 2]]).all() and s[1] == pytest.approx(1 / 127)
    assert not q[[0, 2]].any() and (q[1] == 127).all()


def test_rms_norm_codes_dequantise_to_the_norm():
    rng = np.random.default_rng(2)
    h = bf16_round(rng.standard_normal((5, 640)).astype(np.float32)).astype(np.float64)
    g = bf16_round((1 + 0.2 * rng.standard_normal(640)).astype(np.float32)).astype(np.float64)
    q, s = oracle.rms_norm_codes(h, g, 1e-6)
    y = h * g / np.sqrt((h ** 2).mean(axis=1, keepdims=True) + 1e-6)
    assert (np.abs(q * s[:, None] - y) <= s[:, None] / 2 * (1 + 1e-12)).all()
    assert np.allclose(s * 127, np.abs(y).max(axis=1), rtol=1e-14)


def test_linears_against_python_loops():
    rng = np.random.default_rng(3)
    q, w, w2 = (rng.integers(-128, 128, s).astype(np.int8) for s in ((3, 48), (5, 48), (5, 48)))
    sx, sw, s2 = rng.uniform(0.01, 1, 3), rng.uniform(1e-4, 1e-3, 5), rng.uniform(1e-4, 1e-3, 5)
    b = rng.standard_normal(5)
    y = oracle.w8a8_linear(q, sx, w, sw, b)
    z, _, _ = oracle.w8a8_swiglu(q, sx, w, sw, w2, s2)
    for m in range(3):
        for n in range(5):
            g = sum(int(x) * int(v) for x, v in zip(q[m], w[n])) * sx[m] * sw[n]
            u = sum(int(x) * int(v) for x, v in zip(q[m], w2[n])) * sx[m] * s2[n]
            assert y[m, n] == pytest.approx(g + b[n], rel=1e-12, abs=1e-13)
            assert z[m, n] == pytest.approx(g / (1 + np.exp(-g)) * u, rel=1e-12, abs=1e-13)


# ---------------------------------------------------------------- host validation
def P(mb, off=0):
    return ctypes.c_void_p((mb << 20) + off)


X, Q, S, W, WS, Y, R, G, H, Z = (P(64 * i) for i in range(1, 11))  # fake, 64 MB apart, never dereferenced
MIS = P(64, 8)


@pytest.mark.parametrize("args,expect", [
    ((X, Q, S, 0, 512, 0, None), OK), ((None, None, None, 0, 512, 0, None), OK),   # no rows: nothing enqueued
    ((X, Q, S, -1, 512, 0, None), INVALID), ((X, Q, S, 2, 0, 0, None), INVALID),
    ((X, Q, S, 2, 49153, 0, None), UNSUPPORTED), ((X, Q, S, 2, 512, 2, None), INVALID),
    ((None, Q, S, 2, 512, 0, None), INVALID), ((MIS, Q, S, 2, 512, 0, None), INVALID),
    ((X, P(128, 8), S, 2, 512, 0, None), INVALID), ((X, Q, P(192, 2), 2, 512, 0, None), INVALID),
    ((X, X, S, 2, 512, 0, None), INVALID), ((X, Q, P(128, 512), 2, 512, 0, None), INVALID),
])
def test_quantize_int8_validation(args, expect):
    assert paro.lib.paro_quantize_activations_int8(*args) == expect, paro.lib.paro_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(M=0), OK), (dict(M=-1), INVALID), (dict(d=0), INVALID), (dict(d=49160), UNSUPPORTED),
    (dict(t=7), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(hid=None), INVALID), (dict(res=None), INVALID),
    (dict(res=MIS), INVALID), (dict(g=P(512, 8)), INVALID),
    (dict(hid=P(64, 16)), INVALID),        # overlaps x but is not x
    (dict(hid=P(448, 1024)), INVALID),     # overlaps the residual but is not it
    (dict(q=G), INVALID), (dict(q=H), INVALID), (dict(hid=G), INVALID), (dict(sx=P(128, 4)), INVALID),
])
def test_rms_norm_int8_validation(change, expect):
    a = dict(x=X, res=R, g=G, eps=1e-6, hid=H, q=Q, sx=S, M=2, d=512, t=0) | change
    st = paro.lib.paro_rms_norm_int8(a["x"], a["res"], a["g"], a["eps"], a["hid"], a["q"], a["sx"], a["M"], a["d"],
                                     a["t"], None)
    assert st == expect, paro.lib.paro_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(d_in=500), INVALID), (dict(d_in=0), INVALID), (dict(d_in=49168), UNSUPPORTED), (dict(d_out=0), INVALID),
    (dict(K=17), UNSUPPORTED), (dict(K=-1), INVALID), (dict(K=8, pairs=None), INVALID), (dict(W=None), INVALID),
    (dict(W=MIS), INVALID), (dict(q=MIS), INVALID), (dict(s=None), INVALID), (dict(q=X), INVALID),
    (dict(K=8, ws=None), INVALID), (dict(K=8, ws=X), INVALID), (dict(K=8, ws=Q), INVALID),
])
def test_pack_int8_validation(change, expect):
    a = dict(W=X, d_out=64, d_in=512, K=0, pairs=R, c=G, sn=H, sc=None, ws=Z, q=Q, s=S) | change
    st = paro.lib.paro_pack_weights_int8(a["W"], a["d_out"], a["d_in"], a["K"], a["pairs"], a["c"], a["sn"], a["sc"],
                                         a["ws"], a["q"], a["s"], None)
    assert st == expect, paro.lib.paro_last_error()


LINEAR = dict(q=X, sx=S, w=W, ws=WS, b=None, y=Y, M=4, d_in=512, d_out=100, t=0)


@pytest.mark.parametrize("change,expect", [
    (dict(M=0), OK), (dict(M=0, q=None, y=None), OK), (dict(M=-1), INVALID), (dict(d_in=8), INVALID),
    (dict(d_in=0), INVALID), (dict(d_in=49168), UNSUPPORTED), (dict(d_out=0), INVALID), (dict(t=-1), INVALID),
    (dict(q=None), INVALID), (dict(q=MIS), INVALID), (dict(w=None), INVALID), (dict(w=P(256, 4)), INVALID),
    (dict(ws=P(320, 2)), INVALID), (dict(sx=None), INVALID), (dict(y=P(384, 2)), INVALID), (dict(b=P(512, 1)), INVALID),
    (dict(y=X), INVALID), (dict(y=S), INVALID), (dict(y=P(256, 64)), INVALID), (dict(y=WS), INVALID),
    (dict(b=P(384, 2)), INVALID), (dict(M=(1 << 30) + 1, d_in=16), UNSUPPORTED), (dict(d_out=(1 << 30) + 1, d_in=16), UNSUPPORTED),
])
def test_w8a8_linear_validation(change, expect):
    a = LINEAR | change
    st = paro.lib.paro_w8a8_linear(a["q"], a["sx"], a["w"], a["ws"], a["b"], a["y"], a["M"], a["d_in"], a["d_out"],
                                   a["t"], None)
    assert st == expect, paro.lib.paro_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(M=0), OK), (dict(M=-1), INVALID), (dict(d_in=24), INVALID), (dict(w2=None), INVALID), (dict(s2=None), INVALID),
    (dict(y=R), INVALID), (dict(y=G), INVALID), (dict(w2=P(448, 8)), INVALID),
])
def test_w8a8_swiglu_validation(change, expect):
    a = LINEAR | dict(w2=R, s2=G) | change
    st = paro.lib.paro_w8a8_swiglu(a["q"], a["sx"], a["w"], a["ws"], a["w2"], a["s2"], a["y"], a["M"], a["d_in"],
                                   a["d_out"], a["t"], None)
    assert st == expect, paro.lib.paro_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(M=0), OK), (dict(M=-1), INVALID), (dict(d_in=100), INVALID), (dict(K=17), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(wsb=10), INVALID), (dict(wsp=P(640, 16)), INVALID), (dict(wsp=X), INVALID), (dict(wsp=Y), INVALID),
    (dict(wsp=W), INVALID), (dict(y=X), INVALID), (dict(y=W), INVALID), (dict(b=P(512, 1)), INVALID),
])
def test_rotate_w8a8_validation(change, expect):
    a = dict(x=X, K=8, p=R, c=G, s=H, sc=None, w=W, ws=WS, b=None, y=Y, M=4, d_in=512, d_out=100, wsp=Z,
             wsb=1 << 20) | change
    st = paro.lib.paro_rotate_w8a8_linear(a["x"], a["K"], a["p"], a["c"], a["s"], a["sc"], a["w"], a["ws"], a["b"],
                                          a["y"], a["M"], a["d_in"], a["d_out"], a["wsp"], a["wsb"], None)
    assert st == expect, paro.lib.paro_last_error()


@pytest.mark.parametrize("change", [dict(M=(1 << 30) + 1), dict(d_out=(1 << 30) + 1)])
def test_rotate_w8a8_refuses_sizes_before_it_enqueues(change):
    # the linear's limit on rows is looked at before the transform is launched (which, without
    # a GPU, would be the first to fail); pointers 1 TB apart, never dereferenced
    at = lambda i: ctypes.c_void_p(i << 40)
    a = dict(M=4, d_out=100) | change
    st = paro.lib.paro_rotate_w8a8_linear(at(1), 8, at(2), at(3), at(4), None, at(5), at(6), None, at(7), a["M"], 16,
                                          a["d_out"], at(8), 1 << 40, None)
    assert st == UNSUPPORTED, paro.lib.paro_last_error()


def test_rotate_w8a8_workspace_bytes():
    r = lambda b: (b + 255) // 256 * 256
    for M, d in [(1, 16), (3, 1536), (2048, 4096)]:
        assert paro.paro_rotate_w8a8_workspace_bytes(M, d) == r(2 * M * d) + r(M * d) + r(4 * M)
    assert paro.paro_rotate_w8a8_workspace_bytes(0, 512) == 0


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    q = torch.zeros(2, 16, dtype=torch.int8)
    s = torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        paro.paro_quantize_activations_int8(x)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        paro.paro_quantize_activations_int8(x.float())
    with pytest.raises(ValueError, match="two dimensions"):
        paro.paro_quantize_activations_int8(x[0])
    with pytest.raises(ValueError, match="hidden"):
        paro.paro_rms_norm_int8(x, hidden=x)
    with pytest.raises(ValueError, match="CUDA"):
        paro.paro_w8a8_linear(q, s, q, s)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        paro.paro_w8a8_linear(q, s, q, s, out_dtype=torch.float32)


# ------------------------------------------------------------------ the linears' forms
def test_w8a8_form_validation():
    form = (ctypes.c_int * 3)()
    call = paro.lib.paro_w8a8_form
    assert call(1, 512, 100, 0, form) == OK and list(form) == [16, 128, 4]
    for bad in ((0, 512, 100, 0, form), (-1, 512, 100, 0, form), (1, 500, 100, 0, form), (1, 512, 0, 0, form),
                (1, 512, 100, 0, None)):
        assert call(*bad) == INVALID
    assert call(1, 49168, 100, 0, form) == UNSUPPORTED
    assert call((1 << 30) + 1, 16, 1, 1, form) == UNSUPPORTED


def test_every_form_of_the_int8_linears_is_compared_with_the_exact_product():
    # the shapes of test_gpu_int8_forms.py reach every form that any shape does, so that
    # new constants of the choice cannot leave a kernel without a test
    from tests.test_gpu_int8_forms import FORMS
    key = lambda M, d_in, d_out, gated: (gated,) + paro.paro_w8a8_form(M, d_in, d_out, gated)
    for shape, form in FORMS.items():
        assert key(*shape)[1:] == form, shape
    rng = np.random.default_rng(6)
    u = rng.random((60000, 3))
    seen = set()
    for a, b, c in u:
        M, d_in, d_out = int(8192 ** a), 16 * int((49152 // 16) ** b), int(60000 ** c)
        seen |= {key(M, d_in, d_out, g) for g in (0, 1)}
    assert seen == {key(*s) for s in FORMS}, seen ^ {key(*s) for s in FORMS}
