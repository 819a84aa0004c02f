"""The 8-bit path on the GPU against its oracle (oracle/int8.py) (needs a B200).

Codes and hidden states are compared exactly.  Tolerances, derived:
  * scales: the sum of squares is fp32 with at most 64 additions in a thread and
    10 levels of a tree, each half a step (2^-24), halved by the square root:
    37 * 2^-24, the final rounding and eps as fp32: 40 * 2^-24 in all;
    2^-24 for scales without a norm;
  * linear: exact sums; the conversion to fp32, two products and the bias are
    half a fp32 step each (4 * 2^-24 of |product| + |bias|), then half a step of
    the output type (finfo.eps / 2 of the value, or half its smallest subnormal);
  * gated pair: g and u are within 3 * 2^-24; g / (1 + exp(-g)) turns a relative
    error e of g into at most (1 + |g|) e; fast exp is within 2 + 1.2 |g| steps of
    2^-23 (scaling its argument by log2 e), the fast quotient within 2 steps, the
    product half a step: (2 + |g|) 2^-20 of the value covers their sum; 3e-36 |u|
    where 1 + exp(-g) passes 2^126 and the fast quotient is flushed to zero; then
    the output's rounding.
"""
import numpy as np
import pytest
import torch

import oracle
from synth import linear_problem

pytestmark = pytest.mark.gpu

paro = pytest.importorskip("rotation_int4_weight_b200")
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


def _f64(t):
    return t.detach().double().cpu().numpy()


def _status_ok():
    torch.cuda.synchronize()
    assert paro.paro_get_device_status() == 0


def _scales_close(got, ref, steps):
    got, ref = got.double().cpu().numpy(), np.asarray(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= (steps * 2.0 ** -24 * np.abs(ref) + 2.0 ** -150)[ok]).all()


def _rounding(ref, t):
    f = torch.finfo(t)
    return np.abs(ref) * (f.eps / 2) + f.tiny * f.eps / 2


def _acts(M, d, t, seed, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, d, generator=g, device=DEV)
    if spread:
        x *= torch.rand(M, 1, generator=g, device=DEV) * 30 + 0.01
        x[:, d // 3] *= 20
    return x.to(t)


# ------------------------------------------------------------------------ codes
WIDTHS = [(1, 1), (2, 7), (3, 8), (5, 9), (1, 96), (7, 255), (9, 257), (4, 1000), (33, 1001), (1, 1536), (301, 1536),
          (5, 4095), (2, 4096), (300, 4097), (3, 8191), (16, 8960), (297, 8960), (2, 14336), (300, 14336), (2, 24577),
          (1, 32767), (297, 32768), (2, 40000), (1, 49151), (2, 49152), (298, 49145)]


@pytest.mark.parametrize("t", [BF16, FP16])
@pytest.mark.parametrize("M,d", WIDTHS)
def test_quantize_int8(M, d, t):
    x = _acts(M, d, t, 100 * M + d)
    if M > 2:
        x[1] = 0
    q, sx = paro.paro_quantize_activations_int8(x)
    _status_ok()
    rq, rs = oracle.row_codes(_f64(x))
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 1)


@pytest.mark.parametrize("t", [BF16, FP16])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("M,d", WIDTHS)
def test_rms_norm_int8(M, d, res, t):
    x = _acts(M, d, t, M + d)
    r = _acts(M, d, t, M + d + 1) if res else None
    gain = (1 + 0.3 * torch.randn(d, generator=torch.Generator(device=DEV).manual_seed(d), device=DEV)).to(t)
    if M > 2:
        x[1] = 0
        if res:
            r[1] = 0
    q, sx, hid = paro.paro_rms_norm_int8(x, gain, r, eps=1e-5)
    _status_ok()
    h = x if not res else (x.double() + r.double()).to(t)
    if res:
        assert torch.equal(hid, h)
    else:
        assert hid is None
    rq, rs = oracle.rms_norm_codes(_f64(h), _f64(gain), float(np.float32(1e-5)))
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 40)


@pytest.mark.parametrize("t", [BF16, FP16])
def test_codes_at_every_border(t):
    # a row of a = 127 * 2 in steps of the type: every tie k + 1/2 and its neighbours
    v = torch.arange(-254, 255, device=DEV).float()
    near = torch.cat([v, torch.nextafter(v.to(t), torch.tensor(1e4, dtype=t, device=DEV)).float(),
                      torch.nextafter(v.to(t), torch.tensor(-1e4, dtype=t, device=DEV)).float()]).clamp(-254, 254)
    rows = torch.stack([near, near * 0.5, near * 2.0 ** -10]).to(t)
    q, sx = paro.paro_quantize_activations_int8(rows)
    rq, rs = oracle.row_codes(_f64(rows))
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 1)


@pytest.mark.parametrize("t", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 1001, 4096])
def test_rows_that_are_not_finite_void_themselves_only(d, t):
    x = _acts(6, d, t, 5)
    x[1, d - 1] = float("nan")
    x[3, 0] = float("inf")
    x[4, d // 2] = -float("inf")
    gain = torch.ones(d, dtype=t, device=DEV)
    gain[d // 2] = 0          # 0 * inf is not finite either
    for q, sx in (paro.paro_quantize_activations_int8(x), paro.paro_rms_norm_int8(x, gain)[:2]):
        bad = torch.tensor([False, True, False, True, True, False], device=DEV)
        assert torch.equal(torch.isnan(sx), bad)
        assert not q[bad].any()
    rq, rs = oracle.row_codes(_f64(x))
    assert np.array_equal(paro.paro_quantize_activations_int8(x)[0].cpu().numpy(), rq)
    w, sw = torch.ones(16, 16 * ((d + 15) // 16), dtype=torch.int8, device=DEV), torch.ones(16, device=DEV)
    if d % 16 == 0:
        q, sx = paro.paro_quantize_activations_int8(x)
        y = paro.paro_w8a8_linear(q, sx, w, sw)
        assert torch.equal(torch.isnan(y).all(1), bad) and torch.equal(torch.isnan(y).any(1), bad)


@pytest.mark.parametrize("factor", [2.0 ** -125, 2.0 ** -110, 2.0 ** -60, 2.0 ** 60, 2.0 ** 70, 2.0 ** 110])
def test_rows_at_the_ends_of_the_range(factor):
    # squares beyond fp32's range, or below it; eps 0 so that nothing covers it
    x = (_acts(3, 512, BF16, 3, spread=False).float() * factor).to(BF16)
    gain = torch.full((512,), 0.5, dtype=BF16, device=DEV)
    q, sx, _ = paro.paro_rms_norm_int8(x, gain, eps=0.0)
    rq, rs = oracle.rms_norm_codes(_f64(x), _f64(gain), 0.0)
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 40)
    q, sx = paro.paro_quantize_activations_int8(x)
    rq, rs = oracle.row_codes(_f64(x))
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 1)


def test_zero_gain_and_zero_rows():
    x = _acts(3, 64, BF16, 3)
    q, sx, _ = paro.paro_rms_norm_int8(x, torch.zeros(64, dtype=BF16, device=DEV))
    assert not q.any() and (sx == 1).all()
    q, sx, _ = paro.paro_rms_norm_int8(torch.zeros_like(x), eps=0.0)
    assert not q.any() and (sx == 1).all()


@pytest.mark.parametrize("d", [1000, 1001])
def test_norm_in_place_and_rows_behind_the_last(d):
    M = 9
    x, r = _acts(M, d, BF16, 1), _acts(M, d, BF16, 2)
    gain = _acts(1, d, BF16, 3, spread=False)[0]
    q0, s0, h0 = paro.paro_rms_norm_int8(x, gain, r)
    for which in ("x", "r"):
        a, b = x.clone(), r.clone()
        q, s, h = paro.paro_rms_norm_int8(a, gain, b, hidden=a if which == "x" else b)
        assert h is (a if which == "x" else b)
        assert torch.equal(h, h0) and torch.equal(q, q0) and torch.equal(s, s0)
    # outputs inside larger buffers: the values behind the last row stay
    hb = torch.full((M * d + 64,), 7.0, dtype=BF16, device=DEV)
    qb = torch.full((M * d + 64,), 77, dtype=torch.int8, device=DEV)
    sb = torch.full((M + 8,), 7.0, device=DEV)
    paro.paro_rms_norm_int8(x, gain, r, hidden=hb[:M * d].view(M, d), q=qb[:M * d].view(M, d), sx=sb[:M])
    assert torch.equal(hb[:M * d].view(M, d), h0) and (hb[M * d:] == 7).all()
    assert torch.equal(qb[:M * d].view(M, d), q0) and (qb[M * d:] == 77).all()
    assert torch.equal(sb[:M], s0) and (sb[M:] == 7).all()


@pytest.mark.parametrize("d_out,d_in", [(1, 16), (5, 48), (300, 1536), (1001, 1552), (64, 49152), (300, 40000)])
def test_pack_int8_plain(d_out, d_in):
    g = torch.Generator(device=DEV).manual_seed(d_in)
    W = torch.randn(d_out, d_in, generator=g, device=DEV) * 0.02
    W[:, 3] *= 10
    if d_out > 4:
        W[2] = 0
        W[3] *= 2.0 ** -120
    qw, sw = paro.paro_pack_weights_int8(W)
    _status_ok()
    rq, rs = oracle.row_codes(_f64(W))
    assert np.array_equal(qw.cpu().numpy(), rq)
    _scales_close(sw, rs, 1)


def _tables(p):
    return (torch.from_numpy(p.pairs.view(np.int16)).to(DEV), torch.from_numpy(p.cos_t).to(DEV),
            torch.from_numpy(p.sin_t).to(DEV), torch.from_numpy(p.scale).to(DEV))


@pytest.mark.parametrize("d_out,d_in", [(96, 512), (33, 1552)])
def test_pack_int8_folds_the_transform(d_out, d_in):
    p = linear_problem(81, 0, d_in, d_out, 1, K=8)
    W = torch.from_numpy(p.W).to(DEV)
    ws = torch.empty(d_out, d_in, device=DEV)
    qw, sw = paro.paro_pack_weights_int8(W, *_tables(p), workspace=ws)
    _status_ok()
    # the fold in fp32, against the oracle's fp64 one: 8 stages of two roundings of the row's scale
    ref = oracle.fold_weights(p.W, p.pairs, p.cos_t, p.sin_t, p.scale)
    err = np.abs(_f64(ws) - ref)
    assert (err <= 2.0 ** -19 * np.abs(ref).max(axis=1, keepdims=True)).all()
    rq, rs = oracle.row_codes(_f64(ws))   # the codes of the fold that the call quantised
    assert np.array_equal(qw.cpu().numpy(), rq)
    _scales_close(sw, rs, 1)


# ---------------------------------------------------------------------- linears
def _operands(M, d_in, d_out, seed, extreme=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lo = (lambda s: torch.full(s, -128, dtype=torch.int8, device=DEV)) if extreme else \
        (lambda s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8))
    return (lo((M, d_in)), torch.rand(M, generator=g, device=DEV) * 0.05 + 1e-3, lo((d_out, d_in)),
            torch.rand(d_out, generator=g, device=DEV) * 2e-3 / d_in ** 0.5 + 1e-6,
            torch.randint(-128, 128, (d_out, d_in), generator=g, device=DEV, dtype=torch.int8),
            torch.rand(d_out, generator=g, device=DEV) * 2e-3 / d_in ** 0.5 + 1e-6,
            torch.randn(d_out, generator=g, device=DEV))


def _gpu_product(q, sx, w, sw):
    # fp64 on the device: the same whole numbers as the numpy oracle, faster
    return (q.double() @ w.double().T) * sx.double()[:, None] * sw.double()[None, :]


def assert_linear(y, q, sx, w, sw, bias=None):
    p = _gpu_product(q, sx, w, sw).cpu().numpy()
    b = 0.0 if bias is None else _f64(bias)[None, :]
    ref = p + b
    tol = 4 * 2.0 ** -24 * (np.abs(p) + np.abs(b)) + _rounding(ref, y.dtype)
    err = np.abs(_f64(y) - ref)
    assert (err <= tol * (1 + 1e-3)).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())


def assert_swiglu(y, q, sx, w, sw, w2, s2):
    g, u = _gpu_product(q, sx, w, sw), _gpu_product(q, sx, w2, s2)
    ref = (g * torch.sigmoid(g) * u).cpu().numpy()
    g, u = g.cpu().numpy(), u.cpu().numpy()
    tol = np.abs(ref) * (2 + np.abs(g)) * 2.0 ** -20 + 3e-36 * np.abs(u) + _rounding(ref, y.dtype)
    err = np.abs(_f64(y) - ref)
    assert (err <= tol * (1 + 1e-3)).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())


SHAPES = [(1, 16, 1), (1, 128, 128), (1, 4096, 4096), (2, 1536, 256), (3, 1552, 1001), (4, 512, 512), (5, 144, 333),
          (8, 8960, 1536), (13, 1536, 8960), (16, 14336, 4096), (17, 4096, 1024), (31, 272, 129), (33, 1536, 1536),
          (48, 640, 40), (64, 4096, 4096), (65, 2064, 127), (96, 4096, 520), (127, 512, 2049), (128, 4096, 1024),
          (129, 1536, 1536), (203, 1552, 1100), (255, 16, 300), (256, 4096, 4096), (257, 1040, 515), (300, 48, 5000),
          (511, 2048, 250), (700, 4096, 1537), (1025, 528, 1283), (2048, 1536, 8960), (2049, 1024, 96), (4096, 256, 1)]


@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_w8a8_linear(M, d_in, d_out):
    q, sx, w, sw, _, _, b = _operands(M, d_in, d_out, M + d_in + d_out)
    t = FP16 if (M + d_out) % 2 else BF16
    y = paro.paro_w8a8_linear(q, sx, w, sw, out_dtype=t)
    _status_ok()
    assert y.dtype == t
    assert_linear(y, q, sx, w, sw)
    t = BF16 if t is FP16 else FP16
    y = paro.paro_w8a8_linear(q, sx, w, sw, b.to(t), out_dtype=t)
    _status_ok()
    assert_linear(y, q, sx, w, sw, b.to(t))


@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_w8a8_swiglu(M, d_in, d_out):
    q, sx, w, sw, w2, s2, _ = _operands(M, d_in, d_out, M + d_in + d_out)
    sw, s2 = sw * 20, s2 * 20     # gates of both signs well into silu's curved part
    for t in (BF16, FP16):
        y = paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2, out_dtype=t)
        _status_ok()
        assert_swiglu(y, q, sx, w, sw, w2, s2)


@pytest.mark.parametrize("M", [1, 16, 300])
def test_w8a8_largest_sums(M):
    # every code -128 over the widest input: |sum| = 49152 * 2^14 < 2^31
    q, sx, w, sw, _, _, _ = _operands(M, 49152, 130, 1, extreme=True)
    y = paro.paro_w8a8_linear(q, sx, w, sw)
    _status_ok()
    assert_linear(y, q, sx, w, sw)


@pytest.mark.parametrize("M", [1, 40, 520])
def test_w8a8_outputs_inside_larger_buffers(M):
    d_in, d_out = 528, 321
    q, sx, w, sw, w2, s2, _ = _operands(M, d_in, d_out, 9)
    buf = torch.full((M * d_out + 512,), 7.0, dtype=BF16, device=DEV)
    out = buf[:M * d_out].view(M, d_out)
    y0 = paro.paro_w8a8_linear(q, sx, w, sw)
    assert paro.paro_w8a8_linear(q, sx, w, sw, out=out) is out
    assert torch.equal(out, y0) and (buf[M * d_out:] == 7).all()
    z0 = paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2)
    paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2, out=out)
    assert torch.equal(out, z0) and (buf[M * d_out:] == 7).all()


@pytest.mark.parametrize("M", [1, 16, 200, 600])
def test_w8a8_repeats_bit_for_bit_and_leaves_inputs(M):
    args = _operands(M, 4096, 1536, 4)[:6]
    kept = [a.clone() for a in args]
    y = paro.paro_w8a8_swiglu(*args)
    for _ in range(3):
        assert torch.equal(paro.paro_w8a8_swiglu(*args), y)
    assert all(torch.equal(a, b) for a, b in zip(args, kept))


def test_gates_far_from_zero():
    # g from -2000 to 2000 and u of both signs: no NaN, zeros where silu vanishes
    q = torch.arange(-100, 101, device=DEV).to(torch.int8).view(-1, 1).repeat(1, 16).contiguous()
    M = q.shape[0]
    sx = torch.ones(M, device=DEV)
    w, w2 = torch.ones(4, 16, dtype=torch.int8, device=DEV), -torch.ones(4, 16, dtype=torch.int8, device=DEV)
    sw = torch.tensor([1.25, 0.05, 1e-3, 1e-6], device=DEV)
    y = paro.paro_w8a8_swiglu(q, sx, w, sw, w2, torch.ones(4, device=DEV))
    assert_swiglu(y, q, sx, w, sw, w2, torch.ones(4, device=DEV))


# ------------------------------------------------------------------ as it is used
def _block(x, res, t, W, stream=None):
    """A feed-forward block of 8-bit linears: norm, gate and up, codes, down."""
    q, sx, h = paro.paro_rms_norm_int8(x, W["gain"], res, stream=stream)
    a = paro.paro_w8a8_swiglu(q, sx, *W["gate"], *W["up"], out_dtype=t, stream=stream)
    qa, sa = paro.paro_quantize_activations_int8(a, stream=stream)
    y = paro.paro_w8a8_linear(qa, sa, *W["down"], W["bias"], out_dtype=t, stream=stream)
    return q, sx, h, a, qa, sa, y


def _block_weights(d, ff, t, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda o, i: paro.paro_pack_weights_int8(torch.randn(o, i, generator=g, device=DEV) * 0.02)
    return dict(gate=r(ff, d), up=r(ff, d), down=r(d, ff), bias=torch.randn(d, generator=g, device=DEV).to(t),
                gain=(1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(t))


def _block_check(got, x, res, t, W):
    """Every step against the oracle on what the step before it gave."""
    q, sx, h, a, qa, sa, y = got
    assert torch.equal(h, (x.double() + res.double()).to(t))
    rq, rs = oracle.rms_norm_codes(_f64(h), _f64(W["gain"]), float(np.float32(1e-6)))
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 40)
    assert_swiglu(a, q, sx, *W["gate"], *W["up"])
    rq, rs = oracle.row_codes(_f64(a))
    assert np.array_equal(qa.cpu().numpy(), rq)
    _scales_close(sa, rs, 1)
    assert_linear(y, qa, sa, *W["down"], W["bias"])


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [BF16, FP16])
@pytest.mark.parametrize("M", [1, 16, 130])
def test_feed_forward_block(M, t):
    d, ff = 512, 1552
    W = _block_weights(d, ff, t)
    x, res = _acts(M, d, t, 1, spread=False), _acts(M, d, t, 2, spread=False)
    got = _block(x, res, t, W)
    _status_ok()
    _block_check(got, x, res, t, W)


@pytest.mark.parametrize("M", [1, 16, 130, 600])
def test_feed_forward_block_on_another_stream_and_in_a_graph(M):
    d, ff, t = 512, 1552, BF16
    W = _block_weights(d, ff, t)
    x, res = _acts(M, d, t, 1, spread=False), _acts(M, d, t, 2, spread=False)
    alone = _block(x, res, t, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _block(x, res, t, W, stream=side)
    torch.cuda.synchronize()
    assert _same(got, alone)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _block(x, res, t, W)
    for seed in (3, 4):
        x.copy_(_acts(M, d, t, seed, spread=False))
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, _block(x, res, t, W))
        _block_check(got, x, res, t, W)
    _status_ok()


def test_two_streams_at_once():
    # calls hold no state: many in flight on two streams give what they give alone
    sets = [_operands(M, 4096, 1552, M)[:6] for M in (1, 300)]
    alone = [paro.paro_w8a8_swiglu(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k in (0, 1):
            got[k].append(paro.paro_w8a8_swiglu(*sets[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(y, alone[k]) for y in got[k])
    _status_ok()


def test_both_linear_kernels_at_once():
    # pairs of CTAs with all of tensor memory and clusters with some of it, on three
    # streams: neither may take what the other's half waits for
    big, small = _operands(1500, 2064, 2048, 1)[:4], _operands(100, 2064, 2048, 2)[:4]
    gate = _operands(40, 512, 1552, 3)[:6]
    calls = [lambda s: paro.paro_w8a8_linear(*big, stream=s), lambda s: paro.paro_w8a8_linear(*small, stream=s),
             lambda s: paro.paro_w8a8_swiglu(*gate, stream=s)]
    alone = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(40):
        for k, c in enumerate(calls):
            got[k].append(c(streams[k]))
    torch.cuda.synchronize()
    for k, ys in enumerate(got):
        assert all(torch.equal(y, alone[k]) for y in ys)
    _status_ok()


def test_codes_of_a_matrix_as_weights_right_away():
    # the row codes of a 16-bit matrix are weights too: the linear right behind the call
    # that wrote them reads them whole
    x = _acts(4, 4096, BF16, 1, spread=False)
    for seed in range(6):
        Wm = _acts(1536, 4096, BF16, 10 + seed, spread=False)
        q, sx = paro.paro_quantize_activations_int8(x)
        w, sw = paro.paro_quantize_activations_int8(Wm)
        y = paro.paro_w8a8_linear(q, sx, w, sw)
        y2 = paro.paro_w8a8_linear(q, sx, w, sw)
        torch.cuda.synchronize()
        assert_linear(y, q, sx, w, sw)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("M,d_in,d_out", [(1, 1536, 1536), (5, 512, 333), (40, 1552, 96), (300, 1536, 256)])
def test_rotate_w8a8_linear(M, d_in, d_out):
    p = linear_problem(82, 0, d_in, d_out, M, K=8)
    tables = _tables(p)
    W = torch.from_numpy(p.W).to(DEV)
    qw, sw = paro.paro_pack_weights_int8(W, *tables)
    x = torch.from_numpy(p.x).to(DEV).to(BF16)
    bias = torch.randn(d_out, device=DEV).to(BF16)
    y = paro.paro_rotate_w8a8_linear(x, *tables, qw, sw, bias)
    _status_ok()
    # the same transform alone gives the x~ whose codes the call took
    q, sx = paro.paro_quantize_activations_int8(paro.paro_rotate(x, *tables))
    assert torch.equal(y, paro.paro_w8a8_linear(q, sx, qw, sw, bias))
    assert_linear(y, q, sx, qw, sw, bias)
    # and the whole stays near x W^T: half a code of each operand against the other's magnitude
    xt, wt = q.double() * sx.double()[:, None], qw.double() * sw.double()[:, None]
    near = (sx.double()[:, None] * 0.51 * wt.abs().sum(1)[None, :] + 0.51 * sw.double()[None, :] * xt.abs().sum(1)[:, None]
            + 0.26 * d_in * sx.double()[:, None] * sw.double()[None, :])
    full = x.double() @ W.double().T + bias.double()
    slack = 2.0 ** -7 * (full.abs() + (xt.abs() @ wt.abs().T))
    assert ((y.double() - full).abs() <= near + slack).all()


def test_rotate_w8a8_linear_without_a_transform():
    # K = 0 and no scale: the plain 8-bit linear on bf16 activations
    x = _acts(5, 512, BF16, 1, spread=False)
    qw, sw = paro.paro_pack_weights_int8(torch.randn(96, 512, device=DEV))
    y = paro.paro_rotate_w8a8_linear(x, None, None, None, None, qw, sw)
    _status_ok()
    q, sx = paro.paro_quantize_activations_int8(x)
    assert torch.equal(y, paro.paro_w8a8_linear(q, sx, qw, sw))


@pytest.mark.parametrize("d", [8, 24, 4088, 8184, 49144])
@pytest.mark.parametrize("M", [3, 700])
def test_norm_of_widths_that_are_multiples_of_8_only(M, d):
    x, r = _acts(M, d, BF16, 1), _acts(M, d, BF16, 2)
    gain = _acts(1, d, BF16, 3, spread=False)[0]
    q, sx, h = paro.paro_rms_norm_int8(x, gain, r)
    assert torch.equal(h, (x.double() + r.double()).to(BF16))
    rq, rs = oracle.rms_norm_codes(_f64(h), _f64(gain), float(np.float32(1e-6)))
    assert np.array_equal(q.cpu().numpy(), rq)
    _scales_close(sx, rs, 40)


def test_offsets_beyond_32_bits():
    # more than 2^31 values in x, q and y: the first and last rows are looked at
    M, d = 70001, 32768
    x = torch.zeros(M, d, dtype=BF16, device=DEV)
    rows = [0, 65535, 65536, M - 1]
    x[rows] = _acts(4, d, BF16, 1)
    q, sx = paro.paro_quantize_activations_int8(x)
    rq, rs = oracle.row_codes(_f64(x[rows]))
    assert np.array_equal(q[rows].cpu().numpy(), rq)
    _scales_close(sx[rows], rs, 1)
    assert not q[1000].any() and not q[65537:].any(1)[:-1].any()
    del x, q
    M, d_in, d_out = 70001, 32, 32000
    q, sx, w, sw, _, _, _ = _operands(M, d_in, d_out, 2)
    y = paro.paro_w8a8_linear(q, sx, w, sw)
    _status_ok()
    rows = [0, 1, 67107, 67108, 67109, M - 2, M - 1]   # 2^31 / 32000 = 67108.9
    assert_linear(y[rows], q[rows], sx[rows], w, sw)


def test_more_token_tiles_than_a_grid_has_rows():
    # beyond 65535 tiles of 128 tokens (64 for a gated pair): only the kernel for many tokens takes them
    M, d_in, d_out = 65535 * 128 + 3, 16, 5
    q, sx, w, sw, w2, s2, b = _operands(M, d_in, d_out, 4)
    rows = torch.cat([torch.arange(300, device=DEV), torch.arange(0, M, 4099, device=DEV),
                      torch.arange(M - 300, M, device=DEV)])
    y = paro.paro_w8a8_linear(q, sx, w, sw, b.to(BF16))
    _status_ok()
    assert_linear(y[rows], q[rows], sx[rows], w, sw, b.to(BF16))
    y = paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2)
    _status_ok()
    assert_swiglu(y[rows], q[rows], sx[rows], w, sw, w2, s2)


@pytest.mark.parametrize("M,d_out", [(8, 1536), (100, 520), (1100, 2049)])
def test_scales_that_are_not_finite_void_their_rows_and_channels_only(M, d_out):
    q, sx, w, sw, _, _, _ = _operands(M, 528, d_out, 5)
    alone = paro.paro_w8a8_linear(q, sx, w, sw)
    sx2, sw2 = sx.clone(), sw.clone()
    sx2[[0, M - 1]], sw2[[3, d_out - 1]] = float("nan"), float("nan")
    y = paro.paro_w8a8_linear(q, sx2, w, sw2)
    _status_ok()
    bad = torch.isnan(sx2)[:, None] | torch.isnan(sw2)[None, :]
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], alone[~bad])


def test_calls_from_two_threads():
    import threading
    sets = [_operands(M, 2064, 1100, M)[:4] for M in (3, 700)]
    alone = [paro.paro_w8a8_linear(*s) for s in sets]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[k] = [paro.paro_w8a8_linear(*sets[k]) for _ in range(50)]
            s.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for k in (0, 1):
        assert len(got[k]) == 50 and all(torch.equal(y, alone[k]) for y in got[k])
    _status_ok()


def test_refusals():
    q = torch.zeros(2, 64, dtype=torch.int8, device=DEV)
    s, w, sw = torch.ones(2, device=DEV), torch.zeros(8, 64, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    x = torch.zeros(2, 64, dtype=BF16, device=DEV)
    ok = paro.paro_w8a8_linear(q, s, w, sw)
    assert ok.shape == (2, 8)
    for bad in (dict(sx=torch.ones(1, device=DEV)), dict(sx=s.double()), dict(qweight=w[:, :48]),
                dict(qweight=w.t().contiguous().t()), dict(wscales=sw[:4]), dict(wscales=sw.cpu()),
                dict(bias=torch.ones(8, device=DEV)), dict(bias=torch.ones(7, dtype=BF16, device=DEV)),
                dict(out=torch.zeros(2, 9, dtype=BF16, device=DEV))):
        with pytest.raises(ValueError):
            paro.paro_w8a8_linear(**(dict(q=q, sx=s, qweight=w, wscales=sw) | bad))
    with pytest.raises(paro.ParoError, match="multiple of 16"):
        paro.paro_w8a8_linear(q[:, :40].contiguous(), s, w[:, :40].contiguous(), sw)
    with pytest.raises(paro.ParoError, match="16-byte"):
        paro.paro_quantize_activations_int8(torch.zeros(131, dtype=BF16, device=DEV)[1:129].view(2, 64))
    with pytest.raises(paro.ParoError, match="in-place"):
        b = torch.zeros(3, 64, dtype=BF16, device=DEV)
        paro.paro_rms_norm_int8(b[:2], None, x, hidden=b[1:])
    with pytest.raises(ValueError, match="residual"):
        paro.paro_rms_norm_int8(x, None, x.to(FP16))
    with pytest.raises(ValueError, match="gain"):
        paro.paro_rms_norm_int8(x, torch.ones(63, dtype=BF16, device=DEV))
    with pytest.raises(paro.ParoError, match="eps"):
        paro.paro_rms_norm_int8(x, eps=-1.0)
    # nothing of that was enqueued, and no rows at all are fine
    assert paro.paro_w8a8_linear(q[:0], s[:0], w, sw).shape == (0, 8)
    assert paro.paro_quantize_activations_int8(x[:0])[0].shape == (0, 64)
    _status_ok()
