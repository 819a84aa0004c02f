"""The int8 linears where fp32 would leave its range on the way to a finite result
(needs a B200).  Tolerances as derived in test_gpu_int8.py.
"""
import pytest
import torch

from tests.test_gpu_int8 import BF16, DEV, _operands, _status_ok, assert_linear, assert_swiglu

pytestmark = pytest.mark.gpu

paro = pytest.importorskip("rotation_int4_weight_b200")

SHAPES = [(3, 528, 131), (70, 2064, 130), (200, 4096, 1536), (2041, 144, 8962)]


@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_tokens_of_large_scales(M, d_in, d_out):
    # rows near bf16's largest value have scales up to 2^121: a sum times such a scale passes
    # fp32, the channel's scale brings it back.  Powers of two leave every product's digits alone
    q, sx, w, sw, _, _, b = _operands(M, d_in, d_out, 3)
    y0 = paro.paro_w8a8_linear(q, sx, w, sw, b.to(BF16))
    up = torch.tensor([2.0 ** 100, 2.0 ** 124, 2.0 ** 60, -2.0 ** 110], device=DEV)
    for e in up:
        sx2 = sx.clone()
        sx2[::2] *= e                    # every other token: the others stay as they are
        y = paro.paro_w8a8_linear(q, sx2, w, sw / e.abs())
        _status_ok()
        assert torch.isfinite(y).all()
        assert_linear(y[::2], q[::2], sx2[::2], w, sw / e.abs())
    sx2 = sx.clone()
    sx2[M // 2] = 2.0 ** 120
    y = paro.paro_w8a8_linear(q, sx2, w, sw, b.to(BF16))
    keep = torch.arange(M, device=DEV) != M // 2
    assert torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_gated_pairs_of_tokens_of_large_scales(M, d_in, d_out):
    q, sx, w, sw, w2, s2, _ = _operands(M, d_in, d_out, 3)
    y0 = paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2)
    for e in (2.0 ** 100, 2.0 ** 120):
        sx2 = sx.clone()
        sx2[1::3] *= e
        y = paro.paro_w8a8_swiglu(q, sx2, w, sw / e, w2, s2 / e)
        _status_ok()
        assert torch.isfinite(y[1::3]).all()
        assert_swiglu(y[1::3], q[1::3], sx2[1::3], w, sw / e, w2, s2 / e)
        keep = torch.ones(M, dtype=torch.bool, device=DEV)
        keep[1::3] = False
        y = paro.paro_w8a8_swiglu(q, sx2, w, sw, w2, s2)
        assert torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_a_sum_of_zero_stays_zero_at_any_scale(M, d_in, d_out):
    q, sx, w, sw, _, _, _ = _operands(M, d_in, d_out, 3)
    y = paro.paro_w8a8_linear(q, torch.full_like(sx, 3e38), torch.zeros_like(w), torch.full_like(sw, 3e38))
    _status_ok()
    assert not y.any()
