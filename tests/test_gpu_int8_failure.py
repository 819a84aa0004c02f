"""Waits of the int8 linears that run out, on the GPU without a fault (needs a B200).

The test hook paro_set_test_hooks makes one CTA of every cluster stop its copies
when its ring is full and bounds the waits to a fraction of a millisecond.  The
call then has to end with PARO_ERR_TIMEOUT, write nothing, and leave the context
usable: its copies and MMAs in flight are waited for, also where the two CTAs of
a pair have sent different numbers of stages.
"""
import pytest
import torch

from tests.test_gpu_int8 import BF16, DEV, _operands, _status_ok, assert_linear, assert_swiglu

pytestmark = pytest.mark.gpu

paro = pytest.importorskip("rotation_int4_weight_b200")
TIMEOUT = 4

# sums stored into their owners, sums read between cluster barriers, pairs of CTAs
# (one tile a pair, several); shares of d_in longer than a ring, so that copies stop
SHAPES = [(1, 14336, 1024), (20, 14336, 1000), (64, 14336, 2000), (100, 14336, 1024), (200, 14336, 1536), (1500, 2064, 2048),
          (2081, 1040, 8960)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_copies_that_stop_time_out_without_writing_output(M, d_in, d_out, which, gated):
    q, sx, w, sw, w2, s2, _ = _operands(M, d_in, d_out, 7)
    y = torch.full((M, d_out), float("nan"), dtype=BF16, device=DEV)

    def call():
        if gated:
            paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2, out=y)
        else:
            paro.paro_w8a8_linear(q, sx, w, sw, out=y)

    _status_ok()
    try:
        paro.paro_set_test_hooks(200_000, which)
        call()
        torch.cuda.synchronize()
    finally:
        paro.paro_set_test_hooks(0, False)
    assert paro.paro_get_device_status() == TIMEOUT
    assert torch.isnan(y).all(), "outputs were written although codes never came"
    call()
    _status_ok()
    if gated:
        assert_swiglu(y, q, sx, w, sw, w2, s2)
    else:
        assert_linear(y, q, sx, w, sw)


@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_a_short_bound_alone_still_completes_a_call(M, d_in, d_out):
    q, sx, w, sw, _, _, _ = _operands(M, d_in, d_out, 8)
    try:
        paro.paro_set_test_hooks(20_000_000, False)
        y = paro.paro_w8a8_linear(q, sx, w, sw)
        torch.cuda.synchronize()
    finally:
        paro.paro_set_test_hooks(0, False)
    _status_ok()
    assert_linear(y, q, sx, w, sw)
