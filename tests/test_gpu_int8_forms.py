"""The int8 linears' forms (kernel, token tile, shares of d_in) on the GPU, every
element against the exact product (needs a B200).  Tolerances as derived in
test_gpu_int8.py.
"""
import pytest
import torch

from tests.test_gpu_int8 import BF16, FP16, _operands, _status_ok, assert_linear, assert_swiglu

pytestmark = pytest.mark.gpu

paro = pytest.importorskip("rotation_int4_weight_b200")


@pytest.mark.parametrize("M", [2049, 2081, 2178])
def test_ragged_last_token_tile_among_many_tiles_a_pair(M):
    # the kernel for many tokens, rows of y by TMA: a pair of SMs takes several tiles,
    # some of them behind the last tokens (M % 256 = 1, 33, 130), at a d_in so short that
    # the next tile's sums are there at once.  A tile's stores have to have read their
    # boxes in shared memory before the next tile, whose warps may have no token, takes them.
    d_in, d_out = 128, 8960
    q, sx, w, sw, w2, s2, b = _operands(M, d_in, d_out, M)
    y = paro.paro_w8a8_linear(q, sx, w, sw, b.to(BF16))
    z = paro.paro_w8a8_swiglu(q, sx, w, sw * 20, w2, s2 * 20, out_dtype=FP16)
    _status_ok()
    assert_linear(y, q, sx, w, sw, b.to(BF16))
    assert_swiglu(z, q, sx, w, sw * 20, w2, s2 * 20)
    for _ in range(100):
        again = paro.paro_w8a8_linear(q, sx, w, sw, b.to(BF16))
        assert torch.equal(again, y)
        again = paro.paro_w8a8_swiglu(q, sx, w, sw * 20, w2, s2 * 20, out_dtype=FP16)
        assert torch.equal(again, z)
