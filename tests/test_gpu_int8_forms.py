"""The int8 linears' forms (kernel, token tile, shares of d_in) on the GPU, every
element against the exact product (needs a B200).  Tolerances as derived in
test_gpu_int8.py.
"""
import pytest
import torch

from tests.test_gpu_int8 import BF16, DEV, FP16, _operands, _status_ok, assert_linear, assert_swiglu

pytestmark = pytest.mark.gpu

paro = pytest.importorskip("rotation_int4_weight_b200")

# (M, d_in, d_out, gated) -> (tokens, channels of a tile, shares of d_in); the last of several
# token tiles and channel tiles ragged.  Rows of y of whole 8, 4 and 2 bytes and odd ones.
FORMS = {
    (3, 16, 131, 0): (16, 128, 1), (5, 144, 333, 0): (16, 128, 2), (40, 400, 70, 0): (16, 128, 4), (7, 912, 300, 0): (16, 128, 8),
    (300, 48, 5000, 0): (32, 128, 1), (2414, 144, 50, 0): (32, 128, 2), (203, 1552, 1100, 0): (32, 128, 4), (516, 928, 6, 0): (32, 128, 8),
    (1801, 1216, 1170, 0): (64, 128, 1), (781, 2368, 1293, 0): (64, 128, 2), (548, 2928, 444, 0): (64, 128, 4), (323, 4928, 266, 0): (64, 128, 8),
    (274, 608, 8431, 0): (128, 128, 1), (139, 928, 4504, 0): (128, 128, 2), (259, 2560, 1381, 0): (128, 128, 4), (360, 2736, 724, 0): (128, 128, 8),
    (1219, 1696, 392, 0): (256, 256, 1), (1000, 1040, 5004, 0): (256, 256, 1), (2041, 1552, 4098, 0): (256, 256, 1), (1500, 2064, 2051, 0): (256, 256, 1),
    (3, 16, 131, 1): (16, 128, 1), (5, 144, 333, 1): (16, 128, 2), (40, 400, 70, 1): (16, 128, 4), (7, 912, 300, 1): (16, 128, 8),
    (4770, 272, 2, 1): (32, 128, 1), (2378, 656, 3, 1): (32, 128, 2), (203, 1552, 1100, 1): (32, 128, 4), (525, 2576, 1, 1): (32, 128, 8),
    (150, 560, 9631, 1): (64, 128, 1), (300, 4096, 1552, 1): (64, 128, 4), (259, 1504, 2186, 1): (64, 128, 2), (200, 4096, 1536, 1): (64, 128, 4), (600, 3360, 389, 1): (64, 128, 4), (567, 4832, 213, 1): (64, 128, 8),
    (256, 4096, 4096, 1): (256, 128, 1), (700, 2064, 2052, 1): (256, 128, 1), (513, 1040, 4098, 1): (256, 128, 1), (700, 4096, 1537, 1): (256, 128, 1),
}


@pytest.mark.parametrize("t", [BF16, FP16])
@pytest.mark.parametrize("M,d_in,d_out,gated", FORMS)
def test_every_form_against_the_exact_product(M, d_in, d_out, gated, t):
    q, sx, w, sw, w2, s2, b = _operands(M, d_in, d_out, M + d_in)
    assert paro.paro_w8a8_form(M, d_in, d_out, gated) == FORMS[M, d_in, d_out, gated]
    y = torch.full((M * d_out + 64,), 7.0, dtype=t, device=DEV)
    out = y[:M * d_out].view(M, d_out)
    if gated:
        sw, s2 = sw * 20, s2 * 20
        paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2, out=out)
        _status_ok()
        assert_swiglu(out, q, sx, w, sw, w2, s2)
    else:
        paro.paro_w8a8_linear(q, sx, w, sw, b.to(t), out=out)
        _status_ok()
        assert_linear(out, q, sx, w, sw, b.to(t))
    assert (y[M * d_out:] == 7).all()


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


@pytest.mark.parametrize("t", [BF16, FP16])
@pytest.mark.parametrize("d_in,d_out", [(4096, 1536), (528, 4098), (2064, 5001)])
def test_a_token_does_not_depend_on_the_form_that_takes_it(d_in, d_out, t):
    # the same rows of q alone, in small calls and in large ones: bit for bit
    M = 2100
    q, sx, w, sw, w2, s2, b = _operands(M, d_in, d_out, 11)
    sx[7] = 2.0 ** 100
    b, sw, s2 = b.to(t), sw * 20, s2 * 20
    y = paro.paro_w8a8_linear(q, sx, w, sw, b, out_dtype=t)
    z = paro.paro_w8a8_swiglu(q, sx, w, sw, w2, s2, out_dtype=t)
    forms = {paro.paro_w8a8_form(M, d_in, d_out)}
    for lo, n in ((7, 1), (0, 16), (40, 33), (512, 100), (0, 300), (2099, 1), (1024, 700)):
        rows = slice(lo, lo + n)
        qs, ss = q[rows].contiguous(), sx[rows].contiguous()
        assert torch.equal(paro.paro_w8a8_linear(qs, ss, w, sw, b, out_dtype=t), y[rows])
        assert torch.equal(paro.paro_w8a8_swiglu(qs, ss, w, sw, w2, s2, out_dtype=t), z[rows])
        forms.add(paro.paro_w8a8_form(n, d_in, d_out))
    _status_ok()
    assert len(forms) >= 4
