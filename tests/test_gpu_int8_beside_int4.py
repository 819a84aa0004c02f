"""INT4 and 8-bit calls between one another, on one stream and in one graph (needs a B200).

Both sides start early under the kernel before them: an INT4 decode call fetches
its weights and tables, an 8-bit linear sets up and asks for weights, before the
other's output that it takes is there.  A chain of both, each call on what the call
before wrote, has to give what it gives with a wait for the GPU after every call.
"""
import numpy as np
import pytest
import torch

import oracle
from synth import linear_problem
from tests.test_gpu_int8 import BF16, DEV, _acts, _f64, _status_ok, _tables, assert_linear, assert_swiglu
from tests.tolerances import assert_linear_close

pytestmark = pytest.mark.gpu

paro = pytest.importorskip("rotation_int4_weight_b200")


class _Chain:
    """Layers of: INT4 linears (batched decode call) -> norm -> gated pair -> transformed 8-bit
    linear -> codes -> the next layer's INT4 linears; buffers, weights and workspaces its own."""

    d, side, ff, layers = 1536, 256, 2048, 4

    def __init__(self, M):
        d, ff = self.d, self.ff
        g = torch.Generator(device=DEV).manual_seed(M)
        new = lambda n: torch.empty(M, n, dtype=BF16, device=DEV)
        self.x0 = _acts(M, d, BF16, M, spread=False)
        self.p = [linear_problem(91, i, d, n, M, K=8) for i, n in enumerate((d, self.side))]
        self.int4 = [(_tables(p), paro.paro_pack_weights(torch.from_numpy(p.W).to(DEV), *_tables(p))) for p in self.p]
        r = lambda o, i: torch.randn(o, i, generator=g, device=DEV) / i ** 0.5
        self.gate, self.up = (paro.paro_pack_weights_int8(r(ff, d)) for _ in range(2))
        self.t8 = _tables(linear_problem(92, 0, ff, d, M, K=8))
        self.down = paro.paro_pack_weights_int8(r(d, ff), *self.t8)
        self.gain = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(BF16)
        self.steps, x = [], self.x0
        for _ in range(self.layers):
            a, b, s = new(d), new(self.side), dict(x=x, y=new(d), h=new(d), z=new(ff))
            s["int4"] = [paro.paro_linear(x, *t, *w, o) for (t, w), o in zip(self.int4, (a, b))]
            s |= dict(a=a, b=b, q=torch.empty(M, d, dtype=torch.int8, device=DEV), sx=torch.empty(M, device=DEV),
                      qy=torch.empty(M, d, dtype=torch.int8, device=DEV), sy=torch.empty(M, device=DEV))
            self.steps.append(s)
            x = s["y"]
        need = paro.paro_batched_workspace_bytes(self.steps[0]["int4"])
        self.ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=DEV)
        self.ws8 = torch.empty(paro.paro_rotate_w8a8_workspace_bytes(M, ff), dtype=torch.uint8, device=DEV)

    def run(self, between=lambda: None):
        for s in self.steps:
            paro.paro_rotate_w4_linear_batched(s["int4"], workspace=self.ws)
            between()
            paro.paro_rms_norm_int8(s["a"], self.gain, s["x"], hidden=s["h"], q=s["q"], sx=s["sx"])
            between()
            paro.paro_w8a8_swiglu(s["q"], s["sx"], *self.gate, *self.up, out=s["z"])
            between()
            paro.paro_rotate_w8a8_linear(s["z"], *self.t8, *self.down, out=s["y"], workspace=self.ws8)
            between()
            paro.paro_quantize_activations_int8(s["y"], q=s["qy"], sx=s["sy"])
            between()

    NAMES = ("a", "b", "h", "q", "sx", "z", "y", "qy", "sy")

    def results(self):
        torch.cuda.synchronize()
        return [s[n].clone() for s in self.steps for n in self.NAMES]

    def wipe(self):
        for s in self.steps:
            for n in self.NAMES:
                s[n].zero_() if s[n].dtype == torch.int8 else s[n].fill_(float("nan"))

    def check_first_layer(self):
        s = self.steps[0]
        for p, (t, w), n in zip(self.p, self.int4, "ab"):
            ref = oracle.rotate_w4_linear(_f64(s["x"]).astype(np.float32), p.pairs, p.cos_t, p.sin_t, p.scale,
                                          w[0].cpu().numpy().view(np.uint32), w[1].cpu().numpy(), w[2].cpu().numpy())
            assert_linear_close(s[n].float().cpu().numpy(), ref)
        assert torch.equal(s["h"], (s["a"].double() + s["x"].double()).to(BF16))
        assert np.array_equal(s["q"].cpu().numpy(), oracle.rms_norm_codes(_f64(s["h"]), _f64(self.gain), 1e-6)[0])
        assert_swiglu(s["z"], s["q"], s["sx"], *self.gate, *self.up)
        q, sx = paro.paro_quantize_activations_int8(paro.paro_rotate(s["z"], *self.t8))
        assert_linear(s["y"], q, sx, *self.down)
        assert np.array_equal(s["qy"].cpu().numpy(), oracle.row_codes(_f64(s["y"]))[0])


@pytest.mark.parametrize("M", [1, 4, 16, 40, 200])
def test_int4_calls_between_8_bit_calls(M):
    c = _Chain(M)
    c.run(torch.cuda.synchronize)
    _status_ok()
    alone = c.results()
    assert all(torch.isfinite(t).all() for t in alone)
    c.check_first_layer()
    for _ in range(20):
        c.wipe()
        c.run()
        assert all(torch.equal(a, b) for a, b in zip(c.results(), alone))
    _status_ok()


@pytest.mark.parametrize("M", [1, 4, 16, 200])
def test_int4_calls_between_8_bit_calls_in_a_graph(M):
    c = _Chain(M)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seed in range(3):
        c.x0.copy_(_acts(M, c.d, BF16, 50 + seed, spread=False))
        c.run(torch.cuda.synchronize)
        alone = c.results()
        for _ in range(5):
            c.wipe()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(c.results(), alone))
        c.check_first_layer()
    _status_ok()


def _fork_and_join(side, x, Wm):
    """Codes of Wm on a side stream, codes of x on the current one, then the linear of both
    and the codes of its output on the side stream: the join gives the linear two kernels to wait for."""
    main = torch.cuda.current_stream()
    side.wait_stream(main)
    w, sw = paro.paro_quantize_activations_int8(Wm, stream=side)
    q, sx = paro.paro_quantize_activations_int8(x)
    main.wait_stream(side)
    y = paro.paro_w8a8_linear(q, sx, w, sw)
    side.wait_stream(main)
    z, sz = paro.paro_quantize_activations_int8(y, stream=side)
    main.wait_stream(side)
    return q, sx, w, sw, y, z, sz


@pytest.mark.parametrize("M", [2, 64, 700])
def test_a_linear_that_joins_two_streams(M):
    # the codes of a large matrix take 10 times those of x, so the linear may not go by the kernel
    # before it on its own stream alone; eagerly and in a graph
    x = _acts(M, 4096, BF16, 1, spread=False)
    Wm = _acts(8960, 4096, BF16, 2, spread=False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _fork_and_join(side, x, Wm)
    for seed in range(4):
        x.copy_(_acts(M, 4096, BF16, 10 + seed, spread=False))
        Wm.copy_(_acts(8960, 4096, BF16, 20 + seed, spread=False))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = _fork_and_join(side, x, Wm)
        _status_ok()
        for got in (held, eager):
            q, sx, w, sw, y, z, sz = got
            assert_linear(y, q, sx, w, sw)
            assert torch.equal(z, paro.paro_quantize_activations_int8(y)[0])
            assert torch.equal(q, paro.paro_quantize_activations_int8(x)[0])
            assert torch.equal(w, paro.paro_quantize_activations_int8(Wm)[0])
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
