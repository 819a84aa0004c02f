"""The operators of the 8-bit decoder path: plain forms, cases and measures.

Five operators that work together in a decoder layer whose linears hold 8-bit
weights: the weights' packing, the RMS norm that takes the residual's sum and
gives int8 codes with a scale for each token, the codes of plain activations,
the int8 linear with scales for each token and channel, and the gated pair of
linears with silu(gate) * up as its output.

Codes are whole numbers.  The code of a value v in a row whose largest
magnitude is a is the whole number nearest to 127 v / a, ties to the even one;
the row's scale is a / 127, so that a code stands for code * scale.  Codes and
scales are both returned.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one generated token: latency of the norm in front of a layer's linears
        {"name": "norm_one_token", "op": "norm", "M": 1, "d": 4096, "residual": True, "dtype": "bf16"},
        # an odd batch of an odd width, without a residual (a first layer, a draft head)
        {"name": "norm_odd", "op": "norm", "M": 517, "d": 1001, "residual": False, "dtype": "fp16"},
        # a prompt of 2048 tokens at the width of an 8B model
        {"name": "norm_prompt", "op": "norm", "M": 2048, "d": 4096, "residual": True, "dtype": "bf16"},
        # the input of the last linear of a feed-forward block, 16 sequences decoding
        {"name": "codes_16_tokens", "op": "codes", "M": 16, "d": 8960, "dtype": "bf16"},
        # the same for a prompt
        {"name": "codes_prompt", "op": "codes", "M": 2048, "d": 14336, "dtype": "bf16"},
        # loading a model: a narrow projection, an odd number of rows
        {"name": "pack_narrow", "op": "pack", "d_out": 1001, "d_in": 1536},
        # loading a model: the widest projection
        {"name": "pack_wide", "op": "pack", "d_out": 14336, "d_in": 4096},
        # one generated token through an attention projection
        {"name": "linear_one_token", "op": "linear", "M": 1, "d_in": 4096, "d_out": 4096, "bias": False, "dtype": "bf16"},
        # a short ragged chunk through a projection with a bias, rows and channels off every tile
        {"name": "linear_chunk", "op": "linear", "M": 203, "d_in": 1552, "d_out": 1100, "bias": True, "dtype": "fp16"},
        # a prompt through the last linear of a feed-forward block
        {"name": "linear_prompt", "op": "linear", "M": 2048, "d_in": 14336, "d_out": 4096, "bias": False, "dtype": "bf16"},
        # 16 sequences decoding through gate and up
        {"name": "swiglu_16_tokens", "op": "swiglu", "M": 16, "d_in": 1536, "d_out": 8960, "dtype": "bf16"},
        # a prompt through gate and up
        {"name": "swiglu_prompt", "op": "swiglu", "M": 2048, "d_in": 4096, "d_out": 14336, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm", "codes", "pack", "linear", "linear", "linear", "swiglu", "swiglu"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("norm", "codes"):
        d = _log_int(rng, 96, 16384)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        c = {"op": op, "M": _log_int(rng, 1, min(8192, (1 << 25) // d)), "d": d}
        return {**c, "residual": rng.random() < 0.7, "dtype": dtype} if op == "norm" else {**c, "dtype": dtype}
    d_in = 16 * _log_int(rng, 8, 896)
    d_out = _log_int(rng, 100, 14336)
    if rng.random() < 0.5:
        d_out = max(16, d_out // 16 * 16)
    if op == "pack":
        return {"op": op, "d_out": d_out, "d_in": min(d_in, (14336 * 4096 // d_out) // 16 * 16)}
    M = _log_int(rng, 1, min(4096, 2048 * 4096 * 14336 // (d_in * d_out)))
    c = {"op": op, "M": M, "d_in": d_in, "d_out": d_out}
    return {**c, "bias": rng.random() < 0.5, "dtype": dtype} if op == "linear" else {**c, "dtype": dtype}


def _activations(g, M, d, dtype):
    """Hidden states: a few channels carry values twenty times the others'."""
    x = torch.randn(M, d, generator=g, device="cuda")
    x[:, torch.randint(0, d, (4,), generator=g, device="cuda")] *= 20.0
    return x.to(dtype)


def _weights(g, d_out, d_in):
    """fp32 weights with a few input columns ten times the others."""
    w = torch.randn(d_out, d_in, generator=g, device="cuda").mul_(0.02)
    w[:, torch.randint(0, d_in, (4,), generator=g, device="cuda")] *= 10.0
    return w


def _int8_rows(v):
    """Codes and scales that a loaded checkpoint or the step before has left."""
    a = v.abs().amax(1, keepdim=True)
    return torch.round(v * (127.0 / a)).to(torch.int8), (a / 127.0).squeeze(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    op, s = case["op"], dict(case)
    if op in ("norm", "codes"):
        t = DTYPES[case["dtype"]]
        s["x"] = _activations(g, case["M"], case["d"], t)
        if op == "norm":
            s["gain"] = (1.0 + 0.2 * torch.randn(case["d"], generator=g, device="cuda")).to(t)
            s["res"] = _activations(g, case["M"], case["d"], t) if case["residual"] else None
        return s
    if op == "pack":
        s["W"] = _weights(g, case["d_out"], case["d_in"])
        return s
    s["q"], s["sx"] = _int8_rows(_activations(g, case["M"], case["d_in"], torch.float32))
    s["w"], s["sw"] = _int8_rows(_weights(g, case["d_out"], case["d_in"]))
    if op == "swiglu":
        s["w2"], s["sw2"] = _int8_rows(_weights(g, case["d_out"], case["d_in"]))
    else:
        s["b"] = torch.randn(case["d_out"], generator=g, device="cuda").to(DTYPES[case["dtype"]]) if case["bias"] else None
    return s


EPS = 1e-6


def _codes(v):
    """Codes of fp64 rows, and the rows' largest magnitudes.  In 64 bits: 127 v
    is exact there and a quotient next to a border between two codes stays on
    its side of it."""
    a = v.abs().amax(1, keepdim=True)
    q = torch.round(v * 127.0 / torch.where(a > 0, a, torch.ones_like(a)))
    return q.to(torch.int8), a.squeeze(1)


def _scales(a, r=1.0):
    return torch.where(a > 0, a * r / 127.0, torch.ones_like(a)).float()


def _product(q, sx, w, sw):
    return (q.float() @ w.float().T) * sx[:, None] * sw[None, :]


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
        hd = h.double()
        q, a = _codes(hd * s["gain"].double())
        sx = _scales(a, torch.rsqrt(hd.square().mean(1) + EPS))
        return (q, sx) if s["res"] is None else (q, sx, h)
    if op == "codes":
        q, a = _codes(s["x"].double())
        return q, _scales(a)
    if op == "pack":
        q, a = _codes(s["W"].double())
        return q, _scales(a)
    t = DTYPES[s["dtype"]]
    y = _product(s["q"], s["sx"], s["w"], s["sw"])
    if op == "linear":
        return (y if s["b"] is None else y + s["b"].float()).to(t)
    return (y / (1.0 + torch.exp(-y)) * _product(s["q"], s["sx"], s["w2"], s["sw2"])).to(t)


def _own(s):
    import rotation_int4_weight_b200 as paro
    op = s["op"]
    if op == "norm":
        q, sx, h = paro.paro_rms_norm_int8(s["x"], s["gain"], s["res"], eps=EPS)
        return (q, sx) if s["res"] is None else (q, sx, h)
    if op == "codes":
        return paro.paro_quantize_activations_int8(s["x"])
    if op == "pack":
        return paro.paro_pack_weights_int8(s["W"])
    t = DTYPES[s["dtype"]]
    if op == "linear":
        return paro.paro_w8a8_linear(s["q"], s["sx"], s["w"], s["sw"], s["b"], out_dtype=t)
    return paro.paro_w8a8_swiglu(s["q"], s["sx"], s["w"], s["sw"], s["w2"], s["sw2"], out_dtype=t)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    op = case["op"]
    if op in ("norm", "codes"):
        n, d = case["M"] * case["d"], case["d"]
        rows = 3 * n + 4 * case["M"]  # 16-bit values in, codes and scales out
        if op == "codes":
            return {"bytes": rows, "flops": 4 * n}
        return {"bytes": rows + 2 * d + (4 * n if case["residual"] else 0), "flops": 7 * n}
    if op == "pack":
        n = case["d_out"] * case["d_in"]
        return {"bytes": 5 * n + 4 * case["d_out"], "flops": 4 * n}
    M, k, n = case["M"], case["d_in"], case["d_out"]
    if op == "linear":
        return {"bytes": M * k + 4 * M + n * (k + 4) + (2 * n if case["bias"] else 0) + 2 * M * n, "flops": 2 * M * k * n}
    return {"bytes": M * k + 4 * M + 2 * n * (k + 4) + 2 * M * n, "flops": 4 * M * k * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]

    def nearest(t):
        low = torch.floor(t)
        part = t - low
        up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2.0) == 1.0))
        return low + up.double()

    def rows(v):
        top = torch.maximum(v.amax(dim=1), -v.amin(dim=1))
        some = top != 0
        ratio = (127.0 * v) / torch.where(some, top, 1.0)[:, None]
        return nearest(ratio).to(torch.int64).to(torch.int8), top, some

    if op in ("norm", "codes", "pack"):
        v = s["W"] if op == "pack" else s["x"]
        if op == "norm" and s["res"] is not None:
            h = (v.to(torch.float64) + s["res"].to(torch.float64)).to(v.dtype)
        else:
            h = v
        h64 = h.to(torch.float64)
        q, top, some = rows(h64 * s["gain"].to(torch.float64)[None, :] if op == "norm" else h64)
        if op == "norm":
            top = top / torch.sqrt(torch.sum(h64 * h64, dim=1) / case["d"] + EPS)
        sx = torch.where(some, top / 127.0, 1.0)
        return (q, sx, h64) if op == "norm" and s["res"] is not None else (q, sx)

    def product(w, sw):
        whole = torch.einsum("mk,nk->mn", s["q"].to(torch.float64), w.to(torch.float64))
        return whole * torch.outer(s["sx"].to(torch.float64), sw.to(torch.float64))

    y = product(s["w"], s["sw"])
    if op == "linear":
        return y if s["b"] is None else y + s["b"].to(torch.float64)
    return y * torch.sigmoid(y) * product(s["w2"], s["sw2"])
