"""The microscaled 4-bit product and the layer normalisation, as measurements: their cases, a plain form in
elementary torch operations, and the definition in 64 bits.

Operators (``case["op"]``):

* ``quantize``: x[M][K] to MXFP4 (blocks of 32 along K share a power of two), the values the codes stand for.
* ``product``: Y = Xv Wv^T of two matrices already held as MXFP4 codes (Xv, Wv: the values).
* ``fused``: the same product of an un-quantised x[M][K] and MXFP4 weights.
* ``layernorm``: y = (x - mean) rstd weight + bias over each row, with mean and rstd.
* ``layernorm_backward``: the gradients of x, weight and bias.

The codes' layout in memory is the library's documented one: 1024-byte tiles of 16 rows x 128 columns, 16 bytes
(32 codes, low nibble first) per row and block, and one 32-bit word of four scales (tiles 4c .. 4c + 3) per row
and block.
"""
import math

import torch

own = False

DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of a 4-bit float with 2 exponent bits and 1 mantissa bit
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # latent fp32 weights of one 2B-class up projection, quantised when a model is loaded
        {"name": "quantize_weights_2b", "op": "quantize", "m": 6912, "n": 0, "k": 2560, "x": "f32", "y": "f32"},
        # a batch of token rows whose length is no multiple of a block, a vector or a tile
        {"name": "quantize_acts_ragged", "op": "quantize", "m": 1003, "n": 0, "k": 7001, "x": "bf16", "y": "bf16"},
        # a few dozen sequences decoded together, with odd sizes on every axis
        {"name": "product_37_tokens_ragged", "op": "product", "m": 37, "n": 6909, "k": 2570, "x": "bf16", "y": "f32"},
        # prefill of 2048 tokens through a 2B-class up projection, activations quantised once for gate and up
        {"name": "product_prefill_2b", "op": "product", "m": 2048, "n": 6912, "k": 2560, "x": "bf16", "y": "f32"},
        # one token through a 2B-class up projection: the smallest call, where latency counts
        {"name": "fused_1_token_2b", "op": "fused", "m": 1, "n": 6912, "k": 2560, "x": "bf16", "y": "f32"},
        # 16 sequences' tokens through a 2B-class down projection
        {"name": "fused_16_tokens_2b_down", "op": "fused", "m": 16, "n": 2560, "k": 6912, "x": "bf16", "y": "f32"},
        # one token through a 100B-class down projection: the weights' bytes are what it costs
        {"name": "fused_1_token_100b_down", "op": "fused", "m": 1, "n": 8192, "k": 28672, "x": "f32", "y": "f32"},
        # prefill of 2048 tokens through a 100B-class up projection, output for the next layer in bf16
        {"name": "fused_prefill_100b", "op": "fused", "m": 2048, "n": 28672, "k": 8192, "x": "bf16", "y": "bf16"},
        # the norm in front of one decode step's projections
        {"name": "layernorm_16_tokens_2b", "op": "layernorm", "m": 16, "n": 0, "k": 2560, "x": "bf16", "y": "bf16"},
        # the norm over a long prefill, or over a training batch, of a 100B-class model
        {"name": "layernorm_8192_rows_100b", "op": "layernorm", "m": 8192, "n": 0, "k": 8192, "x": "bf16", "y": "bf16"},
        # a training step's backward over one sequence of a 2B-class model
        {"name": "layernorm_backward_2b", "op": "layernorm_backward", "m": 2048, "n": 0, "k": 2560, "x": "bf16",
         "y": "bf16"},
        # the same in fp32 with sizes that fit no vector and no tile
        {"name": "layernorm_backward_ragged", "op": "layernorm_backward", "m": 1003, "n": 0, "k": 7001, "x": "f32",
         "y": "f32"},
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["quantize", "product", "fused", "fused", "layernorm", "layernorm_backward"])
    x = rng.choice(["f32", "bf16"])
    if op in ("product", "fused"):
        m, n, k = _log(rng, 1, 2048), _log(rng, 16, 28672), _log(rng, 32, 28672)
        if rng.random() < 0.5:  # a decode call
            m = rng.randint(1, 16)
        if rng.random() < 0.5:  # sizes of models are multiples of 64, those of shards need not be
            n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
        n = min(n, 28672 * 8192 // k)
        return {"op": op, "m": m, "n": n, "k": k, "x": x, "y": rng.choice(["f32", "bf16"])}
    m, k = _log(rng, 1, 8192), _log(rng, 32, 28672)
    if rng.random() < 0.5:
        k = max(64, k // 64 * 64)
    m = min(m, 8192 * 8192 * 4 // (k * ESIZE[x] * (3 if op == "layernorm_backward" else 2)))
    return {"op": op, "m": m, "n": 0, "k": k, "x": x, "y": x}


# ---- inputs -------------------------------------------------------------------------------------------------


def _generator(seed, part):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + part)
    return g


def _acts(m, k, dtype, seed):
    """N(0, 1) with 0.5 % of the entries 30 times as large, as the library's prefill workload has them."""
    g = _generator(seed, 1)
    x = torch.randn((m, k), generator=g, device=DEV)
    big = torch.rand((m, k), generator=g, device=DEV) < 0.005
    return torch.where(big, x * 30, x).to(dtype)


def _tiled(codes, exps, m, k):
    """Codes [m][kb * 32] (0 .. 15) and scale bytes [m][kb] in the library's layout."""
    kb = exps.shape[1]
    rb, c, c4 = -(-m // 16), -(-k // 128), -(-k // 512)
    full = torch.zeros((rb * 16, c * 128), dtype=torch.uint8, device=DEV)
    full[:m, :kb * 32] = codes
    two = full[:, 0::2] | (full[:, 1::2] << 4)
    tiles = two.view(rb, 16, c, 4, 16).permute(0, 2, 3, 1, 4).contiguous().view(-1)
    sc = torch.zeros((rb * 16, c4 * 16), dtype=torch.uint8, device=DEV)
    sc[:m, :kb] = exps
    return tiles, sc.view(rb, 16, c4, 4, 4).permute(0, 2, 4, 1, 3).contiguous().view(-1)


def prepare(case, seed):
    m, n, k = case["m"], case["n"], case["k"]
    state = {"case": case}
    if case["op"] in ("layernorm", "layernorm_backward"):
        g = _generator(seed, 2)
        state["x"] = (torch.randn((m, k), generator=g, device=DEV) * 2 + 0.5).to(DT[case["x"]])
        state["weight"] = 1 + 0.1 * torch.randn(k, generator=g, device=DEV)
        state["bias"] = 0.1 * torch.randn(k, generator=g, device=DEV)
        if case["op"] == "layernorm_backward":
            state["dy"] = torch.randn((m, k), generator=g, device=DEV).to(DT[case["x"]])
            mean, rstd = _statistics(state["x"])
            state["mean"], state["rstd"] = mean, rstd
        return state
    x = _acts(m, k, DT[case["x"]], seed) if case["op"] != "quantize" or case["x"] == "bf16" else (
        torch.randn((m, k), generator=_generator(seed, 3), device=DEV) * 0.02)
    if case["op"] == "quantize":
        state["x"] = x
        return state
    w = torch.randn((n, k), generator=_generator(seed, 4), device=DEV) * 0.02
    state["codes"], state["scales"] = _tiled(*_quantize(w)[:2], n, k)
    del w
    if case["op"] == "product":
        state["xcodes"], state["xscales"] = _tiled(*_quantize(x)[:2], m, k)
    else:
        state["x"] = x
    return state


# ---- plain forms --------------------------------------------------------------------------------------------


def _power(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantize(x):
    """Codes [M][kb * 32], scale bytes [M][kb] and values [M][K] in fp32 of x[M][K].  Every step is exact but the
    rounding to the 4-bit grid (nearest, ties to an even mantissa; beyond 6 to 6)."""
    m, k = x.shape
    kb = -(-k // 32)
    b = torch.nn.functional.pad(x.float(), (0, kb * 32 - k)).view(m, kb, 32)
    field = (b.abs().amax(-1).view(torch.int32) >> 23).clamp(min=2)  # exponent field of the largest magnitude
    e = field - 2  # its power of two over the grid's largest, 4: scale 2^(e - 127)
    a = b.abs().double() * _power(127 - e)[:, :, None]  # in 64 bits: 2^(127 - e) need not be an fp32 number
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = (torch.round(a / step) * step).clamp(max=6.0)
    mag = torch.where(v < 2, v * 2, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    codes = mag | (torch.signbit(b).to(torch.uint8) << 3)
    values = (torch.copysign(v, b.double()) * _power(e - 127)[:, :, None]).float().view(m, kb * 32)[:, :k]
    return codes.view(m, kb * 32), e.to(torch.uint8), values


def _rows_of_codes(codes, scales, m, k):
    """Codes [m][k] (0 .. 15) and scale bytes [m][kb] out of the library's layout."""
    rb, c, c4 = -(-m // 16), -(-k // 128), -(-k // 512)
    two = codes.view(rb, c, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(rb * 16, c * 64)[:m]
    q = torch.stack((two & 15, two >> 4), -1).view(m, c * 128)[:, :k]
    e = scales.view(rb, c4, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(rb * 16, c4 * 16)[:m, :-(-k // 32)]
    return q, e


def _values(codes, scales, m, k):
    """The fp32 values [m][k] that the codes stand for."""
    q, e = _rows_of_codes(codes, scales, m, k)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=DEV)
    power = _power(e.int() - 127).float()
    return grid[q.int()] * power.repeat_interleave(32, dim=1)[:, :k]


def _statistics(x):
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    return mean.float(), (1 / torch.sqrt(var + EPS)).float()


def run(state):
    case = state["case"]
    m, n, k, op, out = case["m"], case["n"], case["k"], case["op"], DT[case["y"]]
    if own:
        import bitlinear_fwd_amd as bl

        if op == "quantize":
            return bl.quantize_mxfp4(state["x"], want_values=True)[2]
        if op == "product":
            return bl.forward_mxfp4(state["codes"], state["scales"], state["xcodes"], state["xscales"], m, n, k,
                                    out_dtype=out)
        if op == "fused":
            return bl.forward_mxfp4_fused(state["codes"], state["scales"], state["x"], n, k, out_dtype=out)
        if op == "layernorm":
            return bl.layernorm(state["x"], state["weight"], state["bias"], EPS)
        return bl.layernorm_backward(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"])
    if op == "quantize":
        return _quantize(state["x"])[2].to(out)
    if op == "product":
        xv = _values(state["xcodes"], state["xscales"], m, k)
        return (xv @ _values(state["codes"], state["scales"], n, k).t()).to(out)
    if op == "fused":
        xv = _quantize(state["x"])[2]
        return (xv @ _values(state["codes"], state["scales"], n, k).t()).to(out)
    x = state["x"].float()
    if op == "layernorm":
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = 1 / torch.sqrt((xc * xc).mean(1) + EPS)
        return (xc * rstd[:, None] * state["weight"] + state["bias"]).to(out), mean, rstd
    dy = state["dy"].float()
    xhat = (x - state["mean"][:, None]) * state["rstd"][:, None]
    g = dy * state["weight"]
    dx = state["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx.to(out), (dy * xhat).sum(0), dy.sum(0)


# ---- the cost that no form can do without, and the definition in 64 bits -----------------------------------


def work(case):
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    ex, ey = ESIZE[case["x"]], ESIZE[case["y"]]
    packed = lambda rows: rows * (-(-k // 2) + -(-k // 32))  # noqa: E731
    if op == "quantize":  # x in; codes, scales and values out
        return {"bytes": m * k * (ex + ey) + packed(m), "flops": 4 * m * k}
    if op in ("product", "fused"):
        x = packed(m) if op == "product" else m * k * ex
        return {"bytes": packed(n) + x + m * n * ey, "flops": 2 * m * n * k}
    if op == "layernorm":
        return {"bytes": m * k * (ex + ey) + 8 * k + 8 * m, "flops": 8 * m * k}
    return {"bytes": 3 * m * k * ex + 12 * k + 8 * m, "flops": 14 * m * k}


def _two_to(e):
    """2^e in 64 bits, from a table of the powers that blocks of fp32 numbers can have."""
    return torch.tensor([2.0 ** i for i in range(-149, 129)], dtype=torch.float64, device=DEV)[e.long() + 149]


def _exact_quantized(x):
    """The values of x[M][K] in 64 bits by comparison with the borders between neighbouring grid magnitudes."""
    m, k = x.shape
    kb = -(-k // 32)
    b = torch.zeros((m, kb * 32), dtype=torch.float64, device=DEV)
    b[:, :k] = x.double()
    b = b.view(m, kb, 32)
    exponent = torch.frexp(b.abs().amax(-1))[1] - 1  # floor(log2) of the largest magnitude
    exponent = torch.where(b.abs().amax(-1) == 0, -126, exponent).clamp(min=-125)
    scale = _two_to(exponent - 2).unsqueeze(-1)
    a = b.abs() / scale
    # a tie goes to the even mantissa: 0, 1, 2 and 4 keep theirs, 0.5, 1.5, 3 and 6 give theirs away
    v = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75)
    v = v + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0)
    return (torch.sign(b) * v * scale).view(m, kb * 32)[:, :k]


def _exact_values(codes, scales, m, k):
    q, e = _rows_of_codes(codes, scales, m, k)
    mag = (q & 7).double()
    low, high = mag / 2, torch.exp2((mag / 2).floor() - 1) * (1 + (mag % 2) / 2)
    v = torch.where(mag < 2, low, high) * (1 - 2 * (q >> 3).double())
    return v * _two_to(e.int() - 127).repeat_interleave(32, dim=1)[:, :k]


def exact(case, seed):
    state = prepare(case, seed)
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    if op == "quantize":
        return _exact_quantized(state["x"])
    if op in ("product", "fused"):
        xv = _exact_quantized(state["x"]) if op == "fused" else _exact_values(state["xcodes"], state["xscales"], m, k)
        return xv @ _exact_values(state["codes"], state["scales"], n, k).t().contiguous()
    x, w = state["x"].double(), state["weight"].double()
    if op == "layernorm":
        mean = x.sum(1) / k
        rstd = (((x - mean[:, None]) ** 2).sum(1) / k + EPS) ** -0.5
        return (x - mean[:, None]) * rstd[:, None] * w + state["bias"].double(), mean, rstd
    dy, mean, rstd = state["dy"].double(), state["mean"].double()[:, None], state["rstd"].double()[:, None]
    xhat = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.sum(1, keepdim=True) / k, (g * xhat).sum(1, keepdim=True) / k
    return rstd * (g - c1 - c2 * xhat), (dy * xhat).sum(0), dy.sum(0)
