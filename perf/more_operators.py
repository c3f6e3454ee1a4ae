"""Ternary products with an epilogue, ternary products grouped by expert, and the router in front of them, as
measurements: their cases, a plain form in elementary torch operations, and the definition in 64 bits.

Operators (``case["op"]``), with acc the exact integer product of a token's int8 codes and a row of ternary codes,
gamma the matrix' scale and a the token's:

* ``epilogue``: y[m][n] = act(acc gamma a[m] / 127 + bias[n]) + residual[m][n].
* ``experts``: the same with a matrix per expert.  Slot s of expert e (offsets[e] <= s < offsets[e + 1]) takes token
  rows[s] through matrix e; y has a row per slot.
* ``combine``: the products of slots as above (slot s takes row s of x), added up for each token with the router's
  weights: y[m] = residual[m] + sum_j weights[m][j] act(...)[slots[m][j]].
* ``route``: each token's ``top`` largest logits (ties: the lowest index), their weights (softmax over the chosen
  ones, or over all experts), and the slots ordered by expert, then token: offsets, rows, slots.  A logit of -inf
  is never chosen; choices that are missing for that have the expert -1, the weight 0 and the slot -1.

x is fp32 or bf16 (quantised within the call) or int8 codes with their scales (``"i8"``).  The packed layout is the
library's documented one: 1024-byte tiles of 16 rows x 256 columns, row r's columns 64 g .. 64 g + 63 in the 16 bytes
at 16 (16 g + r), column 16 i + 4 f + b of them in bits 2 f, 2 f + 1 of byte b of word i; 0 -> 00, 1 -> 01, -1 -> 10.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2, "i8": 1, "none": 0}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


def _product(name, op, m, n, k, x, y, act="none", bias=False, res="none", e=1, top=1):
    case = {"op": op, "m": m, "n": n, "k": k, "e": e, "top": top, "x": x, "y": y, "act": act, "bias": bias, "res": res}
    return {"name": name, **case} if name else case


def _route(name, m, e, top, x, renorm, masked):
    case = {"op": "route", "m": m, "e": e, "top": top, "x": x, "renorm": renorm, "masked": masked}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one token through a 2B-class up projection with the feed-forward's squared ReLU: the smallest product
        _product("epilogue_1_token_2b", "epilogue", 1, 6912, 2560, "bf16", "bf16", "relu2"),
        # 16 sequences' tokens through a 2B-class down projection, added to the residual stream
        _product("epilogue_16_tokens_2b_down", "epilogue", 16, 2560, 6912, "f32", "bf16", bias=True, res="bf16"),
        # a few dozen tokens already quantised (for several projections at once), odd sizes on every axis
        _product("epilogue_37_tokens_ragged", "epilogue", 37, 6909, 2570, "i8", "f32", "gelu", True, "f32"),
        # prefill of 2048 tokens through a 2B-class up projection, the activation's output in bf16
        _product("epilogue_prefill_2b", "epilogue", 2048, 6912, 2560, "bf16", "bf16", "silu", True),
        # prefill of 2048 tokens through a 100B-class down projection, added to the residual stream
        _product("epilogue_prefill_100b_down", "epilogue", 2048, 8192, 28672, "bf16", "bf16", res="bf16"),
        # one token, two of 16 experts of the 2B class
        _product("experts_1_token", "experts", 1, 6912, 2560, "bf16", "bf16", "relu2", e=16, top=2),
        # 16 sequences' tokens over 64 narrow experts (a quarter of a 2B-class feed-forward each): one or two a piece
        _product("experts_16_tokens_64", "experts", 16, 1728, 2560, "bf16", "f32", "silu", True, e=64, top=4),
        # prefill of 2048 tokens over 8 experts of the 2B class, two each
        _product("experts_prefill_2b", "experts", 2048, 6912, 2560, "bf16", "bf16", "relu2", e=8, top=2),
        # a short prompt back to the residual stream through experts with odd sizes
        _product("combine_203_tokens_ragged", "combine", 203, 2571, 1733, "f32", "f32", bias=True, res="f32", e=12, top=3),
        # the down projections of the prefill above, added up for each token
        _product("combine_prefill_2b", "combine", 2048, 2560, 6912, "bf16", "bf16", res="bf16", e=8, top=2),
        # the router of one decode step
        _route("route_16_tokens", 16, 64, 4, "f32", True, 0.0),
        # the router of a long prefill with many experts, a tenth of the batch padding
        _route("route_65536_tokens", 65536, 128, 8, "bf16", False, 0.1),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["epilogue", "epilogue", "experts", "experts", "combine", "route"])
    if op == "route":
        e = _log(rng, 2, 256)
        return _route(None, _log(rng, 1, 65536 * 128 // e), e, rng.randint(1, min(e, 8)), rng.choice(["f32", "bf16"]),
                      rng.random() < 0.5, rng.choice([0.0, 0.1]))
    m, n, k = _log(rng, 1, 2048), _log(rng, 16, 28672), _log(rng, 32, 28672)
    if rng.random() < 0.5:  # a decode call
        m = rng.randint(1, 16)
    if rng.random() < 0.5:  # sizes of models are multiples of 64, those of shards need not be
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    e, top, room = 1, 1, 28672 * 8192
    if op != "epilogue":
        e = _log(rng, 2, 64)
        top = rng.randint(1, min(e, 4))
        k = min(k, 8192)
        room = 64 * 1728 * 2560 // e
    n = max(1, min(n, room // k))
    x = rng.choice(["f32", "bf16", "i8"])
    return _product(None, op, m, n, k, x, rng.choice(["f32", "bf16"]), rng.choice(ACTS), rng.random() < 0.5,
                    rng.choice(["none", "f32", "bf16"]), e, top)


# ---- inputs -------------------------------------------------------------------------------------------------


def _generator(seed, part):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + part)
    return g


def _acts(m, k, seed):
    """N(0, 1) with 0.5 % of the entries 30 times as large, as the library's prefill workload has them."""
    g = _generator(seed, 1)
    x = torch.randn((m, k), generator=g, device=DEV)
    big = torch.rand((m, k), generator=g, device=DEV) < 0.005
    return torch.where(big, x * 30, x)


def _random_packed(e, n, k, g):
    """E packed matrices of random ternary codes (31 % zeros, as normally distributed weights give), and padding."""
    nb, c = -(-n // 16), -(-k // 256)
    out = torch.empty((e, nb * c * 1024), dtype=torch.uint8, device=DEV)
    for i in range(e):
        u = torch.empty((nb, c, 4, 16, 4, 4, 4), dtype=torch.uint8, device=DEV)  # [.., g, row, word, byte, field]
        u.random_(0, 256, generator=g)
        code = (u >= 79).to(torch.uint8) + (u >= 167).to(torch.uint8)  # 0, 1 (+1), 2 (-1)
        if n % 16 or k % 256:
            row = torch.arange(nb, device=DEV)[:, None] * 16 + torch.arange(16, device=DEV)
            a = lambda size, shape: torch.arange(size, device=DEV).view(shape)  # noqa: E731
            col = (a(c, (-1, 1, 1, 1, 1)) * 256 + a(4, (-1, 1, 1, 1)) * 64 + a(4, (-1, 1, 1)) * 16 + a(4, (-1, 1))
                   + a(4, (-1,)) * 4)  # [c, g, word, byte, field]
            pad = (row >= n).view(nb, 1, 1, 16, 1, 1, 1) | (col >= k).view(1, c, 4, 1, 4, 4, 4)
            code = torch.where(pad, 3, code).to(torch.uint8)
        shift = torch.tensor([1, 4, 16, 64], dtype=torch.uint8, device=DEV)
        out[i] = (code * shift).sum(-1, dtype=torch.uint8).view(-1)
    return out


def _choices(m, e, top, g):
    """Random routing with busier and idler experts: chosen experts and weights [m][top]."""
    logits = torch.randn((m, e), generator=g, device=DEV) + 0.5 * torch.randn(e, generator=g, device=DEV)
    w, idx = torch.sort(torch.softmax(logits, -1), dim=1, descending=True, stable=True)
    w = w[:, :top]
    return idx[:, :top].contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


def _grouping(idx, e):
    """offsets [e + 1], rows [m top], slots [m][top] of the choices idx (-1: none), ordered by expert, then token."""
    m, top = idx.shape
    key, order = torch.sort(torch.where(idx < 0, e, idx).view(-1), stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(m * top, device=DEV)
    offsets = torch.searchsorted(key, torch.arange(e + 1, device=DEV))
    rows = torch.where(key < e, order // top, -1)
    slots = torch.where(idx < 0, -1, slots.view(m, top))
    return offsets.int(), rows.int(), slots.int()


def prepare(case, seed):
    m, op = case["m"], case["op"]
    state = {"case": case}
    if op == "route":
        g = _generator(seed, 2)
        logits = torch.randn((m, case["e"]), generator=g, device=DEV) * 2 + torch.randn(case["e"], generator=g, device=DEV)
        if case["masked"]:  # padded tokens: no expert at all
            gone = torch.rand((m, 1), generator=g, device=DEV) < case["masked"]
            logits = torch.where(gone, -math.inf, logits)
        state["logits"] = logits.to(DT[case["x"]])
        return state
    n, k, e, top = case["n"], case["k"], case["e"], case["top"]
    g = _generator(seed, 3)
    rows = m
    if op != "epilogue":
        idx, weights = _choices(m, e, top, g)
        state["offsets"], state["rows"], state["slots"] = _grouping(idx, e)
        state["weights"] = weights
        state["bounds"] = state["offsets"].tolist()  # for the plain form
        rows = m * top if op == "combine" else m
    x = _acts(rows, k, seed)
    if case["x"] == "i8":
        state["x"], state["absmax"] = _codes(x)
    else:
        state["x"], state["absmax"] = x.to(DT[case["x"]]), None
    packed = _random_packed(e, n, k, g)
    gamma = 0.016 * (1 + 0.1 * torch.rand(e, generator=g, device=DEV))
    state["packed"], state["gamma"] = (packed[0], gamma) if op == "epilogue" else (packed, gamma)
    state["bias"] = state["residual"] = None
    if case["bias"]:
        bias = 0.2 * torch.randn((e, n), generator=g, device=DEV)
        state["bias"] = bias[0] if op == "epilogue" else bias
    if case["res"] != "none":
        out_rows = m * top if op == "experts" else m
        state["residual"] = torch.randn((out_rows, n), generator=g, device=DEV).to(DT[case["res"]])
    return state


# ---- plain forms --------------------------------------------------------------------------------------------


def _codes(x):
    """int8 codes [M][K_pad] and scales [M] of x: codes round(x * fl32(127 / a)), ties to even, a = max |x|."""
    x = x.float()
    a = x.abs().amax(1)
    s = torch.where(a > 0, torch.full_like(a, 127.0) / a, 0.0)  # (127.0 / a rounds twice: a reciprocal, a product)
    q = torch.round(x * s[:, None]).clamp(-127, 127).to(torch.int8)
    return torch.nn.functional.pad(q, (0, -x.shape[1] % 256)), a


def _weights(packed, n, k):
    """The ternary codes [n][k] of one packed matrix as fp32."""
    nb, c = -(-n // 16), -(-k // 256)
    p = packed.view(nb, c, 4, 16, 4, 4).permute(0, 3, 1, 2, 4, 5)  # [nb, row, c, g, word, byte]
    f = torch.stack([(p >> (2 * i)) & 3 for i in range(4)], -2)  # [.., word, field, byte]
    q = f.reshape(nb * 16, c * 256)[:n, :k]
    return (q == 1).float() - (q == 2).float()


def _act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "relu2":
        return torch.clamp(v, min=0) ** 2
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_product(xq, a, packed, gamma, bias, n, k, act):
    """act(acc gamma a / 127 + bias) in fp32 (the sums of codes are whole numbers below 2^24: exact)."""
    v = (xq[:, :k].float() @ _weights(packed, n, k).t()) * (gamma * a / 127.0)[:, None]
    return _act(v if bias is None else v + bias, act)


def _plain_route(logits, top, renorm):
    x = logits.float()
    order = torch.sort(x, dim=1, descending=True, stable=True)
    values, idx = order[0][:, :top], order[1][:, :top]
    gone = values == -math.inf
    peak = torch.where(gone[:, :1], 0.0, values[:, :1])
    w = torch.exp(values - peak)
    total = w.sum(1, keepdim=True) if renorm else torch.exp(x - peak).sum(1, keepdim=True)
    idx = torch.where(gone, -1, idx)
    return (idx.int(), torch.where(gone, 0.0, w / total)) + _grouping(idx, x.shape[1])


def run(state):
    case = state["case"]
    op = case["op"]
    if op == "route":
        if own:
            import bitlinear_fwd_amd as bl

            r = bl.route_experts(state["logits"], case["top"], renormalize=case["renorm"])
            return r.experts, r.weights, r.offsets, r.rows, r.slots
        return _plain_route(state["logits"], case["top"], case["renorm"])
    n, k, out, act = case["n"], case["k"], DT[case["y"]], case["act"]
    packed, gamma, bias, residual = state["packed"], state["gamma"], state["bias"], state["residual"]
    x, absmax = state["x"], state["absmax"]
    if own:
        import bitlinear_fwd_amd as bl

        if op == "epilogue":
            return bl.forward_epilogue(packed, gamma, x, n, k, absmax=absmax, bias=bias, act=act, residual=residual,
                                       out_dtype=out)
        if op == "experts":
            return bl.forward_experts(packed, gamma, state["offsets"], x, n, k, rows=state["rows"], absmax=absmax,
                                      bias=bias, act=act, residual=residual, out_dtype=out)
        return bl.forward_experts_combine(packed, gamma, state["offsets"], x, n, k, state["slots"], state["weights"],
                                          absmax=absmax, bias=bias, act=act, residual=residual, out_dtype=out)
    xq, a = (x, absmax) if absmax is not None else _codes(x)
    if op == "epilogue":
        y = _plain_product(xq, a, packed, gamma[0], bias, n, k, act)
        return (y if residual is None else y + residual.float()).to(out)
    parts, bounds = [], state["bounds"]
    for e in range(case["e"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            src = slice(lo, hi) if op == "combine" else state["rows"][lo:hi].long()
            parts.append(_plain_product(xq[src], a[src], packed[e], gamma[e], None if bias is None else bias[e], n, k, act))
    y = torch.cat(parts)
    if op == "combine":
        y = (y[state["slots"].long()] * state["weights"][:, :, None]).sum(1)
    return (y if residual is None else y + residual.float()).to(out)


# ---- the cost that no form can do without, and the definition in 64 bits -----------------------------------


def work(case):
    m, e, top = case["m"], case["e"], case["top"]
    if case["op"] == "route":
        return {"bytes": m * e * ESIZE[case["x"]] + m * top * 16 + 4 * (e + 1), "flops": 4 * m * e}
    n, k, op = case["n"], case["k"], case["op"]
    used = e * (1 - (1 - top / e) ** m)  # experts with a token, on average
    slots = m * top
    rows_in, rows_out = slots if op == "combine" else m, slots if op == "experts" else m
    scales = 4 * rows_in if case["x"] == "i8" else 0
    bias = 4 * n * used if case["bias"] else 0
    tables = 0 if op == "epilogue" else 4 * slots + 4 * (e + 1) + (4 * slots if op == "combine" else 0)
    return {"bytes": used * n * k / 4 + rows_in * k * ESIZE[case["x"]] + scales + bias + tables
            + rows_out * n * (ESIZE[case["y"]] + ESIZE[case["res"]]), "flops": 2 * slots * n * k}


def _exact_codes(x):
    """The codes in 64 bits.  The scale and the product that is rounded to a code are fp32 numbers by definition."""
    x = x.double()
    a = x.abs().max(1)[0]
    s = (127.0 / a.clamp(min=1e-300)).float().double() * (a > 0)
    t = (x * s[:, None]).float().double()
    low = torch.floor(t)
    d = t - low
    up = (d > 0.5) | ((d == 0.5) & (torch.remainder(low, 2) == 1))
    return torch.minimum(torch.maximum(low + up, torch.tensor(-127.0, device=DEV)), torch.tensor(127.0, device=DEV)), a


def _exact_weights(packed, n, k):
    """Ternary codes [n][k] in 64 bits, by each column's place."""
    col = torch.arange(k, device=DEV)
    kk = col % 256
    byte = (col // 256) * 1024 + 256 * (kk // 64) + 4 * ((kk % 64) // 16) + kk % 4  # of row 0
    shift = (2 * ((kk % 16) // 4)).to(torch.uint8)
    tiles = packed.view(-(-n // 16), -1)
    rows = [(tiles[:, byte + 16 * r] >> shift) & 3 for r in range(16)]
    q = torch.stack(rows, 1).view(-1, k)[:n]
    return torch.tensor([0.0, 1.0, -1.0, 0.0], dtype=torch.float64, device=DEV)[q.int()]


def _exact_act(v, act):
    if act in ("relu", "relu2"):
        v = torch.where(v > 0, v, torch.zeros_like(v))
        return v if act == "relu" else v * v
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        x = state["logits"].double()
        m, e = x.shape
        top = case["top"]
        left, idx, val = x.clone(), [], []
        for _ in range(top):  # the largest that is left, at the lowest index of those equal to it
            v = left.max(1, keepdim=True)[0]
            i = (left == v).int().argmax(1, keepdim=True)
            left.scatter_(1, i, -math.inf)
            idx.append(torch.where(v > -math.inf, i, -1))
            val.append(v)
        idx, val = torch.cat(idx, 1), torch.cat(val, 1)
        total = torch.logsumexp(val if case["renorm"] else x, 1, keepdim=True)
        w = torch.where(idx < 0, 0.0, torch.exp(val - total))
        one = torch.zeros((m, e + 1), dtype=torch.int32, device=DEV)
        one.scatter_(1, torch.where(idx < 0, e, idx), 1)
        one = one[:, :e]
        counts = one.sum(0)
        offsets = torch.cat((counts.new_zeros(1), torch.cumsum(counts, 0)))
        place = offsets[:e] + torch.cumsum(one, 0) - one  # slot of token m at expert e
        slots = torch.where(idx < 0, -1, place.gather(1, idx.clamp(min=0)))
        rows = torch.full((m * top + 1,), -1, dtype=torch.int64, device=DEV)
        rows[torch.where(slots < 0, m * top, slots).view(-1)] = torch.arange(m, device=DEV).repeat_interleave(top)
        return idx.int(), w, offsets.int(), rows[:m * top].int(), slots.int()
    n, k, op = case["n"], case["k"], case["op"]
    if state["absmax"] is None:
        q, a = _exact_codes(state["x"])
    else:
        q, a = state["x"][:, :k].double(), state["absmax"].double()
    gamma, bias, residual = state["gamma"].double(), state["bias"], state["residual"]
    if op == "epilogue":
        v = q @ _exact_weights(state["packed"], n, k).t().contiguous() * (a * gamma / 127)[:, None]
        y = _exact_act(v if bias is None else v + bias.double(), case["act"])
        return y if residual is None else y + residual.double()
    slots = case["m"] * case["top"]
    y = torch.zeros((slots, n), dtype=torch.float64, device=DEV)
    rows = torch.arange(slots, device=DEV) if op == "combine" else state["rows"].long()
    slot = torch.arange(slots, device=DEV)
    for e in range(case["e"]):
        at = slot[(slot >= state["offsets"][e]) & (slot < state["offsets"][e + 1])]
        if at.numel():
            v = q[rows[at]] @ _exact_weights(state["packed"][e], n, k).t().contiguous()
            v = v * (a[rows[at]] * gamma[e] / 127)[:, None]
            y[at] = _exact_act(v if bias is None else v + bias[e].double(), case["act"])
    if op == "combine":
        w = state["weights"].double()
        y = sum(w[:, j:j + 1] * y[state["slots"][:, j].long()] for j in range(case["top"]))
    return y if residual is None else y + residual.double()
