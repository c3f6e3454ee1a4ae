"""Products with an epilogue, products grouped by expert and the router in 64 bits on the CPU, written from their
definitions, with the error that fp32 arithmetic may have.

u = 2^-24 is half a step of fp32.  v = fl(acc scale + bias) with scale = fl(fl(gamma a) / 127): acc (below 2^24) is
exact, the scale is off by 2 u relative, the fused multiply-add by u of its result.  The activations pass that on
with their largest slope and add their own roundings, counted at each below.  The last rounding is half a step of
the output's type."""
import math

import torch

U = 2.0 ** -24
STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TINY = 1e-34  # results below are not told apart from 0


def pack(q):
    """Ternary codes q [N][K] in the library's layout (uint8)."""
    n, k = q.shape
    nb, c = -(-n // 16), -(-k // 256)
    code = torch.full((nb * 16, c * 256), 3, dtype=torch.uint8)
    code[:n, :k] = torch.where(q < 0, 2, q).to(torch.uint8)
    f = code.view(nb, 16, c, 4, 4, 4, 4)  # block, row, chunk, g, word, field, byte
    f = f.permute(0, 2, 3, 1, 4, 6, 5).to(torch.int32)  # block, chunk, g, row, word, byte, field
    return (f * torch.tensor([1, 4, 16, 64], dtype=torch.int32)).sum(-1).to(torch.uint8).reshape(-1)


def random_codes(n, k, gen):
    return torch.randint(-1, 2, (n, k), generator=gen, dtype=torch.int8)


def quantize(x):
    """Codes [M][K] (int64) and scales of x: the decisions are fp32 numbers by definition."""
    x = x.float()
    a = x.abs().amax(1)
    # (127.0 / a would be torch's reciprocal of a times 127, which rounds twice)
    s = torch.where(a > 0, torch.full_like(a, 127.0) / a, torch.zeros_like(a))
    return torch.round(x * s[:, None]).clamp(-127, 127).long(), a.double()


def act(v, dv, name):
    """(act(v), its error) of v in 64 bits known to dv."""
    if name == "relu":
        return v.clamp(min=0), dv
    if name == "relu2":
        r = v.clamp(min=0)
        return r * r, 2 * r * dv + dv * dv + U * (r + dv) ** 2
    if name == "silu":  # slope up to 1.1; e^-v to 4 u, the sum, the reciprocal (2 u), the product
        s = v * torch.sigmoid(v)
        return s, 1.1 * dv + 10 * U * s.abs() + TINY
    if name == "gelu":  # slope up to 1.13; the argument to 2 u, erf to 2 u of 1, the sum, two products
        return 0.5 * v * torch.erfc(-v / math.sqrt(2)), 1.13 * dv + 8 * U * v.abs()
    if name == "gelu_tanh":  # as silu, of an argument t with five roundings
        t = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        g = v * torch.sigmoid(t)
        return g, 1.13 * dv + (10 + 6 * t.abs()) * U * g.abs() + TINY
    return v, dv


def product(q_x, a, q_w, gamma, bias, name):
    """(act(acc gamma a / 127 + bias), its error) [M][N]."""
    acc = (q_x.double() @ q_w.double().t())
    assert acc.abs().max() < 2 ** 24
    raw = acc * (a * float(gamma) / 127)[:, None]
    v = raw if bias is None else raw + bias.double()
    return act(v, 2.01 * U * raw.abs() + U * v.abs(), name)


def finish(v, dv, residual, dtype):
    """(v + residual, its error) once rounded to dtype."""
    if residual is not None:
        v = v + residual.double()
        dv = dv + U * (v.abs() + dv)
    return v, dv + STEP[dtype] * (v.abs() + dv) * (dtype != torch.float32)


def check(y, ref, err, what=""):
    y = y.double().cpu()
    assert y.shape == ref.shape, (what, y.shape, ref.shape)
    bad = ~((y - ref).abs() <= err)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outputs are off, first at {i}: {y[i]} for {ref[i]}, "
                             f"allowed {err[i]}")


def experts(q_x, a, q_ws, gammas, bias, name, offsets, rows):
    """Slots' products [T][N], their errors, and which slots there are."""
    t, n = (len(rows) if rows is not None else q_x.shape[0]), q_ws[0].shape[0]
    y, dy = torch.zeros(t, n, dtype=torch.float64), torch.zeros(t, n, dtype=torch.float64)
    there = torch.zeros(t, dtype=torch.bool)
    for e, q_w in enumerate(q_ws):
        s = torch.arange(int(offsets[e]), int(offsets[e + 1]))
        r = rows[s].long() if rows is not None else s
        ok = (r >= 0) & (r < q_x.shape[0])
        s, r = s[ok], r[ok]
        if len(s):
            y[s], dy[s] = product(q_x[r], a[r], q_w, gammas[e], None if bias is None else bias[e], name)
            there[s] = True
    return y, dy, there


def combine(y, dy, there, slots, weights):
    """Weighted sums over the slots of a token, and their errors (each step rounds once)."""
    m, k = slots.shape
    out, err, size = (torch.zeros(m, y.shape[1], dtype=torch.float64) for _ in range(3))
    for j in range(k):
        s = slots[:, j].long()
        ok = (s >= 0) & (s < len(there))
        ok[ok.clone()] = there[s[ok]]
        w = weights[ok, j].double()[:, None]
        out[ok] += w * y[s[ok]]
        err[ok] += w.abs() * dy[s[ok]]
        size[ok] += w.abs() * y[s[ok]].abs()
    return out, err + k * U * (size + err)


def route(logits, k, renormalize):
    """experts, weights (64 bits), offsets, rows, slots by a loop over the tokens."""
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), torch.tensor(-math.inf, dtype=torch.float64), x).clamp(max=3.4028234663852886e38)
    m, e = x.shape
    ids, weights = torch.full((m, k), -1, dtype=torch.int32), torch.zeros(m, k, dtype=torch.float64)
    for i in range(m):
        row = x[i].tolist()
        order = sorted((j for j in range(e) if row[j] > -math.inf), key=lambda j: (-row[j], j))
        chosen = order[:k]
        if not chosen:
            continue
        peak = row[chosen[0]]
        total = math.fsum(math.exp(row[j] - peak) for j in (chosen if renormalize else order))
        for j, c in enumerate(chosen):
            ids[i, j], weights[i, j] = c, math.exp(row[c] - peak) / total
    slots, rows, offsets = torch.full((m, k), -1, dtype=torch.int32), [], [0]
    by_expert = [[] for _ in range(e)]
    for i in range(m):
        for j in range(k):
            if ids[i, j] >= 0:
                by_expert[int(ids[i, j])].append((i, j))
    for members in by_expert:
        for i, j in members:
            slots[i, j] = len(rows)
            rows.append(i)
        offsets.append(len(rows))
    rows += [-1] * (m * k - len(rows))
    return ids, weights, torch.tensor(offsets, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32), slots
