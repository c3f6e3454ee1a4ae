"""Products grouped by expert, their sums over a token's slots and the router against 64 bits (experts_reference)."""
import math

import pytest
import torch

import bitlinear_fwd_amd as bl
import experts_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Layer:
    """E experts of random codes, slots as `counts` says, token rows drawn at random (twice in one expert, too)."""

    def __init__(self, counts, n, k, r, x="bf16", seed=0, gather=True, behind=0):
        g = torch.Generator().manual_seed(seed * 1013 + n + k + r + sum(counts))
        self.n, self.k, e, t = n, k, len(counts), sum(counts)
        self.q_w = [ref.random_codes(n, k, g) for _ in range(e)]
        self.gamma = 0.01 + 0.02 * torch.rand(e, generator=g)
        self.bias = 0.3 * torch.randn(e, n, generator=g)
        self.offsets = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
        self.t = t + behind
        self.r = r if gather else self.t
        self.rows = torch.randint(0, r, (self.t,), generator=g, dtype=torch.int32) if gather else None
        self.x = torch.randn(self.r, k, generator=g).to(DT[x])
        self.packed = torch.stack([ref.pack(q) for q in self.q_w]).to(DEV)
        self.g = g

    def tables(self):
        return self.packed, self.gamma.to(DEV), self.offsets.to(DEV)

    def reference(self, act="none", bias=True):
        q, a = ref.quantize(self.x)
        return ref.experts(q, a, self.q_w, self.gamma, self.bias if bias else None, act, self.offsets, self.rows)

    def forward(self, act="none", bias=True, codes=False, **kw):
        x, absmax = (bl.quantize_acts(self.x.to(DEV)) if codes else (self.x.to(DEV), None))
        rows = self.rows.to(DEV) if self.rows is not None else None
        return bl.forward_experts(*self.tables(), x, self.n, self.k, rows=rows, absmax=absmax,
                                  bias=self.bias.to(DEV) if bias else None, act=act, **kw)


COUNTS = {
    "one": [1],
    "one of many": [0] * 5 + [1] + [0] * 3,
    "all in the last": [0, 0, 0, 100],
    "all in the first": [70, 0, 0],
    "a few each": [2, 0, 1, 3, 0, 5, 1, 1],
    "around 16": [15, 16, 17, 0, 31, 32, 33],
    "ragged": [1, 130, 0, 64, 7, 257, 0, 128],
    "many experts": [i % 3 for i in range(200)],
    "65 experts, the last": [0] * 64 + [20],
}


@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
@pytest.mark.parametrize("size", [(1, 1), (40, 300), (130, 513), (16, 2570)], ids=str)
@pytest.mark.parametrize("gather", [True, False], ids=["gather", "in order"])
def test_counts_and_sizes(counts, size, gather):
    layer = Layer(counts, *size, r=23, gather=gather)
    y, dy, there = layer.reference("relu2")
    assert there.all()
    ref.check(layer.forward("relu2"), y, dy)
    ref.check(layer.forward("relu2", codes=True), y, dy)


@pytest.mark.parametrize("counts", ["a few each", "ragged"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_types(counts, x, res, out):
    layer = Layer(COUNTS[counts], 70, 600, r=40, x=x)
    r = torch.randn(layer.t, 70, generator=layer.g).to(DT[res]) if res else None
    y = layer.forward("gelu_tanh", residual=None if r is None else r.to(DEV), out_dtype=DT[out])
    v, dv, _ = layer.reference("gelu_tanh")
    ref.check(y, *ref.finish(v, dv, r, DT[out]))


@pytest.mark.parametrize("counts", ["a few each", "ragged", "one"])
@pytest.mark.parametrize("codes", [False, True], ids=["x", "codes"])
def test_slots_that_are_left_out(counts, codes):
    """Rows of Y behind the last slot, and of slots without a token row, stay as they were."""
    layer = Layer(COUNTS[counts], 40, 300, r=30, behind=9)
    bad = torch.rand(layer.t, generator=layer.g) < 0.3
    layer.rows[bad] = torch.tensor([-1, 30, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.arange(int(bad.sum())) % 4]
    y0 = torch.randn(layer.t, 40, generator=layer.g)
    y = layer.forward("silu", codes=codes, y=y0.to(DEV))
    v, dv, there = layer.reference("silu")
    assert not there[-9:].any()
    ref.check(y[there.to(DEV)], v[there], dv[there])
    assert torch.equal(y.cpu()[~there], y0[~there])


def test_no_slots_at_all():
    layer = Layer([0, 0, 0], 40, 300, r=5, behind=6)
    y = layer.forward(y=torch.full((6, 40), 7.0, device=DEV))
    assert (y == 7).all()


@pytest.mark.parametrize("t", [3, 40, 200])
def test_offsets_against_the_rule_touch_nothing_else(t):
    """Offsets that fall, or lie outside 0 .. T: rows of Y are unspecified, what lies around Y is not touched."""
    layer = Layer([t], 40, 300, r=9)
    guard = torch.full((t + 64, 40), 5.0, device=DEV)
    for offsets in ([-5, t + 1000], [t, 0], [2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1]):
        layer.offsets = torch.tensor(offsets, dtype=torch.int32)
        layer.forward(y=guard[32:32 + t])
    assert (guard[:32] == 5).all() and (guard[32 + t:] == 5).all()
    many = Layer([1] * 6, 40, 300, r=9)
    many.offsets = torch.tensor([0, 6, 0, 6, 0, 6, 6], dtype=torch.int32)  # more slots than T in all
    guard = torch.full((70, 40), 5.0, device=DEV)
    many.forward(y=guard[32:38])
    assert (guard[:32] == 5).all() and (guard[38:] == 5).all()


@pytest.mark.parametrize("m,e,k,n,kk", [(1, 4, 2, 40, 300), (16, 8, 3, 130, 513), (60, 5, 5, 33, 700), (300, 8, 2, 257, 256),
                                        (33, 300, 16, 20, 40)])
@pytest.mark.parametrize("res,out", [(None, "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_combine(m, e, k, n, kk, res, out):
    g = torch.Generator().manual_seed(m + e)
    logits = torch.randn(m, e, generator=g)
    logits[torch.rand(m, e, generator=g) < 0.2] = -math.inf
    if m > 1:
        logits[1] = -math.inf  # a token without any expert
    routed = bl.route_experts(logits.to(DEV), k)
    counts = routed.offsets.cpu().diff().tolist()
    layer = Layer(counts, n, kk, r=m * k, gather=False, behind=m * k - sum(counts))
    r = torch.randn(m, n, generator=g).to(DT[res]) if res else None
    y = bl.forward_experts_combine(*layer.tables(), layer.x.to(DEV), n, kk, routed.slots, routed.weights, bias=layer.bias.to(DEV),
                                   act="relu", residual=None if r is None else r.to(DEV), out_dtype=DT[out])
    v, dv, there = layer.reference("relu")
    v, dv = ref.combine(v, dv, there, routed.slots.cpu(), routed.weights.cpu())
    ref.check(y, *ref.finish(v, dv, r, DT[out]))
    # with rows: one product per token and expert, some slots without a row; in place of the residual
    rows = torch.randint(-1, m, (m * k,), generator=g, dtype=torch.int32)
    layer.rows, layer.x = rows, layer.x[:m]
    y = r.to(DEV).clone() if res else torch.zeros(m, n, device=DEV)
    res_in = y if res else None
    bl.forward_experts_combine(*layer.tables(), layer.x.to(DEV), n, kk, routed.slots, routed.weights, rows=rows.to(DEV),
                               residual=res_in, y=y)
    v, dv, there = layer.reference("none", bias=False)
    v, dv = ref.combine(v, dv, there, routed.slots.cpu(), routed.weights.cpu())
    ref.check(y, *ref.finish(v, dv, r, y.dtype))


def test_combine_entries_out_of_range_and_twice():
    layer = Layer([2, 3], 20, 64, r=5, gather=False, behind=2)
    slots = torch.tensor([[0, 0, 5], [4, -1, 7], [2 ** 31 - 1, -2 ** 31, 6], [1, 2, 3]], dtype=torch.int32)
    weights = torch.tensor([[0.5, 0.25, 9.0], [1.0, 9.0, 9.0], [9.0, 9.0, 9.0], [-1.0, 2.0, 0.0]])
    y = bl.forward_experts_combine(*layer.tables(), layer.x.to(DEV), 20, 64, slots.to(DEV), weights.to(DEV))
    v, dv, there = layer.reference("none", bias=False)
    v, dv = ref.combine(v, dv, there, slots, weights)
    ref.check(y, v, dv)
    assert (y[2] == 0).all()


# ---- the router ---------------------------------------------------------------------------------------------


def check_route(logits, k, renormalize, routed=None):
    r = routed or bl.route_experts(logits.to(DEV), k, renormalize=renormalize)
    ids, weights, offsets, rows, slots = ref.route(logits, k, renormalize)
    assert torch.equal(r.experts.cpu(), ids)
    assert torch.equal(r.offsets.cpu(), offsets)
    assert torch.equal(r.rows.cpu(), rows)
    assert torch.equal(r.slots.cpu(), slots)
    # e^x: the difference of logits rounds once (absolute error u |d|, relative in e^d), then 4 u; sums of up to
    # E terms in a tree of at most 16 steps, the division
    x = logits.double().nan_to_num(0.0).clamp(min=-1e30, max=1e30)
    spread = (x.amax(1, keepdim=True) - x.amin(1, keepdim=True)).clamp(max=110)
    assert ((r.weights.double().cpu() - weights).abs() <= (2 * spread + 30) * ref.U * weights + 1e-37).all()


@pytest.mark.parametrize("m", [1, 2, 63, 256, 257, 1000])
@pytest.mark.parametrize("e,k", [(1, 1), (2, 2), (8, 2), (16, 16), (17, 3), (64, 4), (65, 8), (128, 8), (200, 16), (512, 5)])
def test_route(m, e, k):
    g = torch.Generator().manual_seed(m * 600 + e)
    logits = torch.randn(m, e, generator=g) * 3
    check_route(logits, k, True)
    check_route(logits.to(torch.bfloat16), k, False)


@pytest.mark.parametrize("m,e,k", [(5, 8, 8), (300, 16, 4), (300, 64, 6), (40, 130, 16), (700, 300, 3)])
def test_route_ties_and_what_cannot_be_chosen(m, e, k):
    g = torch.Generator().manual_seed(e)
    logits = torch.randint(-1, 2, (m, e), generator=g).float()  # ties everywhere, 0 and -0 among them
    logits[torch.rand(m, e, generator=g) < 0.2] = -0.0
    for v in (-math.inf, math.nan, math.inf, -math.nan, 3.4028234663852886e38, -3.4028234663852886e38, 1e-45):
        logits[torch.rand(m, e, generator=g) < 0.1] = v
    logits[0] = -math.inf
    logits[m // 2] = math.nan
    logits[m - 1, 1:] = -math.inf
    check_route(logits, k, True)
    check_route(logits, k, False)
    check_route(logits.to(torch.bfloat16), k, True)


@pytest.mark.parametrize("m,e,k", [(70000, 8, 2), (70001, 256, 1)])
def test_route_long(m, e, k):
    """More tokens than the chunks of the shortest kind hold, against torch's stable sort."""
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(m, e, generator=g).to(DEV)
    r = bl.route_experts(logits, k)
    ids = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(r.experts.long(), ids)
    key, order = torch.sort(ids.reshape(-1), stable=True)
    assert torch.equal(r.rows.long(), order // k)
    assert torch.equal(r.slots.view(-1).long()[order], torch.arange(m * k, device=DEV))
    assert torch.equal(r.offsets.long(), torch.searchsorted(key, torch.arange(e + 1, device=DEV)))
    torch.testing.assert_close(r.weights.sum(1), torch.ones(m, device=DEV), rtol=0, atol=4e-6)


@pytest.mark.parametrize("m", [40, 400])
def test_route_graph_and_given_outputs(m):
    e, k = 32, 3
    logits = torch.zeros(m, e, device=DEV)
    out = bl.route_experts(logits, k)
    ws = torch.empty(max(bl.route_experts_ws_bytes(m, e), 1), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert bl.route_experts(logits, k, out=out, workspace=ws) is out
    for i in range(3):
        new = torch.randn(m, e, generator=torch.Generator().manual_seed(i))
        logits.copy_(new)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        check_route(new, k, True, out)


# ---- the whole layer ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("m", [1, 16, 150])
def test_layer_of_experts(m):
    """Router, up projections, squared ReLU, down projections and the residual sum, as a model runs them, each
    step checked against 64 bits on what the step before gave; then all of it captured once and replayed."""
    e, k, h, f = 6, 2, 300, 520
    g = torch.Generator().manual_seed(m)
    q_up, q_down = [ref.random_codes(f, h, g) for _ in range(e)], [ref.random_codes(h, f, g) for _ in range(e)]
    up, down = (torch.stack([ref.pack(q) for q in qs]).to(DEV) for qs in (q_up, q_down))
    gu, gd = 0.01 + 0.01 * torch.rand(e, generator=g), 0.01 + 0.01 * torch.rand(e, generator=g)
    b = 0.1 * torch.randn(e, f, generator=g)
    x = torch.randn(m, h, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(m, e, generator=g).to(DEV)

    def layer():
        r = bl.route_experts(logits, k)
        hidden = bl.forward_experts(up, gu.to(DEV), r.offsets, x, f, h, rows=r.rows, bias=b.to(DEV), act="relu2",
                                    out_dtype=torch.bfloat16)
        y = bl.forward_experts_combine(down, gd.to(DEV), r.offsets, hidden, h, f, r.slots, r.weights, residual=x,
                                       out_dtype=torch.bfloat16)
        return r, hidden, y

    def check(r, hidden, y, what):
        check_route(logits.cpu(), k, True, r)
        q, a = ref.quantize(x.cpu())
        v, dv, _ = ref.experts(q, a, q_up, gu, b, "relu2", r.offsets.cpu(), r.rows.cpu())
        ref.check(hidden, *ref.finish(v, dv, None, torch.bfloat16), what)
        q, a = ref.quantize(hidden.cpu())
        v, dv = ref.combine(*ref.experts(q, a, q_down, gd, None, "none", r.offsets.cpu(), None), r.slots.cpu(), r.weights.cpu())
        ref.check(y, *ref.finish(v, dv, x.cpu(), torch.bfloat16), what)

    gu, gd, b = gu, gd, b
    check(*layer(), "eager")
    gu_d, gd_d, b_d = gu.to(DEV), gd.to(DEV), b.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def captured():
        r = bl.route_experts(logits, k)
        hidden = bl.forward_experts(up, gu_d, r.offsets, x, f, h, rows=r.rows, bias=b_d, act="relu2", out_dtype=torch.bfloat16)
        return r, hidden, bl.forward_experts_combine(down, gd_d, r.offsets, hidden, h, f, r.slots, r.weights, residual=x,
                                                     out_dtype=torch.bfloat16)

    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured()
    for i in range(3):
        logits.copy_(torch.randn(m, e, generator=torch.Generator().manual_seed(100 + i)))
        graph.replay()
        torch.cuda.synchronize()
        check(*out, f"replay {i}")
        r, hidden, y = layer()
        assert torch.equal(y, out[2]) and torch.equal(hidden, out[1])


def test_quantize_expert_weights():
    w = torch.randn(5, 33, 300, generator=torch.Generator().manual_seed(0)).to(DEV) * 0.02
    packed, gamma = bl.quantize_expert_weights(w)
    for i in range(5):
        p, gm = bl.quantize_weights(w[i])
        assert torch.equal(packed[i], p) and torch.equal(gamma[i:i + 1], gm)


# ---- offsets past 32 bits, calls of other kernels' shapes ------------------------------------------------------


@pytest.mark.parametrize("t", [2, 40, 700])
def test_packed_weights_past_4_gib(t):
    """The last of 20 experts of 256 MiB each: the same as that matrix alone (any bytes are valid weights)."""
    e, n, k = 20, 16384, 65536
    g = torch.Generator(device=DEV).manual_seed(t)
    packed = torch.zeros(e, bl.packed_bytes(n, k), dtype=torch.uint8, device=DEV)
    packed[-1].random_(0, 256, generator=g)
    gamma = torch.full((e,), 0.01, device=DEV)
    x = torch.randn(t, k, generator=g, device=DEV).to(torch.bfloat16)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[-1] = t
    y = bl.forward_experts(packed, gamma, offsets, x, n, k, act="relu")
    alone = bl.forward_epilogue(packed[-1], gamma[-1:], x, n, k, act="relu")
    assert torch.equal(y, alone)
    assert (y > 0).any()


def test_outputs_past_4_gib():
    """Rows of Y and of the residual behind 2^32 bytes, of codes behind 2^24 rows' starts: as in a call of their own."""
    m, n, k = 140001, 8200, 260
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(m, k, generator=g, device=DEV)
    packed = torch.randint(0, 256, (bl.packed_bytes(n, k),), generator=g, device=DEV, dtype=torch.uint8)
    gamma = torch.full((1,), 0.01, device=DEV)
    res = torch.randn(m, n, generator=g, device=DEV, dtype=torch.bfloat16)
    y = bl.forward_epilogue(packed, gamma, x, n, k, residual=res)
    for rows in (slice(0, 300), slice(m - 300, m)):
        assert torch.equal(y[rows], bl.forward_epilogue(packed, gamma, x[rows].contiguous(), n, k, residual=res[rows]))


@pytest.mark.parametrize("counts", [[300, 0, 517, 64, 1], [4000, 130], [40] * 30], ids=str)
def test_experts_equal_single_matrices(counts):
    """Large groups: every expert's rows as forward_epilogue gives them for that matrix."""
    layer = Layer(counts, 1100, 700, r=999)
    x = layer.x.to(DEV)
    rows, packed, gamma, bias = layer.rows.to(DEV), layer.packed, layer.gamma.to(DEV), layer.bias.to(DEV)
    r = torch.randn(layer.t, 1100, device=DEV)
    y = bl.forward_experts(packed, gamma, layer.offsets.to(DEV), x, 1100, 700, rows=rows, bias=bias, act="silu", residual=r,
                           out_dtype=torch.bfloat16)
    for e, n in enumerate(counts):
        if n:
            s = slice(int(layer.offsets[e]), int(layer.offsets[e + 1]))
            one = bl.forward_epilogue(packed[e], gamma[e:e + 1], x[rows[s].long()], 1100, 700, bias=bias[e].contiguous(), act="silu",
                                      residual=r[s], out_dtype=torch.bfloat16)
            assert torch.equal(y[s], one)


def test_two_streams_at_once():
    """Calls on two streams with their own buffers do not disturb each other."""
    layers = [Layer([50, 3, 0, 70], 300, 900, r=60, seed=i) for i in range(2)]
    refs = [layer.forward("gelu") for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[], []]
    args = [(layer.tables(), layer.x.to(DEV), layer.rows.to(DEV), layer.bias.to(DEV)) for layer in layers]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                tables, x, rows, bias = args[i]
                outs[i].append(bl.forward_experts(*tables, x, 300, 900, rows=rows, bias=bias, act="gelu"))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, refs[i]) for o in outs[i])
