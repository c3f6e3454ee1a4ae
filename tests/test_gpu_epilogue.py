"""Products with an epilogue against the definition in 64 bits (experts_reference)."""
import pytest
import torch

import bitlinear_fwd_amd as bl
import experts_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = list(bl.ACTIVATIONS)


def make(m, n, k, x="bf16", seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed * 7919 + m * 31 + n * 17 + k)
    q_w = ref.random_codes(n, k, g)
    xv = torch.randn(m, k, generator=g) * spread
    xv[torch.rand(m, k, generator=g) < 0.005] *= 30
    gamma = 0.01 + 0.02 * torch.rand(1, generator=g)
    return q_w, xv.to(DT[x]), gamma, torch.randn(n, generator=g) * 0.3, torch.randn(m, n, generator=g)


def codes_of(x):
    """int8 codes and scales as the library takes them, from the reference's."""
    q, a = ref.quantize(x)
    full = torch.zeros(x.shape[0], (x.shape[1] + 255) // 256 * 256, dtype=torch.int8)
    full[:, :x.shape[1]] = q.to(torch.int8)
    return full.to(DEV), a.float().to(DEV)


def run(m, n, k, x="bf16", act="none", bias=True, res="f32", out="f32", codes=False, seed=0, spread=1.0):
    q_w, xv, gamma, b, r = make(m, n, k, x, seed, spread)
    r = r.to(DT[res]) if res else None
    b = b if bias else None
    packed = ref.pack(q_w).to(DEV)
    arg, absmax = codes_of(xv) if codes else (xv.to(DEV), None)
    y = bl.forward_epilogue(packed, gamma.to(DEV), arg, n, k, absmax=absmax, bias=None if b is None else b.to(DEV), act=act,
                            residual=None if r is None else r.to(DEV), out_dtype=DT[out])
    assert y.dtype == DT[out]
    q, a = ref.quantize(xv)
    v, dv = ref.finish(*ref.product(q, a, q_w, gamma, b, act), r, DT[out])
    ref.check(y, v, dv, f"{(m, n, k, x, act, bias, res, out, codes)}")


SIZES = [(1, 1, 1), (1, 16, 256), (1, 6912, 2560), (2, 17, 300), (3, 1000, 8), (4, 64, 7), (5, 33, 2570), (16, 2560, 6912),
         (16, 65, 512), (17, 64, 256), (31, 200, 300), (32, 48, 1000), (33, 130, 1000), (37, 6909, 257), (48, 16, 4000),
         (64, 256, 2560), (65, 515, 300), (100, 300, 700), (127, 129, 1030), (129, 1000, 513), (300, 2000, 256), (513, 257, 770)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("codes", [False, True], ids=["x", "codes"])
def test_sizes(size, codes):
    run(*size, codes=codes)


@pytest.mark.parametrize("m", [1, 7, 40, 200])
@pytest.mark.parametrize("act", ACTS)
def test_activations(m, act):
    """Arguments from deep in the left tail to far on the right."""
    run(m, 300, 600, act=act, res=None, spread=1.0)
    run(m, 300, 600, act=act, res=None, bias=False, spread=30.0, seed=1)
    run(m, 300, 600, act=act, res="bf16", out="bf16", seed=2)


@pytest.mark.parametrize("m", [1, 16, 50, 260])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_types(m, x, res, out):
    run(m, 515, 700, x=x, res=res, out=out, act="relu2", bias=res is not None)


@pytest.mark.parametrize("m", [1, 16, 40, 150])
def test_equals_forward(m):
    """Without an epilogue: the accumulators of bitlinear_forward, rescaled (four roundings there, three here)."""
    n, k = 515, 700
    q_w, xv, gamma, _, _ = make(m, n, k)
    packed, x = ref.pack(q_w).to(DEV), xv.to(DEV)
    y = bl.forward_epilogue(packed, gamma.to(DEV), x, n, k)
    y0, acc = bl.forward_fused(packed, gamma.to(DEV), x, n, k, want_acc=True)[0]
    torch.testing.assert_close(y, y0, rtol=8 * ref.U, atol=0)
    assert torch.equal(y == 0, acc == 0)


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_in_place_residual_and_parts_of_longer_rows(m):
    n, k = 130, 300
    q_w, xv, gamma, b, r = make(m, n, k)
    q, a = ref.quantize(xv)
    wide = torch.randn(m, 3 * n + 5, device=DEV)
    part = wide[:, n + 1:2 * n + 1]
    part.copy_(r)
    before = wide.clone()
    y = bl.forward_epilogue(ref.pack(q_w).to(DEV), gamma.to(DEV), xv.to(DEV), n, k, bias=b.to(DEV), act="gelu",
                            residual=part, y=part)
    assert y is part
    ref.check(part, *ref.finish(*ref.product(q, a, q_w, gamma, b, "gelu"), r, torch.float32))
    before[:, n + 1:2 * n + 1] = part
    assert torch.equal(before, wide)
    # bf16 rows that start at an odd element, the residual in rows of another length
    out = torch.zeros(m, 2 * n + 1, dtype=torch.bfloat16, device=DEV)[:, 1:n + 1]
    res = torch.zeros(m, n + 3, device=DEV)[:, 2:n + 2]
    res.copy_(r)
    bl.forward_epilogue(ref.pack(q_w).to(DEV), gamma.to(DEV), xv.to(DEV), n, k, residual=res, y=out)
    ref.check(out, *ref.finish(*ref.product(q, a, q_w, gamma, None, "none"), r, torch.bfloat16))


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_rows_of_zeros_and_zero_scale(m):
    n, k = 40, 300
    q_w, xv, gamma, b, r = make(m, n, k)
    xv[0] = 0
    y = bl.forward_epilogue(ref.pack(q_w).to(DEV), gamma.to(DEV), xv.to(DEV), n, k, bias=b.to(DEV))
    assert torch.equal(y[0].cpu(), b)
    y = bl.forward_epilogue(ref.pack(q_w).to(DEV), torch.zeros(1, device=DEV), xv.to(DEV), n, k, bias=b.to(DEV))
    assert torch.equal(y.cpu(), b.expand(m, n))


@pytest.mark.parametrize("m", [1, 3, 16, 40])
def test_x_at_odd_addresses(m):
    """x and y that start anywhere an element can."""
    n, k = 70, 513
    q_w, xv, gamma, b, r = make(m, n, k)
    q, a = ref.quantize(xv)
    buf = torch.zeros(m * k + 1, dtype=torch.bfloat16, device=DEV)[1:]
    buf.copy_(xv.view(-1))
    out = torch.zeros(m * n + 1, dtype=torch.bfloat16, device=DEV)[1:].view(m, n)
    bl.forward_epilogue(ref.pack(q_w).to(DEV), gamma.to(DEV), buf.view(m, k), n, k, bias=b.to(DEV), y=out)
    ref.check(out, *ref.finish(*ref.product(q, a, q_w, gamma, b, "none"), None, torch.bfloat16))


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_graph_replays_and_other_stream(m):
    n, k = 300, 700
    q_w, xv, gamma, b, r = make(m, n, k)
    packed, gm, bd = ref.pack(q_w).to(DEV), gamma.to(DEV), b.to(DEV)
    x, y = xv.to(DEV), torch.zeros(m, n, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bl.forward_epilogue(packed, gm, x, n, k, bias=bd, act="silu", y=y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.forward_epilogue(packed, gm, x, n, k, bias=bd, act="silu", y=y)
    for i in range(3):
        new = torch.randn(m, k, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        x.copy_(new)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        q, a = ref.quantize(new)
        ref.check(y, *ref.product(q, a, q_w, gamma, b, "silu"), f"replay {i}")
        assert torch.equal(y, bl.forward_epilogue(packed, gm, x, n, k, bias=bd, act="silu"))


def exact_on_gpu(q_w, q, a, gamma):
    """The products of codes in 64 bits on the GPU (whole numbers: exact), and the allowed error."""
    raw = (q.to(DEV).double() @ q_w.to(DEV).double().t().contiguous()) * (a.to(DEV) * float(gamma) / 127)[:, None]
    return raw, 3.01 * ref.U * raw.abs()


FORMS = [(1, 700, 1280, "bf16"), (4, 301, 2568, "f32"), (1, 64, 90000, "bf16"), (2, 64, 40000, "f32"), (4, 300, 40000, "f32"),
         (3, 65, 2571, "f32"), (9, 200, 700, "i8"), (9, 4500, 600, "i8"), (33, 9000, 300, "i8"), (64, 6900, 700, "i8"), (1500, 1000, 512, "i8"),
         (1247, 1641, 635, "i8"), (65, 19498, 300, "i8"), (200, 6917, 2560, "i8"), (300, 300, 300, "i8"), (133, 15252, 33, "i8"),
         (700, 3000, 1000, "i8"), (1500, 6900, 1100, "i8"), (6090, 526, 34, "i8"), (2050, 6912, 600, "i8"), (13197, 345, 33, "i8")]


def test_every_form_is_tested():
    plans = [bl.forward_epilogue_plan(m, n, k, None if x == "i8" else x) for m, n, k, x in FORMS]
    seen = {(p["kernel"], p["rows"], p["outputs"]) for p in plans}
    assert {("fused", 16, 16), ("decode", 16, 16), ("decode", 16, 32), ("decode", 16, 64), ("decode", 32, 64)} <= seen
    assert {("gemm", h, w) for h, w in ((32, 128), (64, 128), (64, 256), (96, 256), (128, 256))} <= seen, seen
    assert {p["launches"] for p in plans} == {1, 2}


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_forms(form):
    m, n, k, x = form
    q_w, xv, gamma, _, _ = make(m, n, k, "f32" if x == "i8" else x)
    arg, absmax = codes_of(xv) if x == "i8" else (xv.to(DEV), None)
    q, a = ref.quantize(xv)
    packed, gm = ref.pack(q_w).to(DEV), gamma.to(DEV)
    raw, err = exact_on_gpu(q_w, q, a, gamma)
    y = bl.forward_epilogue(packed, gm, arg, n, k, absmax=absmax)
    assert ((y.double() - raw).abs() <= err).all()
    r = torch.randn(m, n, device=DEV, dtype=torch.bfloat16)
    y = bl.forward_epilogue(packed, gm, arg, n, k, absmax=absmax, act="relu", residual=r, out_dtype=torch.bfloat16)
    v = raw.clamp(min=0) + r.double()
    assert ((y.double() - v).abs() <= err + 1.01 * (2.0 ** -8 + ref.U) * v.abs() + 2 * ref.U * raw.abs()).all()
