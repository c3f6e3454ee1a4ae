"""Products with an epilogue, products by expert and the router: refusals and host-only calls (nothing reaches a GPU),
and the 64-bit reference of the GPU tests against plain loops."""
import ctypes
import math

import pytest
import torch

import bitlinear_fwd_amd as bl
import experts_reference as ref

FAKE = 0x10000  # never dereferenced: calls are refused first
INVALID, UNSUPPORTED = bl.BL_ERR_INVALID_ARG, bl.BL_ERR_UNSUPPORTED


def ep(**kw):
    d = dict(bias=FAKE, residual=FAKE, Y=FAKE, residual_ld=0, y_ld=0, act=0, residual_dt=bl.BL_F32, y_dt=bl.BL_F32)
    d.update(kw)
    return bl.BlEpilogue(**d)


EP_REFUSALS = [(dict(Y=None), INVALID), (dict(act=-1), INVALID), (dict(act=6), INVALID), (dict(y_dt=2), UNSUPPORTED),
               (dict(residual_dt=7), UNSUPPORTED), (dict(bias=FAKE + 2), INVALID), (dict(Y=FAKE + 2), INVALID),
               (dict(Y=FAKE + 1, y_dt=bl.BL_BF16), INVALID), (dict(residual=FAKE + 2), INVALID),
               (dict(residual=FAKE + 1, residual_dt=bl.BL_BF16), INVALID), (dict(y_ld=15), INVALID),
               (dict(residual_ld=15), INVALID), (dict(y_ld=-16), INVALID), (dict(y_ld=1 << 41), INVALID)]
X_REFUSALS = [(dict(X=None, Xq=None), INVALID), (dict(X=None, absmax=None), INVALID), (dict(dt=2), UNSUPPORTED),
              (dict(X=FAKE + 2), INVALID), (dict(X=FAKE + 1, dt=bl.BL_BF16), INVALID), (dict(Xq=FAKE + 8), INVALID),
              (dict(absmax=FAKE + 2), INVALID), (dict(K=0), INVALID), (dict(K=(1 << 24) + 1), INVALID),
              (dict(K=-256), INVALID)]


def epilogue(e=None, **kw):
    d = dict(packed=FAKE, gamma=FAKE, X=FAKE, dt=bl.BL_F32, Xq=FAKE, absmax=FAKE, M=5, N=16, K=256)
    d.update(kw)
    return bl.lib().bitlinear_forward_epilogue(d["packed"], d["gamma"], d["X"], d["dt"], d["Xq"], d["absmax"], d["M"],
                                               d["N"], d["K"], None if e is None else ctypes.byref(e), None)


@pytest.mark.parametrize("kw,status", X_REFUSALS + [
    (dict(packed=None), INVALID), (dict(gamma=None), INVALID), (dict(M=0), INVALID), (dict(N=0), INVALID),
    (dict(M=-1), INVALID), (dict(N=1 << 31), INVALID), (dict(M=1 << 31), INVALID), (dict(packed=FAKE + 8), INVALID),
    (dict(gamma=FAKE + 2), INVALID), (dict(M=(1 << 31) - 1, N=(1 << 31) - 1), UNSUPPORTED),
    (dict(N=1 << 26, K=1 << 24), UNSUPPORTED), (dict(M=1 << 30, K=1 << 20), UNSUPPORTED)])
def test_epilogue_refuses(kw, status):
    assert epilogue(ep(), **kw) == status


@pytest.mark.parametrize("kw,status", EP_REFUSALS)
def test_epilogue_struct_refused(kw, status):
    assert epilogue(ep(**kw)) == status
    assert epilogue(None) == INVALID


def experts(e=None, fn="experts", ex=None, **kw):
    d = dict(packed=FAKE, gamma=FAKE, offsets=FAKE, rows=FAKE, E=4, T=10, N=16, X=FAKE, dt=bl.BL_F32, Xq=FAKE, absmax=FAKE,
             R=5, K=256, slots=FAKE, weights=FAKE, M=5, k=2, ws=FAKE, ws_bytes=10 * 16 * 4)
    d.update(kw)
    x = bl.BlExperts(*(d[n] for n in ("packed", "gamma", "offsets", "rows", "E", "T", "N")))
    px = None if ex == "null" else ctypes.byref(x)
    pe = None if e is None else ctypes.byref(e)
    if fn == "experts":
        return bl.lib().bitlinear_forward_experts(px, d["X"], d["dt"], d["Xq"], d["absmax"], d["R"], d["K"], pe, None)
    return bl.lib().bitlinear_forward_experts_combine(px, d["X"], d["dt"], d["Xq"], d["absmax"], d["R"], d["K"], d["slots"],
                                                      d["weights"], d["M"], d["k"], pe, d["ws"], d["ws_bytes"], None)


@pytest.mark.parametrize("fn", ["experts", "combine"])
@pytest.mark.parametrize("kw,status", X_REFUSALS + [
    (dict(packed=None), INVALID), (dict(gamma=None), INVALID), (dict(offsets=None), INVALID), (dict(offsets=FAKE + 2), INVALID),
    (dict(rows=FAKE + 1), INVALID), (dict(E=0), INVALID), (dict(E=-3), INVALID), (dict(E=4097), UNSUPPORTED),
    (dict(E=1 << 40), UNSUPPORTED), (dict(T=0), INVALID), (dict(T=1 << 31), INVALID), (dict(R=0), INVALID), (dict(R=1 << 31), INVALID),
    (dict(N=0), INVALID), (dict(ex="null"), INVALID), (dict(T=(1 << 31) - 1, N=1 << 20), UNSUPPORTED)])
def test_experts_refuse(fn, kw, status):
    assert experts(ep(), fn, **kw) == status


@pytest.mark.parametrize("fn", ["experts", "combine"])
@pytest.mark.parametrize("kw,status", EP_REFUSALS)
def test_experts_struct_refused(fn, kw, status):
    assert experts(ep(**kw), fn) == status
    assert experts(None, fn) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(slots=None), INVALID), (dict(weights=None), INVALID), (dict(M=0), INVALID), (dict(k=0), INVALID), (dict(k=65), UNSUPPORTED),
    (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID), (dict(ws_bytes=639), INVALID), (dict(slots=FAKE + 2), INVALID),
    (dict(weights=FAKE + 2), INVALID), (dict(M=1 << 31), INVALID)])
def test_combine_refuses(kw, status):
    assert experts(ep(), "combine", **kw) == status


def test_combine_workspace():
    f = bl.lib().bitlinear_forward_experts_combine_ws_bytes
    assert f(10, 16) == 640 and f(0, 16) == -1 and f(3, 0) == -1 and f(1 << 31, 1) == -1 and f((1 << 31) - 1, 1 << 20) == -1
    with pytest.raises(ValueError):
        bl.forward_experts_combine_ws_bytes(0, 4)


def route(**kw):
    d = dict(logits=FAKE, dt=bl.BL_F32, M=1000, E=64, k=4, renorm=1, experts=FAKE, weights=FAKE, offsets=FAKE, rows=FAKE,
             slots=FAKE, ws=FAKE, ws_bytes=1 << 20)
    d.update(kw)
    return bl.lib().bitlinear_route_experts(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(weights=None), INVALID), (dict(offsets=None), INVALID),
    (dict(rows=None), INVALID), (dict(slots=None), INVALID), (dict(M=0), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID),
    (dict(k=65), INVALID), (dict(E=2, k=3), INVALID), (dict(renorm=2), INVALID), (dict(dt=3), UNSUPPORTED),
    (dict(E=513), UNSUPPORTED), (dict(k=17), UNSUPPORTED), (dict(M=1 << 30, k=2), UNSUPPORTED), (dict(M=1 << 31), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=4), INVALID), (dict(ws=FAKE + 2), INVALID), (dict(logits=FAKE + 2), INVALID),
    (dict(logits=FAKE + 1, dt=bl.BL_BF16), INVALID), (dict(slots=FAKE + 1), INVALID)])
def test_route_refuses(kw, status):
    assert route(**kw) == status


def test_route_workspace():
    assert bl.route_experts_ws_bytes(1, 8) == 0
    assert bl.route_experts_ws_bytes(65536, 128) > 0
    with pytest.raises(ValueError):
        bl.route_experts_ws_bytes(0, 8)


def test_plans():
    for m, n, k in [(1, 1, 1), (16, 2560, 6912), (2048, 6912, 2560), (300, 515, 33)]:
        for x in (None, "bf16", "f32"):
            for p in (bl.forward_epilogue_plan(m, n, k, x), bl.forward_experts_plan(8, m, n, k, x)):
                assert p["workgroups"] > 0 and p["threads"] % 64 == 0 and p["launches"] in (1, 2)
                assert x is not None or p["launches"] == 1
    with pytest.raises(bl.BitLinearError):
        bl.forward_epilogue_plan(0, 16, 16)
    with pytest.raises(ValueError):
        bl.forward_experts_plan(0, 16, 16, 16)
    with pytest.raises(ValueError):
        bl.forward_epilogue_plan(1, 16, 16, "f16")


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        bl.route_experts(torch.zeros(4, 4), 2)
    with pytest.raises(ValueError):
        bl.forward_epilogue(torch.zeros(1024, dtype=torch.uint8), torch.zeros(1), torch.zeros(4, 16), 16, 16)


# ---- the reference itself -----------------------------------------------------------------------------------


def test_reference_pack_matches_the_layout():
    g = torch.Generator().manual_seed(0)
    q = ref.random_codes(19, 300, g)
    b = ref.pack(q)
    code = {0: 0, 1: 1, -1: 2}
    for n, k in [(0, 0), (18, 299), (3, 17), (16, 255), (7, 256), (5, 64), (9, 79)]:
        kk = k % 256
        at = (n // 16 * 2 + k // 256) * 1024 + 16 * (16 * (kk // 64) + n % 16) + 4 * (kk % 64 // 16) + kk % 4
        assert int(b[at]) >> (2 * (kk % 16 // 4)) & 3 == code[int(q[n, k])]
    assert int(b[1024 + 16 * 5 + 0]) & 3 == code[int(q[5, 256])]  # columns past K hold 3
    assert int(b[1024 + 16 * (16 * 3 + 5)]) == 255


def test_reference_product_and_combine():
    g = torch.Generator().manual_seed(1)
    qs = [ref.random_codes(3, 5, g) for _ in range(2)]
    x = torch.randn(4, 5, generator=g)
    q, a = ref.quantize(x)
    rows, offsets = torch.tensor([2, 0, 3, -1]), [0, 1, 4]
    bias = torch.randn(2, 3, generator=g)
    y, dy, there = ref.experts(q, a, qs, [0.5, 2.0], bias, "relu2", offsets, rows)
    assert there.tolist() == [True, True, True, False] and (dy[:3] > 0).any()
    for s, e in [(0, 0), (1, 1), (2, 1)]:
        r = int(rows[s])
        for n in range(3):
            v = sum(int(q[r, k]) * int(qs[e][n, k]) for k in range(5)) * [0.5, 2.0][e] * float(a[r]) / 127 + float(bias[e, n])
            assert math.isclose(float(y[s, n]), max(v, 0) ** 2, rel_tol=1e-12, abs_tol=1e-12)
    out, _ = ref.combine(y, dy, there, torch.tensor([[2, 0], [3, -1]]), torch.tensor([[0.25, 4.0], [1.0, 1.0]]))
    assert torch.allclose(out[0], 0.25 * y[2] + 4 * y[0]) and (out[1] == 0).all()


def test_reference_activations():
    v = torch.linspace(-8, 8, 101, dtype=torch.float64)
    zero = torch.zeros_like(v)
    assert torch.allclose(ref.act(v, zero, "silu")[0], torch.nn.functional.silu(v))
    assert torch.allclose(ref.act(v, zero, "gelu")[0], torch.nn.functional.gelu(v))
    assert torch.allclose(ref.act(v, zero, "gelu_tanh")[0], torch.nn.functional.gelu(v, approximate="tanh"))
    assert torch.equal(ref.act(v, zero, "relu2")[0], torch.relu(v) ** 2)


def test_reference_route():
    ids, w, offsets, rows, slots = ref.route(torch.tensor([[1.0, 3.0, 3.0], [-math.inf, 2.0, math.nan]]), 2, True)
    assert ids.tolist() == [[1, 2], [1, -1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0]]
    assert offsets.tolist() == [0, 0, 2, 3] and rows.tolist() == [0, 1, 0, -1] and slots.tolist() == [[0, 2], [1, -1]]
