"""MXFP4 and layer norm on the host: size helpers, refusals, and the tests' own plain forms
checked against hand-derived values.  No call here reaches a GPU."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import bitlinear_fwd_amd as bl
import mxfp4_reference as ref

FAKE = 0x10000  # aligned non-null address; never dereferenced (calls are rejected first)
BAD, UNS = bl.BL_ERR_INVALID_ARG, bl.BL_ERR_UNSUPPORTED


def test_sizes():
    L = bl.lib()
    for r, k in ((1, 1), (16, 128), (17, 129), (6912, 2560), (1003, 7001), (28672, 8192), (5, 513)):
        assert bl.mxfp4_codes_bytes(r, k) == L.bitlinear_mxfp4_codes_bytes(r, k) == -(-r // 16) * -(-k // 128) * 1024
        assert bl.mxfp4_scales_bytes(r, k) == L.bitlinear_mxfp4_scales_bytes(r, k) == -(-r // 16) * -(-k // 512) * 256
    for r, k in ((0, 5), (5, 0), (-1, 3)):
        assert bl.mxfp4_codes_bytes(r, k) == L.bitlinear_mxfp4_codes_bytes(r, k) == -1
        assert bl.mxfp4_scales_bytes(r, k) == L.bitlinear_mxfp4_scales_bytes(r, k) == -1
    assert L.bitlinear_layernorm_backward_ws_bytes(0, 5) == -1
    assert L.bitlinear_layernorm_backward_ws_bytes(5, (1 << 24) + 1) == -1
    assert bl.layernorm_backward_ws_bytes(1, 8) >= 8 * 8
    with pytest.raises(ValueError):
        bl.layernorm_backward_ws_bytes(0, 8)
    with pytest.raises(ValueError):
        bl.forward_mxfp4_fused_ws_bytes(0, 8, 8)
    assert L.bitlinear_forward_mxfp4_fused_ws_bytes(1, 8, 8, 7) == -1


def test_quantize_refusals():
    f = bl.lib().bitlinear_quantize_mxfp4
    ok = [FAKE, bl.BL_F32, 4, 64, FAKE, FAKE, None, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(a0=None) == BAD and call(a4=None) == BAD and call(a5=None) == BAD
    assert call(a1=2) == UNS and call(a1=-1) == UNS
    assert call(a2=0) == BAD and call(a3=0) == BAD and call(a2=1 << 31) == BAD and call(a3=(1 << 24) + 1) == BAD
    assert call(a2=1 << 20, a3=1 << 21) == UNS
    assert call(a0=FAKE + 2) == BAD and call(a4=FAKE + 8) == BAD and call(a5=FAKE + 2) == BAD
    assert call(a1=bl.BL_BF16, a0=FAKE + 1) == BAD and call(a6=FAKE + 2) == BAD


def test_forward_refusals():
    f = bl.lib().bitlinear_forward_mxfp4
    ok = [FAKE, FAKE, FAKE, FAKE, 4, 16, 64, FAKE, bl.BL_F32, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 1, 2, 3, 7):
        assert call(**{f"a{i}": None}) == BAD
    for i in (4, 5, 6):
        assert call(**{f"a{i}": 0}) == BAD and call(**{f"a{i}": 1 << 31}) == BAD
    assert call(a6=(1 << 24) + 1) == BAD
    assert call(a8=2) == UNS
    assert call(a4=(1 << 31) - 1, a5=(1 << 31) - 1, a6=1) == UNS  # too many output tiles
    assert call(a5=1 << 30, a6=1 << 12) == UNS
    assert call(a0=FAKE + 8) == BAD and call(a2=FAKE + 8) == BAD and call(a1=FAKE + 2) == BAD
    assert call(a3=FAKE + 1) == BAD and call(a7=FAKE + 2) == BAD


def test_fused_refusals():
    f = bl.lib().bitlinear_forward_mxfp4_fused
    m, n, k = 2048, 16, 512  # takes a workspace
    need = bl.lib().bitlinear_forward_mxfp4_fused_ws_bytes(m, n, k, bl.BL_BF16)
    assert need > 0
    ok = [FAKE, FAKE, FAKE, bl.BL_BF16, m, n, k, FAKE, bl.BL_F32, FAKE, need, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 1, 2, 7, 9):
        assert call(**{f"a{i}": None}) == BAD
    for i in (4, 5, 6):
        assert call(**{f"a{i}": 0}) == BAD
    assert call(a3=9) == UNS and call(a8=9) == UNS
    assert call(a10=need - 1) == BAD and call(a9=FAKE + 8) == BAD
    assert call(a0=FAKE + 4) == BAD and call(a1=FAKE + 1) == BAD
    assert call(a2=FAKE + 1) == BAD and call(a7=FAKE + 2) == BAD


def test_layernorm_refusals():
    L = bl.lib()
    ok = [FAKE, bl.BL_BF16, 4, 64, FAKE, FAKE, 1e-5, FAKE, FAKE, FAKE, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return L.bitlinear_layernorm(*a)

    assert call(a0=None) == BAD and call(a7=None) == BAD
    assert call(a2=0) == BAD and call(a3=0) == BAD and call(a3=(1 << 24) + 1) == BAD
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert call(a6=eps) == BAD
    assert call(a1=4) == UNS and call(a2=1 << 30, a3=1 << 12) == UNS
    assert call(a0=FAKE + 1) == BAD and call(a4=FAKE + 2) == BAD and call(a5=FAKE + 1) == BAD
    assert call(a7=FAKE + 1) == BAD and call(a8=FAKE + 2) == BAD and call(a9=FAKE + 2) == BAD


def test_layernorm_backward_refusals():
    L = bl.lib()
    need = bl.layernorm_backward_ws_bytes(4, 64)
    ok = [FAKE, FAKE, bl.BL_F32, 4, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, need, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return L.bitlinear_layernorm_backward(*a)

    for i in (0, 1, 6, 7, 11):
        assert call(**{f"a{i}": None}) == BAD
    assert call(a8=None, a9=None, a10=None) == BAD
    assert call(a3=0) == BAD and call(a4=0) == BAD
    assert call(a2=3) == UNS and call(a3=1 << 30, a4=1 << 12) == UNS
    assert call(a12=need - 1) == BAD and call(a11=FAKE + 8) == BAD
    for i in (0, 1, 5, 6, 7, 8, 9, 10):
        assert call(**{f"a{i}": FAKE + 2}) == BAD


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: bl.quantize_mxfp4(x), lambda: bl.layernorm(x),
                 lambda: bl.layernorm_backward(x, x, None, torch.zeros(4), torch.zeros(4)),
                 lambda: bl.forward_mxfp4_fused(x, x, x, 4, 64),
                 lambda: bl.forward_mxfp4(x, x, x, x, 4, 4, 64)):
        with pytest.raises(ValueError):
            call()


def test_reference_grid_by_hand():
    """Every border of the grid, with the block's largest magnitude 6 (scale 1)."""
    pairs = [(0.0, 0), (0.25, 0), (0.26, 1), (0.5, 1), (0.74, 1), (0.75, 2), (1.25, 2), (1.26, 3), (1.74, 3), (1.75, 4),
             (2.5, 4), (2.51, 5), (3.49, 5), (3.5, 6), (5.0, 6), (5.01, 7), (6.0, 7), (7.9, 7)]
    x = np.zeros((2, 32))
    x[0, :18] = [p[0] for p in pairs]
    x[1, :18] = [-p[0] for p in pairs]
    x[:, 31] = 4.0
    codes, scales, values = ref.quantize(x)
    assert scales.tolist() == [[127], [127]]
    assert codes[0, :18].tolist() == [p[1] for p in pairs]
    assert codes[1, 1:18].tolist() == [p[1] + 8 for p in pairs][1:]
    assert values[0, 17] == 6.0 and values[1, 17] == -6.0


def test_reference_scales_by_hand():
    x = np.zeros((7, 40))
    x[1, 5] = 1.0        # E 127: e 125, 1.0 / 2^-2 = 4
    x[2, 5] = 2.0 ** -126
    x[3, 5] = 2.0 ** -149
    x[4, 5] = 2.0 ** -124
    x[5, 5] = 3.4e38
    x[6, 39] = np.inf
    codes, scales, values = ref.quantize(x)
    assert scales[:, 0].tolist() == [0, 125, 0, 0, 1, 252, 0]
    assert codes[1, 5] == 6 and values[1, 5] == 1.0
    assert codes[2, 5] == 4 and values[2, 5] == 2.0 ** -126   # 2 * 2^-127
    assert codes[3, 5] == 0
    assert codes[4, 5] == 6 and values[4, 5] == 2.0 ** -124
    assert values[5, 5] == 6 * 2.0 ** 125
    assert scales[6, 1] == 255 and np.isnan(values[6, 32:]).all() and values[6, 0] == 0
    packed, sc = ref.pack(codes, scales, 40)
    assert packed.size == 1024 and sc.size == 256
    assert packed[16 * 1 + 2] == 6 << 4           # row 1, column 5: byte 2, high nibble
    assert sc[(16 * 1 + 6) * 4] == 255            # row 6, block 1


def test_reference_layernorm_gradients_by_differences():
    """The gradient formulas against central differences in 64 bits (step 1e-5: the error of the
    difference is about 1e-10 of the loss's third derivative, and 1e-11 of rounding)."""
    rng = np.random.default_rng(5)
    x, w, b, r = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=7), rng.normal(size=(3, 7))
    eps = 1e-3

    def loss(x, w, b):
        return float((ref.layernorm(x, w, b, eps)[0] * r).sum())

    _, mean, rstd = ref.layernorm(x, w, b, eps)
    dx, dw, db = ref.layernorm_backward(r, x, w, mean, rstd)[:3]
    for arr, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + 1e-5
            up = loss(x, w, b)
            arr[i] = keep - 1e-5
            down = loss(x, w, b)
            arr[i] = keep
            assert abs((up - down) / 2e-5 - grad[i]) < 1e-6, i


# (M, N, K), the kernel of the product and, of the fused call on bf16, its launches: each shape below is
# one that the GPU tests run, so that every kernel form is reached there
VARIANTS = [((1, 6912, 2560), ("lds", 16, 16), 1), ((16, 64, 8704), ("lds", 16, 16), 2),
            ((16, 40, 28672), ("decode", 16, 16), 2), ((16, 4100, 28672), ("decode", 16, 32), 2),
            ((17, 64, 128), ("decode", 32, 16), 2), ((20, 4100, 1100), ("decode", 32, 32), 2),
            ((64, 2560, 2560), ("decode", 64, 16), 2), ((100, 4100, 1100), ("decode", 64, 32), 2),
            ((520, 300, 640), ("decode", 64, 16), 2), ((600, 515, 2049), ("decode", 64, 32), 2),
            ((2100, 4000, 390), ("gemm", 128, 256), 2), ((2050, 4100, 120), ("gemm", 128, 256), 2),
            ((1030, 1500, 1000), ("gemm", 128, 128), 2), ((2060, 2030, 260), ("gemm", 128, 128), 2),
            ((4100, 300, 640), ("gemm", 128, 128), 2), ((1030, 2000, 1930), ("gemm", 128, 128), 2),
            ((4100, 260, 2177), ("gemm", 128, 128), 2), ((1100, 2000, 4100), ("gemm", 128, 128), 2),
            ((2100, 2000, 6200), ("gemm", 128, 256), 2), ((33000, 130, 600), ("gemm", 128, 256), 2)]


@pytest.mark.parametrize("shape,want,launches", VARIANTS)
def test_plan(shape, want, launches):
    p = bl.forward_mxfp4_plan(*shape)
    assert (p["kernel"], p["tokens"], p["outputs"]) == want and p["launches"] == 1
    f = bl.forward_mxfp4_plan(*shape, x="bf16")
    assert f["launches"] == launches and (launches == 2) == (bl.forward_mxfp4_fused_ws_bytes(*shape) > 0)
    m, n, k = shape
    if p["kernel"] != "lds":  # workgroups cover the output once
        assert p["workgroups"] == -(-m // p["tokens"]) * -(-n // p["outputs"])
    assert p["threads"] in range(64, 1025, 64)


@pytest.mark.parametrize("n,outputs", [(48, 128), (128, 128), (129, 256), (300, 128), (512, 256), (640, 128),
                                       (700, 256), (800, 256), (1100, 256)])
def test_plan_tile_width(n, outputs):
    """Wide tiles of the GEMM only where little of them lies past the last column."""
    p = bl.forward_mxfp4_plan(65536, n, 640)
    assert p["kernel"] == "gemm" and p["outputs"] == outputs


def test_plan_refusals():
    out = (ctypes.c_int32 * 6)()
    f = bl.lib().bitlinear_forward_mxfp4_plan
    assert f(0, 1, 1, -1, out) == BAD and f(1, 1, 1 << 25, -1, out) == BAD and f(1, 1, 1, -1, None) == BAD
    assert f(1, 1, 1, 5, out) == UNS and f(1 << 30, 1 << 30, 1, -1, out) == UNS


def test_lds_limits_are_constants():
    """A kernel's LDS limit is shared by all host threads, so each is set to one constant and never to a call's
    own size, which another thread's larger call could find in its way."""
    csrc = os.path.join(os.path.dirname(bl.__file__), "csrc")
    sizes = []
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            sizes += re.findall(r"hipFuncAttributeMaxDynamicSharedMemorySize,\s*(?:\(int\)\s*)?([\w.]+)", f.read())
    assert len(sizes) >= 2 and all(re.fullmatch(r"k[A-Z]\w*|\d+", v) for v in sizes), sizes


# (M, N, K) of each form of the products' kernels: the GPU tests run all of them, with both output types
FORMS = [("lds", (7, 100, 513)), ("decode 16 16 once", (16, 40, 28672)), ("decode 16 32 once", (16, 4100, 28672)),
         ("decode 32 16 once", (17, 64, 128)), ("decode 32 32 once", (20, 4100, 1100)),
         ("decode 64 16 once", (64, 2560, 2560)), ("decode 64 32 once", (37, 6909, 2570)),
         ("decode 64 32 once", (50, 4099, 1030)), ("decode 64 32 once", (64, 4112, 384)),
         ("decode 64 16 again", (520, 300, 640)), ("decode 64 32 again", (100, 4100, 1100)),
         ("gemm 128", (1030, 1500, 1000)), ("gemm 256", (2100, 4000, 390))]


def form(m, n, k):
    p = bl.forward_mxfp4_plan(m, n, k)
    if p["kernel"] != "decode":
        return p["kernel"] if p["kernel"] == "lds" else f"gemm {p['outputs']}"
    once = "once" if p["workgroups"] == -(-n // p["outputs"]) else "again"
    return f"decode {p['tokens']} {p['outputs']} {once}"


@pytest.mark.parametrize("want,shape", FORMS)
def test_form(want, shape):
    assert form(*shape) == want


def test_every_form_of_the_library_is_listed():
    """The products' kernels in the built library are those of FORMS, each with both output types (and the
    one-launch kernel with its three sources): none that no call reaches, and none that no test runs."""
    with open(bl.LIB_PATH, "rb") as f:
        names = f.read()
    built = {(f"decode {16 * int(tg)} {16 * int(rb)} {'once' if once == b'1' else 'again'}", y.decode())
             for tg, rb, once, y in re.findall(rb"k_mx_decodeILi(\d)ELi(\d)ELb(\d)E([ft])E", names)}
    built |= {(f"gemm {128 * int(tn)}", y.decode()) for tn, y in re.findall(rb"k_mx_gemmILi(\d)E([ft])E", names)}
    built |= {("lds", src.decode() + y.decode()) for src, y in re.findall(rb"k_mx_fewILi(\d)E([ft])E", names)}
    listed = {(w, y) for w in {w for w, _ in FORMS} - {"lds"} for y in "ft"}
    assert built == listed | {("lds", s + y) for s in "012" for y in "ft"}


@pytest.mark.parametrize("name", ["bfloat16", "fp32", "BF16", "", 0, torch.bfloat16])
def test_type_names(name):
    """A type the calls do not know is refused, not described as fp32."""
    with pytest.raises(ValueError):
        bl.forward_mxfp4_plan(16, 64, 512, x=name)
    with pytest.raises(ValueError):
        bl.forward_mxfp4_fused_ws_bytes(16, 64, 512, name)
