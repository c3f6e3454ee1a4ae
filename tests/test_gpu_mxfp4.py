"""MXFP4 on the GPU against the plain 64-bit forms: codes, scales and values bit for bit, products
within a bound on fp32 sums (and bit for bit where every partial sum is an fp32 number)."""
import threading

import numpy as np
import pytest
import torch

import bitlinear_fwd_amd as bl
import mxfp4_reference as ref
from test_mxfp4_cpu import FORMS, VARIANTS
from gpu_helpers import acts_host_f32, check_equal, host

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def outliers(m, k, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((m, k), generator=g, device=DEV)
    return torch.where(torch.rand((m, k), generator=g, device=DEV) < 0.01, x * 30, x).to(dtype)


def check_quantized(x):
    r, k = x.shape
    codes = torch.full((bl.mxfp4_codes_bytes(r, k) + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((bl.mxfp4_scales_bytes(r, k) + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    _, _, values = bl.quantize_mxfp4(x, codes=codes, scales=scales, want_values=True)
    plain = bl.quantize_mxfp4(x)
    q, s, v = ref.quantize(acts_host_f32(x))
    want, wsc = ref.pack(q, s, k)
    check_equal(host(codes)[:want.size], want, "codes")
    check_equal(host(scales)[:wsc.size], wsc, "scales")
    assert (host(codes)[want.size:] == 0xA5).all() and (host(scales)[wsc.size:] == 0xA5).all()
    check_equal(host(plain[0]), want, "codes without values")
    check_equal(host(plain[1]), wsc, "scales without values")
    got = acts_host_f32(values).astype(np.float64)
    assert values.dtype == x.dtype
    check_equal(np.isnan(got), np.isnan(v), "NaN values")
    check_equal(np.nan_to_num(got), np.nan_to_num(v), "values")
    check_equal(np.signbit(got) & ~np.isnan(got), np.signbit(v) & ~np.isnan(v), "signs")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("r,k", [(1, 1), (1, 31), (3, 32), (16, 128), (17, 129), (15, 511), (33, 513), (5, 1000),
                                 (64, 2560), (2, 6912), (37, 7001)])
def test_quantize(r, k, dtype):
    print(f"case: quantize_mxfp4 R={r} K={k} {dtype}", flush=True)
    check_quantized(outliers(r, k, seed=r + k, dtype=DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_wide_range_and_nonfinite(dtype):
    """Blocks over the whole exponent range (subnormals and the largest numbers), zero rows, signed
    zeros, and blocks with a NaN or an infinity among finite ones."""
    g = np.random.default_rng(3)
    x = (g.normal(size=(40, 160)) * np.exp2(g.integers(-150, 127, size=(40, 5)).repeat(32, 1))).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 7], x[3, 40], x[4, 100] = np.nan, np.inf, -np.inf
    x[5, :32] = 3.4e38
    x[6, :32] = 1e-45
    x[7, :64] = np.float32(2.0 ** -126)
    check_quantized(torch.from_numpy(x).to(DEV).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_borders(dtype):
    """Magnitudes at, just under and just over every border between neighbouring grid values, at
    several scales, in blocks whose largest magnitude fixes the scale."""
    rows = []
    for e in (-120, -3, 0, 1, 90):
        for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0):
            v = torch.tensor([border], dtype=DT[dtype])
            bits = v.view(torch.int16 if dtype == "bf16" else torch.int32)
            near = torch.cat([(bits + d).view(DT[dtype]) for d in (-1, 0, 1)]).float()
            row = torch.zeros(32)
            row[:3], row[3:6], row[31] = near, -near, 4.0
            rows.append(torch.ldexp(row, torch.tensor(e)))
    check_quantized(torch.stack(rows).to(DT[dtype]).to(DEV))


def test_quantize_every_bf16_value():
    """Every bf16 bit pattern, 31 of them and one fixed magnitude to a block."""
    bits = np.arange(65536, dtype=np.uint32)
    pad = np.zeros(-(-65536 // 31) * 31, dtype=np.uint32)
    pad[:65536] = bits
    rows = np.zeros((len(pad) // 31, 32), dtype=np.uint32)
    rows[:, :31] = pad.reshape(-1, 31)
    rows[:, 31] = 0x40C0  # 6.0
    x = torch.from_numpy(rows.astype(np.uint16).view(np.int16)).view(torch.bfloat16).to(DEV)
    check_quantized(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_unaligned_source(dtype):
    """A source that starts at an odd element of its storage."""
    flat = outliers(1, 1 + 19 * 333, seed=9, dtype=DT[dtype]).view(-1)
    check_quantized(flat[1:].view(19, 333))


def product_bound(xv, wv, k):
    """|error| of an fp32 sum of the K exact products: every product is an fp32 number times powers
    of two; each matrix instruction adds 128 of them to its accumulator, off by at most 2^-22 of the
    magnitudes it adds, ceil(K / 128) of them in a chain, then up to 16 partial sums."""
    return (-(-k // 128) + 20) * 2.0 ** -22 * (np.abs(xv) @ np.abs(wv).T)


def check_product(y, xv, wv, k):
    want = xv @ wv.T
    got = acts_host_f32(y).astype(np.float64)
    tol = product_bound(xv, wv, k)
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def quantized(x):
    """Codes and scales from the GPU quantiser, the values from the plain form."""
    codes, scales = bl.quantize_mxfp4(x)
    return codes, scales, ref.quantize(acts_host_f32(x))[2]


PRODUCTS = [(1, 16, 32), (1, 1, 1), (2, 17, 33), (1, 6912, 2560), (3, 100, 513), (8, 640, 2560), (15, 333, 1000),
            (16, 2560, 6912), (17, 64, 128), (31, 50, 640), (33, 1003, 777), (48, 48, 4096), (64, 2560, 2560),
            (65, 96, 256), (100, 1000, 1500), (128, 256, 512), (200, 130, 2570), (257, 515, 1029), (300, 1024, 2048)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS + [(520, 300, 640), (2100, 4000, 390), (513, 130, 129), (1000, 257, 2000),
                                              (1500, 600, 390), (1030, 2000, 1930), (4100, 130, 3000)])
def test_forward(m, n, k, dtype):
    print(f"case: forward_mxfp4 M={m} N={n} K={k} {dtype}", flush=True)
    x, w = outliers(m, k, seed=m + 1, dtype=DT[dtype]), outliers(n, k, seed=n + 2) * 0.02
    xc, xs, xv = quantized(x)
    wc, ws, wv = quantized(w)
    y = torch.full((m + 2, n), 777.0, dtype=DT[dtype], device=DEV)
    bl.forward_mxfp4(wc, ws, xc, xs, m, n, k, y=y[:m])
    check_product(y[:m], xv, wv, k)
    assert (y[m:] == 777.0).all()  # rows behind the last token are left alone
    f = bl.forward_mxfp4_fused(wc, ws, x, n, k, out_dtype=DT[dtype])
    check_product(f, xv, wv, k)
    again = bl.forward_mxfp4_fused(wc, ws, x, n, k, out_dtype=DT[dtype])
    assert torch.equal(f, again)


def grid_matrix(r, k, seed, shift=0):
    """Values on the grid times 2^shift, a 4 or a 6 in every block: quantised without error."""
    g = np.random.default_rng(seed)
    v = g.choice(ref.GRID, size=(r, k)) * g.choice([-1.0, 1.0], size=(r, k))
    v[:, ::32] = g.choice([4.0, -6.0], size=v[:, ::32].shape)
    return torch.from_numpy((v * 2.0 ** shift).astype(np.float32)).to(DEV)


@pytest.mark.parametrize("m,n,k", PRODUCTS + [(5, 40, 28672), (70, 90, 28672), (150, 70, 4100)]
                         + [v[0] for v in VARIANTS])
def test_forward_exact_sums(m, n, k):
    """All scales equal and every partial sum a multiple of 1/4 below 2^22: the product is exact, so
    any wrong element, scale or index shows."""
    print(f"case: forward_mxfp4 exact M={m} N={n} K={k}", flush=True)
    x, w = grid_matrix(m, k, m), grid_matrix(n, k, n + 1, shift=-5)
    wc, ws = bl.quantize_mxfp4(w)
    xc, xs = bl.quantize_mxfp4(x)
    want = host(x).astype(np.float64) @ host(w).astype(np.float64).T
    check_equal(host(bl.forward_mxfp4(wc, ws, xc, xs, m, n, k)).astype(np.float64), want, "y")
    check_equal(host(bl.forward_mxfp4_fused(wc, ws, x, n, k)).astype(np.float64), want, "fused y")
    xb = x.to(torch.bfloat16)  # grid values are bf16 numbers
    check_equal(host(bl.forward_mxfp4_fused(wc, ws, xb, n, k)).astype(np.float64), want, "fused bf16 y")


@pytest.mark.parametrize("n,outputs", [(260, 128), (2300, 256)])
def test_forward_every_step_count(n, outputs):
    """The GEMM's pipeline from one step of 128 columns to ten: exact sums, as above, against products in
    64 bits on the GPU."""
    m = 4100
    x, w = grid_matrix(m, 1280, 3), grid_matrix(n, 1280, 4, shift=-5)
    for k in range(128, 1281, 128):
        print(f"case: forward_mxfp4 M={m} N={n} K={k}", flush=True)
        p = bl.forward_mxfp4_plan(m, n, k)
        assert p["kernel"] == "gemm" and p["outputs"] == outputs
        xk, wk = x[:, :k].contiguous(), w[:, :k].contiguous()
        y = bl.forward_mxfp4(*bl.quantize_mxfp4(wk), *bl.quantize_mxfp4(xk), m, n, k)
        assert torch.equal(y.double(), xk.double() @ wk.double().t().contiguous())


@pytest.mark.parametrize("m", [1, 7, 16, 20, 64, 130, 520, 4100])
def test_forward_block_scales(m):
    """One block per row pair at its own power of two: each output is one product of scales."""
    k, n = 640, 48
    x = torch.zeros((m, k), device=DEV)
    w = torch.zeros((n, k), device=DEV)
    for i in range(m):
        x[i, 32 * (i % 20):32 * (i % 20) + 32] = 2.0 ** (i % 60 - 30)
    for j in range(n):
        w[j] = torch.tensor([2.0 ** ((j + b) % 40 - 20) for b in range(20)], device=DEV).repeat_interleave(32)
    wc, ws = bl.quantize_mxfp4(w)
    want = host(x).astype(np.float64) @ host(w).astype(np.float64).T
    check_equal(host(bl.forward_mxfp4_fused(wc, ws, x, n, k)).astype(np.float64), want, "y")


@pytest.mark.parametrize("m", [1, 4, 16, 40, 100, 200, 520, 4100])
def test_forward_nonfinite(m):
    """A NaN or an infinity spoils its token's row of the output, or its weight's column, and
    nothing else."""
    n, k = 70, 600
    x, w = grid_matrix(m, k, 5), grid_matrix(n, k, 6)
    clean = bl.forward_mxfp4_fused(*bl.quantize_mxfp4(w), x, n, k)
    x[m - 1, 599] = float("inf")
    w[33, 64] = float("nan")
    wc, ws = bl.quantize_mxfp4(w)
    for y in (bl.forward_mxfp4_fused(wc, ws, x, n, k), bl.forward_mxfp4(wc, ws, *bl.quantize_mxfp4(x), m, n, k)):
        bad = torch.zeros((m, n), dtype=torch.bool, device=DEV)
        bad[m - 1], bad[:, 33] = True, True
        assert torch.equal(torch.isnan(y), bad)
        assert torch.equal(y[~bad], clean[~bad])


def test_forward_zero_rows_and_large_scales():
    """All-zero tokens give zeros; scales at both ends of their range cancel."""
    n, k = 33, 256
    w = torch.full((n, k), 2.0 ** -100, device=DEV)
    x = torch.zeros((3, k), device=DEV)
    x[1] = 2.0 ** 100
    x[2] = -(2.0 ** 90)
    y = host(bl.forward_mxfp4_fused(*bl.quantize_mxfp4(w), x, n, k))
    assert (y[0] == 0).all() and (y[1] == k).all() and (y[2] == -k / 1024).all()


def test_forward_argument_errors():
    w, x = torch.randn(32, 256, device=DEV), torch.randn(4, 256, device=DEV)
    wc, ws = bl.quantize_mxfp4(w)
    xc, xs = bl.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        bl.forward_mxfp4(wc[:-1], ws, xc, xs, 4, 32, 256)
    with pytest.raises(ValueError):
        bl.forward_mxfp4(wc, ws, xc, xs, 17, 32, 256)
    with pytest.raises(ValueError):
        bl.forward_mxfp4(wc, ws, xc, xs, 4, 32, 256, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        bl.forward_mxfp4(wc, ws, xc, xs, 4, 32, 256, y=torch.empty(4, 33, device=DEV))
    with pytest.raises(ValueError):
        bl.forward_mxfp4_fused(wc, ws, x.half(), 32, 256)
    with pytest.raises(ValueError):
        bl.forward_mxfp4_fused(wc, ws, x.t(), 32, 4)
    with pytest.raises(ValueError):
        bl.forward_mxfp4_fused(wc, ws, x, 32, 255)
    with pytest.raises(ValueError):
        bl.quantize_mxfp4(x[:, ::2])
    with pytest.raises(ValueError):
        bl.quantize_mxfp4(x[:0])
    with pytest.raises(bl.BitLinearError):
        bl.forward_mxfp4(wc, ws, xc, xs, 0, 32, 256)
    with pytest.raises(ValueError):  # a workspace that is too small
        bl.forward_mxfp4_fused(wc, ws, torch.randn(700, 256, device=DEV), 32, 256,
                               workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_forward_offsets_past_32_bits():
    """An output of more than 2^32 elements (8.6 GB) and an input of as many: rows at both ends
    against the same rows computed alone."""
    m, n, k = 65600, 65552, 64
    x, w = grid_matrix(m, k, 1), grid_matrix(n, k, 2)
    wc, ws = bl.quantize_mxfp4(w)
    y = bl.forward_mxfp4_fused(wc, ws, x, n, k, out_dtype=torch.bfloat16)
    for lo in (0, 32768, m - 40):
        want = bl.forward_mxfp4_fused(wc, ws, x[lo:lo + 40].contiguous(), n, k, out_dtype=torch.bfloat16)
        assert torch.equal(y[lo:lo + 40], want)
    del y, want
    r, k = 262200, 16400
    x = torch.zeros((r, k), dtype=torch.bfloat16, device=DEV)
    tail = outliers(37, k, seed=8, dtype=torch.bfloat16)
    x[r - 37:] = tail
    codes, scales, values = bl.quantize_mxfp4(x, want_values=True)
    q, s, v = ref.quantize(acts_host_f32(tail))
    check_equal(acts_host_f32(values[r - 37:]).astype(np.float64), v, "values")
    # the last 8 rows start a row block: r = 16 * 16387 + 8
    want, wsc = ref.pack(q[-8:], s[-8:], k)
    check_equal(host(codes[-want.size:]), want, "codes")
    check_equal(host(scales[-wsc.size:]), wsc, "scales")


@pytest.mark.parametrize("m,n", [(20, 262192), (600, 262192), (262192, 48)])
def test_forward_codes_past_32_bits(m, n):
    """Codes of more than 2^32 bytes (random grid values, all scales 1, so that sums are exact): both ends
    of the long matrix against products of its slices."""
    k, edge = 32768, 96
    print(f"case: forward_mxfp4 M={m} N={n} K={k}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(m)

    def matrix(rows):
        codes = torch.randint(0, 256, (bl.mxfp4_codes_bytes(rows, k),), generator=g, dtype=torch.uint8, device=DEV)
        return codes, torch.full((bl.mxfp4_scales_bytes(rows, k),), 127, dtype=torch.uint8, device=DEV)

    w, x = matrix(n), matrix(m)
    assert max(w[0].numel(), x[0].numel()) > 1 << 32
    y = bl.forward_mxfp4(*w, *x, m, n, k)
    cb, sb = bl.mxfp4_codes_bytes(edge, k), bl.mxfp4_scales_bytes(edge, k)
    ends = [(slice(0, cb), slice(0, sb), slice(0, edge)), (slice(-cb, None), slice(-sb, None), slice(-edge, None))]
    for c, sc, rows in ends:
        if n > m:
            assert torch.equal(y[:, rows], bl.forward_mxfp4(w[0][c], w[1][sc], *x, m, edge, k))
        else:
            assert torch.equal(y[rows], bl.forward_mxfp4(*w, x[0][c], x[1][sc], edge, n, k))


def test_largest_k():
    """The longest rows the calls take, one token (the quantiser, then the decode kernel)."""
    n, k = 3, 1 << 24
    w, x = torch.full((n, k), 2.0 ** -12, device=DEV), torch.full((1, k), 0.5, device=DEV)
    x[0, 1::2] = 1.0
    y = bl.forward_mxfp4_fused(*bl.quantize_mxfp4(w), x, n, k)
    assert (y == k * 0.75 * 2.0 ** -12).all()


def test_graph_replays_and_streams():
    """The products and the quantiser captured into a graph on a side stream, replayed with new
    inputs and eager work between, and two streams at once, against eager results."""
    shapes = [(1, 300, 2560), (16, 128, 6912), (16, 64, 8704), (40, 500, 1000), (600, 600, 1500), (700, 2500, 1000),
              (1030, 2000, 1930)]
    w = [grid_matrix(n, k, i, shift=-3) for i, (m, n, k) in enumerate(shapes)]
    wq = [bl.quantize_mxfp4(t) for t in w]
    xs = [outliers(m, k, seed=i, dtype=torch.bfloat16) for i, (m, n, k) in enumerate(shapes)]

    def run():
        out = []
        for (m, n, k), (c, s), x in zip(shapes, wq, xs):
            out.append(bl.forward_mxfp4_fused(c, s, x, n, k))
            out.append(bl.forward_mxfp4(c, s, *bl.quantize_mxfp4(x), m, n, k, out_dtype=torch.bfloat16))
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = run()
    for turn in range(3):
        for i, x in enumerate(xs):
            x.copy_(outliers(*x.shape, seed=100 * turn + i, dtype=torch.bfloat16))
        g.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), turn
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            both.append([run() for _ in range(3)])
    torch.cuda.synchronize()
    for runs in both:
        for out in runs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_workspace_of_the_caller():
    """A given workspace is used whatever it holds, and one serves calls of several shapes."""
    shapes = [(20, 48, 640), (16, 40, 28672), (530, 200, 513)]
    need = max(bl.forward_mxfp4_fused_ws_bytes(m, n, k, "f32") for m, n, k in shapes)
    assert need > 0 and bl.forward_mxfp4_fused_ws_bytes(1, 64, 2560) == 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    for m, n, k in shapes:
        w, x = bl.quantize_mxfp4(grid_matrix(n, k, 3)), outliers(m, k, seed=m)
        assert torch.equal(bl.forward_mxfp4_fused(*w, x, n, k, workspace=ws), bl.forward_mxfp4_fused(*w, x, n, k))


@pytest.mark.parametrize("tokens", [1, 5, 16, 50, 300, 700])
def test_norm_quantise_product_together(tokens):
    """A layer as it would be used: layer norm, its output quantised once for two projections, squared
    ReLU gating, and the down projection from the un-quantised hidden rows; against 64 bits on the
    values that each quantiser saw."""
    d, h = 640, 1111
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    x = torch.randn((tokens, d), generator=g, device=DEV).to(torch.bfloat16)
    gain, bias = 1 + 0.1 * torch.randn(d, generator=g, device=DEV), 0.1 * torch.randn(d, generator=g, device=DEV)
    wg, wu, wd = (torch.randn(s, generator=g, device=DEV) * 0.05 for s in ((h, d), (h, d), (d, h)))
    (gc, gs), (uc, us), (dc, ds) = (bl.quantize_mxfp4(w) for w in (wg, wu, wd))
    y, mean, rstd = bl.layernorm(x, gain, bias)
    yc, ys = bl.quantize_mxfp4(y)
    gate = bl.forward_mxfp4(gc, gs, yc, ys, tokens, h, d)
    up = bl.forward_mxfp4(uc, us, yc, ys, tokens, h, d)
    hidden = torch.relu(gate) ** 2 * up
    out = bl.forward_mxfp4_fused(dc, ds, hidden, d, h)
    wy = ref.layernorm(acts_host_f32(x), host(gain), host(bias), 1e-5)[0]
    assert np.abs(acts_host_f32(y) - wy).max() <= 2.0 ** -8 * np.abs(wy).max() + 1e-4
    yv = ref.quantize(acts_host_f32(y))[2]
    check_product(gate, yv, ref.quantize(host(wg))[2], d)
    check_product(up, yv, ref.quantize(host(wu))[2], d)
    check_product(out, ref.quantize(host(hidden))[2], ref.quantize(host(wd))[2], h)


def test_host_threads_with_different_lds():
    """Host threads that call at once, each on a stream of its own, with sizes of the one-launch kernel that
    take different amounts of LDS above 64 KiB."""
    n, calls = 64, 150
    cases = []
    assert bl.forward_mxfp4_plan(8, n, 8704, x="f32")["launches"] == 1
    for i, (m, k) in enumerate([(16, 14848), (16, 8704), (8, 8704), (16, 8200)]):
        assert bl.forward_mxfp4_plan(m, n, k)["kernel"] == "lds"
        x, w = grid_matrix(m, k, i), grid_matrix(n, k, i + 9, shift=-5)
        cases.append((m, k, x, bl.quantize_mxfp4(w), bl.quantize_mxfp4(x), x.double() @ w.double().t().contiguous()))
    torch.cuda.synchronize()
    failures = []

    def work(i):
        m, k, x, wq, xq, want = cases[i]
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out = [bl.forward_mxfp4(*wq, *xq, m, n, k) for _ in range(calls)]
                if m == 8:
                    out += [bl.forward_mxfp4_fused(*wq, x, n, k) for _ in range(calls)]
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(y.double(), want) for y in out):
                failures.append((i, "wrong"))
        except Exception as e:  # reported by the main thread
            failures.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", sorted({shape for _, shape in FORMS} | {v[0] for v in VARIANTS}))
def test_forward_exact_sums_of_every_form(m, n, k, out):
    """Exact sums, as above, in every form of the kernels and in both output types (bf16: the exact sum,
    an fp32 number, rounded once); rows behind the last token are left alone."""
    print(f"case: forward_mxfp4 form M={m} N={n} K={k} -> {out}", flush=True)
    x, w = grid_matrix(m, k, m + 3), grid_matrix(n, k, n + 4, shift=-5)
    wq, xq = bl.quantize_mxfp4(w), bl.quantize_mxfp4(x)
    want = torch.from_numpy(host(x).astype(np.float64) @ host(w).astype(np.float64).T).float().to(DT[out])
    for call in (lambda y: bl.forward_mxfp4(*wq, *xq, m, n, k, y=y), lambda y: bl.forward_mxfp4_fused(*wq, x, n, k, y=y),
                 lambda y: bl.forward_mxfp4_fused(*wq, x.to(torch.bfloat16), n, k, y=y)):
        y = torch.full((m + 1, n), 777.0, dtype=DT[out], device=DEV)
        call(y[:m])
        check_equal(acts_host_f32(y[:m]), acts_host_f32(want), "y")
        assert (y[m:] == 777.0).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", sorted({shape for _, shape in FORMS}) + [(2304, 2560, 512), (1, 6912, 2560)])
def test_forward_unaligned_rows(m, n, k, out):
    """x and y that start at an odd element of their storage: exact sums, as above, and nothing written before
    or behind y."""
    print(f"case: forward_mxfp4 unaligned M={m} N={n} K={k} -> {out}", flush=True)
    x, w = grid_matrix(m, k, m + 5), grid_matrix(n, k, n + 6, shift=-5)
    wq = bl.quantize_mxfp4(w)
    want = torch.from_numpy(host(x).astype(np.float64) @ host(w).astype(np.float64).T).float().to(DT[out])
    for dtype in ("f32", "bf16"):
        flat = torch.empty(1 + m * k, dtype=DT[dtype], device=DEV)
        flat[1:] = x.to(DT[dtype]).reshape(-1)
        y = torch.full((m * n + 2,), 777.0, dtype=DT[out], device=DEV)
        bl.forward_mxfp4_fused(*wq, flat[1:].view(m, k), n, k, y=y[1:-1].view(m, n))
        check_equal(acts_host_f32(y[1:-1].view(m, n)), acts_host_f32(want), "y")
        assert (y[[0, -1]] == 777.0).all()
