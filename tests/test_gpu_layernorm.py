"""Layer normalisation and its gradients on the GPU against the plain 64-bit forms."""
import numpy as np
import pytest
import torch

import bitlinear_fwd_amd as bl
import mxfp4_reference as ref
from gpu_helpers import acts_host_f32, host

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24

# one element, rows shared by a wave, by 256 and by 1024 threads, longer rows; odd sizes around each
SIZES = [(1, 1), (3, 7), (2, 8), (5, 64), (9, 513), (4, 2048), (3, 2049), (7, 2560), (6, 5000), (5, 8192), (2, 8193),
         (3, 28672), (2, 32768), (2, 32775), (1, 100003), (700, 40), (1030, 257), (530, 2560),
         # enough rows that a workgroup walks over several, in each form
         (9000, 100), (5300, 600), (1100, 1500), (1700, 2560), (1050, 5001), (1030, 8192), (300, 8000), (600, 12288),
         (300, 12289), (520, 20000)]


def data(m, k, dtype, seed, offset=0.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = (torch.randn((m, k), generator=g, device=DEV) * 2 + offset).to(DT[dtype])
    w = 1 + 0.2 * torch.randn(k, generator=g, device=DEV)
    b = 0.3 * torch.randn(k, generator=g, device=DEV)
    dy = torch.randn((m, k), generator=g, device=DEV).to(DT[dtype])
    return x, w, b, dy


def rounded(tol, want, dtype):
    """The bound with the one rounding to dtype on top."""
    return tol + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (np.abs(want) + tol)


def within(got, want, tol, what):
    bad = ~(np.abs(got.astype(np.float64) - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def check_forward(x, w, b, eps, dtype):
    m, k = x.shape
    y, mean, rstd = bl.layernorm(x, w, b, eps)
    xh = acts_host_f32(x).astype(np.float64)
    wh, bh = (None if w is None else host(w)), (None if b is None else host(b))
    wy, wm, wr = ref.layernorm(xh, wh, bh, eps)
    # a row sum: at most 64 roundings on the way of any term (32 in a thread, 6 in a wave, 16 over waves)
    d = 64 * U * np.abs(xh).mean(1)
    within(host(mean), wm, d + U * np.abs(wm), "mean")
    # the variance moves by d^2 for a mean off by d, and by its own sum's roundings
    rel = 0.5 * (72 * U + d * d * wr * wr) + 4 * U
    within(host(rstd), wr, rel * wr, "rstd")
    a = np.abs(wy - (0 if bh is None else bh))
    ww = 1.0 if wh is None else np.abs(wh)
    tol = ww * (wr * (d + U * np.abs(xh).max(1)))[:, None] * (1 + rel)[:, None] + a * (rel + 6 * U)[:, None]
    tol = tol + 2 * U * (a + (0 if bh is None else np.abs(bh)))
    within(acts_host_f32(y), wy, rounded(tol, wy, dtype), "y")
    return y, mean, rstd


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,k", SIZES)
def test_layernorm(m, k, dtype):
    print(f"case: layernorm M={m} K={k} {dtype}", flush=True)
    x, w, b, _ = data(m, k, dtype, seed=m + k)
    check_forward(x, w, b, 1e-5, dtype)
    check_forward(x, None, b, 1e-2, dtype)
    check_forward(x, w, None, 1e-5, dtype)
    check_forward(x, None, None, 1e-12, dtype)


@pytest.mark.parametrize("k", [33, 1000, 2560, 20000, 40000])
def test_layernorm_large_mean_and_constant_rows(k):
    """A mean a thousand times the spread; a constant row (variance 0); a zero row."""
    x, w, b, _ = data(6, k, "f32", seed=k, offset=2000.0)
    x[2] = 3.0
    x[3] = 0.0
    y, mean, rstd = check_forward(x, w, b, 1e-5, "f32")
    assert torch.equal(y[3], b) and float(mean[3]) == 0.0
    assert abs(float(rstd[3]) - 1e-5 ** -0.5) < 1e-4


def check_backward(dy, x, w, mean, rstd, dtype):
    dx, dw, db = bl.layernorm_backward(dy, x, w, mean, rstd)
    wx, ww, wb, tx, tw, tb = ref.layernorm_backward(acts_host_f32(dy), acts_host_f32(x), None if w is None else host(w),
                                                    host(mean), host(rstd))
    within(acts_host_f32(dx), wx, rounded(tx, wx, dtype), "dx")
    within(host(dw), ww, tw + U * np.abs(ww), "dweight")
    within(host(db), wb, tb + U * np.abs(wb), "dbias")
    return dx, dw, db


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,k", SIZES + [(3000, 72), (2050, 9000)])
def test_layernorm_backward(m, k, dtype):
    print(f"case: layernorm_backward M={m} K={k} {dtype}", flush=True)
    x, w, b, dy = data(m, k, dtype, seed=m + k)
    _, mean, rstd = bl.layernorm(x, w, b, 1e-5)
    dx, dw, db = check_backward(dy, x, w, mean, rstd, dtype)
    check_backward(dy, x, None, mean, rstd, dtype)
    only = bl.layernorm_backward(dy, x, w, mean, rstd, want_params=False)
    assert torch.equal(only, dx)
    again = bl.layernorm_backward(dy, x, w, mean, rstd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)


@pytest.mark.parametrize("m,k", [(5, 100), (40, 2560), (3, 9000), (70, 40000)])
def test_layernorm_backward_subsets(m, k):
    """Each output alone through the C ABI equals the same output of the full call, and the others
    are not written."""
    x, w, b, dy = data(m, k, "f32", seed=k)
    _, mean, rstd = bl.layernorm(x, w, b, 1e-5)
    full = bl.layernorm_backward(dy, x, w, mean, rstd)
    ws = torch.empty(bl.layernorm_backward_ws_bytes(m, k), dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    for i, shape in enumerate([(m, k), (k,), (k,)]):
        out = torch.full(shape, 5.0, device=DEV)
        ptr = [None, None, None]
        ptr[i] = out.data_ptr()
        st = bl.lib().bitlinear_layernorm_backward(dy.data_ptr(), x.data_ptr(), bl.BL_F32, m, k, w.data_ptr(),
                                                   mean.data_ptr(), rstd.data_ptr(), *ptr, ws.data_ptr(), ws.numel(), s)
        assert st == bl.BL_OK
        assert torch.equal(out, full[i])


@pytest.mark.parametrize("m,k", [(5, 100), (7, 3000), (3, 40000)])
def test_layernorm_without_statistics(m, k):
    """mean and rstd may be null, each by itself or both, and so may weight and bias."""
    x, w, b, _ = data(m, k, "bf16", seed=k)
    y, mean, rstd = bl.layernorm(x, w, b, 1e-5)
    s = torch.cuda.current_stream().cuda_stream
    for give in ((True, False), (False, True), (False, False)):
        out = torch.empty_like(x)
        stats = [torch.full((m,), 7.0, device=DEV) for _ in range(2)]
        st = bl.lib().bitlinear_layernorm(x.data_ptr(), bl.BL_BF16, m, k, w.data_ptr(), b.data_ptr(), 1e-5,
                                          out.data_ptr(), *(t.data_ptr() if g else None for t, g in zip(stats, give)), s)
        assert st == bl.BL_OK and torch.equal(out, y)
        for t, g, want in zip(stats, give, (mean, rstd)):
            assert torch.equal(t, want if g else torch.full_like(t, 7.0))


def test_layernorm_nonfinite_rows_stay_apart():
    for k in (100, 3000, 40000):
        x, w, b, dy = data(5, k, "f32", seed=k)
        clean, mean, rstd = bl.layernorm(x, w, b, 1e-5)
        gclean = bl.layernorm_backward(dy, x, w, mean, rstd, want_params=False)
        x[1, k - 1] = float("nan")
        x[3, 0] = float("inf")
        y, mean, rstd = bl.layernorm(x, w, b, 1e-5)
        dx = bl.layernorm_backward(dy, x, w, mean, rstd, want_params=False)
        for r in (0, 2, 4):
            assert torch.equal(y[r], clean[r]) and torch.equal(dx[r], gclean[r])
        assert torch.isnan(y[1]).all() and torch.isnan(dx[1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layernorm_unaligned_rows(dtype):
    """Rows that start at odd elements: an odd row length in storage that starts one element in."""
    m, k = 9, 2563
    x, w, b, dy = data(m, k, dtype, seed=4)

    def moved(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    y, mean, rstd = check_forward(moved(x), moved(w), moved(b), 1e-5, dtype)
    check_backward(moved(dy), moved(x), moved(w), moved(mean), moved(rstd), dtype)


def test_layernorm_argument_errors():
    x, w, b, dy = data(4, 64, "f32", seed=1)
    _, mean, rstd = bl.layernorm(x, w, b)
    for bad in (lambda: bl.layernorm(x.half(), w, b), lambda: bl.layernorm(x.t(), None, None),
                lambda: bl.layernorm(x, w[:-1], b), lambda: bl.layernorm(x, w.bfloat16(), b),
                lambda: bl.layernorm(x, w, b, y=torch.empty(4, 63, device=DEV)),
                lambda: bl.layernorm(x[:0], w, b),
                lambda: bl.layernorm_backward(dy.bfloat16(), x, w, mean, rstd),
                lambda: bl.layernorm_backward(dy[:3], x, w, mean, rstd),
                lambda: bl.layernorm_backward(dy, x, w, None, rstd),
                lambda: bl.layernorm_backward(dy, x, w, mean[:3], rstd),
                lambda: bl.layernorm_backward(dy, x, w, mean, rstd,
                                              workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bl.BitLinearError):
        bl.layernorm(x, w, b, eps=0.0)


def test_layernorm_offsets_past_32_bits():
    """More than 2^32 elements (8.6 GB each way): the last rows against the same rows alone."""
    m, k = 262145, 16400
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    tail, w, b, dy = data(5, k, "bf16", seed=2)
    x[m - 5:] = tail
    y, mean, rstd = bl.layernorm(x, w, b)
    ty, tm, tr = bl.layernorm(tail, w, b)
    assert torch.equal(y[m - 5:], ty) and torch.equal(mean[m - 5:], tm) and torch.equal(rstd[m - 5:], tr)
    assert torch.equal(y[0], b.to(torch.bfloat16)) and float(mean[7]) == 0.0
    y.zero_()
    y[m - 5:] = dy  # as the gradient: zeros but for the last rows
    dx, dw, db = bl.layernorm_backward(y, x, w, mean, rstd)
    tx, tw, tb = bl.layernorm_backward(dy, tail, w, tm, tr)
    assert torch.equal(dx[m - 5:], tx) and not dx[:7].any()
    torch.testing.assert_close(dw, tw, rtol=0, atol=8 * U * float((dy.float().abs() * 5).sum(0).max()))
    torch.testing.assert_close(db, tb, rtol=0, atol=8 * U * float(dy.float().abs().sum(0).max()))


def test_layernorm_graph_replays_and_streams():
    """Forward and backward captured into a graph on a side stream, replayed with new inputs and eager
    work between; then on two streams at once."""
    sizes = [(5, 100, "f32"), (300, 2560, "bf16"), (40, 9000, "f32"), (3, 40000, "bf16")]
    ins = [data(m, k, dt, seed=i) for i, (m, k, dt) in enumerate(sizes)]

    def run():
        out = []
        for x, w, b, dy in ins:
            y, mean, rstd = bl.layernorm(x, w, b)
            out += [y, mean, rstd, *bl.layernorm_backward(dy, x, w, mean, rstd)]
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
        for i, (m, k, dt) in enumerate(sizes):
            for t, new in zip(ins[i], data(m, k, dt, seed=10 * turn + i + 50)):
                t.copy_(new)
        g.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), turn
    streams, both = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            both.append([run() for _ in range(3)])
    torch.cuda.synchronize()
    for runs in both:
        for out in runs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_layernorm_gradients_against_differences():
    """dx, dweight and dbias along random directions against central differences of the kernel's own
    forward pass.  With |r|, |v| <= 1 and rows of 64 values of unit spread the loss is a few tens, its
    fp32 error about 64 * 6 * 64 * U ~ 1.5e-3 in the worst case; at a step of 0.05 that is 0.03 in the
    difference, and the third derivative adds 0.05^2 / 6 of a few tens ~ 0.02."""
    m, k, step = 6, 64, 0.05
    x, w, b, _ = data(m, k, "f32", seed=3)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    r = torch.rand((m, k), generator=g, device=DEV) * 2 - 1

    def loss(x, w, b):
        return float((bl.layernorm(x, w, b)[0].double() * r.double()).sum())

    _, mean, rstd = bl.layernorm(x, w, b)
    for i, grad in enumerate(bl.layernorm_backward(r, x, w, mean, rstd)):
        args = [x, w, b]
        v = torch.rand(args[i].shape, generator=g, device=DEV) * 2 - 1
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * v, args[i] - step * v
        slope = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(slope - float((grad.double() * v.double()).sum())) <= 0.06, i


# (M, K) that reach each form of the forward pass: rows of a wave with one and with two groups a thread,
# of a workgroup with one, two and four, and the long form; each with a row that fills no whole group, and
# with one of whole runs of four columns
FORWARD_FORMS = [(9, 1), (9, 4), (9, 33), (9, 500), (9, 509), (9, 514), (9, 1000), (9, 1023), (9, 1025), (9, 2560),
                 (9, 8191), (1030, 2560), (1030, 2561), (9, 10000), (9, 16383), (9, 20000), (9, 20001), (9, 32767),
                 (9, 32768), (9, 40001)]


def check_forward_near(x, w, b, eps, dtype):
    """check_forward with bounds that go by the distances |x - mean| and not by the mean.  With p an element of the
    row and r the largest |x - mean|, |x - p| <= |x - mean| + r:
    * x - p is off by U (|x - mean| + r), and its mean by 72 U of the mean of that (that rounding, 64 of the sum, those
      of p differing between waves, the division); the returned mean is rounded once more.
    * Of the squares, the common part of these errors enters squared and the rounding of each x - p by twice its product
      with x - mean, together at most 4 U (1 + r rstd) of the variance and eps (the mean of |x - mean| is below 1 / rstd);
      their sum and rstd are rounded as in check_forward."""
    y, mean, rstd = bl.layernorm(x, w, b, eps)
    xh = acts_host_f32(x).astype(np.float64)
    wh, bh = host(w).astype(np.float64), host(b).astype(np.float64)
    wy, wm, wr = ref.layernorm(xh, wh, bh, eps)
    dist = np.abs(xh - wm[:, None])
    r = dist.max(1)
    off = 72 * U * (dist.mean(1) + r) + 2.0 ** -50 * np.abs(xh).mean(1)  # (the last: the plain form's own)
    within(host(mean), wm, off + U * np.abs(wm), "mean")
    rel = 0.5 * (72 * U + 4 * U * (1 + r * wr) + (off * wr) ** 2) + 4 * U
    within(host(rstd), wr, rel * wr, "rstd")
    a = dist * wr[:, None] * np.abs(wh)
    moved = (U * (2 * dist + r[:, None]) + off[:, None]) * wr[:, None] * np.abs(wh)
    tol = moved * (1 + rel)[:, None] + a * (rel + 6 * U)[:, None] + 2 * U * (a + np.abs(bh))
    within(acts_host_f32(y), wy, rounded(tol, wy, dtype), "y")
    return y, mean, rstd


@pytest.mark.parametrize("m,k", FORWARD_FORMS)
def test_layernorm_constant_rows(m, k):
    """Rows of one value, large against eps and not a number whose sums are exact in fp32: the variance
    is 0, so y is the bias, rstd that of eps alone, and the mean the value itself."""
    print(f"case: layernorm constant rows M={m} K={k}", flush=True)
    values = [12345.678, 100000.3, -54321.1, 1e7 + 1, 1e-3 / 3, 123456792.0, -3.3, 7.0, 0.1]
    _, w, b, _ = data(1, k, "f32", seed=k)
    for dtype in ("f32", "bf16"):
        x = torch.tensor([values[i % 9] for i in range(m)], device=DEV).to(DT[dtype])[:, None].repeat(1, k)
        for eps in (1e-5, 1e-12):
            y, mean, rstd = check_forward_near(x, w, b, eps, dtype)
            assert torch.equal(mean, x[:, 0].float())
            assert torch.equal(y, b.to(DT[dtype]).repeat(m, 1))
            assert bool(((rstd.double() * eps ** 0.5 - 1).abs() <= 4 * U).all())


@pytest.mark.parametrize("m,k", FORWARD_FORMS)
def test_layernorm_small_spread_about_a_large_mean(m, k):
    """Rows of 1000 +- 0.01, 100000 +- 0.5 and -30000 +- 100: the result goes by the spread."""
    print(f"case: layernorm small spread M={m} K={k}", flush=True)
    z, w, b, _ = data(m, k, "f32", seed=k, offset=0.0)
    rows = torch.arange(m, device=DEV)[:, None] % 3
    centre = torch.tensor([1000.0, 100000.0, -30000.0], device=DEV)[rows]
    spread = torch.tensor([0.005, 0.25, 50.0], device=DEV)[rows]
    x = centre + spread * z
    for eps in (1e-5, 1e-12):
        check_forward_near(x, w, b, eps, "f32")
    check_forward_near((centre + 30 * spread * z).to(torch.bfloat16), w, b, 1e-5, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,k", [(4, 33), (4, 500), (20, 514), (4, 1000), (4, 2561), (4, 8190), (4, 9000), (4, 12288),
                                 (4, 12290), (3, 40001)])
def test_layernorm_backward_of_large_constant_rows(m, k, dtype):
    """A row of one value whose mean * rstd is beyond fp32: x - mean is 0, so dx is rstd (g - mean(g)), and the columns
    between the row's end and the threads' must not get in the way."""
    print(f"case: layernorm_backward large constant row M={m} K={k} {dtype}", flush=True)
    x, w, b, dy = data(m, k, dtype, seed=k)
    x[1] = 2.5e37
    x[m - 1] = -3e37
    _, mean, rstd = bl.layernorm(x, w, b, 1e-5)
    assert torch.equal(mean[1], x[1, 0].float()) and abs(float(rstd[1]) * 1e-5 ** 0.5 - 1) < 1e-6
    dx, dw, db = check_backward(dy, x, w, mean, rstd, dtype)
    assert torch.isfinite(dx).all()
    assert torch.equal(bl.layernorm_backward(dy, x, w, mean, rstd, want_params=False), dx)
