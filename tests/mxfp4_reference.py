"""Plain 64-bit forms of the MXFP4 format and of the layer norm for the tests, written from the
formulas of include/bitlinear.h (numpy on the host)."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes uint8 [R][K], scale bytes uint8 [R][ceil(K/32)], values float64 [R][K]) of x
    (any float values that fp32 holds), element by element from the definition."""
    x = np.asarray(x, dtype=np.float64)
    r, k = x.shape
    kb = -(-k // 32)
    codes = np.zeros((r, kb * 32), dtype=np.uint8)
    scales = np.zeros((r, kb), dtype=np.uint8)
    values = np.zeros((r, kb * 32))
    pad = np.zeros((r, kb * 32))
    pad[:, :k] = x
    blocks = pad.reshape(r, kb, 32)
    finite = np.isfinite(blocks).all(-1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(blocks), blocks, 0.0)).max(-1), 1.0)
    # exponent field of an fp32 magnitude: floor(log2) + 127, 0 below the smallest normal
    field = np.where(amax >= 2.0 ** -126, np.frexp(np.maximum(amax, 2.0 ** -126))[1] + 126, 0)
    e = np.maximum(field - 2, 0)
    a = np.ldexp(np.abs(np.where(finite[..., None], blocks, 0.0)), (127 - e)[..., None])
    # nearest grid magnitude; of two at the same distance the even index
    dist = np.abs(a[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    near = dist == best
    idx = np.where(near.sum(-1) == 1, near.argmax(-1), 0)
    even = (near & (np.arange(8) % 2 == 0)).argmax(-1)
    idx = np.where(near.sum(-1) == 2, even, idx)
    q = idx.astype(np.uint8) | (np.signbit(blocks).astype(np.uint8) << 3)
    v = np.copysign(np.ldexp(GRID[idx], (e - 127)[..., None]), blocks)
    q = np.where(finite[..., None], q, 0)
    v = np.where(finite[..., None], v, np.nan)
    codes[:] = q.reshape(r, kb * 32)
    values[:] = v.reshape(r, kb * 32)
    scales[:] = np.where(finite, e, 255)
    return codes[:, :k], scales, values[:, :k]


def pack(codes, scales, k):
    """The library's layout of codes [R][K] and scale bytes [R][ceil(K/32)], byte by byte."""
    r = codes.shape[0]
    tiles, groups, rbs = -(-k // 128), -(-k // 512), -(-r // 16)
    out = np.zeros(rbs * tiles * 1024, dtype=np.uint8)
    sc = np.zeros(rbs * groups * 256, dtype=np.uint8)
    rows, cols = np.meshgrid(np.arange(r), np.arange(k), indexing="ij")
    rb, rr, c, kk = rows // 16, rows % 16, cols // 128, cols % 128
    b, i = kk // 32, kk % 32
    addr = (rb * tiles + c) * 1024 + 16 * (16 * b + rr) + i // 2
    np.bitwise_or.at(out, addr.ravel(), (codes.astype(np.uint8) << (4 * (i % 2)).astype(np.uint8)).ravel())
    rows, blk = np.meshgrid(np.arange(r), np.arange(scales.shape[1]), indexing="ij")
    rb, rr, c, b = rows // 16, rows % 16, blk // 4, blk % 4
    sc[((rb * groups + c // 4) * 64 + 16 * b + rr) * 4 + c % 4] = scales
    return out, sc


def layernorm(x, w, b, eps):
    x = x.astype(np.float64)
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / np.sqrt((xc * xc).mean(1) + eps)
    y = xc * rstd[:, None]
    if w is not None:
        y = y * w.astype(np.float64)
    if b is not None:
        y = y + b.astype(np.float64)
    return y, mean, rstd


def layernorm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db) and the sums of magnitudes that their error bounds go by."""
    dy, x = dy.astype(np.float64), x.astype(np.float64)
    mean, rstd = mean.astype(np.float64)[:, None], rstd.astype(np.float64)[:, None]
    xhat = (x - mean) * rstd
    g = dy * (1.0 if w is None else w.astype(np.float64))
    c1, c2 = g.mean(1, keepdims=True), (g * xhat).mean(1, keepdims=True)
    dx = rstd * (g - c1 - xhat * c2)
    u = 2.0 ** -24
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    # row sums: at most 64 roundings on the way of any term; xhat: 3; the rest of the formula: 8
    dx_tol = rstd * (72 * u * (a1 + np.abs(xhat) * a2) + 8 * u * (np.abs(g) + np.abs(c1) + np.abs(xhat * c2)))
    # sums over the rows: a chain over a walker's rows, then over the partial rows
    n = -(-x.shape[0] // 64) + 140
    return (dx, (dy * xhat).sum(0), dy.sum(0), dx_tol, n * u * np.abs(dy * xhat).sum(0), n * u * np.abs(dy).sum(0))
