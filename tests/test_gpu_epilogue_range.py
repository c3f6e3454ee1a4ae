"""Activations of products over the whole range of their argument, in every kernel: tokens of zeros leave the bias, a
number of fp32, as the exact argument."""
import pytest
import torch

import bitlinear_fwd_amd as bl
import experts_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
# kernel of the plan: tokens, columns, x of zeros or codes of zeros
FORMS = {"fused": (2, 264, "bf16"), "decode": (16, 300, None), "gemm": (1500, 300, None)}


def activated(form, bias, act, dtype):
    """act(bias) [N], as the form's kernel gives it for every token (all the same)."""
    m, k, x = FORMS[form]
    n = len(bias)
    assert bl.forward_epilogue_plan(m, n, k, x)["kernel"] == form
    packed = ref.pack(ref.random_codes(n, k, torch.Generator().manual_seed(n))).to(DEV)
    gamma = torch.full((1,), 0.02, device=DEV)
    if x is None:
        xs, absmax = torch.zeros(m, (k + 255) // 256 * 256, dtype=torch.int8, device=DEV), torch.zeros(m, device=DEV)
    else:
        xs, absmax = torch.zeros(m, k, dtype=BF16, device=DEV), None
    y = bl.forward_epilogue(packed, gamma, xs, n, k, absmax=absmax, bias=bias.to(DEV), act=act, out_dtype=dtype)
    assert torch.equal(y.isnan(), y[:1].isnan().expand(m, n))
    assert torch.equal(y.nan_to_num(), y[:1].nan_to_num().expand(m, n))
    return y[0].cpu()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_sigmoid_forms_go_to_zero(form, act, dtype):
    """v times a sigmoid: 0 far to the left, v far to the right, and every order of magnitude between.  Roundings as
    ref.act counts them; e^x is 0 where fp32 has it below its normal numbers, of which |v| < 104 makes 104 2^-126."""
    size = torch.logspace(-3, 38.5, 500, dtype=torch.float64).float()
    v = torch.cat((-size, size, -torch.linspace(80, 110, 301), torch.tensor([0.0, -0.0, -3.4028234663852886e38])))
    y = activated(form, v, act, dtype)
    d = v.double()
    exact, err = ref.act(d, torch.zeros_like(d), act)
    # 2^t to an argument t of 87 at most: further left nothing is left of v e^t
    if act == "gelu_tanh":
        t = 1.5957691216057308 * (d + 0.044715 * d ** 3)
        exact = torch.where(t < -120, torch.zeros_like(d), exact)
        err = (10 + 6 * t.abs().clamp(max=120)) * ref.U * exact.abs()
    err = err + 104 * 2.0 ** -126
    ref.check(y, exact, err + (dtype == BF16) * ref.STEP[BF16] * (exact.abs() + err), f"{form} {act}")
    assert (y[v < -110].double() == 0).all()


def gelu(d):
    return 0.5 * d * torch.erfc(-d / 2 ** 0.5)


FAR = torch.logspace(-30, 38.5, 200, dtype=torch.float64).float()
GELU_ARGS = torch.cat((torch.linspace(-16, 16, 3001), FAR, -FAR, torch.tensor([1.25, -1.25, 0.0])))


@pytest.mark.parametrize("form", FORMS)
def test_gelu_in_fp32(form):
    """On the left relative to the result: t = 1 / (1 + 0.35 a) to 3 half steps, which the result follows at most
    twice; the polynomial's fit and last steps 2; the exponential 2, and its argument a^2 / 2 to 2; three products: 13 + a^2.
    On the right h, at most 0.106 |v| where it is taken, to 15 there, and the difference; below 1.25 Phi(v) - 1/2, at
    most 0.4, to 2.5, the sum and the product: 3 of |v|.  Results below fp32's normal numbers may be 0."""
    v = GELU_ARGS
    y = activated(form, v, "gelu", F32).double()
    d = v.double()
    exact = gelu(d)
    left = (13 + d.clamp(min=-16) ** 2) * ref.U * exact.abs() + 16 * 2.0 ** -126
    err = torch.where(d < 0, left, 3 * ref.U * d)
    ref.check(y, exact, err, form)
    assert (y[d < -1e-30] <= 0).all() and (y[(d < -1e-30) & (d > -12)] < 0).all()


@pytest.mark.parametrize("form", FORMS)
def test_gelu_in_bf16(form):
    """Half a step of bf16 of the result and what the short form adds, all of it relative to the result: 16 half steps
    of fp32, and the exponent's a^2 / 2 to 2 of them."""
    v = GELU_ARGS
    y = activated(form, v, "gelu", BF16)
    d = v.double()
    exact = gelu(d)
    short = (16 + d.abs().clamp(max=16) ** 2) * ref.U * exact.abs() + 16 * 2.0 ** -126
    ref.check(y, exact, short + ref.STEP[BF16] * (exact.abs() + short), form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", ["relu2", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_plus_infinity(form, act, dtype):
    """A sum that overflows fp32 stays infinite."""
    y = activated(form, torch.tensor([float("inf")] + [1.0] * 1303), act, dtype)
    assert y[0] == float("inf") and y[1:].isfinite().all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", list(bl.ACTIVATIONS))
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_nan_stays_nan(form, act, dtype):
    y = activated(form, torch.tensor([float("nan"), -float("nan"), -1.0] + [1.0] * 1301), act, dtype)
    assert y[:2].isnan().all() and y[2:].isfinite().all()


@pytest.mark.parametrize("m,n,k,x", [(1, 700, 1280, BF16), (2, 40, 264, F32), (4, 301, 2568, F32), (4, 301, 2568, BF16),
                                     (3, 40, 256, BF16), (2, 64, 20000, F32), (1, 64, 40000, BF16)], ids=str)
def test_rows_with_nan_or_infinity(m, n, k, x):
    """The quantiser within the kernel passes over NaN and takes infinities as the one in a launch of its own does: the
    same outputs as from its codes and scales."""
    g = torch.Generator().manual_seed(k)
    assert bl.forward_epilogue_plan(m, n, k, "bf16" if x == BF16 else "f32")["kernel"] == "fused"
    packed = ref.pack(ref.random_codes(n, k, g)).to(DEV)
    gamma = torch.full((1,), 0.02, device=DEV)
    nan, inf = float("nan"), float("inf")
    at = [0, k // 2, k - 1]
    for places in ([(0, nan)], [(0, nan), (1, -nan), (2, nan)], [(1, inf)], [(2, -inf), (0, nan)], [(1, -nan)], "all"):
        xs = torch.randn(m, k, generator=g)
        for r in range(0, m, 2):  # every other row
            if places == "all":
                xs[r] = nan
            else:
                for i, v in places:
                    xs[r, at[i]] = v
        xs = xs.to(x).to(DEV)
        codes, absmax = bl.quantize_acts(xs)
        y = bl.forward_epilogue(packed, gamma, xs, n, k)
        z = bl.forward_epilogue(packed, gamma, codes, n, k, absmax=absmax)
        assert torch.equal(y.isnan(), z.isnan()) and torch.equal(y.nan_to_num(), z.nan_to_num()), places
