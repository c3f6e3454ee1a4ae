"""The GEMM's tiles of 32 slots x 256 outputs: long sums (every stage of the ring many times), rows and columns that end
inside a tile, and experts of ragged sizes."""
import pytest
import torch

import bitlinear_fwd_amd as bl
import experts_reference as ref
from test_gpu_epilogue import codes_of, exact_on_gpu, make
from test_gpu_experts import Layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
TILE = ("gemm", 32, 256)


def tile(plan):
    return plan["kernel"], plan["rows"], plan["outputs"]


@pytest.mark.parametrize("m,n,k", [(65, 19498, 300), (326, 11239, 2015), (198, 17013, 2205), (1500, 1000, 512)])
def test_one_matrix(m, n, k):
    assert tile(bl.forward_epilogue_plan(m, n, k)) == TILE
    q_w, xv, gamma, _, _ = make(m, n, k, "f32")
    q, a = ref.quantize(xv)
    codes, absmax = codes_of(xv)
    raw, err = exact_on_gpu(q_w, q, a, gamma)
    y = bl.forward_epilogue(ref.pack(q_w).to(DEV), gamma.to(DEV), codes, n, k, absmax=absmax)
    assert ((y.double() - raw).abs() <= err).all()
    r = torch.randn(m, n, device=DEV, dtype=torch.bfloat16)
    y = bl.forward_epilogue(ref.pack(q_w).to(DEV), gamma.to(DEV), codes, n, k, absmax=absmax, act="relu", residual=r,
                            out_dtype=torch.bfloat16)
    v = raw.clamp(min=0) + r.double()
    assert ((y.double() - v).abs() <= err + ref.STEP[torch.bfloat16] * (v.abs() + err) + 2 * ref.U * raw.abs()).all()


@pytest.mark.parametrize("mean,e,n,k", [(40, 24, 2600, 2570), (25, 6, 6535, 441)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_ragged_experts(mean, e, n, k, dtype):
    """None, one, 32 and 33 slots among them, some of them without a token row."""
    g = torch.Generator().manual_seed(n)
    counts = torch.randint(0, 2 * mean, (e,), generator=g)
    counts[:5] = torch.tensor([0, 1, 32, 33, 64])
    layer = Layer(counts.tolist(), n, k, r=77)
    assert tile(bl.forward_experts_plan(e, layer.t, n, k)) == TILE
    layer.rows[::17] = -1
    y0 = torch.randn(layer.t, n, generator=g).to(dtype)
    y = layer.forward("relu", codes=True, y=y0.to(DEV))
    v, dv, there = layer.reference("relu")
    assert (~there).sum() == len(range(0, layer.t, 17))
    v, dv = ref.finish(v, dv, None, dtype)
    ref.check(y[there.to(DEV)], v[there], dv[there])
    assert torch.equal(y.cpu()[~there], y0[~there])
