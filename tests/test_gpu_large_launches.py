"""Calls whose rows or outputs are more than the threads that one launch can have (2^32)."""
import pytest
import torch

import bitlinear_fwd_amd as bl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_combine_of_more_outputs_than_threads():
    """2^21 + 3 tokens of 8192 outputs, four to a thread: each token's row is the one of its slot times its weight."""
    m, n, k, t = (1 << 21) + 3, 8192, 64, 5
    g = torch.Generator(device=DEV).manual_seed(0)
    packed = torch.randint(0, 256, (1, bl.packed_bytes(n, k)), generator=g, device=DEV, dtype=torch.uint8)
    gamma = torch.full((1,), 0.02, device=DEV)
    x = torch.randn(t, k, generator=g, device=DEV)
    offsets = torch.tensor([0, t], dtype=torch.int32, device=DEV)
    slots = torch.randint(0, t, (m, 1), generator=g, device=DEV, dtype=torch.int32)
    weights = torch.randint(1, 9, (m, 1), generator=g, device=DEV).float()
    y = bl.forward_experts_combine(packed, gamma, offsets, x, n, k, slots, weights, out_dtype=torch.bfloat16)
    rows = bl.forward_experts(packed, gamma, offsets, x, n, k)
    table = (rows[:, None] * torch.arange(9, device=DEV)[:, None]).to(torch.bfloat16).view(t * 9, n)
    at = (slots.long() * 9 + weights.long()).view(-1)
    for lo in range(0, m, 1 << 17):
        assert torch.equal(y[lo:lo + (1 << 17)], table[at[lo:lo + (1 << 17)]]), lo


@pytest.mark.parametrize("k", [8, 9])
def test_more_rows_than_workgroups_of_256_threads(k):
    """2^24 + 9 token rows, a workgroup each in the quantiser: codes, row sums and a product's outputs as from the rows
    around each of its launches' borders in calls of their own."""
    r, n = (1 << 24) + 9, 16
    g = torch.Generator(device=DEV).manual_seed(k)
    x = torch.randn(r, k, generator=g, device=DEV).to(torch.bfloat16)
    packed = torch.randint(0, 256, (bl.packed_bytes(n, k),), generator=g, device=DEV, dtype=torch.uint8)
    gamma = torch.full((1,), 0.02, device=DEV)
    codes, scales, sums = bl.quantize_acts(x, want_rowsum=True)
    y = bl.forward_epilogue(packed, gamma, x, n, k)
    assert torch.equal(scales, x.float().abs().amax(1))
    for at in [i << 21 for i in range(1, 9)] + [r]:
        rows = slice(at - 5, min(at + 5, r))
        part = x[rows].clone()
        c, s, t = bl.quantize_acts(part, want_rowsum=True)
        assert torch.equal(codes[rows], c) and torch.equal(scales[rows], s) and torch.equal(sums[rows], t)
        assert torch.equal(y[rows], bl.forward_epilogue(packed, gamma, part, n, k))
