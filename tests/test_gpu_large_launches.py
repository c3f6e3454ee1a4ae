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
