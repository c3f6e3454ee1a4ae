"""Products whose launch would have 2^32 threads or more are refused, by the plan and by the call before it enqueues
anything (host-only: the pointers are never read)."""
import ctypes

import pytest

import bitlinear_fwd_amd as bl

FAKE = 0x10000
M, N, K = 1 << 20, (1 << 19) - 16, 4096  # 8192 x 2048 tiles of 128 x 256, 256 threads each


@pytest.mark.parametrize("e", [0, 1, 8, 4096])
@pytest.mark.parametrize("x", [None, "bf16", "f32"])
def test_plans_refuse(e, x):
    with pytest.raises(bl.BitLinearError) as refusal:
        bl.forward_experts_plan(e, M, N, K, x) if e else bl.forward_epilogue_plan(M, N, K, x)
    assert refusal.value.status == bl.BL_ERR_UNSUPPORTED
    p = bl.forward_epilogue_plan(M, N - 240, K, x)  # a column of tiles less
    assert p["workgroups"] * p["threads"] < 1 << 32


@pytest.mark.parametrize("x", [None, FAKE])
def test_calls_refuse(x):
    ep = bl.BlEpilogue(None, None, FAKE, 0, 0, 0, 0, bl.BL_F32)
    ex = bl.BlExperts(FAKE, FAKE, FAKE, None, 8, M, N)
    assert bl.lib().bitlinear_forward_epilogue(FAKE, FAKE, x, bl.BL_BF16, FAKE, FAKE, M, N, K, ctypes.byref(ep),
                                               None) == bl.BL_ERR_UNSUPPORTED
    assert bl.lib().bitlinear_forward_experts(ctypes.byref(ex), x, bl.BL_BF16, FAKE, FAKE, M, K, ctypes.byref(ep),
                                              None) == bl.BL_ERR_UNSUPPORTED
    assert bl.lib().bitlinear_forward_experts_combine(ctypes.byref(ex), x, bl.BL_BF16, FAKE, FAKE, M, K, FAKE, FAKE, 5,
                                                      2, ctypes.byref(ep), FAKE, 1 << 62, None) == bl.BL_ERR_UNSUPPORTED
