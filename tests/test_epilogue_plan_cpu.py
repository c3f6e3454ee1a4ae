"""Which products of up to four tokens are one launch with the quantiser: those whose workgroups, which each quantise
all rows again, are few enough (host-only)."""
import pytest

import bitlinear_fwd_amd as bl


@pytest.mark.parametrize("m,n,k,one", [
    (1, 6912, 2560, True), (4, 6912, 2560, True), (4, 2560, 6912, True), (4, 4096, 4096, True), (1, 40, 40960, True),
    (1, 40, 41216, False), (4, 40, 10240, True), (4, 40, 10496, False), (4, 14336, 2560, False), (4, 28672, 1280, False),
    (2, 14336, 4096, False), (1, 28672, 8192, False), (5, 64, 256, False), (1, 64, 257, False)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_one_launch_or_two(m, n, k, one, x):
    p = bl.forward_epilogue_plan(m, n, k, x)
    assert p["launches"] == (1 if one else 2) and (p["kernel"] == "fused") == one
    assert bl.forward_epilogue_plan(m, n, k)["launches"] == 1  # codes
