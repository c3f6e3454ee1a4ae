"""MI355X-native BitNet b1.58 BitLinear forward: thin Python binding of libbitlinear.so.

The binding only marshals arguments: every step of the path (weight absmean + ternarise
+ pack, per-token absmax int8 activation quantisation, the packed-ternary x int8
contraction with exact int32 accumulation, and the fp32 rescale) runs in the HIP kernels
behind the C ABI declared in ``include/bitlinear.h``.  PyTorch supplies device memory
and the current stream.  There is no CPU fallback: if the library is missing or a call
fails, an exception is raised.

The method follows the aratech.ae article "BitNet b1.58: Microsoft's 1-bit LLM that runs
a 100B model on one CPU" (sub-sections "Ternary weights {-1, 0, +1}" and "BitLinear: the
building block") and the 2-bit code table of bhfrc.com news 56965, section 4.1.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbitlinear.so")

BL_OK, BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED, BL_ERR_HIP = 0, -1, -2, -3
BL_F32, BL_BF16 = 0, 1

_lib = None


class BitLinearError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libbitlinear.so (built by ``python -m bitlinear_fwd_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bitlinear_fwd_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, p, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.bitlinear_version.restype = c_int
        L.bitlinear_version.argtypes = []
        L.bitlinear_status_string.restype = ctypes.c_char_p
        L.bitlinear_status_string.argtypes = [c_int]
        for name in ("bitlinear_n_pad", "bitlinear_k_pad"):
            getattr(L, name).restype = i64
            getattr(L, name).argtypes = [i64]
        for name in ("bitlinear_packed_bytes", "bitlinear_wq_workspace_bytes"):
            getattr(L, name).restype = i64
            getattr(L, name).argtypes = [i64, i64]
        L.bitlinear_quantize_weights.restype = c_int
        L.bitlinear_quantize_weights.argtypes = [p, i64, i64, p, p, p, i64, p]
        L.bitlinear_quantize_weights_noalloc.restype = c_int
        L.bitlinear_quantize_weights_noalloc.argtypes = [p, i64, i64, p, p, p]
        L.bitlinear_quantize_acts.restype = c_int
        L.bitlinear_quantize_acts.argtypes = [p, c_int, i64, i64, p, p, p, p]
        L.bitlinear_forward_fused.restype = c_int
        L.bitlinear_forward_fused.argtypes = [p, p, p, c_int, i64, i64, i64, p, p, p, p, p]
        L.bitlinear_forward_plan.restype = c_int
        L.bitlinear_forward_plan.argtypes = [i64, i64, i64, p]
        L.bitlinear_forward_fused_plan.restype = c_int
        L.bitlinear_forward_fused_plan.argtypes = [i64, i64, i64, c_int, p]
        L.bitlinear_forward.restype = c_int
        L.bitlinear_forward.argtypes = [p, p, p, p, i64, i64, i64, p, p, p]
        L.bitlinear_forward_ws_bytes.restype = i64
        L.bitlinear_forward_ws_bytes.argtypes = [i64, i64, i64]
        L.bitlinear_forward_ws.restype = c_int
        L.bitlinear_forward_ws.argtypes = [p, p, p, p, i64, i64, i64, p, p, p, i64, p]
        L.bitlinear_probe_prefill_occupancy.restype = c_int
        L.bitlinear_probe_prefill_occupancy.argtypes = [p]
        L.bitlinear_forward_ws_plan.restype = c_int
        L.bitlinear_forward_ws_plan.argtypes = [i64, i64, i64, p]
        L.bitlinear_probe_stream_words.restype = i64
        L.bitlinear_probe_stream_words.argtypes = [i64]
        L.bitlinear_probe_stream.restype = c_int
        L.bitlinear_probe_stream.argtypes = [p, i64, p, i64, p]
        L.bitlinear_probe_read.restype = c_int
        L.bitlinear_probe_read.argtypes = [p, i64, i64, c_int, p, p]
        L.bitlinear_probe_mfma.restype = c_int
        L.bitlinear_probe_mfma.argtypes = [i64, i64, p, p]
        L.bitlinear_forward_grouped.restype = c_int
        L.bitlinear_forward_grouped.argtypes = [p, c_int, p, c_int, i64, i64, p, p, p]
        f32 = ctypes.c_float
        L.bitlinear_subln_quantize_acts.restype = c_int
        L.bitlinear_subln_quantize_acts.argtypes = [p, c_int, i64, i64, p, f32, p, p, p]
        L.bitlinear_forward_subln.restype = c_int
        L.bitlinear_forward_subln.argtypes = [p, p, p, c_int, i64, i64, i64, p, f32, p, p, p, p, p]
        L.bitlinear_forward_grouped_subln.restype = c_int
        L.bitlinear_forward_grouped_subln.argtypes = [p, c_int, p, c_int, i64, i64, p, f32, p, p, p]
        L.bitlinear_gated_relu2_workspace_bytes.restype = i64
        L.bitlinear_gated_relu2_workspace_bytes.argtypes = [i64, i64]
        L.bitlinear_forward_gated_relu2.restype = c_int
        L.bitlinear_forward_gated_relu2.argtypes = [p, p, p, p, p, c_int, i64, i64, i64, c_int, p, f32, p, p, p, p,
                                                    i64, p]
        L.bitlinear_forward_gated_relu2_plan.restype = c_int
        L.bitlinear_forward_gated_relu2_plan.argtypes = [i64, i64, i64, c_int, c_int, p]
        for name in ("bitlinear_kb_pad",):
            getattr(L, name).restype = i64
            getattr(L, name).argtypes = [i64]
        L.bitlinear_packed_bytes_binary.restype = i64
        L.bitlinear_packed_bytes_binary.argtypes = [i64, i64]
        L.bitlinear_quantize_weights_binary.restype = c_int
        L.bitlinear_quantize_weights_binary.argtypes = [p, i64, i64, p, p, p, i64, p]
        L.bitlinear_forward_binary.restype = c_int
        L.bitlinear_forward_binary.argtypes = [p, p, p, p, i64, i64, i64, p, p, p]
        L.bitlinear_forward_binary_plan.restype = c_int
        L.bitlinear_forward_binary_plan.argtypes = [i64, i64, i64, p]
        L.bitlinear_forward_lut.restype = c_int
        L.bitlinear_forward_lut.argtypes = [p, p, p, p, i64, i64, i64, p, p, p]
        L.bitlinear_forward_lut_plan.restype = c_int
        L.bitlinear_forward_lut_plan.argtypes = [i64, i64, i64, p]
        L.bitlinear_forward_subln_plan.restype = c_int
        L.bitlinear_forward_subln_plan.argtypes = [i64, i64, i64, c_int, p]
        for name in ("bitlinear_mxfp4_codes_bytes", "bitlinear_mxfp4_scales_bytes",
                     "bitlinear_layernorm_backward_ws_bytes"):
            getattr(L, name).restype = i64
            getattr(L, name).argtypes = [i64, i64]
        L.bitlinear_quantize_mxfp4.restype = c_int
        L.bitlinear_quantize_mxfp4.argtypes = [p, c_int, i64, i64, p, p, p, p]
        L.bitlinear_forward_mxfp4.restype = c_int
        L.bitlinear_forward_mxfp4.argtypes = [p, p, p, p, i64, i64, i64, p, c_int, p]
        L.bitlinear_forward_mxfp4_fused_ws_bytes.restype = i64
        L.bitlinear_forward_mxfp4_fused_ws_bytes.argtypes = [i64, i64, i64, c_int]
        L.bitlinear_forward_mxfp4_fused.restype = c_int
        L.bitlinear_forward_mxfp4_fused.argtypes = [p, p, p, c_int, i64, i64, i64, p, c_int, p, i64, p]
        L.bitlinear_forward_mxfp4_plan.restype = c_int
        L.bitlinear_forward_mxfp4_plan.argtypes = [i64, i64, i64, c_int, p]
        L.bitlinear_layernorm.restype = c_int
        L.bitlinear_layernorm.argtypes = [p, c_int, i64, i64, p, p, f32, p, p, p, p]
        L.bitlinear_layernorm_backward.restype = c_int
        L.bitlinear_layernorm_backward.argtypes = [p, p, c_int, i64, i64, p, p, p, p, p, p, p, i64, p]
        for name in ("bitlinear_forward_experts_combine_ws_bytes", "bitlinear_route_experts_ws_bytes"):
            getattr(L, name).restype = i64
            getattr(L, name).argtypes = [i64, i64]
        L.bitlinear_forward_epilogue.restype = c_int
        L.bitlinear_forward_epilogue.argtypes = [p, p, p, c_int, p, p, i64, i64, i64, p, p]
        L.bitlinear_forward_epilogue_plan.restype = c_int
        L.bitlinear_forward_epilogue_plan.argtypes = [i64, i64, i64, c_int, p]
        L.bitlinear_forward_experts.restype = c_int
        L.bitlinear_forward_experts.argtypes = [p, p, c_int, p, p, i64, i64, p, p]
        L.bitlinear_forward_experts_plan.restype = c_int
        L.bitlinear_forward_experts_plan.argtypes = [i64, i64, i64, i64, c_int, p]
        L.bitlinear_forward_experts_combine.restype = c_int
        L.bitlinear_forward_experts_combine.argtypes = [p, p, c_int, p, p, i64, i64, p, p, i64, i64, p, p, i64, p]
        L.bitlinear_route_experts.restype = c_int
        L.bitlinear_route_experts.argtypes = [p, c_int, i64, i64, i64, c_int, p, p, p, p, p, p, i64, p]
        _lib = L
    return _lib


EXPORTED_SYMBOLS = (
    "bitlinear_version", "bitlinear_status_string", "bitlinear_n_pad", "bitlinear_k_pad",
    "bitlinear_packed_bytes", "bitlinear_wq_workspace_bytes", "bitlinear_quantize_weights",
    "bitlinear_quantize_acts", "bitlinear_forward", "bitlinear_forward_fused", "bitlinear_forward_plan",
    "bitlinear_forward_fused_plan", "bitlinear_forward_grouped", "bitlinear_probe_stream_words",
    "bitlinear_probe_stream", "bitlinear_probe_read", "bitlinear_probe_mfma", "bitlinear_subln_quantize_acts",
    "bitlinear_forward_subln",
    "bitlinear_forward_grouped_subln", "bitlinear_forward_subln_plan", "bitlinear_gated_relu2_workspace_bytes",
    "bitlinear_forward_gated_relu2", "bitlinear_forward_gated_relu2_plan", "bitlinear_forward_lut",
    "bitlinear_forward_lut_plan", "bitlinear_kb_pad", "bitlinear_packed_bytes_binary",
    "bitlinear_quantize_weights_binary", "bitlinear_forward_binary", "bitlinear_forward_binary_plan",
    "bitlinear_quantize_weights_noalloc", "bitlinear_forward_ws_bytes", "bitlinear_forward_ws",
    "bitlinear_forward_ws_plan", "bitlinear_probe_prefill_occupancy", "bitlinear_mxfp4_codes_bytes",
    "bitlinear_mxfp4_scales_bytes", "bitlinear_quantize_mxfp4", "bitlinear_forward_mxfp4",
    "bitlinear_forward_mxfp4_fused_ws_bytes", "bitlinear_forward_mxfp4_fused", "bitlinear_layernorm",
    "bitlinear_layernorm_backward_ws_bytes", "bitlinear_layernorm_backward", "bitlinear_forward_mxfp4_plan",
    "bitlinear_forward_epilogue", "bitlinear_forward_epilogue_plan", "bitlinear_forward_experts",
    "bitlinear_forward_experts_plan", "bitlinear_forward_experts_combine",
    "bitlinear_forward_experts_combine_ws_bytes", "bitlinear_route_experts", "bitlinear_route_experts_ws_bytes",
)

MAX_GROUP = 8


class BlMatrix(ctypes.Structure):
    """bl_matrix of bitlinear.h: one weight matrix of a grouped call."""
    _fields_ = [("packed", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("Y", ctypes.c_void_p), ("acc", ctypes.c_void_p)]


class BlEpilogue(ctypes.Structure):
    """bl_epilogue of bitlinear.h: bias, activation and residual of a product, and its output."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("residual_ld", ctypes.c_int64), ("y_ld", ctypes.c_int64), ("act", ctypes.c_int),
                ("residual_dt", ctypes.c_int), ("y_dt", ctypes.c_int)]


class BlExperts(ctypes.Structure):
    """bl_experts of bitlinear.h: the matrices of a layer with experts, and their slots."""
    _fields_ = [("packed", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("E", ctypes.c_int64), ("T", ctypes.c_int64), ("N", ctypes.c_int64)]


def _check(fn: str, status: int) -> None:
    if status != BL_OK:
        raise BitLinearError(fn, status, lib().bitlinear_status_string(status).decode())


def status_string(status: int) -> str:
    return lib().bitlinear_status_string(status).decode()


def version() -> int:
    return lib().bitlinear_version()


def n_pad(n: int) -> int:
    return int(lib().bitlinear_n_pad(n))


def k_pad(k: int) -> int:
    return int(lib().bitlinear_k_pad(k))


def packed_bytes(n: int, k: int) -> int:
    return int(lib().bitlinear_packed_bytes(n, k))


def wq_workspace_bytes(n: int, k: int) -> int:
    return int(lib().bitlinear_wq_workspace_bytes(n, k))


def _plan_dict(out) -> dict:
    if out[0] == 5:
        return {"kernel": "binary", "workgroups": out[1], "threads": out[2], "row_blocks": out[3],
                "tiles_per_wave": out[4]}
    if out[0] == 4:
        return {"kernel": "lut", "workgroups": out[1], "threads": out[2], "row_blocks": out[3],
                "tiles_per_wave": out[4], "lds_bytes": out[5]}
    if out[0] == 3 and out[4] == 4:  # 5..16 tokens: every workgroup quantises the 16 token rows into LDS
        return {"kernel": "fused", "workgroups": out[1], "threads": out[2], "row_blocks": out[3],
                "acts": "lds16", "lds_acts": True, "lds_bytes": 0, "tiles_per_wave": out[5]}
    if out[0] == 3:
        return {"kernel": "fused", "workgroups": out[1], "threads": out[2], "row_blocks": out[3],
                "acts": "registers" if out[4] == 2 else "lds", "lds_acts": out[4] == 1,
                "lds_bytes": out[5] if out[4] == 1 else 0, "tiles_per_wave": out[5] if out[4] == 2 else 0}
    if out[0] == 1:
        acts = {0: "per-tile loads", 1: "lds", 2: "registers"}[out[4]]
        return {"kernel": "decode", "workgroups": out[1], "threads": out[2], "row_blocks": out[3],
                "acts": acts, "lds_acts": out[4] == 1, "lds_bytes": out[5] if out[4] == 1 else 0,
                "tiles_per_wave": out[5] if out[4] == 2 else 0}
    d = {"kernel": "prefill", "workgroups": out[1], "threads": out[2], "tile_m": out[3], "tile_n": out[4],
         "k_groups": out[5]}
    if out[0] == 6:
        d.update(split_tail=True, rounds=out[6], split_tiles=out[7], k_ranges=out[8], chunks_per_range=out[9])
    return d


def forward_plan(m: int, n: int, k: int) -> dict:
    """The launch bitlinear_forward makes for (M, N, K), computed on the host."""
    out = (ctypes.c_int32 * 6)()
    _check("bitlinear_forward_plan", lib().bitlinear_forward_plan(m, n, k, out))
    return _plan_dict(out)


def forward_ws_plan(m: int, n: int, k: int) -> dict:
    """The launch bitlinear_forward_ws makes for (M, N, K), computed on the host."""
    out = (ctypes.c_int32 * 10)()
    _check("bitlinear_forward_ws_plan", lib().bitlinear_forward_ws_plan(m, n, k, out))
    return _plan_dict(out)


def forward_ws_bytes(m: int, n: int, k: int) -> int:
    """Workspace bytes bitlinear_forward_ws needs for (M, N, K) (0: none)."""
    v = int(lib().bitlinear_forward_ws_bytes(m, n, k))
    if v < 0:
        raise ValueError(f"invalid shape {(m, n, k)}")
    return v


def forward_workspace(m: int, n: int, k: int, device):
    """A workspace for bitlinear_forward_ws on (M, N, K) (None when it needs none).  Its
    contents on entry do not matter and nothing carries over between calls, so one
    workspace serves later calls of any shape it is large enough for."""
    import torch

    nb = forward_ws_bytes(m, n, k)
    return torch.zeros(nb, dtype=torch.uint8, device=device) if nb > 0 else None


def forward_fused_plan(m: int, n: int, k: int, dtype: str = "bf16") -> dict:
    """What bitlinear_forward_fused does for (M, N, K): kernel "fused" (one launch) or the
    forward launch that follows the activation quantiser."""
    out = (ctypes.c_int32 * 6)()
    dt = BL_BF16 if dtype == "bf16" else BL_F32
    _check("bitlinear_forward_fused_plan", lib().bitlinear_forward_fused_plan(m, n, k, dt, out))
    return _plan_dict(out)


def forward_subln_plan(m: int, n: int, k: int, dtype: str = "bf16") -> dict:
    """What bitlinear_forward_subln does for (M, N, K): kernel "fused" (one launch) or the
    forward launch that follows the normalising quantiser."""
    out = (ctypes.c_int32 * 6)()
    dt = BL_BF16 if dtype == "bf16" else BL_F32
    _check("bitlinear_forward_subln_plan", lib().bitlinear_forward_subln_plan(m, n, k, dt, out))
    return _plan_dict(out)


def forward_gated_relu2_plan(m: int, n: int, k: int, dtype: str = "bf16", subln: bool = False) -> dict:
    """What bitlinear_forward_gated_relu2 does for (M, N, K): kernel "fused" (one launch)
    or the plan of each of the two forwards."""
    out = (ctypes.c_int32 * 6)()
    dt = BL_BF16 if dtype == "bf16" else BL_F32
    _check("bitlinear_forward_gated_relu2_plan",
           lib().bitlinear_forward_gated_relu2_plan(m, n, k, dt, int(subln), out))
    return _plan_dict(out)


def _stream(device) -> int:
    import torch

    return torch.cuda.current_stream(device).cuda_stream


def _require_cuda(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def quantize_weights(W, packed=None, gamma=None, workspace=None):
    """Ternarise + pack latent weights W[N][K] (fp32, out x in) on the GPU.

    Returns ``(packed uint8 [packed_bytes(N, K)], gamma fp32 [1])``."""
    import torch

    _require_cuda(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    n, k = W.shape
    dev = W.device
    if packed is None:
        packed = torch.empty(packed_bytes(n, k), dtype=torch.uint8, device=dev)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(wq_workspace_bytes(n, k), dtype=torch.uint8, device=dev)
    _check("bitlinear_quantize_weights", lib().bitlinear_quantize_weights(
        W.data_ptr(), n, k, packed.data_ptr(), gamma.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(dev)))
    return packed, gamma


def quantize_weights_noalloc(W, packed=None, gamma=None):
    """bitlinear_quantize_weights_noalloc: the weight quantiser with the library's own static
    scratch in place of a workspace (the C call allocates nothing; outputs not given here
    are allocated by torch before it).  Returns ``(packed, gamma)``."""
    import torch

    _require_cuda(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    n, k = W.shape
    dev = W.device
    if packed is None:
        packed = torch.empty(packed_bytes(n, k), dtype=torch.uint8, device=dev)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=dev)
    _check("bitlinear_quantize_weights_noalloc", lib().bitlinear_quantize_weights_noalloc(
        W.data_ptr(), n, k, packed.data_ptr(), gamma.data_ptr(), _stream(dev)))
    return packed, gamma


def quantize_acts(x, xq=None, absmax=None, rowsum=None, want_rowsum: bool = False):
    """Per-token absmax int8 quantisation of x[M][K] (fp32 or bf16) on the GPU.

    Returns ``(xq int8 [M][K_pad], absmax fp32 [M])``, plus the exact int32 row sums of
    the codes when ``want_rowsum`` is set or ``rowsum`` is given."""
    import torch

    _require_cuda(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [tokens, features]")
    if x.dtype == torch.float32:
        dt = BL_F32
    elif x.dtype == torch.bfloat16:
        dt = BL_BF16
    else:
        raise ValueError("x must be float32 or bfloat16")
    m, k = x.shape
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if absmax is None:
        absmax = torch.empty(m, dtype=torch.float32, device=dev)
    if want_rowsum and rowsum is None:
        rowsum = torch.empty(m, dtype=torch.int32, device=dev)
    _check("bitlinear_quantize_acts", lib().bitlinear_quantize_acts(
        x.data_ptr(), dt, m, k, xq.data_ptr(), absmax.data_ptr(), rowsum.data_ptr() if rowsum is not None else None,
        _stream(dev)))
    return (xq, absmax, rowsum) if rowsum is not None else (xq, absmax)


def forward(packed, gamma, xq, absmax, n: int, k: int, y=None, acc=None, want_y: bool = True,
            want_acc: bool = False):
    """y[M][N] (fp32) and/or acc[M][N] (int32) of the packed-ternary x int8 product.

    Returns y, acc or (y, acc) depending on ``want_y`` / ``want_acc``."""
    import torch

    for t, name in ((packed, "packed"), (gamma, "gamma"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    m = xq.shape[0]
    dev = xq.device
    if want_y and y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    if want_acc and acc is None:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    _check("bitlinear_forward", lib().bitlinear_forward(
        packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), absmax.data_ptr(), m, n, k,
        y.data_ptr() if y is not None else None, acc.data_ptr() if acc is not None else None,
        _stream(dev)))
    if want_y and want_acc:
        return y, acc
    return y if want_y else acc


def forward_ws(packed, gamma, xq, absmax, n: int, k: int, workspace=None, y=None, acc=None, want_y: bool = True,
               want_acc: bool = False):
    """forward() through bitlinear_forward_ws: the same results, with the caller's
    zero-filled workspace (forward_workspace) for the prefill GEMM's split tail tiles."""
    import torch

    for t, name in ((packed, "packed"), (gamma, "gamma"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    m = xq.shape[0]
    dev = xq.device
    if workspace is not None:
        _require_cuda(workspace, "workspace")
    if want_y and y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    if want_acc and acc is None:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    _check("bitlinear_forward_ws", lib().bitlinear_forward_ws(
        packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), absmax.data_ptr(), m, n, k,
        y.data_ptr() if y is not None else None, acc.data_ptr() if acc is not None else None,
        workspace.data_ptr() if workspace is not None else None,
        workspace.numel() * workspace.element_size() if workspace is not None else 0, _stream(dev)))
    if want_y and want_acc:
        return y, acc
    return y if want_y else acc


def kb_pad(k: int) -> int:
    return int(lib().bitlinear_kb_pad(k))


def packed_bytes_binary(n: int, k: int) -> int:
    return int(lib().bitlinear_packed_bytes_binary(n, k))


def quantize_weights_binary(W, packed=None, beta=None, workspace=None):
    """1-bit sign-binary weights: (packed binary buffer, beta = exact mean |W|) on the GPU."""
    import torch

    _require_cuda(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    W = W.contiguous()
    n, k = W.shape
    dev = W.device
    if packed is None:
        packed = torch.empty(packed_bytes_binary(n, k), dtype=torch.uint8, device=dev)
    if beta is None:
        beta = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(wq_workspace_bytes(n, k), dtype=torch.uint8, device=dev)
    _check("bitlinear_quantize_weights_binary", lib().bitlinear_quantize_weights_binary(
        W.data_ptr(), n, k, packed.data_ptr(), beta.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(dev)))
    return packed, beta


def forward_binary_plan(m: int, n: int, k: int):
    """The launch bitlinear_forward_binary makes for (M, N, K), or None where it does not apply."""
    out = (ctypes.c_int32 * 6)()
    st = lib().bitlinear_forward_binary_plan(m, n, k, out)
    if st == BL_ERR_UNSUPPORTED:
        return None
    _check("bitlinear_forward_binary_plan", st)
    return _plan_dict(out)


def forward_binary(packed, beta, xq, absmax, n: int, k: int, y=None, acc=None, want_y: bool = True,
                   want_acc: bool = False):
    """bitlinear_forward with 1-bit sign-binary weights (M <= 4)."""
    import torch

    for t, name in ((packed, "packed"), (beta, "beta"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    m = xq.shape[0]
    dev = xq.device
    if want_y and y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    if want_acc and acc is None:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    _check("bitlinear_forward_binary", lib().bitlinear_forward_binary(
        packed.data_ptr(), beta.data_ptr(), xq.data_ptr(), absmax.data_ptr(), m, n, k,
        y.data_ptr() if y is not None else None, acc.data_ptr() if acc is not None else None, _stream(dev)))
    if want_y and want_acc:
        return y, acc
    return y if want_y else acc


def forward_lut_plan(m: int, n: int, k: int):
    """The launch bitlinear_forward_lut makes for (M, N, K), or None where it does not apply."""
    out = (ctypes.c_int32 * 6)()
    st = lib().bitlinear_forward_lut_plan(m, n, k, out)
    if st == BL_ERR_UNSUPPORTED:
        return None
    _check("bitlinear_forward_lut_plan", st)
    return _plan_dict(out)


def forward_lut(packed, gamma, xq, absmax, n: int, k: int, y=None, acc=None, want_y: bool = True,
                want_acc: bool = False):
    """bitlinear_forward computed by table lookups (comparison variant, M <= 4)."""
    import torch

    for t, name in ((packed, "packed"), (gamma, "gamma"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    m = xq.shape[0]
    dev = xq.device
    if want_y and y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    if want_acc and acc is None:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    _check("bitlinear_forward_lut", lib().bitlinear_forward_lut(
        packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), absmax.data_ptr(), m, n, k,
        y.data_ptr() if y is not None else None, acc.data_ptr() if acc is not None else None, _stream(dev)))
    if want_y and want_acc:
        return y, acc
    return y if want_y else acc


def forward_fused(packed, gamma, x, n: int, k: int, y=None, acc=None, xq=None, absmax=None, want_y: bool = True,
                  want_acc: bool = False):
    """Quantise x[M][K] (fp32/bf16) per token and apply the packed weights in one call.

    Returns (y and/or acc, xq, absmax)."""
    import torch

    for t, name in ((packed, "packed"), (gamma, "gamma"), (x, "x")):
        _require_cuda(t, name)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be [tokens, K]")
    if x.dtype == torch.float32:
        dt = BL_F32
    elif x.dtype == torch.bfloat16:
        dt = BL_BF16
    else:
        raise ValueError("x must be float32 or bfloat16")
    m = x.shape[0]
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if absmax is None:
        absmax = torch.empty(m, dtype=torch.float32, device=dev)
    if want_y and y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    if want_acc and acc is None:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    _check("bitlinear_forward_fused", lib().bitlinear_forward_fused(
        packed.data_ptr(), gamma.data_ptr(), x.data_ptr(), dt, m, n, k,
        y.data_ptr() if y is not None else None, acc.data_ptr() if acc is not None else None,
        xq.data_ptr(), absmax.data_ptr(), _stream(dev)))
    out = (y, acc) if (want_y and want_acc) else (y if want_y else acc)
    return out, xq, absmax


def _group_array(mats):
    """Host bl_matrix array for [(packed, gamma, n, y, acc), ...] (y / acc may be None)."""
    if not 1 <= len(mats) <= MAX_GROUP:
        raise ValueError(f"a group holds 1..{MAX_GROUP} matrices")
    arr = (BlMatrix * len(mats))()
    for i, (packed, gamma, n, y, acc) in enumerate(mats):
        for t, name in ((packed, "packed"), (gamma, "gamma")):
            _require_cuda(t, name)
        arr[i] = BlMatrix(packed.data_ptr(), gamma.data_ptr(), n, y.data_ptr() if y is not None else None,
                          acc.data_ptr() if acc is not None else None)
    return arr


def forward_grouped(mats, x, k: int, xq=None, absmax=None, want_y: bool = True, want_acc: bool = False):
    """Several projections of one input x[M][K] (fp32/bf16): ``mats`` is a list of
    (packed, gamma, n).  The activations are quantised once.  Returns (outs, xq, absmax)
    with outs[i] = y_i, acc_i or (y_i, acc_i) as for forward_fused."""
    import torch

    _require_cuda(x, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be [tokens, K]")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be float32 or bfloat16")
    dt = BL_BF16 if x.dtype == torch.bfloat16 else BL_F32
    m = x.shape[0]
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if absmax is None:
        absmax = torch.empty(m, dtype=torch.float32, device=dev)
    full, outs = [], []
    for packed, gamma, n in mats:
        y = torch.empty((m, n), dtype=torch.float32, device=dev) if want_y else None
        acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
        full.append((packed, gamma, n, y, acc))
        outs.append((y, acc) if (want_y and want_acc) else (y if want_y else acc))
    arr = _group_array(full)
    _check("bitlinear_forward_grouped", lib().bitlinear_forward_grouped(
        ctypes.addressof(arr), len(full), x.data_ptr(), dt, m, k, xq.data_ptr(), absmax.data_ptr(), _stream(dev)))
    return outs, xq, absmax


def _acts_dtype(x, k=None) -> int:
    import torch

    _require_cuda(x, "x")
    if x.dim() != 2 or (k is not None and x.shape[1] != k):
        raise ValueError("x must be 2-D [tokens, K]")
    if x.dtype == torch.float32:
        return BL_F32
    if x.dtype == torch.bfloat16:
        return BL_BF16
    raise ValueError("x must be float32 or bfloat16")


def _gain_ptr(gain, k: int):
    import torch

    if gain is None:
        return None
    _require_cuda(gain, "gain")
    if gain.dtype != torch.float32 or gain.dim() != 1 or gain.shape[0] != k or not gain.is_contiguous():
        raise ValueError("gain must be a contiguous float32 [K] tensor")
    return gain.data_ptr()


def subln_quantize_acts(x, gain=None, eps: float = 1e-5, xq=None, scale=None):
    """Sub-layer RMS normalisation (per-feature gain, eps) fused with the per-token absmax
    int8 quantiser.  Returns ``(xq int8 [M][K_pad], scale fp32 [M])``; scale is the
    absmax of the normalised row and takes the place of absmax in ``forward``."""
    import torch

    dt = _acts_dtype(x)
    m, k = x.shape
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty(m, dtype=torch.float32, device=dev)
    _check("bitlinear_subln_quantize_acts", lib().bitlinear_subln_quantize_acts(
        x.data_ptr(), dt, m, k, _gain_ptr(gain, k), eps, xq.data_ptr(), scale.data_ptr(), _stream(dev)))
    return xq, scale


def forward_subln(packed, gamma, x, n: int, k: int, gain=None, eps: float = 1e-5, y=None, acc=None, xq=None,
                  scale=None, want_y: bool = True, want_acc: bool = False):
    """Sub-layer normalisation, quantisation and the packed-weight product in one call.
    Returns (y and/or acc, xq, scale) as forward_fused."""
    import torch

    for t, name in ((packed, "packed"), (gamma, "gamma")):
        _require_cuda(t, name)
    dt = _acts_dtype(x, k)
    m = x.shape[0]
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty(m, dtype=torch.float32, device=dev)
    if want_y and y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=dev)
    if want_acc and acc is None:
        acc = torch.empty((m, n), dtype=torch.int32, device=dev)
    _check("bitlinear_forward_subln", lib().bitlinear_forward_subln(
        packed.data_ptr(), gamma.data_ptr(), x.data_ptr(), dt, m, n, k, _gain_ptr(gain, k), eps,
        y.data_ptr() if y is not None else None, acc.data_ptr() if acc is not None else None,
        xq.data_ptr(), scale.data_ptr(), _stream(dev)))
    out = (y, acc) if (want_y and want_acc) else (y if want_y else acc)
    return out, xq, scale


def forward_grouped_subln(mats, x, k: int, gain=None, eps: float = 1e-5, xq=None, scale=None,
                          want_y: bool = True, want_acc: bool = False):
    """forward_grouped behind the sub-layer normalisation: one normalising quantisation,
    shared by every matrix.  Returns (outs, xq, scale)."""
    import torch

    dt = _acts_dtype(x, k)
    m = x.shape[0]
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty(m, dtype=torch.float32, device=dev)
    full, outs = [], []
    for packed, gamma, n in mats:
        y = torch.empty((m, n), dtype=torch.float32, device=dev) if want_y else None
        acc = torch.empty((m, n), dtype=torch.int32, device=dev) if want_acc else None
        full.append((packed, gamma, n, y, acc))
        outs.append((y, acc) if (want_y and want_acc) else (y if want_y else acc))
    arr = _group_array(full)
    _check("bitlinear_forward_grouped_subln", lib().bitlinear_forward_grouped_subln(
        ctypes.addressof(arr), len(full), x.data_ptr(), dt, m, k, _gain_ptr(gain, k), eps, xq.data_ptr(),
        scale.data_ptr(), _stream(dev)))
    return outs, xq, scale


def forward_gated_relu2(gate, up, x, n: int, k: int, subln: bool = False, gain=None, eps: float = 1e-5, h=None,
                        xq=None, scale=None, workspace=None):
    """Gate / up pair of one input with the squared-ReLU gating: ``gate`` and ``up`` are
    (packed, gamma) of two N x K matrices.  Returns (h fp32 [M][N], xq, scale)."""
    import torch

    for t, name in ((gate[0], "gate packed"), (gate[1], "gate gamma"), (up[0], "up packed"), (up[1], "up gamma")):
        _require_cuda(t, name)
    dt = _acts_dtype(x, k)
    m = x.shape[0]
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k_pad(k)), dtype=torch.int8, device=dev)
    if scale is None:
        scale = torch.empty(m, dtype=torch.float32, device=dev)
    if h is None:
        h = torch.empty((m, n), dtype=torch.float32, device=dev)
    fused = forward_gated_relu2_plan(m, n, k, "bf16" if dt == BL_BF16 else "f32", subln)["kernel"] == "fused"
    fused = fused and x.data_ptr() % 16 == 0 and (not subln or gain is None or gain.data_ptr() % 16 == 0)
    if workspace is None and not fused:
        workspace = torch.empty(int(lib().bitlinear_gated_relu2_workspace_bytes(m, n)), dtype=torch.uint8,
                                device=dev)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("bitlinear_forward_gated_relu2", lib().bitlinear_forward_gated_relu2(
        gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), x.data_ptr(), dt, m, n, k,
        int(subln), _gain_ptr(gain, k) if subln else None, eps, h.data_ptr(), xq.data_ptr(), scale.data_ptr(),
        ws_ptr, ws_len, _stream(dev)))
    return h, xq, scale


def probe_stream(buf, out=None):
    """Read the uint8 device tensor ``buf`` with the decode access pattern (measurement
    probe); returns the per-32-KiB-block XOR checksums (uint32 device tensor)."""
    import torch

    _require_cuda(buf, "buf")
    nbytes = buf.numel() * buf.element_size()
    words = int(lib().bitlinear_probe_stream_words(nbytes))
    if words < 0:
        raise ValueError("probe_stream needs a multiple of 1024 bytes")
    if out is None:
        out = torch.empty(words, dtype=torch.int32, device=buf.device)
    _check("bitlinear_probe_stream", lib().bitlinear_probe_stream(buf.data_ptr(), nbytes, out.data_ptr(),
                                                                  out.numel(), _stream(buf.device)))
    return out


def probe_read(buf, workgroups: int, nontemporal: bool = True, out=None):
    """Read the device tensor ``buf`` with a plain grid-stride loop of ``workgroups`` x 256
    lanes (measurement probe); returns the per-workgroup XOR checksums (int32 device tensor)."""
    import torch

    _require_cuda(buf, "buf")
    nbytes = buf.numel() * buf.element_size()
    if out is None:
        out = torch.empty(workgroups, dtype=torch.int32, device=buf.device)
    if out.numel() < workgroups:
        raise ValueError("out needs one word per workgroup")
    _check("bitlinear_probe_read", lib().bitlinear_probe_read(buf.data_ptr(), nbytes, workgroups, int(nontemporal),
                                                              out.data_ptr(), _stream(buf.device)))
    return out


def probe_mfma(iters: int, workgroups: int, out):
    """Matrix-core probe: workgroups x 4 waves x 16 independent int8 MFMAs per iteration."""
    _require_cuda(out, "out")
    if out.numel() < workgroups:
        raise ValueError("out needs one word per workgroup")
    _check("bitlinear_probe_mfma", lib().bitlinear_probe_mfma(iters, workgroups, out.data_ptr(), _stream(out.device)))
    return out


def prefill_occupancy() -> dict:
    """Resident workgroups per compute unit of the one-group prefill kernels, from the HIP
    runtime: {"whole": {256: n, 192: n}, "split": {256: n, 192: n}} by tile width."""
    out = (ctypes.c_int32 * 4)()
    _check("bitlinear_probe_prefill_occupancy", lib().bitlinear_probe_prefill_occupancy(out))
    return {"whole": {256: out[0], 192: out[1]}, "split": {256: out[2], 192: out[3]}}


class PreparedCall:
    """One C-ABI call with its arguments marshalled once: raw device pointers, sizes and the
    stream handle, converted to ctypes values up front.  Calling it re-issues the same
    launch for the cost of one foreign call, for launch loops where the per-call Python
    work of the functions above would take longer than the kernel itself.  The caller keeps
    the tensors the pointers came from alive.  The stream is the one current when the call
    was prepared: to record the call into a HIP graph, prepare it inside the capture."""

    def __init__(self, fn: str, *args):
        self._name = fn
        self._fn = getattr(lib(), fn)
        self._args = tuple(t(a) for t, a in zip(self._fn.argtypes, args))
        if len(self._args) != len(self._fn.argtypes):
            raise ValueError(f"{fn} takes {len(self._fn.argtypes)} arguments")

    def __call__(self) -> None:
        st = self._fn(*self._args)
        if st != BL_OK:
            _check(self._name, st)


def prepare_forward_fused(packed, gamma, x, n: int, k: int, y, xq, absmax) -> PreparedCall:
    """bitlinear_forward_fused on these tensors (y fp32 output), marshalled once."""
    import torch

    for t, name in ((packed, "packed"), (gamma, "gamma"), (x, "x"), (y, "y"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    dt = BL_BF16 if x.dtype == torch.bfloat16 else BL_F32
    return PreparedCall("bitlinear_forward_fused", packed.data_ptr(), gamma.data_ptr(), x.data_ptr(), dt,
                        x.shape[0], n, k, y.data_ptr(), None, xq.data_ptr(), absmax.data_ptr(), _stream(x.device))


def prepare_forward_grouped(mats, x, k: int, xq, absmax) -> PreparedCall:
    """bitlinear_forward_grouped on these tensors: ``mats`` is a list of
    (packed, gamma, n, y) with fp32 outputs y, marshalled once."""
    import torch

    for t, name in ((x, "x"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    arr = _group_array([(pk, g, n, y, None) for pk, g, n, y in mats])
    dt = BL_BF16 if x.dtype == torch.bfloat16 else BL_F32
    call = PreparedCall("bitlinear_forward_grouped", ctypes.addressof(arr), len(mats), x.data_ptr(), dt,
                        x.shape[0], k, xq.data_ptr(), absmax.data_ptr(), _stream(x.device))
    call._keep = arr  # the host descriptor array must outlive the call object
    return call


def prepare_forward_subln(packed, gamma, x, n: int, k: int, gain, eps: float, y, xq, scale) -> PreparedCall:
    """bitlinear_forward_subln on these tensors (y fp32 output), marshalled once."""
    for t, name in ((packed, "packed"), (gamma, "gamma"), (y, "y"), (xq, "xq"), (scale, "scale")):
        _require_cuda(t, name)
    dt = _acts_dtype(x, k)
    return PreparedCall("bitlinear_forward_subln", packed.data_ptr(), gamma.data_ptr(), x.data_ptr(), dt,
                        x.shape[0], n, k, _gain_ptr(gain, k), eps, y.data_ptr(), None, xq.data_ptr(),
                        scale.data_ptr(), _stream(x.device))


def prepare_forward_grouped_subln(mats, x, k: int, gain, eps: float, xq, scale) -> PreparedCall:
    """bitlinear_forward_grouped_subln on these tensors: ``mats`` is a list of
    (packed, gamma, n, y) with fp32 outputs y, marshalled once."""
    for t, name in ((xq, "xq"), (scale, "scale")):
        _require_cuda(t, name)
    dt = _acts_dtype(x, k)
    arr = _group_array([(pk, g, n, y, None) for pk, g, n, y in mats])
    call = PreparedCall("bitlinear_forward_grouped_subln", ctypes.addressof(arr), len(mats), x.data_ptr(), dt,
                        x.shape[0], k, _gain_ptr(gain, k), eps, xq.data_ptr(), scale.data_ptr(), _stream(x.device))
    call._keep = arr
    return call


def prepare_subln_quantize_acts(x, gain, eps: float, xq, scale) -> PreparedCall:
    """bitlinear_subln_quantize_acts on these tensors, marshalled once."""
    for t, name in ((xq, "xq"), (scale, "scale")):
        _require_cuda(t, name)
    dt = _acts_dtype(x)
    return PreparedCall("bitlinear_subln_quantize_acts", x.data_ptr(), dt, x.shape[0], x.shape[1],
                        _gain_ptr(gain, x.shape[1]), eps, xq.data_ptr(), scale.data_ptr(), _stream(x.device))


def prepare_forward_gated_relu2(gate, up, x, n: int, k: int, subln: bool, gain, eps: float, h, xq, scale,
                                workspace=None) -> PreparedCall:
    """bitlinear_forward_gated_relu2 on these tensors, marshalled once."""
    for t, name in ((h, "h"), (xq, "xq"), (scale, "scale")):
        _require_cuda(t, name)
    dt = _acts_dtype(x, k)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return PreparedCall("bitlinear_forward_gated_relu2", gate[0].data_ptr(), gate[1].data_ptr(), up[0].data_ptr(),
                        up[1].data_ptr(), x.data_ptr(), dt, x.shape[0], n, k, int(subln),
                        _gain_ptr(gain, k) if subln else None, eps, h.data_ptr(), xq.data_ptr(), scale.data_ptr(),
                        ws_ptr, ws_len, _stream(x.device))


def prepare_forward_lut(packed, gamma, xq, absmax, n: int, k: int, y) -> PreparedCall:
    """bitlinear_forward_lut on these tensors (y fp32 output), marshalled once."""
    for t, name in ((packed, "packed"), (gamma, "gamma"), (xq, "xq"), (absmax, "absmax"), (y, "y")):
        _require_cuda(t, name)
    return PreparedCall("bitlinear_forward_lut", packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), absmax.data_ptr(),
                        xq.shape[0], n, k, y.data_ptr(), None, _stream(xq.device))


def prepare_forward_binary(packed, beta, xq, absmax, n: int, k: int, y) -> PreparedCall:
    """bitlinear_forward_binary on these tensors (y fp32 output), marshalled once."""
    for t, name in ((packed, "packed"), (beta, "beta"), (xq, "xq"), (absmax, "absmax"), (y, "y")):
        _require_cuda(t, name)
    return PreparedCall("bitlinear_forward_binary", packed.data_ptr(), beta.data_ptr(), xq.data_ptr(),
                        absmax.data_ptr(), xq.shape[0], n, k, y.data_ptr(), None, _stream(xq.device))


def prepare_quantize_acts(x, xq, absmax) -> PreparedCall:
    """bitlinear_quantize_acts on these tensors, marshalled once."""
    import torch

    for t, name in ((x, "x"), (xq, "xq"), (absmax, "absmax")):
        _require_cuda(t, name)
    dt = BL_BF16 if x.dtype == torch.bfloat16 else BL_F32
    return PreparedCall("bitlinear_quantize_acts", x.data_ptr(), dt, x.shape[0], x.shape[1], xq.data_ptr(),
                        absmax.data_ptr(), None, _stream(x.device))


def prepare_forward_ws(packed, gamma, xq, absmax, n: int, k: int, y, workspace) -> PreparedCall:
    """bitlinear_forward_ws on these tensors (y fp32 output), marshalled once."""
    for t, name in ((packed, "packed"), (gamma, "gamma"), (xq, "xq"), (absmax, "absmax"), (y, "y")):
        _require_cuda(t, name)
    return PreparedCall("bitlinear_forward_ws", packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), absmax.data_ptr(),
                        xq.shape[0], n, k, y.data_ptr(), None,
                        workspace.data_ptr() if workspace is not None else None,
                        workspace.numel() * workspace.element_size() if workspace is not None else 0,
                        _stream(xq.device))


def prepare_forward(packed, gamma, xq, absmax, n: int, k: int, y) -> PreparedCall:
    """bitlinear_forward on these tensors (y fp32 output), marshalled once."""
    for t, name in ((packed, "packed"), (gamma, "gamma"), (xq, "xq"), (absmax, "absmax"), (y, "y")):
        _require_cuda(t, name)
    return PreparedCall("bitlinear_forward", packed.data_ptr(), gamma.data_ptr(), xq.data_ptr(), absmax.data_ptr(),
                        xq.shape[0], n, k, y.data_ptr(), None, _stream(xq.device))


class BitLinear:
    """Inference-time BitLinear: weights quantised once, forward per token batch."""

    def __init__(self, W):
        self.n, self.k = W.shape
        self.packed, self.gamma = quantize_weights(W)

    def __call__(self, x):
        y, _, _ = forward_fused(self.packed, self.gamma, x.contiguous(), self.n, self.k)
        return y


# The calls below take a few microseconds of host time each, a launch included, so what they need of
# torch and of the library is looked up once, their checks read every attribute once, and they
# allocate nothing that the caller has given.  The current stream and device are asked for below
# torch's public functions, as its own generated code does (0.08 us for the stream, 1.1 through
# torch.cuda.current_stream).


class _Runtime:
    """torch and the library, bound on the first call."""

    def __init__(self):
        import torch

        L = lib()
        self.torch, self.empty, self.empty_like = torch, torch.empty, torch.empty_like
        self.stream, self.current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self.u8, self.f32 = torch.uint8, torch.float32
        self.codes = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}
        self.quantize_mxfp4 = L.bitlinear_quantize_mxfp4
        self.forward_mxfp4 = L.bitlinear_forward_mxfp4
        self.forward_mxfp4_fused = L.bitlinear_forward_mxfp4_fused
        self.fused_ws_bytes = L.bitlinear_forward_mxfp4_fused_ws_bytes
        self.layernorm = L.bitlinear_layernorm
        self.layernorm_backward = L.bitlinear_layernorm_backward
        self.backward_ws_bytes = L.bitlinear_layernorm_backward_ws_bytes
        self.i8, self.i32 = torch.int8, torch.int32
        self.forward_epilogue = L.bitlinear_forward_epilogue
        self.forward_experts = L.bitlinear_forward_experts
        self.forward_experts_combine = L.bitlinear_forward_experts_combine
        self.route_experts = L.bitlinear_route_experts


_RT = None


def _runtime() -> _Runtime:
    global _RT
    if _RT is None:
        _RT = _Runtime()
    return _RT


def _call(rt, f, index: int, args) -> None:
    """The library call `f` on the device's current stream, with the device the current one."""
    if rt.current() == index:
        st = f(*args, rt.stream(index))
    else:
        with rt.torch.cuda.device(index):
            st = f(*args, rt.stream(index))
    if st != BL_OK:
        _check(f.__name__, st)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _dtype_code(rt, dtype, name: str) -> int:
    code = rt.codes.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code


def _require_rows(rt, t, name: str) -> int:
    """A contiguous GPU matrix of fp32 or bf16 rows; returns its bl_dtype."""
    if t.is_cuda and t.is_contiguous() and t.dim() == 2 and t.numel():
        code = rt.codes.get(t.dtype)
        return code if code is not None else _dtype_code(rt, t.dtype, name)
    raise ValueError(f"{name} must be a non-empty contiguous 2-D GPU tensor")


def _given(t, name: str, shape, dtype, index: int):
    """`t`, an output or vector given by the caller, checked: contiguous, of this shape (a
    tuple), type and device."""
    if t.get_device() != index or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on cuda:{index}")
    return t


def _bytes_at_least(rt, t, name: str, nbytes: int, index: int) -> int:
    """The address of `t`, checked to be a contiguous uint8 tensor of at least nbytes on the
    device."""
    if t.get_device() != index or t.dtype != rt.u8 or not t.is_contiguous() or t.numel() < nbytes:
        raise ValueError(f"{name} must be a contiguous uint8 tensor of at least {nbytes} bytes on cuda:{index}")
    return t.data_ptr()


def mxfp4_codes_bytes(rows: int, k: int) -> int:
    """Bytes of the MXFP4 codes of a rows x k matrix (16-row x 128-column tiles of 1024 bytes)."""
    return ((rows + 15) >> 4) * ((k + 127) >> 7) << 10 if rows >= 1 and k >= 1 else -1


def mxfp4_scales_bytes(rows: int, k: int) -> int:
    """Bytes of the MXFP4 block scales of a rows x k matrix."""
    return ((rows + 15) >> 4) * ((k + 511) >> 9) << 8 if rows >= 1 and k >= 1 else -1


def quantize_mxfp4(x, codes=None, scales=None, values=None, want_values: bool = False):
    """MXFP4 quantisation of x[R][K] (fp32 or bf16) on the GPU: blocks of 32 columns share a
    power of two, each element is a 4-bit float (weights and activations alike).

    Returns ``(codes uint8, scales uint8)`` in the layout of bitlinear.h, plus ``values``
    ([R][K] of x's type, what the codes stand for) when ``want_values`` is set or ``values``
    is given."""
    rt = _RT or _runtime()
    dt = _require_rows(rt, x, "x")
    r, k = x.shape
    dev = x.get_device()
    nc, ns = mxfp4_codes_bytes(r, k), mxfp4_scales_bytes(r, k)
    if codes is None:
        codes = rt.empty(nc, dtype=rt.u8, device=x.device)
    if scales is None:
        scales = rt.empty(ns, dtype=rt.u8, device=x.device)
    if values is not None:
        _given(values, "values", (r, k), x.dtype, dev)
    elif want_values:
        values = rt.empty_like(x)
    _call(rt, rt.quantize_mxfp4, dev, (x.data_ptr(), dt, r, k, _bytes_at_least(rt, codes, "codes", nc, dev),
                                       _bytes_at_least(rt, scales, "scales", ns, dev), _ptr(values)))
    return (codes, scales, values) if values is not None else (codes, scales)


def _product_output(rt, y, out_dtype, m: int, n: int, like):
    """(y, its bl_dtype) of a product: the caller's or a new one on like's device."""
    if y is not None:
        dtype = out_dtype or y.dtype
        return _given(y, "y", (m, n), dtype, like.get_device()), _dtype_code(rt, dtype, "out_dtype")
    dtype = out_dtype or rt.f32
    ydt = _dtype_code(rt, dtype, "out_dtype")
    if m < 0 or n < 0:
        m = n = 0  # refused by the library
    return rt.empty(m, n, dtype=dtype, device=like.device), ydt  # (a tuple of sizes takes 0.4 us longer)


def forward_mxfp4(codes, scales, xcodes, xscales, m: int, n: int, k: int, y=None, out_dtype=None):
    """y[M][N] = Xv Wv^T of MXFP4 activations (xcodes, xscales: M rows) and weights (codes,
    scales: N rows), both of K columns, accumulated in fp32; y in ``out_dtype`` (fp32, or
    bf16), or in that of the given ``y``."""
    rt = _RT or _runtime()
    dev = codes.get_device()
    if dev < 0:
        raise ValueError("codes must be a GPU tensor")
    wc = _bytes_at_least(rt, codes, "codes", mxfp4_codes_bytes(n, k), dev)
    ws = _bytes_at_least(rt, scales, "scales", mxfp4_scales_bytes(n, k), dev)
    xc = _bytes_at_least(rt, xcodes, "xcodes", mxfp4_codes_bytes(m, k), dev)
    xs = _bytes_at_least(rt, xscales, "xscales", mxfp4_scales_bytes(m, k), dev)
    y, ydt = _product_output(rt, y, out_dtype, m, n, codes)
    _call(rt, rt.forward_mxfp4, dev, (wc, ws, xc, xs, m, n, k, y.data_ptr(), ydt))
    return y


def _named_dtype(name: str) -> int:
    """The bl_dtype of "f32" or "bf16"."""
    if name not in ("f32", "bf16"):
        raise ValueError(f'a type must be "f32" or "bf16", not {name!r}')
    return BL_BF16 if name == "bf16" else BL_F32


def forward_mxfp4_plan(m: int, n: int, k: int, x=None) -> dict:
    """The launches of forward_mxfp4 (``x`` None) or of forward_mxfp4_fused (``x`` "bf16" or "f32")
    for (M, N, K), computed on the host."""
    out = (ctypes.c_int32 * 6)()
    xdt = -1 if x is None else _named_dtype(x)
    _check("bitlinear_forward_mxfp4_plan", lib().bitlinear_forward_mxfp4_plan(m, n, k, xdt, out))
    return {"kernel": {7: "lds", 8: "decode", 9: "gemm"}[out[0]], "workgroups": out[1], "threads": out[2],
            "tokens": out[3], "outputs": out[4], "launches": out[5]}


def forward_mxfp4_fused_ws_bytes(m: int, n: int, k: int, dtype: str = "bf16") -> int:
    """Workspace bytes bitlinear_forward_mxfp4_fused needs for (M, N, K) and x of ``dtype`` "bf16"
    or "f32" (0: none)."""
    v = int(lib().bitlinear_forward_mxfp4_fused_ws_bytes(m, n, k, _named_dtype(dtype)))
    if v < 0:
        raise ValueError(f"invalid shape {(m, n, k)}")
    return v


def forward_mxfp4_fused(codes, scales, x, n: int, k: int, y=None, workspace=None, out_dtype=None):
    """Quantise x[M][K] (fp32 or bf16) to MXFP4 and apply MXFP4 weights (codes, scales: N
    rows) in one call; y[M][N] as forward_mxfp4.  A workspace of at least
    forward_mxfp4_fused_ws_bytes is allocated unless one is given."""
    rt = _RT or _runtime()
    dt = _require_rows(rt, x, "x")
    m, cols = x.shape
    if cols != k:
        raise ValueError("x must be [tokens, K]")
    dev = x.get_device()
    wc = _bytes_at_least(rt, codes, "codes", mxfp4_codes_bytes(n, k), dev)
    ws = _bytes_at_least(rt, scales, "scales", mxfp4_scales_bytes(n, k), dev)
    y, ydt = _product_output(rt, y, out_dtype, m, n, x)
    need = rt.fused_ws_bytes(m, n, k, dt)
    if workspace is not None:
        _bytes_at_least(rt, workspace, "workspace", need, dev)
    elif need > 0:
        workspace = rt.empty(need, dtype=rt.u8, device=x.device)
    _call(rt, rt.forward_mxfp4_fused, dev, (wc, ws, x.data_ptr(), dt, m, n, k, y.data_ptr(), ydt, _ptr(workspace),
                                            workspace.numel() if workspace is not None else 0))
    return y


def layernorm(x, weight=None, bias=None, eps: float = 1e-5, y=None, mean=None, rstd=None):
    """Layer normalisation of the rows of x[M][K] (fp32 or bf16) with fp32 weight and bias
    (None: ones, zeros).  Returns ``(y, mean fp32 [M], rstd fp32 [M])``; y has x's type.

    Like every call here it builds no autograd graph, also where an input requires a gradient:
    a training program takes the gradients from layernorm_backward."""
    rt = _RT or _runtime()
    dt = _require_rows(rt, x, "x")
    m, k = x.shape
    dev, f32, device = x.get_device(), rt.f32, x.device
    if weight is not None:
        _given(weight, "weight", (k,), f32, dev)
    if bias is not None:
        _given(bias, "bias", (k,), f32, dev)
    y = rt.empty_like(x) if y is None else _given(y, "y", (m, k), x.dtype, dev)
    mean = rt.empty(m, dtype=f32, device=device) if mean is None else _given(mean, "mean", (m,), f32, dev)
    rstd = rt.empty(m, dtype=f32, device=device) if rstd is None else _given(rstd, "rstd", (m,), f32, dev)
    _call(rt, rt.layernorm, dev, (x.data_ptr(), dt, m, k, _ptr(weight), _ptr(bias), eps, y.data_ptr(),
                                  mean.data_ptr(), rstd.data_ptr()))
    return y, mean, rstd


def layernorm_backward_ws_bytes(m: int, k: int) -> int:
    """Workspace bytes bitlinear_layernorm_backward needs for dweight and dbias of x[M][K]."""
    v = int(lib().bitlinear_layernorm_backward_ws_bytes(m, k))
    if v < 0:
        raise ValueError(f"invalid shape {(m, k)}")
    return v


def layernorm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None,
                       want_params: bool = True):
    """Gradients of layernorm: dy and x [M][K], weight fp32 [K] (None: ones), mean and rstd
    from the forward call.  Returns ``(dx, dweight, dbias)``, or ``dx`` alone with
    ``want_params=False``; dx has x's type, the others are fp32 and overwritten.  A workspace
    of at least layernorm_backward_ws_bytes is allocated unless one is given."""
    rt = _RT or _runtime()
    dt = _require_rows(rt, x, "x")
    m, k = x.shape
    dev, f32, device = x.get_device(), rt.f32, x.device
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward call are needed")
    _given(dy, "dy", (m, k), x.dtype, dev)
    _given(mean, "mean", (m,), f32, dev)
    _given(rstd, "rstd", (m,), f32, dev)
    if weight is not None:
        _given(weight, "weight", (k,), f32, dev)
    dx = rt.empty_like(x) if dx is None else _given(dx, "dx", (m, k), x.dtype, dev)
    if want_params:
        dweight = (rt.empty(k, dtype=f32, device=device) if dweight is None
                   else _given(dweight, "dweight", (k,), f32, dev))
        dbias = (rt.empty(k, dtype=f32, device=device) if dbias is None
                 else _given(dbias, "dbias", (k,), f32, dev))
        need = rt.backward_ws_bytes(m, k)
        if workspace is None:
            workspace = rt.empty(max(need, 0), dtype=rt.u8, device=device)
        else:
            _bytes_at_least(rt, workspace, "workspace", need, dev)
    else:
        dweight = dbias = workspace = None
    _call(rt, rt.layernorm_backward, dev,
          (dy.data_ptr(), x.data_ptr(), dt, m, k, _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
           _ptr(dweight), _ptr(dbias), _ptr(workspace), workspace.numel() if workspace is not None else 0))
    return (dx, dweight, dbias) if want_params else dx


ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4, "gelu_tanh": 5}


@functools.lru_cache(maxsize=4096)
def _products_plan(e: int, t: int, n: int, k: int, xdt: int):
    """out[0..5] of the plan calls (e = 0: one matrix); the rule goes by sizes and types alone."""
    out = (ctypes.c_int32 * 6)()
    if e:
        _check("bitlinear_forward_experts_plan", lib().bitlinear_forward_experts_plan(e, t, n, k, xdt, out))
    else:
        _check("bitlinear_forward_epilogue_plan", lib().bitlinear_forward_epilogue_plan(t, n, k, xdt, out))
    return tuple(out)


def _products_plan_dict(e: int, t: int, n: int, k: int, x) -> dict:
    out = _products_plan(e, t, n, k, -1 if x is None else _named_dtype(x))
    return {"kernel": {10: "fused", 11: "gemm", 12: "decode"}[out[0]], "workgroups": out[1], "threads": out[2], "rows": out[3],
            "outputs": out[4], "launches": out[5]}


def forward_epilogue_plan(m: int, n: int, k: int, x=None) -> dict:
    """The launches of forward_epilogue for (M, N, K) and an x of int8 codes (``x`` None), "bf16" or
    "f32", computed on the host."""
    return _products_plan_dict(0, m, n, k, x)


def forward_experts_plan(e: int, t: int, n: int, k: int, x=None) -> dict:
    """The launches of forward_experts for E experts and T slots, as forward_epilogue_plan."""
    if e < 1:
        raise ValueError("at least one expert")
    return _products_plan_dict(e, t, n, k, x)


def _strided(rt, t, name: str, rows: int, n: int, index: int):
    """(bl_dtype, row distance) of a [rows][n] matrix on the device whose rows are contiguous."""
    if t.get_device() != index or t.shape != (rows, n) or (n > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a [{rows}, {n}] tensor with contiguous rows on cuda:{index}")
    ld = t.stride(0) if rows > 1 else n
    if ld < n:
        raise ValueError(f"{name} must not have rows that overlap")
    return _dtype_code(rt, t.dtype, name), ld


def _vector(rt, t, name: str, shape, dtype, index: int) -> int:
    """The address of a contiguous tensor of this shape and type on the device."""
    if t.get_device() != index or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _tokens(rt, x, k: int, absmax, e: int, t, n: int):
    """The token rows x: (address of x or None, its bl_dtype, codes, scales, rows, what has to stay alive)."""
    dev = x.get_device()
    if x.dtype == rt.i8:
        if dev < 0 or x.dim() != 2 or not x.is_contiguous() or not x.numel() or x.shape[1] != (k + 255) // 256 * 256:
            raise ValueError("codes must be a non-empty contiguous [tokens, K_pad] GPU tensor")
        if absmax is None:
            raise ValueError("codes need their scales, absmax")
        r = x.shape[0]
        return None, 0, x.data_ptr(), _vector(rt, absmax, "absmax", (r,), rt.f32, dev), r, None
    if absmax is not None:
        raise ValueError("absmax goes with int8 codes")
    dt = _require_rows(rt, x, "x")
    r, cols = x.shape
    if cols != k:
        raise ValueError("x must be [tokens, K]")
    if n < 1 or _products_plan(e, r if t is None else t, n, k, dt)[5] == 1:
        return x.data_ptr(), dt, None, None, r, None
    codes = r * ((k + 255) // 256 * 256)
    scratch = rt.empty(codes + 4 * r, dtype=rt.u8, device=x.device)  # the codes, then the scales
    at = scratch.data_ptr()
    return x.data_ptr(), dt, at, at + codes, r, scratch


def _epilogue(rt, y, out_dtype, rows: int, n: int, like, bias, bias_shape, act: str, residual):
    """(y, its bl_epilogue)."""
    dev = like.get_device()
    if y is None:
        dtype = out_dtype or rt.f32
        ydt, yld = _dtype_code(rt, dtype, "out_dtype"), 0
        y = rt.empty(rows, max(n, 0), dtype=dtype, device=like.device)
    else:
        if out_dtype is not None and y.dtype != out_dtype:
            raise ValueError(f"y must be {out_dtype}")
        ydt, yld = _strided(rt, y, "y", rows, n, dev)
    rdt, rld, rptr = 0, 0, None
    if residual is not None:
        rdt, rld = _strided(rt, residual, "residual", rows, n, dev)
        rptr = residual.data_ptr()
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, not {act!r}")
    bptr = _vector(rt, bias, "bias", bias_shape, rt.f32, dev) if bias is not None else None
    return y, BlEpilogue(bptr, rptr, y.data_ptr(), rld, yld, code, rdt, ydt)


def forward_epilogue(packed, gamma, x, n: int, k: int, absmax=None, bias=None, act: str = "none", residual=None,
                     y=None, out_dtype=None):
    """y[M][N] = act(x W^T + bias) + residual in one call, for weights from quantize_weights.

    x: [M][K] fp32 or bf16, or the int8 codes [M][K_pad] with their scales ``absmax`` (quantize_acts).
    bias: fp32 [N].  act: a name of ``ACTIVATIONS``.  residual: [M][N] fp32 or bf16; it may be ``y``
    itself.  y: [M][N] in ``out_dtype`` (fp32, or bf16), or the given tensor; rows of y and residual
    may be parts of longer ones."""
    rt = _RT or _runtime()
    dev = x.get_device()
    wp = _bytes_at_least(rt, packed, "packed", (n + 15) // 16 * 4 * ((k + 255) // 256 * 256), dev)
    gp = _vector(rt, gamma, "gamma", (1,), rt.f32, dev)
    xp, dt, xq, a, m, keep = _tokens(rt, x, k, absmax, 0, None, n)
    y, ep = _epilogue(rt, y, out_dtype, m, n, x, bias, (n,), act, residual)
    _call(rt, rt.forward_epilogue, dev, (wp, gp, xp, dt, xq, a, m, n, k, ctypes.byref(ep)))
    return y


def _experts(rt, packed, gamma, offsets, rows, t: int, n: int, k: int, dev: int) -> BlExperts:
    e = gamma.shape[0] if gamma.dim() == 1 else 0
    if e < 1:
        raise ValueError("gamma must hold a scale per expert")
    wp = _bytes_at_least(rt, packed, "packed", e * ((n + 15) // 16 * 4 * ((k + 255) // 256 * 256)), dev)
    return BlExperts(wp, _vector(rt, gamma, "gamma", (e,), rt.f32, dev),
                     _vector(rt, offsets, "offsets", (e + 1,), rt.i32, dev),
                     _vector(rt, rows, "rows", (t,), rt.i32, dev) if rows is not None else None, e, t, n)


def quantize_expert_weights(W):
    """Ternary weights of E experts, W[E][N][K] fp32 on the GPU, each with its own scale: (packed uint8
    [E][packed_bytes], gamma fp32 [E])."""
    import torch

    _require_cuda(W, "W")
    if W.dim() != 3 or not W.numel():
        raise ValueError("W must be a non-empty [experts, N, K] tensor")
    e, n, k = W.shape
    packed = torch.empty((e, packed_bytes(n, k)), dtype=torch.uint8, device=W.device)
    gamma = torch.empty(e, dtype=torch.float32, device=W.device)
    workspace = torch.empty(wq_workspace_bytes(n, k), dtype=torch.uint8, device=W.device)
    for i in range(e):
        quantize_weights(W[i], packed[i], gamma[i:i + 1], workspace)
    return packed, gamma


def forward_experts(packed, gamma, offsets, x, n: int, k: int, rows=None, absmax=None, bias=None, act: str = "none",
                    residual=None, y=None, out_dtype=None):
    """Products grouped by expert: slot s of expert e (offsets[e] <= s < offsets[e + 1]) is token row
    rows[s] of x (row s without ``rows``) through matrix e; y[T][N] has a row per slot, with act, bias
    ([E][N]) and residual ([T][N]) as forward_epilogue.  Rows of slots without an expert, or with a row
    that x does not have, stay as they were.

    packed, gamma: quantize_expert_weights.  offsets, rows: int32 tables of route_experts."""
    rt = _RT or _runtime()
    dev = x.get_device()
    t = rows.shape[0] if rows is not None else x.shape[0]
    ex = _experts(rt, packed, gamma, offsets, rows, t, n, k, dev)
    xp, dt, xq, a, r, keep = _tokens(rt, x, k, absmax, ex.E, t, n)
    y, ep = _epilogue(rt, y, out_dtype, t, n, x, bias, (ex.E, n), act, residual)
    _call(rt, rt.forward_experts, dev, (ctypes.byref(ex), xp, dt, xq, a, r, k, ctypes.byref(ep)))
    return y


@functools.lru_cache(maxsize=4096)
def forward_experts_combine_ws_bytes(t: int, n: int) -> int:
    """Workspace bytes of forward_experts_combine for T slots of N outputs."""
    v = int(lib().bitlinear_forward_experts_combine_ws_bytes(t, n))
    if v < 0:
        raise ValueError(f"invalid shape {(t, n)}")
    return v


def forward_experts_combine(packed, gamma, offsets, x, n: int, k: int, slots, weights, rows=None, absmax=None,
                            bias=None, act: str = "none", residual=None, y=None, out_dtype=None, workspace=None):
    """forward_experts with the slots of each token added up: y[m] = residual[m] + sum_j weights[m][j]
    act(...) at slot slots[m][j] (-1: none).  slots int32 and weights fp32 [M][k] of route_experts."""
    rt = _RT or _runtime()
    dev = x.get_device()
    t = rows.shape[0] if rows is not None else x.shape[0]
    ex = _experts(rt, packed, gamma, offsets, rows, t, n, k, dev)
    if slots.dim() != 2 or not slots.numel():
        raise ValueError("slots must be a non-empty [tokens, choices] tensor")
    m, top = slots.shape
    sp = _vector(rt, slots, "slots", (m, top), rt.i32, dev)
    wt = _vector(rt, weights, "weights", (m, top), rt.f32, dev)
    xp, dt, xq, a, r, keep = _tokens(rt, x, k, absmax, ex.E, t, n)
    y, ep = _epilogue(rt, y, out_dtype, m, n, x, bias, (ex.E, n), act, residual)
    need = forward_experts_combine_ws_bytes(t, n)
    if workspace is None:
        workspace = rt.empty(need, dtype=rt.u8, device=x.device)
    ws = _bytes_at_least(rt, workspace, "workspace", need, dev)
    _call(rt, rt.forward_experts_combine, dev, (ctypes.byref(ex), xp, dt, xq, a, r, k, sp, wt, m, top,
                                                ctypes.byref(ep), ws, workspace.numel()))
    return y


class Route(NamedTuple):
    """What route_experts chose: experts and weights [M][k], and the slots by expert, then token:
    offsets [E + 1], rows [M k] (the token of each slot) and slots [M][k] (the slot of each choice)."""
    experts: object
    weights: object
    offsets: object
    rows: object
    slots: object


@functools.lru_cache(maxsize=4096)
def route_experts_ws_bytes(m: int, e: int) -> int:
    """Workspace bytes of route_experts for M tokens and E experts (0: none)."""
    v = int(lib().bitlinear_route_experts_ws_bytes(m, e))
    if v < 0:
        raise ValueError(f"invalid shape {(m, e)}")
    return v


def route_experts(logits, k: int, renormalize: bool = True, out: Route = None, workspace=None) -> Route:
    """The k largest of each token's logits[M][E] (fp32 or bf16; equal ones: the lowest index first),
    their weights (softmax over the chosen ones, or over all E without ``renormalize``), and the slots
    that forward_experts takes.  -inf and NaN are never chosen; missing choices are -1 with weight 0."""
    rt = _RT or _runtime()
    dt = _require_rows(rt, logits, "logits")
    m, e = logits.shape
    dev = logits.get_device()
    if out is None:
        if not 0 < k <= e:
            raise ValueError(f"k must be 1 .. {e}")
        new, on = rt.empty, logits.device
        out = Route(new(m, k, dtype=rt.i32, device=on), new(m, k, dtype=rt.f32, device=on),
                    new(e + 1, dtype=rt.i32, device=on), new(m * k, dtype=rt.i32, device=on),
                    new(m, k, dtype=rt.i32, device=on))
        ptrs = [t.data_ptr() for t in out]
    else:
        ptrs = [_vector(rt, t, name, shape, dtype, dev) for t, name, shape, dtype in zip(
            out, Route._fields, ((m, k), (m, k), (e + 1,), (m * k,), (m, k)), (rt.i32, rt.f32, rt.i32, rt.i32, rt.i32))]
    need = route_experts_ws_bytes(m, e)
    if workspace is not None:
        _bytes_at_least(rt, workspace, "workspace", need, dev)
    elif need > 0:
        workspace = rt.empty(need, dtype=rt.u8, device=logits.device)
    _call(rt, rt.route_experts, dev, (logits.data_ptr(), dt, m, e, k, int(bool(renormalize)), *ptrs, _ptr(workspace),
                                      workspace.numel() if workspace is not None else 0))
    return out
