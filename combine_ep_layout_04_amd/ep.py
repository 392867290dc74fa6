"""Python binding of libep.so (the C ABI in include/ep.h).

Argument marshalling only: every step of layout, dispatch and combine runs
in the HIP kernels behind the C ABI.  PyTorch provides device memory and
the stream.  There is no fallback: if the library is missing or a call
fails, an exception is raised.

Two levels, with the C names:

* ``lib()`` returns the raw ``ctypes`` handle whose functions take integer
  device addresses (``tensor.data_ptr()``) and a stream handle;
* ``ep_layout``, ``ep_dispatch``, ``ep_combine`` take torch tensors, check
  dtype / shape / device, allocate outputs with torch when not given, and
  launch on ``stream`` (default: torch's current stream).
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep.so")

EP_SUCCESS = 0
EP_INVALID_ARGUMENT = 1
EP_UNSUPPORTED = 2
EP_RUNTIME_ERROR = 3
EP_OUT_BF16 = 0
EP_OUT_FP8_E4M3 = 1
EP_OUT_FP8_E5M2 = 2
EP_SCALE_FP32 = 0
EP_SCALE_FP32_POW2 = 1
EP_SCALE_UE8M0 = 2
_FORMATS = {"e4m3": EP_OUT_FP8_E4M3, "e5m2": EP_OUT_FP8_E5M2}
_SCALES = {"fp32": EP_SCALE_FP32, "pow2": EP_SCALE_FP32_POW2, "ue8m0": EP_SCALE_UE8M0}
EP_MAX_EXPERTS = 1024
EP_MAX_TOPK = 64
EP_MAX_HIDDEN = 65536
EP_MAX_ALIGNMENT = 4096
EP_MAX_RANKS = 64
EP_MAX_GROUPS = 64
EP_MAX_W4_ROWS = 1 << 20
EP_MAX_OUT_FEATURES = 1 << 20
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # ep_dtype_t
_SCORES = {"softmax": 0, "sigmoid": 1}

# every symbol include/ep.h declares
SYMBOLS = ("ep_version", "ep_status_string", "ep_last_error", "ep_layout_workspace_size",
           "ep_layout", "ep_layout_noalloc", "ep_layout_ex", "ep_layout_max_rows", "ep_dispatch", "ep_dispatch_ex",
           "ep_dispatch_prequantized", "ep_combine",
           "ep_combine_backward", "ep_dispatch_backward", "ep_routing_map",
           "ep_rank_layout_workspace_size", "ep_rank_layout", "ep_dispatch_ranked",
           "ep_dispatch_ranked_prequantized", "ep_dispatch_ranked_fp8", "ep_dispatch_fused_permute",
           "ep_dispatch_fused_permute_prequantized", "ep_combine_ranked",
           "ep_dispatch_ranked_backward", "ep_dispatch_colmajor_workspace_size",
           "ep_dispatch_colmajor_scales", "ep_dispatch_prequantized_colmajor",
           "ep_router", "ep_router_backward", "ep_permute", "ep_permute_backward", "ep_unpermute",
           "ep_unpermute_backward", "ep_w4_packed_size", "ep_w4_pack", "ep_expert_matmul_w4",
           "ep_expert_matmul", "ep_expert_glu", "ep_expert_matmul_backward",
           "ep_expert_backward_workspace_size", "ep_expert_glu_backward", "ep_expert_matmul_fp8")


class EpError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}: {message}")


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libep.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m combine_ep_layout_04_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.ep_version.argtypes = []
        L.ep_version.restype = i32
        L.ep_status_string.argtypes = [i32]
        L.ep_status_string.restype = ctypes.c_char_p
        L.ep_last_error.argtypes = []
        L.ep_last_error.restype = ctypes.c_char_p
        L.ep_layout_workspace_size.argtypes = [i64, i32, i32]
        L.ep_layout_workspace_size.restype = sz
        L.ep_layout.argtypes = [P, i64, i32, i32, P, P, P, P, P, P, sz, P]
        L.ep_layout.restype = i32
        L.ep_layout_noalloc.argtypes = [P, i64, i32, i32, P, P, P, P, P, P]
        L.ep_layout_noalloc.restype = i32
        L.ep_layout_ex.argtypes = [P, i64, i32, i32, i32, i64, P, P, P, P, P, P, P, sz, P]
        L.ep_layout_ex.restype = i32
        L.ep_layout_max_rows.argtypes = [i64, i32, i32, i32, i64]
        L.ep_layout_max_rows.restype = i64
        L.ep_dispatch.argtypes = [P, i64, i32, i32, P, P, i32, P, P, P, P]
        L.ep_dispatch.restype = i32
        L.ep_dispatch_ex.argtypes = [P, i64, i32, i32, P, P, i32, i32, P, P, P, i64, P]
        L.ep_dispatch_ex.restype = i32
        L.ep_dispatch_colmajor_workspace_size.argtypes = [i64, i32, i32]
        L.ep_dispatch_colmajor_workspace_size.restype = sz
        L.ep_dispatch_colmajor_scales.argtypes = [P, i64, i32, i32, P, P, P, i32, i32, P, P, P, i64,
                                                  i64, P, sz, P]
        L.ep_dispatch_colmajor_scales.restype = i32
        L.ep_dispatch_prequantized.argtypes = [P, P, i64, i32, i32, P, P, P, P, P, i64, P]
        L.ep_dispatch_prequantized.restype = i32
        L.ep_dispatch_prequantized_colmajor.argtypes = [P, P, i64, i32, i32, P, P, P, P, P, P, i64,
                                                        i64, P]
        L.ep_dispatch_prequantized_colmajor.restype = i32
        L.ep_combine.argtypes = [P, P, P, i64, i32, i32, P, P]
        L.ep_combine.restype = i32
        L.ep_combine_backward.argtypes = [P, P, P, P, i64, i32, i32, P, P, P]
        L.ep_combine_backward.restype = i32
        L.ep_dispatch_backward.argtypes = [P, P, P, i64, i32, i32, P, P, P]
        L.ep_dispatch_backward.restype = i32
        L.ep_routing_map.argtypes = [P, i64, i32, i32, P, P, P]
        L.ep_routing_map.restype = i32
        L.ep_rank_layout_workspace_size.argtypes = [i64, i32, i32]
        L.ep_rank_layout_workspace_size.restype = sz
        L.ep_rank_layout.argtypes = [P, i64, i32, i32, i32, i32, P, P, P, P, P, P, P, P, sz, P]
        L.ep_rank_layout.restype = i32
        L.ep_dispatch_ranked.argtypes = [P, P, P, i64, i32, i32, i32, i32, P, P, P, i64, P]
        L.ep_dispatch_ranked.restype = i32
        L.ep_dispatch_ranked_prequantized.argtypes = [P, P, P, P, i64, i32, i32, i32, i32, P, P, P,
                                                      P, i64, P]
        L.ep_dispatch_ranked_prequantized.restype = i32
        L.ep_dispatch_ranked_fp8.argtypes = [P, P, P, i64, i32, i32, i32, i32, P, i32, i32, P, P,
                                             P, i64, P]
        L.ep_dispatch_ranked_fp8.restype = i32
        L.ep_dispatch_fused_permute.argtypes = [P, P, P, i64, i32, i32, i32, i32, i32, P, P, P, P,
                                                i64, P, P, P]
        L.ep_dispatch_fused_permute.restype = i32
        L.ep_dispatch_fused_permute_prequantized.argtypes = [P, P, P, P, i64, i32, i32, i32, i32,
                                                             i32, P, P, P, P, i64, P, P, P, P]
        L.ep_dispatch_fused_permute_prequantized.restype = i32
        L.ep_combine_ranked.argtypes = [P, i64, P, i64, i32, i32, P, P]
        L.ep_combine_ranked.restype = i32
        L.ep_dispatch_ranked_backward.argtypes = [P, P, i64, P, P, i64, i32, i32, i32, i32, P, P,
                                                  P]
        L.ep_dispatch_ranked_backward.restype = i32
        f32 = ctypes.c_float
        L.ep_router.argtypes = [P, i32, i64, i32, i64, i32, i32, P, i32, i32, i32, i32, f32, P, P,
                                P, P]
        L.ep_router.restype = i32
        L.ep_router_backward.argtypes = [P, i32, i64, i32, i64, i32, i32, i32, f32, P, P, P, P, P]
        L.ep_router_backward.restype = i32
        L.ep_permute.argtypes = [P, i32, i64, i32, i64, i32, P, P, P, i64, i64, P, P, i32, P]
        L.ep_permute.restype = i32
        L.ep_permute_backward.argtypes = [P, i32, i64, i32, i64, i64, i32, P, P, P, i64, P, i64, P,
                                          P]
        L.ep_permute_backward.restype = i32
        L.ep_unpermute.argtypes = [P, i32, i64, i32, i64, i64, i32, P, P, P, i64, P]
        L.ep_unpermute.restype = i32
        L.ep_unpermute_backward.argtypes = [P, i32, i64, i32, i64, i32, P, P, P, i64, P, i64, i64,
                                            P, P, P, i32, P]
        L.ep_unpermute_backward.restype = i32
        L.ep_w4_packed_size.argtypes = [i32, i32, i32, i32, i32, i32]
        L.ep_w4_packed_size.restype = sz
        L.ep_w4_pack.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, P, sz, P]
        L.ep_w4_pack.restype = i32
        L.ep_expert_matmul_w4.argtypes = [P, i32, i64, i64, P, P, sz, i32, i32, i32, i32, i32, i32,
                                          P, P, i64, P, i64, P]
        L.ep_expert_matmul_w4.restype = i32
        L.ep_expert_matmul.argtypes = [P, i32, i64, i64, P, P, i32, i32, i32, P, P, i64, P, i64, P]
        L.ep_expert_matmul.restype = i32
        L.ep_expert_glu.argtypes = [P, i32, i64, i64, P, P, i32, i32, i32, P, P, i64, P, i64, P, i64,
                                    P]
        L.ep_expert_glu.restype = i32
        L.ep_expert_matmul_backward.argtypes = [P, i32, i64, P, i64, i64, P, P, i32, i32, i32, P, P,
                                                i64, P, i64, P, i32, P, sz, P]
        L.ep_expert_matmul_backward.restype = i32
        L.ep_expert_backward_workspace_size.argtypes = [i64, i32, i32, i32, i32]
        L.ep_expert_backward_workspace_size.restype = sz
        L.ep_expert_glu_backward.argtypes = [P, i32, i64, P, i64, P, i64, i64, P, P, i32, i32, i32, P,
                                             P, i64, P, i64, P, i32, P, sz, P]
        L.ep_expert_glu_backward.restype = i32
        L.ep_expert_matmul_fp8.argtypes = [P, i32, i64, i64, P, i32, i64, i64, P, P, P, i32, i32, i32,
                                           i32, P, P, i64, P, i32, i64, P]
        L.ep_expert_matmul_fp8.restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ep_status_string(int(status)).decode()


def last_error() -> str:
    return lib().ep_last_error().decode()


def version() -> int:
    return int(lib().ep_version())


def layout_workspace_size(num_tokens: int, num_topk: int, num_experts: int) -> int:
    return int(lib().ep_layout_workspace_size(int(num_tokens), int(num_topk), int(num_experts)))


def layout_max_rows(num_tokens: int, num_topk: int, num_experts: int, alignment: int = 1,
                    capacity: int = 0) -> int:
    """Rows a receive buffer needs for any routing of this shape (-1 if the
    arguments are invalid)."""
    return int(lib().ep_layout_max_rows(int(num_tokens), int(num_topk), int(num_experts),
                                        int(alignment), int(capacity)))


def _check(status: int, where: str) -> None:
    if status != EP_SUCCESS:
        raise EpError(status, where, last_error())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, numel: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")


# ------------------------------------------------------------------ layout --

def ep_layout(topk_idx: torch.Tensor, num_experts: int, *, alignment: int = 1, capacity: int = 0,
              counts=None, offsets=None, slot=None, src=None, num_invalid=None,
              num_dropped=None, workspace=None, want_src: bool = True,
              want_invalid: bool = True, stream=None):
    """Routing layout of ``topk_idx`` (int64 [T, k], -1 = masked).

    ``alignment`` / ``capacity`` select ep_layout_ex's segment placement
    (packed segments starting on multiples of ``alignment``, or a fixed
    ``capacity`` rows per expert with overflow dropped).

    Returns (counts int32 [E], offsets int32 [E+1], slot int32 [T, k],
    src int32 [rows] or None, num_invalid int32 [1] or None); with a
    capacity, ``num_dropped`` (int32 [1]) is filled when given.  ``rows`` is
    layout_max_rows(...).
    """
    _need(topk_idx, "topk_idx", torch.int64)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be 2-D [num_tokens, num_topk]")
    T, k = topk_idx.shape
    E = int(num_experts)
    rows = layout_max_rows(T, k, E, alignment, capacity)
    if rows < 0:
        raise ValueError("invalid layout shape, alignment or capacity")
    dev = topk_idx.device
    i32 = dict(dtype=torch.int32, device=dev)
    counts = torch.empty(E, **i32) if counts is None else counts
    offsets = torch.empty(E + 1, **i32) if offsets is None else offsets
    slot = torch.empty((T, k), **i32) if slot is None else slot
    if want_src and src is None:
        src = torch.empty(max(rows, 1), **i32)
    if want_invalid and num_invalid is None:
        num_invalid = torch.empty(1, **i32)
    need = layout_workspace_size(T, k, E)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need(counts, "counts", torch.int32, E)
    _need(offsets, "offsets", torch.int32, E + 1)
    _need(slot, "slot", torch.int32, T * k)
    if src is not None:
        _need(src, "src", torch.int32, rows)
    if num_invalid is not None:
        _need(num_invalid, "num_invalid", torch.int32, 1)
    if num_dropped is not None:
        _need(num_dropped, "num_dropped", torch.int32, 1)
    _need(workspace, "workspace", torch.uint8)
    if alignment == 1 and capacity == 0 and num_dropped is None:
        st = lib().ep_layout(_ptr(topk_idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(slot),
                             _ptr(src), _ptr(num_invalid), _ptr(workspace), workspace.numel(),
                             _stream(stream))
    else:
        st = lib().ep_layout_ex(_ptr(topk_idx), T, k, E, int(alignment), int(capacity),
                                _ptr(counts), _ptr(offsets), _ptr(slot), _ptr(src),
                                _ptr(num_invalid), _ptr(num_dropped), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check(st, "ep_layout")
    return counts, offsets, slot, src, num_invalid


def ep_layout_noalloc(topk_idx: torch.Tensor, num_experts: int, counts: torch.Tensor,
                      offsets: torch.Tensor, slot: torch.Tensor, src: Optional[torch.Tensor] = None,
                      num_invalid: Optional[torch.Tensor] = None, stream=None):
    """ep_layout with the library's fixed per-device scratch: no workspace,
    and nothing allocated here or in the library (every output is the
    caller's).  Outputs as ep_layout; returns them."""
    _need(topk_idx, "topk_idx", torch.int64)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be 2-D [num_tokens, num_topk]")
    T, k = topk_idx.shape
    E = int(num_experts)
    _need(counts, "counts", torch.int32, E)
    _need(offsets, "offsets", torch.int32, E + 1)
    _need(slot, "slot", torch.int32, T * k)
    if src is not None:
        _need(src, "src", torch.int32, T * k)
    if num_invalid is not None:
        _need(num_invalid, "num_invalid", torch.int32, 1)
    st = lib().ep_layout_noalloc(_ptr(topk_idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(slot),
                                 _ptr(src), _ptr(num_invalid), _stream(stream))
    _check(st, "ep_layout_noalloc")
    return counts, offsets, slot, src, num_invalid


# ---------------------------------------------------------------- dispatch --

def ep_dispatch(x: torch.Tensor, slot: torch.Tensor, topk_weights: Optional[torch.Tensor] = None,
                *, fp8: bool = False, fmt: str = "e4m3", scale: str = "fp32", recv_x=None,
                recv_scales=None, recv_weights=None,
                want_weights: bool = False, rows: Optional[int] = None,
                trust_slots: bool = False, scale_ld: int = 0, stream=None):
    """Permute (bf16) or cast (fp8 e4m3 + per-128 fp32 scales) the rows of
    ``x`` (bf16 [T, H]) into the expert-grouped buffer named by ``slot``.

    With ``fp8`` the cast format is ``fmt`` ("e4m3" / "e5m2") and the scale
    ``scale`` ("fp32", "pow2", "ue8m0" -- the last gives uint8 scales);
    ``scale_ld`` > 0 stores the scales column-major, [H/128, scale_ld]
    (scale_ld >= rows, a multiple of 4 fp32 / 16 UE8M0 scales).

    Returns (recv_x, recv_scales or None, recv_weights or None); recv_x is
    bf16 [rows, H] or uint8 [rows, H].  ``rows`` is the layout's row bound
    (layout_max_rows; T*k for the compact layout) and output buffers given
    by the caller must hold that many, unless ``trust_slots`` says the
    caller knows every slot is below the rows it passed.
    """
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [num_tokens, hidden]")
    T, H = x.shape
    _need(slot, "slot", torch.int32)
    if slot.dim() != 2 or slot.shape[0] != T:
        raise ValueError("slot must be 2-D [num_tokens, num_topk]")
    k = slot.shape[1]
    R = T * k if rows is None else int(rows)
    dev = x.device
    if recv_x is None:
        recv_x = torch.empty((R, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    sdt = torch.uint8 if scale == "ue8m0" else torch.float32
    nb = H // 128
    if scale_ld:
        if scale_ld < R:
            raise ValueError(f"scale_ld {scale_ld} is below the layout's {R} rows")
    if fp8 and recv_scales is None:
        recv_scales = torch.empty((nb, scale_ld) if scale_ld else (R, nb), dtype=sdt, device=dev)
    if want_weights and recv_weights is None:
        recv_weights = torch.empty(R, dtype=torch.float32, device=dev)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    cap = 0 if trust_slots else R
    _need(recv_x, "recv_x", torch.uint8 if fp8 else torch.bfloat16, cap * H)
    if recv_x.shape[-1] != H:
        raise ValueError("recv_x rows must have hidden elements")
    if recv_scales is not None:
        _need(recv_scales, "recv_scales", sdt, nb * scale_ld if scale_ld else cap * nb)
    if recv_weights is not None:
        _need(recv_weights, "recv_weights", torch.float32, cap)
    st = lib().ep_dispatch_ex(_ptr(x), T, H, k, _ptr(slot), _ptr(topk_weights),
                              _FORMATS[fmt] if fp8 else EP_OUT_BF16,
                              _SCALES[scale] if fp8 else EP_SCALE_FP32, _ptr(recv_x),
                              _ptr(recv_scales), _ptr(recv_weights), int(scale_ld),
                              _stream(stream))
    _check(st, "ep_dispatch")
    return recv_x, recv_scales, recv_weights


def ep_dispatch_colmajor_workspace_size(num_tokens: int, hidden: int, scale: str = "fp32") -> int:
    return int(lib().ep_dispatch_colmajor_workspace_size(int(num_tokens), int(hidden), _SCALES[scale]))


def ep_dispatch_colmajor_scales(x: torch.Tensor, slot: torch.Tensor, src: torch.Tensor,
                                topk_weights: Optional[torch.Tensor] = None, *, fmt: str = "e4m3",
                                scale: str = "fp32", scale_ld: int, rows: Optional[int] = None,
                                recv_x=None, recv_scales=None, recv_weights=None,
                                want_weights: bool = False, workspace=None, stream=None):
    """The 8-bit cast with column-major scales [H/128, scale_ld] written in
    two passes through a workspace (allocated here with torch when not
    given).  ``src`` is the layout's int32 source token of each of the
    ``rows`` receive rows (T*k by default).  Returns (recv_x uint8 [rows, H],
    recv_scales, recv_weights or None)."""
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [num_tokens, hidden]")
    T, H = x.shape
    _need(slot, "slot", torch.int32)
    if slot.dim() != 2 or slot.shape[0] != T:
        raise ValueError("slot must be 2-D [num_tokens, num_topk]")
    k = slot.shape[1]
    R = T * k if rows is None else int(rows)
    if scale_ld < R:
        raise ValueError(f"scale_ld {scale_ld} is below the {R} rows")
    _need(src, "src", torch.int32, R)
    dev = x.device
    sdt = torch.uint8 if scale == "ue8m0" else torch.float32
    nb = H // 128
    if recv_x is None:
        recv_x = torch.empty((R, H), dtype=torch.uint8, device=dev)
    if recv_scales is None:
        recv_scales = torch.empty((nb, scale_ld), dtype=sdt, device=dev)
    if want_weights and recv_weights is None:
        recv_weights = torch.empty(R, dtype=torch.float32, device=dev)
    need = ep_dispatch_colmajor_workspace_size(T, H, scale)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need(recv_x, "recv_x", torch.uint8, R * H)
    _need(recv_scales, "recv_scales", sdt, nb * scale_ld)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    if recv_weights is not None:
        _need(recv_weights, "recv_weights", torch.float32, R)
    _need(workspace, "workspace", torch.uint8)
    st = lib().ep_dispatch_colmajor_scales(_ptr(x), T, H, k, _ptr(slot), _ptr(src),
                                           _ptr(topk_weights), _FORMATS[fmt], _SCALES[scale],
                                           _ptr(recv_x), _ptr(recv_scales), _ptr(recv_weights),
                                           int(scale_ld), R, _ptr(workspace), workspace.numel(),
                                           _stream(stream))
    _check(st, "ep_dispatch_colmajor_scales")
    return recv_x, recv_scales, recv_weights


def ep_dispatch_prequantized(x_q: torch.Tensor, x_scales: torch.Tensor, slot: torch.Tensor,
                             topk_weights: Optional[torch.Tensor] = None, *, recv_q=None,
                             recv_scales=None, recv_weights=None, want_weights: bool = False,
                             rows: Optional[int] = None, scale_ld: int = 0, stream=None):
    """Copy pre-quantized rows (uint8 [T, H]) and their fp32 scales
    ([T, H/128]) to the expert-grouped buffer (scales column-major
    [H/128, scale_ld] when scale_ld > 0).  Returns (recv_q, recv_scales,
    recv_weights or None)."""
    _need(x_q, "x_q", torch.uint8)
    _need(x_scales, "x_scales", torch.float32)
    _need(slot, "slot", torch.int32)
    if x_q.dim() != 2 or slot.dim() != 2 or slot.shape[0] != x_q.shape[0]:
        raise ValueError("x_q must be [T, H] and slot [T, k]")
    T, H = x_q.shape
    k = slot.shape[1]
    if x_scales.numel() < T * (H // 128):
        raise ValueError("x_scales must hold T * H/128 values")
    R = T * k if rows is None else int(rows)
    dev = x_q.device
    if recv_q is None:
        recv_q = torch.empty((R, H), dtype=torch.uint8, device=dev)
    nb = H // 128
    if scale_ld and scale_ld < R:
        raise ValueError(f"scale_ld {scale_ld} is below the layout's {R} rows")
    if recv_scales is None:
        recv_scales = torch.empty((nb, scale_ld) if scale_ld else (R, nb), dtype=torch.float32,
                                  device=dev)
    if want_weights and recv_weights is None:
        recv_weights = torch.empty(R, dtype=torch.float32, device=dev)
    _need(recv_q, "recv_q", torch.uint8, R * H)
    _need(recv_scales, "recv_scales", torch.float32, nb * scale_ld if scale_ld else R * nb)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    if recv_weights is not None:
        _need(recv_weights, "recv_weights", torch.float32, R)
    st = lib().ep_dispatch_prequantized(_ptr(x_q), _ptr(x_scales), T, H, k, _ptr(slot),
                                        _ptr(topk_weights), _ptr(recv_q), _ptr(recv_scales),
                                        _ptr(recv_weights), int(scale_ld), _stream(stream))
    _check(st, "ep_dispatch_prequantized")
    return recv_q, recv_scales, recv_weights


def ep_dispatch_prequantized_colmajor(x_q: torch.Tensor, x_scales: torch.Tensor,
                                      slot: torch.Tensor, src: torch.Tensor,
                                      topk_weights: Optional[torch.Tensor] = None, *,
                                      scale_ld: int, rows: Optional[int] = None, recv_q=None,
                                      recv_scales=None, recv_weights=None,
                                      want_weights: bool = False, stream=None):
    """The pre-quantized copy with column-major scales [H/128, scale_ld]
    written in two passes (the code rows, then the scale columns from
    x_scales).  ``src`` is the layout's int32 source token of each of the
    ``rows`` receive rows (T*k by default).  Returns (recv_q, recv_scales,
    recv_weights or None)."""
    _need(x_q, "x_q", torch.uint8)
    _need(x_scales, "x_scales", torch.float32)
    _need(slot, "slot", torch.int32)
    if x_q.dim() != 2 or slot.dim() != 2 or slot.shape[0] != x_q.shape[0]:
        raise ValueError("x_q must be [T, H] and slot [T, k]")
    T, H = x_q.shape
    k = slot.shape[1]
    nb = H // 128
    if x_scales.numel() < T * nb:
        raise ValueError("x_scales must hold T * H/128 values")
    R = T * k if rows is None else int(rows)
    if scale_ld < R:
        raise ValueError(f"scale_ld {scale_ld} is below the {R} rows")
    _need(src, "src", torch.int32, R)
    dev = x_q.device
    if recv_q is None:
        recv_q = torch.empty((R, H), dtype=torch.uint8, device=dev)
    if recv_scales is None:
        recv_scales = torch.empty((nb, scale_ld), dtype=torch.float32, device=dev)
    if want_weights and recv_weights is None:
        recv_weights = torch.empty(R, dtype=torch.float32, device=dev)
    _need(recv_q, "recv_q", torch.uint8, R * H)
    _need(recv_scales, "recv_scales", torch.float32, nb * scale_ld)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    if recv_weights is not None:
        _need(recv_weights, "recv_weights", torch.float32, R)
    st = lib().ep_dispatch_prequantized_colmajor(_ptr(x_q), _ptr(x_scales), T, H, k, _ptr(slot),
                                                 _ptr(src), _ptr(topk_weights), _ptr(recv_q),
                                                 _ptr(recv_scales), _ptr(recv_weights),
                                                 int(scale_ld), R, _stream(stream))
    _check(st, "ep_dispatch_prequantized_colmajor")
    return recv_q, recv_scales, recv_weights


# ----------------------------------------------------------------- combine --

def ep_combine(y: torch.Tensor, slot: torch.Tensor, topk_weights: Optional[torch.Tensor],
               *, out=None, rows: Optional[int] = None, trust_slots: bool = False,
               stream=None) -> torch.Tensor:
    """out[t] = bf16(sum_j w[t,j] * y[slot[t,j]]) for y bf16 [rows, H] and
    slot int32 [T, k]; ``topk_weights`` None means unit weights.  y must
    hold ``rows`` rows (the layout's bound, T*k by default) unless
    ``trust_slots`` says every slot is below its rows."""
    _need(y, "y", torch.bfloat16)
    _need(slot, "slot", torch.int32)
    if slot.dim() != 2 or y.dim() != 2:
        raise ValueError("slot must be [num_tokens, num_topk] and y [rows, hidden]")
    T, k = slot.shape
    H = y.shape[-1]
    R = T * k if rows is None else int(rows)
    if not trust_slots and y.shape[0] < R:
        raise ValueError(f"y has {y.shape[0]} rows, the layout may use {R}")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _need(out, "out", torch.bfloat16, T * H)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    st = lib().ep_combine(_ptr(y), _ptr(slot), _ptr(topk_weights), T, H, k, _ptr(out),
                          _stream(stream))
    _check(st, "ep_combine")
    return out


# ---------------------------------------------------------------- backward --

def ep_combine_backward(grad_out: torch.Tensor, y: Optional[torch.Tensor], slot: torch.Tensor,
                        topk_weights: Optional[torch.Tensor], *, grad_y=None,
                        grad_topk_weights=None, want_weight_grad: bool = True,
                        rows: Optional[int] = None, stream=None):
    """Gradients of ep_combine: returns (grad_y bf16 [rows, H],
    grad_topk_weights fp32 [T, k] or None).  The weight gradient needs y."""
    _need(grad_out, "grad_out", torch.bfloat16)
    _need(slot, "slot", torch.int32)
    if slot.dim() != 2 or grad_out.dim() != 2 or slot.shape[0] != grad_out.shape[0]:
        raise ValueError("grad_out must be [T, H] and slot [T, k]")
    T, H = grad_out.shape
    k = slot.shape[1]
    R = T * k if rows is None else int(rows)
    if grad_y is None:
        grad_y = torch.empty((R, H), dtype=torch.bfloat16, device=grad_out.device)
    _need(grad_y, "grad_y", torch.bfloat16, R * H)
    if y is not None:
        _need(y, "y", torch.bfloat16, R * H)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    if want_weight_grad and y is not None and grad_topk_weights is None:
        grad_topk_weights = torch.empty((T, k), dtype=torch.float32, device=grad_out.device)
    if grad_topk_weights is not None:
        _need(grad_topk_weights, "grad_topk_weights", torch.float32, T * k)
    st = lib().ep_combine_backward(_ptr(grad_out), _ptr(y), _ptr(slot), _ptr(topk_weights), T, H, k,
                                   _ptr(grad_y), _ptr(grad_topk_weights), _stream(stream))
    _check(st, "ep_combine_backward")
    return grad_y, grad_topk_weights


def ep_dispatch_backward(grad_recv: torch.Tensor, grad_recv_weights: Optional[torch.Tensor],
                         slot: torch.Tensor, *, grad_x=None, grad_topk_weights=None,
                         rows: Optional[int] = None, stream=None):
    """Gradients of ep_dispatch: returns (grad_x bf16 [T, H],
    grad_topk_weights fp32 [T, k] or None)."""
    _need(grad_recv, "grad_recv", torch.bfloat16)
    _need(slot, "slot", torch.int32)
    if slot.dim() != 2 or grad_recv.dim() != 2:
        raise ValueError("slot must be [T, k] and grad_recv [rows, H]")
    T, k = slot.shape
    H = grad_recv.shape[1]
    R = T * k if rows is None else int(rows)
    if grad_recv.shape[0] < R:
        raise ValueError(f"grad_recv has {grad_recv.shape[0]} rows, the layout may use {R}")
    if grad_x is None:
        grad_x = torch.empty((T, H), dtype=torch.bfloat16, device=grad_recv.device)
    _need(grad_x, "grad_x", torch.bfloat16, T * H)
    if grad_recv_weights is not None:
        _need(grad_recv_weights, "grad_recv_weights", torch.float32, R)
        if grad_topk_weights is None:
            grad_topk_weights = torch.empty((T, k), dtype=torch.float32, device=grad_recv.device)
        _need(grad_topk_weights, "grad_topk_weights", torch.float32, T * k)
    st = lib().ep_dispatch_backward(_ptr(grad_recv), _ptr(grad_recv_weights), _ptr(slot), T, H, k,
                                    _ptr(grad_x), _ptr(grad_topk_weights), _stream(stream))
    _check(st, "ep_dispatch_backward")
    return grad_x, grad_topk_weights


# ------------------------------------------------- per-(token, rank) path --

def ep_routing_map(topk_idx: torch.Tensor, num_experts: int, *, routing_map=None,
                   num_invalid=None, want_invalid: bool = True, stream=None):
    """Routing bitmap of ``topk_idx`` (int64 [T, k]): uint8 [T, ceil(E/8)],
    bit e % 8 of byte e // 8 set iff the token selects expert e.  Returns
    (routing_map, num_invalid int32 [1] or None)."""
    _need(topk_idx, "topk_idx", torch.int64)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be 2-D [num_tokens, num_topk]")
    T, k = topk_idx.shape
    E = int(num_experts)
    W = (E + 7) // 8
    dev = topk_idx.device
    if routing_map is None:
        routing_map = torch.empty((T, W), dtype=torch.uint8, device=dev)
    _need(routing_map, "routing_map", torch.uint8, T * W)
    if want_invalid and num_invalid is None:
        num_invalid = torch.empty(1, dtype=torch.int32, device=dev)
    if num_invalid is not None:
        _need(num_invalid, "num_invalid", torch.int32, 1)
    st = lib().ep_routing_map(_ptr(topk_idx), T, k, E, _ptr(routing_map), _ptr(num_invalid),
                              _stream(stream))
    _check(st, "ep_routing_map")
    return routing_map, num_invalid


def rank_layout_workspace_size(tokens_per_rank: int, num_experts: int, num_ranks: int) -> int:
    return int(lib().ep_rank_layout_workspace_size(int(tokens_per_rank), int(num_experts),
                                                   int(num_ranks)))


class RankLayout:
    """Outputs of :func:`ep_rank_layout` (device tensors)."""

    FIELDS = ("sparse_to_dense", "local_map", "recv_src", "recv_topk_idx", "expert_counts",
              "num_recv", "num_overflow")

    def __init__(self, **kw):
        self.__dict__.update(kw)


def ep_rank_layout(global_map: torch.Tensor, tokens_per_rank: int, num_experts: int,
                   num_ranks: int, rank: int, k_out: int, *, out: Optional[RankLayout] = None,
                   workspace=None, stream=None) -> RankLayout:
    """Metadata preprocessing of rank ``rank`` from the all-gathered routing
    map (uint8 [G*T, ceil(E/8)]).  Returns a RankLayout with
    sparse_to_dense int32 [T, G], local_map uint8 [G*T, E/G], recv_src int32
    [G*T], recv_topk_idx int64 [G*T, k_out], expert_counts int32 [E/G],
    num_recv int32 [1], num_overflow int32 [1]."""
    T, E, G = int(tokens_per_rank), int(num_experts), int(num_ranks)
    if G < 1 or E % G:
        raise ValueError("num_experts must be a multiple of num_ranks")
    El = E // G
    R = G * T
    W = (E + 7) // 8
    _need(global_map, "global_map", torch.uint8, R * W)
    dev = global_map.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = RankLayout(sparse_to_dense=torch.empty((T, G), **i32),
                         local_map=torch.empty((R, El), dtype=torch.uint8, device=dev),
                         recv_src=torch.empty(R, **i32),
                         recv_topk_idx=torch.empty((R, int(k_out)), dtype=torch.int64, device=dev),
                         expert_counts=torch.empty(El, **i32), num_recv=torch.empty(1, **i32),
                         num_overflow=torch.empty(1, **i32))
    _need(out.sparse_to_dense, "sparse_to_dense", torch.int32, T * G)
    _need(out.local_map, "local_map", torch.uint8, R * El)
    _need(out.recv_src, "recv_src", torch.int32, R)
    _need(out.recv_topk_idx, "recv_topk_idx", torch.int64, R * int(k_out))
    _need(out.expert_counts, "expert_counts", torch.int32, El)
    _need(out.num_recv, "num_recv", torch.int32, 1)
    if out.num_overflow is not None:
        _need(out.num_overflow, "num_overflow", torch.int32, 1)
    need = rank_layout_workspace_size(T, E, G)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8)
    st = lib().ep_rank_layout(_ptr(global_map), T, E, G, int(rank), int(k_out),
                              _ptr(out.sparse_to_dense), _ptr(out.local_map), _ptr(out.recv_src),
                              _ptr(out.recv_topk_idx), _ptr(out.expert_counts), _ptr(out.num_recv),
                              _ptr(out.num_overflow), _ptr(workspace), workspace.numel(),
                              _stream(stream))
    _check(st, "ep_rank_layout")
    return out


def _ptr_table(tensors):
    arr = (ctypes.c_void_p * len(tensors))(*[None if t is None else t.data_ptr() for t in tensors])
    return arr, ctypes.addressof(arr)


def ep_dispatch_ranked(x: torch.Tensor, sparse_to_dense: torch.Tensor, dest_x, num_experts: int,
                       *, topk_idx: Optional[torch.Tensor] = None,
                       topk_weights: Optional[torch.Tensor] = None, dest_weights=None,
                       stream=None):
    """Send the rows of ``x`` (bf16 [T, H]) once to every rank that receives
    them: ``dest_x`` is a list of G bf16 [rows_d, H] tensors, ``dest_weights``
    None or a list of G fp32 [rows_d, k] tensors (entries may be None; needs
    ``topk_idx``).  Rows at or past the smallest rows_d are not written."""
    _need(x, "x", torch.bfloat16)
    _need(sparse_to_dense, "sparse_to_dense", torch.int32)
    if x.dim() != 2 or sparse_to_dense.dim() != 2 or sparse_to_dense.shape[0] != x.shape[0]:
        raise ValueError("x must be [T, H] and sparse_to_dense [T, G]")
    T, H = x.shape
    G = sparse_to_dense.shape[1]
    if len(dest_x) != G:
        raise ValueError("one destination buffer per rank")
    for d, t in enumerate(dest_x):
        _need(t, f"dest_x[{d}]", torch.bfloat16)
        if t.dim() != 2 or t.shape[1] != H:
            raise ValueError(f"dest_x[{d}] must be [rows, {H}]")
    rows = min(int(t.shape[0]) for t in dest_x)
    k = 1
    if topk_idx is not None:
        _need(topk_idx, "topk_idx", torch.int64)
        if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
            raise ValueError("topk_idx must be [T, k]")
        k = topk_idx.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    wtab = None
    if dest_weights is not None:
        if topk_idx is None:
            raise ValueError("dest_weights needs topk_idx")
        if len(dest_weights) != G:
            raise ValueError("one weight buffer (or None) per rank")
        for d, t in enumerate(dest_weights):
            if t is not None:
                _need(t, f"dest_weights[{d}]", torch.float32, rows * k)
        wtab = _ptr_table(dest_weights)
    xtab = _ptr_table(dest_x)
    st = lib().ep_dispatch_ranked(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, H, k,
                                  int(num_experts), G, _ptr(sparse_to_dense), xtab[1],
                                  None if wtab is None else wtab[1], rows, _stream(stream))
    _check(st, "ep_dispatch_ranked")
    return dest_x, dest_weights


def ep_dispatch_ranked_prequantized(x_q: torch.Tensor, x_scales: torch.Tensor,
                                    sparse_to_dense: torch.Tensor, dest_q, dest_scales,
                                    num_experts: int, *, topk_idx: Optional[torch.Tensor] = None,
                                    topk_weights: Optional[torch.Tensor] = None, dest_weights=None,
                                    stream=None):
    """Once-per-rank dispatch of 8-bit tokens: ``x_q`` uint8 [T, H] and
    ``x_scales`` fp32 [T, H/128] go to the G ranks' ``dest_q`` (uint8
    [rows_d, H]) and ``dest_scales`` (fp32 [rows_d, H/128]); weights as
    ep_dispatch_ranked.  Rows at or past the smallest rows_d are not
    written."""
    _need(x_q, "x_q", torch.uint8)
    _need(x_scales, "x_scales", torch.float32)
    _need(sparse_to_dense, "sparse_to_dense", torch.int32)
    if x_q.dim() != 2 or sparse_to_dense.dim() != 2 or sparse_to_dense.shape[0] != x_q.shape[0]:
        raise ValueError("x_q must be [T, H] and sparse_to_dense [T, G]")
    T, H = x_q.shape
    nb = H // 128
    _need(x_scales, "x_scales", torch.float32, T * nb)
    G = sparse_to_dense.shape[1]
    if len(dest_q) != G or len(dest_scales) != G:
        raise ValueError("one code and one scale buffer per rank")
    for d in range(G):
        _need(dest_q[d], f"dest_q[{d}]", torch.uint8)
        if dest_q[d].dim() != 2 or dest_q[d].shape[1] != H:
            raise ValueError(f"dest_q[{d}] must be [rows, {H}]")
        _need(dest_scales[d], f"dest_scales[{d}]", torch.float32)
    rows = min(int(t.shape[0]) for t in dest_q)
    for d in range(G):
        _need(dest_scales[d], f"dest_scales[{d}]", torch.float32, rows * nb)
    k = 1
    if topk_idx is not None:
        _need(topk_idx, "topk_idx", torch.int64)
        k = topk_idx.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    wtab = None
    if dest_weights is not None:
        if topk_idx is None or len(dest_weights) != G:
            raise ValueError("dest_weights needs topk_idx and one buffer (or None) per rank")
        for d, t in enumerate(dest_weights):
            if t is not None:
                _need(t, f"dest_weights[{d}]", torch.float32, rows * k)
        wtab = _ptr_table(dest_weights)
    qtab = _ptr_table(dest_q)
    stab = _ptr_table(dest_scales)
    st = lib().ep_dispatch_ranked_prequantized(_ptr(x_q), _ptr(x_scales), _ptr(topk_idx),
                                               _ptr(topk_weights), T, H, k, int(num_experts), G,
                                               _ptr(sparse_to_dense), qtab[1], stab[1],
                                               None if wtab is None else wtab[1], rows,
                                               _stream(stream))
    _check(st, "ep_dispatch_ranked_prequantized")
    return dest_q, dest_scales, dest_weights


def ep_dispatch_ranked_fp8(x: torch.Tensor, sparse_to_dense: torch.Tensor, dest_q, dest_scales,
                           num_experts: int, *, fmt: str = "e4m3", scale: str = "fp32",
                           topk_idx: Optional[torch.Tensor] = None,
                           topk_weights: Optional[torch.Tensor] = None, dest_weights=None,
                           stream=None):
    """Once-per-rank dispatch with the 8-bit cast on the way: ``x`` bf16
    [T, H] (H a multiple of 128) is cast as ep_dispatch casts it (``fmt``
    "e4m3" / "e5m2", ``scale`` "fp32" / "pow2" / "ue8m0") and each token's
    codes and scales go to the G ranks' ``dest_q`` (uint8 [rows_d, H]) and
    ``dest_scales`` ([rows_d, H/128], fp32, or uint8 for "ue8m0"); weights as
    ep_dispatch_ranked.  Rows at or past the smallest rows_d are not
    written."""
    _need(x, "x", torch.bfloat16)
    _need(sparse_to_dense, "sparse_to_dense", torch.int32)
    if x.dim() != 2 or sparse_to_dense.dim() != 2 or sparse_to_dense.shape[0] != x.shape[0]:
        raise ValueError("x must be [T, H] and sparse_to_dense [T, G]")
    T, H = x.shape
    nb = H // 128
    G = sparse_to_dense.shape[1]
    sdt = torch.uint8 if scale == "ue8m0" else torch.float32
    if len(dest_q) != G or len(dest_scales) != G:
        raise ValueError("one code and one scale buffer per rank")
    for d in range(G):
        _need(dest_q[d], f"dest_q[{d}]", torch.uint8)
        if dest_q[d].dim() != 2 or dest_q[d].shape[1] != H:
            raise ValueError(f"dest_q[{d}] must be [rows, {H}]")
    rows = min(int(t.shape[0]) for t in dest_q)
    for d in range(G):
        _need(dest_scales[d], f"dest_scales[{d}]", sdt, rows * nb)
    k = 1
    if topk_idx is not None:
        _need(topk_idx, "topk_idx", torch.int64)
        k = topk_idx.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, T * k)
    wtab = None
    if dest_weights is not None:
        if topk_idx is None or len(dest_weights) != G:
            raise ValueError("dest_weights needs topk_idx and one buffer (or None) per rank")
        for d, t in enumerate(dest_weights):
            if t is not None:
                _need(t, f"dest_weights[{d}]", torch.float32, rows * k)
        wtab = _ptr_table(dest_weights)
    qtab = _ptr_table(dest_q)
    stab = _ptr_table(dest_scales)
    st = lib().ep_dispatch_ranked_fp8(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, H, k,
                                      int(num_experts), G, _ptr(sparse_to_dense), _FORMATS[fmt],
                                      _SCALES[scale], qtab[1], stab[1],
                                      None if wtab is None else wtab[1], rows, _stream(stream))
    _check(st, "ep_dispatch_ranked_fp8")


def _fused_permute_tables(G, T, k, R, src_topk_idx, src_topk_weights, recv_weights):
    itab = wtab = None
    if recv_weights is not None:
        _need(recv_weights, "recv_weights", torch.float32, R)
        if src_topk_idx is None or len(src_topk_idx) != G:
            raise ValueError("recv_weights needs src_topk_idx for every rank")
        for d, t in enumerate(src_topk_idx):
            _need(t, f"src_topk_idx[{d}]", torch.int64, T * k)
        itab = _ptr_table(src_topk_idx)
        if src_topk_weights is not None:
            for d, t in enumerate(src_topk_weights):
                if t is not None:
                    _need(t, f"src_topk_weights[{d}]", torch.float32, T * k)
            wtab = _ptr_table(src_topk_weights)
    return itab, wtab


def _fused_permute_routing(G, T, recv_src, recv_topk_idx, slot, num_recv):
    _need(recv_src, "recv_src", torch.int32, G * T)
    _need(recv_topk_idx, "recv_topk_idx", torch.int64)
    _need(slot, "slot", torch.int32)
    if slot.dim() != 2 or slot.shape[0] != G * T or recv_topk_idx.shape != slot.shape:
        raise ValueError("slot and recv_topk_idx must be [G*T, k]")
    if num_recv is not None:
        _need(num_recv, "num_recv", torch.int32, 1)
    return slot.shape[1]


def ep_dispatch_fused_permute(src_x, recv_src: torch.Tensor, recv_topk_idx: torch.Tensor,
                              slot: torch.Tensor, num_experts: int, rank: int, *, rows: int,
                              src_topk_idx=None, src_topk_weights=None, num_recv=None,
                              recv_x=None, recv_weights=None, want_weights: bool = False,
                              stream=None):
    """The receiving rank's dispatch with the permute fused in: ``src_x`` is
    a list of the G ranks' tokens (bf16 [T, H]); ``recv_src`` /
    ``recv_topk_idx`` come from ep_rank_layout and ``slot`` from ep_layout of
    recv_topk_idx over E/G experts; ``rows`` is the expert-grouped buffer's
    row count.  Weights need ``src_topk_idx`` (list of int64 [T, k]) and
    optionally ``src_topk_weights`` (list of fp32 [T, k] or None).
    ``num_recv`` (int32 [1] on the device, from ep_rank_layout) bounds the
    rows visited; None visits all G*T.  Returns (recv_x bf16 [rows, H],
    recv_weights fp32 [rows] or None)."""
    G = len(src_x)
    for d, t in enumerate(src_x):
        _need(t, f"src_x[{d}]", torch.bfloat16)
    T, H = src_x[0].shape
    for t in src_x:
        if tuple(t.shape) != (T, H):
            raise ValueError("every src_x must be [T, H]")
    k = _fused_permute_routing(G, T, recv_src, recv_topk_idx, slot, num_recv)
    R = int(rows)
    dev = src_x[0].device
    if recv_x is None:
        recv_x = torch.empty((max(R, 1), H), dtype=torch.bfloat16, device=dev)
    _need(recv_x, "recv_x", torch.bfloat16, R * H)
    if want_weights and recv_weights is None:
        recv_weights = torch.empty(max(R, 1), dtype=torch.float32, device=dev)
    itab, wtab = _fused_permute_tables(G, T, k, R, src_topk_idx, src_topk_weights, recv_weights)
    xtab = _ptr_table(src_x)
    st = lib().ep_dispatch_fused_permute(xtab[1], None if itab is None else itab[1],
                                         None if wtab is None else wtab[1], T, H, k,
                                         int(num_experts), G, int(rank), _ptr(recv_src),
                                         _ptr(recv_topk_idx), _ptr(num_recv), _ptr(slot), R,
                                         _ptr(recv_x),
                                         _ptr(recv_weights), _stream(stream))
    _check(st, "ep_dispatch_fused_permute")
    return recv_x, recv_weights


def ep_dispatch_fused_permute_prequantized(src_q, src_scales, recv_src: torch.Tensor,
                                           recv_topk_idx: torch.Tensor, slot: torch.Tensor,
                                           num_experts: int, rank: int, *, rows: int,
                                           src_topk_idx=None, src_topk_weights=None,
                                           num_recv=None, recv_q=None, recv_scales=None,
                                           recv_weights=None, want_weights: bool = False,
                                           stream=None):
    """ep_dispatch_fused_permute for tokens the senders already cast to
    8 bits: ``src_q`` is a list of the G ranks' code rows (uint8 [T, H], H a
    multiple of 128) and ``src_scales`` their scale rows (fp32 [T, H/128]).
    Returns (recv_q uint8 [rows, H], recv_scales fp32 [rows, H/128],
    recv_weights fp32 [rows] or None)."""
    G = len(src_q)
    if len(src_scales) != G:
        raise ValueError("one scale tensor per rank")
    for d, t in enumerate(src_q):
        _need(t, f"src_q[{d}]", torch.uint8)
    T, H = src_q[0].shape
    nb = H // 128
    for d in range(G):
        if tuple(src_q[d].shape) != (T, H):
            raise ValueError("every src_q must be [T, H]")
        _need(src_scales[d], f"src_scales[{d}]", torch.float32, T * nb)
    k = _fused_permute_routing(G, T, recv_src, recv_topk_idx, slot, num_recv)
    R = int(rows)
    dev = src_q[0].device
    if recv_q is None:
        recv_q = torch.empty((max(R, 1), H), dtype=torch.uint8, device=dev)
    if recv_scales is None:
        recv_scales = torch.empty((max(R, 1), max(nb, 1)), dtype=torch.float32, device=dev)
    _need(recv_q, "recv_q", torch.uint8, R * H)
    _need(recv_scales, "recv_scales", torch.float32, R * nb)
    if want_weights and recv_weights is None:
        recv_weights = torch.empty(max(R, 1), dtype=torch.float32, device=dev)
    itab, wtab = _fused_permute_tables(G, T, k, R, src_topk_idx, src_topk_weights, recv_weights)
    qtab = _ptr_table(src_q)
    stab = _ptr_table(src_scales)
    st = lib().ep_dispatch_fused_permute_prequantized(
        qtab[1], stab[1], None if itab is None else itab[1], None if wtab is None else wtab[1], T,
        H, k, int(num_experts), G, int(rank), _ptr(recv_src), _ptr(recv_topk_idx),
        _ptr(num_recv), _ptr(slot), R, _ptr(recv_q), _ptr(recv_scales), _ptr(recv_weights),
        _stream(stream))
    _check(st, "ep_dispatch_fused_permute_prequantized")
    return recv_q, recv_scales, recv_weights


def ep_combine_ranked(src_y, sparse_to_dense: torch.Tensor, *, out=None, stream=None) -> torch.Tensor:
    """out[t] = bf16(sum over ranks d holding token t of src_y[d][row]) with
    ``src_y`` a list of G bf16 [rows_d, H] tensors; rows at or past the
    smallest rows_d read as 0."""
    _need(sparse_to_dense, "sparse_to_dense", torch.int32)
    if sparse_to_dense.dim() != 2:
        raise ValueError("sparse_to_dense must be [T, G]")
    T, G = sparse_to_dense.shape
    if len(src_y) != G:
        raise ValueError("one source buffer per rank")
    H = None
    for d, t in enumerate(src_y):
        _need(t, f"src_y[{d}]", torch.bfloat16)
        if t.dim() != 2 or (H is not None and t.shape[1] != H):
            raise ValueError("every src_y must be [rows, H] with the same H")
        H = t.shape[1]
    rows = min(int(t.shape[0]) for t in src_y)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=sparse_to_dense.device)
    _need(out, "out", torch.bfloat16, T * H)
    ytab = _ptr_table(src_y)
    st = lib().ep_combine_ranked(ytab[1], rows, _ptr(sparse_to_dense), T, H, G, _ptr(out),
                                 _stream(stream))
    _check(st, "ep_combine_ranked")
    return out


def ep_dispatch_ranked_backward(sparse_to_dense: torch.Tensor, num_experts: int, *,
                                grad_recv_x=None, grad_recv_weights=None,
                                topk_idx: Optional[torch.Tensor] = None, grad_x=None,
                                grad_topk_weights=None, stream=None):
    """Backward of ep_dispatch_ranked for this rank's tokens.
    ``grad_recv_x``: None or a list of G bf16 [rows, H] row gradients (gives
    grad_x [T, H], the combine over ranks); ``grad_recv_weights``: None or a
    list of G fp32 [rows, k] weight gradients (entries may be None; gives
    grad_topk_weights [T, k], needs ``topk_idx``).  Rows at or past the
    smallest buffer's rows read as 0.  Returns (grad_x, grad_topk_weights)."""
    _need(sparse_to_dense, "sparse_to_dense", torch.int32)
    if sparse_to_dense.dim() != 2:
        raise ValueError("sparse_to_dense must be [T, G]")
    T, G = sparse_to_dense.shape
    dev = sparse_to_dense.device
    rows = None
    H = 0
    k = 1
    xtab = wtab = None
    if grad_recv_x is not None:
        if len(grad_recv_x) != G:
            raise ValueError("one row-gradient buffer per rank")
        for d, t in enumerate(grad_recv_x):
            _need(t, f"grad_recv_x[{d}]", torch.bfloat16)
            if t.dim() != 2 or (H and t.shape[1] != H):
                raise ValueError("every grad_recv_x must be [rows, H] with the same H")
            H = t.shape[1]
        rows = min(int(t.shape[0]) for t in grad_recv_x)
        if grad_x is None:
            grad_x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        _need(grad_x, "grad_x", torch.bfloat16, T * H)
        xtab = _ptr_table(grad_recv_x)
    if grad_recv_weights is not None:
        if topk_idx is None:
            raise ValueError("grad_recv_weights needs topk_idx")
        _need(topk_idx, "topk_idx", torch.int64, T)
        k = topk_idx.shape[1]
        if len(grad_recv_weights) != G:
            raise ValueError("one weight-gradient buffer per rank")
        wrows = []
        for d, t in enumerate(grad_recv_weights):
            if t is None:
                continue
            _need(t, f"grad_recv_weights[{d}]", torch.float32)
            if t.dim() != 2 or t.shape[1] != k:
                raise ValueError("every grad_recv_weights must be [rows, k]")
            wrows.append(int(t.shape[0]))
        if wrows:
            rows = min(wrows + ([rows] if rows is not None else []))
        if grad_topk_weights is None:
            grad_topk_weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        _need(grad_topk_weights, "grad_topk_weights", torch.float32, T * k)
        wtab = _ptr_table(grad_recv_weights)
    st = lib().ep_dispatch_ranked_backward(
        None if xtab is None else xtab[1], None if wtab is None else wtab[1], rows or 0,
        _ptr(topk_idx), _ptr(sparse_to_dense), T, H or 8, k, int(num_experts), G,
        _ptr(grad_x) if xtab is not None else None,
        _ptr(grad_topk_weights) if wtab is not None else None, _stream(stream))
    _check(st, "ep_dispatch_ranked_backward")
    return (grad_x if xtab is not None else None,
            grad_topk_weights if wtab is not None else None)


# -------------------------------------- router, row movement, 4-bit products --
# Outputs that are not given are allocated with torch on the stream of the
# call; every tensor of a call lives on one device, which need not be the
# current one.  No call takes part in torch's autograd: outputs carry no
# gradient function whatever their inputs require, and each backward is a call
# of its own.

def _rows_of(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None,
             cols: Optional[int] = None, device=None) -> int:
    """The row stride of a 2-D device tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16, float16 or float32'}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    n, h = t.shape
    if cols is not None and h != cols:
        raise ValueError(f"{name} must have {cols} columns, has {h}")
    if n <= 1 and (h <= 1 or t.stride(1) == 1):
        return h
    if (h > 1 and t.stride(1) != 1) or t.stride(0) < h:
        raise ValueError(f"{name} must have contiguous rows that do not overlap (strides "
                         f"{tuple(t.stride())})")
    return t.stride(0)


def _need_on(t, name, dtype, device, numel=None):
    _need(t, name, dtype, numel)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _stream_handle(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without a Stream object: 0.1 us against 1.8 of
# the 10 that a call takes on the host.  The name is torch's own and may be
# missing from a build: then through the Stream.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)


class _On:
    """The device and stream of a call: ``empty`` allocates for that stream,
    ``call`` launches on it."""

    __slots__ = ("device", "stream", "ctx")

    def __init__(self, device, stream):
        self.device = device
        self.ctx = None
        if stream is None:
            self.stream = _raw_stream(device.index)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.stream = stream.cuda_stream
            self.ctx = stream

    def empty(self, shape, dtype):
        if self.ctx is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.ctx):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def call(self, where, fn, *args):
        if self.device.index == torch.cuda.current_device():
            st = fn(*args, self.stream)
        else:
            with torch.cuda.device(self.device):
                st = fn(*args, self.stream)
        if st != EP_SUCCESS:
            _check(st, where)


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"unknown score {score!r} (softmax or sigmoid)")
    return _SCORES[score]


def ep_router(logits: torch.Tensor, num_topk: int, *, score: str = "softmax",
              bias: Optional[torch.Tensor] = None, num_groups: int = 1, topk_groups: int = 1,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
              topk_idx=None, topk_weights=None, probs=None, want_probs: bool = False, stream=None):
    """Choose ``num_topk`` experts per token from ``logits`` (bf16 / fp16 /
    fp32 [T, E], rows may be strided; -inf masks an expert).

    ``score`` is "softmax" or "sigmoid"; ``bias`` (fp32 [E]) is added to the
    scores for the choice only; with ``num_groups`` > 1 the choice is among
    the ``topk_groups`` groups whose ``group_top`` (1 or 2) best values sum
    highest.  Weights are the chosen scores, divided by their sum with
    ``renormalize``, times ``scale``.

    Returns (topk_idx int64 [T, k], -1 where no expert is left, topk_weights
    fp32 [T, k], probs fp32 [T, E] or None), all outside autograd: their
    gradient is ep_router_backward.
    """
    ld = _rows_of(logits, "logits")
    T, E = logits.shape
    k = int(num_topk)
    dev = logits.device
    on = _On(dev, stream)
    if k < 1:
        raise ValueError("num_topk must be positive")
    if topk_idx is None:
        topk_idx = on.empty((T, k), torch.int64)
    else:
        _need_on(topk_idx, "topk_idx", torch.int64, dev, T * k)
    if topk_weights is None:
        topk_weights = on.empty((T, k), torch.float32)
    else:
        _need_on(topk_weights, "topk_weights", torch.float32, dev, T * k)
    if probs is not None:
        _need_on(probs, "probs", torch.float32, dev, T * E)
    elif want_probs:
        probs = on.empty((T, E), torch.float32)
    if bias is not None:
        _need_on(bias, "bias", torch.float32, dev, E)
    on.call("ep_router", lib().ep_router, logits.data_ptr(), _DTYPES[logits.dtype], T, E, ld, k,
            _score(score), _ptr(bias), int(num_groups), int(topk_groups), int(group_top),
            int(bool(renormalize)), float(scale), topk_idx.data_ptr(), topk_weights.data_ptr(),
            _ptr(probs))
    return topk_idx, topk_weights, probs


def ep_router_backward(logits: torch.Tensor, topk_idx: torch.Tensor, grad_weights: torch.Tensor,
                       grad_probs: Optional[torch.Tensor] = None, *, score: str = "softmax",
                       renormalize: bool = True, scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of ep_router's weights (and probs) back to the logits, the
    choice ``topk_idx`` held constant; ``score``, ``renormalize`` and ``scale``
    as given to ep_router.  Returns grad_logits [T, E] in the logits' type."""
    ld = _rows_of(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    _need_on(topk_idx, "topk_idx", torch.int64, dev)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError("topk_idx must be 2-D [num_tokens, num_topk]")
    k = topk_idx.shape[1]
    _need_on(grad_weights, "grad_weights", torch.float32, dev, T * k)
    if grad_probs is not None:
        _need_on(grad_probs, "grad_probs", torch.float32, dev, T * E)
    on = _On(dev, stream)
    if grad_logits is None:
        grad_logits = on.empty((T, E), logits.dtype)
    else:
        _need_on(grad_logits, "grad_logits", logits.dtype, dev, T * E)
    on.call("ep_router_backward", lib().ep_router_backward, logits.data_ptr(),
            _DTYPES[logits.dtype], T, E, ld, k, _score(score), int(bool(renormalize)), float(scale),
            topk_idx.data_ptr(), grad_weights.data_ptr(), _ptr(grad_probs), grad_logits.data_ptr())
    return grad_logits


def _pairs_of(slot, topk_weights, T, device):
    _need_on(slot, "slot", torch.int32, device)
    if slot.dim() != 2 or (T is not None and slot.shape[0] != T):
        raise ValueError("slot must be 2-D [num_tokens, num_topk]")
    if topk_weights is not None:
        _need_on(topk_weights, "topk_weights", torch.float32, device, slot.numel())
    return slot.shape


def _clear_of(clear, device):
    if clear is None:
        return None, None, 0
    counts, offsets = clear
    _need_on(counts, "counts", torch.int32, device)
    E = counts.numel()
    _need_on(offsets, "offsets", torch.int32, device, E + 1)
    return counts.data_ptr(), offsets.data_ptr(), E


def ep_permute(x: torch.Tensor, slot: torch.Tensor, topk_weights: Optional[torch.Tensor] = None, *,
               rows: Optional[int] = None, out=None, clear=None, stream=None):
    """Rows sorted by expert: ``out[slot[t, j]] = topk_weights[t, j] * x[t]``
    (unit weights without ``topk_weights``).  ``x`` is bf16 / fp16 / fp32
    [T, H], of any width, rows may be strided.

    ``rows`` (T*k by default) is the layout's row bound.  ``clear`` =
    (counts, offsets) of the layout clears the rows that no slot names; else
    they are not written.  Returns out [rows, H], outside autograd: its
    gradient is ep_permute_backward."""
    ld = _rows_of(x, "x")
    T, H = x.shape
    dev = x.device
    _, k = _pairs_of(slot, topk_weights, T, dev)
    on = _On(dev, stream)
    if out is None:
        R, ld_out = T * k if rows is None else int(rows), H
        out = on.empty((R, H), x.dtype)
    else:
        R, ld_out = out.shape[0], _rows_of(out, "out", x.dtype, H, dev)
        if rows is not None and R < rows:
            raise ValueError(f"out has {R} rows, needs {rows}")
    c, o, E = _clear_of(clear, dev)
    on.call("ep_permute", lib().ep_permute, x.data_ptr(), _DTYPES[x.dtype], T, H, ld, k,
            slot.data_ptr(), _ptr(topk_weights), out.data_ptr(), ld_out, R, c, o, E)
    return out


def ep_permute_backward(grad_rows: torch.Tensor, slot: torch.Tensor,
                        topk_weights: Optional[torch.Tensor] = None,
                        x: Optional[torch.Tensor] = None, *, grad_x=None, grad_weights=None,
                        stream=None):
    """Backward of ep_permute: (grad_x [T, H], grad_weights fp32 [T, k]); the
    latter None unless ``topk_weights`` and ``x`` are given, which a
    ``grad_weights`` buffer needs."""
    if grad_weights is not None and (topk_weights is None or x is None):
        raise ValueError("grad_weights needs topk_weights and x")
    ld = _rows_of(grad_rows, "grad_rows")
    R, H = grad_rows.shape
    dev, dt = grad_rows.device, grad_rows.dtype
    T, k = _pairs_of(slot, topk_weights, None, dev)
    on = _On(dev, stream)
    ld_x = 0
    if topk_weights is None or x is None:
        x = None
    else:
        ld_x = _rows_of(x, "x", dt, H, dev)
        if x.shape[0] != T:
            raise ValueError(f"x has {x.shape[0]} rows, slot {T}")
        if grad_weights is None:
            grad_weights = on.empty((T, k), torch.float32)
        else:
            _need_on(grad_weights, "grad_weights", torch.float32, dev, T * k)
    if grad_x is None:
        grad_x, ld_gx = on.empty((T, H), dt), H
    else:
        ld_gx = _rows_of(grad_x, "grad_x", dt, H, dev)
        if grad_x.shape[0] != T:
            raise ValueError(f"grad_x has {grad_x.shape[0]} rows, slot {T}")
    on.call("ep_permute_backward", lib().ep_permute_backward, grad_rows.data_ptr(), _DTYPES[dt], T,
            H, ld, R, k, slot.data_ptr(), _ptr(topk_weights), _ptr(x), ld_x, grad_x.data_ptr(),
            ld_gx, _ptr(grad_weights))
    return grad_x, grad_weights


def ep_unpermute(y: torch.Tensor, slot: torch.Tensor, topk_weights: Optional[torch.Tensor] = None,
                 *, out=None, stream=None):
    """Rows back in token order: ``out[t] = sum_j topk_weights[t, j] *
    y[slot[t, j]]``, in fp32, j ascending.  ``y`` is bf16 / fp16 / fp32
    [rows, H], of any width, rows may be strided.  Returns out [T, H], outside
    autograd: its gradient is ep_unpermute_backward."""
    ld = _rows_of(y, "y")
    R, H = y.shape
    dev = y.device
    T, k = _pairs_of(slot, topk_weights, None, dev)
    on = _On(dev, stream)
    if out is None:
        out, ld_out = on.empty((T, H), y.dtype), H
    else:
        ld_out = _rows_of(out, "out", y.dtype, H, dev)
        if out.shape[0] != T:
            raise ValueError(f"out has {out.shape[0]} rows, slot {T}")
    on.call("ep_unpermute", lib().ep_unpermute, y.data_ptr(), _DTYPES[y.dtype], T, H, ld, R, k,
            slot.data_ptr(), _ptr(topk_weights), out.data_ptr(), ld_out)
    return out


def ep_unpermute_backward(grad_out: torch.Tensor, slot: torch.Tensor,
                          topk_weights: Optional[torch.Tensor] = None,
                          y: Optional[torch.Tensor] = None, *, rows: Optional[int] = None,
                          grad_y=None, grad_weights=None, clear=None, stream=None):
    """Backward of ep_unpermute: (grad_y [rows, H], grad_weights fp32 [T, k]);
    the latter None unless ``topk_weights`` and ``y`` are given, which a
    ``grad_weights`` buffer needs.  ``rows`` and ``clear`` as in ep_permute
    (``rows`` is y's with ``y``)."""
    if grad_weights is not None and (topk_weights is None or y is None):
        raise ValueError("grad_weights needs topk_weights and y")
    ld = _rows_of(grad_out, "grad_out")
    T, H = grad_out.shape
    dev, dt = grad_out.device, grad_out.dtype
    _, k = _pairs_of(slot, topk_weights, T, dev)
    on = _On(dev, stream)
    ld_y = 0
    if y is not None and rows is None:
        rows = y.shape[0]
    if topk_weights is None or y is None:
        y = None
    else:
        ld_y = _rows_of(y, "y", dt, H, dev)
        if grad_weights is None:
            grad_weights = on.empty((T, k), torch.float32)
        else:
            _need_on(grad_weights, "grad_weights", torch.float32, dev, T * k)
    if grad_y is None:
        R, ld_gy = T * k if rows is None else int(rows), H
        grad_y = on.empty((R, H), dt)
    else:
        R, ld_gy = grad_y.shape[0], _rows_of(grad_y, "grad_y", dt, H, dev)
        if rows is not None and R < rows:
            raise ValueError(f"grad_y has {R} rows, needs {rows}")
    if y is not None and y.shape[0] < R:
        raise ValueError(f"y has {y.shape[0]} rows, grad_y {R}")
    c, o, E = _clear_of(clear, dev)
    on.call("ep_unpermute_backward", lib().ep_unpermute_backward, grad_out.data_ptr(), _DTYPES[dt],
            T, H, ld, k, slot.data_ptr(), _ptr(topk_weights), _ptr(y), ld_y, grad_y.data_ptr(),
            ld_gy, R, _ptr(grad_weights), c, o, E)
    return grad_y, grad_weights


class W4Weights(NamedTuple):
    """4-bit expert weights as ep_w4_pack lays them out."""
    packed: torch.Tensor
    num_experts: int
    out_features: int
    in_features: int
    group_size: int
    dtype: torch.dtype
    has_zeros: bool
    gated: bool


def ep_w4_packed_size(num_experts: int, out_features: int, in_features: int, group_size: int = 128,
                      has_zeros: bool = False, gated: bool = False) -> int:
    """Bytes of the packed weights (0 if the shape is invalid)."""
    return int(lib().ep_w4_packed_size(int(num_experts), int(out_features), int(in_features),
                                       int(group_size), int(bool(has_zeros)), int(bool(gated))))


def ep_w4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None, *,
               group_size: int = 128, gated: bool = False, packed=None, stream=None) -> W4Weights:
    """Lay out 4-bit weights, once, for ep_expert_matmul_w4.

    ``codes`` uint8 [E, N, K/2] (the even input's code in the low four bits),
    ``scales`` bf16 or fp16 [E, N, ceil(K / group_size)], ``zeros`` uint8 of
    the scales' shape, or None: 8 everywhere.  ``gated``: the N rows are two
    halves, gate then up."""
    _need(codes, "codes", torch.uint8)
    if codes.dim() != 3:
        raise ValueError("codes must be 3-D [num_experts, out_features, in_features / 2]")
    E, N, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    dev = codes.device
    if scales.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"scales must be bfloat16 or float16, got {scales.dtype}")
    need = ep_w4_packed_size(E, N, K, group_size, zeros is not None, gated)
    if need == 0:
        raise ValueError(f"invalid 4-bit weights: {E} x {N} x {K}, groups of {group_size}, "
                         f"gated={gated}")
    shape = (E, N, (K + group_size - 1) // group_size)
    for t, name, dt in ((scales, "scales", scales.dtype), (zeros, "zeros", torch.uint8)):
        if t is not None:
            _need_on(t, name, dt, dev)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, is {tuple(t.shape)}")
    on = _On(dev, stream)
    if packed is None:
        packed = on.empty(need, torch.uint8)
    else:
        _need_on(packed, "packed", torch.uint8, dev, need)
    on.call("ep_w4_pack", lib().ep_w4_pack, codes.data_ptr(), scales.data_ptr(), _ptr(zeros),
            _DTYPES[scales.dtype], E, N, K, int(group_size), int(bool(gated)), packed.data_ptr(),
            packed.numel())
    return W4Weights(packed, E, N, K, int(group_size), scales.dtype, zeros is not None, bool(gated))


def ep_expert_matmul_w4(x: torch.Tensor, weights: W4Weights, offsets: Optional[torch.Tensor] = None,
                        *, src: Optional[torch.Tensor] = None, counts=None,
                        rows: Optional[int] = None, out=None, stream=None):
    """The experts' products with 4-bit weights: row r of expert e (rows
    ``offsets[e]`` to ``offsets[e+1]``, or ``counts[e]`` of them) gives
    ``out[r] = W[e] @ x[r]``, or ``W[e] @ x[src[r]]`` with ``src`` (the
    layout's), or silu(gate) * up of its two halves for gated weights.

    ``x`` has the scales' type and may have strided rows; ``offsets`` may be
    left out with one expert.  ``rows`` is the layout's row bound (src's
    length, or x's rows).  Returns out [rows, N] (N/2 if gated), outside
    autograd and without a backward call; rows of no expert are not written."""
    w = weights
    ld = _rows_of(x, "x", w.dtype, w.in_features)
    dev = x.device
    _need_on(w.packed, "weights.packed", torch.uint8, dev)
    if src is not None:
        _need_on(src, "src", torch.int32, dev, rows)
    R = int(rows) if rows is not None else (src.numel() if src is not None else x.shape[0])
    if offsets is not None:
        _need_on(offsets, "offsets", torch.int32, dev, w.num_experts + 1)
    if counts is not None:
        _need_on(counts, "counts", torch.int32, dev, w.num_experts)
    on = _On(dev, stream)
    n = w.out_features // 2 if w.gated else w.out_features
    if out is None:
        out, ld_out = on.empty((R, n), w.dtype), n
    else:
        ld_out = _rows_of(out, "out", w.dtype, n, dev)
        if out.shape[0] < R:
            raise ValueError(f"out has {out.shape[0]} rows, needs {R}")
    on.call("ep_expert_matmul_w4", lib().ep_expert_matmul_w4, x.data_ptr(), _DTYPES[w.dtype], ld,
            x.shape[0], _ptr(src), w.packed.data_ptr(), w.packed.numel(), w.num_experts,
            w.out_features, w.in_features, w.group_size, int(w.has_zeros), int(w.gated),
            _ptr(offsets), _ptr(counts), R, out.data_ptr(), ld_out)
    return out


# ------------------------------------------ full-width and 8-bit products --

_HALVES = (torch.bfloat16, torch.float16)


def _expert_weights(t, name, dtype, device):
    _need_on(t, name, dtype, device)
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [num_experts, out_features, in_features]")
    return t.shape


def _segments_of(E, offsets, counts, device):
    if offsets is not None:
        _need_on(offsets, "offsets", torch.int32, device, E + 1)
    if counts is not None:
        _need_on(counts, "counts", torch.int32, device, E)


def _out_of(on, out, name, R, cols, dtype, device):
    if out is None:
        return on.empty((R, cols), dtype), cols
    ld = _rows_of(out, name, dtype, cols, device)
    if out.shape[0] < R:
        raise ValueError(f"{name} has {out.shape[0]} rows, needs {R}")
    return out, ld


def _expert_rows(x, weights, offsets, src, counts, rows):
    """(E, N, K, x's row stride, rows of the product) of a 16-bit product."""
    if isinstance(x, torch.Tensor) and x.dtype not in _HALVES:
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    ld = _rows_of(x, "x")
    dev = x.device
    E, N, K = _expert_weights(weights, "weights", x.dtype, dev)
    if x.shape[1] != K:
        raise ValueError(f"x must have {K} columns, has {x.shape[1]}")
    if src is not None:
        _need_on(src, "src", torch.int32, dev, rows)
    R = int(rows) if rows is not None else (src.numel() if src is not None else x.shape[0])
    _segments_of(E, offsets, counts, dev)
    return E, N, K, ld, R


def ep_expert_matmul(x: torch.Tensor, weights: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                     src: Optional[torch.Tensor] = None, counts=None, rows: Optional[int] = None,
                     out=None, stream=None):
    """The experts' products: row r of expert e (rows ``offsets[e]`` to
    ``offsets[e+1]``, or ``counts[e]`` of them) gives ``out[r] = W[e] @ x[r]``,
    or ``W[e] @ x[src[r]]`` with ``src`` (the layout's).

    ``x`` is bf16 or fp16 and may have strided rows, ``weights`` [E, N, K] has
    its type; ``offsets`` may be left out with one expert.  ``rows`` is the
    layout's row bound (src's length, or x's rows).  Returns out [rows, N],
    outside autograd: its gradients are ep_expert_matmul_backward.  Rows of no
    expert are not written."""
    E, N, K, ld, R = _expert_rows(x, weights, offsets, src, counts, rows)
    dev, dt = x.device, x.dtype
    on = _On(dev, stream)
    out, ld_out = _out_of(on, out, "out", R, N, dt, dev)
    on.call("ep_expert_matmul", lib().ep_expert_matmul, x.data_ptr(), _DTYPES[dt], ld, x.shape[0],
            _ptr(src), weights.data_ptr(), E, N, K, _ptr(offsets), _ptr(counts), R, out.data_ptr(),
            ld_out)
    return out


def ep_expert_glu(x: torch.Tensor, weights: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                  src: Optional[torch.Tensor] = None, counts=None, rows: Optional[int] = None,
                  out=None, pre=None, want_pre: bool = False, stream=None):
    """The experts' gated block: ``out[r] = silu(gate) * up``, gate and up the
    two halves of ``W[e] @ x[r]`` (the rows of ``weights`` [E, N, K] are gate,
    then up), in one kernel; arguments as ep_expert_matmul.

    Returns (out [rows, N/2], pre): with ``want_pre`` or a ``pre`` buffer
    [rows, N] gate and up, which ep_expert_glu_backward takes, else None."""
    E, N, K, ld, R = _expert_rows(x, weights, offsets, src, counts, rows)
    if N % 2:
        raise ValueError(f"gated weights have two halves, got {N} rows")
    dev, dt = x.device, x.dtype
    on = _On(dev, stream)
    out, ld_out = _out_of(on, out, "out", R, N // 2, dt, dev)
    ld_pre = 0
    if pre is not None or want_pre:
        pre, ld_pre = _out_of(on, pre, "pre", R, N, dt, dev)
    on.call("ep_expert_glu", lib().ep_expert_glu, x.data_ptr(), _DTYPES[dt], ld, x.shape[0],
            _ptr(src), weights.data_ptr(), E, N, K, _ptr(offsets), _ptr(counts), R, out.data_ptr(),
            ld_out, _ptr(pre), ld_pre)
    return out, pre


def ep_expert_backward_workspace_size(num_rows: int, out_features: int, in_features: int,
                                      gated: bool = False, gathered: bool = False) -> int:
    """Bytes of the backward's workspace, of ep_expert_glu_backward with
    ``gated``, of a call with ``src`` with ``gathered`` (0 if none is needed or
    the shape is invalid).  A call without the weights' gradient takes those of
    ``in_features`` 8 and no ``gathered``."""
    return int(lib().ep_expert_backward_workspace_size(int(num_rows), int(out_features), int(in_features),
                                                       int(bool(gated)), int(bool(gathered))))


def _expert_backward(grad_out, x, weights, offsets, src, counts, grad_rows, grad_weights, want_rows,
                     want_weights, weights_dtype, workspace, stream,
                     gated):
    E, N, K, ld_x, _ = _expert_rows(x, weights, offsets, src, counts, None)
    dev, dt = x.device, x.dtype
    if gated and N % 2:
        raise ValueError(f"gated weights have two halves, got {N} rows")
    ld_g = _rows_of(grad_out, "grad_out", dt, N // 2 if gated else N, dev)
    R = grad_out.shape[0]
    if src is not None and src.numel() < R:
        raise ValueError(f"src has {src.numel()} elements, needs {R}")
    if src is None and x.shape[0] < R:
        raise ValueError(f"x has {x.shape[0]} rows, grad_out {R}")
    want_rows, want_weights = want_rows or grad_rows is not None, want_weights or grad_weights is not None
    if not want_rows and not want_weights:
        raise ValueError("neither gradient is wanted")
    if weights_dtype is None:
        weights_dtype = dt if grad_weights is None else grad_weights.dtype
    if weights_dtype not in (dt, torch.float32):
        raise TypeError(f"the weights' gradient must be {dt} or float32, not {weights_dtype}")
    on = _On(dev, stream)
    ld_gr = 0
    if want_rows:
        grad_rows, ld_gr = _out_of(on, grad_rows, "grad_rows", R, K, dt, dev)
    if want_weights:
        if grad_weights is None:
            grad_weights = on.empty((E, N, K), weights_dtype)
        else:
            _need_on(grad_weights, "grad_weights", weights_dtype, dev)
            if tuple(grad_weights.shape) != (E, N, K):
                raise ValueError(f"grad_weights must be {(E, N, K)}, is {tuple(grad_weights.shape)}")
    # x is laid out for the weights' gradient only
    need = ep_expert_backward_workspace_size(R, N, K if want_weights else 8, gated, want_weights and src is not None)
    if workspace is not None:
        _need_on(workspace, "workspace", torch.uint8, dev, need)
    elif need:
        workspace = on.empty(need, torch.uint8)
    tail = (x.data_ptr(), ld_x, x.shape[0], _ptr(src), weights.data_ptr(), E, N, K, _ptr(offsets),
            _ptr(counts), R, _ptr(grad_rows), ld_gr, _ptr(grad_weights), _DTYPES[weights_dtype],
            _ptr(workspace), 0 if workspace is None else workspace.numel())
    return on, N, R, ld_g, tail, grad_rows, grad_weights, workspace


def ep_expert_matmul_backward(grad_out: torch.Tensor, x: torch.Tensor, weights: torch.Tensor,
                              offsets: Optional[torch.Tensor] = None, *,
                              src: Optional[torch.Tensor] = None, counts=None, grad_rows=None,
                              grad_weights=None, want_rows: bool = True, want_weights: bool = True,
                              weights_dtype: Optional[torch.dtype] = None, workspace=None, stream=None):
    """Backward of ep_expert_matmul from ``grad_out`` [rows, N]: (grad_rows
    [rows, K], grad_weights [E, N, K]); the latter in ``weights_dtype``, the
    weights' own type or float32 (summed in fp32 either way), zeros for experts
    without rows.

    With ``src`` the rows' gradients still come per row of the layout;
    ep_permute_backward sums them per token.  ``want_rows`` / ``want_weights``
    False leaves one out (None).  Rows of no expert are not written.

    ``workspace`` (uint8, ep_expert_backward_workspace_size bytes) holds rows
    that are gathered or padded first, those of x for grad_weights only; torch
    allocates it when it is not given."""
    on, N, R, ld_g, tail, grad_rows, grad_weights, workspace = _expert_backward(
        grad_out, x, weights, offsets, src, counts, grad_rows, grad_weights, want_rows, want_weights,
        weights_dtype, workspace, stream, False)
    on.call("ep_expert_matmul_backward", lib().ep_expert_matmul_backward, grad_out.data_ptr(),
            _DTYPES[grad_out.dtype], ld_g, *tail)
    return grad_rows, grad_weights


def ep_expert_glu_backward(grad_out: torch.Tensor, pre: torch.Tensor, x: torch.Tensor,
                           weights: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                           src: Optional[torch.Tensor] = None, counts=None, grad_rows=None,
                           grad_weights=None, want_rows: bool = True, want_weights: bool = True,
                           weights_dtype: Optional[torch.dtype] = None, workspace=None, stream=None):
    """Backward of ep_expert_glu from ``grad_out`` [rows, N/2] and the ``pre``
    [rows, N] that it left; otherwise as ep_expert_matmul_backward.

    ``workspace`` (uint8, ep_expert_backward_workspace_size bytes) also holds
    the gradients of gate and up, in the rows' type (fp16: infinite past 65504,
    0 below 2^-25)."""
    on, N, R, ld_g, tail, grad_rows, grad_weights, workspace = _expert_backward(
        grad_out, x, weights, offsets, src, counts, grad_rows, grad_weights, want_rows, want_weights,
        weights_dtype, workspace, stream, True)
    ld_p = _rows_of(pre, "pre", x.dtype, N, x.device)
    if pre.shape[0] < R:
        raise ValueError(f"pre has {pre.shape[0]} rows, grad_out {R}")
    on.call("ep_expert_glu_backward", lib().ep_expert_glu_backward, grad_out.data_ptr(),
            _DTYPES[grad_out.dtype], ld_g, pre.data_ptr(), ld_p, *tail)
    return grad_rows, grad_weights


def ep_expert_matmul_fp8(x: torch.Tensor, x_scales: torch.Tensor, weights: torch.Tensor,
                         weight_scales: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                         fmt: str = "e4m3", gated: bool = False,
                         src: Optional[torch.Tensor] = None, counts=None, rows: Optional[int] = None,
                         dtype: torch.dtype = torch.bfloat16, out=None, stream=None):
    """The experts' products of 8-bit rows and weights, scaled per 128 inputs:
    ``out[r, n] = sum_b x_scales[r, b] * weight_scales[e, n // 128, b] *
    sum_{k in b} x[r, k] * W[e, n, k]``, or silu(gate) * up of its halves with
    ``gated``.

    ``x`` uint8 [M, K]: codes of ``fmt`` ("e4m3" or "e5m2") as ep_dispatch
    writes them, rows may be strided; ``x_scales`` [M, ceil(K / 128)] fp32, or
    uint8 powers of two (UE8M0), of any strides (``scales.t()[:M]`` for
    column-major ones); ``weights`` uint8 [E, N, K] E4M3 codes;
    ``weight_scales`` fp32 [E, ceil(N / 128), ceil(K / 128)].  The rest as
    ep_expert_matmul.  Returns out [rows, N] (N/2 if gated) in ``dtype``
    (bfloat16 or float16), outside autograd and without a backward call.

    Sums are fp32; with more than a few rows per expert, of each 8 neighbouring
    products what lies 2^-13 below the largest is dropped, so that a row's last
    bits may differ with the number of rows around it."""
    if fmt not in _FORMATS:
        raise ValueError(f"unknown fmt {fmt!r} (e4m3 or e5m2)")
    if not isinstance(x, torch.Tensor) or x.dtype != torch.uint8:
        raise TypeError("x must be uint8 codes")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    dev = x.device
    E, N, K = _expert_weights(weights, "weights", torch.uint8, dev)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be 2-D with {K} columns, is {tuple(x.shape)}")
    M = x.shape[0]
    ld = x.stride(0) if M > 1 else (K + 15) // 16 * 16
    if (K > 1 and x.stride(1) != 1) or ld < K:
        raise ValueError(f"x must have contiguous rows that do not overlap (strides {tuple(x.stride())})")
    if gated and N % 2:
        raise ValueError(f"gated weights have two halves, got {N} rows")
    blocks = (K + 127) // 128
    if not isinstance(x_scales, torch.Tensor) or x_scales.dtype not in (torch.float32, torch.uint8):
        raise TypeError("x_scales must be float32 or uint8")
    if x_scales.device != dev:
        raise ValueError(f"x_scales is on {x_scales.device}, not on {dev}")
    if tuple(x_scales.shape) != (M, blocks):
        raise ValueError(f"x_scales must be {(M, blocks)}, is {tuple(x_scales.shape)}")
    _need_on(weight_scales, "weight_scales", torch.float32, dev)
    if tuple(weight_scales.shape) != (E, (N + 127) // 128, blocks):
        raise ValueError(f"weight_scales must be {(E, (N + 127) // 128, blocks)}, is "
                         f"{tuple(weight_scales.shape)}")
    if dtype not in _HALVES:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    if src is not None:
        _need_on(src, "src", torch.int32, dev, rows)
    R = int(rows) if rows is not None else (src.numel() if src is not None else M)
    _segments_of(E, offsets, counts, dev)
    on = _On(dev, stream)
    out, ld_out = _out_of(on, out, "out", R, N // 2 if gated else N, dtype, dev)
    on.call("ep_expert_matmul_fp8", lib().ep_expert_matmul_fp8, x.data_ptr(), _FORMATS[fmt], ld, M,
            x_scales.data_ptr(), EP_SCALE_UE8M0 if x_scales.dtype == torch.uint8 else EP_SCALE_FP32,
            x_scales.stride(0), x_scales.stride(1), _ptr(src), weights.data_ptr(),
            weight_scales.data_ptr(), E, N, K, int(bool(gated)), _ptr(offsets), _ptr(counts), R,
            out.data_ptr(), _DTYPES[dtype], ld_out)
    return out


# ------------------------------------------------------ C-ABI names, 1:1 --
# Every function include/ep.h declares is reachable here under its own name.
# The helpers above keep short names and ep_layout / ep_dispatch take the
# _ex arguments as keywords; these are the same calls under the header's
# names.

ep_version = version
ep_status_string = status_string
ep_last_error = last_error
ep_layout_workspace_size = layout_workspace_size
ep_layout_max_rows = layout_max_rows
ep_rank_layout_workspace_size = rank_layout_workspace_size


def ep_layout_ex(topk_idx: torch.Tensor, num_experts: int, alignment: int, capacity: int, **kw):
    """ep_layout with segment starts aligned to ``alignment`` rows, or a fixed
    ``capacity`` rows per expert (overflow dropped, counted in num_dropped)."""
    return ep_layout(topk_idx, num_experts, alignment=alignment, capacity=capacity, **kw)


def ep_dispatch_ex(x: torch.Tensor, slot: torch.Tensor, topk_weights: Optional[torch.Tensor] = None,
                   *, out_dtype: str = "e4m3", scale: str = "fp32", scale_ld: int = 0, **kw):
    """ep_dispatch with the output type named: ``out_dtype`` "bf16" (a copy),
    "e4m3" or "e5m2" (a cast with ``scale`` "fp32", "pow2" or "ue8m0" block
    scales, row-major or, with ``scale_ld`` > 0, column-major)."""
    if out_dtype == "bf16":
        if scale_ld:
            raise ValueError("bf16 output takes no scale_ld")
        return ep_dispatch(x, slot, topk_weights, **kw)
    if out_dtype not in _FORMATS:
        raise ValueError(f"unknown out_dtype {out_dtype!r}")
    return ep_dispatch(x, slot, topk_weights, fp8=True, fmt=out_dtype, scale=scale,
                       scale_ld=scale_ld, **kw)
