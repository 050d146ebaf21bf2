"""GB300-native low-precision MoE expert path: NVFP4 per-token forward, MXFP8 backward.

A thin binding over ``libfme.so`` (C ABI in ``include/fme.h``): ctypes, and a compiled
module for the FP8 block-128, bf16, 4-bit and router calls, whose host side would outlast
their kernels in Python.  Every step of the path runs in the library's CUDA
kernels; the binding only turns torch tensors into pointers, allocates outputs
with torch when the caller does not pass them, and turns status codes into
exceptions.  There is no fallback: if the library is missing or the device is not
a GB300, calls raise.

With `stream` a call runs there and not on the current stream: its inputs must be ready on it and must live
until it is done with them.  What the call allocates then comes from that stream's memory; the outputs may be used
on the current stream once that waits for it, and freed at any time.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libfme.so")

ROWWISE = 0
COLWISE = 1
MAX_GROUPS = 1024
MX_SCALE_CEIL = 0x100
DW_BF16 = 0
DW_FP32 = 1
DW_FP32_ADD = 2
DEV_TIMEOUT = 0x1
DEV_BAD_OFFSETS = 0x2
DEV_BAD_INDEX = 0x4
# status codes (fme_status) of include/fme.h
OK = 0
ERR_INVALID_ARGUMENT = 1
ERR_MISALIGNED = 2
ERR_UNSUPPORTED_SHAPE = 3
ERR_UNSUPPORTED_DEVICE = 4
ERR_CUDA = 5
ERR_DEVICE_TIMEOUT = 6
ERR_DEVICE_BAD_OFFSETS = 7
ERR_DEVICE_BAD_INDEX = 8

_lib = None
_lock = threading.Lock()


class FmeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: status {status}"
        if _lib is not None:
            msg += f" ({_lib.fme_error_string(status).decode()})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


def ensure_built() -> str:
    """Build libfme.so and the binding if they are missing or older than their sources."""
    from . import build as _build

    return _build.refresh()


def lib() -> ctypes.CDLL:
    """The loaded CUDA library.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY):
                raise RuntimeError(f"{LIBRARY} is missing: build it with "
                                   "`python -m fp8_moe_expert_gb300.build` (no CPU fallback exists)")
            _lib = _declare(ctypes.CDLL(LIBRARY))
    return _lib


SYMBOLS = {
    # name: (restype, argtypes)
    "quantize_nvfp4_pertoken": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p", "p", "p"]),
    "quantize_nvfp4_pertensor": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p", "p", "p", "p"]),
    "swiglu_quantize_nvfp4": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p", "p", "p", "p"]),
    "quantize_mxfp8": ("i32", ["p", "i64", "i64", "i32", "p", "i32", "p", "p", "p", "p", "p"]),
    "quantize_mxfp8_rowcol": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p", "p", "p", "p", "p"]),
    "swiglu_backward_quantize_mxfp8": ("i32", ["p", "p", "i64", "i64", "p", "i32", "p", "p", "p", "p", "p", "p",
                                               "p", "p"]),
    "grouped_gemm_fwd_nvfp4": ("i32", ["p", "p", "p", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p", "p",
                                       "p"]),
    "grouped_gemm_fwd_nvfp4_swiglu": ("i32", ["p", "p", "p", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p",
                                              "p", "p"]),
    "grouped_gemm_fwd_mxfp8": ("i32", ["p", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p", "p", "p"]),
    "grouped_gemm_dgrad_mxfp8": ("i32", ["p", "p", "p", "p", "i64", "p", "i32", "i64", "i64", "i64", "p", "p",
                                         "p"]),
    "grouped_gemm_wgrad_mxfp8": ("i32", ["p", "p", "i64", "p", "p", "i64", "p", "i32", "i64", "i64", "p", "p",
                                         "p"]),
    "moe_route": ("i32", ["p", "i64", "i32", "i32", "p", "p", "p", "p", "i64", "p", "p"]),
    "moe_route_noalloc": ("i32", ["p", "i64", "i32", "i32", "p", "p", "p", "p", "p"]),
    "permute_quantize_nvfp4": ("i32", ["p", "i64", "i64", "p", "i32", "p", "i32", "p", "p", "p", "p", "p"]),
    "permute_quantize_mxfp8": ("i32", ["p", "i64", "i64", "p", "i32", "p", "i32", "p", "p", "p", "p"]),
    "moe_combine": ("i32", ["p", "i64", "p", "p", "i64", "i32", "i64", "p", "p", "p"]),
    "grouped_gemm_wgrad_mxfp8_accumulate": ("i32", ["p", "p", "i64", "p", "p", "i64", "p", "i32", "i64", "i64", "p",
                                                    "p", "p"]),
    "quantize_fp8_block128": ("i32", ["p", "i64", "i64", "i32", "p", "i32", "p", "p", "p", "p", "p"]),
    "quantize_fp8_block128_rowcol": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p", "p", "p", "p", "p"]),
    "permute_quantize_fp8_block128": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p", "p"]),
    "quantize_fp8_block128_weights": ("i32", ["p", "i32", "i64", "i64", "p", "p", "p"]),
    "grouped_gemm_fwd_fp8_block128": ("i32", ["p", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p", "p", "p"]),
    "grouped_gemm_dgrad_fp8_block128": ("i32", ["p", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p", "p", "p"]),
    "grouped_gemm_wgrad_fp8_block128": ("i32", ["p", "p", "p", "p", "i64", "p", "i32", "i64", "i64", "p", "i32", "p",
                                                "p"]),
    "grouped_gemm_fwd_bf16": ("i32", ["p", "p", "p", "i32", "i64", "i64", "i64", "p", "p", "p"]),
    "grouped_gemm_dgrad_bf16": ("i32", ["p", "p", "p", "i32", "i64", "i64", "i64", "p", "p", "p"]),
    "grouped_gemm_wgrad_bf16": ("i32", ["p", "p", "i64", "p", "i32", "i64", "i64", "p", "i32", "p", "p"]),
    "grouped_gemv_nvfp4": ("i32", ["p", "i64", "p", "i32", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p", "p",
                                   "p"]),
    "grouped_gemv_nvfp4_swiglu": ("i32", ["p", "i64", "p", "i32", "p", "p", "p", "p", "i32", "i64", "i64", "i64", "p",
                                          "p", "p"]),
    "swiglu": ("i32", ["p", "i64", "i64", "p", "p"]),
    "swiglu_backward": ("i32", ["p", "p", "i64", "i64", "p", "p"]),
    "moe_permute": ("i32", ["p", "i64", "i64", "p", "i32", "p", "p", "p"]),
    "moe_gate": ("i32", ["p", "i32", "i64", "i32", "i32", "i32", "i32", "f32", "p", "p", "p", "p"]),
    "moe_gate_backward": ("i32", ["p", "i32", "p", "p", "i64", "i32", "i32", "i32", "i32", "f32", "p", "p", "p"]),
    "moe_balance_loss": ("i32", ["p", "i32", "p", "i64", "i32", "i32", "i32", "f32", "p", "i64", "p", "p", "p", "p",
                                 "p", "i64", "p", "p"]),
    "moe_balance_loss_backward": ("i32", ["p", "i32", "p", "p", "p", "i64", "i32", "i32", "i32", "f32", "p", "i64",
                                          "p", "p", "i32", "p"]),
    "moe_combine_backward": ("i32", ["p", "p", "i64", "p", "p", "i64", "i32", "i64", "p", "p", "p", "p"]),
    "fme_balance_workspace_bytes": ("i64", ["i64", "i64", "i32"]),
    "fme_route_workspace_bytes": ("i64", ["i64", "i32", "i32"]),
    "fme_sf_padded_rows": ("i64", ["i64", "i32"]),
    "fme_sf_bytes": ("i64", ["i64", "i64", "i32", "i32"]),
    "fme_colwise_ld": ("i64", ["i64", "i32"]),
    "fme_read_device_status": ("i32", ["p", "p", "p"]),
    "fme_error_string": ("s", ["i32"]),
    "fme_last_cuda_error": ("s", []),
    "fme_version": ("s", []),
}

_CT = {"f32": ctypes.c_float, "i32": ctypes.c_int32, "i64": ctypes.c_int64, "p": ctypes.c_void_p, "s": ctypes.c_char_p}


def _declare(handle):
    for name, (res, args) in SYMBOLS.items():
        fn = getattr(handle, name)
        fn.restype = _CT[res]
        fn.argtypes = [_CT[a] for a in args]
    return handle


# ------------------------------------------------------------------ helpers --
def sf_padded_rows(rows: int, num_groups: int = 1) -> int:
    return int(lib().fme_sf_padded_rows(rows, num_groups))


def sf_bytes(rows: int, cols: int, block: int, num_groups: int = 1) -> int:
    return int(lib().fme_sf_bytes(rows, cols, block, num_groups))


def colwise_ld(rows: int, num_groups: int = 1) -> int:
    return int(lib().fme_colwise_ld(rows, num_groups))


def route_workspace_bytes(tokens: int, top_k: int, num_experts: int) -> int:
    return int(lib().fme_route_workspace_bytes(tokens, top_k, num_experts))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch

        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        detail = lib().fme_last_cuda_error().decode() if status == 5 else ""
        raise FmeError(status, where, detail)


def _groups(offsets, num_groups):
    if offsets is None:
        return None, 1 if num_groups is None else num_groups
    n = offsets.numel() - 1 if num_groups is None else num_groups
    return offsets, n


def _empty(shape, dtype, device, stream=None):
    """A new tensor for a call on `stream` (None: the current one), from that stream's memory: a block of the current
    stream's, just freed, may still be used by work queued there.  The caller goes on with it on the current stream, so
    its memory waits for that one as well when it is freed."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    outer = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(outer)
    return t


# --------------------------------------------------------------- the five calls --
def quantize_nvfp4_pertoken(x, offsets=None, num_groups=None, *, codes=None, sf=None, row_scale=None,
                            status=None, stream=None):
    """NVFP4 per-token quantization of bf16 x [rows, k] -> (codes [rows, k/2] u8,
    sf (tiled E4M3 scales) u8, row_scale [rows] f32)."""
    import torch

    rows, k = x.shape
    offsets, g = _groups(offsets, num_groups)
    dev = x.device
    if codes is None:
        codes = _empty((rows, k // 2), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty((max(sf_bytes(rows, k, 16, g), 16),), torch.uint8, dev, stream)
    if row_scale is None:
        row_scale = _empty((rows,), torch.float32, dev, stream)
    st = lib().quantize_nvfp4_pertoken(_ptr(x), rows, k, _ptr(offsets), g, _ptr(codes), _ptr(sf), _ptr(row_scale),
                                       _ptr(status), _stream(stream))
    _check(st, "quantize_nvfp4_pertoken")
    return codes, sf, row_scale


def quantize_nvfp4_pertensor(x, offsets=None, num_groups=None, *, codes=None, sf=None, row_scale=None,
                             tensor_amax=None, status=None, stream=None):
    """Standard NVFP4 (one FP32 scale for the tensor) of bf16 x [rows, k] ->
    (codes, sf, row_scale (S in every row), tensor_amax [1])."""
    import torch

    rows, k = x.shape
    offsets, g = _groups(offsets, num_groups)
    dev = x.device
    if codes is None:
        codes = _empty((rows, k // 2), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty((max(sf_bytes(rows, k, 16, g), 16),), torch.uint8, dev, stream)
    if row_scale is None:
        row_scale = _empty((max(rows, 1),), torch.float32, dev, stream)
    if tensor_amax is None:
        tensor_amax = _empty((4,), torch.float32, dev, stream)
    st = lib().quantize_nvfp4_pertensor(_ptr(x), rows, k, _ptr(offsets), g, _ptr(codes), _ptr(sf),
                                        _ptr(row_scale), _ptr(tensor_amax), _ptr(status), _stream(stream))
    _check(st, "quantize_nvfp4_pertensor")
    return codes, sf, row_scale[:rows], tensor_amax[:1]


def swiglu_quantize_nvfp4(gate_up, offsets=None, num_groups=None, *, codes=None, sf=None, row_scale=None, h=None,
                          want_h=True, status=None, stream=None):
    """h = silu(g) * u of gate_up [rows x 2*inter] (bf16), NVFP4-quantized per
    token -> (codes, sf, row_scale, h or None)."""
    import torch

    rows, two_inter = gate_up.shape
    inter = two_inter // 2
    offsets, g = _groups(offsets, num_groups)
    dev = gate_up.device
    if codes is None:
        codes = _empty((rows, inter // 2), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty((max(sf_bytes(rows, inter, 16, g), 16),), torch.uint8, dev, stream)
    if row_scale is None:
        row_scale = _empty((rows,), torch.float32, dev, stream)
    if h is None and want_h:
        h = _empty((rows, inter), torch.bfloat16, dev, stream)
    st = lib().swiglu_quantize_nvfp4(_ptr(gate_up), rows, inter, _ptr(offsets), g, _ptr(codes), _ptr(sf),
                                     _ptr(row_scale), _ptr(h), _ptr(status), _stream(stream))
    _check(st, "swiglu_quantize_nvfp4")
    return codes, sf, row_scale, h


def quantize_mxfp8(x, axis=ROWWISE, offsets=None, num_groups=None, *, codes=None, sf=None, padded_offsets=None,
                   status=None, stream=None):
    """MXFP8 quantization of bf16 x [rows, cols].

    ROWWISE -> (codes [rows, cols] u8, sf tiled E8M0 u8).
    COLWISE -> (codes [cols, ld] u8, sf tiled u8, padded_offsets [G+1] i32, ld)."""
    import torch

    rows, cols = x.shape
    offsets, g = _groups(offsets, num_groups)
    dev = x.device
    if (axis & ~MX_SCALE_CEIL) == ROWWISE:
        if codes is None:
            codes = _empty((rows, cols), torch.uint8, dev, stream)
        if sf is None:
            sf = _empty((max(sf_bytes(rows, cols, 32, g), 16),), torch.uint8, dev, stream)
        st = lib().quantize_mxfp8(_ptr(x), rows, cols, axis, _ptr(offsets), g, _ptr(codes), _ptr(sf), None,
                                  _ptr(status), _stream(stream))
        _check(st, "quantize_mxfp8")
        return codes, sf
    ld = colwise_ld(rows, g)
    if codes is None:
        codes = _empty((cols, ld), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty((max(sf_bytes(cols, ld, 32, 1), 16),), torch.uint8, dev, stream)
    if padded_offsets is None:
        padded_offsets = _empty((g + 1,), torch.int32, dev, stream)
    st = lib().quantize_mxfp8(_ptr(x), rows, cols, axis, _ptr(offsets), g, _ptr(codes), _ptr(sf),
                              _ptr(padded_offsets), _ptr(status), _stream(stream))
    _check(st, "quantize_mxfp8")
    return codes, sf, padded_offsets, ld


def quantize_mxfp8_rowcol(x, offsets=None, num_groups=None, *, row_codes=None, row_sf=None, col_codes=None,
                          col_sf=None, padded_offsets=None, status=None, stream=None):
    """Row-wise and column-wise MXFP8 of bf16 x [rows, cols] in one pass ->
    ((row_codes, row_sf), (col_codes, col_sf, padded_offsets, ld))."""
    import torch

    rows, cols = x.shape
    offsets, g = _groups(offsets, num_groups)
    dev = x.device
    ld = colwise_ld(rows, g)
    if row_codes is None:
        row_codes = _empty((rows, cols), torch.uint8, dev, stream)
    if row_sf is None:
        row_sf = _empty((max(sf_bytes(rows, cols, 32, g), 16),), torch.uint8, dev, stream)
    if col_codes is None:
        col_codes = _empty((cols, ld), torch.uint8, dev, stream)
    if col_sf is None:
        col_sf = _empty((max(sf_bytes(cols, ld, 32, 1), 16),), torch.uint8, dev, stream)
    if padded_offsets is None:
        padded_offsets = _empty((g + 1,), torch.int32, dev, stream)
    st = lib().quantize_mxfp8_rowcol(_ptr(x), rows, cols, _ptr(offsets), g, _ptr(row_codes), _ptr(row_sf),
                                     _ptr(col_codes), _ptr(col_sf), _ptr(padded_offsets), _ptr(status),
                                     _stream(stream))
    _check(st, "quantize_mxfp8_rowcol")
    return (row_codes, row_sf), (col_codes, col_sf, padded_offsets, ld)


def swiglu_backward_quantize_mxfp8(gate_up, dh, offsets=None, num_groups=None, *, row_codes=None, row_sf=None,
                                   col_codes=None, col_sf=None, padded_offsets=None, d_gate_up=None,
                                   want_d=False, status=None, stream=None):
    """d(gate/up) of h = silu(g) * u given dh, quantized to MXFP8 row-wise and
    column-wise -> (row_codes, row_sf, col_codes, col_sf, padded_offsets, ld,
    d_gate_up or None)."""
    import torch

    rows, two_inter = gate_up.shape
    inter = two_inter // 2
    offsets, g = _groups(offsets, num_groups)
    dev = gate_up.device
    ld = colwise_ld(rows, g)
    if row_codes is None:
        row_codes = _empty((rows, two_inter), torch.uint8, dev, stream)
    if row_sf is None:
        row_sf = _empty((max(sf_bytes(rows, two_inter, 32, g), 16),), torch.uint8, dev, stream)
    if col_codes is None:
        col_codes = _empty((two_inter, ld), torch.uint8, dev, stream)
    if col_sf is None:
        col_sf = _empty((max(sf_bytes(two_inter, ld, 32, 1), 16),), torch.uint8, dev, stream)
    if padded_offsets is None:
        padded_offsets = _empty((g + 1,), torch.int32, dev, stream)
    if d_gate_up is None and want_d:
        d_gate_up = _empty((rows, two_inter), torch.bfloat16, dev, stream)
    st = lib().swiglu_backward_quantize_mxfp8(_ptr(gate_up), _ptr(dh), rows, inter, _ptr(offsets), g,
                                              _ptr(row_codes), _ptr(row_sf), _ptr(col_codes), _ptr(col_sf),
                                              _ptr(padded_offsets), _ptr(d_gate_up), _ptr(status), _stream(stream))
    _check(st, "swiglu_backward_quantize_mxfp8")
    return row_codes, row_sf, col_codes, col_sf, padded_offsets, ld, d_gate_up


def grouped_gemm_fwd_nvfp4(a_codes, a_sf, a_scale, b_codes, b_sf, b_scale, offsets, n, k, *, y=None,
                           status=None, stream=None):
    import torch

    m = a_codes.shape[0]
    e = offsets.numel() - 1
    if y is None:
        y = _empty((m, n), torch.bfloat16, a_codes.device, stream)
    st = lib().grouped_gemm_fwd_nvfp4(_ptr(a_codes), _ptr(a_sf), _ptr(a_scale), _ptr(b_codes), _ptr(b_sf),
                                      _ptr(b_scale), _ptr(offsets), e, m, n, k, _ptr(y), _ptr(status),
                                      _stream(stream))
    _check(st, "grouped_gemm_fwd_nvfp4")
    return y


def grouped_gemm_fwd_nvfp4_swiglu(a_codes, a_sf, a_scale, b_codes, b_sf, b_scale, offsets, n, k, *, h=None,
                                  status=None, stream=None):
    """The gate/up projection's NVFP4 forward with SwiGLU in the epilogue:
    h [m x n / 2] = silu(gate) * up (bf16), gate and up the first and last n / 2
    rows of each expert's weights."""
    import torch

    m = a_codes.shape[0]
    e = offsets.numel() - 1
    if h is None:
        h = _empty((m, n // 2), torch.bfloat16, a_codes.device, stream)
    st = lib().grouped_gemm_fwd_nvfp4_swiglu(_ptr(a_codes), _ptr(a_sf), _ptr(a_scale), _ptr(b_codes), _ptr(b_sf),
                                             _ptr(b_scale), _ptr(offsets), e, m, n, k, _ptr(h), _ptr(status),
                                             _stream(stream))
    _check(st, "grouped_gemm_fwd_nvfp4_swiglu")
    return h


def grouped_gemm_fwd_mxfp8(a_codes, a_sf, b_codes, b_sf, offsets, n, k, *, y=None, status=None, stream=None):
    """MXFP8 forward: Y [m x n] bf16 from row-wise MXFP8 of X [m x k] and of the
    stacked weights [E*n x k]."""
    import torch

    m = a_codes.shape[0]
    e = offsets.numel() - 1
    if y is None:
        y = _empty((m, n), torch.bfloat16, a_codes.device, stream)
    st = lib().grouped_gemm_fwd_mxfp8(_ptr(a_codes), _ptr(a_sf), _ptr(b_codes), _ptr(b_sf), _ptr(offsets), e, m, n, k,
                                      _ptr(y), _ptr(status), _stream(stream))
    _check(st, "grouped_gemm_fwd_mxfp8")
    return y


def grouped_gemm_dgrad_mxfp8(a_codes, a_sf, b_codes, b_sf, ldb, offsets, n, k, *, y=None, status=None,
                             stream=None):
    import torch

    m = a_codes.shape[0]
    e = offsets.numel() - 1
    if y is None:
        y = _empty((m, n), torch.bfloat16, a_codes.device, stream)
    st = lib().grouped_gemm_dgrad_mxfp8(_ptr(a_codes), _ptr(a_sf), _ptr(b_codes), _ptr(b_sf), ldb, _ptr(offsets),
                                        e, m, n, k, _ptr(y), _ptr(status), _stream(stream))
    _check(st, "grouped_gemm_dgrad_mxfp8")
    return y


def grouped_gemm_wgrad_mxfp8(a_codes, a_sf, lda, b_codes, b_sf, ldb, padded_offsets, m, n, *, y=None,
                             status=None, stream=None):
    import torch

    e = padded_offsets.numel() - 1
    if y is None:
        y = _empty((e, m, n), torch.bfloat16, padded_offsets.device, stream)
    st = lib().grouped_gemm_wgrad_mxfp8(_ptr(a_codes), _ptr(a_sf), lda, _ptr(b_codes), _ptr(b_sf), ldb,
                                        _ptr(padded_offsets), e, m, n, _ptr(y), _ptr(status), _stream(stream))
    _check(st, "grouped_gemm_wgrad_mxfp8")
    return y


# ------------------------------------------------------------------ routing --
def moe_route(topk_ids, num_experts, *, offsets=None, row_of=None, src_row=None, workspace=None, status=None,
              stream=None):
    """Group the assignments of topk_ids [tokens, top_k] (int32 expert ids) by
    expert, stably -> (offsets [E+1], row_of [tokens, top_k], src_row [tokens*top_k]),
    all int32."""
    import torch

    tokens, top_k = topk_ids.shape
    dev = topk_ids.device
    if offsets is None:
        offsets = _empty((num_experts + 1,), torch.int32, dev, stream)
    if row_of is None:
        row_of = _empty((tokens, top_k), torch.int32, dev, stream)
    if src_row is None:
        src_row = _empty((tokens * top_k,), torch.int32, dev, stream)
    need = route_workspace_bytes(tokens, top_k, num_experts)
    if workspace is None:
        workspace = _empty((need,), torch.uint8, dev, stream)
    st = lib().moe_route(_ptr(topk_ids), tokens, top_k, num_experts, _ptr(offsets), _ptr(row_of), _ptr(src_row),
                         _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                         _stream(stream))
    _check(st, "moe_route")
    return offsets, row_of, src_row


def moe_route_noalloc(topk_ids, num_experts, offsets, row_of, src_row, *, status=None, stream=None):
    """moe_route into caller-owned outputs, with the library's static counters as
    the workspace: neither this call nor the library allocates memory."""
    import torch

    tokens, top_k = topk_ids.shape
    for name, t, n in (("topk_ids", topk_ids, tokens * top_k), ("offsets", offsets, num_experts + 1),
                       ("row_of", row_of, tokens * top_k), ("src_row", src_row, tokens * top_k)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"moe_route_noalloc: {name} must be a contiguous int32 CUDA tensor of {n} elements")
        if t.device != topk_ids.device:
            raise ValueError(f"moe_route_noalloc: {name} is on {t.device}, topk_ids on {topk_ids.device}")
    st = lib().moe_route_noalloc(_ptr(topk_ids), tokens, top_k, num_experts, _ptr(offsets), _ptr(row_of),
                                 _ptr(src_row), _ptr(status), _stream(stream))
    _check(st, "moe_route_noalloc")
    return offsets, row_of, src_row


def permute_quantize_nvfp4(x, src_row, top_k, offsets, *, codes=None, sf=None, row_scale=None, status=None,
                           stream=None):
    """NVFP4 per-token quantization of the grouped rows x[src_row // top_k] ->
    (codes [tokens*top_k, k/2], sf, row_scale [tokens*top_k])."""
    import torch

    tokens, k = x.shape
    rows = tokens * top_k
    g = offsets.numel() - 1
    dev = x.device
    if codes is None:
        codes = _empty((rows, k // 2), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty((max(sf_bytes(rows, k, 16, g), 16),), torch.uint8, dev, stream)
    if row_scale is None:
        row_scale = _empty((rows,), torch.float32, dev, stream)
    st = lib().permute_quantize_nvfp4(_ptr(x), tokens, k, _ptr(src_row), top_k, _ptr(offsets), g, _ptr(codes),
                                      _ptr(sf), _ptr(row_scale), _ptr(status), _stream(stream))
    _check(st, "permute_quantize_nvfp4")
    return codes, sf, row_scale


def permute_quantize_mxfp8(x, src_row, top_k, offsets, *, codes=None, sf=None, status=None, stream=None):
    """MXFP8 row-wise quantization of the grouped rows x[src_row // top_k] ->
    (codes [tokens*top_k, k], sf)."""
    import torch

    tokens, k = x.shape
    rows = tokens * top_k
    g = offsets.numel() - 1
    dev = x.device
    if codes is None:
        codes = _empty((rows, k), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty((max(sf_bytes(rows, k, 32, g), 16),), torch.uint8, dev, stream)
    st = lib().permute_quantize_mxfp8(_ptr(x), tokens, k, _ptr(src_row), top_k, _ptr(offsets), g, _ptr(codes),
                                      _ptr(sf), _ptr(status), _stream(stream))
    _check(st, "permute_quantize_mxfp8")
    return codes, sf


def moe_combine(y, row_of, weights, *, out=None, status=None, stream=None):
    """out[t] = bf16(sum_k weights[t, k] * y[row_of[t, k]]) (fp32, k in order) for
    grouped expert outputs y [rows_y, n] bf16 -> out [tokens, n] bf16."""
    import torch

    rows_y, n = y.shape
    tokens, top_k = row_of.shape
    if out is None:
        out = _empty((tokens, n), torch.bfloat16, y.device, stream)
    st = lib().moe_combine(_ptr(y), rows_y, _ptr(row_of), _ptr(weights), tokens, top_k, n, _ptr(out), _ptr(status),
                           _stream(stream))
    _check(st, "moe_combine")
    return out


def grouped_gemm_wgrad_mxfp8_accumulate(a_codes, a_sf, lda, b_codes, b_sf, ldb, padded_offsets, m, n, dw_acc, *,
                                        status=None, stream=None):
    """dw_acc [E, m, n] (fp32) += dY_e^T H_e, the wgrad's fp32 result per expert."""
    e = padded_offsets.numel() - 1
    st = lib().grouped_gemm_wgrad_mxfp8_accumulate(_ptr(a_codes), _ptr(a_sf), lda, _ptr(b_codes), _ptr(b_sf), ldb,
                                                   _ptr(padded_offsets), e, m, n, _ptr(dw_acc), _ptr(status),
                                                   _stream(stream))
    _check(st, "grouped_gemm_wgrad_mxfp8_accumulate")
    return dw_acc


# ------------------------------------------------------------ FP8 block-128 --
_native = None


def _bind():
    """The compiled half of the binding (csrc/binding.cpp): checks the tensors (ValueError), allocates outputs, calls
    the library.  Raises if it has not been built."""
    global _native
    if _native is None:
        lib()
        import torch  # noqa: F401  (the module's symbols come from torch's libraries)

        from .build import binding_target

        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the binding is missing or was built for another torch: build it with "
                               "`python -m fp8_moe_expert_gb300.build`") from e
        if _binding.built_for != binding_target():
            raise RuntimeError(f"the binding was built for {_binding.built_for}, this is {binding_target()}: build it "
                               "with `python -m fp8_moe_expert_gb300.build`")
        _binding.set_error(FmeError)
        _native = _binding
    return _native


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def quantize_fp8_block128(x, axis=ROWWISE, offsets=None, num_groups=None, *, src_row=None, top_k=1, codes=None,
                          scale=None, padded_offsets=None, status=None, stream=None):
    """FP8 (E4M3) of bf16 x [rows, cols] with one fp32 scale per 128 values.

    ROWWISE -> (codes [rows, cols] u8, scale [ceil(cols/128), rows] f32); with src_row
    (int32 [tokens*top_k], from moe_route) the rows are x[src_row // top_k].
    COLWISE -> (codes [ld, cols] u8, scale [ld/128, cols] f32, padded_offsets [G+1] i32),
    blocks along each group's rows, each group padded with zeros to a multiple of 128."""
    if axis == ROWWISE:
        return _bind().quantize_rows(x, src_row, top_k, codes, scale, status, _raw(stream))
    if axis != COLWISE:
        raise FmeError(ERR_INVALID_ARGUMENT, "quantize_fp8_block128")
    if src_row is not None:
        raise ValueError("quantize_fp8_block128: src_row is for ROWWISE only")
    return _bind().quantize_cols(x, offsets, num_groups, codes, scale, padded_offsets, status, _raw(stream))


def quantize_fp8_block128_rowcol(x, offsets=None, num_groups=None, *, row_codes=None, row_scale=None, col_codes=None,
                                 col_scale=None, padded_offsets=None, status=None, stream=None):
    """Both layouts of quantize_fp8_block128 from one read of x ->
    ((row_codes, row_scale), (col_codes, col_scale, padded_offsets))."""
    r = _bind().quantize_rowcol(x, offsets, num_groups, row_codes, row_scale, col_codes, col_scale, padded_offsets,
                                status, _raw(stream))
    return r[:2], r[2:]


def quantize_fp8_block128_weights(w, *, codes=None, scale=None, stream=None):
    """FP8 of expert weights w [E, n, k] (bf16) with one fp32 scale per 128 x 128 block ->
    (codes [E, n, k] u8, scale [E, ceil(n/128), ceil(k/128)] f32)."""
    return _bind().quantize_weights(w, codes, scale, _raw(stream))


def grouped_gemm_fwd_fp8_block128(a_codes, a_scale, w_codes, w_scale, offsets, *, y=None, status=None, stream=None):
    """Y [m, n] (bf16) = X_e W_e^T per expert, from quantize_fp8_block128(ROWWISE) of
    X [m, k] and quantize_fp8_block128_weights of W [E, n, k]."""
    return _bind().fwd(a_codes, a_scale, w_codes, w_scale, offsets, y, status, _raw(stream))


def grouped_gemm_dgrad_fp8_block128(dy_codes, dy_scale, w_codes, w_scale, offsets, *, dx=None, status=None,
                                    stream=None):
    """dX [m, k] (bf16) = dY_e W_e per expert, from quantize_fp8_block128(ROWWISE) of
    dY [m, n] and the forward's weight codes."""
    return _bind().dgrad(dy_codes, dy_scale, w_codes, w_scale, offsets, dx, status, _raw(stream))


def grouped_gemm_wgrad_fp8_block128(dy_codes, dy_scale, x_codes, x_scale, padded_offsets, *, dw=None, dtype=None,
                                    accumulate=False, status=None, stream=None):
    """dW [E, n, k] = dY_e^T X_e per expert, from quantize_fp8_block128(COLWISE) of dY [rows, n]
    and X [rows, k] with the same offsets.  dtype bfloat16 (default) or float32; with accumulate
    the result is added into dw (float32)."""
    mode = _dw_mode("grouped_gemm_wgrad_fp8_block128", dw, dtype, accumulate)
    return _bind().wgrad(dy_codes, dy_scale, x_codes, x_scale, padded_offsets, dw, mode, status, _raw(stream))


def _dw_mode(where, dw, dtype, accumulate):
    import torch

    if dtype is None:
        dtype = torch.bfloat16 if dw is None else dw.dtype
    if dtype not in (torch.bfloat16, torch.float32) or (accumulate and (dw is None or dtype != torch.float32)):
        raise ValueError(f"{where}: dw is bfloat16 or float32, and a given float32 tensor to accumulate into")
    return DW_BF16 if dtype == torch.bfloat16 else DW_FP32_ADD if accumulate else DW_FP32


# ------------------------------------------------------------ bf16 products --
def grouped_gemm_fwd_bf16(x, w, offsets, *, y=None, status=None, stream=None):
    """Y [m, n] (bf16) = X_e W_e^T per expert, from bf16 rows x [m, k] grouped by expert (moe_permute) and weights
    w [E, n, k]; offsets int32 [E+1].  n and k are multiples of 8."""
    return _bind().fwd_bf16(x, w, offsets, y, status, _raw(stream))


def grouped_gemm_dgrad_bf16(dy, w, offsets, *, dx=None, status=None, stream=None):
    """dX [m, k] (bf16) = dY_e W_e per expert, from dy [m, n] and the forward's weights."""
    return _bind().dgrad_bf16(dy, w, offsets, dx, status, _raw(stream))


def grouped_gemm_wgrad_bf16(dy, x, offsets, *, dw=None, dtype=None, accumulate=False, status=None, stream=None):
    """dW [E, n, k] = dY_e^T X_e per expert, from dy [m, n] and x [m, k] grouped with the same offsets.  dtype bfloat16
    (default) or float32; with accumulate the result is added into dw (float32)."""
    mode = _dw_mode("grouped_gemm_wgrad_bf16", dw, dtype, accumulate)
    return _bind().wgrad_bf16(dy, x, offsets, dw, mode, status, _raw(stream))


def moe_permute(x, src_row, top_k, *, out=None, status=None, stream=None):
    """The bf16 rows x[src_row // top_k] in grouped order -> out [tokens*top_k, n]; src_row int32 from moe_route.  Its
    gradient is moe_combine of the rows' gradients with weights 1."""
    return _bind().permute(x, src_row, top_k, out, status, _raw(stream))


def swiglu(gate_up, *, h=None, stream=None):
    """h [rows, inter] = silu(g) * u of gate_up [rows, 2*inter] = [g | u] (bf16): the h of swiglu_quantize_nvfp4."""
    return _bind().swiglu(gate_up, h, _raw(stream))


def swiglu_backward(gate_up, dh, *, d_gate_up=None, stream=None):
    """The gradient of swiglu for dh [rows, inter] -> d_gate_up [rows, 2*inter] (bf16)."""
    return _bind().swiglu_backward(gate_up, dh, d_gate_up, _raw(stream))


# ------------------------------------------------- NVFP4 weights, few rows --
def grouped_gemv_nvfp4(x, w_codes, w_sf, w_scale, offsets, *, src_row=None, top_k=1, y=None, status=None, stream=None):
    """Y [m, n] (bf16) = X_e W_e^T per expert for few bf16 rows and NVFP4 weights: w_codes [E*n, k/2], w_sf and w_scale
    [E*n] from quantize_nvfp4_pertoken of W [E*n, k] as one group; x [m, k], or with src_row (int32 [tokens*top_k], from
    moe_route) the rows x[src_row // top_k] of x [tokens, k].  k is a multiple of 64."""
    return _bind().gemv(x, w_codes, w_sf, w_scale, offsets, src_row, top_k, y, status, _raw(stream))


def grouped_gemv_nvfp4_swiglu(x, w_codes, w_sf, w_scale, offsets, *, src_row=None, top_k=1, h=None, status=None,
                              stream=None):
    """grouped_gemv_nvfp4 of the gate/up weights with the activation: h [m, n/2] = silu(gate) * up (bf16), gate and up the
    first and last n/2 rows of each expert's weights, not rounded in between.  n is a multiple of 256."""
    return _bind().gemv_swiglu(x, w_codes, w_sf, w_scale, offsets, src_row, top_k, h, status, _raw(stream))


# ------------------------------------------------------------------- router --
def moe_gate(logits, top_k, *, score="softmax", bias=None, normalize=True, scale=1.0, ids=None, weights=None,
             stream=None):
    """The top_k experts of each token by logits [tokens, E] (+ bias [E]), largest first, and
    their weights, scale * s / sum of the chosen s (normalize) or scale * s, s the softmax or
    sigmoid of the logits -> (ids [tokens, top_k] int32, weights [tokens, top_k] f32)."""
    return _bind().gate(logits, top_k, score, bias, normalize, scale, ids, weights, _raw(stream))


def moe_gate_backward(logits, ids, d_weights, *, score="softmax", normalize=True, scale=1.0, d_logits=None, status=None,
                      stream=None):
    """The gradient of moe_gate's weights -> d_logits [tokens, E] in the logits' type."""
    return _bind().gate_backward(logits, ids, d_weights, score, normalize, scale, d_logits, status, _raw(stream))


def balance_workspace_bytes(tokens: int, num_seqs: int, num_experts: int) -> int:
    return int(lib().fme_balance_workspace_bytes(tokens, num_seqs, num_experts))


def moe_balance_loss(logits, ids, *, score="softmax", alpha=1.0, seq_offsets=None, token_mask=None, loss=None,
                     counts=None, seq_tokens=None, workspace=None, status=None, stream=None):
    """alpha times the sequence-wise load-balance loss of routing logits [tokens, E] to ids
    [tokens, top_k] -> (loss [1] f32, counts [S, E] int32, seq_tokens [S] int32).

    seq_offsets: int32 [S+1], rising from 0 to tokens (None: one sequence); token_mask: bool or
    uint8 [tokens], the tokens that count (None: all)."""
    return _bind().balance_loss(logits, ids, score, alpha, seq_offsets, token_mask, loss, counts, seq_tokens, workspace,
                                status, _raw(stream))


def moe_balance_loss_backward(logits, counts, seq_tokens, d_loss, top_k, *, score="softmax", alpha=1.0,
                              seq_offsets=None, token_mask=None, d_logits=None, accumulate=False, stream=None):
    """The gradient of d_loss [1] times moe_balance_loss -> d_logits [tokens, E] in the logits'
    type; with accumulate it is added to the given d_logits."""
    return _bind().balance_loss_backward(logits, counts, seq_tokens, d_loss, top_k, score, alpha, seq_offsets, token_mask,
                                         d_logits, accumulate, _raw(stream))


def moe_combine_backward(d_out, y, row_of, weights, *, d_y=None, d_weights=None, status=None, stream=None):
    """The gradient of moe_combine for d_out [tokens, n] bf16 -> (d_y [rows_y, n] bf16,
    d_weights [tokens, top_k] f32)."""
    return _bind().combine_backward(d_out, y, row_of, weights, d_y, d_weights, status, _raw(stream))


def read_device_status(status, stream=None) -> tuple[int, int]:
    """Synchronise the stream and read a device status word -> (status code, raw bits)."""
    raw = ctypes.c_int32(0)
    st = lib().fme_read_device_status(_ptr(status), _stream(stream), ctypes.byref(raw))
    return int(st), int(raw.value)
