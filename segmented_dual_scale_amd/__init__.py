"""segmented_dual_scale_amd -- SegQuant's DualScale x SegLinear W8A8 linear
layer on AMD Instinct MI355X (gfx950).

This module is a thin ctypes binding over the C ABI of ``libsegquant.so``
(``include/segquant.h``).  Each function has the name of its C entry point and
only marshals arguments: torch supplies device memory and the current HIP
stream, every step of the layer runs in the library's HIP kernels.  If the
library is not built, every call raises: there is no other path.

    from segmented_dual_scale_amd import (segquant_calibrate_amax,
        segquant_quantize_weight, segquant_gemm_w8a8_seg)
    act = segquant_calibrate_amax(x, kseg=[64] * 24)            # offline
    wq, ws = segquant_quantize_weight(w, kseg=[64] * 24)        # offline
    y = segquant_gemm_w8a8_seg(x, wq, ws, act, kseg=[64] * 24)  # one launch

Pages: "SegQuant: A Semantics-Aware and Generalizable Quantization Framework
for Diffusion Models" (papernotes.org notes, "SegLinear" and "DualScale"
sections) and "SegQuant" (hliangzhao.me, sections 2 and 3).
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence, Tuple

__all__ = [
    "SegQuantError", "library_path", "load_library",
    "segquant_calibrate_amax", "segquant_quantize_dualscale", "segquant_weight_packed_bytes",
    "segquant_quantize_weight", "segquant_unpack_weight", "segquant_gemm_w8a8_seg",
    "segquant_gemm_kernel_for", "segquant_status_string", "segquant_last_error",
    "segquant_version", "SEGQ_Q_SIGNED", "SEGQ_Q_PLANES", "SEGQ_GEMM_AUTO",
    "SEGQ_GEMM_FORCE_TILE", "SEGQ_GEMM_FORCE_SMALLM", "SEGQ_GEMM_FUSED_QUANT",
    "SEGQ_GEMM_SINGLE_SCALE", "segquant_calibrate_amax_single",
    "SEGQ_ACT_SILU", "SEGQ_ACT_GELU", "segquant_activate_quantize", "SEGQ_GEMM_W4", "SEGQ_KERNEL_TILE", "SEGQ_KERNEL_SMALLM",
    "segquant_gemm_halves", "segquant_gemm_w8a8_seg_noalloc", "SEGQ_NOALLOC_SCRATCH_BYTES",
    "SEGQ_ACT_NONE", "segquant_groupnorm_workspace_bytes", "segquant_groupnorm_quantize",
    "segquant_adanorm_quantize", "segquant_adapter_workspace_bytes", "segquant_adapter_add",
    "SEGQ_ADAPTER_RANK_STEP", "SEGQ_ADAPTER_RANK_MAX", "segquant_rmsnorm_quantize",
    "segquant_mxfp4_bytes", "segquant_quantize_mxfp4", "segquant_quantize_weight_mxfp4",
    "segquant_unpack_mxfp4", "segquant_gemm_mxfp4", "segquant_gemm_mxfp4_workspace_bytes",
    "SEGQ_ROTARY_PAIRS", "SEGQ_ROTARY_HALVES", "SEGQ_ROTARY_MAX_AXES", "SEGQ_ROTARY_MAX_HEAD",
    "segquant_rotary_frequencies", "segquant_qk_rotary",
]

SEGQ_OK = 0
SEGQ_ERR_NULL = -1
SEGQ_ERR_SHAPE = -2
SEGQ_ERR_SEGMENTS = -3
SEGQ_ERR_ALIGN = -4
SEGQ_ERR_UNSUPPORTED = -5
SEGQ_ERR_HIP = -6
SEGQ_MAX_KSEG = 128
SEGQ_MAX_KSEG_WIDTH = 132104
SEGQ_Q_SIGNED = 0
SEGQ_Q_PLANES = 1
SEGQ_GEMM_AUTO = 0
SEGQ_GEMM_FORCE_TILE = 1
SEGQ_GEMM_FORCE_SMALLM = 2
SEGQ_GEMM_FUSED_QUANT = 4
SEGQ_GEMM_SINGLE_SCALE = 8
SEGQ_GEMM_W4 = 16
SEGQ_ACT_NONE = 0
SEGQ_ACT_SILU = 1
SEGQ_ACT_GELU = 2
SEGQ_KERNEL_TILE = 1
SEGQ_KERNEL_SMALLM = 2
SEGQ_NOALLOC_SCRATCH_BYTES = 64 << 20
SEGQ_ADAPTER_RANK_STEP = 16
SEGQ_ADAPTER_RANK_MAX = 256
SEGQ_ROTARY_PAIRS = 0
SEGQ_ROTARY_HALVES = 1
SEGQ_ROTARY_MAX_AXES = 8
SEGQ_ROTARY_MAX_HEAD = 512

_HERE = os.path.dirname(os.path.abspath(__file__))
# SEGQUANT_LIBRARY names another build of the same library (the tests use it
# for a build whose host code carries address and undefined-behaviour
# sanitizers); by default the in-tree build is loaded.
_LIB_PATH = os.environ.get("SEGQUANT_LIBRARY") or os.path.join(_HERE, "libsegquant.so")
_lib = None


class SegQuantError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({segquant_status_string(status)}): {detail}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libsegquant.so (built in-tree by segmented_dual_scale_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run `python -m segmented_dual_scale_amd.build` "
                           "(the layer has no other implementation)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
    F32 = ctypes.c_float
    sig = {
        "segquant_calibrate_amax": [P, I64, I64, I64, I32, P, P, P, P],
        "segquant_calibrate_amax_single": [P, I64, I64, I64, I32, P, P, P, P],
        "segquant_activate_quantize": [P, I64, I64, I64, I32, I32, P, P, P, P, I64, I32, P, I64,
                                       P],
        "segquant_quantize_dualscale": [P, I64, I64, I64, I32, P, P, P, P, I64, I32, P],
        "segquant_quantize_weight": [P, I64, I64, I64, I32, P, P, I32, P, P, I32, P, P, P],
        "segquant_unpack_weight": [P, I64, I64, P, I64, P],
        "segquant_unpack_weight_w4": [P, I64, I64, P, I64, P],
        "segquant_quantize_weight_w4": [P, I64, I64, I64, I32, P, P, I32, P, P, I32, P, P, P],
        "segquant_weight_packed_bytes_w4": [I64, I64],
        "segquant_gemm_w8a8_seg": [I64, I64, I64, P, I64, P, I64, I32, P, P, I32, P, P, P, P, I64,
                                   P, P, ctypes.c_size_t, U32, P],
        "segquant_gemm_w8a8_seg_noalloc": [I64, I64, I64, P, I64, P, I64, I32, P, P, I32, P, P,
                                           P, P, I64, P, U32, P],
        "segquant_gemm_workspace_bytes": [I64, I64, I64, I32, P, P, U32],
        "segquant_gemm_kernel_for": [I64, I64, I64, U32],
        "segquant_groupnorm_quantize": [P, I64, I64, I64, I64, I32, F32, P, P, P, P, I64, I32, I32,
                                        P, P, P, P, I64, I32, P, I64, P, ctypes.c_size_t, P],
        "segquant_groupnorm_workspace_bytes": [I64, I64, I64, I32],
        "segquant_adanorm_quantize": [P, I64, I64, I64, P, I64, P, P, I64, F32, P, P, P, P, I64,
                                      I32, P, I32, P, P, P, P, I64, I32, P, I64, P],
        "segquant_adapter_add": [I64, I64, I64, P, I64, I32, P, P, I32, I32, P, P, P, P, I32, P, P,
                                 P, I64, P, I64, P, ctypes.c_size_t, P],
        "segquant_adapter_workspace_bytes": [I64, I64, I64, I32, I32, I32, P, P],
        "segquant_mxfp4_code_bytes": [I64, I64],
        "segquant_mxfp4_scale_bytes": [I64, I64],
        "segquant_quantize_mxfp4": [P, I64, I64, I64, I32, P, P, P],
        "segquant_quantize_weight_mxfp4": [P, I64, I64, I64, P, P, P],
        "segquant_unpack_mxfp4": [P, P, I64, I64, P, I64, P],
        "segquant_gemm_mxfp4": [I64, I64, I64, P, I64, I32, P, P, P, P, P, I64, P,
                                ctypes.c_size_t, P],
        "segquant_gemm_mxfp4_workspace_bytes": [I64, I64, I64],
        "segquant_rmsnorm_quantize": [P, I64, I64, I64, P, I64, P, I64, F32, P, I32, P, P, P, P,
                                      I64, I32, P, I64, P, P, P],
        "segquant_rotary_frequencies": [I32, P, ctypes.c_double, P],
        "segquant_qk_rotary": [I64, I64, I32, P, I32, P, P, P, P, I32, P, P, P, I32, F32, P, P, P,
                               I64, I32, P, P, I32, P],
        "segquant_gemm_halves": [P, I32],
        "segquant_version": [],
        "segquant_status_string": [ctypes.c_int],
        "segquant_last_error": [],
        "segquant_weight_packed_bytes": [I64, I64],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.segquant_status_string.restype = ctypes.c_char_p
    lib.segquant_last_error.restype = ctypes.c_char_p
    lib.segquant_weight_packed_bytes.restype = ctypes.c_size_t
    lib.segquant_weight_packed_bytes_w4.restype = ctypes.c_size_t
    lib.segquant_gemm_workspace_bytes.restype = ctypes.c_size_t
    lib.segquant_groupnorm_workspace_bytes.restype = ctypes.c_size_t
    lib.segquant_adapter_workspace_bytes.restype = ctypes.c_size_t
    lib.segquant_mxfp4_code_bytes.restype = ctypes.c_size_t
    lib.segquant_mxfp4_scale_bytes.restype = ctypes.c_size_t
    lib.segquant_gemm_mxfp4_workspace_bytes.restype = ctypes.c_size_t
    _lib = lib
    return lib


# ----------------------------------------------------------------- helpers --
def _segs(widths: Optional[Sequence[int]], total: int):
    return _seg_lists((total,) if widths is None else tuple(map(int, widths)))


@functools.lru_cache(maxsize=256)
def _seg_lists(widths: Tuple[int, ...]):
    """(offsets, widths) as int32 arrays, read only: calls share them."""
    import numpy as np
    w = np.asarray(widths, dtype=np.int32)
    off = np.zeros_like(w)
    if len(w) > 1:
        off[1:] = np.cumsum(w)[:-1]
    off.flags.writeable = w.flags.writeable = False
    return off, w


def _arr_ptr(a):
    return a.ctypes.data if a is not None else None


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(t):
    import torch
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    # torch.cuda.current_stream() takes 2 us
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _check(rc: int, where: str):
    if rc != SEGQ_OK:
        raise SegQuantError(rc, where, segquant_last_error())


def _ld(t, what: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{what} must be a 2-D tensor with unit stride in its last dimension")
    return t.stride(0)


# --------------------------------------------------------------- the ABI ----
def segquant_status_string(status: int) -> str:
    return load_library().segquant_status_string(status).decode()


def segquant_last_error() -> str:
    return load_library().segquant_last_error().decode()


def segquant_version() -> int:
    return load_library().segquant_version()


def segquant_weight_packed_bytes(K: int, N: int) -> int:
    return int(load_library().segquant_weight_packed_bytes(K, N))


def segquant_gemm_kernel_for(M: int, N: int, K: int, flags: int = SEGQ_GEMM_AUTO) -> int:
    return int(load_library().segquant_gemm_kernel_for(M, N, K, flags))


def segquant_gemm_halves(act) -> int:
    """SEGQ_GEMM_SINGLE_SCALE when the scale table `act` ([4][n_kseg], device
    or host tensor, or a numpy array) has no negative half, else 0.  A device
    table is copied to the host (once per layer: the scales are static)."""
    import numpy as np
    if hasattr(act, "detach"):
        act = act.detach().cpu().numpy()
    a = np.ascontiguousarray(np.asarray(act, dtype=np.float32))
    if a.ndim != 2 or a.shape[0] != 4:
        raise ValueError(f"scale table of shape {a.shape}, expected [4][n_kseg]")
    r = load_library().segquant_gemm_halves(a.ctypes.data, a.shape[1])
    if r < 0:
        raise SegQuantError(r, "segquant_gemm_halves", segquant_last_error())
    return int(r)


def _calibrate(fn, name, x, kseg, out):
    import torch
    M, K = x.shape
    off, wid = _segs(kseg, K)
    if out is None:
        out = torch.empty((4, len(wid)), dtype=torch.float32, device=x.device)
    _check(fn(_ptr(x), M, K, _ld(x, "x"), len(wid), _arr_ptr(off), _arr_ptr(wid), _ptr(out),
              _stream(x)), name)
    return out


def segquant_calibrate_amax(x, kseg: Optional[Sequence[int]] = None, out=None):
    """AMax calibration: returns the fp32 [4][n_kseg] table (s+, s-, inv+,
    inv-) for bf16 X [M][K] (device)."""
    return _calibrate(load_library().segquant_calibrate_amax, "segquant_calibrate_amax", x, kseg,
                      out)


def segquant_calibrate_amax_single(x, kseg: Optional[Sequence[int]] = None, out=None):
    """Single-scale calibration: the same table layout with s+ = s- =
    max|x|/127 and inv+ = inv- = 127/max|x| per K-segment (use with
    SEGQ_GEMM_SINGLE_SCALE)."""
    return _calibrate(load_library().segquant_calibrate_amax_single,
                      "segquant_calibrate_amax_single", x, kseg, out)


def segquant_quantize_dualscale(x, act_scales, kseg: Optional[Sequence[int]] = None,
                                layout: int = SEGQ_Q_SIGNED, out=None):
    """Polarity split + dual-scale quantisation of bf16 X -> int8: [M][K]
    signed codes, or [2][M][K] planes (q+, q-)."""
    import torch
    lib = load_library()
    M, K = x.shape
    off, wid = _segs(kseg, K)
    if out is None:
        ldq = (K + 15) // 16 * 16
        shape = (M, ldq) if layout == SEGQ_Q_SIGNED else (2, M, ldq)
        out = torch.empty(shape, dtype=torch.int8, device=x.device)
    ld_q = out.stride(-2)
    _check(lib.segquant_quantize_dualscale(_ptr(x), M, K, _ld(x, "x"), len(wid), _arr_ptr(off),
                                           _arr_ptr(wid), _ptr(act_scales), _ptr(out), ld_q,
                                           layout, _stream(x)),
           "segquant_quantize_dualscale")
    return out


def segquant_activate_quantize(z, act_kind: int, act_scales=None,
                               kseg: Optional[Sequence[int]] = None,
                               layout: int = SEGQ_Q_SIGNED, out=None, x_out=None,
                               want_codes: bool = True):
    """SiLU/GELU of bf16 pre-activation Z fused with the dual-scale
    quantisation.  Returns (codes or None, x_out or None): codes as
    segquant_quantize_dualscale (when act_scales is given and want_codes),
    x_out the bf16 activation if a tensor is passed (or x_out=True to
    allocate one)."""
    import torch
    lib = load_library()
    M, K = z.shape
    off, wid = _segs(kseg, K)
    if want_codes and act_scales is not None and out is None:
        ldq = (K + 15) // 16 * 16
        shape = (M, ldq) if layout == SEGQ_Q_SIGNED else (2, M, ldq)
        out = torch.empty(shape, dtype=torch.int8, device=z.device)
    if not (want_codes and act_scales is not None):
        out = None
    if x_out is True:
        x_out = torch.empty((M, K), dtype=torch.bfloat16, device=z.device)
    ld_q = out.stride(-2) if out is not None else 0
    ld_xo = _ld(x_out, "x_out") if x_out is not None else 0
    _check(lib.segquant_activate_quantize(_ptr(z), M, K, _ld(z, "z"), act_kind, len(wid),
                                          _arr_ptr(off), _arr_ptr(wid), _ptr(act_scales), _ptr(out),
                                          ld_q, layout, _ptr(x_out), ld_xo, _stream(z)),
           "segquant_activate_quantize")
    return out, x_out


def segquant_quantize_weight(w, kseg: Optional[Sequence[int]] = None,
                             nseg: Optional[Sequence[int]] = None, per_column: bool = False,
                             out_packed=None, out_scale=None, bits: int = 8) -> Tuple:
    """Per-group symmetric int8 (bits=8) or 4-bit (bits=4, W4A8) quantisation
    of fp32 W [K][N] (device): returns (packed weight, fp32 w_scale
    [n_kseg][N])."""
    import torch
    lib = load_library()
    if bits not in (4, 8):
        raise ValueError("bits must be 8 or 4")
    K, N = w.shape
    koff, kwid = _segs(kseg, K)
    noff, nwid = _segs(nseg, N)
    if out_packed is None:
        nbytes = (segquant_weight_packed_bytes(K, N) if bits == 8
                  else int(lib.segquant_weight_packed_bytes_w4(K, N)))
        out_packed = torch.empty(max(nbytes, 16), dtype=torch.int8, device=w.device)
    if out_scale is None:
        out_scale = torch.empty((len(kwid), N), dtype=torch.float32, device=w.device)
    fn = lib.segquant_quantize_weight if bits == 8 else lib.segquant_quantize_weight_w4
    _check(fn(_ptr(w), K, N, _ld(w, "w"), len(kwid), _arr_ptr(koff), _arr_ptr(kwid), len(nwid),
              _arr_ptr(noff), _arr_ptr(nwid), int(bool(per_column)), _ptr(out_packed),
              _ptr(out_scale), _stream(w)),
           "segquant_quantize_weight" + ("" if bits == 8 else "_w4"))
    return out_packed, out_scale


def segquant_unpack_weight(w_packed, K: int, N: int, out=None, bits: int = 8):
    """Packed weight (int8, or 4-bit with bits=4) -> int8 W_q [K][N]."""
    import torch
    lib = load_library()
    if out is None:
        out = torch.empty((K, N), dtype=torch.int8, device=w_packed.device)
    fn = lib.segquant_unpack_weight if bits == 8 else lib.segquant_unpack_weight_w4
    _check(fn(_ptr(w_packed), K, N, _ptr(out), _ld(out, "out"), _stream(w_packed)),
           "segquant_unpack_weight" + ("" if bits == 8 else "_w4"))
    return out


def segquant_gemm_workspace_bytes(M: int, N: int, K: int, kseg: Optional[Sequence[int]] = None,
                                  flags: int = SEGQ_GEMM_AUTO) -> int:
    off, wid = _segs(kseg, K)
    return int(load_library().segquant_gemm_workspace_bytes(M, N, K, len(wid), _arr_ptr(off),
                                                            _arr_ptr(wid), flags))


def segquant_gemm_w8a8_seg(x, w_packed, w_scale, act_scales, kseg: Optional[Sequence[int]] = None,
                           N: Optional[int] = None, xq=None, q_layout: int = SEGQ_Q_SIGNED,
                           out=None, acc_debug=None, workspace="auto",
                           flags: int = SEGQ_GEMM_AUTO):
    """The DualScale x SegLinear W8A8 layer (one launch, or quantisation
    then GEMM when a workspace is given and the library asks for one).

    x: bf16 [M][K] (or None with xq = the output of
    segquant_quantize_dualscale); w_packed/w_scale from
    segquant_quantize_weight; act_scales from segquant_calibrate_amax.
    Returns bf16 Y [M][N].  acc_debug, if given, is an int32 tensor
    [2][n_kseg][M][N] that receives the per-segment accumulators.
    workspace: a device tensor, None (always the fused launch), or "auto"
    (a tensor of segquant_gemm_workspace_bytes() bytes from torch's
    allocator when that is nonzero)."""
    import torch
    lib = load_library()
    src = x if x is not None else xq
    if x is not None:
        M, K = x.shape
        ld_x, ld_q = _ld(x, "x"), 0
    else:
        M = xq.shape[-2]
        K = sum(kseg) if kseg is not None else None
        if K is None:
            raise ValueError("kseg is required with a pre-quantised input")
        ld_x, ld_q = 0, xq.stride(-2)
    if N is None:
        N = w_scale.shape[1]
    off, wid = _segs(kseg, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=src.device)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, None or 'auto'")
        nb = segquant_gemm_workspace_bytes(M, N, K, kseg, flags)
        workspace = torch.empty(nb, dtype=torch.uint8, device=src.device) if nb else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.segquant_gemm_w8a8_seg(M, N, K, _ptr(x), ld_x, _ptr(xq), ld_q, q_layout,
                                      _ptr(w_packed), _ptr(w_scale), len(wid), _arr_ptr(off),
                                      _arr_ptr(wid), _ptr(act_scales), _ptr(out), _ld(out, "out"),
                                      _ptr(acc_debug), _ptr(workspace), ws_bytes, flags,
                                      _stream(src)),
           "segquant_gemm_w8a8_seg")
    return out


def segquant_gemm_w8a8_seg_noalloc(x, w_packed, w_scale, act_scales, out,
                                   kseg: Optional[Sequence[int]] = None, N: Optional[int] = None,
                                   xq=None, q_layout: int = SEGQ_Q_SIGNED, acc_debug=None,
                                   flags: int = SEGQ_GEMM_AUTO):
    """segquant_gemm_w8a8_seg through its no-allocation entry point: no
    workspace, no device allocation in the call (the library's own scratch
    array stands in for the workspace).  `out` (bf16 [M][N]) is required:
    this path allocates nothing, here or in the library."""
    lib = load_library()
    src = x if x is not None else xq
    if x is not None:
        M, K = x.shape
        ld_x, ld_q = _ld(x, "x"), 0
    else:
        M = xq.shape[-2]
        if kseg is None:
            raise ValueError("kseg is required with a pre-quantised input")
        K = sum(kseg)
        ld_x, ld_q = 0, xq.stride(-2)
    if N is None:
        N = w_scale.shape[1]
    off, wid = _segs(kseg, K)
    _check(lib.segquant_gemm_w8a8_seg_noalloc(M, N, K, _ptr(x), ld_x, _ptr(xq), ld_q, q_layout,
                                              _ptr(w_packed), _ptr(w_scale), len(wid),
                                              _arr_ptr(off), _arr_ptr(wid), _ptr(act_scales),
                                              _ptr(out), _ld(out, "out"), _ptr(acc_debug), flags,
                                              _stream(src)),
           "segquant_gemm_w8a8_seg_noalloc")
    return out


# ------------------------------------- norms before and adapters beside ----
# These run in microseconds, so the checks look at each operand once.
@functools.lru_cache(maxsize=256)
def _seg_arrays(widths: Tuple[int, ...]):
    off, wid = _seg_lists(widths)
    # the widths as a key, and the arrays that the addresses belong to
    return len(wid), off.ctypes.data, wid.ctypes.data, widths, (off, wid)


def _segments(widths, total: int):
    return _seg_arrays((total,) if widths is None else tuple(map(int, widths)))


def _want(t, name: str, dtype, shape, at: int):
    """Check an operand (None: not given; at: the GPU's index) and return its
    address."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == at and t.shape == shape:
        return t.data_ptr()
    raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on the GPU of the first "
                     f"operand ({at}), got {t.dtype} {tuple(t.shape)} on {t.device}")


def _want_array(t, name: str, dtype, shape, at: int):
    """_want for an operand without a leading dimension of its own."""
    if t is None:
        return None
    if (t.dtype is dtype and t.get_device() == at and t.shape == shape and
            t.is_contiguous()):
        return t.data_ptr()
    _want(t, name, dtype, shape, at)
    raise ValueError(f"{name} must be contiguous")


def _row_ld(t, name: str) -> int:
    """Elements between the rows of a [..., K] tensor whose rows are evenly
    spaced (any value fits a single row)."""
    if t is None:
        return 0
    shape = t.shape
    K = shape[-1]
    if not K & 7 and t.is_contiguous():
        return K
    stride = t.stride()
    if stride[-1] != 1 and K > 1 and t.numel():
        raise ValueError(f"{name} must have unit stride in its last dimension")
    ld, below = None, 1  # rows inside one step of dimension d
    for d in range(len(shape) - 2, -1, -1):
        if shape[d] != 1:
            if ld is None:
                ld = stride[d]
            elif stride[d] != ld * below and t.numel():
                raise ValueError(f"{name}: its rows are not evenly spaced")
            below *= shape[d]
    return -(-K // 8) * 8 if ld is None else ld


def _mod_ld(rows: int, params, names: str) -> int:
    """The row distance that a request's parameters share."""
    ld = None
    for t in params:
        if t is not None:
            if ld is None:
                ld, first = _row_ld(t, names), t
            elif t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError(f"{names} must have unit stride in their last dimension")
            elif rows > 1 and t.stride(0) != first.stride(0):
                raise ValueError(f"{names} must have the same row stride")
    return ld or 0


def _on(at: int, fn, *args):
    """fn(*args, stream) on the current stream of GPU `at`, with it current."""
    import torch
    if at < 0:
        raise ValueError("tensors must be on a GPU")
    stream = torch._C._cuda_getCurrentRawStream(at)  # current_stream() takes 2 us
    if at == torch._C._cuda_getDevice():
        return fn(*args, stream)
    with torch.cuda.device(at):
        return fn(*args, stream)


def _workspace(workspace, size, sizes, device):
    """A workspace argument ("auto": size(*sizes) bytes from torch's
    allocator) -> the tensor to keep, its address and bytes."""
    import torch
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, None or 'auto'")
        nbytes = size(*sizes)
        if not nbytes:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    if workspace is None:
        return None, None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _codes_out(out, M: int, K: int, layout: int, device, new):
    """The int8 output tensor, its address and leading dimension."""
    import torch
    if out is None:
        ldq = (K + 15) // 16 * 16
        out = new((M, ldq) if layout == SEGQ_Q_SIGNED else (2, M, ldq), dtype=torch.int8,
                  device=device)
    planes = layout != SEGQ_Q_SIGNED
    if (out.dtype != torch.int8 or out.device != device or out.dim() != (3 if planes else 2) or
            out.shape[-2] != M or out.shape[-1] < K or (planes and out.shape[0] != 2)):
        raise ValueError(f"out must be an int8 tensor of {'2 planes of ' if planes else ''}{M} rows "
                         f"of at least {K} codes on {device}, got {out.dtype} {tuple(out.shape)} on "
                         f"{out.device}")
    ld = _row_ld(out[0] if planes else out, "out")
    if M <= 1:
        ld = out.stride(0) if planes and M else (out.shape[-1] + 15) // 16 * 16
    if planes and M and out.stride(0) != M * ld:
        raise ValueError("out: the second plane must follow the first")
    return out, out.data_ptr(), ld


def segquant_groupnorm_workspace_bytes(B: int, P: int, C: int, groups: int) -> int:
    return int(load_library().segquant_groupnorm_workspace_bytes(B, P, C, groups))


# workspace sizes depend on the sizes alone
_groupnorm_bytes = functools.lru_cache(maxsize=256)(segquant_groupnorm_workspace_bytes)


def segquant_groupnorm_quantize(z, groups: int, eps: float = 1e-5, gamma=None, beta=None,
                                scale=None, shift=None, act_kind: int = SEGQ_ACT_NONE,
                                act_scales=None, kseg: Optional[Sequence[int]] = None,
                                layout: int = SEGQ_Q_SIGNED, out=None, x_out=None,
                                want_codes: bool = True, workspace="auto"):
    """Channels-last group norm of bf16 z [B][P][C] (P pixels of C channels;
    an image [B][H][W][C] is z.flatten(1, 2)), with optional fp32 gamma and
    beta [C], bf16 modulation scale and shift [B][C], and activation.
    Returns (codes or None, x or None): codes [B*P][C] as
    segquant_quantize_dualscale (when act_scales is given and want_codes), x
    the bf16 [B][P][C] result if a tensor is passed (or x_out=True to allocate
    one).  workspace: a device tensor, None, or "auto" (from torch's allocator
    when the library asks for one)."""
    import torch
    fn = load_library().segquant_groupnorm_quantize
    bf, f32 = torch.bfloat16, torch.float32
    if z.dim() != 3 or z.dtype is not bf:
        raise ValueError(f"z must be bfloat16 [B][P][C], got {z.dtype} {tuple(z.shape)}")
    shape, dev, at = z.shape, z.device, z.get_device()
    B, P, C = shape
    if x_out is True:
        x_out = torch.empty((B, P, -(-C // 8) * 8), dtype=bf, device=dev)[:, :, :C]
    n, off, wid, *_ = _segments(kseg, C)
    act = q = None
    ld_q = 0
    if act_scales is not None and want_codes:
        act = _want_array(act_scales, "act_scales", f32, (4, n), at)
        out, q, ld_q = _codes_out(out, B * P, C, layout, dev, torch.empty)
    else:
        out = None
    workspace, ws, ws_bytes = _workspace(
        workspace, _groupnorm_bytes, (B, P, C, groups), dev)
    _check(_on(at, fn, z.data_ptr(), B, P, C, _row_ld(z, "z"), groups, eps,
               _want_array(gamma, "gamma", f32, (C,), at),
               _want_array(beta, "beta", f32, (C,), at),
               _want(scale, "scale", bf, (B, C), at), _want(shift, "shift", bf, (B, C), at),
               _mod_ld(B, (scale, shift), "scale and shift"), act_kind, n, off, wid, act, q, ld_q, layout,
               _want(x_out, "x_out", bf, shape, at), _row_ld(x_out, "x_out"), ws, ws_bytes),
           "segquant_groupnorm_quantize")
    return out, x_out


def segquant_adanorm_quantize(h, eps: float = 1e-6, gamma=None, beta=None, scale=None, shift=None,
                              gate=None, branch=None, row_offset=None, n_req: Optional[int] = None,
                              act_scales=None, kseg: Optional[Sequence[int]] = None,
                              layout: int = SEGQ_Q_SIGNED, out=None, x_out=None, h_out=None,
                              want_codes: bool = True):
    """The AdaNorm block before a layer, on bf16 rows h [M][K]: h' = h + gate *
    branch (when branch is given), layer norm of h' with optional fp32 gamma
    and beta [K], then * (1 + scale) + shift with the bf16 parameters [R][K]
    of the row's request.  row_offset (int32 [R + 1] on the device) says which
    rows each request has; without it the R = n_req (default: the rows of
    scale, shift or gate, else 1) requests are equal.  Returns (codes or None,
    x or None, h' or None): codes as segquant_quantize_dualscale (when
    act_scales is given and want_codes), x and h' if a tensor is passed (or
    True to allocate one).  Rows of no request are left as they are, zeros in
    a tensor allocated here."""
    import torch
    fn = load_library().segquant_adanorm_quantize
    bf, f32 = torch.bfloat16, torch.float32
    if h.dim() != 2 or h.dtype is not bf:
        raise ValueError(f"h must be bfloat16 [M][K], got {h.dtype} {tuple(h.shape)}")
    shape, dev, at = h.shape, h.device, h.get_device()
    M, K = shape
    mod = scale if scale is not None else shift if shift is not None else gate
    if row_offset is not None:
        if n_req is not None and n_req != row_offset.numel() - 1:
            raise ValueError(f"n_req {n_req} with row_offset of {row_offset.numel()} offsets")
        n_req = row_offset.numel() - 1
    elif n_req is None:
        n_req = mod.shape[0] if mod is not None else 1
    new = torch.empty if row_offset is None else torch.zeros
    if x_out is True:
        x_out = new((M, -(-K // 8) * 8), dtype=bf, device=dev)[:, :K]
    if h_out is True:
        h_out = new((M, -(-K // 8) * 8), dtype=bf, device=dev)[:, :K]
    n, off, wid, *_ = _segments(kseg, K)
    act = q = None
    ld_q = 0
    if act_scales is not None and want_codes:
        act = _want_array(act_scales, "act_scales", f32, (4, n), at)
        out, q, ld_q = _codes_out(out, M, K, layout, dev, new)
    else:
        out = None
    params = (n_req, K)
    _check(_on(at, fn, h.data_ptr(), M, K, _row_ld(h, "h"), _want(branch, "branch", bf, shape, at),
               _row_ld(branch, "branch"), _want(gate, "gate", bf, params, at),
               _want(h_out, "h_out", bf, shape, at), _row_ld(h_out, "h_out"), eps,
               _want_array(gamma, "gamma", f32, (K,), at),
               _want_array(beta, "beta", f32, (K,), at),
               _want(scale, "scale", bf, params, at), _want(shift, "shift", bf, params, at),
               _mod_ld(n_req, (scale, shift, gate), "scale, shift and gate"), n_req,
               _want_array(row_offset, "row_offset", torch.int32, (n_req + 1,), at), n, off, wid,
               act, q, ld_q, layout, _want(x_out, "x_out", bf, shape, at),
               _row_ld(x_out, "x_out")), "segquant_adanorm_quantize")
    return out, x_out, h_out


def segquant_adapter_workspace_bytes(M: int, N: int, K: int, n_req: int, rank: int,
                                     nseg: Optional[Sequence[int]] = None) -> int:
    n, off, wid, *_ = _segments(nseg, N)
    return int(load_library().segquant_adapter_workspace_bytes(M, N, K, n_req, rank, n, off, wid))


_adapter_bytes = functools.lru_cache(maxsize=256)(segquant_adapter_workspace_bytes)


def segquant_adapter_add(x, a, b, adapter, row_offset, base=None, alpha=None, rank=None,
                         nseg: Optional[Sequence[int]] = None, out=None, workspace="auto"):
    """Low-rank adapters of many requests beside a shared layer: y = base +
    alpha (x a^T) b^T with the adapter of each row's request.

    x: bf16 [M][K], the layer's input; a: bf16 [n_adapters][n_nseg * r][K]
    and b: bf16 [n_adapters][N][r], r the stored rank (a multiple of 16);
    adapter: int32 [R], each request's adapter (-1: none); row_offset: int32
    [R + 1]; base: bf16 [M][N], the layer's output (None: 0); alpha: fp32
    [n_adapters]; rank: int32 [n_adapters], the true ranks; nseg: the layer's
    N-segments.  Everything but nseg is on the device.  Returns bf16 y [M][N];
    out may be base.  Rows of no request are left as they are, zeros in a
    tensor allocated here.  workspace: a device tensor, None, or "auto" (from
    torch's allocator when the library asks for one)."""
    import torch
    fn = load_library().segquant_adapter_add
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, x.device
    if x.dim() != 2 or x.dtype is not bf or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be bfloat16 [M][K], a and b 3-D")
    at = x.get_device()
    M, K = x.shape
    n_adapters, N, r = b.shape
    n_req = adapter.numel()
    n, off, wid, widths, _ = _segments(nseg, N)
    y_shape = (M, N)
    if out is None:
        out = torch.zeros(y_shape, dtype=bf, device=dev)
    workspace, ws, ws_bytes = _workspace(
        workspace, _adapter_bytes, (M, N, K, n_req, r, widths), dev)
    _check(_on(at, fn, M, N, K, x.data_ptr(), _row_ld(x, "x"), n_req,
               _want_array(row_offset, "row_offset", i32, (n_req + 1,), at),
               _want_array(adapter, "adapter", i32, (n_req,), at), n_adapters, r,
               _want_array(rank, "rank", i32, (n_adapters,), at),
               _want_array(a, "a", bf, (n_adapters, n * r, K), at),
               _want_array(b, "b", bf, (n_adapters, N, r), at),
               _want_array(alpha, "alpha", f32, (n_adapters,), at), n, off, wid,
               _want(base, "base", bf, y_shape, at), _row_ld(base, "base"),
               _want(out, "out", bf, y_shape, at), _row_ld(out, "out"), ws, ws_bytes),
           "segquant_adapter_add")
    return out


# ------------------------- the 4-bit layer, the norm before it, q and k behind --
@functools.lru_cache(maxsize=256)
def segquant_mxfp4_bytes(R: int, K: int) -> Tuple[int, int]:
    """Bytes of the codes and of the scales of an MXFP4 matrix of R rows."""
    lib = load_library()
    codes = int(lib.segquant_mxfp4_code_bytes(R, K))
    if R and not codes:
        raise ValueError(segquant_last_error())
    return codes, int(lib.segquant_mxfp4_scale_bytes(R, K))


def _mx_new(R: int, K: int, device):
    import torch
    codes, scales = segquant_mxfp4_bytes(R, K)
    return (torch.empty(codes, dtype=torch.uint8, device=device),
            torch.empty(scales, dtype=torch.uint8, device=device))


def _mx_ptrs(mx, name: str, R: int, K: int, at: int):
    """The two arrays of an MXFP4 matrix (None: not given) -> their addresses."""
    import torch
    if mx is None:
        return None, None
    codes, scales = mx
    n, m = segquant_mxfp4_bytes(R, K)
    u8 = torch.uint8
    if (codes.dtype is u8 and scales.dtype is u8 and codes.get_device() == at and
            scales.get_device() == at and codes.dim() == 1 and scales.dim() == 1 and
            codes.numel() == n and scales.numel() == m and codes.is_contiguous() and
            scales.is_contiguous()):
        return codes.data_ptr(), scales.data_ptr()
    return (_want_array(codes, name + " codes", torch.uint8, (n,), at),
            _want_array(scales, name + " scales", torch.uint8, (m,), at))


def segquant_quantize_mxfp4(z, act_kind: int = SEGQ_ACT_NONE, out=None):
    """bf16 z [M][K] -> the MXFP4 matrix (codes, scales) of its activation: two
    uint8 arrays of segquant_mxfp4_bytes(M, K)."""
    import torch
    fn = load_library().segquant_quantize_mxfp4
    if z.dim() != 2 or z.dtype is not torch.bfloat16:
        raise ValueError(f"z must be bfloat16 [M][K], got {z.dtype} {tuple(z.shape)}")
    M, K = z.shape
    at = z.get_device()
    if out is None:
        out = _mx_new(M, K, z.device)
    _check(_on(at, fn, z.data_ptr(), M, K, _row_ld(z, "z"), act_kind,
               *_mx_ptrs(out, "out", M, K, at)), "segquant_quantize_mxfp4")
    return out


def segquant_quantize_weight_mxfp4(w, out=None):
    """fp32 W [K][N] (Y = X W) -> the MXFP4 matrix (codes, scales) of N rows and
    K columns.  Offline."""
    import torch
    fn = load_library().segquant_quantize_weight_mxfp4
    if w.dim() != 2 or w.dtype is not torch.float32:
        raise ValueError(f"w must be float32 [K][N], got {w.dtype} {tuple(w.shape)}")
    K, N = w.shape
    at = w.get_device()
    if out is None:
        out = _mx_new(N, K, w.device)
    _check(_on(at, fn, w.data_ptr(), K, N, _ld(w, "w"), *_mx_ptrs(out, "out", N, K, at)),
           "segquant_quantize_weight_mxfp4")
    return out


def segquant_unpack_mxfp4(mx, R: int, K: int, out=None):
    """An MXFP4 matrix (codes, scales) -> its values, fp32 [R][K]."""
    import torch
    fn = load_library().segquant_unpack_mxfp4
    at = mx[0].get_device()
    if out is None:
        out = torch.empty((R, K), dtype=torch.float32, device=mx[0].device)
    _check(_on(at, fn, *_mx_ptrs(mx, "mx", R, K, at), R, K,
               _want(out, "out", torch.float32, (R, K), at), _ld(out, "out")),
           "segquant_unpack_mxfp4")
    return out


def segquant_gemm_mxfp4_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load_library().segquant_gemm_mxfp4_workspace_bytes(M, N, K))


_gemm_mx_bytes = functools.lru_cache(maxsize=256)(segquant_gemm_mxfp4_workspace_bytes)


def segquant_gemm_mxfp4(z, w, N: int, K: Optional[int] = None, xq=None, M: Optional[int] = None,
                        act_kind: int = SEGQ_ACT_NONE, out=None, workspace="auto"):
    """The linear layer on MXFP4 weights and activations: bf16 y [M][N].

    z: bf16 [M][K], quantised by the call behind its activation; or None with
    xq = an MXFP4 matrix (codes, scales) of M rows and K columns (M may be left
    to out).  w: the (codes, scales) of segquant_quantize_weight_mxfp4, N its
    columns.  workspace: a device tensor, None, or "auto" (from torch's
    allocator when the library asks for one)."""
    import torch
    fn = load_library().segquant_gemm_mxfp4
    bf = torch.bfloat16
    ld_z = ws_bytes = 0
    ptr = ws = None
    if (z is None) == (xq is None):
        raise ValueError("exactly one of z and xq must be given")
    if z is not None:
        if z.dim() != 2 or z.dtype is not bf:
            raise ValueError(f"z must be bfloat16 [M][K], got {z.dtype} {tuple(z.shape)}")
        if M not in (None, z.shape[0]) or K not in (None, z.shape[1]):
            raise ValueError(f"z of shape {tuple(z.shape)} with M {M} and K {K}")
        M, K = z.shape
        dev, at, ptr, ld_z = z.device, z.get_device(), z.data_ptr(), _row_ld(z, "z")
        workspace, ws, ws_bytes = _workspace(workspace, _gemm_mx_bytes, (M, N, K), dev)
    else:
        if M is None and out is not None:
            M = out.shape[0]
        if M is None or K is None:
            raise ValueError("M (or out) and K are required with a pre-quantised input")
        dev, at = xq[0].device, xq[0].get_device()
    if out is None:
        out = torch.empty((M, N), dtype=bf, device=dev)
    _check(_on(at, fn, M, N, K, ptr, ld_z, act_kind, *_mx_ptrs(xq, "xq", M, K, at),
               *_mx_ptrs(w, "w", N, K, at), _want(out, "out", bf, (M, N), at),
               _row_ld(out, "out"), ws, ws_bytes), "segquant_gemm_mxfp4")
    return out


def segquant_rmsnorm_quantize(h, eps: float = 1e-6, gamma=None, branch=None, act_scales=None,
                              kseg: Optional[Sequence[int]] = None, layout: int = SEGQ_Q_SIGNED,
                              out=None, x_out=None, h_out=None, mx_out=None,
                              want_codes: bool = True):
    """The residual update and root-mean-square norm before a layer, on bf16
    rows h [M][K]: h' = h + branch (when branch is given), x = h' / rms(h') with
    optional fp32 gamma [K].  Returns (codes or None, x or None, h' or None,
    (MXFP4 codes, scales) or None): codes as segquant_quantize_dualscale (when
    act_scales is given and want_codes), the others if tensors are passed (or
    True to allocate them)."""
    import torch
    fn = load_library().segquant_rmsnorm_quantize
    bf, f32 = torch.bfloat16, torch.float32
    if h.dim() != 2 or h.dtype is not bf:
        raise ValueError(f"h must be bfloat16 [M][K], got {h.dtype} {tuple(h.shape)}")
    shape, dev, at = h.shape, h.device, h.get_device()
    M, K = shape
    if x_out is True:
        x_out = torch.empty((M, -(-K // 8) * 8), dtype=bf, device=dev)[:, :K]
    if h_out is True:
        h_out = torch.empty((M, -(-K // 8) * 8), dtype=bf, device=dev)[:, :K]
    if mx_out is True:
        mx_out = _mx_new(M, K, dev)
    n, off, wid, *_ = _segments(kseg, K)
    act = q = None
    ld_q = 0
    if act_scales is not None and want_codes:
        act = _want_array(act_scales, "act_scales", f32, (4, n), at)
        out, q, ld_q = _codes_out(out, M, K, layout, dev, torch.empty)
    else:
        out = None
    _check(_on(at, fn, h.data_ptr(), M, K, _row_ld(h, "h"), _want(branch, "branch", bf, shape, at),
               _row_ld(branch, "branch"), _want(h_out, "h_out", bf, shape, at),
               _row_ld(h_out, "h_out"), eps, _want_array(gamma, "gamma", f32, (K,), at), n, off,
               wid, act, q, ld_q, layout, _want(x_out, "x_out", bf, shape, at),
               _row_ld(x_out, "x_out"), *_mx_ptrs(mx_out, "mx_out", M, K, at)),
           "segquant_rmsnorm_quantize")
    return out, x_out, h_out, mx_out


@functools.lru_cache(maxsize=256)
def _axes(widths: Tuple[int, ...]):
    import numpy as np
    w = np.asarray(widths, dtype=np.int32)
    w.flags.writeable = False
    return len(w), w.ctypes.data, sum(widths), w  # the address belongs to the array


def segquant_rotary_frequencies(widths: Sequence[int], theta: float = 10000.0):
    """theta^(-2j / width) for the pairs of each axis: fp64 [sum(widths) / 2] on
    the CPU."""
    import torch
    n, ptr, R, _ = _axes(tuple(map(int, widths)))
    freq = torch.empty(max(R, 0) // 2, dtype=torch.float64)
    _check(load_library().segquant_rotary_frequencies(n, ptr, theta, freq.data_ptr() or None),
           "segquant_rotary_frequencies")
    return freq


@functools.lru_cache(maxsize=1024)
def _stride_array(stride):
    return (ctypes.c_int64 * 3)(*stride[:3])


def _head_strides(t, name: str, shape, at: int, dtype):
    """A [B][L][heads][D] tensor -> its address and its strides (an array, read
    only: calls share it)."""
    if t.dtype is not dtype or t.get_device() != at or t.shape != shape:
        _want(t, name, dtype, shape, at)
    stride = t.stride()
    if stride[3] != 1 and shape[3] > 1 and t.numel():
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return t.data_ptr(), _stride_array(stride)


def segquant_qk_rotary(q, k, positions, freq, widths: Sequence[int],
                       style: int = SEGQ_ROTARY_PAIRS, q_gamma=None, k_gamma=None,
                       eps: float = 1e-6, norm: bool = True, q_out=None, k_out=None):
    """Root-mean-square norm of each head (when norm), then rotary positions of
    the axes whose widths are given, on bf16 q [B][L][Hq][D] and k
    [B][L][Hk][D] (or None) of any strides with unit stride in D: views of a
    packed QKV matrix, heads before tokens.  positions: int32 [L][axes] or
    [B][L][axes]; freq: fp64 [sum(widths) / 2], radians per position
    (segquant_rotary_frequencies, moved to the GPU); q_gamma, k_gamma: fp32 [D].
    Returns (q', k'): q_out and k_out, which may be q and k, or contiguous
    tensors allocated here."""
    import torch
    fn = load_library().segquant_qk_rotary
    bf, f32 = torch.bfloat16, torch.float32
    if q.dim() != 4 or q.dtype is not bf:
        raise ValueError(f"q must be bfloat16 [B][L][heads][D], got {q.dtype} {tuple(q.shape)}")
    q_shape = q.shape
    B, L, Hq, D = q_shape
    at = q.get_device()
    n, axes, R, _ = _axes(tuple(map(int, widths)))
    if q_out is None:
        q_out = torch.empty(q_shape, dtype=bf, device=q.device)
    q_args = _head_strides(q, "q", q_shape, at, bf)
    q_out_args = _head_strides(q_out, "q_out", q_shape, at, bf)
    if k is not None:
        if k.dim() != 4:
            raise ValueError(f"k must be bfloat16 [B][L][heads][D], got {tuple(k.shape)}")
        Hk = k.shape[2]
        k_shape = (B, L, Hk, D)
        if k_out is None:
            k_out = torch.empty(k_shape, dtype=bf, device=q.device)
        k_args = _head_strides(k, "k", k_shape, at, bf)
        k_out_args = _head_strides(k_out, "k_out", k_shape, at, bf)
    elif k_out is not None or k_gamma is not None:
        raise ValueError("k_out or k_gamma without k")
    else:
        Hk, k_args, k_out_args = 0, (None, None), (None, None)
    if positions.dim() == 3:
        pos, per = _want_array(positions, "positions", torch.int32, (B, L, n), at), L * n
    else:
        pos, per = _want_array(positions, "positions", torch.int32, (L, n), at), 0
    _check(_on(at, fn, B, L, D, q_args[0], Hq, q_args[1], *q_out_args, k_args[0], Hk, k_args[1],
               *k_out_args, 1 if norm else 0, eps, _want_array(q_gamma, "q_gamma", f32, (D,), at),
               _want_array(k_gamma, "k_gamma", f32, (D,), at), pos, per, n, axes,
               _want_array(freq, "freq", torch.float64, (R // 2,), at), style),
           "segquant_qk_rotary")
    return q_out, k_out
