"""Fused gate-up SwiGLU for AMD MI355X: Python binding of libswiglu_gateup.so.

The binding only marshals arguments: it flattens leading dimensions into rows,
reads row strides, allocates outputs with torch, and passes device pointers
and torch's current HIP stream to the C ABI (include/swiglu_gateup.h). Every
step of the computation runs in the HIP kernels. There is no fallback: if the
library is missing or cannot be loaded, every call raises.

Layout (Liger-Kernel Megatron SwiGLU page, §Background): x is the packed fc1
output [..., 2n] with the gate in [..., :n] and up in [..., n:]; 2D and 3D
inputs are accepted (§Megatron feature compatibility).
"""

from __future__ import annotations

import ctypes
import functools
import os

__all__ = ["swiglu_gateup_fwd", "swiglu_gateup_bwd", "swiglu_silu_mul_fwd", "swiglu_silu_mul_bwd",
           "swiglu_gateup_bias_scale_fwd", "swiglu_gateup_bias_scale_bwd",
           "swiglu_gateup_bias_scale_workspace_size", "swiglu_gateup_bias_scale_bwd_noalloc",
           "swiglu_fc1_fwd", "swiglu_fc1_workspace_size", "swiglu_grouped_mm", "swiglu_grouped_fc1",
           "swiglu_grouped_mm_dgrad", "swiglu_grouped_mm_wgrad", "swiglu_grouped_workspace_size",
           "swiglu_ckpt8_fwd", "swiglu_ckpt8_bwd", "swiglu_ckpt8_workspace_size",
           "swiglu_status_string", "SwiGLUError",
           "library_path",
           "load_library", "EXPORTS", "NOALLOC_SCRATCH_BYTES"]

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG_DIR, "libswiglu_gateup.so")

# Status codes and dtype codes of include/swiglu_gateup.h.
SWIGLU_OK = 0
SWIGLU_ERR_NULL_POINTER = 1
SWIGLU_ERR_BAD_SHAPE = 2
SWIGLU_ERR_BAD_STRIDE = 3
SWIGLU_ERR_BAD_DTYPE = 4
SWIGLU_ERR_ALIASING = 5
SWIGLU_ERR_HIP = 6
SWIGLU_ERR_WORKSPACE = 7
SWIGLU_ERR_SCRATCH_LIMIT = 8
NOALLOC_SCRATCH_BYTES = 64 << 20     # SWIGLU_NOALLOC_SCRATCH_BYTES of the header
SWIGLU_DTYPE_F32 = 0
SWIGLU_DTYPE_BF16 = 1
_BAD_DTYPE_CODE = -1    # passed for any other torch dtype; the library rejects it

EXPORTS = ("swiglu_gateup_fwd", "swiglu_gateup_bwd", "swiglu_silu_mul_fwd", "swiglu_silu_mul_bwd",
           "swiglu_gateup_bias_scale_fwd", "swiglu_gateup_bias_scale_bwd",
           "swiglu_gateup_bias_scale_workspace_size", "swiglu_gateup_bias_scale_bwd_noalloc",
           "swiglu_fc1_fwd", "swiglu_fc1_workspace_size", "swiglu_grouped_mm", "swiglu_grouped_fc1",
           "swiglu_grouped_mm_dgrad", "swiglu_grouped_mm_wgrad", "swiglu_grouped_workspace_size",
           "swiglu_ckpt8_fwd", "swiglu_ckpt8_bwd", "swiglu_ckpt8_workspace_size",
           "swiglu_status_string")

_lib = None


class SwiGLUError(RuntimeError):
    """A nonzero swiglu_status from the library."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {swiglu_status_string(status)}")


class SwiGLUArgumentError(SwiGLUError, ValueError):
    """The library rejected the arguments (nothing was launched)."""


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libswiglu_gateup.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is not built; run `python -m swiglu_activation_amd.build` "
            "(or __graft_entry__.build()) first. There is no non-HIP fallback.")
    lib = ctypes.CDLL(_LIB_PATH)
    i64, vp, cint = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.swiglu_gateup_fwd.argtypes = [vp, i64, vp, i64, i64, i64, cint, vp]
    lib.swiglu_gateup_fwd.restype = cint
    lib.swiglu_gateup_bwd.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, cint, cint, vp]
    lib.swiglu_gateup_bwd.restype = cint
    lib.swiglu_silu_mul_fwd.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, cint, vp]
    lib.swiglu_silu_mul_fwd.restype = cint
    lib.swiglu_silu_mul_bwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64,
                                        cint, cint, vp]
    lib.swiglu_silu_mul_bwd.restype = cint
    lib.swiglu_gateup_bias_scale_fwd.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, i64, cint, vp]
    lib.swiglu_gateup_bias_scale_fwd.restype = cint
    lib.swiglu_gateup_bias_scale_workspace_size.argtypes = [i64, i64, cint, cint]
    lib.swiglu_gateup_bias_scale_workspace_size.restype = ctypes.c_size_t
    lib.swiglu_gateup_bias_scale_bwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp,
                                                 i64, vp, ctypes.c_size_t, i64, i64, cint, cint, vp]
    lib.swiglu_gateup_bias_scale_bwd.restype = cint
    lib.swiglu_gateup_bias_scale_bwd_noalloc.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64,
                                                         vp, vp, i64, i64, i64, cint, cint, vp]
    lib.swiglu_gateup_bias_scale_bwd_noalloc.restype = cint
    lib.swiglu_fc1_fwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, cint, vp, vp]
    lib.swiglu_fc1_fwd.restype = cint
    lib.swiglu_fc1_workspace_size.argtypes = []
    lib.swiglu_fc1_workspace_size.restype = ctypes.c_size_t
    sz = ctypes.c_size_t
    lib.swiglu_grouped_mm.argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, i64, i64, i64, i64, cint, vp,
                                      sz, vp]
    lib.swiglu_grouped_mm.restype = cint
    lib.swiglu_grouped_workspace_size.argtypes = [cint, i64, i64, i64, i64]
    lib.swiglu_grouped_workspace_size.restype = sz
    lib.swiglu_grouped_fc1.argtypes = [vp, i64, vp, i64, i64, vp, vp, i64, vp, i64, i64, i64, i64,
                                       i64, cint, vp, sz, vp]
    lib.swiglu_grouped_fc1.restype = cint
    lib.swiglu_grouped_mm_dgrad.argtypes = lib.swiglu_grouped_mm.argtypes
    lib.swiglu_grouped_mm_dgrad.restype = cint
    lib.swiglu_grouped_mm_wgrad.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, i64, i64,
                                            cint, cint, vp, sz, vp]
    lib.swiglu_grouped_mm_wgrad.restype = cint
    lib.swiglu_ckpt8_fwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, cint, vp]
    lib.swiglu_ckpt8_fwd.restype = cint
    lib.swiglu_ckpt8_bwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                     vp, sz, i64, i64, cint, vp]
    lib.swiglu_ckpt8_workspace_size.argtypes = [i64, i64, cint]
    lib.swiglu_ckpt8_workspace_size.restype = sz
    lib.swiglu_ckpt8_bwd.restype = cint
    lib.swiglu_status_string.argtypes = [cint]
    lib.swiglu_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def swiglu_status_string(status: int) -> str:
    return load_library().swiglu_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status == SWIGLU_OK:
        return
    if status == SWIGLU_ERR_HIP:
        raise SwiGLUError(status, what)
    raise SwiGLUArgumentError(status, what)


# ---------------------------------------------------------------------------
# Tensor marshalling
# ---------------------------------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return SWIGLU_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return SWIGLU_DTYPE_BF16
    return _BAD_DTYPE_CODE


def _rows_and_stride(t, name: str):
    """View t as [rows, width] with unit column stride: (rows, row_stride)."""
    if t.dim() == 2:                # (the common case, without the loops below)
        rows, width = t.shape
        row_stride, unit = t.stride()
        if width > 1 and unit != 1:
            raise ValueError(f"{name} must have unit stride in its last dimension")
        return rows, (row_stride if rows != 1 else width)
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    rows = 1
    for s in t.shape[:-1]:
        rows *= int(s)
    if t.dim() == 1:
        return rows, int(t.shape[-1])
    # leading dims must collapse into one row index with a single stride
    row_stride = None
    expect = None
    for d in range(t.dim() - 2, -1, -1):
        if t.shape[d] == 1:
            continue
        if row_stride is None:
            row_stride = int(t.stride(d))
            expect = row_stride * int(t.shape[d])
        else:
            if int(t.stride(d)) != expect:
                raise ValueError(f"leading dimensions of {name} do not collapse into rows")
            expect = int(t.stride(d)) * int(t.shape[d])
    if row_stride is None:          # a single row
        row_stride = int(t.shape[-1])
    return rows, row_stride


def _require_device(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on a HIP device (device pointers only)")
        d = t.get_device()
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError("all tensors must be on the same device")


def _stream_handle(device, stream):
    import torch
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


class _Stay:
    """In place of a device guard where the device is the current one already."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_STAY = _Stay()


def _on_device(device):
    """Guard that makes `device` current for the call (a launch goes to the
    current device). torch's own guard takes 1.4 us, also where nothing changes."""
    import torch
    return _STAY if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def swiglu_gateup_fwd(x, y=None, *, stream=None):
    """y = silu(x[..., :n]) * x[..., n:] for x of shape [..., 2n] (fp32 or bf16).

    ``y`` (optional) is the [..., n] output; allocated when omitted. The
    kernel is enqueued on ``stream`` (default: torch's current stream)."""
    import torch
    lib = load_library()
    _require_device(x, y)
    if x.dim() < 1 or x.shape[-1] % 2:
        raise ValueError("last dimension of x must be even (2n)")
    n = x.shape[-1] // 2
    if y is None:
        y = torch.empty(tuple(x.shape[:-1]) + (n,), dtype=x.dtype, device=x.device)
    if y.dtype != x.dtype:
        raise ValueError("x and y must have the same dtype")
    rows, xs = _rows_and_stride(x, "x")
    yrows, ys = _rows_and_stride(y, "y")
    if yrows != rows or y.shape[-1] != n:
        raise ValueError(f"y must hold {rows} rows of {n} elements")
    with _on_device(x.device):
        st = lib.swiglu_gateup_fwd(x.data_ptr(), xs, y.data_ptr(), ys, rows, n,
                                   _dtype_code(x), _stream_handle(x.device, stream))
    _check(st, "swiglu_gateup_fwd")
    return y


def swiglu_gateup_bwd(dy, x, dx=None, *, in_place: bool = False, stream=None):
    """Gradient of swiglu_gateup_fwd with respect to x: [dgate | dup], [..., 2n].

    silu is recomputed from the saved input ``x``. Out of place (default) the
    result goes to ``dx`` (allocated when omitted). With ``in_place=True`` it
    overwrites ``x``, which is returned."""
    import torch
    lib = load_library()
    _require_device(dy, x, dx)
    if x.dim() < 1 or x.shape[-1] % 2:
        raise ValueError("last dimension of x must be even (2n)")
    n = x.shape[-1] // 2
    if dy.dtype != x.dtype:
        raise ValueError("dy and x must have the same dtype")
    rows, xs = _rows_and_stride(x, "x")
    dyrows, dys = _rows_and_stride(dy, "dy")
    if dyrows != rows or dy.shape[-1] != n:
        raise ValueError(f"dy must hold {rows} rows of {n} elements")
    if in_place:
        if dx is not None and dx.data_ptr() != x.data_ptr():
            raise ValueError("in_place backward writes into x; pass dx=None or dx=x")
        dx_ptr, dxs = None, 0
        out = x
    else:
        if dx is None:
            dx = torch.empty(tuple(x.shape), dtype=x.dtype, device=x.device)
        if dx.dtype != x.dtype:
            raise ValueError("dx and x must have the same dtype")
        dxrows, dxs = _rows_and_stride(dx, "dx")
        if dxrows != rows or dx.shape[-1] != 2 * n:
            raise ValueError(f"dx must hold {rows} rows of {2 * n} elements")
        dx_ptr = dx.data_ptr()
        out = dx
    with _on_device(x.device):
        st = lib.swiglu_gateup_bwd(dy.data_ptr(), dys, x.data_ptr(), xs, dx_ptr, dxs, rows, n,
                                   _dtype_code(x), 1 if in_place else 0,
                                   _stream_handle(x.device, stream))
    _check(st, "swiglu_gateup_bwd")
    return out


def _same_rows(t, rows, n, name):
    r, s = _rows_and_stride(t, name)
    if r != rows or t.shape[-1] != n:
        raise ValueError(f"{name} must hold {rows} rows of {n} elements")
    return s


def swiglu_silu_mul_fwd(gate, up, y=None, *, stream=None):
    """y = silu(gate) * up for two tensors of the same shape [..., n]."""
    import torch
    lib = load_library()
    _require_device(gate, up, y)
    if gate.shape != up.shape:
        raise ValueError("gate and up must have the same shape")
    if gate.dtype != up.dtype:
        raise ValueError("gate and up must have the same dtype")
    n = gate.shape[-1] if gate.dim() else 1
    rows, gs = _rows_and_stride(gate, "gate")
    us = _same_rows(up, rows, n, "up")
    if y is None:
        y = torch.empty(tuple(gate.shape), dtype=gate.dtype, device=gate.device)
    if y.dtype != gate.dtype:
        raise ValueError("y must have the dtype of gate")
    ys = _same_rows(y, rows, n, "y")
    with _on_device(gate.device):
        st = lib.swiglu_silu_mul_fwd(gate.data_ptr(), gs, up.data_ptr(), us, y.data_ptr(), ys,
                                     rows, n, _dtype_code(gate), _stream_handle(gate.device, stream))
    _check(st, "swiglu_silu_mul_fwd")
    return y


def swiglu_silu_mul_bwd(dy, gate, up, dgate=None, dup=None, *, in_place: bool = False, stream=None):
    """(dgate, dup) for y = silu(gate) * up. With in_place=True they overwrite
    gate and up, which are returned."""
    import torch
    lib = load_library()
    _require_device(dy, gate, up, dgate, dup)
    if gate.shape != up.shape or dy.shape != gate.shape:
        raise ValueError("dy, gate and up must have the same shape")
    if not (dy.dtype == gate.dtype == up.dtype):
        raise ValueError("dy, gate and up must have the same dtype")
    n = gate.shape[-1] if gate.dim() else 1
    rows, gs = _rows_and_stride(gate, "gate")
    us = _same_rows(up, rows, n, "up")
    dys = _same_rows(dy, rows, n, "dy")
    if in_place:
        for t, src, name in ((dgate, gate, "dgate"), (dup, up, "dup")):
            if t is not None and t.data_ptr() != src.data_ptr():
                raise ValueError(f"in_place backward writes into the inputs; pass {name}=None")
        dgate, dup = gate, up
        dg_ptr = du_ptr = None
        dgs = dus = 0
    else:
        if dgate is None:
            dgate = torch.empty(tuple(gate.shape), dtype=gate.dtype, device=gate.device)
        if dup is None:
            dup = torch.empty(tuple(gate.shape), dtype=gate.dtype, device=gate.device)
        if dgate.dtype != gate.dtype or dup.dtype != gate.dtype:
            raise ValueError("dgate and dup must have the dtype of gate")
        dgs = _same_rows(dgate, rows, n, "dgate")
        dus = _same_rows(dup, rows, n, "dup")
        dg_ptr, du_ptr = dgate.data_ptr(), dup.data_ptr()
    with _on_device(gate.device):
        st = lib.swiglu_silu_mul_bwd(dy.data_ptr(), dys, gate.data_ptr(), gs, up.data_ptr(), us,
                                     dg_ptr, dgs, du_ptr, dus, rows, n, _dtype_code(gate),
                                     1 if in_place else 0, _stream_handle(gate.device, stream))
    _check(st, "swiglu_silu_mul_bwd")
    return dgate, dup


# ---------------------------------------------------------------------------
# Bias and per-token scale variants
# ---------------------------------------------------------------------------

def _bias_arg(bias, x, n):
    if bias is None:
        return None
    _require_device(bias, x)
    if bias.dim() != 1 or bias.shape[0] != 2 * n or (n and bias.stride(0) != 1):
        raise ValueError(f"bias must be a contiguous [{2 * n}] tensor")
    if bias.dtype != x.dtype:
        raise ValueError("bias must have the dtype of x")
    return bias.data_ptr()


def _per_row_arg(t, x, rows, name):
    """A per-row fp32 tensor shaped like x's leading dims, optionally with a
    trailing 1: (pointer, stride)."""
    import torch
    if t is None:
        return None, 1
    _require_device(t, x)
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    lead = tuple(x.shape[:-1])
    if tuple(t.shape) == lead:
        t2 = t.unsqueeze(-1)
    elif tuple(t.shape) == lead + (1,):
        t2 = t
    else:
        raise ValueError(f"{name} must have shape {lead} or {lead + (1,)}")
    r, s_ = _rows_and_stride(t2, name)
    assert r == rows
    if rows > 1 and s_ < 1:         # a stride of 1 would read past the one value it has
        raise ValueError(f"{name} must not be an expanded view")
    return t.data_ptr(), max(1, s_)


def swiglu_gateup_bias_scale_workspace_size(rows: int, n: int, want_dbias: bool,
                                            want_dscale: bool) -> int:
    return int(load_library().swiglu_gateup_bias_scale_workspace_size(
        int(rows), int(n), int(bool(want_dbias)), int(bool(want_dscale))))


def swiglu_gateup_bias_scale_fwd(x, bias=None, scale=None, y=None, *, stream=None):
    """y = scale * silu(z[..., :n]) * z[..., n:] with z = x + bias.

    bias: [2n] of x's dtype or None; scale: float32 per row (shape
    x.shape[:-1], optionally with a trailing 1) or None."""
    import torch
    lib = load_library()
    _require_device(x, y)
    if x.dim() < 1 or x.shape[-1] % 2:
        raise ValueError("last dimension of x must be even (2n)")
    n = x.shape[-1] // 2
    rows, xs = _rows_and_stride(x, "x")
    bp = _bias_arg(bias, x, n)
    sp, ss = _per_row_arg(scale, x, rows, "scale")
    if y is None:
        y = torch.empty(tuple(x.shape[:-1]) + (n,), dtype=x.dtype, device=x.device)
    if y.dtype != x.dtype:
        raise ValueError("x and y must have the same dtype")
    ys = _same_rows(y, rows, n, "y")
    with _on_device(x.device):
        st = lib.swiglu_gateup_bias_scale_fwd(x.data_ptr(), xs, bp, sp, ss, y.data_ptr(), ys, rows,
                                              n, _dtype_code(x), _stream_handle(x.device, stream))
    _check(st, "swiglu_gateup_bias_scale_fwd")
    return y


def swiglu_gateup_bias_scale_bwd(dy, x, bias=None, scale=None, dx=None, *, want_dbias=None,
                                 want_dscale=None, in_place: bool = False, workspace=None,
                                 stream=None):
    """Backward of swiglu_gateup_bias_scale_fwd: returns (dx, dbias, dscale).

    dbias ([2n] float32) is computed when want_dbias (default: bias given),
    dscale (float32, shaped like scale) when want_dscale (default: scale
    given). workspace: a device tensor of at least
    swiglu_gateup_bias_scale_workspace_size(...) bytes, allocated if None."""
    import torch
    lib = load_library()
    _require_device(dy, x, dx)
    if x.dim() < 1 or x.shape[-1] % 2:
        raise ValueError("last dimension of x must be even (2n)")
    n = x.shape[-1] // 2
    if dy.dtype != x.dtype:
        raise ValueError("dy and x must have the same dtype")
    rows, xs = _rows_and_stride(x, "x")
    dys = _same_rows(dy, rows, n, "dy")
    bp = _bias_arg(bias, x, n)
    sp, ss = _per_row_arg(scale, x, rows, "scale")
    want_dbias = bias is not None if want_dbias is None else bool(want_dbias)
    want_dscale = scale is not None if want_dscale is None else bool(want_dscale)
    dbias = torch.empty(2 * n, dtype=torch.float32, device=x.device) if want_dbias else None
    dscale = (torch.empty(tuple(scale.shape), dtype=torch.float32, device=x.device)
              if want_dscale and scale is not None else None)
    if want_dscale and scale is None:
        dscale = torch.empty(tuple(x.shape[:-1]), dtype=torch.float32, device=x.device)
    dsp, dss = _per_row_arg(dscale, x, rows, "dscale") if dscale is not None else (None, 1)
    if in_place:
        if dx is not None and dx.data_ptr() != x.data_ptr():
            raise ValueError("in_place backward writes into x; pass dx=None or dx=x")
        dx_ptr, dxs, out = None, 0, x
    else:
        if dx is None:
            dx = torch.empty(tuple(x.shape), dtype=x.dtype, device=x.device)
        if dx.dtype != x.dtype:
            raise ValueError("dx and x must have the same dtype")
        dxs = _same_rows(dx, rows, 2 * n, "dx")
        dx_ptr, out = dx.data_ptr(), dx
    need = swiglu_gateup_bias_scale_workspace_size(rows, n, want_dbias, want_dscale)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if workspace is not None:
        _require_device(workspace, x)
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        wp, wb = None, 0
    with _on_device(x.device):
        st = lib.swiglu_gateup_bias_scale_bwd(
            dy.data_ptr(), dys, x.data_ptr(), xs, bp, sp, ss, dx_ptr, dxs,
            dbias.data_ptr() if dbias is not None else None, dsp, dss, wp, wb, rows, n,
            _dtype_code(x), 1 if in_place else 0, _stream_handle(x.device, stream))
    _check(st, "swiglu_gateup_bias_scale_bwd")
    return out, dbias, dscale


def swiglu_gateup_bias_scale_bwd_noalloc(dy, x, dx=None, dbias=None, dscale=None, *, bias=None,
                                         scale=None, in_place: bool = False, stream=None):
    """swiglu_gateup_bias_scale_bwd without any allocation: the caller passes
    every output (dx, unless in_place; dbias [2n] float32 to get dbias;
    dscale float32 shaped like scale to get dscale) and the partial sums go to
    the library's static per-GPU scratch. Calls that may overlap in time on
    one GPU race on that scratch. Problems needing more than
    NOALLOC_SCRATCH_BYTES of partials raise (SWIGLU_ERR_SCRATCH_LIMIT).
    Returns (dx or x, dbias, dscale)."""
    lib = load_library()
    _require_device(dy, x, dx, dbias, dscale)
    if x.dim() < 1 or x.shape[-1] % 2:
        raise ValueError("last dimension of x must be even (2n)")
    n = x.shape[-1] // 2
    if dy.dtype != x.dtype:
        raise ValueError("dy and x must have the same dtype")
    rows, xs = _rows_and_stride(x, "x")
    dys = _same_rows(dy, rows, n, "dy")
    bp = _bias_arg(bias, x, n)
    sp, ss = _per_row_arg(scale, x, rows, "scale")
    if dbias is not None:
        import torch
        if dbias.dtype != torch.float32 or dbias.dim() != 1 or dbias.shape[0] != 2 * n or \
                (n and dbias.stride(0) != 1):
            raise ValueError(f"dbias must be a contiguous float32 [{2 * n}] tensor")
    dsp, dss = _per_row_arg(dscale, x, rows, "dscale") if dscale is not None else (None, 1)
    if in_place:
        if dx is not None and dx.data_ptr() != x.data_ptr():
            raise ValueError("in_place backward writes into x; pass dx=None or dx=x")
        dx_ptr, dxs, out = None, 0, x
    else:
        if dx is None:
            raise ValueError("the allocation-free backward needs dx (or in_place=True)")
        if dx.dtype != x.dtype:
            raise ValueError("dx and x must have the same dtype")
        dxs = _same_rows(dx, rows, 2 * n, "dx")
        dx_ptr, out = dx.data_ptr(), dx
    import torch
    with _on_device(x.device):
        st = lib.swiglu_gateup_bias_scale_bwd_noalloc(
            dy.data_ptr(), dys, x.data_ptr(), xs, bp, sp, ss, dx_ptr, dxs,
            dbias.data_ptr() if dbias is not None else None, dsp, dss, rows, n,
            _dtype_code(x), 1 if in_place else 0, _stream_handle(x.device, stream))
    _check(st, "swiglu_gateup_bias_scale_bwd_noalloc")
    return out, dbias, dscale


# ---------------------------------------------------------------------------
# fc1 projection with the SwiGLU epilogue
# ---------------------------------------------------------------------------

def swiglu_fc1_workspace_size() -> int:
    return int(load_library().swiglu_fc1_workspace_size())


# One zeroed fc1 workspace per (device, stream): the kernel leaves it zeroed,
# and launches on one stream never overlap.
_fc1_workspaces: dict = {}


def _fc1_workspace(device, stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(device)
    if torch.cuda.is_current_stream_capturing():
        # memory allocated under capture belongs to the graph's pool: the
        # captured launch uses one workgroup per tile instead
        return None
    key = (torch.device(device).index, s.cuda_stream)
    ws = _fc1_workspaces.get(key)
    if ws is None:
        with torch.cuda.stream(s):
            ws = torch.zeros(swiglu_fc1_workspace_size(), dtype=torch.uint8, device=device)
        _fc1_workspaces[key] = ws
    return ws


def swiglu_fc1_fwd(a, w, y=None, *, x_out=None, stream=None, workspace=None):
    """y = silu(a @ w[:n].T) * (a @ w[n:].T) for bf16 a [..., k] and w [2n, k].

    x_out: None, True (allocate) or a [..., 2n] tensor that receives a @ w.T.
    Returns y, or (y, x_out) when x_out is requested. n and k must be
    multiples of 64, rows 16-byte aligned, and the row strides of a and w at
    most 2^28 elements; anything else raises ValueError (the C entry point's
    status).

    workspace: None (a zeroed buffer kept per device and stream; none while
    the stream is being captured into a graph), False (none: one workgroup
    per tile), or a device tensor of swiglu_fc1_workspace_size() bytes that
    is all zero and not in use by another launch. The outputs are the same
    bits either way."""
    import torch
    lib = load_library()
    _require_device(a, w, y, x_out if isinstance(x_out, torch.Tensor) else None)
    if w.dim() != 2 or w.shape[0] % 2:
        raise ValueError("w must be [2n, k]")
    n, k = w.shape[0] // 2, w.shape[1]
    if a.shape[-1] != k:
        raise ValueError(f"a must have {k} columns")
    if a.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise ValueError("swiglu_fc1_fwd needs bfloat16 a and w")
    m, lda = _rows_and_stride(a, "a")
    _, ldw = _rows_and_stride(w, "w")
    if y is None:
        y = torch.empty(tuple(a.shape[:-1]) + (n,), dtype=a.dtype, device=a.device)
    if y.dtype != torch.bfloat16:
        raise ValueError("y must be bfloat16")
    ldy = _same_rows(y, m, n, "y")
    want_x = x_out is not None and x_out is not False
    if x_out is True:
        x_out = torch.empty(tuple(a.shape[:-1]) + (2 * n,), dtype=a.dtype, device=a.device)
    xp, ldx = None, 0
    if want_x:
        if x_out.dtype != torch.bfloat16:
            raise ValueError("x_out must be bfloat16")
        ldx = _same_rows(x_out, m, 2 * n, "x_out")
        xp = x_out.data_ptr()
    if workspace is None:
        workspace = _fc1_workspace(a.device, stream)
    elif workspace is False:
        workspace = None
    wsp = None
    if workspace is not None:
        _require_device(workspace, a)
        if workspace.numel() * workspace.element_size() < swiglu_fc1_workspace_size():
            raise ValueError("fc1 workspace smaller than swiglu_fc1_workspace_size()")
        wsp = workspace.data_ptr()
    with _on_device(a.device):
        st = lib.swiglu_fc1_fwd(a.data_ptr(), lda, w.data_ptr(), ldw, y.data_ptr(), ldy, xp, ldx,
                                m, n, k, _dtype_code(a), wsp, _stream_handle(a.device, stream))
    _check(st, "swiglu_fc1_fwd")
    return (y, x_out) if want_x else y


# ---------------------------------------------------------------------------
# Products grouped by expert
# ---------------------------------------------------------------------------

_calls = None           # _torch_calls (csrc/torch_calls.cpp): ordinary calls without ctypes


class _ThroughCtypes:
    """In place of that module where it is not built or does not load: leaves every
    call to the code here."""

    def _leave(*args):
        return None

    mm = fc1 = mm_dgrad = mm_wgrad = ckpt8_fwd = ckpt8_bwd = staticmethod(_leave)


def _native():
    """The module for the ordinary call of the operators below: tensors on the
    current device, outputs and workspace allocated by the call, torch's current
    stream. Its functions return None for any other call, which the code here then takes.
    Without the module that code takes them all (the same kernels, 5 to 14 us more
    on the host), after one warning."""
    global _calls
    if _calls is None:
        import torch  # noqa: F401  (the module needs torch's libraries loaded)
        load_library()
        try:
            from . import _torch_calls as calls
        except ImportError as e:
            import warnings
            warnings.warn(f"_torch_calls.so is missing or does not load ({e}); calls go through ctypes. "
                          "Build it with `python -m swiglu_activation_amd.build`.", RuntimeWarning,
                          stacklevel=3)
            calls = _ThroughCtypes()
        _calls = calls
    return _calls


def _done(r, what):
    """r, unless it is a status: that raises."""
    if r.__class__ is int:
        _check(r, what)
    return r


def _grouped_tokens(t, name, width=None):
    """(rows, width, row stride) of a token matrix [..., width] in bf16."""
    import torch
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    rows, stride = _rows_and_stride(t, name)
    if width is not None and t.shape[-1] != width:
        raise ValueError(f"{name} must have {width} columns")
    return rows, int(t.shape[-1]), stride


def _grouped_weights(w, name, dtypes):
    """(experts, height, width, row stride, expert stride) of a [E, n, k] tensor."""
    if w.dim() != 3:
        raise ValueError(f"{name} must be [experts, n, k]")
    if w.dtype not in dtypes:
        raise ValueError(f"{name} must be " + " or ".join(str(d)[6:] for d in dtypes))
    e, h, c = w.shape
    es, ld, unit = w.stride()
    if c > 1 and unit != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    # the stride of a dimension of size one (or of an empty tensor) is not used
    if h <= 1 or c == 0:
        ld = c
    if e <= 1 or h * c == 0:
        es = max(h * ld, 1)
    return e, h, c, ld, es


def _grouped_ends(ends, experts):
    import torch
    if ends.dtype != torch.int32 or ends.dim() != 1 or ends.shape[0] != experts or \
            (experts > 1 and ends.stride(0) != 1):
        raise ValueError(f"ends must be a contiguous int32 [{experts}] tensor")
    return ends.data_ptr()


def _grouped_out(out, like, width, name):
    import torch
    if out is None:
        return like.new_empty(like.shape[:-1] + (width,))
    if out.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    return out


# Codes of swiglu_grouped_op in include/swiglu_gateup.h.
GROUPED_OPS = {"mm": 0, "fc1": 1, "mm_dgrad": 2, "mm_wgrad": 3}


def swiglu_grouped_workspace_size(op: str, rows: int, experts: int, n: int, k: int) -> int:
    """Bytes of workspace that swiglu_grouped_<op> uses for these sizes (0: none)."""
    return _workspace_size(op, int(rows), int(experts), int(n), int(k))


@functools.lru_cache(maxsize=4096)          # of the sizes alone
def _workspace_size(op, rows, experts, n, k):
    return int(load_library().swiglu_grouped_workspace_size(GROUPED_OPS[op], rows, experts, n, k))


def _scratch(need, like, stream):
    """need bytes on like's device, taken on the stream that uses them: freed, they
    go to later work of that stream only."""
    import torch
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def _span_of_workspace(workspace, like):
    """(pointer, bytes) of a caller's workspace: its elements have to be its memory (an
    expanded view has more of them than bytes behind its pointer)."""
    _require_device(workspace, like)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _grouped_workspace(op, rows, e, n, k, workspace, like, stream):
    """(tensor kept alive for the call, pointer, bytes). workspace None: taken
    from torch's allocator, on the stream the kernels run on."""
    if workspace is None:
        need = _workspace_size(op, rows, e, n, k)
        if need == 0:
            return None, None, 0
        workspace = _scratch(need, like, stream)
    elif workspace is False:
        return None, None, 0
    return (workspace, *_span_of_workspace(workspace, like))


def swiglu_grouped_mm(a, w, ends, y=None, *, workspace=None, stream=None):
    """y[r] = a[r] @ w[e].T for the rows r in [ends[e-1], ends[e]) of expert e.

    a [..., k] and w [experts, n, k] in bf16; ends [experts] int32 on the
    device, non-decreasing. Rows past ends[-1] are spare: y is zero there.
    Nothing is read back to the host.

    workspace (all four products): None (taken from torch's allocator where
    swiglu_grouped_workspace_size asks for one), False (none: a product of few output
    tiles then runs on few CUs), or a device tensor of at least that size."""
    if y is None and workspace is None and stream is None:
        r = (_calls or _native()).mm(a, w, ends)
        if r is not None:
            return _done(r, "swiglu_grouped_mm")
    import torch
    lib = load_library()
    _require_device(a, w, ends, y)
    e, n, k, ldw, es = _grouped_weights(w, "w", (torch.bfloat16,))
    rows, _, lda = _grouped_tokens(a, "a", k)
    ep = _grouped_ends(ends, e)
    y = _grouped_out(y, a, n, "y")
    ldy = _same_rows(y, rows, n, "y")
    workspace, wp, wb = _grouped_workspace("mm", rows, e, n, k, workspace, a, stream)
    with _on_device(a.device):
        st = lib.swiglu_grouped_mm(a.data_ptr(), lda, w.data_ptr(), ldw, es, ep, y.data_ptr(), ldy,
                                   rows, e, n, k, _dtype_code(a), wp, wb,
                                   _stream_handle(a.device, stream))
    _check(st, "swiglu_grouped_mm")
    return y


def swiglu_grouped_fc1(a, w, ends, scale=None, y=None, *, workspace=None, stream=None):
    """y[r] = scale[r] * silu(a[r] @ w[e, :n].T) * (a[r] @ w[e, n:].T): the
    routed experts' first projection with its activation, the product kept in
    fp32 (for inference: nothing is saved for a backward).

    a [..., k] and w [experts, 2n, k] in bf16; scale float32 per row (shape
    a.shape[:-1], optionally with a trailing 1) or None; ends as in
    swiglu_grouped_mm."""
    if y is None and workspace is None and stream is None:
        r = (_calls or _native()).fc1(a, w, ends, scale)
        if r is not None:
            return _done(r, "swiglu_grouped_fc1")
    import torch
    lib = load_library()
    _require_device(a, w, ends, y)
    e, n2, k, ldw, es = _grouped_weights(w, "w", (torch.bfloat16,))
    if n2 % 2:
        raise ValueError("w must be [experts, 2n, k]")
    n = n2 // 2
    rows, _, lda = _grouped_tokens(a, "a", k)
    ep = _grouped_ends(ends, e)
    sp, ss = _per_row_arg(scale, a, rows, "scale")
    y = _grouped_out(y, a, n, "y")
    ldy = _same_rows(y, rows, n, "y")
    workspace, wp, wb = _grouped_workspace("fc1", rows, e, n, k, workspace, a, stream)
    with _on_device(a.device):
        st = lib.swiglu_grouped_fc1(a.data_ptr(), lda, w.data_ptr(), ldw, es, ep, sp, ss,
                                    y.data_ptr(), ldy, rows, e, n, k, _dtype_code(a), wp, wb,
                                    _stream_handle(a.device, stream))
    _check(st, "swiglu_grouped_fc1")
    return y


def swiglu_grouped_mm_dgrad(dy, w, ends, da=None, *, workspace=None, stream=None):
    """Gradient of swiglu_grouped_mm with respect to a: da[r] = dy[r] @ w[e]
    (zero for spare rows). dy [..., n], w [experts, n, k], da [..., k]."""
    if da is None and workspace is None and stream is None:
        r = (_calls or _native()).mm_dgrad(dy, w, ends)
        if r is not None:
            return _done(r, "swiglu_grouped_mm_dgrad")
    import torch
    lib = load_library()
    _require_device(dy, w, ends, da)
    e, n, k, ldw, es = _grouped_weights(w, "w", (torch.bfloat16,))
    rows, _, lddy = _grouped_tokens(dy, "dy", n)
    ep = _grouped_ends(ends, e)
    da = _grouped_out(da, dy, k, "da")
    ldda = _same_rows(da, rows, k, "da")
    workspace, wp, wb = _grouped_workspace("mm_dgrad", rows, e, n, k, workspace, dy, stream)
    with _on_device(dy.device):
        st = lib.swiglu_grouped_mm_dgrad(dy.data_ptr(), lddy, w.data_ptr(), ldw, es, ep,
                                         da.data_ptr(), ldda, rows, e, n, k, _dtype_code(dy), wp, wb,
                                         _stream_handle(dy.device, stream))
    _check(st, "swiglu_grouped_mm_dgrad")
    return da


def swiglu_grouped_mm_wgrad(dy, a, ends, dw=None, *, dtype=None, workspace=None, stream=None):
    """Gradient of swiglu_grouped_mm with respect to w: dw[e] = sum over
    expert e's rows of dy[r].T a[r], [experts, n, k], zero for an expert
    without rows. dtype (of a new dw): torch.bfloat16 (default) or
    torch.float32, to which the fp32 sums are written unrounded."""
    import torch
    if dw is None and workspace is None and stream is None and \
            (dtype is None or dtype is torch.bfloat16 or dtype is torch.float32):
        r = (_calls or _native()).mm_wgrad(dy, a, ends, dtype is torch.float32)
        if r is not None:
            return _done(r, "swiglu_grouped_mm_wgrad")
    lib = load_library()
    _require_device(dy, a, ends, dw)
    rows, n, lddy = _grouped_tokens(dy, "dy")
    arows, k, lda = _grouped_tokens(a, "a")
    if arows != rows:
        raise ValueError(f"a must hold {rows} rows")
    if dw is None:
        dw = torch.empty(ends.shape[0] if ends.dim() else 0, n, k,
                         dtype=torch.bfloat16 if dtype is None else dtype, device=dy.device)
    elif dtype is not None and dw.dtype != dtype:
        raise ValueError("dw must have the dtype asked for")
    e, h, c, lddw, es = _grouped_weights(dw, "dw", (torch.bfloat16, torch.float32))
    if (h, c) != (n, k):
        raise ValueError(f"dw must be [experts, {n}, {k}]")
    ep = _grouped_ends(ends, e)
    workspace, wp, wb = _grouped_workspace("mm_wgrad", rows, e, n, k, workspace, dy, stream)
    with _on_device(dy.device):
        st = lib.swiglu_grouped_mm_wgrad(dy.data_ptr(), lddy, a.data_ptr(), lda, ep, dw.data_ptr(),
                                         lddw, es, rows, e, n, k, _dtype_code(dy), _dtype_code(dw),
                                         wp, wb, _stream_handle(dy.device, stream))
    _check(st, "swiglu_grouped_mm_wgrad")
    return dw


# ---------------------------------------------------------------------------
# SwiGLU with its input kept in 8 bits
# ---------------------------------------------------------------------------

CKPT8_BLOCK = 32         # columns that share a scale


def swiglu_ckpt8_fwd(x, scale=None, y=None, q=None, qs=None, *, stream=None):
    """y = scale * silu(x[..., :n]) * x[..., n:], and x in 8 bits for the backward.

    Returns (y, q, qs): q [..., 2n] float8_e4m3fn and qs [..., 2 ceil(n/32)]
    uint8, with x ~ q * 2^(qs - 127) in blocks of 32 columns of each half
    (gate scales first, then up). scale: float32 per row (shape
    x.shape[:-1], optionally with a trailing 1) or None."""
    if y is None and q is None and qs is None and stream is None:
        r = (_calls or _native()).ckpt8_fwd(x, scale)
        if r is not None:
            return _done(r, "swiglu_ckpt8_fwd")
    import torch
    lib = load_library()
    _require_device(x, y, q, qs)
    if x.dim() < 1 or x.shape[-1] % 2:
        raise ValueError("last dimension of x must be even (2n)")
    n = x.shape[-1] // 2
    nb = (n + CKPT8_BLOCK - 1) // CKPT8_BLOCK
    lead = tuple(x.shape[:-1])
    rows, xs = _rows_and_stride(x, "x")
    sp, ss = _per_row_arg(scale, x, rows, "scale")
    if y is None:
        y = x.new_empty(lead + (n,))
    if q is None:
        q = x.new_empty(lead + (2 * n,), dtype=torch.float8_e4m3fn)
    if qs is None:
        qs = x.new_empty(lead + (2 * nb,), dtype=torch.uint8)
    if y.dtype != x.dtype:
        raise ValueError("x and y must have the same dtype")
    if q.dtype != torch.float8_e4m3fn or qs.dtype != torch.uint8:
        raise ValueError("q must be float8_e4m3fn and qs uint8")
    ys = _same_rows(y, rows, n, "y")
    qst = _same_rows(q, rows, 2 * n, "q")
    qss = _same_rows(qs, rows, 2 * nb, "qs")
    with _on_device(x.device):
        st = lib.swiglu_ckpt8_fwd(x.data_ptr(), xs, sp, ss, y.data_ptr(), ys, q.data_ptr(), qst,
                                  qs.data_ptr(), qss, rows, n, _dtype_code(x),
                                  _stream_handle(x.device, stream))
    _check(st, "swiglu_ckpt8_fwd")
    return y, q, qs


def swiglu_ckpt8_workspace_size(rows: int, n: int, dtype) -> int:
    """Bytes of workspace that swiglu_ckpt8_bwd takes to give dscale for rows of
    n columns in dtype (torch.float32 or torch.bfloat16)."""
    import torch
    code = {torch.float32: SWIGLU_DTYPE_F32, torch.bfloat16: SWIGLU_DTYPE_BF16}.get(dtype, _BAD_DTYPE_CODE)
    return int(load_library().swiglu_ckpt8_workspace_size(int(rows), int(n), code))


def swiglu_ckpt8_bwd(dy, q, qs, scale=None, dx=None, *, want_y: bool = False, want_dscale=None,
                     y=None, workspace=None, stream=None):
    """Backward of swiglu_ckpt8_fwd at the values kept in (q, qs): returns
    (dx, y, dscale).

    dx [..., 2n] in dy's dtype. y (with want_y, or into a given y) is the
    forward's output again, from the kept values, for a weight gradient that
    needs it. dscale (float32, shaped like scale; default: scale given) is the
    sum over columns of dy * silu(g) * u. workspace: a device tensor of at least
    swiglu_ckpt8_workspace_size(...) bytes, allocated if None."""
    want_dscale = scale is not None if want_dscale is None else bool(want_dscale)
    if dx is None and y is None and workspace is None and stream is None:
        r = (_calls or _native()).ckpt8_bwd(dy, q, qs, scale, bool(want_y), want_dscale)
        if r is not None:
            return _done(r, "swiglu_ckpt8_bwd")
    import torch
    lib = load_library()
    _require_device(dy, q, qs, dx, y, workspace)
    if q.dtype != torch.float8_e4m3fn or qs.dtype != torch.uint8:
        raise ValueError("q must be float8_e4m3fn and qs uint8")
    if dy.dim() < 1:
        raise ValueError("dy must have at least one dimension")
    n = int(dy.shape[-1])
    nb = (n + CKPT8_BLOCK - 1) // CKPT8_BLOCK
    rows, dys = _rows_and_stride(dy, "dy")
    qst = _same_rows(q, rows, 2 * n, "q")
    qss = _same_rows(qs, rows, 2 * nb, "qs")
    sp, ss = _per_row_arg(scale, dy, rows, "scale")
    if want_dscale and scale is None:
        raise ValueError("dscale needs scale")
    dscale = torch.empty(tuple(scale.shape), dtype=torch.float32, device=dy.device) \
        if want_dscale else None
    dsp, dss = _per_row_arg(dscale, dy, rows, "dscale") if want_dscale else (None, 1)
    if dx is None:
        dx = torch.empty(tuple(dy.shape[:-1]) + (2 * n,), dtype=dy.dtype, device=dy.device)
    if y is None and want_y:
        y = torch.empty(tuple(dy.shape), dtype=dy.dtype, device=dy.device)
    if dx.dtype != dy.dtype or (y is not None and y.dtype != dy.dtype):
        raise ValueError("dx and y must have the dtype of dy")
    dxs = _same_rows(dx, rows, 2 * n, "dx")
    yp, ys = (y.data_ptr(), _same_rows(y, rows, n, "y")) if y is not None else (None, n)
    need = lib.swiglu_ckpt8_workspace_size(rows, n, _dtype_code(dy)) if want_dscale else 0
    if workspace is None and need:
        workspace = _scratch(need, dy, stream)
    wp, wb = _span_of_workspace(workspace, dy) if workspace is not None else (None, 0)
    with _on_device(dy.device):
        st = lib.swiglu_ckpt8_bwd(dy.data_ptr(), dys, q.data_ptr(), qst, qs.data_ptr(), qss, sp, ss,
                                  dx.data_ptr(), dxs, yp, ys, dsp, dss, wp, wb, rows, n,
                                  _dtype_code(dy), _stream_handle(dy.device, stream))
    _check(st, "swiglu_ckpt8_bwd")
    return dx, y, dscale
