"""Microscaled matrices (the ``mx*`` entry points of ``include/ciera.h``):
BF16 matrices held in 8 bits (mx8) or 4 bits (mx4) per value with one
power-of-two scale per 32 values of a row, and the products of a linear layer
on them.

    mx8_encoded_size(rows, cols)          mx4_encoded_size(rows, cols)
    mx8_encode(x, out, stream=None)       mx4_encode(x, out, stream=None)
    mx8_decode(inp, y, stream=None)       mx4_decode(inp, y, stream=None)
    mx_workspace_size(tokens, n, k, groups=1)
    mx4_matmul(x, w, y, ws, offsets=None, stream=None)                 y = x W^T
    mx4_matmul_mx8(xq, k, w, y, ws, offsets=None, stream=None, scaled=False)   y = x W^T, x in mx8
    mx4_matmul_dx(dy, w, dx, ws, offsets=None, stream=None)            dx = dy W
    mx8_wgrad(dy, xq, dw, ws, offsets=None, accumulate=False, stream=None)   dW = dy^T x

Matrices are two-dimensional BF16 tensors (bfloat16, or int16/uint16
patterns) whose rows may lie any stride of at least their length apart;
outputs of the products may be float32 too.  ``xq`` and ``w`` are uint8
tensors holding encoded matrices.  With ``offsets`` (int64, groups + 1 row
numbers on the device) the rows offsets[g] .. offsets[g+1] - 1 belong to
group g and ``w`` holds groups matrices one behind the other; ``dw`` is then
(groups, n, k).  Every tensor is on one device; a call made while another
device is current runs on the tensors' own, on that device's current stream.

Nothing here is recorded by autograd: the calls write through addresses, an
input's ``requires_grad`` has no effect, and the gradients are the calls
``mx4_matmul_dx`` and ``mx8_wgrad``, made by the caller.
"""
from __future__ import annotations

import ctypes

import torch

from . import _raise, load_library

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_f32, _i64, _u8 = torch.float32, torch.int64, torch.uint8
_vp, _u64, _u32, _i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
_SCALED = 4  # CIERA_MX_SCALED
_bound = None
# the current device without the check that the GPU is initialised (a device tensor was there first; 0.2 us a call)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# the current stream's handle without the Stream object around it (1 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _lib():
    global _bound
    if _bound is None:
        lib = load_library()
        for name in ("mx8_encoded_size", "mx4_encoded_size"):
            getattr(lib, name).argtypes, getattr(lib, name).restype = [_u64, _u64], _u64
        lib.mx_workspace_size.argtypes, lib.mx_workspace_size.restype = [_u64, _u64, _u64, _u32], _u64
        tail = [_u64, _u64, _u64, _u32, _vp, _vp, _u64, _vp]  # tokens, n, k, groups, offsets, ws, ws_bytes, stream
        sigs = {
            "mx8_encode": [_vp, _u64, _u64, _u64, _vp, _u64, _vp],
            "mx4_encode": [_vp, _u64, _u64, _u64, _vp, _u64, _vp],
            "mx8_decode": [_vp, _u64, _u64, _u64, _vp, _u64, _vp],
            "mx4_decode": [_vp, _u64, _u64, _u64, _vp, _u64, _vp],
            "mx4_matmul": [_vp, _u64, _vp, _u64, _vp, _u64, _u32] + tail,
            "mx4_matmul_mx8": [_vp, _u64, _vp, _u64, _vp, _u64, _u32] + tail,
            "mx4_matmul_dx": [_vp, _u64, _vp, _u64, _vp, _u64, _u32] + tail,
            "mx8_wgrad": [_vp, _u64, _vp, _u64, _vp, _u32, _u32] + tail,
        }
        for name, args in sigs.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, _i32
        _bound = lib
    return _bound


def _rows(t, name, f32=False):
    """Rows, columns and row stride of a matrix; f32: FP32 allowed too."""
    dtype = t.dtype
    if dtype not in _BF16 and not (f32 and dtype is _f32):
        raise TypeError(f"{name} must hold BF16 patterns (bfloat16/int16/uint16){' or float32' if f32 else ''}, "
                        f"got {dtype}")
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a two-dimensional device tensor")
    rows, cols = t.shape
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name}'s rows must be contiguous and must not overlap")
    return rows, cols, ld


def _bytes(t, name):
    """Address and length of a buffer of bytes."""
    if t.dtype is not _u8 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 device tensor")
    n = t.numel()
    return (t.data_ptr() if n else None), n


def _call(name, device, others, stream, *args):
    """The C call ``name`` on the tensors' device: the current stream there
    unless one is given."""
    for o in others:
        if o.get_device() != device:
            raise ValueError(f"tensors on cuda:{device} and {o.device} in one call")
    f = getattr(_lib(), name)
    s = _raw_stream(device) if stream is None else stream.cuda_stream
    if device == _current_device():
        st = f(*args, s)
    else:
        with torch.cuda.device(device):
            st = f(*args, s)
    if st:
        _raise(st, name)


def mx8_encoded_size(rows: int, cols: int) -> int:
    return _lib().mx8_encoded_size(rows, cols)


def mx4_encoded_size(rows: int, cols: int) -> int:
    return _lib().mx4_encoded_size(rows, cols)


def mx_workspace_size(tokens: int, n: int, k: int, groups: int = 1) -> int:
    return _lib().mx_workspace_size(tokens, n, k, groups)


def _encode(name, x, out, stream):
    rows, cols, ld = _rows(x, "x")
    to, size = _bytes(out, "out")
    _call(name, x.get_device(), (out,), stream, x.data_ptr(), rows, cols, ld, to, size)


def _decode(name, inp, y, stream):
    rows, cols, ld = _rows(y, "y")
    src, size = _bytes(inp, "inp")
    _call(name, y.get_device(), (inp,), stream, src, size, rows, cols, y.data_ptr(), ld)


def mx8_encode(x, out, stream=None) -> None:
    """The matrix x in 8 bits a value into ``out`` (at least
    mx8_encoded_size(*x.shape) bytes)."""
    _encode("mx8_encode", x, out, stream)


def mx4_encode(x, out, stream=None) -> None:
    """The matrix x in 4 bits a value into ``out`` (at least
    mx4_encoded_size(*x.shape) bytes)."""
    _encode("mx4_encode", x, out, stream)


def mx8_decode(inp, y, stream=None) -> None:
    """What the mx8 matrix of y's shape in ``inp`` stands for, as BF16."""
    _decode("mx8_decode", inp, y, stream)


def mx4_decode(inp, y, stream=None) -> None:
    """What the mx4 matrix of y's shape in ``inp`` stands for, as BF16."""
    _decode("mx4_decode", inp, y, stream)


def _groups(offsets):
    """Number of groups, the table's address, and the table among the tensors of the call."""
    if offsets is None:
        return 1, None, ()
    if offsets.dtype is not _i64 or not offsets.is_cuda or not offsets.is_contiguous() or offsets.numel() < 2:
        raise ValueError("offsets must be a contiguous int64 device tensor of groups + 1 row numbers")
    return offsets.numel() - 1, offsets.data_ptr(), (offsets,)


def _product(name, a, lead, width, w, out, ws, offsets, tokens, n, k, stream, bf16=0):
    """One call of a matmul-shaped entry point; ``lead`` is its left operand's
    pointer and stride or size, ``width`` the output's columns, ``bf16`` what a
    BF16 output is asked for with."""
    rows, cols, ldo = _rows(out, "the output", f32=True)
    if rows != tokens or cols != width:
        raise ValueError(f"the output is {rows} x {cols}, the product {tokens} x {width}")
    wp, wn = _bytes(w, "w")
    sp, sn = _bytes(ws, "ws")
    groups, offs, table = _groups(offsets)
    _call(name, out.get_device(), (a, w, ws, *table), stream, *lead, wp, wn, out.data_ptr(), ldo,
          1 if out.dtype is _f32 else bf16, tokens, n, k, groups, offs, sp, sn)


def mx4_matmul(x, w, y, ws, offsets=None, stream=None) -> None:
    """y = x W^T: x (tokens, k) BF16, w the groups' (n, k) weights in mx4, y
    (tokens, n) BF16 or float32; ws at least mx_workspace_size bytes."""
    tokens, k, ldx = _rows(x, "x")
    n = y.shape[-1]
    _product("mx4_matmul", x, (x.data_ptr(), ldx), n, w, y, ws, offsets, tokens, n, k, stream)


def mx4_matmul_mx8(xq, k: int, w, y, ws, offsets=None, stream=None, scaled: bool = False) -> None:
    """y = x W^T with x (y's rows, k) in mx8.  ``scaled`` (y in BF16) takes the
    scaled matrix instructions: faster on many rows, and within each block of
    32 they cut what lies below 2^-13 of the largest product."""
    if y.dim() != 2:
        raise ValueError("the output must be a two-dimensional device tensor")
    if scaled and y.dtype is _f32:
        raise ValueError("the scaled matrix instructions are for a BF16 output")
    tokens, n = y.shape
    _product("mx4_matmul_mx8", xq, _bytes(xq, "xq"), n, w, y, ws, offsets, tokens, n, k, stream,
             _SCALED if scaled else 0)


def mx4_matmul_dx(dy, w, dx, ws, offsets=None, stream=None) -> None:
    """dx = dy W: dy (tokens, n) BF16, dx (tokens, k) BF16 or float32."""
    tokens, n, ld = _rows(dy, "dy")
    k = dx.shape[-1]
    _product("mx4_matmul_dx", dy, (dy.data_ptr(), ld), k, w, dx, ws, offsets, tokens, n, k, stream)


def mx8_wgrad(dy, xq, dw, ws, offsets=None, accumulate: bool = False, stream=None) -> None:
    """dW = dy^T x per group: dy (tokens, n) BF16, xq the (tokens, k) mx8
    checkpoint of x, dw (groups, n, k), or (n, k) for one group, contiguous,
    BF16 or float32; accumulate adds to dw instead of writing it."""
    tokens, n, ld = _rows(dy, "dy")
    groups, offs, table = _groups(offsets)
    if dw.dtype not in _BF16 and dw.dtype is not _f32:
        raise TypeError(f"dw must hold BF16 patterns (bfloat16/int16/uint16) or float32, got {dw.dtype}")
    shape = tuple(dw.shape) if dw.dim() == 3 else (1, *dw.shape)
    if not dw.is_cuda or not dw.is_contiguous() or len(shape) != 3 or shape[:2] != (groups, n):
        raise ValueError(f"dw must be a contiguous device tensor ({groups}, {n}, k), got {tuple(dw.shape)}")
    xp, xn = _bytes(xq, "xq")
    sp, sn = _bytes(ws, "ws")
    _call("mx8_wgrad", dy.get_device(), (xq, dw, ws, *table), stream, dy.data_ptr(), ld, xp, xn, dw.data_ptr(),
          1 if dw.dtype is _f32 else 0, 1 if accumulate else 0, tokens, n, shape[2], groups, offs, sp, sn)
