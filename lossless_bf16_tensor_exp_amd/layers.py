"""What stands around the products of a layer (the ``rms_norm*``,
``expert_*`` and ``low_rank_*`` entry points of ``include/ciera.h``).

    rms_norm(x, weight, y=None, yq=None, residual=None, h=None, rstd=None, eps=1e-6, stream=None)
    rms_norm_backward(dy, h, weight, rstd, dx, dw, ws=None, dh=None, accumulate=False, stream=None)
    rms_norm_workspace_size(rows, cols)
    expert_sort(ids, offsets, place, order, ws, stream=None)
    expert_workspace_size(tokens, choices, experts)
    expert_dispatch(x, place, out=None, outq=None, rows=None, stream=None)
    expert_combine(rows, place, out, weights=None, residual=None, stream=None)
    expert_combine_backward(dout, rows, place, drows, dweights, weights=None, stream=None)
    low_rank_add(x, a, b, offsets, y, ws, base=None, order=None, scales=None, stream=None)
    low_rank_workspace_size(tokens, n, k, rank, adapters)

Matrices, streams and devices are as for the products (``mx.py``): two
dimensions, rows any stride apart, outputs the caller's, on the current stream
of the tensors' device unless one is given.  Nothing here is recorded by
autograd; the gradients are calls of their own.
"""
from __future__ import annotations

import ctypes

import torch

from . import _raise, load_library
from .mx import _BF16, _current_device, _f32, _i64, _raw_stream, _rows, _u8

_i32 = torch.int32
_vp, _u64, _u32, _int = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
_functions = {}


def _bind():
    """The C functions by name.  The table is seen when all of it is there:
    another thread may make its first call meanwhile."""
    global _functions
    if not _functions:
        lib, table = load_library(), {}
        m = [_vp, _u64]  # a matrix and its row stride, or a buffer and its length
        sigs = {
            "rms_norm_workspace_size": [_u64] * 2,
            "expert_workspace_size": [_u64, _u64, _u32],
            "low_rank_workspace_size": [_u64] * 4 + [_u32],
            "rms_norm": m + m + [_vp, ctypes.c_float] + m + m + m + [_vp, _u64, _u64, _vp],
            "rms_norm_backward": m + m + [_vp, _vp] + m + m + [_vp, _u32, _u32, _u64, _u64] + m + [_vp],
            "expert_sort": [_vp, _u32, _u64, _u64, _u32, _vp, _vp, _vp] + m + [_vp],
            "expert_dispatch": m + [_vp] + [_u64] * 4 + m + m + [_vp],
            "expert_combine": m + [_u32, _u64, _vp, _vp] + m + m + [_u32, _u64, _u64, _u64, _vp],
            "expert_combine_backward": m + m + [_u32, _u64, _vp, _vp] + m + [_vp, _u64, _u64, _u64, _vp],
            "low_rank_add": m + [_vp] * 5 + m + [_u32] + m + [_u32] + [_u64] * 4 + [_u32] + m + [_vp],
        }
        for name, args in sigs.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, _u64 if name.endswith("_size") else _int
            table[name] = f
        _functions = table
    return _functions


def _elsewhere(t, name, device):
    raise ValueError(f"{name} is on {t.device}" + (f", the call's first tensor on cuda:{device}" if device >= 0 else ""))


def _matrix(t, name, device, rows, cols, f32=False):
    """Address and row stride of a matrix of rows x cols; none for None."""
    if t is None:
        return None, 0
    dtype = t.dtype
    if dtype not in _BF16 and not (f32 and dtype is _f32):
        _rows(t, name, f32)  # says what is wrong
    if t.get_device() != device or device < 0:
        _elsewhere(t, name, device)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} is {tuple(t.shape)}, not {(rows, cols)}")
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name}'s rows must be contiguous and must not overlap")
    return t.data_ptr(), ld


def _vector(t, name, device, dtypes, shape):
    """Address of a contiguous tensor of a type and shape; none for None."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must hold {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.get_device() != device or device < 0:
        _elsewhere(t, name, device)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _buffer(t, name, device):
    """Address and length of a buffer of bytes; none for None."""
    if t is None:
        return None, 0
    if t.dtype is not _u8 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 device tensor")
    if t.get_device() != device or device < 0:
        _elsewhere(t, name, device)
    n = t.numel()
    return (t.data_ptr() if n else None), n


def _entries(t, name, device, dtypes):
    """Tokens, choices and address of a table of entries; one dimension: one choice a token."""
    shape = t.shape
    if len(shape) not in (1, 2):
        raise ValueError(f"{name} must be (tokens, choices) or (tokens,), got {tuple(shape)}")
    return shape[0], shape[1] if len(shape) == 2 else 1, _vector(t, name, device, dtypes, shape)


def _call(name, device, stream, *args):
    """The C call ``name`` on the tensors' device: the current stream there
    unless one is given."""
    f = _functions[name]
    s = _raw_stream(device) if stream is None else stream.cuda_stream
    if device == _current_device():
        st = f(*args, s)
    else:
        with torch.cuda.device(device):
            st = f(*args, s)
    if st:
        _raise(st, name)


def rms_norm_workspace_size(rows: int, cols: int) -> int:
    return _bind()["rms_norm_workspace_size"](rows, cols)


def expert_workspace_size(tokens: int, choices: int, experts: int) -> int:
    return _bind()["expert_workspace_size"](tokens, choices, experts)


def low_rank_workspace_size(tokens: int, n: int, k: int, rank: int, adapters: int) -> int:
    return _bind()["low_rank_workspace_size"](tokens, n, k, rank, adapters)


def rms_norm(x, weight, y=None, yq=None, residual=None, h=None, rstd=None, eps: float = 1e-6, stream=None) -> None:
    """h = x + residual, y = h weight / sqrt(mean(h^2) + eps) of every row: y in
    BF16, ``yq`` in mx8 (mx8_encode's bytes of y), or both.  ``h`` (with a
    residual; x or residual itself may be given) and ``rstd`` (rows, float32)
    are what the backward pass takes."""
    _bind()
    rows, cols, ldx = _rows(x, "x")
    on = x.get_device()
    _call("rms_norm", on, stream, x.data_ptr(), ldx, *_matrix(residual, "residual", on, rows, cols),
          _vector(weight, "weight", on, _BF16, (cols,)), eps, *_matrix(h, "h", on, rows, cols),
          *_matrix(y, "y", on, rows, cols), *_buffer(yq, "yq", on), _vector(rstd, "rstd", on, (_f32,), (rows,)), rows, cols)


def rms_norm_backward(dy, h, weight, rstd, dx, dw, ws=None, dh=None, accumulate: bool = False, stream=None) -> None:
    """The gradients of rms_norm: ``dx`` of h (so of x and of the residual), with
    ``dh``, what h has from elsewhere, added; ``dw`` (cols, BF16 or float32) of
    the weight, added to what is there with ``accumulate``.  Either may be None;
    ``dw`` needs the workspace.  ``h`` is x where there was no residual."""
    _bind()
    rows, cols, lddy = _rows(dy, "dy")
    on = dy.get_device()
    _call("rms_norm_backward", on, stream, dy.data_ptr(), lddy, *_matrix(h, "h", on, rows, cols),
          _vector(weight, "weight", on, _BF16, (cols,)), _vector(rstd, "rstd", on, (_f32,), (rows,)),
          *_matrix(dh, "dh", on, rows, cols), *_matrix(dx, "dx", on, rows, cols),
          _vector(dw, "dw", on, (*_BF16, _f32), (cols,)), 1 if dw is not None and dw.dtype is _f32 else 0,
          1 if accumulate else 0, rows, cols, *_buffer(ws, "ws", on))


def expert_sort(ids, offsets, place, order, ws, stream=None) -> None:
    """Entries sorted by expert: ``ids`` (tokens, choices), or (tokens,) for one
    choice, int32 or int64, -1 for none; ``offsets`` (experts + 1) int64 is what
    the products take; ``place`` (as ids, int32) is each entry's row; ``order``
    (all entries, int32, or None) each row's entry."""
    _bind()
    on = ids.get_device()
    tokens, choices, at = _entries(ids, "ids", on, (_i32, _i64))
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must hold experts + 1 row numbers")
    experts = offsets.numel() - 1
    _call("expert_sort", on, stream, at, 1 if ids.dtype is _i64 else 0, tokens, choices, experts,
          _vector(offsets, "offsets", on, (_i64,), (experts + 1,)), _vector(place, "place", on, (_i32,), ids.shape),
          _vector(order, "order", on, (_i32,), (tokens * choices,)), *_buffer(ws, "ws", on))


def expert_dispatch(x, place, out=None, outq=None, rows=None, stream=None) -> None:
    """Row t of x to the rows ``place[t]`` of ``out`` (BF16) and of the mx8 matrix
    ``outq`` of ``rows`` rows (out's number of rows, or every entry's, unless
    given)."""
    _bind()
    n, cols, ldx = _rows(x, "x")
    on = x.get_device()
    tokens, choices, at = _entries(place, "place", on, (_i32,))
    if n != tokens:
        raise ValueError(f"{n} rows of x and {tokens} of place")
    if rows is None:
        rows = out.shape[0] if out is not None else tokens * choices
    _call("expert_dispatch", on, stream, x.data_ptr(), ldx, at, tokens, choices, cols, rows,
          *_matrix(out, "out", on, rows, cols), *_buffer(outq, "outq", on))


def expert_combine(rows, place, out, weights=None, residual=None, stream=None) -> None:
    """out[t] = residual[t] + sum over the choices of weights[t, j] *
    rows[place[t, j]]: rows BF16 or float32, out BF16 or float32, weights
    float32 in place's shape, None for ones.  Without weights and residual it is
    the gradient of expert_dispatch."""
    _bind()
    n, cols, ld = _rows(rows, "rows", True)
    on = rows.get_device()
    tokens, choices, at = _entries(place, "place", on, (_i32,))
    _call("expert_combine", on, stream, rows.data_ptr(), ld, 1 if rows.dtype is _f32 else 0, n, at,
          _vector(weights, "weights", on, (_f32,), place.shape), *_matrix(residual, "residual", on, tokens, cols),
          *_matrix(out, "out", on, tokens, cols, True), 1 if out.dtype is _f32 else 0, tokens, choices, cols)


def expert_combine_backward(dout, rows, place, drows, dweights, weights=None, stream=None) -> None:
    """The gradients of expert_combine from that of its output: ``drows`` (BF16)
    of the rows, ``dweights`` (float32, in place's shape) of the weights; either
    may be None."""
    _bind()
    n, cols, ld = _rows(rows, "rows", True)
    on = rows.get_device()
    tokens, choices, at = _entries(place, "place", on, (_i32,))
    shape = place.shape
    _call("expert_combine_backward", on, stream, *_matrix(dout, "dout", on, tokens, cols), rows.data_ptr(), ld,
          1 if rows.dtype is _f32 else 0, n, at, _vector(weights, "weights", on, (_f32,), shape),
          *_matrix(drows, "drows", on, n, cols), _vector(dweights, "dweights", on, (_f32,), shape), tokens, choices, cols)


def low_rank_add(x, a, b, offsets, y, ws, base=None, order=None, scales=None, stream=None) -> None:
    """y = base + scales[a] * B_a (A_a x) for every row's adapter a: x (tokens, k)
    BF16, ``a`` (adapters, rank, k) and ``b`` (adapters, n, rank) BF16, y and
    base (tokens, n) BF16 or float32, base None for zeros, or y itself.
    ``offsets`` (adapters + 1, int64) and ``order`` (tokens, int32; None: the
    rows lie sorted) are expert_sort's; rows of no adapter are base."""
    _bind()
    tokens, k, ldx = _rows(x, "x")
    on = x.get_device()
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a must be (adapters, rank, k) and b (adapters, n, rank)")
    (adapters, rank, _), n = a.shape, b.shape[1]
    _call("low_rank_add", on, stream, x.data_ptr(), ldx, _vector(a, "a", on, _BF16, (adapters, rank, k)),
          _vector(b, "b", on, _BF16, (adapters, n, rank)), _vector(scales, "scales", on, (_f32,), (adapters,)),
          _vector(offsets, "offsets", on, (_i64,), (adapters + 1,)), _vector(order, "order", on, (_i32,), (tokens,)),
          *_matrix(base, "base", on, tokens, n, True), 1 if base is not None and base.dtype is _f32 else 0,
          *_matrix(y, "y", on, tokens, n, True), 1 if y.dtype is _f32 else 0, tokens, n, k, rank, adapters,
          *_buffer(ws, "ws", on))
