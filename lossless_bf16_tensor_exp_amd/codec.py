"""Buffer owners for the C ABI: allocate the stream, workspace, size slot and
exponent caches once with torch, then call the library on them.  ``MxLinear``
does the same for a linear layer on microscaled matrices.

Allocation happens only in the constructors; ``encode``/``decode`` only pass
pointers.
"""
from __future__ import annotations

import torch

from . import (CieraError, ciera_decode, ciera_encode, ciera_encode_e0, ciera_encode_spec, ciera_max_encoded_size,
               ciera_read_error, ciera_workspace_size, mx4_encode, mx4_encoded_size, mx4_matmul, mx4_matmul_dx,
               mx4_matmul_mx8, mx8_encode, mx8_encoded_size, mx8_wgrad, mx_workspace_size, zip3_decode, zip3_encode,
               zip3_encode_e0, zip3_encode_spec, zip3_max_encoded_size, zip3_workspace_size)


class Zip3Codec:
    """3-bit exponent code only (no cross-iteration state)."""

    def __init__(self, n: int, device="cuda"):
        self.n = n
        self.capacity = zip3_max_encoded_size(n)
        self.out = torch.empty(self.capacity, dtype=torch.uint8, device=device)
        self.ws = torch.empty(zip3_workspace_size(n), dtype=torch.uint8, device=device)
        self.size = torch.zeros(1, dtype=torch.int64, device=device)

    def encode(self, x, e0_override: int = -1, stream=None):
        zip3_encode(x, self.out, self.ws, self.size, e0_override, stream)

    def encode_e0(self, x, stream=None):
        """Single-read encode with the window base of the previous stream in
        ``out`` (its header byte 7, read on the device before it is
        rewritten); the previous call must have been an encode."""
        zip3_encode_e0(x, self.out, self.out, self.ws, self.size, 7, stream)

    def encode_spec(self, x, stream=None):
        """``encode``'s stream, with x read once when the previous stream's
        window base (its header byte 7 in ``out``) is still the one x's sigma
        gives; the previous call must have been an encode."""
        zip3_encode_spec(x, self.out, self.out, self.ws, self.size, 7, stream)

    def decode(self, stream_bytes, in_size: int, y, stream=None):
        zip3_decode(stream_bytes, in_size, y, self.ws, stream)

    def nbytes(self) -> int:
        return int(self.size.item())

    def error(self, stream=None) -> int:
        return ciera_read_error(self.ws, stream)


class CieraCodec:
    """Exponent reuse with block size B plus the 3-bit code; keeps a sender
    and a receiver exponent cache (both start at zero)."""

    def __init__(self, n: int, B: int, device="cuda"):
        self.n, self.B = n, B
        self.capacity = ciera_max_encoded_size(n, B)
        if self.capacity == 0:
            raise ValueError(f"invalid block size {B}")
        self.out = torch.empty(self.capacity, dtype=torch.uint8, device=device)
        self.ws = torch.empty(ciera_workspace_size(n, B), dtype=torch.uint8, device=device)
        self.ws_dec = torch.empty(ciera_workspace_size(n, B), dtype=torch.uint8, device=device)
        self.size = torch.zeros(1, dtype=torch.int64, device=device)
        self.send_cache = torch.zeros(max(n, 1), dtype=torch.uint8, device=device)
        self.recv_cache = torch.zeros(max(n, 1), dtype=torch.uint8, device=device)

    def encode(self, x, e0_override: int = -1, stream=None):
        ciera_encode(x, self.B, self.send_cache, self.out, self.ws, self.size, e0_override, stream)

    def encode_e0(self, x, stream=None):
        """Single-read encode (x and the sender cache read once) with the
        window base of the previous stream in ``out`` (its header byte 7,
        read on the device before it is rewritten); the previous call must
        have been an encode."""
        ciera_encode_e0(x, self.B, self.send_cache, self.out, self.out, self.ws, self.size, 7, stream)

    def encode_spec(self, x, stream=None):
        """``encode``'s stream and cache update, with x and the sender cache
        read once when the previous stream's window base (its header byte 7
        in ``out``) is still the one x's sigma gives; the previous call must
        have been an encode."""
        ciera_encode_spec(x, self.B, self.send_cache, self.out, self.out, self.ws, self.size, 7, stream)

    def decode(self, stream_bytes, in_size: int, y, stream=None):
        ciera_decode(stream_bytes, in_size, y, self.B, self.recv_cache, self.ws_dec, stream)

    def nbytes(self) -> int:
        return int(self.size.item())

    def error(self, stream=None) -> int:
        """Device status of the last encode."""
        return ciera_read_error(self.ws, stream)

    def decode_error(self, stream=None) -> int:
        """Device status of the last decode."""
        return ciera_read_error(self.ws_dec, stream)


class MxLinear:
    """y = x W^T with the weights in 4 bits, and its gradients from an 8-bit
    checkpoint of x: one linear layer, or with ``offsets`` (groups + 1 row
    numbers) the experts of a mixture-of-experts layer, whose groups (n, k)
    matrices lie one behind the other.  Takes up to ``tokens`` rows a call.
    With ``scaled``, ``keep`` takes a BF16 y from the scaled matrix
    instructions (``mx4_matmul_mx8``: faster on many rows, less exact than FP32).

    ``keep`` and the calls that read the checkpoint share one buffer, so one
    layer's forward and backward belong to one stream, or are ordered by the
    caller.  ``backward`` takes the offsets its ``keep`` had.  Autograd records
    none of this; ``backward`` is the caller's to call."""

    def __init__(self, tokens: int, n: int, k: int, groups: int = 1, device="cuda", scaled: bool = False):
        self.tokens, self.n, self.k, self.groups, self.scaled = tokens, n, k, groups, scaled
        size = mx_workspace_size(tokens, n, k, groups)
        if size == 0:
            raise ValueError(f"no workspace for {tokens} x {n} x {k} in {groups} groups")
        self.w = torch.empty(mx4_encoded_size(groups * n, k), dtype=torch.uint8, device=device)
        self.xq = torch.empty(mx8_encoded_size(tokens, k), dtype=torch.uint8, device=device)
        self.ws = torch.empty(size, dtype=torch.uint8, device=device)
        self.kept = None  # rows of the checkpoint in xq, None while there is none

    def load(self, weights, stream=None):
        """The BF16 weights, (groups, n, k) or their rows one behind the other,
        (groups * n, k), into ``w``.  Rows may lie further apart than k, the
        same everywhere."""
        flat = (self.groups * self.n, self.k)
        self._shape("the weights", weights, (self.groups, self.n, self.k), flat)
        try:
            rows = weights.view(flat)
        except RuntimeError:
            raise ValueError(f"the weights' rows do not lie equally far apart: strides {weights.stride()}") from None
        mx4_encode(rows, self.w, stream)

    def _shape(self, name: str, t, *wanted):
        """The calls take n and k from their tensors, and would read the layer's buffers as those of a smaller matrix."""
        if tuple(t.shape) not in wanted:
            raise ValueError(f"{name} is {tuple(t.shape)}, the layer's {' or '.join(map(str, wanted))}")

    def _product(self, x, y, offsets):
        rows = x.shape[0]
        if rows > self.tokens:
            raise ValueError(f"{rows} rows in a layer made for {self.tokens}")
        self._shape("x", x, (rows, self.k))
        self._shape("y", y, (rows, self.n))
        self._table(offsets)

    def _table(self, offsets):
        if (1 if offsets is None else offsets.numel() - 1) != self.groups:
            raise ValueError(f"offsets must hold {self.groups} + 1 row numbers")

    def forward(self, x, y, offsets=None, stream=None):
        """y = x W^T; nothing is kept."""
        self._product(x, y, offsets)
        mx4_matmul(x, self.w, y, self.ws, offsets, stream)

    def keep(self, x, y, offsets=None, stream=None):
        """The checkpoint of x into ``xq``, and y from it: what ``backward``
        sees is what the product took."""
        self._product(x, y, offsets)
        self.kept = None  # until both calls are made: the first one overwrites xq
        mx8_encode(x, self.xq, stream)
        mx4_matmul_mx8(self.xq, self.k, self.w, y, self.ws, offsets, stream,
                       self.scaled and y.dtype is not torch.float32)
        self.kept = x.shape[0]

    def backward(self, dy, dx, dw, offsets=None, accumulate: bool = False, stream=None):
        """dx = dy W and dw = dy^T x from the checkpoint that ``keep`` left;
        either output may be None."""
        self._table(offsets)
        if dy.shape[0] != self.kept:
            raise ValueError(f"{dy.shape[0]} rows of dy for " +
                             ("no checkpoint" if self.kept is None else f"a checkpoint of {self.kept}"))
        self._shape("dy", dy, (self.kept, self.n))
        if dx is not None:
            self._shape("dx", dx, (self.kept, self.k))
        if dw is not None:
            stack = (self.groups, self.n, self.k)
            self._shape("dw", dw, stack, *([stack[1:]] if self.groups == 1 else []))
        if dx is not None:
            mx4_matmul_dx(dy, self.w, dx, self.ws, offsets, stream)
        if dw is not None:
            mx8_wgrad(dy, self.xq, dw, self.ws, offsets, accumulate, stream)

    def error(self, stream=None) -> int:
        """Status of the last product (CIERA_ERR_ARG for offsets that are not
        in order); synchronises."""
        return ciera_read_error(self.ws, stream)


# One-shot calls: allocate the stream and workspace with torch, run one
# encode or decode on the current stream, and return the result.  Reading the
# compressed size back synchronizes the stream; the classes above keep their
# buffers and do not.

def _raise_device_error(ws, what: str) -> None:
    st = ciera_read_error(ws)
    if st:
        raise CieraError(st, what)


def zip3_encode_tensor(x):
    """3-bit code of the BF16 values x (a CUDA tensor, read as raw 16-bit
    patterns).  Returns (stream bytes, size)."""
    n = x.numel()
    out = torch.empty(zip3_max_encoded_size(n), dtype=torch.uint8, device=x.device)
    ws = torch.empty(zip3_workspace_size(n), dtype=torch.uint8, device=x.device)
    size = torch.zeros(1, dtype=torch.int64, device=x.device)
    zip3_encode(x, out, ws, size)
    _raise_device_error(ws, "zip3_encode")
    k = int(size.item())
    return out[:k], k


def zip3_decode_tensor(stream_bytes, n: int):
    """Inverse of zip3_encode_tensor: the n values as an int16 tensor of raw patterns."""
    y = torch.empty(n, dtype=torch.int16, device=stream_bytes.device)
    ws = torch.empty(zip3_workspace_size(n), dtype=torch.uint8, device=stream_bytes.device)
    zip3_decode(stream_bytes, stream_bytes.numel(), y, ws)
    _raise_device_error(ws, "zip3_decode")
    return y


def ciera_encode_tensor(x, B: int, prev_exp):
    """Exponent reuse against the sender cache prev_exp (n bytes, updated in
    place) plus the 3-bit code.  Returns (stream bytes, size)."""
    n = x.numel()
    cap = ciera_max_encoded_size(n, B)
    if cap == 0:
        raise ValueError(f"invalid block size {B}")
    out = torch.empty(cap, dtype=torch.uint8, device=x.device)
    ws = torch.empty(ciera_workspace_size(n, B), dtype=torch.uint8, device=x.device)
    size = torch.zeros(1, dtype=torch.int64, device=x.device)
    ciera_encode(x, B, prev_exp, out, ws, size)
    _raise_device_error(ws, "ciera_encode")
    k = int(size.item())
    return out[:k], k


def ciera_decode_tensor(stream_bytes, n: int, B: int, prev_exp):
    """Inverse of ciera_encode_tensor against the receiver cache prev_exp
    (updated in place)."""
    y = torch.empty(n, dtype=torch.int16, device=stream_bytes.device)
    ws = torch.empty(ciera_workspace_size(n, B), dtype=torch.uint8, device=stream_bytes.device)
    ciera_decode(stream_bytes, stream_bytes.numel(), y, B, prev_exp, ws)
    _raise_device_error(ws, "ciera_decode")
    return y
