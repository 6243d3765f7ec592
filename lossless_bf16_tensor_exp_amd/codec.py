"""Buffer owners for the C ABI: allocate the stream, workspace, size slot and
exponent caches once with torch, then call the library on them.  ``MxLinear``
does the same for a linear layer on microscaled matrices; ``RmsNorm``,
``ExpertRows`` and ``LowRankAdapters`` for what stands around its products.

Allocation happens only in the constructors; ``encode``/``decode`` only pass
pointers.  The constructors fill what needs a value on the current stream:
calls on another one are ordered behind that by the caller.
"""
from __future__ import annotations

import torch

from . import (CieraError, ciera_decode, ciera_encode, ciera_encode_e0, ciera_encode_spec, ciera_max_encoded_size,
               ciera_read_error, ciera_workspace_size, expert_combine, expert_combine_backward, expert_dispatch,
               expert_sort, expert_workspace_size, low_rank_add, low_rank_workspace_size, mx4_encode, mx4_encoded_size,
               mx4_matmul, mx4_matmul_dx, mx4_matmul_mx8, mx8_encode, mx8_encoded_size, mx8_wgrad, mx_workspace_size,
               rms_norm, rms_norm_backward, rms_norm_workspace_size, zip3_decode, zip3_encode, zip3_encode_e0,
               zip3_encode_spec, zip3_max_encoded_size, zip3_workspace_size)

_WS_HEAD = 256  # bytes of a workspace before its status words; their number is in there


def _workspace(size: int, device):
    """A workspace without status words, which reads as CIERA_OK: ``error``
    before any call would else take their number from what the memory held."""
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    ws[:_WS_HEAD].zero_()
    return ws


class Zip3Codec:
    """3-bit exponent code only (no cross-iteration state)."""

    def __init__(self, n: int, device="cuda"):
        self.n = n
        self.capacity = zip3_max_encoded_size(n)
        self.out = torch.empty(self.capacity, dtype=torch.uint8, device=device)
        self.ws = _workspace(zip3_workspace_size(n), device)
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
        self.ws = _workspace(ciera_workspace_size(n, B), device)
        self.ws_dec = _workspace(ciera_workspace_size(n, B), device)
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
        self.ws = _workspace(size, device)
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

    def keep_dispatched(self, x, experts: "ExpertRows", y, stream=None):
        """``keep`` of the rows that ``experts`` makes of the tokens x: they go
        right into the checkpoint.  y has a row for every entry of the sort;
        ``backward`` takes ``experts.offsets``."""
        rows = experts.rows()
        if rows > self.tokens:
            raise ValueError(f"{rows} rows in a layer made for {self.tokens}")
        self._shape("x", x, (experts.tokens(), self.k))
        self._shape("y", y, (rows, self.n))
        self._table(experts.offsets)
        self.kept = None
        expert_dispatch(x, experts.place, outq=self.xq, rows=rows, stream=stream)
        mx4_matmul_mx8(self.xq, self.k, self.w, y, self.ws, experts.offsets, stream,
                       self.scaled and y.dtype is not torch.float32)
        self.kept = rows

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


class RmsNorm:
    """y = h w / sqrt(mean(h^2) + eps), h = x + residual, of up to ``rows`` rows
    of ``cols``; keeps the weight, what the backward pass needs of a call's rows
    (``rstd``) and its workspace.  ``forward`` and the ``backward`` that belongs
    to it are on one stream, or ordered by the caller; autograd records
    neither."""

    def __init__(self, rows: int, cols: int, eps: float = 1e-6, device="cuda"):
        size = rms_norm_workspace_size(rows, cols)
        if size == 0:
            raise ValueError(f"no norm of {rows} x {cols}")
        self.rows, self.cols, self.eps = rows, cols, eps
        self.weight = torch.ones(cols, dtype=torch.bfloat16, device=device)
        self.rstd = torch.empty(rows, dtype=torch.float32, device=device)
        self.ws = torch.empty(size, dtype=torch.uint8, device=device)
        self.kept = None  # rows of the last forward pass

    def forward(self, x, y=None, yq=None, residual=None, h=None, stream=None):
        """y in BF16, in mx8 (yq), or both; h where a residual is given."""
        rows = x.shape[0]
        if rows > self.rows:
            raise ValueError(f"{rows} rows in a norm made for {self.rows}")
        rms_norm(x, self.weight, y, yq, residual, h, self.rstd[:rows], self.eps, stream)
        self.kept = rows

    def backward(self, dy, h, dx, dw, dh=None, accumulate: bool = False, stream=None):
        """dx and dw of the last forward pass, h being what it left there (x
        without a residual), and dh the gradient that h has from elsewhere."""
        if dy.shape[0] != self.kept:
            raise ValueError(f"{dy.shape[0]} rows of dy for " +
                             ("no forward pass" if self.kept is None else f"a forward pass of {self.kept}"))
        rms_norm_backward(dy, h, self.weight, self.rstd[:self.kept], dx, dw, self.ws, dh, accumulate, stream)


class ExpertRows:
    """The rows of up to ``tokens`` tokens, ``choices`` entries each, by expert:
    ``sort`` keeps the entries' rows (``place``), the rows' entries (``order``)
    and the experts' ``offsets``, which the products take; the other calls move
    rows by them.  A sort and the calls that use it belong to one stream, or are
    ordered by the caller."""

    def __init__(self, tokens: int, choices: int, experts: int, device="cuda"):
        size = expert_workspace_size(tokens, choices, experts)
        if size == 0:
            raise ValueError(f"no sort of {tokens} x {choices} by {experts} experts")
        self.most, self.choices, self.experts = tokens, choices, experts
        self.offsets = torch.zeros(experts + 1, dtype=torch.int64, device=device)
        self._place = torch.empty(tokens, choices, dtype=torch.int32, device=device)
        self._order = torch.empty(tokens * choices, dtype=torch.int32, device=device)
        self.ws = _workspace(size, device)
        self.place, self.order = self._place[:0], self._order[:0]

    def tokens(self) -> int:
        return self.place.shape[0]

    def rows(self) -> int:
        """Entries of the last sort: rows that a buffer of dispatched rows has,
        the last ones unused where entries have no expert."""
        return self.order.shape[0]

    def sort(self, ids, stream=None):
        """ids (tokens, choices) int32 or int64, -1 for no expert."""
        if ids.dim() != 2 or ids.shape[1] != self.choices or ids.shape[0] > self.most:
            raise ValueError(f"ids are {tuple(ids.shape)}, the sort was made for {(self.most, self.choices)}")
        tokens = ids.shape[0]
        place, order = self._place[:tokens], self._order[:tokens * self.choices]
        expert_sort(ids, self.offsets, place, order, self.ws, stream)
        self.place, self.order = place, order

    def dispatch(self, x, out=None, outq=None, stream=None):
        """Each token's row to its entries' rows, in BF16 or mx8."""
        expert_dispatch(x, self.place, out, outq, self.rows() if out is None else None, stream)

    def dispatch_backward(self, drows, dx, stream=None):
        """dx = the sum of a token's entries' gradients."""
        expert_combine(drows, self.place, dx, stream=stream)

    def combine(self, rows, out, weights=None, residual=None, stream=None):
        """out = residual + a token's rows by its weights."""
        expert_combine(rows, self.place, out, weights, residual, stream)

    def combine_backward(self, dout, rows, drows, dweights, weights=None, stream=None):
        expert_combine_backward(dout, rows, self.place, drows, dweights, weights, stream)

    def error(self, stream=None) -> int:
        """Status of the last sort (CIERA_ERR_ARG for a number of no expert);
        synchronises."""
        return ciera_read_error(self.ws, stream)


class LowRankAdapters:
    """``adapters`` low-rank adapters, B (n, rank) and A (rank, k) each, beside a
    projection that all requests share: y = base + scale B (A x) by the adapter
    of each of up to ``tokens`` rows.  ``plan`` sorts a step's rows once for all
    its projections (another adapters' plan of the same rows can be given to
    ``add``); rows of adapter -1 are base.  ``load``, ``plan`` and ``add`` belong
    to one stream, or are ordered by the caller.  For serving: there is no
    gradient."""

    def __init__(self, tokens: int, n: int, k: int, rank: int, adapters: int, device="cuda"):
        size = low_rank_workspace_size(tokens, n, k, rank, adapters)
        if size == 0:
            raise ValueError(f"no adapters of rank {rank} for {tokens} x {n} x {k}")
        self.n, self.k, self.rank, self.adapters = n, k, rank, adapters
        self.a = torch.zeros(adapters, rank, k, dtype=torch.bfloat16, device=device)
        self.b = torch.zeros(adapters, n, rank, dtype=torch.bfloat16, device=device)
        self.scales = torch.ones(adapters, dtype=torch.float32, device=device)
        self.rows = self.taken = ExpertRows(tokens, 1, adapters, device)  # taken: the plan of the last add
        self.ws = _workspace(size, device)

    def load(self, index: int, a, b, scale: float = 1.0, stream=None):
        """Adapter ``index``: a (r, k) and b (n, r), r at most the rank; their
        values alone, autograd records nothing."""
        r = a.shape[0]
        if r > self.rank or tuple(a.shape) != (r, self.k) or tuple(b.shape) != (self.n, r):
            raise ValueError(f"a is {tuple(a.shape)} and b {tuple(b.shape)}, the adapters' are of rank {self.rank} for "
                             f"{self.n} x {self.k}")
        with torch.no_grad(), torch.cuda.stream(stream):
            self.a[index].zero_()
            self.b[index].zero_()
            self.a[index, :r] = a
            self.b[index, :, :r] = b
            self.scales[index] = scale

    def plan(self, ids, stream=None):
        """ids (tokens,) int32 or int64: each row's adapter, -1 for none."""
        self.rows.sort(ids.view(-1, 1), stream)

    def add(self, x, y, base=None, plan: "LowRankAdapters | None" = None, stream=None):
        """y = base + the adapters' part; base may be y, or None for zeros."""
        rows = (self if plan is None else plan).rows
        low_rank_add(x, self.a, self.b, rows.offsets, y, self.ws, base, rows.order, self.scales, stream)
        self.taken = rows

    def error(self, stream=None) -> int:
        """Status of the last ``plan`` (CIERA_ERR_ARG for a number of no
        adapter), of the plan that the last ``add`` took, and of that ``add``;
        synchronises."""
        taken = 0 if self.taken is self.rows else self.taken.error(stream)
        return self.rows.error(stream) or taken or ciera_read_error(self.ws, stream)


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
