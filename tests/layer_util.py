"""What stands around a layer's products, plainly, in 64 bits on the CPU, and
the inputs of its tests."""
import torch

import mx_util as mx

bf16 = torch.bfloat16
GUARD = 64


def guarded(rows, cols, dtype, wider=0, shift=0, fill=7.0):
    """A matrix on the GPU with rows cols + wider values apart, the first `shift` (and GUARD) values into its buffer."""
    ld = cols + wider
    buf = torch.full((2 * GUARD + shift + rows * ld,), fill, dtype=dtype, device="cuda")
    view = buf[GUARD + shift:GUARD + shift + rows * ld].view(rows, ld)[:, :cols]
    return buf, view


def put(t, wider=0, shift=0):
    """t on the GPU at a stride and alignment of its own, NaN between its rows."""
    buf, view = guarded(*t.shape, t.dtype, wider, shift, float("nan"))
    view.copy_(t)
    return view


def untouched(buf, view, fill=7.0):
    """Nothing outside the matrix was written."""
    keep = view.clone()
    view.fill_(fill)
    ok = bool((buf == fill).all())
    view.copy_(keep)
    assert ok, "a value outside the matrix was written"


def within(got, want, room, half_step=0.0):
    """|got - want| within room, and half a step of the output's type; NaN and infinities in the same places."""
    got, want = got.double().cpu(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.nan_to_num(got[~fine], 1e300, 5e300, -5e300), torch.nan_to_num(want[~fine], 1e300, 5e300, -5e300))
    room = (room + half_step * (want.abs() + room) + (2.0 ** -134 if half_step > 2.0 ** -20 else 2.0 ** -149)).expand_as(want)
    off = (got - want).abs()[fine] - room[fine]
    assert off.numel() == 0 or (off <= 0).all(), f"off by up to {off.max().item():.3e} more than the bound"


HALF = {bf16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def sort(ids, experts):
    """offsets, place, order of a table of expert numbers (any not in 0 .. experts - 1: none)."""
    flat = ids.reshape(-1).tolist()
    by = [[] for _ in range(experts + 1)]
    for i, e in enumerate(flat):
        by[e if 0 <= e < experts else experts].append(i)
    offsets, order, place = [0], [], [-1] * len(flat)
    for e in range(experts):
        for i in by[e]:
            place[i] = len(order)
            order.append(i)
        offsets.append(len(order))
    order += by[experts]
    return (torch.tensor(offsets), torch.tensor(place, dtype=torch.int32).view(ids.shape),
            torch.tensor(order, dtype=torch.int32))


def choose(gen, tokens, choices, experts, none=0.1):
    """Different experts for each token, a share of the entries without one."""
    ids = torch.rand(tokens, experts, generator=gen).argsort(1)[:, :choices].to(torch.int32)
    ids[torch.rand(tokens, choices, generator=gen) < none] = -1
    return ids.contiguous()


def norm(x, residual, w, eps):
    """h (BF16), s, y in 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(bf16)
    hd = h.double()
    s = (hd.square().mean(1) + eps) ** -0.5
    return h, s, hd * s[:, None] * w.double()


def combine(rows, place, weights, residual):
    """out and the sum of the magnitudes added."""
    tokens, choices = place.shape
    out = torch.zeros(tokens, rows.shape[1], dtype=torch.float64) if residual is None else residual.double()
    size = out.abs()
    for j in range(choices):
        has = place[:, j] >= 0
        r = rows.double()[place[:, j][has].long()]
        w = torch.ones(int(has.sum()), 1, dtype=torch.float64) if weights is None else weights[has, j].double()[:, None]
        out[has] += w * r
        size[has] += (w * r).abs()
    return out, size


def low_rank(x, a, b, scales, offsets, order, base):
    """y, and the sum of the magnitudes of the products behind each value."""
    y = base.double().clone()
    size = torch.zeros_like(y)
    for g in range(a.shape[0]):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if lo == hi:
            continue
        at = torch.arange(lo, hi) if order is None else order[lo:hi].long()
        xd, ad, bd, s = x[at].double(), a[g].double(), b[g].double(), 1.0 if scales is None else float(scales[g])
        y[at] += s * (xd @ ad.T) @ bd.T
        size[at] += abs(s) * (xd.abs() @ ad.abs().T) @ bd.abs().T
    return y, size


__all__ = ["mx", "bf16", "guarded", "put", "untouched", "within", "HALF", "sort", "choose", "norm", "combine", "low_rank"]
