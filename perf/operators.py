"""Microscaled matrices: what is measured of them, and their plain forms.

A microscaled matrix holds a BF16 matrix in 8 bits (mx8: e4m3 values) or 4
bits (mx4: e2m1 values) per value, with one power-of-two scale byte per 32
consecutive values of a row.  The operators:

  checkpoint   mx8_encode + mx8_decode: activations kept in 8 bits
  weights      mx4_encode + mx4_decode: weights in 4 bits
  matmul       y = x W^T with W in mx4, x in BF16 or an mx8 checkpoint
  dx           dx = dy W, the gradient of x, from the same 4-bit W
  wgrad        dW = dy^T x, the gradient of W, from the 8-bit checkpoint of x

The products take the experts of a mixture-of-experts layer in one call: rows
offsets[g] .. offsets[g+1] - 1 of x, y, dy and dx belong to expert g, whose
weights are rows g N .. (g+1) N - 1 of W.  Rows behind the last expert's are
not read and stay as they were.

Format of a rows x cols matrix, one buffer of bytes: Kp is cols rounded up to
128; first the values, row by row (mx8: Kp bytes a row; mx4: Kp / 2, value 2j
in the low and 2j + 1 in the high half of byte j), zero-filled up to a
multiple of 128 bytes; then one scale byte per block of 32 values, Kp / 32 a
row.  Scale byte b stands for 2^(b - 127): the smallest for which no value of
the block exceeds the largest that e4m3 (448) or e2m1 (6) holds, at least
2^-126.  Values are rounded to nearest, ties to even.  A block with an
infinity or a NaN gets scale byte 255 and values 0, and stands for NaN.
Columns cols .. Kp - 1 are zeros.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
TOP = {"mx8": 448.0, "mx4": 6.0}
E4M3 = [(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127] + [math.nan]
E4M3 += [-v for v in E4M3]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 += [-v for v in E2M1]


# ---------------------------------------------------------------- the format

def _pitch(cols):
    return -(-cols // 128) * 128


def _sections(kind, rows, cols):
    """Bytes of a row of values, where the scales start, and the whole size."""
    kp = _pitch(cols)
    line = kp if kind == "mx8" else kp // 2
    at = -(-rows * line // 128) * 128
    return line, at, at + rows * (kp // BLOCK)


def _power(e):
    """2^e in float32 for a whole-number tensor e in -126 .. 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(kind, x):
    rows, cols = x.shape
    kp = _pitch(cols)
    v = torch.zeros(rows, kp, dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, kp // BLOCK, BLOCK)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(amax)
    m, p = torch.frexp(torch.where(bad, torch.ones_like(amax), amax))
    mt, pt = math.frexp(TOP[kind])
    e = p - pt + (m > mt).to(p.dtype)
    e = torch.where(amax < 2.0 ** -126, torch.full_like(e, -126), e).clamp(min=-126)
    t = torch.where(bad[:, :, None], torch.zeros_like(v), v * _power(-e)[:, :, None])
    if kind == "mx8":
        g = (torch.frexp(t)[1] - 4).clamp(min=-9)  # four significant digits, or the grid of the subnormals
        g = torch.where(t == 0, torch.full_like(g, -9), g)
        q = 8 * (g + 9) + torch.round(t / _power(g)).abs().to(torch.int32)
        q = (q + 128 * torch.signbit(t)).to(torch.uint8).view(rows, kp)
    else:
        a = t.abs()
        q = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
        q = (q + 8 * torch.signbit(t)).view(rows, kp)
        q = q[:, 0::2] | (q[:, 1::2] << 4)
    line, at, size = _sections(kind, rows, cols)
    out = torch.zeros(size, dtype=torch.uint8, device=x.device)
    out[:rows * line] = q.reshape(-1)
    out[at:] = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8).reshape(-1)
    return out


def _decode(kind, buf, rows, cols):
    """The values as float32 (rows, cols)."""
    line, at, size = _sections(kind, rows, cols)
    kp = _pitch(cols)
    q = buf[:rows * line].view(rows, line)
    if kind == "mx8":
        v = torch.tensor(E4M3, device=buf.device)[q.int()]
    else:
        grid = torch.tensor(E2M1, device=buf.device)
        v = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), 2)
    b = buf[at:size].view(rows, kp // BLOCK).to(torch.int32)
    s = torch.where(b == 255, torch.full_like(b, -1).to(torch.float32) * math.nan, _power(b.clamp(1, 254) - 127))
    v = v.reshape(rows, kp // BLOCK, BLOCK) * s[:, :, None]
    return v.view(rows, kp)[:, :cols]


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # a decoding step's activations, kept for a few tokens: latency
        {"name": "checkpoint_step", "op": "checkpoint", "rows": 8, "cols": 2048},
        # a layer's activations of a training batch, 16,384 tokens
        {"name": "checkpoint_batch", "op": "checkpoint", "rows": 16384, "cols": 2048},
        # one attention projection
        {"name": "weights_attention", "op": "weights", "rows": 2048, "cols": 2048},
        # the gate matrices of 64 experts
        {"name": "weights_experts", "op": "weights", "rows": 64 * 1024, "cols": 2048},
        # serving: one new token through an attention projection
        {"name": "matmul_token", "op": "matmul", "x": "bf16", "out": "bf16", "rows": 1, "pad": 0, "n": 2048, "k": 2048,
         "groups": 1, "active": 1},
        # serving: a batch of 8 tokens, each sent to 8 of 64 experts
        {"name": "matmul_step_experts", "op": "matmul", "x": "bf16", "out": "bf16", "rows": 64, "pad": 0, "n": 1024,
         "k": 2048, "groups": 64, "active": 42},
        # a prompt of 4,001 tokens through an attention projection
        {"name": "matmul_prompt", "op": "matmul", "x": "bf16", "out": "bf16", "rows": 4001, "pad": 0, "n": 2048, "k": 2048,
         "groups": 1, "active": 1},
        # training, forward: 4,096 tokens sent to 8 of 64 experts each, from the 8-bit checkpoint
        {"name": "matmul_train_experts", "op": "matmul", "x": "mx8", "out": "bf16", "rows": 32768, "pad": 0, "n": 1024,
         "k": 2048, "groups": 64, "active": 64},
        # backward of a short batch over 66 experts of another width, a buffer with room for more rows
        {"name": "dx_short_experts", "op": "dx", "out": "bf16", "rows": 999, "pad": 25, "n": 1408, "k": 2048, "groups": 66,
         "active": 61},
        # training, gradient of the activations
        {"name": "dx_train_experts", "op": "dx", "out": "bf16", "rows": 32768, "pad": 0, "n": 1024, "k": 2048,
         "groups": 64, "active": 64},
        # training, gradient of an attention projection, in 32 bits
        {"name": "wgrad_attention", "op": "wgrad", "out": "f32", "rows": 8191, "pad": 1, "n": 2048, "k": 2048, "groups": 1,
         "active": 1},
        # training, gradients of 64 experts' weights
        {"name": "wgrad_train_experts", "op": "wgrad", "out": "bf16", "rows": 32768, "pad": 0, "n": 1024, "k": 2048,
         "groups": 64, "active": 64},
    ]


MOST_PRODUCT = 32768 * 1024 * 2048
MOST_WEIGHTS = 64 * 1024 * 2048


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["checkpoint", "weights", "matmul", "matmul", "dx", "wgrad"])
    if op in ("checkpoint", "weights"):
        cols = _spread(rng, 17, 8192)
        cols = rng.choice([cols, -(-cols // 32) * 32])
        return {"op": op, "rows": _spread(rng, 1, min(65536, MOST_WEIGHTS // cols)), "cols": cols}
    while True:
        n, k = _spread(rng, 48, 8192), _spread(rng, 48, 8192)
        n, k = rng.choice([n, -(-n // 64) * 64]), rng.choice([k, -(-k // 64) * 64])
        groups = rng.choice([1, 1, _spread(rng, 2, 96)])
        rows = _spread(rng, 1, 32768)
        if rows * n * k <= MOST_PRODUCT and groups * n * k <= MOST_WEIGHTS and rows * max(n, k) <= MOST_WEIGHTS:
            break
    case = {"op": op, "out": rng.choice(["bf16", "bf16", "f32"]), "rows": rows, "pad": rng.choice([0, rng.randrange(1, 40)]),
            "n": n, "k": k, "groups": groups, "active": rng.randint(max(1, min(groups, rows) // 2), min(groups, rows))}
    if op == "matmul":
        case["x"] = rng.choice(["bf16", "mx8"])
    return case


# ---------------------------------------------------------------- the inputs

def _normal(gen, rows, cols, std, loud=0.0):
    """BF16 values around zero; `loud` of the columns are 16 times larger, as a few channels of activations are."""
    x = torch.randn(rows, cols, generator=gen, device="cuda") * std
    if loud:
        x[:, torch.rand(cols, generator=gen, device="cuda") < loud] *= 16
    return x.to(torch.bfloat16)


def _offsets(case, seed):
    """Rows of each expert: `active` of them have some, unevenly."""
    rng = np.random.default_rng([7, seed])
    has = np.sort(rng.permutation(case["groups"])[:case["active"]])
    share = rng.dirichlet(np.full(case["active"], 4.0))
    count = np.zeros(case["groups"], dtype=np.int64)
    count[has] = 1 + rng.multinomial(case["rows"] - case["active"], share)
    return [0] + [int(c) for c in np.cumsum(count)]


def _tensors(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "checkpoint":
        return {"x": _normal(gen, case["rows"], case["cols"], 1.0, 0.01)}
    if case["op"] == "weights":
        return {"x": _normal(gen, case["rows"], case["cols"], 0.02)}
    rows, total, n, k = case["rows"], case["rows"] + case["pad"], case["n"], case["k"]
    got = {"offsets": _offsets(case, seed)}
    if case["op"] in ("matmul", "wgrad"):
        got["x"] = _normal(gen, total, k, 1.0, 0.01)
        got["x"][rows:] = math.nan
    if case["op"] in ("dx", "wgrad"):
        got["dy"] = _normal(gen, total, n, 1e-3)
        got["dy"][rows:] = math.nan
    if case["op"] in ("matmul", "dx"):
        got["w"] = _encode("mx4", _normal(gen, case["groups"] * n, k, 0.02))
    if case["op"] == "wgrad" or case.get("x") == "mx8":
        got["xq"] = _encode("mx8", got.pop("x"))
    return got


def prepare(case, seed):
    s = dict(case, **_tensors(case, seed))
    s["bounds"] = s.pop("offsets", None)
    dtype = torch.float32 if case.get("out") == "f32" else torch.bfloat16
    if case["op"] in ("checkpoint", "weights"):
        kind = "mx8" if case["op"] == "checkpoint" else "mx4"
        s["kind"], s["y"] = kind, torch.empty_like(s["x"])
        s["buf"] = torch.empty(_sections(kind, case["rows"], case["cols"])[2], dtype=torch.uint8, device="cuda")
    else:
        total, n, k, g = case["rows"] + case["pad"], case["n"], case["k"], case["groups"]
        shape = {"matmul": (total, n), "dx": (total, k), "wgrad": (g, n, k)}[case["op"]]
        s["y"] = torch.zeros(shape, dtype=dtype, device="cuda")
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int64, device="cuda")
        if own:
            import lossless_bf16_tensor_exp_amd as ciera
            s["ws"] = torch.empty(ciera.mx_workspace_size(total, n, k, g), dtype=torch.uint8, device="cuda")
    if own:
        import lossless_bf16_tensor_exp_amd as ciera
        s["lib"] = ciera
    return s


# ------------------------------------------------------------------ the pass

def _run_own(s):
    lib, op = s["lib"], s["op"]
    if op == "checkpoint":
        lib.mx8_encode(s["x"], s["buf"])
        lib.mx8_decode(s["buf"], s["y"])
    elif op == "weights":
        lib.mx4_encode(s["x"], s["buf"])
        lib.mx4_decode(s["buf"], s["y"])
    elif op == "matmul" and "xq" in s:
        lib.mx4_matmul_mx8(s["xq"], s["k"], s["w"], s["y"], s["ws"], s["offsets"])
    elif op == "matmul":
        lib.mx4_matmul(s["x"], s["w"], s["y"], s["ws"], s["offsets"])
    elif op == "dx":
        lib.mx4_matmul_dx(s["dy"], s["w"], s["y"], s["ws"], s["offsets"])
    else:
        lib.mx8_wgrad(s["dy"], s["xq"], s["y"], s["ws"], s["offsets"])
    return s["y"]


def run(s):
    if own:
        return _run_own(s)
    op, y = s["op"], s["y"]
    if op in ("checkpoint", "weights"):
        s["buf"].copy_(_encode(s["kind"], s["x"]))
        y.copy_(_decode(s["kind"], s["buf"], s["rows"], s["cols"]))
        return y
    total, n, k, groups = s["rows"] + s["pad"], s["n"], s["k"], s["groups"]
    if op in ("matmul", "dx"):
        w = _decode("mx4", s["w"], groups * n, k).view(groups, n, k)
    if "xq" in s:
        x = _decode("mx8", s["xq"], total, k)
    elif op == "matmul":
        x = s["x"].float()
    if "dy" in s:
        dy = s["dy"].float()
    for g in range(groups):
        a, b = s["bounds"][g], s["bounds"][g + 1]
        if op == "wgrad":
            y[g] = dy[a:b].t() @ x[a:b]
        elif a < b and op == "matmul":
            y[a:b] = x[a:b] @ w[g].t()
        elif a < b:
            y[a:b] = dy[a:b] @ w[g]
    return y


# ------------------------------------------------------------------ the work

def work(case):
    """Inputs and outputs once; of the weights, those of the experts that have rows."""
    def size(kind, rows, cols):
        return _sections(kind, rows, cols)[2]

    if case["op"] in ("checkpoint", "weights"):
        # the encoded form is the encode's output and the decode's input
        kind = "mx8" if case["op"] == "checkpoint" else "mx4"
        values = case["rows"] * case["cols"]
        return {"bytes": 2 * values + 2 * size(kind, case["rows"], case["cols"]) + 2 * values, "flops": 4 * values}
    rows, n, k = case["rows"], case["n"], case["k"]
    ob = 4 if case["out"] == "f32" else 2
    w = size("mx4", case["active"] * n, k)
    if case["op"] == "matmul":
        moved = (size("mx8", rows, k) if case["x"] == "mx8" else 2 * rows * k) + w + ob * rows * n
    elif case["op"] == "dx":
        moved = 2 * rows * n + w + ob * rows * k
    else:
        moved = 2 * rows * n + size("mx8", rows, k) + ob * case["groups"] * n * k
    return {"bytes": moved, "flops": 2 * rows * n * k}


# ------------------------------------------------------- 64 bits, from the definition

def _power64(e):
    """2^e in float64 for whole numbers e in -1022 .. 1023."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(t, digits, least):
    """t (float64) rounded to `digits` significant binary digits, ties to even, the grid no finer than 2^least."""
    _, p = torch.frexp(t)
    step = _power64((p - digits).clamp(min=least))
    return torch.round(t / step) * step


def _stands_for(kind, x):
    """What the encoded x stands for, in float64."""
    rows, cols = x.shape
    fill = -cols % BLOCK
    v = torch.nn.functional.pad(x.double(), (0, fill)).view(rows, -1, BLOCK)
    amax = v.abs().amax(2, keepdim=True)
    scale = torch.full_like(amax, 2.0 ** -126)
    e = torch.ceil(torch.log2(torch.nan_to_num(amax, 1.0, 1.0).clamp(min=2.0 ** -140) / TOP[kind])).clamp(min=-126)
    for step in (-1, 0, 1):  # the logarithm may be off by one next to a border: the smallest that holds
        c = _power64((e - step).clamp(min=-126))
        scale = torch.where(amax <= TOP[kind] * c, c, scale)
    digits, least = (4, -9) if kind == "mx8" else (2, -1)
    out = _nearest(v / scale, digits, least) * scale
    out = torch.where(torch.isfinite(amax), out, torch.full_like(out, math.nan))
    return out.view(rows, cols + fill)[:, :cols]


def exact(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("checkpoint", "weights"):
        if case["op"] == "checkpoint":
            return _stands_for("mx8", _normal(gen, case["rows"], case["cols"], 1.0, 0.01))
        return _stands_for("mx4", _normal(gen, case["rows"], case["cols"], 0.02))
    rows, total, n, k, groups = case["rows"], case["rows"] + case["pad"], case["n"], case["k"], case["groups"]
    bounds = _offsets(case, seed)
    x = dy = w = None
    if case["op"] in ("matmul", "wgrad"):
        x = _normal(gen, total, k, 1.0, 0.01)
        x = _stands_for("mx8", x) if case["op"] == "wgrad" or case["x"] == "mx8" else x.double()
    if case["op"] in ("dx", "wgrad"):
        dy = _normal(gen, total, n, 1e-3).double()
    if case["op"] in ("matmul", "dx"):
        w = _stands_for("mx4", _normal(gen, groups * n, k, 0.02)).view(groups, n, k)
    shape = {"matmul": (total, n), "dx": (total, k), "wgrad": (groups, n, k)}[case["op"]]
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for g in range(groups):
        a, b = bounds[g], bounds[g + 1]
        if a == b:
            continue
        if case["op"] == "wgrad":
            out[g] = dy[a:b].t().contiguous() @ x[a:b]
        elif case["op"] == "matmul":
            out[a:b] = x[a:b] @ w[g].t().contiguous()
        else:
            out[a:b] = dy[a:b] @ w[g]
    return out
