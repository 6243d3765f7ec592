"""What stands around the products of a layer on microscaled matrices: what is
measured of it, and the plain forms.

  norm               h = x + residual;  y = h w / sqrt(mean(h^2) + eps), in
                     BF16, kept in 8 bits (mx8), or both
  norm_backward      the gradients of h and w, with h's own gradient added
  dispatch           entries (token, choice) sorted by expert, and the tokens'
                     rows laid out in that order, in BF16 or mx8
  combine            out = residual + sum over a token's choices of weight * row
  combine_backward   the gradients of the rows and of the weights
  adapters           y = base + s_a B_a (A_a x): low-rank adapters of many
                     requests beside a projection that they share

h is rounded to BF16 and the norm is that of the rounded h; y is rounded to
BF16 and the 8-bit form is made of the rounded y.  Sorting is stable: entries
of one expert keep their order, and those of no expert (-1) come last.
offsets[e] .. offsets[e+1] - 1 are expert e's rows; place holds the row of each
entry, -1 for one of no expert; order the entry of each row.  Rows behind the
last expert's stay as they were.

mx8: 32 consecutive values of a row share the smallest power of two s, at least
2^-126, for which no |v| exceeds 448 s; each is kept as v / s rounded to
nearest e4m3 (four significant bits, the subnormals' step 2^-9), ties to even.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BLOCK = 32
bf16 = torch.bfloat16


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # a decoding step of 8 requests: the norm before a projection whose input is kept in 8 bits
        {"name": "norm_step", "op": "norm", "rows": 8, "cols": 2048, "residual": True, "out": "mx8"},
        # a training batch of 16,384 tokens: BF16 for the router, 8 bits for the products
        {"name": "norm_batch", "op": "norm", "rows": 16384, "cols": 2048, "residual": True, "out": "both"},
        # backward of a short batch at another width, in BF16
        {"name": "norm_backward_short", "op": "norm_backward", "rows": 999, "cols": 1408, "dh": True, "dw": "bf16"},
        # backward of the training batch
        {"name": "norm_backward_batch", "op": "norm_backward", "rows": 16384, "cols": 2048, "dh": True, "dw": "f32"},
        # serving: 8 tokens, each sent to 8 of 64 experts
        {"name": "dispatch_step", "op": "dispatch", "tokens": 8, "padded": 0, "choices": 8, "experts": 64, "cols": 2048,
         "out": "bf16"},
        # training: 4,096 tokens to 8 of 64 experts each, right into the 8-bit checkpoint of the experts' input
        {"name": "dispatch_train", "op": "dispatch", "tokens": 4096, "padded": 0, "choices": 8, "experts": 64, "cols": 2048,
         "out": "mx8"},
        # serving: back from the experts
        {"name": "combine_step", "op": "combine", "tokens": 8, "padded": 0, "choices": 8, "experts": 64, "cols": 2048,
         "rows": "bf16", "out": "bf16", "residual": True},
        # training: back from the experts, onto the residual
        {"name": "combine_train", "op": "combine", "tokens": 4096, "padded": 0, "choices": 8, "experts": 64, "cols": 2048,
         "rows": "bf16", "out": "bf16", "residual": True},
        # backward of a short padded batch, 6 of 66 experts
        {"name": "combine_backward_short", "op": "combine_backward", "tokens": 167, "padded": 25, "choices": 6,
         "experts": 66, "cols": 2048, "rows": "bf16"},
        # training, backward
        {"name": "combine_backward_train", "op": "combine_backward", "tokens": 4096, "padded": 0, "choices": 8,
         "experts": 64, "cols": 2048, "rows": "bf16"},
        # serving: a step of 64 requests, 24 adapters among them, 5 requests without one
        {"name": "adapters_step", "op": "adapters", "tokens": 64, "bare": 5, "n": 2048, "k": 2048, "rank": 16,
         "adapters": 64, "active": 24, "out": "bf16"},
        # prompts of 9 requests, 4,001 tokens in all
        {"name": "adapters_prompts", "op": "adapters", "tokens": 4001, "bare": 300, "n": 2048, "k": 2048, "rank": 64,
         "adapters": 16, "active": 9, "out": "bf16"},
    ]


MOST_NORM = 16384 * 2048
MOST_ROWS = 32768 * 2048
MOST_TOKENS = 4001


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "dispatch", "combine", "combine_backward", "adapters", "adapters"])
    cols = _spread(rng, 17, 8192)
    cols = rng.choice([cols, -(-cols // 32) * 32])
    if op in ("norm", "norm_backward"):
        case = {"op": op, "rows": _spread(rng, 1, min(65536, MOST_NORM // cols)), "cols": cols}
        if op == "norm":
            return dict(case, residual=rng.random() < 0.7, out=rng.choice(["bf16", "mx8", "both"]))
        return dict(case, dh=rng.random() < 0.7, dw=rng.choice(["f32", "bf16"]))
    if op == "adapters":
        tokens, rank, adapters = _spread(rng, 1, MOST_TOKENS), _spread(rng, 1, 128), _spread(rng, 1, 128)
        while True:
            n, k = _spread(rng, 48, 8192), _spread(rng, 48, 8192)
            n, k = rng.choice([n, -(-n // 64) * 64]), rng.choice([k, -(-k // 64) * 64])
            if max(tokens, 1000) * rank * (n + k) <= 4001 * 64 * 4096:
                break
            rank = max(1, rank // 2)
        bare = rng.choice([0, 0, rng.randrange(0, tokens + 1)])
        return {"op": op, "tokens": tokens, "bare": bare, "n": n, "k": k, "rank": rank, "adapters": adapters,
                "active": min(tokens - bare, rng.randint(1, adapters)), "out": rng.choice(["bf16", "f32"])}
    choices = rng.randint(1, 8)
    tokens = _spread(rng, 1, min(32768, MOST_ROWS // (choices * cols)))
    case = {"op": op, "tokens": tokens, "padded": rng.choice([0, rng.randrange(0, min(tokens, 40))]), "choices": choices,
            "experts": max(choices, _spread(rng, 1, 256)), "cols": cols}
    if op == "dispatch":
        return dict(case, out=rng.choice(["bf16", "mx8"]))
    wide = tokens * choices * cols <= MOST_ROWS // 2  # rows in 32 bits move twice the bytes
    case["rows"] = rng.choice(["bf16", "f32"]) if wide else "bf16"
    if op == "combine":
        case.update(out=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.6)
    return case


# ---------------------------------------------------------------- the inputs

def _normal(gen, rows, cols, std, loud=0.0, dtype=bf16):
    """Values around zero; `loud` of the columns are 16 times larger, as a few channels of activations are."""
    x = torch.randn(rows, cols, generator=gen, device="cuda") * std
    if loud:
        x[:, torch.rand(cols, generator=gen, device="cuda") < loud] *= 16
    return x.to(dtype)


def _choices(gen, case):
    """Each token's experts, some of them more in demand than others, by falling score, and the weights of their
    scores; tokens behind the last real one have none."""
    tokens, experts, c = case["tokens"], case["experts"], case["choices"]
    score = torch.randn(tokens, experts, generator=gen, device="cuda")
    score += 0.7 * torch.randn(experts, generator=gen, device="cuda")
    top, ids = torch.sort(score, 1, descending=True)
    ids, weights = ids[:, :c].to(torch.int32).contiguous(), torch.softmax(top[:, :c], 1).contiguous()
    ids[tokens - case["padded"]:] = -1
    return ids, weights


def _wants(gen, case):
    """Each request's adapter: `active` of them are wanted, each at least once; -1 for none."""
    t, a, bare = case["tokens"], case["active"], case["bare"]
    which = torch.randperm(case["adapters"], generator=gen, device="cuda")[:a]
    ids = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    if a:
        many = torch.randint(0, a, (t - bare,), generator=gen, device="cuda")
        many[:a] = torch.arange(a, device="cuda")
        ids[:t - bare] = which[many]
    return ids[torch.randperm(t, generator=gen, device="cuda")].to(torch.int32)


def _sorted(ids, groups):
    """offsets, place and order of the entries `ids`."""
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where(flat < 0, torch.full_like(flat, groups), flat)
    order = torch.sort(key, stable=True)[1]
    count = torch.zeros(groups + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat((torch.zeros_like(count[:1]), torch.cumsum(count, 0)[:groups]))
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=ids.device)
    place = torch.where(flat < 0, torch.full_like(place, -1), place)
    return offsets, place.to(torch.int32).view(ids.shape), order.to(torch.int32)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {}
    if op in ("norm", "norm_backward"):
        rows, cols = case["rows"], case["cols"]
        s["w"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(bf16)
        if op == "norm":
            s["x"] = _normal(gen, rows, cols, 0.5)
            if case["residual"]:
                s["residual"] = _normal(gen, rows, cols, 1.0, 0.01)
        else:
            s["hidden"] = _normal(gen, rows, cols, 1.0, 0.01)
            s["rstd"] = torch.rsqrt(s["hidden"].double().square().mean(1) + EPS).float()  # as the forward pass keeps it
            s["dy"] = _normal(gen, rows, cols, 1e-3)
            if case["dh"]:
                s["dh"] = _normal(gen, rows, cols, 1e-3)
    elif op == "adapters":
        t, n, k, r, a = (case[m] for m in ("tokens", "n", "k", "rank", "adapters"))
        s["x"] = _normal(gen, t, k, 1.0, 0.01)
        s["a"] = _normal(gen, a * r, k, k ** -0.5).view(a, r, k)
        s["b"] = _normal(gen, a * n, r, 0.2 * r ** -0.5).view(a, n, r)
        s["scales"] = torch.rand(a, generator=gen, device="cuda") * 2
        s["base"] = _normal(gen, t, n, 1.0, dtype=bf16 if case["out"] == "bf16" else torch.float32)
        s["ids"] = _wants(gen, case)
    else:
        t, cols = case["tokens"], case["cols"]
        s["ids"], s["weights"] = _choices(gen, case)
        if op == "dispatch":
            s["x"] = _normal(gen, t, cols, 1.0, 0.01)
        else:
            rows = t * case["choices"]
            s["rows"] = _normal(gen, rows, cols, 0.5, dtype=bf16 if case["rows"] == "bf16" else torch.float32)
            if op == "combine" and case["residual"]:
                s["residual"] = _normal(gen, t, cols, 1.0, 0.01)
            if op == "combine_backward":
                s["dout"] = _normal(gen, t, cols, 1e-3)
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    op = case["op"]
    if op == "adapters":  # sorted once for all projections of a step
        s["offsets"], _, s["order"] = _sorted(s["ids"], case["adapters"])
        s["bounds"] = s["offsets"].tolist()
    elif op.startswith("combine"):  # the dispatch's
        s["place"] = _sorted(s["ids"], case["experts"])[1]
    if op == "dispatch":
        s["out"] = torch.zeros(case["tokens"] * case["choices"], case["cols"], dtype=bf16, device="cuda")
    if op == "combine_backward":
        s["drows"] = torch.zeros_like(s["rows"], dtype=bf16)
    if own:
        _own_buffers(s)
    return s


def _own_buffers(s):
    import lossless_bf16_tensor_exp_amd as ciera
    s["lib"], case, op = ciera, s["case"], s["case"]["op"]

    def new(*shape, dtype=bf16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def kept(rows):  # zeros: rows of no expert are not written
        return torch.zeros(ciera.mx8_encoded_size(rows, case["cols"]), dtype=torch.uint8, device="cuda")

    if op == "norm":
        shape = (case["rows"], case["cols"])
        s["h"] = new(*shape) if case["residual"] else None
        s["y"] = new(*shape) if case["out"] != "mx8" else None
        s["yq"], s["kept"] = (kept(case["rows"]), new(*shape)) if case["out"] != "bf16" else (None, None)
        s["rstd"] = new(case["rows"], dtype=torch.float32)
    elif op == "norm_backward":
        s["dx"] = new(case["rows"], case["cols"])
        s["dw"] = new(case["cols"], dtype=bf16 if case["dw"] == "bf16" else torch.float32)
        s["ws"] = new(ciera.rms_norm_workspace_size(case["rows"], case["cols"]), dtype=torch.uint8)
    elif op == "dispatch":
        s["offsets"] = new(case["experts"] + 1, dtype=torch.int64)
        s["place"] = torch.empty_like(s["ids"])
        s["order"] = new(s["ids"].numel(), dtype=torch.int32)
        s["ws"] = new(ciera.expert_workspace_size(case["tokens"], case["choices"], case["experts"]), dtype=torch.uint8)
        if case["out"] == "mx8":
            s["outq"] = kept(s["out"].shape[0])
    elif op == "combine":
        s["y"] = new(case["tokens"], case["cols"], dtype=bf16 if case["out"] == "bf16" else torch.float32)
    elif op == "combine_backward":
        s["dweights"] = torch.empty_like(s["weights"])
    else:
        s["y"] = torch.empty_like(s["base"])
        s["ws"] = new(ciera.low_rank_workspace_size(case["tokens"], case["n"], case["k"], case["rank"], case["adapters"]),
                      dtype=torch.uint8)


# ------------------------------------------------------------------ the pass

def _run_own(s):
    lib, case, op = s["lib"], s["case"], s["case"]["op"]
    if op == "norm":
        lib.rms_norm(s["x"], s["w"], y=s["y"], yq=s["yq"], residual=s.get("residual"), h=s["h"], rstd=s["rstd"], eps=EPS)
        if s["yq"] is not None:
            lib.mx8_decode(s["yq"], s["kept"])
        return [s["h"], s["y"], s["kept"], s["rstd"]]
    if op == "norm_backward":
        lib.rms_norm_backward(s["dy"], s["hidden"], s["w"], s["rstd"], s["dx"], s["dw"], s["ws"], dh=s.get("dh"))
        return [s["dx"], s["dw"]]
    if op == "dispatch":
        lib.expert_sort(s["ids"], s["offsets"], s["place"], s["order"], s["ws"])
        if case["out"] == "mx8":
            lib.expert_dispatch(s["x"], s["place"], outq=s["outq"])
            lib.mx8_decode(s["outq"], s["out"])
        else:
            lib.expert_dispatch(s["x"], s["place"], out=s["out"])
        return [s["offsets"], s["place"], s["order"], s["out"]]
    if op == "combine":
        lib.expert_combine(s["rows"], s["place"], s["y"], weights=s["weights"], residual=s.get("residual"))
        return s["y"]
    if op == "combine_backward":
        lib.expert_combine_backward(s["dout"], s["rows"], s["place"], s["drows"], s["dweights"], weights=s["weights"])
        return [s["drows"], s["dweights"]]
    lib.low_rank_add(s["x"], s["a"], s["b"], s["offsets"], s["y"], s["ws"], base=s["base"], order=s["order"],
                     scales=s["scales"])
    return s["y"]


def _power(e):
    """2^e in float32 for a whole-number tensor e in -126 .. 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _in_8_bits(y):
    """What the mx8 form of the BF16 matrix y stands for, in BF16."""
    rows, cols = y.shape
    v = torch.nn.functional.pad(y.float(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    m, p = torch.frexp(v.abs().amax(2, keepdim=True))
    s = _power((p - 9 + (m > 0.875)).clamp(min=-126))  # 448 = 0.875 * 2^9
    t = v / s
    step = _power((torch.frexp(t)[1] - 4).clamp(min=-9))
    return (torch.round(t / step) * step * s).view(rows, -1)[:, :cols].to(bf16)


def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        h = (s["x"].float() + s["residual"].float()).to(bf16) if case["residual"] else s["x"]
        rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
        y = (h.float() * rstd[:, None] * s["w"].float()).to(bf16)
        return [h if case["residual"] else None, y if case["out"] != "mx8" else None,
                _in_8_bits(y) if case["out"] != "bf16" else None, rstd]
    if op == "norm_backward":
        h, rstd, dy = s["hidden"].float(), s["rstd"][:, None], s["dy"].float()
        g = dy * s["w"].float()
        dx = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
        if case["dh"]:
            dx = dx + s["dh"].float()
        dw = (dy * h * rstd).sum(0)
        return [dx.to(bf16), dw.to(bf16) if case["dw"] == "bf16" else dw]
    if op == "dispatch":
        offsets, place, order = _sorted(s["ids"], case["experts"])
        has = place.reshape(-1) >= 0
        at, token = place.reshape(-1)[has].long(), torch.arange(has.numel(), device="cuda")[has] // case["choices"]
        x = _in_8_bits(s["x"]) if case["out"] == "mx8" else s["x"]
        s["out"][at] = x[token]
        return [offsets, place, order, s["out"]]
    if op == "adapters":
        order, base, x = s["order"].long(), s["base"].float(), s["x"].float()
        y = base.clone()
        for a in range(case["adapters"]):
            lo, hi = s["bounds"][a], s["bounds"][a + 1]
            if lo < hi:
                at = order[lo:hi]
                y[at] += s["scales"][a] * ((x[at] @ s["a"][a].float().t()) @ s["b"][a].float().t())
        return y.to(s["base"].dtype)
    place, has = s["place"].long(), s["place"] >= 0
    rows, w = s["rows"].float(), torch.where(has, s["weights"], torch.zeros_like(s["weights"]))
    if op == "combine":
        # a token's choices one after the other; one without expert adds nothing
        y = s["residual"].float() if case["residual"] else torch.zeros(case["tokens"], case["cols"], device="cuda")
        for j in range(case["choices"]):
            y = y + torch.where(has[:, j:j + 1], w[:, j:j + 1] * rows[place[:, j].clamp(min=0)], torch.zeros_like(y))
        return y.to(bf16) if case["out"] == "bf16" else y
    dout, dw = s["dout"].float(), torch.zeros_like(w)
    for j in range(case["choices"]):
        at, token = place[:, j][has[:, j]], torch.nonzero(has[:, j]).view(-1)
        s["drows"][at] = (w[token, j][:, None] * dout[token]).to(bf16)
        dw[token, j] = (dout[token] * rows[at]).sum(1)
    return [s["drows"], dw]


# ------------------------------------------------------------------ the work

def _kept_size(rows, cols):
    kp = -(-cols // 128) * 128
    return rows * kp + rows * (kp // BLOCK)


def work(case):
    """Inputs and outputs once; of the adapters, those that have requests.  What is kept in 8 bits is written, and read
    and written as values once more."""
    op = case["op"]
    if op == "norm":
        v = case["rows"] * case["cols"]
        kept = 2 * _kept_size(case["rows"], case["cols"]) + 2 * v if case["out"] != "bf16" else 0
        moved = 2 * v + (4 * v if case["residual"] else 0) + (2 * v if case["out"] != "mx8" else 0) + kept
        return {"bytes": moved + 4 * case["rows"] + 2 * case["cols"], "flops": 6 * v}
    if op == "norm_backward":
        v = case["rows"] * case["cols"]
        return {"bytes": (8 if case["dh"] else 6) * v + 4 * case["rows"] + 6 * case["cols"], "flops": 12 * v}
    if op == "adapters":
        t, n, k, r = case["tokens"], case["n"], case["k"], case["rank"]
        live, ob = t - case["bare"], 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * live * k + 2 * ob * t * n + 2 * case["active"] * r * (n + k) + 4 * t,
                "flops": 2 * live * r * (n + k) + live * n}
    entries = case["tokens"] * case["choices"]
    live = entries - case["padded"] * case["choices"]
    t, c = case["tokens"] - case["padded"], case["cols"]
    if op == "dispatch":
        out = 2 * _kept_size(live, c) + 2 * live * c if case["out"] == "mx8" else 2 * live * c
        return {"bytes": 12 * entries + 8 * (case["experts"] + 1) + 2 * t * c + out, "flops": 2 * t * c}
    rb = 2 if case["rows"] == "bf16" else 4
    if op == "combine":
        ob = 2 if case["out"] == "bf16" else 4
        return {"bytes": 8 * entries + rb * live * c + ((2 if case["residual"] else 0) + ob) * case["tokens"] * c,
                "flops": 2 * live * c}
    return {"bytes": 12 * entries + rb * live * c + 2 * t * c + 2 * live * c, "flops": 3 * live * c}


# ------------------------------------------------------- 64 bits, from the definition

def _power64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _rounded(t, digits, least):
    """t (float64) to `digits` significant binary digits, ties to even, the grid no finer than 2^least."""
    step = _power64((torch.frexp(t)[1] - digits).clamp(min=least))
    return torch.round(t / step) * step


def _bf16_64(t):
    return _rounded(t, 8, -133)


def _kept_64(y):
    """The mx8 form of y (float64 holding BF16 values), block by block."""
    rows, cols = y.shape
    v = torch.nn.functional.pad(y, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    top = v.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).clamp(min=-126)
    s = torch.full_like(top, 2.0 ** -126)
    for step in (-1, 0, 1):  # the logarithm may be off by one next to a border: the smallest that holds
        c = _power64((e - step).clamp(min=-126))
        s = torch.where(top <= 448.0 * c, c, s)
    return (_rounded(v / s, 4, -9) * s).view(rows, -1)[:, :cols]


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    d = {m: v.double() for m, v in s.items() if v.is_floating_point()}
    if op == "norm":
        h = _bf16_64(d["x"] + d["residual"]) if case["residual"] else d["x"]
        rstd = (h.pow(2).sum(1) / case["cols"] + EPS) ** -0.5
        y = h * rstd[:, None] * d["w"]
        return [h if case["residual"] else None, y if case["out"] != "mx8" else None,
                _kept_64(_bf16_64(y)) if case["out"] != "bf16" else None, rstd]
    if op == "norm_backward":
        unit = d["hidden"] * d["rstd"][:, None]  # d y / d h = rstd (w - unit (unit w)' / cols)
        g = d["dy"] * d["w"]
        dx = d["rstd"][:, None] * (g - unit * ((g * unit).sum(1, keepdim=True) / case["cols"])) + d.get("dh", 0.0)
        return [dx, (d["dy"] * unit).sum(0)]
    if op == "adapters":
        # every adapter's inner values, those of the row's own adapter kept
        t, r, groups = case["tokens"], case["rank"], case["adapters"]
        y, ids = d["base"].clone(), s["ids"].long()
        for a in ids.unique().tolist():
            if a >= 0:
                at = (ids == a).nonzero().view(-1)
                y[at] += d["scales"][a] * torch.mm(torch.mm(d["x"][at], d["a"][a].t().contiguous()),
                                                   d["b"][a].t().contiguous())
        return y
    # where each entry goes, from counts
    flat = s["ids"].cpu().numpy().reshape(-1)
    live = np.flatnonzero(flat >= 0)
    at = np.empty(live.size, dtype=np.int64)
    at[np.lexsort((live, flat[live]))] = np.arange(live.size)
    at, entry = torch.from_numpy(at).cuda(), torch.from_numpy(live).cuda()
    token, choices = entry // case["choices"], case["choices"]
    if op == "dispatch":
        out = torch.zeros(flat.size, case["cols"], dtype=torch.float64, device="cuda")
        out[at] = (_kept_64(d["x"]) if case["out"] == "mx8" else d["x"])[token]
        return [None, None, None, out]
    w = d["weights"].view(-1)[entry][:, None]
    if op == "combine":
        out = d["residual"] if case["residual"] else torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        for j in range(choices):  # a token at most once in each step
            of = entry % choices == j
            out = out.index_add(0, token[of], w[of] * d["rows"][at[of]])
        return out
    drows = torch.zeros(flat.size, case["cols"], dtype=torch.float64, device="cuda")
    drows[at] = w * d["dout"][token]
    dweights = torch.zeros(flat.size, dtype=torch.float64, device="cuda")
    dweights[entry] = (d["dout"][token] * d["rows"][at]).sum(1)
    return [drows, dweights.view(-1, choices)]
