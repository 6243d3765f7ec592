"""The microscaled matrices without a GPU: the plain implementation that the
GPU tests compare with (tests/mx_util.py) against the format's definition, the
size queries, and every argument error, which returns before a launch."""
import ctypes
import math
import os

import pytest

import mx_util as mx

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    import lossless_bf16_tensor_exp_amd as ciera
    if not os.path.exists(ciera.library_path()):
        from lossless_bf16_tensor_exp_amd import build
        build.build()
    from lossless_bf16_tensor_exp_amd import mx as calls
    return calls._lib()


@pytest.mark.parametrize("bits", [8, 4])
def test_plain_form_all_bf16_values(bits):
    """Every BF16 value alone in a block: the smallest scale that holds it,
    the nearest code, and a decoded value within half a step."""
    x = torch.arange(-32768, 32768).to(torch.int16).view(torch.bfloat16)
    m = torch.zeros(65536, 32, dtype=torch.bfloat16)
    m[:, 7] = x
    buf = mx.encode(bits, m)
    line, at, size = mx.sections(bits, 65536, 32)
    sb = buf[at:size].view(65536, -1)[:, 0].long()
    finite = torch.isfinite(x)
    assert torch.equal(sb == 255, ~finite)
    a, s = x.double().abs()[finite], torch.ldexp(torch.ones(int(finite.sum()), dtype=torch.float64), sb[finite] - 127)
    assert (a <= mx.TOP[bits] * s).all()
    assert ((a > mx.TOP[bits] * s / 2) | (sb[finite] == 1)).all()
    y = mx.decode(bits, buf, 65536, 32)
    assert torch.isnan(y[~finite]).all()
    grid = torch.tensor(mx.E4M3[:127] if bits == 8 else mx.E2M1[:8], dtype=torch.float64)
    best = ((a / s)[:, None] - grid).abs().amin(1)
    assert torch.equal((y[finite, 7].abs() / s - a / s).abs(), best)
    assert (torch.signbit(y[finite, 7]) == torch.signbit(x[finite])).all()


def test_plain_form_ties_go_to_even():
    m = torch.zeros(1, 32, dtype=torch.bfloat16)
    m[0, :9] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25])
    assert mx.decode(4, mx.encode(4, m), 1, 32)[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.0]
    m[0, :5] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])
    assert mx.decode(8, mx.encode(8, m), 1, 32)[0, :5].tolist() == [448, 16, 20, 0, 2.0 ** -8]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,cols", [(0, 5), (1, 1), (3, 31), (7, 33), (5, 128), (2, 129), (1000, 1408)])
def test_encoded_sizes(lib, bits, rows, cols):
    f = lib.mx8_encoded_size if bits == 8 else lib.mx4_encoded_size
    assert f(rows, cols) == mx.sections(bits, rows, cols)[2]


def test_size_limits(lib):
    assert lib.mx8_encoded_size((1 << 31) + 1, 1) == 0 and lib.mx4_encoded_size(1, (1 << 21) + 1) == 0
    assert lib.mx8_encoded_size(1 << 31, 1 << 21) == (1 << 52) + (1 << 47)
    assert lib.mx_workspace_size(0, 1, 1, 1) >= 512
    for bad in [(1 << 31, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, 4097), (1, (1 << 21) + 1, 1, 1),
                (1, 1, (1 << 21) + 1, 1), (1, 1 << 20, 1, 4096)]:
        assert lib.mx_workspace_size(*bad) == 0, bad


def test_argument_errors_return_before_any_launch(lib):
    p, odd, mis = ctypes.c_void_p(1 << 16), ctypes.c_void_p((1 << 16) + 1), ctypes.c_void_p((1 << 16) + 8)
    big = 1 << 40
    for enc, dec in ((lib.mx8_encode, lib.mx8_decode), (lib.mx4_encode, lib.mx4_decode)):
        assert enc(None, 4, 40, 40, p, big, None) == 1
        assert enc(odd, 4, 40, 40, p, big, None) == 1
        assert enc(p, 4, 40, 40, None, big, None) == 1
        assert enc(p, 4, 40, 40, mis, big, None) == 1
        assert enc(p, 4, 40, 39, p, big, None) == 1
        assert enc(p, 4, 40, (1 << 22) + 1, p, big, None) == 1
        assert enc(p, (1 << 31) + 1, 40, 40, p, 1 << 60, None) == 1
        assert enc(p, 4, (1 << 21) + 1, (1 << 21) + 1, p, big, None) == 1
        assert enc(p, 4, 40, 40, p, 100, None) == 2
        assert enc(None, 0, 40, 40, None, 0, None) == 0
        assert enc(None, 4, 0, 0, None, 0, None) == 0
        assert dec(p, big, 4, 40, None, 40, None) == 1
        assert dec(mis, big, 4, 40, p, 40, None) == 1
        assert dec(p, big, 4, 40, p, 39, None) == 1
        assert dec(p, 100, 4, 40, p, 40, None) == 5
        assert dec(None, 0, 0, 40, None, 40, None) == 0
    # (x, ldx, w, w_bytes, y, ldy, f32, tokens, n, k, groups, offsets, ws, ws_bytes, stream)
    good = dict(x=p, ldx=64, w=p, wb=big, y=p, ldy=48, f32=0, t=8, n=48, k=64, g=1, off=None, ws=p, wsb=big)

    def matmul(f, **kw):
        a = dict(good, **kw)
        return f(a["x"], a["ldx"], a["w"], a["wb"], a["y"], a["ldy"], a["f32"], a["t"], a["n"], a["k"], a["g"], a["off"],
                 a["ws"], a["wsb"], None)

    for f in (lib.mx4_matmul, lib.mx4_matmul_mx8, lib.mx4_matmul_dx):
        wide = dict(ldy=64) if f is lib.mx4_matmul_dx else {}
        if f is lib.mx4_matmul_mx8:
            wide["ldx"] = big
        for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None), dict(w=mis), dict(ws=mis), dict(y=odd),
                   dict(f32=2), dict(f32=1, y=ctypes.c_void_p((1 << 16) + 2)), dict(n=0), dict(k=0), dict(g=0),
                   dict(g=2), dict(g=4097, off=p), dict(g=2, off=ctypes.c_void_p((1 << 16) + 4)), dict(t=1 << 31),
                   dict(ldy=47), dict(off=odd)):
            assert matmul(f, **dict(wide, **kw)) == 1, (f.__name__, kw)
        if f is not lib.mx4_matmul_mx8:
            assert matmul(f, **dict(wide, ldx=40)) == 1
            assert matmul(f, **dict(wide, x=odd)) == 1
        else:
            assert matmul(f, **dict(wide, x=mis)) == 1
            assert matmul(f, **dict(wide, ldx=100)) == 5
        assert matmul(f, **dict(wide, wb=100)) == 5
        assert matmul(f, **dict(wide, wsb=100)) == 3

    def wgrad(**kw):
        # (dy, lddy, xq, xq_bytes, dw, f32, accumulate, tokens, n, k, groups, offsets, ws, ws_bytes, stream)
        a = dict(dict(dy=p, ld=48, xq=p, xb=big, dw=p, f32=0, acc=0, t=8, n=48, k=64, g=1, off=None, ws=p, wsb=big), **kw)
        return lib.mx8_wgrad(a["dy"], a["ld"], a["xq"], a["xb"], a["dw"], a["f32"], a["acc"], a["t"], a["n"], a["k"],
                             a["g"], a["off"], a["ws"], a["wsb"], None)

    for kw in (dict(dy=None), dict(xq=None), dict(dw=None), dict(ws=None), dict(dy=odd), dict(xq=mis), dict(dw=odd),
               dict(ws=mis), dict(ld=47), dict(f32=2), dict(acc=2), dict(n=0), dict(k=0), dict(g=2), dict(t=1 << 31),
               dict(f32=1, dw=ctypes.c_void_p((1 << 16) + 2))):
        assert wgrad(**kw) == 1, kw
    assert wgrad(xb=100) == 5 and wgrad(wsb=100) == 3


def test_binding_refuses_what_is_not_a_matrix():
    import lossless_bf16_tensor_exp_amd as ciera
    assert not math.isnan(ciera.mx8_encoded_size(3, 3))
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ciera.mx8_encode(x, torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ciera.mx4_encode(x.float(), torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ciera.mx8_wgrad(x.half(), x, x, x)
    with pytest.raises(AttributeError):
        ciera.mx9_encode
