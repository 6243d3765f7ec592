"""What the calls around a layer's products refuse on the host, before any
launch, and their sizes; no GPU needed."""
import ctypes

import pytest

import layer_util as lu

torch = pytest.importorskip("torch")

P, ODD, BYTE = ctypes.c_void_p(16 * 1024), ctypes.c_void_p(16 * 1024 + 1), ctypes.c_void_p(16 * 1024 + 4)
ARG, CAPACITY, WORKSPACE = 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from lossless_bf16_tensor_exp_amd import layers, load_library
    layers._bind()
    return load_library()


def norm(lib, x=P, ldx=64, r=None, w=P, eps=1e-6, h=None, y=P, yq=None, size=BIG, rstd=None, rows=4, cols=64):
    return lib.rms_norm(x, ldx, r, 64, w, eps, h, 64, y, 64, yq, size, rstd, rows, cols, None)


def test_norm(lib):
    for bad in (dict(x=None), dict(x=ODD), dict(ldx=63), dict(ldx=(1 << 22) + 1), dict(w=None), dict(w=ODD), dict(y=None), dict(h=P),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-60), dict(cols=0),
                dict(cols=32769, ldx=40000), dict(rows=(1 << 31) + 1), dict(r=ODD), dict(rstd=ctypes.c_void_p(16 * 1024 + 2)),
                dict(yq=BYTE), dict(rows=1 << 31, cols=32768, ldx=32768)):
        assert norm(lib, **bad) == ARG, bad
    assert norm(lib, yq=P, size=4 * 128 + 4 * 4 - 1) == CAPACITY
    assert norm(lib, x=None, y=None, rows=0) == 0


def norm_back(lib, dy=P, h=P, w=P, rstd=P, dh=None, dx=P, dw=P, f32=1, more=0, rows=4, cols=64, ws=P, size=BIG):
    return lib.rms_norm_backward(dy, 64, h, 64, w, rstd, dh, 64, dx, 64, dw, f32, more, rows, cols, ws, size, None)


def test_norm_backward(lib):
    for bad in (dict(dy=None), dict(h=ODD), dict(w=None), dict(rstd=None), dict(dh=P, dx=None), dict(dx=None, dw=None), dict(f32=2),
                dict(more=2), dict(ws=None), dict(ws=BYTE), dict(dw=ctypes.c_void_p(16 * 1024 + 2)), dict(cols=0), dict(dh=ODD)):
        assert norm_back(lib, **bad) == ARG, bad
    assert norm_back(lib, size=lib.rms_norm_workspace_size(4, 64) - 1) == WORKSPACE
    assert norm_back(lib, rows=0, dy=None, h=None, rstd=None, dx=None, dw=None) == 0
    assert lib.rms_norm_workspace_size(1, 0) == lib.rms_norm_workspace_size(1, 32769) == lib.rms_norm_workspace_size((1 << 31) + 1, 8) == 0
    for cols in (1, 64, 2048, 2049, 8192, 32768):  # one workspace serves fewer rows
        sizes = [lib.rms_norm_workspace_size(rows, cols) for rows in (0, 1, 2, 63, 500, 4096, 70000, 1 << 31)]
        assert sizes == sorted(sizes) and sizes[0] >= cols * 4


def sort(lib, ids=P, wide=0, tokens=4, choices=2, experts=3, offsets=P, place=P, order=P, ws=P, size=BIG):
    return lib.expert_sort(ids, wide, tokens, choices, experts, offsets, place, order, ws, size, None)


def test_sort(lib):
    for bad in (dict(ids=None), dict(ids=ODD), dict(ids=BYTE, wide=1), dict(wide=2), dict(choices=0), dict(choices=65), dict(experts=0),
                dict(experts=4097), dict(offsets=None), dict(offsets=BYTE), dict(place=None), dict(order=ODD), dict(ws=None),
                dict(ws=BYTE), dict(tokens=1 << 31, choices=1), dict(tokens=1 << 26, choices=32), dict(tokens=1 << 63)):
        assert sort(lib, **bad) == ARG, bad
    assert sort(lib, size=lib.expert_workspace_size(4, 2, 3) - 1) == WORKSPACE
    for args in ((1, 0, 4), (1, 65, 4), (1, 1, 0), (1, 1, 4097), (1 << 31, 1, 4), (1 << 62, 4, 4)):
        assert lib.expert_workspace_size(*args) == 0, args
    for experts in (1, 64, 1023, 1024, 4096):
        sizes = [lib.expert_workspace_size(t, 8, experts) for t in (0, 1, 500, 4096, 70000, 1 << 27)]
        assert sizes == sorted(sizes) and sizes[0] >= 512


def test_rows(lib):
    def dispatch(x=P, ldx=64, place=P, tokens=4, choices=2, cols=64, rows=8, out=P, outq=None, size=BIG):
        return lib.expert_dispatch(x, ldx, place, tokens, choices, cols, rows, out, 64, outq, size, None)

    def combine(rows_at=P, f32=0, rows=8, place=P, weights=P, residual=None, out=P, out_f32=0, tokens=4, choices=2, cols=64):
        return lib.expert_combine(rows_at, 64, f32, rows, place, weights, residual, 64, out, 64, out_f32, tokens, choices, cols, None)

    def back(dout=P, rows_at=P, f32=0, rows=8, place=P, weights=P, drows=P, dweights=P, tokens=4, choices=2, cols=64):
        return lib.expert_combine_backward(dout, 64, rows_at, 64, f32, rows, place, weights, drows, 64, dweights, tokens, choices, cols,
                                           None)

    for bad in (dict(x=None), dict(x=ODD), dict(ldx=63), dict(place=None), dict(place=ODD), dict(choices=0), dict(choices=65),
                dict(tokens=1 << 31, choices=1), dict(cols=(1 << 21) + 1), dict(rows=(1 << 31) + 1), dict(out=None), dict(out=ODD),
                dict(outq=BYTE), dict(tokens=(1 << 24) + 1, cols=2048, ldx=2048)):
        assert dispatch(**bad) == ARG, bad
    assert dispatch(outq=P, size=8 * 128 + 8 * 4 - 1) == CAPACITY
    assert dispatch(tokens=0, x=None, place=None) == dispatch(rows=0, out=None) == dispatch(cols=0, x=None, out=P) == 0
    for bad in (dict(rows_at=None), dict(f32=2), dict(out_f32=2), dict(rows_at=ctypes.c_void_p(16 * 1024 + 2), f32=1), dict(place=None),
                dict(weights=ODD), dict(residual=ODD), dict(out=None), dict(out=ctypes.c_void_p(16 * 1024 + 2), out_f32=1), dict(choices=65)):
        assert combine(**bad) == ARG, bad
    assert combine(tokens=0, out=None, place=None) == 0
    for bad in (dict(dout=None), dict(rows_at=None), dict(drows=None, dweights=None), dict(f32=2), dict(weights=ODD), dict(drows=ODD),
                dict(dweights=ODD), dict(place=ODD)):
        assert back(**bad) == ARG, bad
    assert back(tokens=0, dout=None, place=None) == 0


def low_rank(lib, x=P, ldx=64, a=P, b=P, scales=None, offsets=P, order=None, base=P, ldb=64, base_f32=0, y=P, ldy=64, y_f32=0, tokens=4,
             n=64, k=64, rank=8, adapters=2, ws=P, size=BIG):
    return lib.low_rank_add(x, ldx, a, b, scales, offsets, order, base, ldb, base_f32, y, ldy, y_f32, tokens, n, k, rank, adapters, ws,
                            size, None)


def test_low_rank(lib):
    for bad in (dict(x=None), dict(x=ODD), dict(ldx=63), dict(a=None), dict(a=ODD), dict(b=None), dict(scales=ODD), dict(offsets=None),
                dict(offsets=BYTE), dict(order=ODD), dict(base=ODD), dict(ldb=10), dict(base_f32=2), dict(y=None), dict(y_f32=2),
                dict(y=ctypes.c_void_p(16 * 1024 + 2), y_f32=1), dict(n=0), dict(k=0), dict(rank=0), dict(rank=129), dict(adapters=0),
                dict(adapters=4097), dict(tokens=(1 << 31) + 1), dict(n=(1 << 21) + 1), dict(ws=None), dict(ws=BYTE), dict(ldb=65),
                dict(y_f32=1), dict(base_f32=1), dict(tokens=1 << 31, n=1 << 20, ldy=1 << 20, base=None)):
        assert low_rank(lib, **bad) == ARG, bad
    assert low_rank(lib, size=lib.low_rank_workspace_size(4, 64, 64, 8, 2) - 1) == WORKSPACE
    assert lib.low_rank_workspace_size(4, 64, 64, 129, 2) == 0 and lib.low_rank_workspace_size(4, 64, 64, 8, 0) == 0


def test_tensors_off_the_gpu_are_refused():
    import lossless_bf16_tensor_exp_amd as c
    m, w = torch.zeros(4, 64, dtype=lu.bf16), torch.ones(64, dtype=lu.bf16)
    ids, table = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    ws, a = torch.zeros(4096, dtype=torch.uint8), torch.zeros(2, 8, 64, dtype=lu.bf16)
    for bad in (lambda: c.rms_norm(m, w, y=m), lambda: c.rms_norm_backward(m, m, w, torch.ones(4), m, None),
                lambda: c.expert_sort(ids, table, ids, None, ws), lambda: c.expert_dispatch(m, ids, out=m),
                lambda: c.expert_combine(m, ids, m), lambda: c.expert_combine_backward(m, m, ids, m, None),
                lambda: c.low_rank_add(m, a, a.transpose(1, 2).contiguous(), table, m, ws)):
        with pytest.raises(ValueError):
            bad()


def test_the_plain_sort():
    ids = torch.tensor([[2, -1], [0, 2], [5, 0]])
    offsets, place, order = lu.sort(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4] and place.tolist() == [[2, -1], [0, 3], [-1, 1]] and order.tolist() == [2, 5, 0, 3, 1, 4]
