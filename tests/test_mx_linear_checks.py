"""What MxLinear refuses, without a GPU: the library's calls are replaced by
ones that record that they were reached."""
import pytest

torch = pytest.importorskip("torch")

CALLS = ("mx4_encode", "mx4_matmul", "mx8_encode", "mx4_matmul_mx8", "mx4_matmul_dx", "mx8_wgrad")


@pytest.fixture
def made(monkeypatch):
    """make(...) a layer on the CPU; made.reached lists the calls it made."""
    from lossless_bf16_tensor_exp_amd import codec

    class Made:
        reached, fails = [], set()

        def __call__(self, *args, **kw):
            return codec.MxLinear(*args, device="cpu", **kw)

    made = Made()
    made.reached, made.fails = [], set()
    for name in CALLS:
        def call(*args, name=name, **kw):
            made.reached.append(name)
            if name in made.fails:
                raise TypeError(name)
        monkeypatch.setattr(codec, name, call)
    return made


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("x,y", [((8, 128), (8, 64)), ((8, 256), (8, 32)), ((8, 256), (8, 65)), ((8, 257), (8, 64)),
                                 ((8, 256), (7, 64)), ((64, 256), (64, 64)), ((8,), (8, 64)), ((8, 256), (8,)),
                                 ((1, 8, 256), (8, 64))])
def test_forward_and_keep_take_the_layers_shapes_only(made, x, y):
    layer = made(16, 64, 256)
    for call in (layer.forward, layer.keep):
        with pytest.raises(ValueError):
            call(bf(*x), bf(*y))
    assert made.reached == []
    layer.forward(bf(8, 256), bf(8, 64))
    layer.keep(bf(8, 256), bf(8, 64))
    assert made.reached == ["mx4_matmul", "mx8_encode", "mx4_matmul_mx8"]


@pytest.mark.parametrize("groups,dy,dx,dw", [(1, (8, 32), None, (64, 256)), (1, (8, 64), (8, 128), None),
                                             (1, (8, 64), (7, 256), None), (1, (8, 64), None, (64, 128)),
                                             (1, (8, 64), None, (32, 256)), (1, (8, 64), None, (2, 64, 256)),
                                             (2, (8, 64), None, (64, 256)), (2, (8, 64), None, (2, 64, 128)),
                                             (2, (8, 32), (8, 256), (2, 32, 256)), (1, (7, 64), (7, 256), None),
                                             (1, (8,), (8, 256), None), (1, (8, 64), (8, 256), (64, 255))])
def test_backward_takes_the_layers_shapes_only(made, groups, dy, dx, dw):
    layer = made(16, 64, 256, groups)
    offsets = None if groups == 1 else torch.tensor([0, 3, 8])
    layer.keep(bf(8, 256), bf(8, 64), offsets)
    del made.reached[:]
    with pytest.raises(ValueError):
        layer.backward(bf(*dy), None if dx is None else bf(*dx), None if dw is None else bf(*dw), offsets)
    assert made.reached == [], "a refused call computes neither gradient"
    layer.backward(bf(8, 64), bf(8, 256), bf(groups, 64, 256), offsets)
    assert made.reached == ["mx4_matmul_dx", "mx8_wgrad"]


def test_one_groups_gradient_has_two_or_three_dimensions(made):
    layer = made(16, 64, 256)
    layer.keep(bf(8, 256), bf(8, 64))
    layer.backward(bf(8, 64), None, bf(64, 256))
    layer.backward(bf(8, 64), None, bf(1, 64, 256))
    assert made.reached[-2:] == ["mx8_wgrad"] * 2


def test_a_keep_that_fails_leaves_no_checkpoint(made):
    """The new x overwrites the buffer before the product can refuse: what an earlier call kept is gone then."""
    layer = made(16, 64, 256)
    for call in ("mx4_matmul_mx8", "mx8_encode"):
        layer.keep(bf(8, 256), bf(8, 64))
        layer.backward(bf(8, 64), None, bf(64, 256))
        made.fails = {call}
        with pytest.raises(TypeError):
            layer.keep(bf(12, 256), bf(12, 64))
        del made.reached[:]
        for rows in (8, 12, 0):
            with pytest.raises(ValueError):
                layer.backward(bf(rows, 64), bf(rows, 256), bf(64, 256))
        assert made.reached == []
        made.fails = set()


def test_backward_needs_a_checkpoint(made):
    layer = made(16, 64, 256)
    with pytest.raises(ValueError):
        layer.backward(bf(0, 64), None, bf(64, 256))
    layer.keep(bf(0, 256), bf(0, 64))
    layer.backward(bf(0, 64), None, bf(64, 256))
    assert made.reached[-1] == "mx8_wgrad"


def test_load_takes_weights_that_lie_apart(made, monkeypatch):
    """Rows of a wider buffer, in two dimensions or three; a copy is never made in silence."""
    from lossless_bf16_tensor_exp_amd import codec
    seen = []
    monkeypatch.setattr(codec, "mx4_encode", lambda rows, out, stream=None: seen.append((rows.shape, rows.stride(), rows.data_ptr())))
    layer = made(16, 64, 256, 3)
    wide = torch.zeros(3, 64, 300, dtype=torch.bfloat16)
    for w, stride in ((wide[:, :, :256], 300), (wide[:, :, 8:264], 300), (wide.view(192, 300)[:, :256], 300),
                      (torch.zeros(3, 64, 256, dtype=torch.bfloat16), 256)):
        layer.load(w)
        assert seen[-1] == ((192, 256), (stride, 1), w.data_ptr())
    for w in (torch.zeros(3, 70, 256, dtype=torch.bfloat16)[:, :64], torch.zeros(64, 3, 256, dtype=torch.bfloat16).transpose(0, 1)):
        with pytest.raises(ValueError, match="apart"):
            layer.load(w)
    for shape in ((2, 64, 256), (64, 256), (3, 64, 255), (3, 1, 64, 256), (192 * 256,)):
        with pytest.raises(ValueError):
            layer.load(bf(*shape))
    assert len(seen) == 4
    one = made(16, 1, 256, 3)  # a row a group, each from a matrix of its own
    one.load(torch.zeros(3, 5, 256, dtype=torch.bfloat16)[:, 2:3])
    assert seen[-1][:2] == ((3, 256), (1280, 1))
