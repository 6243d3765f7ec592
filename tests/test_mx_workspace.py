"""Sizes of the microscaled products' workspace (host arithmetic only)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("n,k,groups", [(4096, 4224, 1), (2048, 2048, 1), (1024, 2048, 64), (512, 128, 1), (600, 16384, 3),
                                        (40, 72, 5), (2 ** 20, 2 ** 15, 1)])
def test_a_workspace_serves_every_smaller_number_of_rows(n, k, groups):
    from lossless_bf16_tensor_exp_amd import mx_workspace_size
    sizes = [mx_workspace_size(t, n, k, groups) for t in
             [*range(0, 300), *range(300, 20000, 97), 2 ** 17, 2 ** 20, 2 ** 30]]
    assert sizes[0] > 0
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
