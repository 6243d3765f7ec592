"""Which kernel the microscaled products choose (no GPU: mx_rules.h compiled
for the host).  Each listed choice is the faster of the two that were timed, or
within a tenth of it."""
import ctypes
import os
import random

import pytest

from mx_rules import kernel, rules

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("op", ["bf16", "mx8"])
@pytest.mark.parametrize("groups", [1, 4, 64, 1000])
def test_no_workgroup_walks_many_rows(op, groups):
    """k_mx_few takes a group's rows 16 at a time, one pass after the other: few passes only, however narrow the product."""
    for n in (1, 16, 48, 64, 100, 512, 4096):
        for tokens in (groups * r for r in (1, 16, 64, 65, 100, 500, 2000, 8000)):
            if kernel(op, tokens, n, 2048, groups).startswith("few"):
                assert tokens <= 64 * groups, (tokens, n)


@pytest.mark.parametrize("op,tokens,n,groups,want", [
    # one group: the split form up to 48 rows (x in mx8: 64) at any width
    ("bf16", 1, 2048, 1, "few16"), ("bf16", 1, 16384, 1, "few128"), ("bf16", 8, 16384, 1, "few128"),
    ("bf16", 32, 48, 1, "few16"), ("bf16", 32, 2048, 1, "few16"), ("bf16", 16, 8192, 1, "few16"),
    ("bf16", 64, 48, 1, "32x128"), ("bf16", 128, 64, 1, "32x128"), ("bf16", 2000, 64, 1, "32x128"),
    ("bf16", 500, 256, 1, "32x128"), ("bf16", 24, 8192, 1, "32x128"), ("bf16", 8000, 16, 1, "32x128"),
    ("mx8", 64, 256, 1, "few16"), ("mx8", 64, 1024, 1, "few16"), ("mx8", 128, 48, 1, "64x128"), ("mx8", 512, 48, 1, "64x128"),
    # groups: by the rows of each, and their passes in the larger groups
    ("bf16", 64, 1024, 64, "few128"), ("bf16", 128, 1024, 64, "few128"), ("bf16", 256, 512, 64, "few128"),
    ("bf16", 64, 2048, 16, "few128"), ("bf16", 512, 256, 64, "32x128"), ("bf16", 128, 1024, 16, "32x128"),
    ("bf16", 512, 1024, 64, "32x128"), ("bf16", 96, 48, 4, "few16"), ("bf16", 128, 256, 16, "few16"),
    ("bf16", 96, 1024, 16, "few128"), ("bf16", 384, 256, 64, "32x128"), ("bf16", 256, 256, 16, "few16"),
    ("bf16", 384, 256, 16, "32x128"), ("bf16", 128, 256, 4, "32x128"), ("bf16", 512, 48, 64, "few16"), ("bf16", 2000, 48, 64, "32x128"), ("bf16", 512, 48, 16, "32x128"),
    ("mx8", 256, 512, 64, "few128"), ("mx8", 512, 256, 64, "few128"), ("mx8", 512, 128, 16, "few16"),
    ("mx8", 1024, 48, 16, "64x128"), ("mx8", 256, 1024, 16, "64x128"),
])
def test_few_rows_or_tiles(op, tokens, n, groups, want):
    assert kernel(op, tokens, n, 2048, groups) == want


@pytest.mark.parametrize("op,tokens,n,k,groups,want", [
    # dx: 128 rows for one group of many; groups, whose last tiles are part empty, from four times as many tiles on
    ("dx", 4096, 2048, 2048, 1, "64x256"), ("dx", 8192, 2048, 2048, 1, "128x256"), ("dx", 8192, 512, 2048, 1, "128x256"),
    ("dx", 8192, 2048, 2048, 2, "64x256"), ("dx", 8192, 1024, 2048, 8, "64x256"), ("dx", 8192, 512, 4096, 4, "64x256"),
    ("dx", 16384, 2048, 2048, 8, "64x256"), ("dx", 32768, 1024, 2048, 64, "64x256"), ("dx", 32768, 2048, 2048, 4, "128x256"),
    ("dx", 65536, 1024, 2048, 16, "128x256"),
    # and the smaller ones
    ("dx", 512, 2048, 2048, 1, "64x128"), ("dx", 2048, 2048, 2048, 1, "64x128"), ("dx", 999, 1408, 2048, 66, "32x256"),
    ("dx", 3000, 1024, 2048, 64, "32x256"), ("dx", 4000, 1024, 2048, 64, "64x256"),
    # x in mx8: groups take 128 columns
    ("mx8", 32768, 1024, 2048, 64, "128x128"), ("mx8", 16384, 2048, 2048, 8, "128x128"), ("mx8", 8192, 4096, 8192, 1, "128x256"),
    ("mx8", 32768, 2048, 2048, 1, "128x256"), ("bf16", 32768, 1024, 2048, 64, "128x256"), ("bf16", 8192, 1024, 2048, 8, "128x128"),
    ("mx8", 4000, 1024, 2048, 64, "64x128"), ("bf16", 4001, 2048, 2048, 1, "128x128"),
])
def test_tile_of_many_rows(op, tokens, n, k, groups, want):
    assert kernel(op, tokens, n, k, groups) == want


MOST = (2 ** 32 - 1) // 256  # workgroups of 256 threads


def workgroups(op, tokens, n, k, groups):
    r = rules()
    if op == "wgrad":
        return r.tile_groups(2, 256, 128, tokens, n, k, groups, 1, r.wgrad_parts(tokens, n, k, groups))
    name = kernel(op, tokens, n, k, groups)
    if name.startswith("few"):
        return 2 * -(-n // (128 if name == "few128" else 16))  # of 512 threads; the groups are another dimension
    return r.tile_groups({"bf16": 0, "dx": 1, "mx8": 3, "scaled": 3}[op], *map(int, name.split("x")), tokens, n, k, groups,
                         int(groups > 1), 1)


def test_what_the_contract_allows_is_launched():
    """Every kernel of sizes that the header does not except has less than 2^32 threads."""
    gen = random.Random(1)
    top = {"bf16": 0, "mx8": 0, "scaled": 0, "dx": 0, "wgrad": 0}
    for _ in range(20000):
        groups = min(4096, int(2 ** gen.uniform(0, 12.01)))
        tokens = int(2 ** gen.uniform(0, 31)) - 1
        n = min(2 ** 21, 2 ** 31 // groups, int(2 ** gen.uniform(0, 21.01)))
        k = min(2 ** 21, int(2 ** gen.uniform(0, 21.01)))
        for op in top:
            if op == "wgrad":
                count = groups * (-(-(-(-n // 256) * -(-k // 128)) // 8) * 8)
            else:
                count = (tokens // 32 + groups + 1) * -(-(k if op == "dx" else n) // 128)
            if count < 2 ** 24:
                need = workgroups(op, tokens, n, k, groups)
                assert need <= MOST, (op, tokens, n, k, groups)
                top[op] = max(top[op], need)
    assert all(t > MOST // 16 for t in top.values()), top  # the search came near the border
    for rows, cols, ok in ((2 ** 29 - 32, 128, True), (2 ** 29 - 31, 128, False), (2 ** 31, 24, True), (2 ** 31, 25, False),
                           (2 ** 31, 32, False), (2 ** 15 - 1, 2 ** 21, True), (2 ** 15, 2 ** 21, False)):
        assert (rules().unit_groups(rows, cols) <= MOST) == ok, (rows, cols)
        assert ok == (rows * (-(-cols // 8) * 8) <= 2 ** 36 - 4096)


def test_what_needs_more_threads_is_refused_before_a_launch():
    import lossless_bf16_tensor_exp_amd as ciera
    if not os.path.exists(ciera.library_path()):
        from lossless_bf16_tensor_exp_amd import build
        build.build()
    from lossless_bf16_tensor_exp_amd import mx as calls
    lib, p, big = calls._lib(), ctypes.c_void_p(1 << 16), 1 << 62
    for enc in (lib.mx8_encode, lib.mx4_encode):
        assert enc(p, 2 ** 29, 1, 1, p, big, None) == 1
        assert enc(p, 2 ** 15, 2 ** 21, 2 ** 21, p, big, None) == 1
    for dec in (lib.mx8_decode, lib.mx4_decode):
        assert dec(p, big, 2 ** 31, 32, p, 32, None) == 1
    g, n = 4096, 2 ** 19
    for f in (lib.mx4_matmul, lib.mx4_matmul_mx8):
        ldx = big if f is lib.mx4_matmul_mx8 else 64
        assert workgroups("mx8" if f is lib.mx4_matmul_mx8 else "bf16", 4096, n, 64, g) > MOST
        assert f(p, ldx, p, big, p, n, 0, 4096, n, 64, g, p, p, big, None) == 1
    assert workgroups("scaled", 4096, n, 64, g) > MOST
    assert lib.mx4_matmul_mx8(p, big, p, big, p, n, 4, 4096, n, 64, g, p, p, big, None) == 1
    n = 2 ** 21
    assert workgroups("dx", 4096, 64, n, g) > MOST
    assert lib.mx4_matmul_dx(p, 64, p, big, p, n, 0, 4096, 64, n, g, p, p, big, None) == 1
    assert workgroups("wgrad", 64, 1, 2 ** 21, g) > MOST
    assert lib.mx8_wgrad(p, 1, p, big, p, 0, 0, 64, 1, 2 ** 21, g, p, p, big, None) == 1


def test_only_the_mx8_product_takes_the_scaled_instructions():
    from lossless_bf16_tensor_exp_amd import mx as calls
    lib, p, big = calls._lib(), ctypes.c_void_p(1 << 16), 1 << 40
    assert lib.mx4_matmul(p, 64, p, big, p, 48, 4, 8, 48, 64, 1, None, p, big, None) == 1
    assert lib.mx4_matmul_dx(p, 48, p, big, p, 64, 4, 8, 48, 64, 1, None, p, big, None) == 1
    assert lib.mx8_wgrad(p, 48, p, big, p, 4, 0, 8, 48, 64, 1, None, p, big, None) == 1
    for kind in (2, 3, 5, 8):
        assert lib.mx4_matmul_mx8(p, big, p, big, p, 48, kind, 8, 48, 64, 1, None, p, big, None) == 1
    for bad in (dict(q=None), dict(y=None), dict(ws=100), dict(wb=100), dict(qb=100)):  # as for the others
        a = dict(dict(q=p, qb=big, wb=big, y=p, ws=big), **bad)
        st = lib.mx4_matmul_mx8(a["q"], a["qb"], p, a["wb"], a["y"], 48, 4, 8, 48, 64, 1, None, p, a["ws"], None)
        assert st == {"q": 1, "y": 1, "ws": 3, "wb": 5, "qb": 5}[next(iter(bad))]
