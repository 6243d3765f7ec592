"""Which kernel the microscaled products choose (no GPU: mx_rules.h compiled
for the host).  Each listed choice is the faster of the two that were timed, or
within a tenth of it."""
import pytest

from mx_rules import kernel


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
    ("bf16", 512, 48, 64, "few16"), ("bf16", 2000, 48, 64, "32x128"), ("bf16", 512, 48, 16, "32x128"),
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
