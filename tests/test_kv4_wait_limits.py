"""The wait of attention over the 4-bit cache that lasts as long as a piece: its limit covers the longest piece that the header
allows (no GPU needed)."""
import os
import re

import pytest

import kv4_shapes

CSRC = os.path.dirname(kv4_shapes.SOURCE)
TILE_NS = 900  # what a tile of 128 keys takes a CTA at most, with 16 heads a group (24 sequences of up to 32K keys: 840)


def read(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return f.read()


@pytest.mark.parametrize("L_cap", [16, 4096, 1 << 20, 1 << 27, (1 << 27) + 128, 1 << 29, (1 << 31) - 1024])
def test_the_finishing_warps_wait_long_enough_for_a_piece(L_cap):
    """One CTA may have a whole segment: sequences whose tables share their pages are as long as the table. Twice its time."""
    limit = int(re.search(r"kWaitLimitNs = (\d+)ull;", read("moe_device.cuh"))[1])
    src = read("kv4_decode.cu")
    e = re.search(r"p\.piece_waits = ([^;]+);", src)
    waits = 1
    if e and re.search(r"i < p\.piece_waits && !mbar_wait\(h_full, [^)]*\);\) \+\+i;\n\s+wait\(h_full,", src):
        waits = eval(e[1].replace("p.L_cap", str(L_cap)).replace("kv4::kKeys", "128").replace("/", "//"))
    tiles = -(-L_cap // 128) + 1
    assert waits * limit >= 2 * tiles * TILE_NS
    assert waits == 1 or L_cap > 1 << 26, "ordinary lengths keep one limit"
