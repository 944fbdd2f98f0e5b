"""The waits between the warps of lora_tile_kernel, run through in every order on the CPU: no
copy into the ring of row scales may come before the last read of what it replaces.

The kernel's warps as steps that wait for one another (lora.cu has the same names):
  * a converting warp, at block b: asks for the scales of block b + kTileRaw - 1 (and before the
    first block for those of the blocks below kTileRaw - 1); waits until the products of block
    b - kTileXStages are known complete (s_xempty); converts block b (s_xfull).
  * the issuing thread: product p, of block p // groups, when its block is converted and every sum
    warp has released the accumulator of product p - kTileAccs (s_tempty).
  * a sum warp, at product p: sees it complete (s_tfull), reads its block's scales, releases
    the accumulator.  The first one, on seeing a block's last product, says so (s_xempty).
Products complete and copies land as soon as they may, which is when a missing wait shows.
"""
import os
import re

import pytest

from conftest import ROOT


def _constants():
    with open(os.path.join(ROOT, "serving_lightning_indexer_gb300", "csrc", "lora.cu")) as f:
        text = f.read()
    return {k: int(re.search(rf"\b{k} = (\d+)[,;]", text).group(1)) for k in ("kTileXStages", "kTileRaw", "kTileAccs", "kTileScales")}


def _first_overwrite(c, groups, blocks):
    """None, or (block copied, block still to be read in its slot) of some order of the steps."""
    products = blocks * groups
    ahead = c["kTileRaw"] - 1
    # blocks asked for, blocks converted, products issued, products the first sum warp has seen and
    # read, products the slowest one has read
    start = (min(ahead, blocks), 0, 0, 0, 0, 0)
    todo, known = [start], {start}
    while todo:
        asked, converted, issued, seen, read0, read1 = todo.pop()
        after = []
        if asked < blocks and asked == converted + ahead:
            oldest = min(read0, read1) // groups
            if oldest <= asked - c["kTileScales"]:
                return asked, asked - c["kTileScales"]
            after.append((asked + 1, converted, issued, seen, read0, read1))
        if converted < blocks and asked == min(blocks, converted + ahead + 1):
            complete = seen // groups                      # blocks whose last product has been seen
            if converted < c["kTileXStages"] or complete > converted - c["kTileXStages"]:
                after.append((asked, converted + 1, issued, seen, read0, read1))
        if issued < products and issued // groups < converted and min(read0, read1) > issued - c["kTileAccs"]:
            after.append((asked, converted, issued + 1, seen, read0, read1))
        if seen < issued and seen == read0:
            after.append((asked, converted, issued, seen + 1, read0, read1))
        if read0 < seen:
            after.append((asked, converted, issued, seen, read0 + 1, read1))
        if read1 < issued:
            after.append((asked, converted, issued, seen, read0, read1 + 1))
        for s in after:
            if s not in known:
                known.add(s)
                todo.append(s)
    assert (blocks, blocks, products, products, products, products) in known   # and every order ends
    return None


@pytest.mark.parametrize("groups", [1, 2, 3, 4, 5, 8])
def test_no_scale_is_replaced_before_it_is_read(groups):
    assert _first_overwrite(_constants(), groups, 24) is None


@pytest.mark.parametrize("groups,slots", [(1, 11), (2, 9), (3, 9), (4, 8)])
def test_the_model_finds_a_ring_that_is_too_short(groups, slots):
    c = dict(_constants(), kTileXStages=3, kTileRaw=4, kTileAccs=4)
    assert _first_overwrite(dict(c, kTileScales=slots), groups, 24) is None
    assert _first_overwrite(dict(c, kTileScales=slots - 1), groups, 24) is not None
