"""Rows in error beside rows that are not: what decode over shared pages reads for a group."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests.test_gpu_shared_decode import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("hq,hkv,d,layout", [(32, 8, 128, pgd.PAGE_MAJOR), (14, 2, 64, pgd.HEAD_MAJOR)])
def test_a_row_in_error_lends_its_group_no_pages(hq, hkv, d, layout):
    """The first rows of groups, and of a group's second block, are in error; their tables name
    other pages of the pool.  The other rows' results are theirs."""
    groups, own = [(2, None), (4, 6), (3, 2), (80, 5)], np.full(89, 90)
    b = Batch(41, groups, own, hq, hkv, d, layout)
    good, true = b.want, b.positions.copy()
    bad = [2, 3, 6, 9, 10, 45, 73]                # (blocks of the last group: 9, 45 or 73, 81)
    table = b.table.copy()

    def want(scale, sinks=None):
        at, b.positions, names, b.table = b.positions, true, b.table, table
        r = good(scale, sinks)
        b.positions, b.table = at, names
        return r
    b.want = want
    b.positions = true.copy()
    b.positions[[2, 6, 9, 45]] = 70               # in the groups' pages
    b.positions[[3, 10, 73]] = b.width * 64 + 5   # beyond the table
    b.table = table.copy()
    for r in bad:
        b.table[r, :6] = (b.table[r, :6] + 1) % b.pages
    b.check(status=pgd.EDEVICE_BOUNDS, bad=bad)
    # nobody else is left in a group: nothing is read for it
    b.positions[[4, 5]] = 1, -1
    b.table[[4, 5], :6] = -9
    gone = b.want

    def without(scale, sinks=None):
        r = gone(scale, sinks)
        for x in r:
            x[5] = 0
        return r
    b.want = without
    b.check(status=pgd.EDEVICE_BOUNDS, bad=bad + [4])
