"""Rows in error beside rows that are not: what fork_rows reports, and what decode over shared
pages reads for a group."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import page_side as side
from tests.test_gpu_shared_decode import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def fork(state, parents, keep=None):
    """The call's outputs as arrays, in the model's order, the model's, and the status."""
    table, lengths, shares, free, head, pages = state
    t, s, f = dev(table), dev(shares), dev(free)
    plan = pgd.fork_rows(t, dev(lengths), dev(parents), s, f, free_head=dev([head]),
                         keep=None if keep is None else dev(keep))
    status = pgd.get_device_error()
    want, _ = side.fork_rows(np.asarray(table), lengths, list(parents), keep, shares, free, head,
                             pages)
    return [a.cpu().numpy().reshape(-1) for a in (t, s, f) + tuple(plan)], want, status


def same(got, want):
    for name, g, w in zip(("table", "shares", "free_pages") + pgd.ForkPlan._fields, got, want):
        np.testing.assert_array_equal(g, np.asarray(w).reshape(-1), err_msg=name)


# one cluster's table, and one that all SMs take
@pytest.mark.parametrize("requests,beams,width", [(3, 4, 12), (400, 8, 12)])
@pytest.mark.parametrize("cut", [False, True])
def test_an_entry_outside_the_pool_in_a_row_with_one_child(requests, beams, width, cut):
    """A row that goes on as it is, or as another one, reports its entries outside the pool; one
    past its pages, or in a row that nobody reads, is nobody's."""
    rng = np.random.default_rng(31)
    state = side.random_state(rng, requests, beams, 500, 90, width=width)
    table, lengths, shares, free, head, pages = state
    lengths[5] = 4 * 64 + 9
    fresh = free[head:head + 5]
    for p in table[5]:
        if 0 <= p < pages and shares[p]:
            shares[p] -= 1
    table[5, :5], head = fresh, head + 5
    shares[fresh] = 0
    rows = requests * beams
    state = table, lengths, shares, free, head, pages
    keep = np.full(rows, 2 ** 31 - 1)
    if cut:
        keep[[5, 6]] = 2 * 64 + 3
    itself = np.arange(rows)
    swapped = itself.copy()
    swapped[[5, 6]] = 6, 5
    for parents in (itself, swapped):
        got, want, status = fork(state, parents, keep)
        assert status == pgd.OK
        same(got, want)
        for e in (0, 1, 2) if cut else (0, 1, 3, 4):
            for page in (-1, pages):
                holes = table.copy()
                holes[5, e] = page
                got, want, status = fork((holes,) + state[1:], parents, keep)
                same(got, want)
                assert status == pgd.EDEVICE_BOUNDS, (e, page)
    past = table.copy()
    past[5, 5:] = pages
    got, want, status = fork((past,) + state[1:], swapped, keep)
    same(got, want)
    assert status == pgd.OK


def rows_of_two_pages(rows, width):
    """Row r holds pages 2 r and 2 r + 1, 100 positions; then row 1's last page is row 0's."""
    table = np.full((rows, width), -7)
    table[:, :2] = np.arange(2 * rows).reshape(rows, 2)
    table[1, 1] = 1
    return table, np.full(rows, 100), np.zeros(2 * rows + 40, dtype=int), \
        np.r_[np.delete(np.arange(2 * rows), 3), 2 * rows:2 * rows + 40], 2 * rows - 1, 2 * rows + 40


# one cluster's table, and one that all SMs take
@pytest.mark.parametrize("rows,width", [(5, 3), (2600, 11)])
def test_more_rows_leave_a_page_than_its_shares_say(rows, width):
    """Rows 0 and 1 hold page 1, shares say one does.  Whatever becomes of it, it is an error, the
    same outputs come of it every time, and no page is both held and listed, or listed twice."""
    state = rows_of_two_pages(rows, width)
    itself = np.arange(rows)
    released, crossed = itself.copy(), itself.copy()
    released[0] = -1                # gives it up; row 1 stays
    crossed[2] = 1                  # three rows leave it
    for parents in (released, itself, crossed):
        runs = [fork(state, parents) for _ in range(20 if rows < 100 else 5)]
        for got, want, status in runs:
            assert status == pgd.EDEVICE_BOUNDS
            for a, b in zip(got, runs[0][0]):
                np.testing.assert_array_equal(a, b)
        got, want, _ = runs[0]
        if parents is released:
            same(got, want)
        table, _, free, lengths, _, targets, _, head = got
        table = table.reshape(rows, width)
        held = {p for r in range(rows) for p in table[r, :side.pages_of(lengths[r])]}
        listed = list(free[head[0]:])
        assert len(set(listed)) == len(listed) and not held & set(listed)
        assert list(targets[:3] >= 0) == [False, True, parents is crossed]


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


def step(b, kernel, written, **kw):
    """A step of new values: the pools afterwards hold those of the rows `written`, and nothing
    else that is new, bit for bit.  Returns the outputs and the status."""
    rows = len(b.positions)
    new = [torch.randn(rows, b.hkv, b.d, generator=b.gen).bfloat16() for _ in range(2)]
    for r in written:
        n = b.positions[r]
        for pool, x in zip((b.k, b.v), new):
            pool[b.table[r, n // 64], :, n % 64] = x[r]
    out = b.call(*(x.to(DEV) for x in new), kernel=kernel, **kw)
    status = pgd.get_device_error()
    for pool, host in ((b.k_pool, b.k), (b.v_pool, b.v)):
        assert torch.equal(pool.view(torch.int16), b.lay(host).view(torch.int16))
    return out, status


@pytest.mark.parametrize("hq,hkv,d,layout", [(32, 8, 128, pgd.PAGE_MAJOR), (14, 2, 64, pgd.HEAD_MAJOR)])
def test_what_a_step_writes_of_rows_in_error(hq, hkv, d, layout):
    """Rows with a page outside the pool among the group's (written), among their own (not),
    with positions in error (not)."""
    b = Batch(42, [(4, 6), (3, 2), (2, None)], [90] * 9, hq, hkv, d, layout)
    good = b.table.copy()
    b.table[4:7, 1] = b.pages                     # of the second group
    b.table[1, 6] = -1                            # row 1's own first page, not the new token's
    b.table[8, 1] = b.pages                       # row 8's, the new token's
    true = b.positions.copy()
    b.positions[2], b.positions[7] = 100, b.width * 64
    out, status = step(b, pgd.KERNEL_PREFILL_UMMA, (0, 3, 4, 5, 6))
    assert status == pgd.EDEVICE_BOUNDS
    bad = (1, 2, 4, 5, 6, 7, 8)
    assert not out[list(bad)].any()
    at = b.positions.copy()
    at[list(bad)] = -1
    b.positions, b.table = at, good
    b.compare(out, d ** -0.5)
    # starts that decrease, pages of a group out of range: nothing of their rows is written
    b = Batch(43, [(4, 6), (3, 2), (2, None)], [90] * 9, hq, hkv, d, layout)
    shared = b.shared
    b.shared = [6, 10 ** 6]
    out, status = step(b, pgd.KERNEL_PREFILL_UMMA, (0, 1, 2, 3, 7, 8))
    assert status == pgd.EDEVICE_BOUNDS and not out[4:7].any() and bool((out[:4] != 0).any())
    b.shared, b.starts = shared, [0, 8, 7]
    out, status = step(b, pgd.KERNEL_PREFILL_UMMA, ())
    assert status == pgd.EDEVICE_BOUNDS and not out.any()


def test_what_a_step_writes_row_by_row():
    """A page outside the pool in a split before the last one: the row is written, its output zero."""
    b = Batch(44, [(4, 40)], [1500] * 4, 32, 8, 128)  # 64 pages a row, splits of 24
    good = b.table.copy()
    b.table[1, 3] = b.table[2, 63] = b.pages
    out, status = step(b, pgd.KERNEL_TENSOR_CORE, (0, 1, 3))
    assert status == pgd.EDEVICE_BOUNDS and not out[1:3].any()
    at = b.positions.copy()
    at[1:3] = -1
    b.positions, b.table = at, good
    b.compare(out, 128 ** -0.5)
