"""assign_pages against the plain request-by-request implementation: every
output is a whole number and has to be equal, the table's untouched entries
included."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import step_reference as ref

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


def batch(rng, requests, cached_hi, new_hi, width=None, spare=5, zeros=0.2):
    cached = rng.integers(0, cached_hi + 1, requests)
    new = rng.integers(0, new_hi + 1, requests) * (rng.random(requests) >= zeros)
    have, need = -(-cached // 64), -(-(cached + new) // 64)
    width = width or int(need.max(initial=0)) + 2
    total = int(need.sum()) + spare
    order = rng.permutation(total)
    table = np.full((requests, width), -7, dtype=np.int64)   # entries out of use: any value
    used = 0
    for r in range(requests):
        table[r, :have[r]] = order[used:used + have[r]]
        used += have[r]
    return cached, new, table, order[used:], total


def check(cached, new, table, free, num_tokens, num_pages, head=None, status=None, out=None):
    t, f = dev(table), dev(free)
    h = None if head is None else dev([head])
    keep = [dev(cached), dev(new), f.clone()]
    plan = pgd.assign_pages(t, keep[0], keep[1], f, num_tokens=num_tokens, num_pages=num_pages,
                            free_head=h, out=out)
    got_status = pgd.get_device_error()
    want = ref.assign_pages(np.asarray(table), cached, new, free, num_tokens, num_pages, head or 0)
    for name, got, w in zip(("table",) + pgd.PagePlan._fields, (t,) + tuple(plan), want):
        np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1),
                                      err_msg=name)
    assert got_status == (pgd.EDEVICE_BOUNDS if want[-1] else pgd.OK)
    if status is not None:
        assert got_status == status
    assert torch.equal(f, keep[2])
    return plan


@pytest.mark.parametrize("requests,cached_hi,new_hi,pad", [
    (1, 0, 1, 0), (1, 63, 1, 3), (1, 64, 64, 0), (1, 5000, 3000, 100),
    (4, 300, 1, 60), (64, 32768, 1, 0), (31, 200, 700, 13), (1000, 100, 40, 1),
    (1024, 10, 3, 0), (1025, 70, 65, 5), (4095, 64, 2, 0), (4096, 65, 5, 7),
    (4097, 127, 3, 0), (9001, 40, 9, 33), (20000, 3, 1, 0),
])
def test_matches_the_plain_form(requests, cached_hi, new_hi, pad):
    rng = np.random.default_rng(requests + new_hi)
    cached, new, table, free, total = batch(rng, requests, cached_hi, new_hi)
    check(cached, new, table, free, int(new.sum()) + pad, total, status=pgd.OK)


def test_head_and_reused_plan():
    rng = np.random.default_rng(5)
    cached, new, table, free, total = batch(rng, 50, 500, 90, spare=40)
    tokens = int(new.sum()) + 9
    plan = check(cached, new, table, free, tokens, total, head=17)
    again = check(cached, new, table, free, tokens, total, head=40, out=plan)
    assert all(a is b for a, b in zip(plan, again))


def test_no_requests_no_tokens_no_pages():
    check(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 3), int), np.arange(4), 5, 9, head=2,
          status=pgd.OK)
    check(np.array([64, 3]), np.array([0, 0]), np.full((2, 2), 1), np.zeros(0, int), 0, 9,
          status=pgd.OK)
    check(np.array([63, 3]), np.array([1, 2]), np.full((2, 2), 1), np.zeros(0, int), 3, 9,
          status=pgd.OK)   # every token fits a page in use


@pytest.mark.parametrize("short", [1, 3, 50])
def test_too_few_free_pages(short):
    rng = np.random.default_rng(7)
    cached, new, table, free, total = batch(rng, 200, 300, 100, spare=0)
    check(cached, new, table, free[:-short], int(new.sum()), total, status=pgd.EDEVICE_BOUNDS)


@pytest.mark.parametrize("short", [1, 64, 5000])
def test_too_few_places(short):
    rng = np.random.default_rng(8)
    cached, new, table, free, total = batch(rng, 5000, 30, 4)
    check(cached, new, table, free, max(0, int(new.sum()) - short), total,
          status=pgd.EDEVICE_BOUNDS)


def test_bad_lengths_are_left_out_and_reported():
    table = np.arange(20).reshape(5, 4)
    top = 2 ** 31 - 1
    check(np.array([-1, 10, 250, top, 5]), np.array([3, -2, 7, top, 60]), table,
          np.arange(20, 30), 100, 30, status=pgd.EDEVICE_BOUNDS)


def test_sums_past_int32():
    # 40 requests of 2^26 - 64 positions each in wide rows: the sum of the tokens passes 2^31
    width, requests = 2 ** 20, 40
    cached, new = np.zeros(requests, int), np.full(requests, width * 64)
    t = torch.full((requests, width), -7, dtype=torch.int32, device=DEV)
    plan = pgd.assign_pages(t, dev(cached), dev(new), dev(np.arange(100)), num_tokens=1000,
                            num_pages=200)
    assert pgd.get_device_error() == pgd.EDEVICE_BOUNDS
    assert int(plan.free_head) == 0 and int(plan.positions.max()) == -1
    assert plan.starts.tolist() == [0] + [1000] * requests and int(plan.lengths.abs().max()) == 0
    assert int((t != -7).sum()) == 0


@pytest.mark.parametrize("head", [-1, 12])
def test_bad_head(head):
    table = np.arange(8).reshape(2, 4)
    check(np.array([64, 10]), np.array([1, 5]), table, np.arange(8, 18), 8, 30, head=head,
          status=pgd.EDEVICE_BOUNDS)


def test_pages_outside_the_pool():
    table = np.array([[3, 0, 0], [99, 0, 0]])
    check(np.array([10, 20]), np.array([60, 50]), table, np.array([-4, 5, 6]), 120, 30,
          status=pgd.EDEVICE_BOUNDS)


def test_stream_graph_and_two_at_once():
    rng = np.random.default_rng(9)
    cached, new, table, free, total = batch(rng, 300, 200, 50)
    tokens = int(new.sum())
    side = torch.cuda.Stream()
    t1, t2, c, n, f = dev(table), dev(table), dev(cached), dev(new), dev(free)
    side.wait_stream(torch.cuda.current_stream())
    a = pgd.assign_pages(t1, c, n, f, num_tokens=tokens, num_pages=total, stream=side)
    b = pgd.assign_pages(t2, c, n, f, num_tokens=tokens, num_pages=total)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(t1, t2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pgd.assign_pages(t2, c, n, f, num_tokens=tokens, num_pages=total, out=a)
    # another batch in the same places: the replay sees it
    cached2, new2 = cached[::-1].copy(), np.minimum(new, 30)[::-1].copy()
    have2 = -(-cached2 // 64)
    table2 = np.where(np.arange(table.shape[1])[None] < have2[:, None], 1, 0)
    t2.copy_(dev(table2)), c.copy_(dev(cached2)), n.copy_(dev(new2))
    graph.replay()
    assert pgd.get_device_error() == pgd.OK
    want = ref.assign_pages(table2, cached2, new2, free, tokens, total)
    for got, w in zip((t2,) + tuple(a), want):
        np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


def test_rejects_wrong_tensors():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    kw = dict(num_tokens=4, num_pages=9)
    with pytest.raises(ValueError):
        pgd.assign_pages(i(2, 3), i(3), i(3), i(4), **kw)
    with pytest.raises(ValueError):
        pgd.assign_pages(i(2, 3).long(), i(2), i(2), i(4), **kw)
    with pytest.raises(ValueError):
        pgd.assign_pages(i(3, 2).T, i(2), i(2), i(4), **kw)
    c = i(2)
    with pytest.raises(pgd.PgdError):   # the length written over the one read
        plan = pgd.PagePlan(i(4), i(4), i(4), i(3), c, i(1))
        pgd.assign_pages(i(2, 3), c, i(2), i(4), out=plan, **kw)
    with pytest.raises(ValueError):
        pgd.assign_pages(i(2, 3), c, i(2), i(4), out=pgd.PagePlan(i(3), i(4), i(4), i(3), i(2),
                                                                  i(1)), **kw)
