"""fork_rows against the plain row-by-row model: every output is a whole number and
has to be equal, entries out of use included."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import page_side as side

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


def check(state, parents, keep=None, status=None, out=None, pass_head=True):
    table, lengths, shares, free, head, pages = state
    t, n, q, s, f = dev(table), dev(lengths), dev(parents), dev(shares), dev(free)
    k = None if keep is None else dev(keep)
    plan = pgd.fork_rows(t, n, q, s, f, free_head=dev([head]) if pass_head else None, keep=k,
                         out=out)
    got_status = pgd.get_device_error()
    want, error = side.fork_rows(np.asarray(table), lengths, parents, keep, shares, free,
                                 head if pass_head else 0, pages)
    names = ("table", "shares", "free_pages") + pgd.ForkPlan._fields
    for name, got, w in zip(names, (t, s, f) + tuple(plan), want):
        np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1),
                                      err_msg=name)
    assert got_status == (pgd.EDEVICE_BOUNDS if error else pgd.OK)
    if status is not None:
        assert got_status == status
    assert torch.equal(n, dev(lengths)) and torch.equal(q, dev(parents))
    # the state afterwards
    return want[0], np.asarray(want[3]), np.asarray(want[1]), np.asarray(want[2]), want[7], pages


@pytest.mark.parametrize("requests,beams,hi,grown", [
    (1, 1, 300, 0), (1, 4, 500, 70), (8, 4, 1500, 200), (3, 7, 64, 64), (5, 5, 63, 1),
    (33, 3, 900, 129), (1, 64, 2000, 0), (300, 4, 400, 90), (1, 1, 0, 0),
])
def test_random_reordering_again_and_again(requests, beams, hi, grown):
    rng = np.random.default_rng(requests * 100 + beams)
    state = side.random_state(rng, requests, beams, hi, grown)
    rows = requests * beams
    for step in range(4):
        first = np.arange(rows) // beams * beams
        parents = first + rng.integers(0, beams, rows)
        keep = None
        if step >= 2:
            parents = np.where(rng.random(rows) < 0.1, -1, parents)
            keep = np.where(rng.random(rows) < 0.3, rng.integers(0, hi + grown + 2, rows), 2 ** 31 - 1)
        state = check(state, parents, keep, status=pgd.OK)
        # pages' holders and the list add up
        table, lengths, shares, free, head, pages = state
        held = np.zeros(pages, dtype=int)
        for r in range(rows):
            at, count = np.unique(table[r, :side.pages_of(lengths[r])], return_counts=True)
            held[at] += count
        assert np.array_equal(np.maximum(held - 1, 0), shares)
        assert sorted(free[head:]) == sorted(np.nonzero(held == 0)[0])


def test_as_it_was():
    """Every row its own parent: nothing moves."""
    rng = np.random.default_rng(3)
    state = side.random_state(rng, 4, 3, 700, 100)
    after = check(state, np.arange(12), status=pgd.OK)
    for a, b in zip(state, after):
        np.testing.assert_array_equal(a, b)


def test_one_row_into_all_and_all_released():
    rng = np.random.default_rng(4)
    state = side.random_state(rng, 40, 1, 900, 1)
    state = check(state, np.full(40, 17), status=pgd.OK)
    state = check(state, np.full(40, -1), status=pgd.OK)
    assert state[4] == 0 and sorted(state[3]) == list(range(state[5]))


@pytest.mark.parametrize("length", [1, 63, 64, 65, 128])
@pytest.mark.parametrize("keep", [0, 1, 63, 64, 65, 127, 128, -5])
def test_cuts_at_page_borders(length, keep):
    """Two rows of one prompt and a third one: one cut, one as it is, one forked and cut."""
    rng = np.random.default_rng(length)
    state = side.random_state(rng, 1, 1, 0, 0, width=3, spare=8)
    table = np.full((3, 3), -7)
    need = side.pages_of(length)
    table[0, :need] = state[3][:need]
    table[1, :length // 64] = state[3][:length // 64]
    state = (table, np.array([length, length // 64 * 64, 0]),
             np.array([(int(p in table[0]) + int(p in table[1]) - 1 if p in table[0] else 0)
                       for p in range(state[5])]), state[3], need, state[5])
    big = 2 ** 31 - 1
    check(state, np.array([0, 1, 0]), np.array([keep, big, big]), status=pgd.OK)
    check(state, np.array([0, 1, 0]), np.array([keep, keep, keep]), status=pgd.OK)
    check(state, np.array([0, 0, 0]), np.array([big, keep, keep]), status=pgd.OK)
    check(state, np.array([2, 0, 1]), np.array([big, keep, big]), status=pgd.OK)


def test_wide_tables_and_many_rows():
    rng = np.random.default_rng(8)
    for requests, beams, hi, grown in ((2, 3, 40000, 300), (1500, 2, 100, 70), (600, 8, 2000, 100)):
        rows = requests * beams
        state = side.random_state(rng, requests, beams, hi, grown)
        parents = np.arange(rows) // beams * beams + rng.integers(0, beams, rows)
        check(state, parents, status=pgd.OK)


def test_the_most_rows():
    rows = 8192
    table = np.zeros((rows, 1), dtype=np.int64)
    table[:, 0] = np.arange(rows)
    lengths = np.full(rows, 64)
    lengths[5] = 9
    parents = np.full(rows, 5)
    t, s = dev(table), dev(np.zeros(rows + 20))
    free = np.concatenate([np.arange(rows), np.arange(rows, rows + 20)])
    f = dev(free)
    plan = pgd.fork_rows(t, dev(lengths), dev(parents), s, f, free_head=dev([rows]))
    # all pages but row 5's come back, in order; rows in order take them again
    assert pgd.get_device_error() == pgd.OK
    want = [p for p in range(rows) if p != 5]
    targets = plan.targets.cpu().numpy()
    assert targets[0] == -1 and list(targets[1:]) == want
    assert torch.equal(plan.lengths.cpu(), torch.full((rows,), 9, dtype=torch.int32))
    assert list(t.cpu().numpy()[:, 0]) == [5] + want
    assert not s.any() and plan.free_head.item() == rows
    bad = torch.zeros(rows + 1, dtype=torch.int32, device=DEV)
    with pytest.raises(pgd.PgdError) as e:
        pgd.fork_rows(bad.view(-1, 1), torch.zeros_like(bad), torch.zeros_like(bad), s, f)
    assert e.value.status == pgd.EUNSUPPORTED


def test_no_rows_and_no_list():
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    plan = pgd.fork_rows(torch.empty(0, 3, dtype=torch.int32, device=DEV), empty, empty,
                         torch.zeros(4, dtype=torch.int32, device=DEV), dev([1, 2]),
                         free_head=dev([1]))
    assert plan.free_head.item() == 1 and pgd.get_device_error() == pgd.OK
    state = side.random_state(np.random.default_rng(1), 2, 2, 300, 20)
    table, lengths, shares, free, head, pages = state
    check((table, lengths, shares, np.array([], dtype=np.int64), 0, pages), np.arange(4),
          status=pgd.OK)


# ----------------------------------------------------------------- device errors

def test_too_few_pages_for_the_copies():
    rng = np.random.default_rng(5)
    table, lengths, shares, free, head, pages = side.random_state(rng, 2, 4, 200, 40)
    for left in (0, 1, 2, 3):
        check((table, lengths, shares, free[:head + left], head, pages),
              np.arange(8) // 4 * 4 + (np.arange(8) % 4 == 3) * 2)


def test_a_list_without_room_below_its_head():
    rng = np.random.default_rng(6)
    table, lengths, shares, free, head, pages = side.random_state(rng, 3, 2, 400, 60)
    check((table, lengths, shares, free[head - 2:], 2, pages), np.full(6, -1),
          status=pgd.EDEVICE_BOUNDS)
    check((table, lengths, shares, free[head:], 0, pages), np.array([0, 0, 2, 2, 4, 4]),
          pass_head=False)


@pytest.mark.parametrize("head", [-1, 10 ** 6])
def test_a_head_outside_its_list(head):
    table, lengths, shares, free, _, pages = side.random_state(np.random.default_rng(7), 3, 2, 400, 60)
    check((table, lengths, shares, free, head, pages), np.array([0, 0, 3, 2, -1, 4]),
          status=pgd.EDEVICE_BOUNDS)


def test_bad_lengths_parents_and_entries():
    state = side.random_state(np.random.default_rng(9), 3, 4, 500, 90)
    table, lengths, shares, free, head, pages = state
    parents = np.array([0, 0, 2, 2, 5, 4, -9, 12, 8, 9, 9, 2 ** 31 - 1])
    check((table, lengths, shares, free, head, pages), parents, status=pgd.EDEVICE_BOUNDS)
    broken = lengths.copy()
    broken[0], broken[6] = -1, 64 * table.shape[1] + 1
    # (pages that only the rows of unknown length held are not given back)
    check((table, broken, shares, free, head, pages), np.arange(12) // 2 * 2,
          status=pgd.EDEVICE_BOUNDS)
    holes = table.copy()
    holes[1, 0], holes[4, 1], holes[9, side.pages_of(lengths[9]) - 1] = -1, pages, 2 ** 31 - 1
    check((holes, lengths, shares, free, head, pages), np.arange(12) // 2 * 2 + 1)


def test_pages_outside_the_pool_on_the_list():
    table, lengths, shares, free, head, pages = side.random_state(np.random.default_rng(2), 1, 6, 300, 0)
    lengths[:] = 300
    free = free.copy()
    free[head], free[head + 2] = pages, -4
    check((table, lengths, shares, free, head, pages), np.zeros(6, dtype=int))


def test_a_page_given_back_more_often_than_held():
    table = np.array([[0, 1], [0, 2], [3, 4]])
    state = (table, np.array([128, 128, 128]), np.zeros(8, dtype=int), np.arange(8), 5, 8)
    # page 0 is held twice, its shares say once
    check(state, np.array([-1, -1, 2]), status=pgd.EDEVICE_BOUNDS)


def test_refusals():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    good = dict(table=i(2, 3), lengths=i(2), parents=i(2), shares=i(9), free_pages=i(5))
    for name, bad in (("lengths", i(3)), ("parents", i(2, 1)), ("shares", i(3, 3)),
                      ("free_pages", i(5, 1)), ("table", i(6))):
        with pytest.raises(ValueError, match="shapes"):
            pgd.fork_rows(**dict(good, **{name: bad}))
    with pytest.raises(ValueError, match="int32"):
        pgd.fork_rows(**dict(good, parents=i(2).long()))
    with pytest.raises(ValueError, match="shapes"):
        pgd.fork_rows(**good, keep=i(3))
    with pytest.raises(ValueError, match="out.targets"):
        pgd.fork_rows(**good, out=pgd.ForkPlan(i(2), i(2), i(3), i(2), i(1)))
    # outputs over inputs
    with pytest.raises(pgd.PgdError) as e:
        pgd.fork_rows(**good, out=pgd.ForkPlan(good["lengths"], i(2), i(2), i(2), i(1)))
    assert e.value.status == pgd.EINVAL
    with pytest.raises(pgd.PgdError) as e:
        pgd.fork_rows(**dict(good, shares=good["table"].view(-1)))
    assert e.value.status == pgd.EINVAL
    assert pgd.get_device_error() == pgd.OK


def test_captured_and_replayed():
    """Beam steps replayed from a graph whose plan feeds the next step."""
    rng = np.random.default_rng(12)
    state = side.random_state(rng, 4, 4, 300, 30)
    state[1][:] = np.repeat(state[1][::4], 4) // 64 * 64   # whole pages: no copies by the first step
    for r in range(16):
        assert side.pages_of(state[1][r]) <= side.pages_of(state[1][r - r % 4])
    table, lengths, _, free, _, pages = state
    shares = np.zeros(pages, dtype=int)
    for r in range(16):
        shares[table[r, :lengths[r] // 64]] += 1
    used = [p for p in range(pages) if shares[p]]
    free = np.array(used + [p for p in range(pages) if not shares[p]])
    state = (table, lengths, np.maximum(shares - 1, 0), free, len(used), pages)
    t, n, s, f, h = (dev(a) for a in (table, lengths, state[2], free, [len(used)]))
    parents = dev(np.zeros(16))
    plan = pgd.ForkPlan(*(torch.empty(k, dtype=torch.int32, device=DEV) for k in (16, 16, 16, 16, 1)))
    side_stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side_stream):
        pgd.fork_rows(t, n, parents, s, f, free_head=h, out=plan)
        n.copy_(plan.lengths)
        h.copy_(plan.free_head)
    for step in range(5):
        chosen = np.arange(16) // 4 * 4 + rng.integers(0, 4, 16)
        parents.copy_(dev(chosen))
        graph.replay()
        want, error = side.fork_rows(state[0], state[1], list(chosen), None, state[2], state[3],
                                     state[4], pages)
        assert not error
        for got, w in zip((t, s, f) + tuple(plan), want):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        state = (want[0], np.asarray(want[3]), np.asarray(want[1]), want[2], want[7], pages)
    assert pgd.get_device_error() == pgd.OK


def test_many_entries_take_all_sms():
    """Past the entries that one cluster takes; then with cuts, releases, too few pages and errors."""
    rng = np.random.default_rng(21)
    for requests, beams, hi, grown in ((40, 8, 9000, 300), (500, 8, 900, 200)):
        rows = requests * beams
        state = side.random_state(rng, requests, beams, hi, grown)
        assert state[0].size > 40000
        for step in range(3):
            parents = np.arange(rows) // beams * beams + rng.integers(0, beams, rows)
            keep = np.where(rng.random(rows) < 0.2, rng.integers(0, hi, rows), 2 ** 31 - 1)
            parents = np.where(rng.random(rows) < 0.05, -1, parents)
            state = check(state, parents, keep if step else None, status=pgd.OK)
    table, lengths, shares, free, head, pages = state
    parents = np.arange(rows) // beams * beams + rng.integers(0, beams, rows)
    few = free[:head + 20]
    check((table, lengths, shares, few, head, pages), parents)
    check((table, lengths, shares, free[head - 3:], 3, pages), np.full(rows, -1),
          status=pgd.EDEVICE_BOUNDS)
    check((table, lengths, shares, free, -7, pages), parents, status=pgd.EDEVICE_BOUNDS)
    holes, wrong = table.copy(), lengths.copy()
    holes[rng.random(table.shape) < 0.01] = pages
    wrong[5] = -1
    parents[17], parents[33] = rows, -2
    check((holes, wrong, shares, free, head, pages), parents, status=pgd.EDEVICE_BOUNDS)


def test_the_most_rows_of_a_large_table():
    rng = np.random.default_rng(22)
    state = side.random_state(rng, 1024, 8, 300, 40, width=9)
    rows = 8192
    assert state[0].shape == (rows, 9)
    for step in range(2):
        parents = np.arange(rows) // 8 * 8 + rng.integers(0, 8, rows)
        keep = np.where(rng.random(rows) < 0.3, rng.integers(0, 300, rows), 2 ** 31 - 1)
        state = check(state, parents, keep, status=pgd.OK)


def test_large_tables_on_two_streams_and_replayed():
    """Calls whose blocks meet, at once and out of a graph."""
    rng = np.random.default_rng(23)
    states = [side.random_state(rng, 60, 8, 5000, 300) for _ in range(2)]
    rows = 480
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for state, stream in zip(states, streams):
        table, lengths, shares, free, head, pages = state
        assert table.size > 20000
        parents = np.arange(rows) // 8 * 8 + rng.integers(0, 8, rows)
        first = tuple(dev(a) for a in (table, shares, free))
        work = tuple(a.clone() for a in first)
        plan = pgd.ForkPlan(*(torch.empty(k, dtype=torch.int32, device=DEV)
                              for k in (rows, rows, rows, rows, 1)))
        args = dev(lengths), dev(parents), dev([head])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for to, a in zip(work, first):
                to.copy_(a)
            pgd.fork_rows(work[0], args[0], args[1], work[1], work[2], free_head=args[2], out=plan)
        want, error = side.fork_rows(table, lengths, list(parents), None, shares, free, head, pages)
        assert not error
        runs.append((graph, stream, work, plan, want, first, args))
    for _ in range(10):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, work, plan, want, _, _ in runs:
        for got, w in zip(work + tuple(plan), want):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    assert pgd.get_device_error() == pgd.OK
