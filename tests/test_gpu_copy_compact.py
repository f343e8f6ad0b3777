"""copy_pages and compact_pages against plain models: copies and whole numbers, equal
to the last bit, whatever the values are (NaN patterns among them)."""
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


# ----------------------------------------------------------------- copy_pages

def pools(rng, layers, pages, hkv, d):
    """Any bits, page-major [pages, Hkv, 64, D], as int16 on the host."""
    return [rng.integers(-2 ** 15, 2 ** 15, (pages, hkv, 64, d), dtype=np.int16)
            for _ in range(2 * layers)]


def lay(pool, layout):
    p = pool if layout == pgd.PAGE_MAJOR else np.ascontiguousarray(pool.transpose(1, 0, 2, 3))
    return torch.from_numpy(p).to(DEV).view(torch.bfloat16)


def check_copy(rng, layers, pages, hkv, d, layout, sources, targets, counts, status=pgd.OK):
    host = pools(rng, layers, pages, hkv, d)
    on = [lay(p, layout) for p in host]
    pgd.copy_pages(on[:layers], on[layers:], dev(sources), dev(targets),
                   None if counts is None else dev(counts), num_kv_heads=hkv, head_dim=d,
                   layout=layout)
    assert pgd.get_device_error() == status
    for p, got in zip(host, on):
        for i, (a, b) in enumerate(zip(sources, targets)):
            n = 64 if counts is None else counts[i]
            if min(a, b) >= 0 and max(a, b) < pages and 0 <= n <= 64:
                p[b, :, :n] = p[a, :, :n]
        want = p if layout == pgd.PAGE_MAJOR else p.transpose(1, 0, 2, 3)
        np.testing.assert_array_equal(got.view(torch.int16).cpu().numpy(), want)


@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (1, 128), (3, 64)])
@pytest.mark.parametrize("layout", [pgd.PAGE_MAJOR, pgd.HEAD_MAJOR])
@pytest.mark.parametrize("layers,copies", [(1, 1), (3, 7), (2, 50)])
@pytest.mark.parametrize("partial", [False, True])
def test_copies(hkv, d, layout, layers, copies, partial):
    rng = np.random.default_rng(layers * 100 + copies)
    pages = 2 * copies + 3
    order = rng.permutation(pages)
    counts = rng.integers(0, 65, copies) if partial else None
    sources, targets = order[:copies].copy(), order[copies:2 * copies].copy()
    if copies > 5:
        sources[3] = targets[3] = -1     # a row without a copy
        sources[4] = sources[0]          # a page copied twice
    check_copy(rng, layers, pages, hkv, d, layout, sources, targets, counts)


def test_more_layers_than_a_launch_takes():
    rng = np.random.default_rng(1)
    check_copy(rng, 67, 4, 1, 64, pgd.PAGE_MAJOR, [0, 3], [1, 2], [64, 5])


def test_no_copies_and_no_layers():
    rng = np.random.default_rng(1)
    check_copy(rng, 1, 4, 1, 64, pgd.PAGE_MAJOR, [], [], None)
    pgd.copy_pages([], [], dev([1]), dev([2]), num_kv_heads=1, head_dim=64)
    one = lay(pools(rng, 1, 2, 2, 64)[0], pgd.PAGE_MAJOR)
    pgd.copy_pages(one, one.clone(), dev([0]), dev([1]), num_kv_heads=2, head_dim=64)
    assert torch.equal(one[0].view(torch.int16), one[1].view(torch.int16))


def test_pages_and_counts_out_of_range_are_left_out():
    rng = np.random.default_rng(2)
    check_copy(rng, 2, 6, 2, 64, pgd.PAGE_MAJOR, [0, 6, 1, 2, -1], [3, 4, 2 ** 31 - 1, 5, 1],
               [64, 64, 64, 64, 64], status=pgd.EDEVICE_BOUNDS)
    check_copy(rng, 2, 6, 2, 64, pgd.HEAD_MAJOR, [0, 1, 2], [3, 4, 5], [65, -1, 64],
               status=pgd.EDEVICE_BOUNDS)


def test_a_pool_past_32_bits_of_bytes_and_values():
    pages = 70000                                  # 4.6 GB a pool, 2.3e9 values
    k = torch.zeros(pages, 4, 64, 128, dtype=torch.bfloat16, device=DEV)
    for layout, at in ((pgd.PAGE_MAJOR, lambda p, h: (p * 4 + h) * 64),
                       (pgd.HEAD_MAJOR, lambda p, h: (h * pages + p) * 64)):
        flat = k.view(-1, 128)
        flat.zero_()
        a, b = pages - 1, pages - 2
        for h in range(4):
            flat[at(a, h):at(a, h) + 64] = h + 1.0
        pgd.copy_pages(k, k, dev([a]), dev([b]), dev([63]), num_kv_heads=4, head_dim=128,
                       layout=layout)
        for h in range(4):
            assert bool((flat[at(b, h):at(b, h) + 63] == h + 1).all())
            assert not flat[at(b, h) + 63].any()
    assert pgd.get_device_error() == pgd.OK


def test_copy_refusals():
    p = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16, device=DEV)
    kw = dict(num_kv_heads=2, head_dim=64)
    with pytest.raises(ValueError, match="same layers"):
        pgd.copy_pages([p, p], [p], dev([0]), dev([1]), **kw)
    with pytest.raises(ValueError, match="one shape"):
        pgd.copy_pages([p, p], [p, p[:2]], dev([0]), dev([1]), **kw)
    with pytest.raises(ValueError, match="bfloat16"):
        pgd.copy_pages(p, p.half(), dev([0]), dev([1]), **kw)
    with pytest.raises(ValueError, match=r"\[n\]"):
        pgd.copy_pages(p, p, dev([0]), dev([1, 2]), **kw)
    with pytest.raises(ValueError, match="whole number"):
        pgd.copy_pages(p, p, dev([0]), dev([1]), num_kv_heads=3, head_dim=64)
    for bad, status in ((dict(head_dim=32), pgd.EUNSUPPORTED), (dict(layout=pgd.ROW_MAJOR), pgd.EUNSUPPORTED)):
        with pytest.raises(pgd.PgdError) as e:
            pgd.copy_pages(p, p, dev([0]), dev([1]), **dict(kw, **bad))
        assert e.value.status == status


# ----------------------------------------------------------------- compact_pages

def check_compact(table, lengths, shares, free, head, pages, moves, in_place=False,
                  pass_head=True):
    t, n, s, f = dev(table), dev(lengths), dev(shares), dev(free)
    out = None
    if in_place:
        empty = lambda k: torch.full((k,), 99, dtype=torch.int32, device=DEV)  # noqa: E731
        out = pgd.CompactPlan(t, s, f, empty(moves), empty(moves), empty(1))
    kept = [x.clone() for x in (t, s, f)]
    plan = pgd.compact_pages(t, n, s, f, free_head=dev([head]) if pass_head else None,
                             max_moves=moves, out=out)
    status = pgd.get_device_error()
    limit = pages // 2 if moves is None else moves
    want = side.compact_pages(np.asarray(table), lengths, shares, free, head if pass_head else 0,
                              pages, limit)
    assert status == (pgd.EDEVICE_BOUNDS if want[-1] is None else pgd.OK)
    for name, got, w in zip(pgd.CompactPlan._fields, plan, want):
        if w is not None:
            np.testing.assert_array_equal(got.cpu().numpy().reshape(-1),
                                          np.asarray(w).reshape(-1), err_msg=name)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(kept, (t, s, f)))
    return plan


@pytest.mark.parametrize("requests,beams,hi,spare", [
    (1, 1, 100, 0), (4, 3, 800, 40), (60, 2, 500, 1000), (2, 1, 40, 31), (300, 4, 700, 37), (5, 5, 0, 3),
])
@pytest.mark.parametrize("moves", [None, 0, 1, 7, 500])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(requests, beams, hi, spare, moves, in_place):
    if in_place and moves is None:
        pytest.skip("an own plan says how many moves")
    rng = np.random.default_rng(requests + spare)
    table, lengths, shares, free, head, pages = side.random_state(rng, requests, beams, hi, 50,
                                                                  spare=spare)
    # pages of the user's own: neither listed nor held
    listed = np.concatenate([free[:head], rng.permutation(free[head:])[:max(0, pages - head - 3)]])
    check_compact(table, lengths, shares, listed, head, pages, moves, in_place)


def test_compact_already_and_full_and_empty():
    table = np.array([[0, 1, 2], [3, 1, 9]])
    shares = np.array([0, 1, 0, 0, 0, 0, 0, 0])
    check_compact(table, np.array([192, 128]), shares, np.arange(8), 4, 8, None)
    check_compact(table, np.array([192, 128]), shares[:4], np.arange(4), 4, 4, 2)   # none free
    check_compact(table, np.array([0, 0]), np.zeros(8), np.arange(8)[::-1], 0, 8, 4)  # none held
    check_compact(table[:0], np.array([], dtype=int), np.zeros(8), np.arange(8), 2, 8, 4)
    # all held pages above all free ones, and the pool's last page
    check_compact(np.array([[7, 6], [5, 6]]), np.array([65, 128]), np.array([0] * 6 + [1, 0]),
                  np.array([9, 3, 1, 4, 0, 2]), 1, 8, 4)
    check_compact(np.array([[7]]), np.array([1]), np.zeros(8), np.array([3]), 0, 8, 4,
                  pass_head=False)


@pytest.mark.parametrize("pages", [31, 32, 33, 1023, 1024, 1025, 32769])
def test_compact_at_the_bitmaps_borders(pages):
    rng = np.random.default_rng(pages)
    order = rng.permutation(pages)
    held = pages // 3
    width = 11
    rows = -(-held // width)
    table = np.full((rows, width), -1)
    table.reshape(-1)[:held] = order[:held]
    lengths = np.full(rows, 64 * width)
    lengths[-1] = 64 * (held - (rows - 1) * width)
    check_compact(table, lengths, np.zeros(pages), order, held, pages, None)
    check_compact(table, lengths, np.zeros(pages), order, held, pages, held // 2 + 1, True)


def test_compact_a_large_pool():
    """More words than prefixes in shared memory: several words a prefix."""
    pages = 2_500_003
    rng = np.random.default_rng(1)
    order = rng.permutation(pages)
    held = 5000
    table = order[:held].reshape(50, 100)
    check_compact(table, np.full(50, 6400), np.zeros(pages), order, held, pages, 6000)


@pytest.mark.parametrize("what", ["length", "negative", "entry", "listed", "twice", "both", "head"])
def test_nothing_moves_where_the_state_is_wrong(what):
    rng = np.random.default_rng(3)
    table, lengths, shares, free, head, pages = side.random_state(rng, 4, 2, 600, 50, spare=30)
    table, lengths, free = table.copy(), lengths.copy(), free.copy()
    if what == "length":
        lengths[2] = table.shape[1] * 64 + 1
    elif what == "negative":
        lengths[2] = -1
    elif what == "entry":
        lengths[3] = max(lengths[3], 1)
        table[3, 0] = pages
    elif what == "listed":
        free[head + 1] = -1
    elif what == "twice":
        free[head + 1] = free[head + 4]
    elif what == "both":
        free[-1] = table[int(np.argmax(lengths)), 0]
    else:
        head = len(free) + 1
    check_compact(table, lengths, shares, free, head, pages, 20)
    check_compact(table, lengths, shares, free, head, pages, 20, True)


def test_compact_refusals():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    good = dict(table=i(2, 3), lengths=i(2), shares=i(9), free_pages=i(5))
    for name, bad in (("lengths", i(3)), ("shares", i(3, 3)), ("free_pages", i(5, 1)), ("table", i(6))):
        with pytest.raises(ValueError, match="shapes"):
            pgd.compact_pages(**dict(good, **{name: bad}))
    with pytest.raises(ValueError, match="max_moves"):
        pgd.compact_pages(**good, max_moves=-1)
    with pytest.raises(ValueError, match="out.sources"):
        pgd.compact_pages(**good, max_moves=3, out=pgd.CompactPlan(i(2, 3), i(9), i(5), i(2), i(3), i(1)))
    with pytest.raises(pgd.PgdError) as e:   # sources over the lengths
        pgd.compact_pages(**good, max_moves=2,
                          out=pgd.CompactPlan(i(2, 3), i(9), i(5), good["lengths"], i(2), i(1)))
    assert e.value.status == pgd.EINVAL
    assert pgd.get_device_error() == pgd.OK


@pytest.mark.parametrize("moves", [0, 5, 30000, None])
def test_compact_on_all_sms(moves):
    """More entries and pages than one cluster takes, then the same state gone wrong."""
    rng = np.random.default_rng(5)
    table, lengths, shares, free, head, pages = side.random_state(rng, 300, 4, 9000, 300,
                                                                  spare=20000)
    assert table.size + pages > 100000
    check_compact(table, lengths, shares, free, head, pages, moves)
    if moves is not None:
        check_compact(table, lengths, shares, free, head, pages, moves, True)
        twice = free.copy()
        twice[-1] = twice[-9]
        check_compact(table, lengths, shares, twice, head, pages, moves, True)


def test_large_pools_on_two_streams_and_replayed():
    rng = np.random.default_rng(6)
    runs = []
    for k in range(2):
        table, lengths, shares, free, head, pages = side.random_state(rng, 200, 4, 9000, 300,
                                                                      spare=20000)
        assert table.size + pages > 100000
        args = tuple(dev(a) for a in (table, lengths, shares, free))
        h = dev([head])
        want = check_compact(table, lengths, shares, free, head, pages, 4000)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            plan = pgd.compact_pages(*args, free_head=h, max_moves=4000)
        runs.append((graph, stream, plan, want, args, h))
    for _ in range(10):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, plan, want, _, _ in runs:
        for a, b in zip(plan, want):
            assert torch.equal(a, b)
    assert pgd.get_device_error() == pgd.OK
