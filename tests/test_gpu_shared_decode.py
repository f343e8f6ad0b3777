"""Decode over shared pages against the plain 64-bit attention of each row over its own
table entries, within the bound of page_side."""
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


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(DEV)


class Batch:
    """Groups of rows over shared pages.  groups: (rows, shared pages) in order, with
    shared None for rows in no group (at the start or the end only); own: positions of
    each row's own (0: an inactive row).  Pool positions out of use hold NaN."""

    def __init__(self, seed, groups, own, hq, hkv, d, layout=pgd.PAGE_MAJOR, width=None,
                 scale_k=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.layout = hq, hkv, d, layout
        rows = len(own)
        own = np.asarray(own)
        shared = np.concatenate([np.full(n, p or 0) for n, p in groups]).astype(int)
        need = side.pages_of(own)
        self.positions = np.where(own > 0, shared * 64 + own - 1, -1)
        self.width = width or max(1, int((shared + need).max()))
        self.pages = int(need.sum()) + sum(p or 0 for _, p in groups) + 3
        order = list(rng.permutation(self.pages))
        self.table = np.full((rows, self.width), 2 ** 30)       # entries out of use: any value
        self.starts, self.shared, b = [], [], 0
        for n, p in groups:
            if p is not None:
                if not self.starts:
                    self.starts.append(b)
                self.starts.append(b + n)
                self.shared.append(p)
                pages = [order.pop() for _ in range(p)]
                self.table[b:b + n, :p] = pages
            for r in range(b, b + n):
                for e in range(need[r]):
                    self.table[r, shared[r] + e] = order.pop()
            b += n
        assert b == rows
        g = torch.Generator().manual_seed(seed)
        shape = (self.pages, hkv, 64, d)
        self.k = (torch.randn(shape, generator=g) * scale_k).bfloat16()
        self.v = torch.randn(shape, generator=g).bfloat16()
        used = np.zeros((self.pages, 64), dtype=bool)
        for r, n in enumerate(self.positions):
            for s in range(0, n + 1, 64):
                used[self.table[r, s // 64], :min(64, n + 1 - s)] = True
        gone = torch.from_numpy(~used)
        for pool in (self.k, self.v):
            pool.permute(0, 2, 1, 3)[gone] = float("nan")
        self.q = torch.randn(rows, hq, d, generator=g).bfloat16()
        self.gen = g
        self.k_pool, self.v_pool = self.lay(self.k), self.lay(self.v)

    def lay(self, pool):
        return (pool if self.layout == pgd.PAGE_MAJOR else pool.transpose(0, 1)).contiguous().to(DEV)

    def want(self, scale, sinks=None):
        host = lambda t: t.double().numpy()  # noqa: E731
        return side.attention(host(self.q), host(self.k), host(self.v), self.table,
                              self.positions, scale, sinks)

    def call(self, k_new=None, v_new=None, **kw):
        args = (dev(self.table), dev(self.positions))
        kw = dict(dict(num_kv_heads=self.hkv, layout=self.layout, group_starts=dev(self.starts or [0]),
                       group_pages=dev(self.shared),
                       kernel=pgd.KERNEL_PREFILL_UMMA), **kw)
        if k_new is None:
            return pgd.paged_decode_attention(self.q.to(DEV), self.k_pool, self.v_pool, *args, **kw)
        return pgd.paged_decode_step(self.q.to(DEV), k_new, v_new, self.k_pool, self.v_pool, *args,
                                     **kw)

    def check(self, scale=None, sinks=None, status=pgd.OK, bad=(), **kw):
        out = self.call(scale=scale, sinks=None if sinks is None else dev(sinks, np.float32), **kw)
        assert pgd.get_device_error() == status
        self.compare(out, scale or self.d ** -0.5, sinks, bad)
        return out

    def compare(self, out, scale, sinks=None, bad=()):
        want, mass, size, every = self.want(scale, sinks)
        for b in bad:
            want[b] = 0
        limit = side.bound(want, mass, size, every, self.d)
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got)), "non-finite output"
        excess = np.abs(got - want) - limit
        at = np.unravel_index(np.argmax(excess), excess.shape)
        assert excess.max() <= 0, f"at {at}: {got[at]} for {want[at]}, bound {limit[at]}"


HEADS = [(14, 2, 64), (64, 8, 64), (32, 8, 128), (8, 8, 128), (16, 8, 64), (3, 1, 128), (6, 2, 128),
         (5, 1, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("layout", [pgd.PAGE_MAJOR, pgd.HEAD_MAJOR])
def test_groups_of_all_sizes(hq, hkv, d, layout):
    rng = np.random.default_rng(hq + d)
    groups = [(2, None), (4, 5), (1, 3), (17, 2), (0, 4), (70, 1), (3, 0), (5, 7), (2, None)]
    rows = sum(n for n, _ in groups)
    own = rng.integers(1, 200, rows)
    own[::9] = rng.integers(1, 3, len(own[::9]))
    own[5], own[7], own[40] = 64, 65, 0
    b = Batch(1, groups, own, hq, hkv, d, layout)
    b.check()
    b.check(sinks=rng.normal(size=hq))


@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (32, 8, 128)])
def test_one_token_and_one_page(hq, hkv, d):
    for groups, own in (([(1, 1)], [1]), ([(1, 0)], [1]), ([(1, None)], [1]), ([(2, 1)], [64, 1]),
                        ([(4, 4)], [1, 30, 2, 40]), ([(3, 2)], [0, 0, 0]), ([(3, 2)], [0, 5, 0])):
        Batch(2, groups, own, hq, hkv, d).check()


def test_no_groups():
    Batch(3, [(9, None)], np.arange(1, 900, 100), 32, 8, 128).check(sinks=np.zeros(32))


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 64), (32, 8, 128), (14, 2, 64)])
def test_long_prefix_under_many_rows(hq, hkv, d):
    rng = np.random.default_rng(4)
    Batch(4, [(150, 40)], rng.integers(1, 300, 150), hq, hkv, d).check(sinks=rng.normal(size=hq))


def test_long_prefix_under_few_rows():
    Batch(5, [(3, 900), (2, 1)], [1, 100, 64, 3, 500], 16, 8, 64).check()


def test_long_own_parts():
    Batch(6, [(2, 3), (3, None)], [9000, 1, 20000, 7, 12345], 32, 8, 128).check()


def test_many_small_groups():
    rng = np.random.default_rng(7)
    groups = [(int(n), int(p)) for n, p in zip(rng.integers(0, 5, 150), rng.integers(0, 9, 150))]
    Batch(7, groups, rng.integers(0, 150, sum(n for n, _ in groups)), 16, 8, 64).check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 3.0])
def test_scales(scale):
    b = Batch(8, [(5, 6), (3, None)], [1, 70, 128, 5, 200, 3, 64, 90], 32, 8, 128)
    out = b.call(scale=scale)
    b.compare(out, scale)


def test_scores_that_rise_and_fall_over_the_pages():
    """The running maximum is raised again and again, in the shared pages and after them."""
    for rising in (True, False):
        b = Batch(9, [(6, 30), (2, None)], [500, 1, 64, 300, 90, 70, 2000, 1], 32, 8, 128)
        key = b.k.float().numpy()
        for r, n in enumerate(b.positions):
            for j in range(n // 64 + 1):
                far = j if rising else n // 64 - j
                key[b.table[r, j], :, :, 0] = 4.0 * far
        b.k = torch.from_numpy(key).bfloat16()
        gone = torch.isnan(b.v)
        b.k[gone] = float("nan")
        b.k_pool = b.lay(b.k)
        b.q[:, :, 0] = 8.0
        b.check()


def test_equal_keys_give_the_mean():
    b = Batch(10, [(40, 10)], [64] * 40, 8, 8, 128)
    b.q[:] = 0
    b.check()


def test_a_row_of_nan_stays_in_its_row():
    b = Batch(11, [(70, 3), (1, None)], [30] * 71, 32, 8, 128)
    b.q[33, 5] = float("nan")
    out = b.call()
    assert pgd.get_device_error() == pgd.OK
    assert bool(torch.isnan(out[33, 5]).all())
    got = out.clone()
    got[33, 5] = 0
    b.q[33, 5] = 0
    want, mass, size, every = b.want(128 ** -0.5)
    want[33, 5] = 0
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= side.bound(want, mass, size, every, 128))


@pytest.mark.parametrize("hq,hkv,d,layout", [(14, 2, 64, pgd.PAGE_MAJOR), (32, 8, 128, pgd.HEAD_MAJOR),
                                             (8, 8, 128, pgd.PAGE_MAJOR)])
def test_step_appends_first(hq, hkv, d, layout):
    own = [1, 64, 65, 128, 2, 0, 300, 1, 63]
    b = Batch(12, [(7, 4), (2, None)], own, hq, hkv, d, layout)
    k_new, v_new = (torch.randn(9, hkv, d, generator=b.gen).bfloat16() for _ in range(2))
    for r, n in enumerate(b.positions):
        page, s = (b.table[r, n // 64], n % 64) if n >= 0 else (0, 0)
        if n >= 0:
            b.k[page, :, s], b.v[page, :, s] = k_new[r], v_new[r]
    # the pools still hold other values at the new positions
    out = b.call(k_new.to(DEV), v_new.to(DEV))
    assert pgd.get_device_error() == pgd.OK
    b.compare(out, d ** -0.5)
    for pool, host in ((b.k_pool, b.k), (b.v_pool, b.v)):
        assert torch.equal(pool.view(torch.int16), b.lay(host).view(torch.int16))


def test_the_same_as_without_groups():
    """Grouped and ungrouped calls agree within two roundings and the bound's."""
    b = Batch(13, [(20, 9), (4, 2)], np.arange(1, 25) * 7, 64, 8, 64)
    b.check()
    plain = pgd.paged_decode_attention(b.q.to(DEV), b.k_pool, b.v_pool, dev(np.where(
        b.table < b.pages, b.table, 0)), dev(b.positions), num_kv_heads=8)
    b.compare(plain, 64 ** -0.5)


def test_equal_calls_give_equal_bits():
    b = Batch(14, [(50, 20), (9, 3)], np.arange(1, 60) * 5, 32, 8, 128)
    outs = [b.call() for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ----------------------------------------------------------------- device errors

def test_a_page_outside_the_pool():
    b = Batch(15, [(4, 6), (3, 2), (2, None)], [90] * 9, 32, 8, 128)
    b.table[4:7, 1] = b.pages                     # of the second group
    b.table[1, 7] = -1                            # of row 1's own pages
    args = dict(status=pgd.EDEVICE_BOUNDS, bad=(1, 4, 5, 6))
    keep, b.want = b.want, None
    good = Batch(15, [(4, 6), (3, 2), (2, None)], [90] * 9, 32, 8, 128)
    b.want = good.want
    b.check(**args)
    b.want = keep


def test_rows_beyond_their_table_or_in_their_groups_pages():
    b = Batch(16, [(4, 3), (2, None)], [90] * 6, 32, 8, 128)
    good = b.want
    true = b.positions.copy()
    b.positions = true.copy()
    b.positions[1] = b.width * 64                 # beyond the table
    b.positions[2] = 3 * 64 - 1                   # in the shared pages

    def want(scale, sinks=None):
        at, b.positions = b.positions, true
        r = good(scale, sinks)
        b.positions = at
        return r
    b.want = want
    b.check(status=pgd.EDEVICE_BOUNDS, bad=(1, 2))


@pytest.mark.parametrize("starts,pages,bad", [
    ([0, 4, 3, 6], [3, 3, 3], range(6)),           # decreasing
    ([0, 4, 6, 7], [3, 0, 0], range(6)),           # past the rows
    ([-1, 4, 4, 6], [3, 0, 0], range(6)),
    ([0, 4, 5, 6], [3, -1, 0], [4]),
    ([0, 4, 5, 6], [3, 0, 1000], [5]),
])
def test_bad_groups(starts, pages, bad):
    b = Batch(17, [(4, 3), (2, None)], [90] * 6, 32, 8, 128)
    b.starts, b.shared = starts, pages
    b.check(status=pgd.EDEVICE_BOUNDS, bad=bad)


def test_refusals():
    b = Batch(18, [(4, 3)], [90] * 4, 32, 8, 128)
    with pytest.raises(ValueError, match="together"):
        b.call(group_pages=None)
    for kw in (dict(window=64), dict(softcap=30.0), dict(first_key=dev([0] * 4)),
               dict(alibi_slopes=torch.zeros(32, device=DEV))):
        with pytest.raises(ValueError, match="full attention"):
            b.call(**kw)
    with pytest.raises(ValueError, match="library's"):
        b.call(pages_per_split=4)
    for kernel, status in ((pgd.KERNEL_CUDA_CORE, pgd.EUNSUPPORTED), (9, pgd.EINVAL)):
        with pytest.raises(pgd.PgdError) as e:
            b.call(kernel=kernel)
        assert e.value.status == status
    with pytest.raises(ValueError, match=r"\[S"):
        b.call(group_starts=dev([0, 2, 4]))
    with pytest.raises(ValueError, match="int32"):
        b.call(group_pages=dev([3]).long())
    with pytest.raises(pgd.PgdError) as e:
        b.call(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == pgd.EWORKSPACE
    with pytest.raises(pgd.PgdError) as e:
        b.call(layout=pgd.ROW_MAJOR)
    assert e.value.status in (pgd.EUNSUPPORTED, pgd.EINVAL)
    assert pgd.get_device_error() == pgd.OK


def test_captured_with_changing_groups():
    """One graph, replayed over other tables, positions, groups and values."""
    rows, hq, hkv, d, pages, width = 24, 32, 8, 128, 400, 30
    t = torch.zeros(rows, width, dtype=torch.int32, device=DEV)
    n, starts, shared = (torch.zeros(k, dtype=torch.int32, device=DEV) for k in (rows, 4, 3))
    q = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=DEV)
    kp, vp = (torch.zeros(pages, hkv, 64, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.empty_like(q)
    call = lambda: pgd.paged_decode_attention(  # noqa: E731
        q, kp, vp, t, n, num_kv_heads=hkv, out=out, group_starts=starts, group_pages=shared,
        kernel=pgd.KERNEL_PREFILL_UMMA)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    rng = np.random.default_rng(19)
    for step in range(4):
        cut = np.sort(rng.integers(0, rows + 1, 2))
        groups = [(int(cut[0]), 5), (int(cut[1] - cut[0]), int(rng.integers(0, 12))),
                  (int(rows - cut[1]), 1)]
        b = Batch(20 + step, groups, rng.integers(0, 400, rows), hq, hkv, d, width=width)
        t.copy_(dev(b.table))
        n.copy_(dev(b.positions))
        starts.copy_(dev(b.starts))
        shared.copy_(dev(b.shared))
        q.copy_(b.q)
        kp[:b.pages], vp[:b.pages] = b.k_pool, b.v_pool
        graph.replay()
        assert pgd.get_device_error() == pgd.OK
        b.compare(out, d ** -0.5)


def test_on_a_side_stream():
    b = Batch(21, [(30, 8)], np.arange(1, 31) * 9, 64, 8, 64)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    outs = [b.call(stream=stream) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(stream)
    assert pgd.get_device_error(stream) == pgd.OK
    for out in outs:
        b.compare(out, 64 ** -0.5)


def test_more_rows_and_groups_than_threads():
    """A thread of the cut sums several items; odd counts of everything."""
    rng = np.random.default_rng(30)
    groups = [(1, None)] + [(int(n), int(p)) for n, p in zip(rng.integers(0, 9, 301),
                                                            rng.integers(0, 4, 301))] + [(2, None)]
    own = rng.integers(0, 130, sum(n for n, _ in groups))
    assert len(own) > 1000
    b = Batch(30, groups, own, 3, 1, 64)
    b.check(sinks=rng.normal(size=3))
    b.starts[7] = b.starts[8] + 1                 # decreasing, seen by every thread
    b.check(status=pgd.EDEVICE_BOUNDS, bad=range(len(own)))


def test_inactive_rows_may_hold_anything():
    """The first rows of groups and of blocks among them, their table entries out of the pool."""
    own = np.full(180, 50)
    own[:3] = own[64:100] = own[150:153] = 0
    own[160:170] = 0                               # a whole group
    b = Batch(31, [(150, 5), (10, 3), (10, 4), (10, 2)], own, 32, 8, 128)
    b.table[np.asarray(own) == 0] = -5
    b.check()
    own = np.full(40, 70)
    own[:39] = 0
    b = Batch(32, [(40, 6)], own, 14, 2, 64)
    b.table[:39] = 2 ** 30
    b.check()


@pytest.mark.parametrize("kernel", [pgd.KERNEL_AUTO, pgd.KERNEL_TENSOR_CORE])
def test_row_by_row(kernel):
    """Small calls by AUTO, any by choice: the rows' own table entries, the step among them."""
    groups = [(2, None), (4, 5), (1, 3), (9, 2), (1, None)]
    own = np.arange(17) * 13 % 150 + 1
    own[4] = 0
    for hq, hkv, d in ((14, 2, 64), (16, 4, 128)):
        b = Batch(33, groups, own, hq, hkv, d)
        b.check(sinks=np.linspace(-1, 1, hq), kernel=kernel)
        k_new, v_new = (torch.randn(17, hkv, d, generator=b.gen).bfloat16() for _ in range(2))
        for r, n in enumerate(b.positions):
            if n >= 0:
                page = b.table[r, n // 64]
                b.k[page, :, n % 64], b.v[page, :, n % 64] = k_new[r], v_new[r]
        out = b.call(k_new.to(DEV), v_new.to(DEV), kernel=kernel)
        assert pgd.get_device_error() == pgd.OK
        b.compare(out, d ** -0.5)
        assert torch.equal(b.k_pool.view(torch.int16), b.lay(b.k).view(torch.int16))
    # the groups are not looked at
    b.starts, b.shared = [9, 3], [1000]
    b.check(kernel=kernel)


def test_auto_goes_by_the_tables_pages():
    """The same rows in a table of 128 MB of pages and in one a page wider."""
    rows, hkv, d = 32, 8, 64
    width = (128 << 20) // (rows * hkv * 64 * d * 4)
    for more in (0, 1):
        b = Batch(34, [(rows, 3)], np.arange(1, rows + 1) * 7, 16, hkv, d, width=width + more)
        auto, umma, single = (b.call(kernel=k) for k in (pgd.KERNEL_AUTO, pgd.KERNEL_PREFILL_UMMA,
                                                        pgd.KERNEL_TENSOR_CORE))
        assert torch.equal(auto, umma if more else single)
        b.compare(auto, d ** -0.5)


@pytest.mark.parametrize("at", [0, 16])
def test_a_workspace_at_any_16_bytes(at):
    b = Batch(35, [(5, 3), (70, 2)], np.arange(1, 76) * 5, 32, 8, 128)
    dims = pgd.make_dims(rows=75, num_q_heads=32, num_kv_heads=8, head_dim=128,
                         num_pages=b.k.shape[0], max_pages_per_row=b.table.shape[1])
    need = pgd.shared_decode_workspace_bytes(dims, 2)
    whole = torch.full((need + 64,), 0xa5, dtype=torch.uint8, device=DEV)
    assert whole.data_ptr() % 32 == 0
    b.check(workspace=whole[at:at + need])
    assert (whole[:at] == 0xa5).all() and (whole[at + need:] == 0xa5).all()


@pytest.mark.parametrize("layout", [pgd.PAGE_MAJOR, pgd.HEAD_MAJOR])
def test_pools_past_32_bits_of_bytes_and_values(layout):
    """A small batch's pages at the ends of pools of 2.3e9 values, the step among them."""
    b = Batch(36, [(6, 3), (2, None)], np.arange(1, 9) * 30, 16, 4, 128, layout)
    pages = 70000
    place = np.r_[0:3, pages - (b.pages - 3):pages]        # page i of the batch is page place[i]
    rng = np.random.default_rng(1)
    place = rng.permutation(place)
    big = [torch.zeros(pages, 4, 64, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    k_new, v_new = (torch.randn(8, 4, 128, generator=b.gen).bfloat16() for _ in range(2))
    views = [x if layout == pgd.PAGE_MAJOR else x.view(4, pages, 64, 128).transpose(0, 1) for x in big]
    for view, small in zip(views, (b.k, b.v)):
        view[torch.from_numpy(place).to(DEV)] = small.to(DEV)
    for r, n in enumerate(b.positions):
        page = b.table[r, n // 64]
        b.k[page, :, n % 64], b.v[page, :, n % 64] = k_new[r], v_new[r]
    table = np.where(b.table < b.pages, place[np.minimum(b.table, b.pages - 1)], -1)
    out = pgd.paged_decode_step(
        b.q.to(DEV), k_new.to(DEV), v_new.to(DEV), *big, dev(table), dev(b.positions), num_kv_heads=4,
        layout=layout, group_starts=dev(b.starts), group_pages=dev(b.shared),
        kernel=pgd.KERNEL_PREFILL_UMMA)
    assert pgd.get_device_error() == pgd.OK
    b.compare(out, 128 ** -0.5)
    for view, small in zip(views, (b.k, b.v)):
        got = view[torch.from_numpy(place).to(DEV)].cpu()
        assert torch.equal(got.view(torch.int16), small.view(torch.int16))


def test_two_calls_at_once():
    """Captured steps of two batches, each with its own workspace, replayed on two streams."""
    batches = [Batch(37, [(200, 40), (9, 3)], np.arange(209) * 7 % 300 + 1, 32, 8, 128),
               Batch(38, [(3, 30)] * 20, np.arange(60) * 11 % 200 + 1, 64, 8, 64)]
    runs = []
    for b in batches:
        args = (b.q.to(DEV), b.k_pool, b.v_pool, dev(b.table), dev(b.positions))
        kw = dict(num_kv_heads=b.hkv, group_starts=dev(b.starts), group_pages=dev(b.shared),
                  kernel=pgd.KERNEL_PREFILL_UMMA)
        want = pgd.paged_decode_attention(*args, **kw)
        b.compare(want, b.d ** -0.5)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(5):
                out = pgd.paged_decode_attention(*args, **kw)
        runs.append((graph, stream, out, want, args, kw))
    for _ in range(10):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, _, _ in runs:
        assert torch.equal(out, want)
    assert pgd.get_device_error() == pgd.OK
