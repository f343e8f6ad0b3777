"""The operators of shared pages together, as a serving loop uses them: prompts in, forked
into beams, steps of assign_pages, paged_decode_step over shared pages, reordering by
fork_rows with copy_pages, rows cut back and released, the pool compacted -- against
rows that keep their whole keys and values on the host."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import page_side as side

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LAYERS = 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Server:
    """Requests of `beams` rows each.  history[layer][row]: (keys, values), [n, Hkv, D]."""

    def __init__(self, seed, prompts, beams, hq, hkv, d, layout, kernel=pgd.KERNEL_PREFILL_UMMA):
        self.kernel = kernel
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.beams, self.hq, self.hkv, self.d, self.layout = beams, hq, hkv, d, layout
        self.prompts, self.requests = np.asarray(prompts), len(prompts)
        self.rows = self.requests * beams
        width = int(side.pages_of(self.prompts).max()) + 4
        self.pages = int(side.pages_of(self.prompts).sum()) + 4 * self.rows + 5
        shape = (self.pages, hkv, 64, d) if layout == pgd.PAGE_MAJOR else (hkv, self.pages, 64, d)
        nan = lambda: torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.k, self.v = [nan() for _ in range(LAYERS)], [nan() for _ in range(LAYERS)]
        self.table = dev(np.full((self.rows, width), 2 ** 29))
        self.lengths = dev(np.zeros(self.rows))
        self.shares = dev(np.zeros(self.pages))
        self.free = dev(self.rng.permutation(self.pages))
        self.head = dev([0])
        self.history = [[(np.zeros((0, hkv, d)),) * 2 for _ in range(self.rows)]
                        for _ in range(LAYERS)]
        self.starts = dev(np.arange(self.requests + 1) * beams)

    def values(self, tokens, heads):
        return torch.randn(tokens, heads, self.d, generator=self.gen).bfloat16().to(DEV)

    def extend(self, layer, rows, k, v):
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        for t, r in enumerate(rows):
            old = self.history[layer][r]
            self.history[layer][r] = (np.concatenate([old[0], k[t:t + 1]]),
                                      np.concatenate([old[1], v[t:t + 1]]))

    def assign(self, new):
        plan = pgd.assign_pages(self.table, self.lengths, dev(new), self.free,
                                num_tokens=int(np.sum(new)), num_pages=self.pages,
                                free_head=self.head)
        self.lengths, self.head = plan.lengths, plan.free_head
        return plan

    def prefill(self):
        """Each request's prompt into its first row."""
        new = np.where(np.arange(self.rows) % self.beams == 0, np.repeat(self.prompts, self.beams), 0)
        plan = self.assign(new)
        rows = np.repeat(np.arange(self.rows), new)
        for layer in range(LAYERS):
            k, v = self.values(len(rows), self.hkv), self.values(len(rows), self.hkv)
            pgd.kv_write_slots(k, v, plan.slots, self.k[layer], self.v[layer], layout=self.layout)
            self.extend(layer, rows, k, v)

    def fork(self, parents, keep=None):
        plan = pgd.fork_rows(self.table, self.lengths, dev(parents), self.shares, self.free,
                             free_head=self.head, keep=None if keep is None else dev(keep))
        pgd.copy_pages(self.k, self.v, plan.sources, plan.targets, plan.counts,
                       num_kv_heads=self.hkv, head_dim=self.d, layout=self.layout)
        self.lengths, self.head = plan.lengths, plan.free_head
        none = (np.zeros((0, self.hkv, self.d)),) * 2
        for layer in range(LAYERS):
            old = list(self.history[layer])
            cut = lambda r, q: tuple(x[: None if keep is None else keep[r]] for x in old[q])  # noqa: E731
            self.history[layer] = [none if q < 0 else cut(r, q) for r, q in enumerate(parents)]

    def shared_pages(self):
        """Pages that all rows of each request with a token in the cache hold."""
        table = self.table.cpu().numpy()
        out = []
        for g in range(self.requests):
            rows = [r for r in range(g * self.beams, (g + 1) * self.beams)
                    if len(self.history[0][r][0])]
            same = 0
            whole = min([len(self.history[0][r][0]) // 64 for r in rows], default=0)
            first = table[g * self.beams]
            while rows and rows[0] == g * self.beams and same < whole and \
                    all(table[r, same] == first[same] for r in rows):
                same += 1
            out.append(same)
        return out

    def step(self):
        """One token for every row that has any; checked layer by layer."""
        live = np.array([len(h[0]) > 0 for h in self.history[0]])
        groups = dev(self.shared_pages())
        before = self.lengths.clone()
        self.assign(live.astype(int))
        positions = torch.where(dev(live) > 0, before, -1).int()
        for layer in range(LAYERS):
            q = self.values(self.rows, self.hq)
            k, v = self.values(self.rows, self.hkv), self.values(self.rows, self.hkv)
            out = pgd.paged_decode_step(q, k, v, self.k[layer], self.v[layer], self.table,
                                        positions, num_kv_heads=self.hkv, layout=self.layout,
                                        group_starts=self.starts, group_pages=groups,
                                        kernel=self.kernel)
            at = np.nonzero(live)[0]
            self.extend(layer, at, k[dev(at).long()], v[dev(at).long()])
            assert pgd.get_device_error() == pgd.OK
            want, mass, size, every = side.attend_rows(
                q.double().cpu().numpy(),
                [tuple(x.transpose(1, 0, 2) for x in h) if len(h[0]) else None
                 for h in self.history[layer]], self.d ** -0.5)
            got = out.double().cpu().numpy()
            assert np.all(np.isfinite(got))
            excess = np.abs(got - want) - side.bound(want, mass, size, every, self.d)
            assert excess.max() <= 0, (layer, np.unravel_index(np.argmax(excess), excess.shape))
        return groups.cpu().numpy()

    def books(self):
        """Shares and the list say what the table does."""
        table, n = self.table.cpu().numpy(), self.lengths.cpu().numpy()
        held = np.zeros(self.pages, dtype=int)
        for r in range(self.rows):
            np.add.at(held, table[r, :side.pages_of(n[r])], 1)
        assert np.array_equal(np.maximum(held - 1, 0), self.shares.cpu().numpy())
        free = self.free.cpu().numpy()[self.head.item():]
        assert sorted(free) == sorted(np.nonzero(held == 0)[0])
        return held


@pytest.mark.parametrize("hq,hkv,d,layout,kernel", [
    (14, 2, 64, pgd.PAGE_MAJOR, pgd.KERNEL_PREFILL_UMMA),
    (32, 8, 128, pgd.HEAD_MAJOR, pgd.KERNEL_PREFILL_UMMA),
    (8, 8, 128, pgd.PAGE_MAJOR, pgd.KERNEL_AUTO)])
def test_beam_search_over_shared_pages(hq, hkv, d, layout, kernel):
    s = Server(1, [200, 63, 64, 129], 4, hq, hkv, d, layout, kernel)
    s.prefill()
    s.books()
    first = np.arange(s.rows) // 4 * 4
    s.fork(first)                                   # each prompt into four beams
    s.books()
    assert list(s.step()) == [3, 0, 1, 2]
    for turn in range(70):                          # past a page's end
        s.fork(first + s.rng.integers(0, 4, s.rows))
        if turn % 10 == 0 or turn > 60:
            s.books()
            s.step()
        else:                                       # (the same step, unchecked)
            plan = s.assign(np.ones(s.rows, dtype=int))
            for layer in range(LAYERS):
                k, v = s.values(s.rows, hkv), s.values(s.rows, hkv)
                pgd.kv_write_slots(k, v, plan.slots, s.k[layer], s.v[layer], layout=layout)
                s.extend(layer, range(s.rows), k, v)
    # a request finishes, another goes back to its prompt's middle, one beam is dropped
    parents = np.where(np.arange(s.rows) // 4 == 1, -1, np.arange(s.rows))
    parents[13] = -1
    keep = np.where(np.arange(s.rows) // 4 == 3, 100, 2 ** 31 - 1)
    s.fork(parents, keep)
    s.books()
    s.step()
    # the pool's upper end is given up
    plan = pgd.compact_pages(s.table, s.lengths, s.shares, s.free, free_head=s.head)
    pgd.copy_pages(s.k, s.v, plan.sources, plan.targets, num_kv_heads=hkv, head_dim=d,
                   layout=layout)
    s.table, s.shares, s.free = plan.table, plan.shares, plan.free_pages
    held = s.books()
    assert plan.end.item() == (held > 0).sum()      # nothing between the pages in use
    if layout == pgd.PAGE_MAJOR:
        for pool in s.k + s.v:
            pool[plan.end.item():] = float("nan")
    s.step()
    s.fork(np.full(s.rows, -1))
    assert s.head.item() == 0 and not s.shares.any()


def test_a_step_captured_with_its_reordering():
    """fork_rows, copy_pages, assign_pages and the attention in one graph, replayed with other
    parents and values; no memory but what the graph was given."""
    hq, hkv, d, beams = 14, 2, 64, 4
    s = Server(2, [150, 70], beams, hq, hkv, d, pgd.PAGE_MAJOR)
    s.prefill()
    s.fork(np.arange(s.rows) // beams * beams)
    s.step()
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    parents = i32(s.rows)
    q, k, v = s.values(s.rows, hq), s.values(s.rows, hkv), s.values(s.rows, hkv)
    out = torch.empty_like(q)
    fork = pgd.ForkPlan(i32(s.rows), i32(s.rows), i32(s.rows), i32(s.rows), i32(1))
    page = pgd.PagePlan(i32(s.rows), i32(s.rows), i32(s.rows), i32(s.rows + 1), i32(s.rows), i32(1))
    ones, groups = dev(np.ones(s.rows)), dev([2, 1])
    dims = pgd.make_dims(rows=s.rows, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                         num_pages=s.pages, max_pages_per_row=s.table.shape[1])
    work = torch.empty(pgd.shared_decode_workspace_bytes(dims, 2), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pgd.fork_rows(s.table, s.lengths, parents, s.shares, s.free, free_head=s.head, out=fork)
        pgd.copy_pages(s.k, s.v, fork.sources, fork.targets, fork.counts, num_kv_heads=hkv,
                       head_dim=d)
        pgd.assign_pages(s.table, fork.lengths, ones, s.free, num_tokens=s.rows, num_pages=s.pages,
                         free_head=fork.free_head, out=page)
        s.lengths.copy_(page.lengths)
        s.head.copy_(page.free_head)
        pgd.paged_decode_step(q, k, v, s.k[0], s.v[0], s.table, page.positions, num_kv_heads=hkv,
                              out=out, workspace=work, group_starts=s.starts, group_pages=groups,
                              kernel=pgd.KERNEL_PREFILL_UMMA)
    for turn in range(80):
        chosen = np.arange(s.rows) // beams * beams + s.rng.integers(0, beams, s.rows)
        parents.copy_(dev(chosen))
        for t in (q, k, v):
            t.copy_(s.values(s.rows, t.shape[1]))
        graph.replay()
        s.history[0] = [s.history[0][r] for r in chosen]
        s.extend(0, range(s.rows), k, v)
        if turn % 20 == 19 or turn < 2:
            assert pgd.get_device_error() == pgd.OK
            s.books()
            want, mass, size, every = side.attend_rows(
                q.double().cpu().numpy(),
                [tuple(x.transpose(1, 0, 2) for x in h) for h in s.history[0]], d ** -0.5)
            excess = np.abs(out.double().cpu().numpy() - want) - \
                side.bound(want, mass, size, every, d)
            assert excess.max() <= 0
