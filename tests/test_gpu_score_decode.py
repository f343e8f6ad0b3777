"""Decode attention with capped and biased scores and first visible keys, against
the plain 64-bit implementation; steps, dense rows, layouts, splits, rows whose
mask leaves nothing, values in masked places, graphs and streams."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests.score_side import DEV, Paged, check, i32

pytestmark = pytest.mark.gpu

CONTEXTS = [1, 2, 63, 64, 65, 128, 129, 700, 1000, 2049]
MODS = [dict(softcap=50.0), dict(softcap=1.0), dict(alibi=True), dict(first=True),
        dict(softcap=20.0, alibi=True, first=True, sinks=True),
        dict(softcap=30.0, window=100), dict(alibi=True, window=300, sinks=True, first=True)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def mods(kw, hq, positions, seed=3):
    """Arguments of a call and of the check for the modifications `kw`."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    a = dict(softcap=kw.get("softcap", 0.0), alibi_slopes=None, first_key=None)
    if kw.get("alibi"):
        a["alibi_slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).to(DEV)
    if kw.get("first"):
        a["first_key"] = i32([rng.integers(0, max(1, n) + 1) for n in positions])
    sinks = torch.randn(hq, generator=g).to(DEV) if kw.get("sinks") else None
    window = kw.get("window", 0)
    return a, sinks, window, dict(softcap=a["softcap"], slopes=a["alibi_slopes"],
                                  first=a["first_key"], sinks=sinks, window=window)


@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (64, 8, 64), (32, 8, 128), (8, 8, 128),
                                      (3, 1, 64), (10, 2, 128)])
@pytest.mark.parametrize("kw", MODS, ids=str)
@pytest.mark.parametrize("pages_per_split", [0, 1, 5])
def test_decode(hq, hkv, d, kw, pages_per_split):
    b = Paged(1, CONTEXTS, hq, hkv, d, width=40)
    positions = [n - 1 for n in CONTEXTS]
    a, sinks, window, c = mods(kw, hq, positions)
    q = b.queries(len(positions))
    out = torch.full_like(q, float("nan"))
    pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32(positions), sinks, window,
                               num_kv_heads=hkv, pages_per_split=pages_per_split, out=out, **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, range(len(positions)), positions, scale=d ** -0.5, **c)


@pytest.mark.parametrize("layout", [pgd.PAGE_MAJOR, pgd.HEAD_MAJOR, pgd.ROW_MAJOR])
@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (32, 8, 128)])
def test_step_appends_and_attends(layout, hq, hkv, d):
    contexts = [1, 64, 65, 300, 5]
    b = Paged(2, contexts, hq, hkv, d, width=6, layout=layout)
    positions = [0, 63, 64, 299, -1]
    a, sinks, window, c = mods(dict(softcap=30.0, alibi=True, sinks=True, first=True), hq,
                               positions)
    a["first_key"][1] = 64            # sees nothing, and is appended all the same
    q = b.queries(5)
    k_new = torch.randn(5, hkv, d, generator=b.gen).bfloat16().to(DEV)
    v_new = torch.randn(5, hkv, d, generator=b.gen).bfloat16().to(DEV)
    for r, n in enumerate(positions):
        if n >= 0:
            b.k_rows[r][:, n] = k_new[r].double().cpu().numpy()
            b.v_rows[r][:, n] = v_new[r].double().cpu().numpy()
    k2, v2 = b.k_pool.clone(), b.v_pool.clone()
    out = pgd.paged_decode_step(q, k_new, v_new, b.k_pool, b.v_pool, b.table, i32(positions),
                                sinks, window, num_kv_heads=hkv, layout=layout, **a)
    pgd.kv_append_paged(k_new, v_new, b.table, i32(positions), k2, v2, layout=layout)
    two = pgd.paged_decode_attention(q, k2, v2, b.table, i32(positions), sinks, window,
                                     num_kv_heads=hkv, layout=layout, **a)
    assert pgd.get_device_error() == pgd.OK
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731
    assert same(b.k_pool, k2) and same(b.v_pool, v2) and same(out, two)
    assert not out[1].any() and not out[4].any()
    check(out, b, q, range(5), positions, scale=d ** -0.5, **c)
    if layout == pgd.ROW_MAJOR:
        cache = lambda t: t.view(5, hkv, 6 * 64, d)  # noqa: E731
        rows = pgd.decode_rows_attention(q, cache(k2), cache(v2), i32(positions), sinks, window,
                                         **a)
        assert same(rows, out)
        rows = pgd.decode_rows_step(q, k_new, v_new, cache(k2), cache(v2), i32(positions), sinks,
                                    window, **a)
        assert same(rows, out)


def test_first_keys_at_the_borders():
    n = 200
    firsts = [0, -5, 1, 63, 64, 65, 127, 128, 199, 200, 201, 2 ** 31 - 1, -2 ** 31]
    b = Paged(4, [n] * len(firsts), 8, 2, 64, width=9)
    q = b.queries(len(firsts))
    for pages_per_split in (0, 1, 2):
        for sinks in (None, torch.zeros(8, device=DEV)):
            out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table,
                                             i32([n - 1] * len(firsts)), sinks, num_kv_heads=2,
                                             first_key=i32(firsts),
                                             pages_per_split=pages_per_split)
            check(out, b, q, range(len(firsts)), [n - 1] * len(firsts), scale=0.125, sinks=sinks,
                  first=firsts)
            assert not out[9:12].any()
    assert pgd.get_device_error() == pgd.OK


def test_values_in_masked_places():
    """NaN and infinities before the first key, past the position and in unused pages."""
    b = Paged(5, [300, 300], 8, 8, 128, width=5)
    q = b.queries(2)
    first, last = 70, 250
    want = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32([last, last]),
                                      num_kv_heads=8, softcap=5.0, first_key=i32([first] * 2))
    for bad in (float("nan"), float("inf"), -3.3e38):
        for pool in (b.k_pool, b.v_pool):
            for r in range(2):
                for n in list(range(first)) + list(range(last + 1, 320)):
                    pool[b.table_np[r, n // 64], :, n % 64] = bad
        out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32([last, last]),
                                         num_kv_heads=8, softcap=5.0, first_key=i32([first] * 2))
        assert torch.equal(out, want)


@pytest.mark.parametrize("softcap,gain", [(2.0, 40.0), (50.0, 30.0), (1000.0, 1.0), (0.01, 1.0)])
@pytest.mark.parametrize("scale", [0.125, -0.3, 0.0])
def test_scores_far_past_the_cap(softcap, gain, scale):
    b = Paged(6, [500, 77], 16, 2, 64)
    q = (b.queries(2) * gain)
    out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32([499, 76]), None, 0, scale,
                                     num_kv_heads=2, softcap=softcap)
    check(out, b, q, range(2), [499, 76], scale=scale, softcap=softcap)


@pytest.mark.parametrize("slopes", [[0.0] * 8, [1.0] * 8, [-0.01] * 8, [0.5, 0, 0, 0, 3, 0, 0, 1]])
def test_slopes(slopes):
    b = Paged(7, [700, 1, 64], 8, 1, 64)
    q = b.queries(3)
    s = torch.tensor(slopes, device=DEV)
    out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32([699, 0, 63]),
                                     num_kv_heads=1, alibi_slopes=s)
    check(out, b, q, range(3), [699, 0, 63], scale=0.125, slopes=s)


def test_long_row_and_no_modification():
    """A row of many splits; and a cap too wide to matter, no bias: the plain call's result."""
    b = Paged(8, [33000, 31000], 8, 1, 64, scale_v=0.5)
    q = b.queries(2)
    pos = i32([32999, 30999])
    s = torch.full((8,), 2.0 ** -12, device=DEV)
    out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, pos, num_kv_heads=1,
                                     softcap=50.0, alibi_slopes=s)
    check(out, b, q, range(2), [32999, 30999], scale=0.125, softcap=50.0, slopes=s)
    plain = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, pos, num_kv_heads=1)
    masked = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, pos, num_kv_heads=1,
                                        first_key=i32([0, 0]))
    assert torch.equal(plain, masked)


def test_bad_pages_and_positions():
    b = Paged(9, [200, 200, 200], 8, 2, 64, width=4)
    q = b.queries(3)
    table = b.table.clone()
    table[0, 2], table[1, 0] = 10 ** 6, -1
    for pages_per_split in (0, 1):
        out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, table, i32([199, 199, 256]),
                                         num_kv_heads=2, softcap=9.0, first_key=i32([0, 64, 0]),
                                         pages_per_split=pages_per_split)
        assert pgd.get_device_error() == pgd.EDEVICE_BOUNDS
        assert not out[0].any() and not out[2].any()
        # the bad page of row 1 lies before its first key: not read
        check(out[1:2], b, q[1:2], [1], [199], scale=0.125, softcap=9.0, first=[64])


def test_graph_stream_and_shared_pages():
    b = Paged(10, [900, 130], 32, 8, 128)
    table = i32([b.table_np[0], b.table_np[0], b.table_np[1]])       # two rows share pages
    q, pos, first = b.queries(3), i32([899, 500, 129]), i32([100, 0, 5])
    kw = dict(num_kv_heads=8, softcap=25.0, first_key=first)
    out = torch.empty_like(q)
    dims = pgd.make_dims(rows=3, num_q_heads=32, num_kv_heads=8, head_dim=128, num_pages=b.pages,
                         max_pages_per_row=b.width)
    ws = torch.empty(max(16, pgd.paged_decode_workspace_bytes(dims)), dtype=torch.uint8,
                     device=DEV)
    call = lambda: pgd.paged_decode_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, table, pos, out=out, workspace=ws, **kw)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pos.copy_(i32([700, 899, 100]))
    first.copy_(i32([0, 640, 100]))
    out.fill_(float("nan"))
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, table, pos, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(other, out)
    check(out, b, q, [0, 0, 1], [700, 899, 100], scale=128 ** -0.5, softcap=25.0,
          first=[0, 640, 100])


@pytest.mark.parametrize("seed", range(40))
def test_random(seed):
    rng = np.random.default_rng(500 + seed)
    hkv = int(rng.choice([1, 2, 3, 8]))
    hq, d = hkv * int(rng.integers(1, 9)), int(rng.choice([64, 128]))
    rows = int(rng.integers(1, 9))
    contexts = [int(rng.integers(1, int(rng.choice([70, 700, 2500])))) for _ in range(rows)]
    b = Paged(seed, contexts, hq, hkv, d, width=int(rng.integers(40, 60)))
    positions = [n - 1 if rng.random() < 0.9 else -1 for n in contexts]
    kw = dict(softcap=float(rng.choice([0.0, 0.5, 15.0, 50.0])), alibi=rng.random() < 0.5,
              first=rng.random() < 0.5, sinks=rng.random() < 0.5,
              window=int(rng.choice([0, 0, 1, 100, 1000])))
    if not (kw["softcap"] or kw["alibi"] or kw["first"]):
        kw["first"] = True
    a, sinks, window, c = mods(kw, hq, positions, seed)
    q = b.queries(rows)
    out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32(positions), sinks, window,
                                     num_kv_heads=hkv, pages_per_split=int(rng.integers(0, 9)), **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, range(rows), positions, scale=d ** -0.5, **c)


def test_refusals():
    b = Paged(11, [10], 8, 2, 64)
    q = b.queries(1)
    call = lambda **kw: pgd.paged_decode_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, b.table, i32([9]), num_kv_heads=2, **kw)
    f = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
               dict(alibi_slopes=f(7)), dict(alibi_slopes=f(8).double()),
               dict(alibi_slopes=f(16)[::2]), dict(first_key=i32([1, 2])),
               dict(first_key=f(1)), dict(first_key=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call(**kw)
    for kernel in (pgd.KERNEL_CUDA_CORE, pgd.KERNEL_PREFILL_TILED, pgd.KERNEL_PREFILL_PAIR):
        with pytest.raises(pgd.PgdError) as e:
            call(softcap=5.0, kernel=kernel)
        assert e.value.status == pgd.EUNSUPPORTED
    with pytest.raises(pgd.PgdError):
        call(softcap=5.0, kernel=pgd.KERNEL_PREFILL_UMMA)
    with pytest.raises(pgd.PgdError) as e:
        call(softcap=5.0, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == pgd.EWORKSPACE


@pytest.mark.parametrize("softcap", [1e4, 1e6, 4e8, 1e12])
def test_a_cap_far_above_the_scores(softcap):
    """Scores up to s differ from uncapped ones by s^3 / (3 softcap^2): here by less than 1e-6."""
    b = Paged(21, [300, 65], 8, 2, 64)
    q = b.queries(2)
    out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32([299, 64]),
                                     num_kv_heads=2, softcap=softcap)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, [0, 1], [299, 64], scale=0.125)
