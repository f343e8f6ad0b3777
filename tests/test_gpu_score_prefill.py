"""Prefill attention with capped and biased scores, documents and bidirectional
prefixes, against the plain 64-bit implementation; on the tcgen05 kernel, its
key parts and the per-token kernel; steps; masks that leave nothing; values in
masked places; bad entries; graphs and streams."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests.score_side import DEV, Paged, i32
from tests.score_side import check as check_score

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def check(*args, kernel=pgd.KERNEL_PREFILL_UMMA, **kw):
    check_score(*args, rounded=kernel != pgd.KERNEL_TENSOR_CORE, **kw)


def packed(cached, chunks):
    rows = np.repeat(np.arange(len(cached)), chunks)
    positions = np.concatenate([np.arange(c, c + t) for c, t in zip(cached, chunks)])
    return rows, positions


def mods(kw, b, rows, positions, seed=3):
    hq = b.hq
    g = torch.Generator().manual_seed(seed)
    a = dict(softcap=kw.get("softcap", 0.0), alibi_slopes=None, first_key=None, prefix_len=None)
    if kw.get("alibi"):
        a["alibi_slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).to(DEV)
    if kw.get("docs"):
        a["first_key"] = i32(positions // kw["docs"] * kw["docs"])
    if kw.get("prefix"):
        a["prefix_len"] = i32(np.minimum(b.lengths, kw["prefix"]))
    sinks = torch.randn(hq, generator=g).to(DEV) if kw.get("sinks") else None
    window = kw.get("window", 0)
    return a, sinks, window, dict(softcap=a["softcap"], slopes=a["alibi_slopes"],
                                  first=a["first_key"], prefix=a["prefix_len"], sinks=sinks,
                                  window=window)


MODS = [dict(softcap=50.0), dict(softcap=1.0, sinks=True), dict(alibi=True), dict(docs=50),
        dict(prefix=90), dict(softcap=20.0, alibi=True, docs=77, prefix=33, sinks=True),
        dict(softcap=30.0, window=100), dict(alibi=True, window=65, prefix=150, sinks=True)]
KERNELS = [pgd.KERNEL_AUTO, pgd.KERNEL_TENSOR_CORE, pgd.KERNEL_PREFILL_UMMA]


@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (16, 2, 64), (8, 8, 64), (8, 2, 128),
                                      (3, 3, 128), (10, 2, 128)])
@pytest.mark.parametrize("kw", MODS, ids=str)
@pytest.mark.parametrize("kernel", KERNELS)
def test_prefill(hq, hkv, d, kw, kernel):
    cached, chunks = [0, 65, 300, 31], [130, 70, 45, 1]
    b = Paged(1, np.add(cached, chunks), hq, hkv, d, width=7)
    rows, positions = packed(cached, chunks)
    a, sinks, window, c = mods(kw, b, rows, positions)
    q = b.queries(len(rows))
    out = torch.full_like(q, float("nan"))
    pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), sinks,
                                window, num_kv_heads=hkv, kernel=kernel, out=out, **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, kernel=kernel, scale=d ** -0.5, **c)


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 64), (4, 1, 128)])
@pytest.mark.parametrize("kw", MODS, ids=str)
def test_key_parts(hq, hkv, d, kw):
    """Few items over a long cached prefix: AUTO cuts them into key parts."""
    cached, chunks = [2370], [200]
    b = Paged(2, [2570], hq, hkv, d)
    rows, positions = packed(cached, chunks)
    kw = dict(kw)
    if "docs" in kw:
        kw["docs"] = 2450
    a, sinks, window, c = mods(kw, b, rows, positions)
    q = b.queries(len(rows))
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      sinks, window, num_kv_heads=hkv, **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=d ** -0.5, **c)


@pytest.mark.parametrize("layout", [pgd.PAGE_MAJOR, pgd.HEAD_MAJOR, pgd.ROW_MAJOR])
@pytest.mark.parametrize("kernel", KERNELS)
def test_step(layout, kernel):
    cached, chunks = [0, 100, 5], [100, 28, 60]
    b = Paged(3, np.add(cached, chunks), 14, 2, 64, width=3, layout=layout)
    rows, positions = packed(cached, chunks)
    a, sinks, window, c = mods(dict(softcap=20.0, alibi=True, prefix=40, docs=64, sinks=True), b,
                               rows, positions)
    q = b.queries(len(rows))
    k_new = torch.randn(len(rows), 2, 64, generator=b.gen).bfloat16().to(DEV)
    v_new = torch.randn(len(rows), 2, 64, generator=b.gen).bfloat16().to(DEV)
    for t, (r, n) in enumerate(zip(rows, positions)):
        b.k_rows[r][:, n], b.v_rows[r][:, n] = (x[t].double().cpu().numpy() for x in (k_new, v_new))
    k2, v2 = b.k_pool.clone(), b.v_pool.clone()
    out = pgd.paged_prefill_step(q, k_new, v_new, b.k_pool, b.v_pool, b.table, i32(rows),
                                 i32(positions), sinks, window, num_kv_heads=2, layout=layout,
                                 kernel=kernel, **a)
    b.write(k2, rows, positions, k_new)
    b.write(v2, rows, positions, v_new)
    two = pgd.paged_prefill_attention(q, k2, v2, b.table, i32(rows), i32(positions), sinks, window,
                                      num_kv_heads=2, layout=layout, kernel=kernel, **a)
    assert pgd.get_device_error() == pgd.OK
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731
    assert same(b.k_pool, k2) and same(b.v_pool, v2) and same(out, two)
    check(out, b, q, rows, positions, kernel=kernel, scale=0.125, **c)


@pytest.mark.parametrize("kernel", KERNELS)
def test_odd_token_orders(kernel):
    """Tokens of a row out of order, repeated, interleaved with other rows and inactive."""
    b = Paged(4, [400, 200], 8, 2, 64)
    rng = np.random.default_rng(1)
    rows = rng.integers(0, 2, 90)
    positions = np.array([rng.integers(0, b.lengths[r]) for r in rows])
    positions[[3, 40, 41]] = -1
    first = rng.integers(-3, 300, 90)          # some past their token: those see nothing
    a = dict(softcap=10.0, first_key=i32(first), prefix_len=i32([-4, 60]))
    q = b.queries(90)
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      num_kv_heads=2, kernel=kernel, **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, kernel=kernel, scale=0.125, softcap=10.0, first=first,
          prefix=[-4, 60])
    empty = (positions >= 0) & (first > np.maximum(positions, np.array([-4, 60])[rows] - 1))
    assert empty.any() and not out[torch.from_numpy(empty)].any()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("sinks", [False, True])
def test_masks_that_leave_nothing(kernel, sinks):
    b = Paged(5, [300], 8, 1, 64)
    rows, positions = packed([100], [200])
    s = torch.zeros(8, device=DEV) if sinks else None
    q = b.queries(200)
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), s,
                                      num_kv_heads=1, kernel=kernel, softcap=3.0,
                                      first_key=i32(np.where(positions < 280, 2 ** 31 - 1, 290)))
    assert pgd.get_device_error() == pgd.OK
    first = np.where(positions < 280, 2 ** 31 - 1, 290)
    check(out, b, q, rows, positions, kernel=kernel, scale=0.125, softcap=3.0, sinks=s, first=first)
    assert not out[:190].any() and out[190:].any()


@pytest.mark.parametrize("kernel", KERNELS)
def test_values_in_masked_places(kernel):
    """NaN and infinities in documents before a run's own, past its last visible position and
    in unused pages; a cap that masked values must not disturb."""
    b = Paged(6, [500, 500], 16, 2, 128, width=9)
    rows, positions = packed([260, 300], [60, 40])
    first = np.where(positions < 290, 70, 130)
    call = lambda: pgd.paged_prefill_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), num_kv_heads=2, softcap=6.0,
        first_key=i32(first), prefix_len=i32([333, 0]), kernel=kernel)
    q = b.queries(100)
    want = call()
    for bad in (float("nan"), float("inf"), -3.3e38):
        for pool in (b.k_pool, b.v_pool):
            for r, lo, hi in ((0, 70, 332), (1, 130, 339)):
                for n in list(range(lo)) + list(range(hi + 1, 512)):
                    pool[b.table_np[r, n // 64], :, n % 64] = bad
        assert torch.equal(call(), want)
    check(want, b, q, rows, positions, kernel=kernel, scale=128 ** -0.5, softcap=6.0, first=first,
          prefix=[333, 0])


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("softcap,gain,scale", [(2.0, 40.0, 0.125), (50.0, 30.0, -0.2),
                                                (0.01, 1.0, 0.125), (30.0, 1.0, 0.0),
                                                (1000.0, 1.0, 0.125)])
def test_scores_far_past_the_cap(kernel, softcap, gain, scale):
    b = Paged(7, [200, 90], 16, 2, 64)
    rows, positions = packed([100, 0], [100, 90])
    q = b.queries(190) * gain
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      None, 0, scale, num_kv_heads=2, softcap=softcap,
                                      kernel=kernel)
    check(out, b, q, rows, positions, kernel=kernel, scale=scale, softcap=softcap)


@pytest.mark.parametrize("kernel", KERNELS)
def test_bad_entries(kernel):
    b = Paged(8, [200, 200, 200, 200], 8, 2, 64, width=4)
    rows, positions = packed([100, 100, 100, 100], [40, 40, 40, 40])
    rows = rows.copy()
    rows[35:40] = 9                                   # no such table row
    table = b.table.clone()
    table[1, 0], table[2, 1] = 10 ** 6, -1
    q = b.queries(160)
    first = np.where(rows == 1, 64, 0)                # row 1 does not read its bad page
    prefix = [0, 0, 0, 257]                           # past row 3's table
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, table, i32(rows), i32(positions),
                                      num_kv_heads=2, softcap=8.0, first_key=i32(first),
                                      prefix_len=i32(prefix), kernel=kernel)
    assert pgd.get_device_error() == pgd.EDEVICE_BOUNDS
    good = np.r_[0:35, 40:80]
    check(out[good], b, q[good], rows[good], positions[good], kernel=kernel, scale=0.125,
          softcap=8.0, first=first[good], prefix=prefix)
    assert not out[35:40].any() and not out[80:].any()


def test_graph_and_streams():
    b = Paged(9, [1000, 300], 32, 8, 128)
    rows, positions = packed([700, 0], [300, 300])
    q, n, r = b.queries(600), i32(positions), i32(rows)
    prefix = i32([0, 100])
    kw = dict(num_kv_heads=8, softcap=25.0, prefix_len=prefix)
    out = torch.empty_like(q)
    dims = pgd.make_dims(rows=600, num_q_heads=32, num_kv_heads=8, head_dim=128, num_pages=b.pages,
                         max_pages_per_row=b.width)
    ws = torch.empty(max(16, pgd.paged_decode_workspace_bytes(dims)), dtype=torch.uint8,
                     device=DEV)
    call = lambda: pgd.paged_prefill_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, b.table, r, n, out=out, workspace=ws, **kw)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    prefix.copy_(i32([900, 0]))
    n.sub_((n >= 700).int() * 100)
    out.fill_(float("nan"))
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, r, n, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(other, out)
    pos = n.cpu().numpy()
    check(out, b, q, rows, pos, scale=128 ** -0.5, softcap=25.0, prefix=[900, 0])


@pytest.mark.parametrize("seed", range(40))
def test_random(seed):
    rng = np.random.default_rng(900 + seed)
    hkv = int(rng.choice([1, 2, 3]))
    hq, d = hkv * int(rng.integers(1, 9)), int(rng.choice([64, 128]))
    n = int(rng.integers(1, 5))
    cached = rng.integers(0, int(rng.choice([1, 100, 900])), n)
    chunks = rng.integers(1, int(rng.choice([3, 60, 200])), n)
    b = Paged(seed, cached + chunks, hq, hkv, d, width=int(rng.integers(18, 30)))
    rows, positions = packed(cached, chunks)
    kw = dict(softcap=float(rng.choice([0.0, 0.5, 15.0, 50.0])), alibi=rng.random() < 0.5,
              docs=int(rng.choice([0, 0, 1, 30, 200])), prefix=int(rng.choice([0, 0, 1, 64, 500])),
              sinks=rng.random() < 0.5, window=int(rng.choice([0, 0, 1, 50, 500])))
    if not (kw["softcap"] or kw["alibi"] or kw["docs"] or kw["prefix"]):
        kw["softcap"] = 4.0
    a, sinks, window, c = mods(kw, b, rows, positions, seed)
    q = b.queries(len(rows))
    kernel = int(rng.choice(KERNELS))
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      sinks, window, num_kv_heads=hkv, kernel=kernel, **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, kernel=kernel, scale=d ** -0.5, **c)


def test_refusals():
    b = Paged(11, [10], 8, 2, 64)
    q, n = b.queries(10), i32(np.arange(10))
    call = lambda **kw: pgd.paged_prefill_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, b.table, i32([0] * 10), n, num_kv_heads=2, **kw)
    for kw in (dict(prefix_len=i32([1, 2])), dict(prefix_len=torch.zeros(1, device=DEV)),
               dict(first_key=i32([0])), dict(softcap=-2.0)):
        with pytest.raises(ValueError):
            call(**kw)
    for kernel in (pgd.KERNEL_CUDA_CORE, pgd.KERNEL_PREFILL_TILED, pgd.KERNEL_PREFILL_PAIR):
        with pytest.raises(pgd.PgdError) as e:
            call(prefix_len=i32([3]), kernel=kernel)
        assert e.value.status == pgd.EUNSUPPORTED


def ramp(b, gains):
    """Keys of each row times a gain per position (rounded to bf16 again)."""
    for r, n in enumerate(b.lengths):
        k = torch.from_numpy(b.k_rows[r]).transpose(0, 1) * torch.as_tensor(gains[:n])[:, None, None]
        k = k.bfloat16()
        b.k_rows[r] = k.transpose(0, 1).double().numpy()
        b.write(b.k_pool, [r] * n, range(n), k.to(DEV))


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("kernel", [pgd.KERNEL_AUTO, pgd.KERNEL_PREFILL_UMMA])
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("kw", [
    dict(docs=10000), dict(softcap=50.0), dict(softcap=53.0), dict(softcap=300.0),
    dict(slopes=-0.05), dict(slopes=0.05), dict(softcap=70.0, slopes=-0.02)], ids=str)
def test_scores_that_grow(hq, hkv, d, kernel, falling, kw):
    """Scores that grow, or fall, from page to page by more than a row's reference allows:
    every page raises it, or (a reference that stays) the caps' forms change on the way."""
    b = Paged(12, [1100, 700], hq, hkv, d)
    gains = np.linspace(0.2, 12.0, 1100)
    ramp(b, gains[::-1].copy() if falling else gains)
    rows, positions = packed([900, 560], [200, 140])
    q = b.queries(340)
    softcap = kw.get("softcap", 0.0)
    slopes = torch.full((hq,), kw["slopes"], device=DEV) if "slopes" in kw else None
    first = positions // kw["docs"] if "docs" in kw else None
    out = pgd.paged_prefill_attention(
        q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), num_kv_heads=hkv,
        kernel=kernel, softcap=softcap, alibi_slopes=slopes,
        first_key=None if first is None else i32(first))
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=d ** -0.5, softcap=softcap, slopes=slopes, first=first)


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("softcap", [1.0, 50.0, 52.6, 52.8, 100.0, 1000.0])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("sinks", [False, True])
def test_all_scores_at_one_end_of_the_cap(hq, hkv, d, softcap, sign, sinks):
    """Every score near -cap (or cap): weights far from 1 against a reference that stays;
    values of 2^20 with them."""
    b = Paged(13, [300, 65], hq, hkv, d, scale_v=2.0 ** 20)
    ramp(b, np.ones(300))
    for r, n in enumerate(b.lengths):
        k = (torch.from_numpy(b.k_rows[r]).abs() + 0.5).bfloat16()
        b.k_rows[r] = k.double().numpy()
        b.write(b.k_pool, [r] * n, range(n), k.transpose(0, 1).to(DEV))
    rows, positions = packed([200, 0], [100, 65])
    q = b.queries(165).abs() + 0.25
    scale = sign * softcap / d                    # products of about 1.3 d: well past the cap
    s = torch.linspace(-60.0, 60.0, hq, device=DEV) if sinks else None
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      s, 0, scale, num_kv_heads=hkv, softcap=softcap,
                                      kernel=pgd.KERNEL_PREFILL_UMMA)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=scale, softcap=softcap, sinks=s)


@pytest.mark.parametrize("kernel", KERNELS)
def test_one_row_of_nan(kernel):
    """A token's own NaN (or infinite) query reaches its own outputs only."""
    b = Paged(14, [300], 16, 2, 64)
    rows, positions = packed([100], [200])
    q = b.queries(200)
    args = (b.k_pool, b.v_pool, b.table, i32(rows), i32(positions))
    kw = dict(num_kv_heads=2, softcap=9.0, alibi_slopes=torch.full((16,), 0.1, device=DEV),
              kernel=kernel)
    want = pgd.paged_prefill_attention(q, *args, **kw)
    bad = q.clone()
    bad[77], bad[150, 3] = float("nan"), float("inf")
    got = pgd.paged_prefill_attention(bad, *args, **kw)
    same = torch.ones(200, 16, dtype=torch.bool, device=DEV)
    same[77], same[150, 3] = False, False
    assert torch.equal(got[same], want[same])
    assert torch.isnan(got[77]).all()


def test_a_nan_row_in_key_parts():
    """As above where the keys are cut into parts: the row's outputs are NaN, not left over."""
    b = Paged(15, [2570], 4, 1, 128)
    rows, positions = packed([2370], [200])
    q = b.queries(200)
    q[33] = float("nan")
    out = torch.full_like(q, 7.0)
    pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                num_kv_heads=1, softcap=20.0, out=out)
    assert pgd.get_device_error() == pgd.OK
    good = np.r_[0:33, 34:200]
    check(out[good], b, q[good], rows[good], positions[good], scale=128 ** -0.5, softcap=20.0)
    assert torch.isnan(out[33]).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap", [1e4, 1e6, 4e8, 1e12])
def test_a_cap_far_above_the_scores(kernel, d, softcap):
    """Scores up to s differ from uncapped ones by s^3 / (3 softcap^2): here by less than 1e-6."""
    b = Paged(16, [300, 65], 8, 2, d)
    rows, positions = packed([200, 0], [100, 65])
    q = b.queries(165)
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      num_kv_heads=2, softcap=softcap, kernel=kernel)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, kernel=kernel, scale=d ** -0.5)


def test_scratch_on_a_side_stream():
    """A call's own workspace is not handed out while the call runs on another stream."""
    b = Paged(17, [3000], 8, 2, 64)
    rows, positions = packed([2900], [100])
    q = b.queries(100)
    args = (b.k_pool, b.v_pool, b.table, i32(rows), i32(positions))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(pgd.paged_prefill_attention(q, *args, num_kv_heads=2, softcap=9.0, stream=side))
        for size in (1 << 20, 1 << 22, 1 << 23):          # (would take the block if it were free)
            torch.full((size,), float("nan"), device=DEV)
    torch.cuda.synchronize()
    check(outs[0], b, q, rows, positions, scale=0.125, softcap=9.0)
    assert all(torch.equal(o, outs[0]) for o in outs)
