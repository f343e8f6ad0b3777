"""Attention with modified scores at the ends of what its arguments allow: outputs near
cancellation, NaN rows in calls cut into parts, steep distance biases, values of any size,
many tokens, prefix lengths at the ends of int32."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests.score_side import DEV, Paged, check, i32

pytestmark = pytest.mark.gpu

UMMA = pgd.KERNEL_PREFILL_UMMA


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def packed(cached, chunks):
    rows = np.repeat(np.arange(len(cached)), chunks)
    positions = np.concatenate([np.arange(c, c + t) for c, t in zip(cached, chunks)])
    return rows, positions


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (16, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("kernel", [pgd.KERNEL_AUTO, UMMA])
def test_many_items_that_end_in_runs_without_pages(hq, hkv, d, softcap, kernel):
    """Blocks of a few visible tokens each, then padding, unseen tokens and other rows' tokens
    in turn: short page streams whose descriptors end in runs that copy nothing."""
    b = Paged(23, [130, 70, 300], hq, hkv, d)
    block = 2 * (128 // (hq // hkv))
    rng = np.random.default_rng(4)
    tokens = 40 * block
    rows = rng.integers(0, 3, tokens)
    positions = np.array([rng.integers(0, b.lengths[r]) for r in rows])
    first = rng.integers(0, 60, tokens)
    at = np.arange(tokens) % block
    positions[(at > 6) & (at % 3 == 0)] = -1
    first[(at > 6) & (at % 3 != 0)] = 2 ** 31 - 1
    q = b.queries(tokens)
    out = torch.full_like(q, float("nan"))
    for _ in range(3):
        pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                    num_kv_heads=hkv, softcap=softcap, first_key=i32(first),
                                    kernel=kernel, out=out)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=d ** -0.5, softcap=softcap, first=first, rounded=True)


def slopes_of(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).to(DEV)


KINDS = [dict(), dict(first=True), dict(alibi=True), dict(softcap=20.0), dict(softcap=100.0),
         dict(softcap=100.0, alibi=True)]


def of_kind(kw, hq, tokens):
    """Arguments of a call and of the check (no modification: the plain call)."""
    a = dict(softcap=kw.get("softcap", 0.0), alibi_slopes=slopes_of(hq) if kw.get("alibi") else None,
             first_key=i32([1] * tokens) if kw.get("first") else None)
    return a, dict(softcap=a["softcap"], slopes=a["alibi_slopes"], first=a["first_key"])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("with_sinks", [False, True])
def test_a_nan_query_in_prefill_cut_into_key_parts(d, kw, with_sinks):
    """As in calls that are not cut: NaN for that token's heads, nothing else changed."""
    b = Paged(15, [2570], 4, 1, d)
    rows, positions = packed([2370], [200])
    q = b.queries(200)
    q[33], q[150, 2] = float("nan"), float("nan")
    a, c = of_kind(kw, 4, 200)
    sinks = torch.zeros(4, device=DEV) if with_sinks else None
    out = torch.full_like(q, 7.0)
    pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), sinks,
                                num_kv_heads=1, out=out, **a)
    assert pgd.get_device_error() == pgd.OK
    assert torch.isnan(out[33]).all() and torch.isnan(out[150, 2]).all()
    assert torch.isfinite(out[150, [0, 1, 3]]).all()
    good = np.r_[0:33, 34:150, 151:200]
    if c["first"] is not None:
        c["first"] = c["first"][good]
    check(out[good], b, q[good], rows[good], positions[good], scale=d ** -0.5, sinks=sinks,
          rounded=True, **c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("with_sinks", [False, True])
@pytest.mark.parametrize("pages_per_split", [0, 5])
def test_a_nan_query_in_decode_cut_into_splits(d, kw, with_sinks, pages_per_split):
    contexts = [2049, 2300, 64]
    b = Paged(16, contexts, 8, 2, d)
    positions = [n - 1 for n in contexts]
    q = b.queries(3)
    q[0], q[1, 5] = float("nan"), float("nan")
    a, c = of_kind(kw, 8, 3)
    sinks = torch.zeros(8, device=DEV) if with_sinks else None
    out = pgd.paged_decode_attention(q, b.k_pool, b.v_pool, b.table, i32(positions), sinks,
                                     num_kv_heads=2, pages_per_split=pages_per_split, **a)
    assert pgd.get_device_error() == pgd.OK
    assert torch.isnan(out[0]).all() and torch.isnan(out[1, 5]).all()
    assert torch.isfinite(out[1, [0, 1, 2, 3, 4, 6, 7]]).all()
    if c["first"] is not None:
        c["first"] = c["first"][2:]
    check(out[2:], b, q[2:], [2], positions[2:], scale=d ** -0.5, sinks=sinks, **c)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("slope", [1e2, 1e4, 1e6, 1e8, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(prefix=120)], ids=str)
@pytest.mark.parametrize("cut", [False, True])
def test_steep_slopes(hq, hkv, d, slope, kw, cut):
    """Slopes that leave a token its own key alone: out = v_n / (1 + e^(sink - x_n)), whatever
    n mod 16 is."""
    cached, chunk = (2370, 200) if cut else (40, 90)
    b = Paged(18, [cached + chunk], hq, hkv, d)
    rows, positions = packed([cached], [chunk])
    q = b.queries(chunk)
    sinks = torch.linspace(-2.0, 2.0, hq, device=DEV)
    softcap = kw.get("softcap", 0.0)
    out = pgd.paged_prefill_attention(
        q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), sinks, num_kv_heads=hkv,
        softcap=softcap, alibi_slopes=torch.full((hq,), slope, device=DEV),
        prefix_len=i32([kw["prefix"]]) if "prefix" in kw else None,
        kernel=pgd.KERNEL_AUTO if cut else UMMA)
    assert pgd.get_device_error() == pgd.OK
    group = hq // hkv
    k = np.repeat(b.k_rows[0][:, positions], group, axis=0).transpose(1, 0, 2)
    v = np.repeat(b.v_rows[0][:, positions], group, axis=0).transpose(1, 0, 2)
    qd = q.double().cpu().numpy()
    x, size = ((qd * k).sum(-1) * d ** -0.5, np.abs(qd * k).sum(-1) * d ** -0.5)
    if softcap:
        x = softcap * np.tanh(x / softcap)
    want = v / (1.0 + np.exp(sinks.double().cpu().numpy() - x))[..., None]
    # the weights' errors of score_side; the key's own bias is zero and no other key has weight
    weight = (2 * d * 2.0 ** -24 * size + softcap * 2.0 ** -20 + 2.0 ** -14)[..., None]
    bound = 2 * weight * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want)
    excess = np.abs(out.double().cpu().numpy() - want) - bound
    assert excess.max() <= 0, (excess.max(), np.unravel_index(np.argmax(excess), excess.shape))


@pytest.mark.parametrize("slope", [3.0, 3.9, 4.1, 60.0, -0.3, -5.0])
@pytest.mark.parametrize("kernel", [pgd.KERNEL_TENSOR_CORE, UMMA])
def test_slopes_on_both_sides_of_the_linear_form(slope, kernel):
    """A slope per head, some heads of a tile steep and some not."""
    b = Paged(19, [300, 200], 16, 2, 64)
    rows, positions = packed([150, 0], [150, 200])
    q = b.queries(350)
    slopes = torch.linspace(slope, slope / 7, 16, device=DEV)
    sinks = torch.zeros(16, device=DEV)
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      sinks, num_kv_heads=2, alibi_slopes=slopes,
                                      prefix_len=i32([260, 0]), kernel=kernel)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=0.125, slopes=slopes, prefix=[260, 0], sinks=sinks,
          rounded=True)


@pytest.mark.parametrize("kernel", [pgd.KERNEL_AUTO, pgd.KERNEL_TENSOR_CORE, UMMA])
def test_prefix_lengths_that_mean_none(kernel):
    """Lengths of 0 and less, down to the end of int32, are no prefix."""
    b = Paged(20, [100] * 5, 8, 2, 64)
    rows, positions = packed([20] * 5, [80] * 5)
    q = b.queries(400)
    args = (q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions))
    kw = dict(num_kv_heads=2, softcap=20.0, kernel=kernel)
    prefix = [0, -1, -2 ** 31, -2 ** 31 + 1, -2 ** 31]
    out = pgd.paged_prefill_attention(*args, prefix_len=i32(prefix), **kw)
    assert pgd.get_device_error() == pgd.OK
    assert torch.equal(out, pgd.paged_prefill_attention(*args, **kw))
    check(out, b, q, rows, positions, scale=0.125, softcap=20.0, rounded=True)


MANY = 65_600  # tokens: more than a grid's third dimension


@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_more_tokens_than_the_per_token_grid_holds(softcap):
    """AUTO takes them in blocks, few to a table row as they are."""
    b = Paged(24, [200] * 64, 1, 1, 64)
    count = MANY // 4
    rows = np.repeat(np.arange(count), 4)
    positions = np.tile([17, 64, 130, 199], count)
    table = b.table.repeat(count // 64 + 1, 1)[:count].contiguous()
    q = b.queries(MANY)
    out = torch.full_like(q, float("nan"))
    pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, table, i32(rows), i32(positions),
                                num_kv_heads=1, softcap=softcap, out=out)
    assert pgd.get_device_error() == pgd.OK
    assert torch.isfinite(out).all()
    some = np.r_[0:300, 65_500:MANY]
    check(out[some], b, q[some], rows[some] % 64, positions[some], scale=0.125, softcap=softcap,
          rounded=True)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_refused_calls_of_many_tokens_leave_the_pools(softcap):
    b = Paged(25, [64], 1, 1, 64)
    b.k_pool.zero_(), b.v_pool.zero_()
    q = b.queries(MANY)
    n, rows = i32(np.zeros(MANY)), i32(np.zeros(MANY))
    kw = dict(num_kv_heads=1, softcap=softcap)
    with pytest.raises(pgd.PgdError) as e:
        pgd.paged_prefill_step(q, q, q, b.k_pool, b.v_pool, b.table, rows, n,
                               kernel=pgd.KERNEL_TENSOR_CORE, **kw)
    assert e.value.status == pgd.EUNSUPPORTED
    many = b.table.repeat(MANY, 1)
    with pytest.raises(pgd.PgdError) as e:
        pgd.paged_decode_step(q, q, q, b.k_pool, b.v_pool, many, n, **kw)
    assert e.value.status == pgd.EUNSUPPORTED
    torch.cuda.synchronize()
    assert not b.k_pool.any() and not b.v_pool.any() and pgd.get_device_error() == pgd.OK


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 9.0])
def test_dense_rows_check_their_output(step, softcap):
    cache = [torch.zeros(2, 2, 64, 64, device=DEV).bfloat16() for _ in range(2)]
    q, n = torch.ones(2, 8, 64, device=DEV).bfloat16(), i32([3, 5])
    k = torch.ones(2, 2, 64, device=DEV).bfloat16()
    for out in (q[:1].clone(), q.float(), q.view(2, 64, 8)):
        with pytest.raises(ValueError, match="out"):
            if step:
                pgd.decode_rows_step(q, k, k, *cache, n, softcap=softcap, out=out)
            else:
                pgd.decode_rows_attention(q, *cache, n, softcap=softcap, out=out)
    assert not cache[0].any()


@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("kw", [dict(first=True), dict(softcap=50.0), dict(alibi=True),
                                dict(softcap=50.0, alibi=True)], ids=str)
@pytest.mark.parametrize("cut", [False, True])
def test_prefill_carries_the_weights_residual(hq, hkv, d, kw, cut):
    """The bound of the framework's other attention kernels, whose weights are a bf16 head and
    residual: outputs near cancellation err by far less than a rounded weight would make them."""
    cached, chunks = ([2370], [140]) if cut else ([0, 5, 300], [40, 70, 45])
    b = Paged(21, np.add(cached, chunks), hq, hkv, d)
    rows, positions = packed(cached, chunks)
    q = b.queries(len(rows))
    a, c = of_kind(kw, hq, len(rows))
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      num_kv_heads=hkv, kernel=pgd.KERNEL_AUTO if cut else UMMA,
                                      **a)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=d ** -0.5, **c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap", [20.0, 50.0, 52.6, 53.0])
@pytest.mark.parametrize("log2_v", [-30, 40, 80])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("kernel", [pgd.KERNEL_TENSOR_CORE, UMMA])
def test_capped_scores_with_values_of_any_size(d, softcap, log2_v, far, kernel):
    """Scores as they come, or (far) all near the cap, where weights are at their largest."""
    b = Paged(22, [400, 65], 8, 2, d, scale_v=2.0 ** log2_v)
    if far:
        for r, n in enumerate(b.lengths):
            k = (torch.from_numpy(b.k_rows[r]).abs() + 0.5).bfloat16()
            b.k_rows[r] = k.double().numpy()
            b.write(b.k_pool, [r] * n, range(n), k.transpose(0, 1).to(DEV))
    rows, positions = packed([200, 0], [200, 65])
    q = b.queries(265)
    if far:
        q = q.abs() + 0.25
    scale = softcap / d if far else d ** -0.5
    out = pgd.paged_prefill_attention(q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions),
                                      None, 0, scale, num_kv_heads=2, softcap=softcap,
                                      kernel=kernel)
    assert pgd.get_device_error() == pgd.OK
    check(out, b, q, rows, positions, scale=scale, softcap=softcap, rounded=True)


