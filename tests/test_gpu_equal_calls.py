"""Equal calls give equal bits: no sum's order depends on when a block runs."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests.score_side import DEV, Paged, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("kw", [dict(softcap=50.0), dict(alibi=True), dict(softcap=1.0, alibi=True),
                                dict(first=True)], ids=str)
@pytest.mark.parametrize("cached,chunks", [([2370], [200]), ([0, 900, 31], [300, 70, 500])])
def test_prefill(kw, cached, chunks):
    b = Paged(41, np.add(cached, chunks), 16, 2, 64)
    rows = np.repeat(np.arange(len(cached)), chunks)
    positions = np.concatenate([np.arange(c, c + t) for c, t in zip(cached, chunks)])
    q = b.queries(len(rows))
    call = lambda: pgd.paged_prefill_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, b.table, i32(rows), i32(positions), num_kv_heads=2,
        softcap=kw.get("softcap", 0.0),
        alibi_slopes=torch.full((16,), 0.2, device=DEV) if kw.get("alibi") else None,
        first_key=i32(positions // 100 * 100) if kw.get("first") else None)
    want = call()
    assert all(torch.equal(call(), want) for _ in range(10))


def test_decode():
    b = Paged(42, [2000, 70, 900], 8, 2, 128)
    q, n = b.queries(3), i32([1999, 69, 899])
    call = lambda: pgd.paged_decode_attention(  # noqa: E731
        q, b.k_pool, b.v_pool, b.table, n, num_kv_heads=2, softcap=20.0, pages_per_split=3)
    want = call()
    assert all(torch.equal(call(), want) for _ in range(10))
