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


