"""Memory that the binding makes for a call with `stream=`: never a block that work still
pending on the current stream uses, and a result's block is kept while that stream reads it."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests.score_side import DEV, Paged, i32

pytestmark = pytest.mark.gpu

PENDING = 60_000_000  # cycles that the current stream is busy (some 30 ms)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def calls():
    b = Paged(31, [2900 + 100, 700], 8, 2, 64, width=47)
    rows = np.repeat([0, 1], [100, 30])
    positions = np.r_[2900:3000, 600:630]
    q, r, n = b.queries(130), i32(rows), i32(positions)
    pools = (b.k_pool, b.v_pool, b.table)
    q2, n2 = q[:2].contiguous(), i32([2999, 629])
    k, v = (torch.randn(130, 2, 64, generator=b.gen).bfloat16().to(DEV) for _ in range(2))
    kp, vp = torch.zeros(8, 2, 64, 64, device=DEV).bfloat16(), torch.zeros(8, 2, 64, 64,
                                                                          device=DEV).bfloat16()
    rotary, slots = pgd.Rotary(64, 1e4), i32(np.arange(130))
    dense = [torch.randn(2, 2, 3008, 64, generator=b.gen).bfloat16().to(DEV) for _ in range(2)]
    lens = i32([70, 5])
    table = lambda: torch.zeros(2, 9, dtype=torch.int32, device=DEV)  # noqa: E731
    tables = iter([table() for _ in range(8)])
    return {
        "prefill": lambda s: pgd.paged_prefill_attention(q, *pools, r, n, num_kv_heads=2,
                                                         softcap=9.0, stream=s),
        "prefill_plain": lambda s: pgd.paged_prefill_attention(q, *pools, r, n, num_kv_heads=2,
                                                               stream=s),
        "decode": lambda s: pgd.paged_decode_attention(q2, *pools, n2, num_kv_heads=2, softcap=9.0,
                                                       pages_per_split=4, stream=s),
        "decode_plain": lambda s: pgd.paged_decode_attention(q2, *pools, n2, num_kv_heads=2,
                                                             pages_per_split=4, stream=s),
        "rows": lambda s: pgd.decode_rows_attention(q2, *dense, n2, pages_per_split=4, stream=s),
        "rotary": lambda s: pgd.rotary_append_paged(q, k, v, n, kp, vp, rotary=rotary, slots=slots,
                                                    stream=s),
        "slots": lambda s: pgd.page_slots(b.table, n, r, num_pages=b.pages, stream=s),
        "assign": lambda s: pgd.assign_pages(next(tables), lens, lens, i32(np.arange(9)),
                                             num_tokens=200, num_pages=9, stream=s).slots,
    }


NAMES = ["prefill", "prefill_plain", "decode", "decode_plain", "rows", "rotary", "slots", "assign"]


@pytest.mark.parametrize("name", NAMES)
def test_blocks_freed_under_pending_work(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None).clone()
    torch.cuda.synchronize()
    sizes = [64, 512, 1 << 12, 1 << 14, 1 << 16, 1 << 18, 1 << 20, 1 << 22]
    torch.cuda.empty_cache()
    blocks = [torch.empty(s, dtype=torch.int32, device=DEV) for s in sizes for _ in range(3)]
    torch.cuda.synchronize()
    spans = [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in blocks]
    torch.cuda._sleep(PENDING)
    for t in blocks:
        t.fill_(0x7fc07fc0)
    del blocks, t
    got = call(side)
    at = got.data_ptr()
    assert not any(a <= at < e for a, e in spans), "a block that a pending fill writes"
    torch.cuda.synchronize()
    assert torch.equal(got, want) and pgd.get_device_error() == pgd.OK


@pytest.mark.parametrize("name", NAMES)
def test_results_read_on_the_current_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = got.clone()
    torch.cuda._sleep(PENDING)
    read = got + 0
    shape, dtype = got.shape, got.dtype
    del got
    with torch.cuda.stream(side):  # would take the result's block if it were free
        later = [torch.full(shape, 3, dtype=dtype, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(read, want) and len(later) == 4


def test_scratch_of_calls_in_a_row_on_a_side_stream():
    call = calls()["prefill"]
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        torch.cuda._sleep(PENDING // 30)
        x = torch.empty(1 << 20, dtype=torch.int32, device=DEV)
        x.fill_(0x7fc07fc0)
        del x
        outs.append(call(side))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
