"""rotary_append_paged and the calls beside it: slots into dense rows."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def normal(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def test_slots_into_row_major_pools():
    """Slots alone do not say how many pages a dense row has: given, or refused."""
    rows, hkv, d, width = 3, 2, 64, 4
    k = normal(70, 5, hkv, d)
    v = normal(71, 5, hkv, d)
    q = normal(72, 5, 4, d)
    positions = i32([0, 70, 255, 3, 130])
    row = np.array([0, 2, 1, 1, 2])
    slots = i32(row * width * 64 + np.array([0, 70, 255, 3, 130]))
    pools = lambda: (torch.zeros(rows, hkv, width * 64, d, device=DEV).bfloat16() for _ in range(2))  # noqa: E731
    rotary = pgd.Rotary(d, 1e4)
    k1, v1 = pools()
    with pytest.raises(ValueError, match="max_pages_per_row"):
        pgd.rotary_append_paged(q, k, v, positions, k1, v1, rotary=rotary, slots=slots,
                                layout=pgd.ROW_MAJOR)
    assert not k1.any() and not v1.any()
    got = pgd.rotary_append_paged(q, k, v, positions, k1, v1, rotary=rotary, slots=slots,
                                  layout=pgd.ROW_MAJOR, max_pages_per_row=width)
    k2, v2 = pools()
    same = pgd.rotary_append_paged(q, k, v, positions, k2, v2, rotary=rotary, rows=i32(row),
                                   table_rows=rows, layout=pgd.ROW_MAJOR, max_pages_per_row=width)
    assert pgd.get_device_error() == pgd.OK
    assert torch.equal(got, same) and torch.equal(k1, k2) and torch.equal(v1, v2)
    assert torch.equal(v1[torch.from_numpy(row), :, positions.long().cpu()], v)
    with pytest.raises(ValueError, match="max_pages_per_row"):
        pgd.rotary_append_paged(q, k, v, positions, k1, v1, rotary=rotary, layout=pgd.ROW_MAJOR,
                                rows=i32(row), table_rows=rows)


def test_write_slots_into_row_major_pools():
    rows, hkv, d, width = 3, 2, 64, 4
    k, v = normal(73, 4, hkv, d), normal(74, 4, hkv, d)
    row, n = np.array([0, 2, 1, 2]), np.array([0, 70, 255, 130])
    slots = i32(row * width * 64 + n)
    k1, v1 = (torch.zeros(rows, hkv, width * 64, d, device=DEV).bfloat16() for _ in range(2))
    pgd.kv_write_slots(k, v, slots, k1, v1, layout=pgd.ROW_MAJOR, max_pages_per_row=width)
    k2, v2 = torch.zeros_like(k1), torch.zeros_like(v1)
    for t in range(4):
        k2[row[t], :, n[t]], v2[row[t], :, n[t]] = k[t], v[t]
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    assert pgd.get_device_error() == pgd.OK
