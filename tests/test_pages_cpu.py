"""Refusals of the calls over shared pages, on the host: nothing is launched, with or
without a device."""
import ctypes

import pytest
import torch

import paged_gqa_decode_gb300 as pgd


@pytest.fixture(scope="module", autouse=True)
def ext():
    from paged_gqa_decode_gb300 import build
    build.build_library()
    return pgd.load_extension()


def places(sizes):
    """A buffer, and where in it arrays of these many int32s lie, one after another."""
    buf = (ctypes.c_int32 * (sum(sizes.values()) + 64))()
    at = (ctypes.addressof(buf) + 15) & ~15
    out = {}
    for name, n in sizes.items():
        out[name] = at
        at += 4 * ((n + 3) // 4 * 4)
    return buf, out


# ----------------------------------------------------------------- fork_rows

FORK = dict(table=6, lengths=2, parents=2, keep=2, shares=9, free=5, head=1, new_lengths=2,
            sources=2, targets=2, counts=2, head_out=1)


def fork(ext, over=None, by=0, **kw):
    """2 rows of width 3, 9 pages, 5 listed; `over`: (array, other, words in) laid over it."""
    buf, at = places(FORK)
    sizes = dict(rows=2, width=3, pages=9, num_free=5)
    for k, v in kw.items():
        (sizes if k in sizes else at)[k] = v
    if over:
        at[over[0]] = at[over[1]] + 4 * over[2]
    if by:
        at["sources"] += by
    return ext.pgdx_fork_rows(
        sizes["rows"], sizes["width"], sizes["pages"], at["table"], at["lengths"], at["parents"],
        at["keep"], at["shares"], at["free"], sizes["num_free"], at["head"], at["new_lengths"],
        at["sources"], at["targets"], at["counts"], at["head_out"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=0), dict(pages=0), dict(num_free=-1), dict(table=None),
    dict(lengths=None), dict(parents=None), dict(shares=None), dict(free=None),
    dict(new_lengths=None), dict(sources=None), dict(targets=None), dict(counts=None),
    dict(head_out=None), dict(by=2),
    dict(over=("new_lengths", "lengths", 0)), dict(over=("sources", "parents", 1)),
    dict(over=("targets", "keep", 0)), dict(over=("head_out", "head", 0)),
    dict(over=("counts", "table", 5)), dict(over=("targets", "shares", 8)),
    dict(over=("sources", "free", 4)), dict(over=("shares", "table", 4)),
    dict(over=("free", "shares", 1)), dict(over=("sources", "targets", 1)),
])
def test_fork_rows_refuses(ext, kw):
    assert fork(ext, **kw) == pgd.EINVAL


def test_fork_rows_refuses_sizes(ext):
    assert fork(ext, width=2 ** 26) == pgd.EUNSUPPORTED         # positions past int32
    assert fork(ext, rows=0, pages=2 ** 26) == pgd.EUNSUPPORTED
    far = ctypes.addressof((ctypes.c_char * 16)())
    many = dict(rows=8193, width=1)
    # (arrays of that length somewhere else: only their addresses are looked at)
    base = (far + 15) & ~15
    spread = {k: base + i * (1 << 34) for i, k in enumerate(FORK)}
    assert fork(ext, **many, **spread) == pgd.EUNSUPPORTED
    assert fork(ext, rows=8000, width=2 ** 18, **spread) == pgd.EUNSUPPORTED   # 2^30 entries and more


# ----------------------------------------------------------------- copy_pages

def copy(ext, layers=1, copies=2, layout=pgd.PAGE_MAJOR, head_dim=64, pools=None, **kw):
    buf, at = places(dict(pool=64, sources=2, targets=2, counts=2))
    at.update(kw)
    d = pgd.make_dims(rows=2, num_q_heads=2, num_kv_heads=2, head_dim=head_dim, num_pages=4,
                      max_pages_per_row=1, layout=layout)
    arr = (ctypes.c_void_p * max(1, layers if layers > 0 else 1))(
        *[at["pool"] if pools is None else pools] * max(1, layers))
    return ext.pgdx_copy_pages(ctypes.byref(d), layers, kw.get("k_pools", arr),
                               kw.get("v_pools", arr), copies, at["sources"], at["targets"],
                               at["counts"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layers=-1), 1), (dict(copies=-1), 1), (dict(layout=pgd.ROW_MAJOR), 2),
    (dict(layout=7), 1), (dict(head_dim=96), 2), (dict(sources=None), 1), (dict(targets=None), 1),
    (dict(k_pools=None), 1), (dict(v_pools=None), 1), (dict(pools=0), 1), (dict(pools=24), 1),
])
def test_copy_pages_refuses(ext, kw, status):
    assert copy(ext, **kw) == status


def test_copy_pages_of_nothing(ext):
    assert copy(ext, layers=0) == pgd.OK
    assert copy(ext, copies=0) == pgd.OK


# ----------------------------------------------------------------- compact_pages

COMPACT = dict(table=6, lengths=2, shares=40, free=5, head=1, new_table=6, new_shares=40, new_free=5,
               sources=4, targets=4, end=1, workspace=64)


def compact(ext, over=None, workspace_bytes=None, **kw):
    buf, at = places(COMPACT)
    sizes = dict(rows=2, width=3, pages=40, num_free=5, moves=4)
    for k, v in kw.items():
        (sizes if k in sizes else at)[k] = v
    if over:
        at[over[0]] = at[over[1]] + 4 * over[2]
    need = ext.pgdx_compact_workspace_bytes(sizes["pages"]) if sizes["pages"] > 0 else 0
    return ext.pgdx_compact_pages(
        sizes["rows"], sizes["width"], sizes["pages"], at["table"], at["lengths"], at["shares"],
        at["free"], sizes["num_free"], at["head"], sizes["moves"], at["new_table"],
        at["new_shares"], at["new_free"], at["sources"], at["targets"], at["end"],
        at["workspace"], need if workspace_bytes is None else workspace_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=0), dict(pages=0), dict(num_free=-1), dict(moves=-1),
    dict(table=None), dict(lengths=None), dict(shares=None), dict(free=None),
    dict(new_table=None), dict(new_shares=None), dict(new_free=None), dict(sources=None),
    dict(targets=None), dict(end=None), dict(workspace=None),
    dict(over=("new_table", "table", 1)), dict(over=("new_shares", "shares", 1)),
    dict(over=("new_free", "free", -1)), dict(over=("sources", "lengths", 0)),
    dict(over=("end", "head", 0)), dict(over=("sources", "targets", 3)),
    dict(over=("workspace", "new_shares", 0)), dict(over=("new_table", "shares", 0)),
])
def test_compact_pages_refuses(ext, kw):
    assert compact(ext, **kw) == pgd.EINVAL


def test_compact_pages_workspace(ext):
    assert compact(ext, workspace_bytes=ext.pgdx_compact_workspace_bytes(40) - 1) == pgd.EWORKSPACE
    assert ext.pgdx_compact_workspace_bytes(0) == 0
    # two bitmaps at least
    assert ext.pgdx_compact_workspace_bytes(1 << 20) >= (1 << 20) // 4
    assert compact(ext, pages=2 ** 26) == pgd.EUNSUPPORTED


# ----------------------------------------------------------------- shared_decode

def shared(ext, groups=1, scale=0.125, workspace_bytes=None, kernel=0, **kw):
    buf = ctypes.create_string_buffer(1 << 14)
    at = (ctypes.addressof(buf) + 15) & ~15
    names = ("q", "k_pool", "v_pool", "out", "starts", "pages", "table", "positions", "workspace")
    ptr = {n: at + 1024 * i for i, n in enumerate(names)}
    ptr.update(k_new=None, v_new=None)
    dims = dict(rows=2, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=4,
                max_pages_per_row=3, layout=pgd.PAGE_MAJOR)
    for k, v in kw.items():
        (dims if k in dims else ptr)[k] = (at + v[1] if isinstance(v, tuple) else v)
    d = pgd.make_dims(**dims)
    need = ext.pgdx_shared_decode_workspace_bytes(ctypes.byref(d), groups)
    return ext.pgdx_shared_decode(
        ctypes.byref(d), groups, ptr["starts"], ptr["pages"], ptr["q"], ptr["k_new"], ptr["v_new"],
        ptr["k_pool"], ptr["v_pool"], ptr["table"], ptr["positions"], None, scale, ptr["out"],
        ptr["workspace"], need if workspace_bytes is None else workspace_bytes,
        ctypes.byref(pgd.DecodeOptions(0, kernel)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(kernel=6), 1), (dict(kernel=-1), 1), (dict(kernel=pgd.KERNEL_CUDA_CORE), 2),
    (dict(kernel=pgd.KERNEL_PREFILL_PAIR), 2),
    (dict(groups=-1), 1), (dict(groups=8193), 2), (dict(rows=65536), 2), (dict(rows=-1), 1),
    (dict(layout=pgd.ROW_MAJOR, num_pages=6), 2), (dict(head_dim=32), 2),
    (dict(num_q_heads=18), 2), (dict(num_q_heads=3), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(k_pool=None), 1), (dict(v_pool=None), 1),
    (dict(table=None), 1), (dict(positions=None), 1), (dict(out=None), 1), (dict(starts=None), 1),
    (dict(pages=None), 1), (dict(workspace=None), 1), (dict(k_new=("at", 0)), 1),
    (dict(v_new=("at", 0)), 1), (dict(q=("at", 8)), 1), (dict(out=("at", 8)), 1),
    (dict(workspace=("at", 8)), 1), (dict(starts=("at", 2)), 1), (dict(workspace_bytes=64), 6),
])
def test_shared_decode_refuses(ext, kw, status):
    assert shared(ext, **kw) == status


def test_shared_decode_of_no_rows(ext):
    assert shared(ext, rows=0) == pgd.OK


def test_shared_decode_workspace(ext):
    d = pgd.make_dims(rows=256, num_q_heads=32, num_kv_heads=8, head_dim=128, num_pages=9000,
                      max_pages_per_row=600)
    size = pgd.shared_decode_workspace_bytes(d, 4)
    assert size > 256 * 32 * 5 * 130 * 4 and size % 8 == 0
    assert pgd.shared_decode_workspace_bytes(d, 8193) == 0
    d.head_dim = 96
    assert pgd.shared_decode_workspace_bytes(d, 4) == 0


def test_python_checks_without_a_device():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pgd.fork_rows(i(2, 3), i(2), i(2), i(9), i(5))
    with pytest.raises(ValueError, match="CUDA"):
        pgd.compact_pages(i(2, 3), i(2), i(9), i(5))
    p = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pgd.copy_pages(p, p, i(1), i(1), num_kv_heads=2, head_dim=64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for kw in (dict(group_starts=i(2)), dict(group_pages=i(1))):
        with pytest.raises(ValueError, match="together"):
            pgd.paged_decode_attention(q, p, p, i(2, 3), i(2), num_kv_heads=2, **kw)
