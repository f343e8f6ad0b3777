"""The C ABI of libpgd_ext without a GPU: it builds for sm_103a, loads, exports
exactly the symbols include/pgd_ext.h declares, refuses bad arguments on the
host before touching a device, and computes the rotary frequencies (host code)
as the plain 64-bit implementation does."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import step_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pgd_ext.h")


@pytest.fixture(scope="module", autouse=True)
def ext():
    from paged_gqa_decode_gb300 import build
    build.build_library()
    return pgd.load_extension()


def test_library_exports_every_declared_symbol_and_nothing_else():
    declared = set(re.findall(r"PGD_API\s+[\w\s\*]+?\b(pgdx_\w+)\s*\(", open(HEADER).read()))
    out = subprocess.run(["nm", "-D", "--defined-only", pgd.EXT_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert {s for s in exported if not s.startswith("_")} == declared and declared


# ----------------------------------------------------------------- assign_pages

def _assign(ext, **kw):
    a = (ctypes.c_int32 * 64)()
    at = ctypes.addressof(a)
    # 2 requests of width 3, 4 tokens, 5 free pages, each array its own place in the buffer
    args = dict(requests=2, width=3, pages=9, tokens=4, table=at, cached=at + 24, new=at + 32,
                free=at + 40, num_free=5, head=at + 60, rows=at + 64, positions=at + 80,
                slots=at + 96, starts=at + 112, lengths=at + 124, head_out=at + 132)
    args.update({k: (at + v[1] if isinstance(v, tuple) else v) for k, v in kw.items()})
    return ext.pgdx_assign_pages(*args.values(), None)


@pytest.mark.parametrize("kw", [
    dict(requests=-1), dict(width=0), dict(pages=0), dict(tokens=-1), dict(num_free=-1),
    dict(table=None), dict(cached=None), dict(new=None), dict(free=None), dict(rows=None),
    dict(positions=None), dict(slots=None), dict(starts=None), dict(lengths=None),
    dict(head_out=None),
    dict(lengths=("at", 24)),      # over cached
    dict(head_out=("at", 60)),     # over head
    dict(slots=("at", 84)),        # over positions
    dict(table=("at", 44)),        # over the free pages
    dict(rows=("at", 66)),         # misaligned
])
def test_assign_pages_refuses(ext, kw):
    assert _assign(ext, **kw) == pgd.EINVAL


def test_assign_pages_refuses_positions_past_int32(ext):
    assert _assign(ext, pages=2 ** 26) == pgd.EUNSUPPORTED
    assert _assign(ext, requests=0, width=2 ** 26) == pgd.EUNSUPPORTED


def test_assign_pages_python_checks():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pgd.assign_pages(i(2, 3), i(2), i(2), i(4), num_tokens=4, num_pages=9)


# ----------------------------------------------------------------- rotary

def turns_of(rotary):
    half = rotary.plan.rotary_dim // 2
    return np.array([int(rotary.plan.turns[i]) for i in range(half)], dtype=np.float64) / 2.0 ** 64


@pytest.mark.parametrize("rotary_dim", [16, 48, 64, 128])
@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=32.0, original=4096.0),
    dict(scaling="yarn", factor=40.0, original=2048.0, beta_fast=16.0, beta_slow=2.0,
         exact_bounds=True),
    dict(scaling="banded", factor=8.0, original=8192.0, low_band=1.0, high_band=4.0),
])
@pytest.mark.parametrize("theta", [1e4, 1.5e5, 1e6])
def test_rotary_frequencies(rotary_dim, kw, theta):
    freq, factor = ref.frequencies(rotary_dim, theta, **kw)
    names = {"original": "original_positions"}
    rot = pgd.Rotary(rotary_dim, theta, **{names.get(k, k): v for k, v in kw.items()})
    # a frequency comes out of a few 64-bit operations (exponents up to about 16): 2^-48 is ample;
    # it is kept in whole multiples of 2^-64 turns
    np.testing.assert_allclose(turns_of(rot) * 2 * np.pi, freq, rtol=2.0 ** -48,
                               atol=2 * np.pi * 2.0 ** -64)
    assert rot.plan.factor == np.float32(factor)
    assert all(int(t) == 0 for t in rot.plan.turns[rotary_dim // 2:])


def test_rotary_attention_factor():
    assert pgd.Rotary(64, 1e4, attention_factor=1.25).plan.factor == 1.25
    assert pgd.Rotary(64, 1e4, scaling="yarn", factor=4.0, original_positions=4096.0,
                      attention_factor=1.0).plan.factor == 1.0


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=24), 2), (dict(rotary_dim=0), 2), (dict(rotary_dim=144), 2),
    (dict(theta=1.0), 1), (dict(theta=float("inf")), 1), (dict(theta=float("nan")), 1),
    (dict(scaling="linear", factor=0.5), 1), (dict(scaling="ntk", factor=float("nan")), 1),
    (dict(scaling="yarn", factor=2.0), 1),                                  # no original_positions
    (dict(scaling="yarn", factor=2.0, original_positions=64.0, beta_fast=1.0), 1),
    (dict(scaling="banded", factor=2.0, original_positions=64.0, low_band=4.0), 1),
])
def test_rotary_refuses(kw, status):
    args = dict(rotary_dim=64, theta=1e4)
    args.update(kw)
    with pytest.raises(pgd.PgdError) as e:
        pgd.Rotary(**args)
    assert e.value.status == status


def test_rotary_refuses_unknown_scaling_and_bad_factor():
    with pytest.raises(ValueError):
        pgd.Rotary(64, 1e4, scaling="cubic")
    with pytest.raises(ValueError):
        pgd.Rotary(64, 1e4, attention_factor=-1.0)


def _append(ext, dims=None, rotary=None, **kw):
    buf = ctypes.create_string_buffer(8192)
    at = (ctypes.addressof(buf) + 15) & ~15
    d = dims or pgd.make_dims(rows=2, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=4,
                              max_pages_per_row=2)
    rot = rotary or pgd.Rotary(64, 1e4)
    args = dict(q=at, q_stride=256, q_out=at + 2048, k=at + 4096, k_stride=128, v=at + 5120,
                v_stride=128, table=at, table_rows=2, rows=None, positions=at, slots=None,
                k_pool=at + 6144, v_pool=at + 7168)
    args.update({k: (at + v[1] if isinstance(v, tuple) else v) for k, v in kw.items()})
    return ext.pgdx_rotary_append(ctypes.byref(d), ctypes.byref(rot.plan), *args.values(), None)


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(positions=None), dict(k_pool=None), dict(v_pool=None),
    dict(q=None), dict(q_out=None), dict(table=None),
    dict(rows=("at", 0), table_rows=0),
    dict(q_stride=250), dict(q_stride=252), dict(k_stride=120), dict(v_stride=132),
    dict(q=("at", 8)), dict(k=("at", 4098)),
    dict(q_out=("at", 0), q_stride=384),      # in place needs contiguous q
    dict(q_out=("at", 512)),                  # overlaps q
])
def test_rotary_append_refuses(ext, kw):
    assert _append(ext, **kw) == pgd.EINVAL


def test_rotary_append_refuses_shapes(ext):
    dims = lambda **kw: pgd.make_dims(**dict(dict(  # noqa: E731
        rows=2, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=4, max_pages_per_row=2), **kw))
    assert _append(ext, rotary=pgd.Rotary(128, 1e4)) == pgd.EINVAL        # wider than the head
    assert _append(ext, dims=dims(head_dim=96)) == pgd.EUNSUPPORTED
    assert _append(ext, dims=dims(layout=pgd.ROW_MAJOR, num_pages=2), table=None) == pgd.EINVAL
    bad = pgd.Rotary(64, 1e4)
    bad.plan.rotary_dim = 20
    assert _append(ext, rotary=bad) == pgd.EINVAL
    assert _append(ext, dims=dims(rows=0), k=None) == pgd.OK


def test_rotary_append_python_checks():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pgd.rotary_append_paged(None, b(2, 1, 64), b(2, 1, 64), torch.zeros(2, dtype=torch.int32),
                                b(1, 1, 64, 64), b(1, 1, 64, 64), rotary=pgd.Rotary(64, 1e4))


# ----------------------------------------------------------------- attention

def _dims(**kw):
    return pgd.make_dims(**dict(dict(rows=2, num_q_heads=4, num_kv_heads=2, head_dim=64,
                                     num_pages=4, max_pages_per_row=2), **kw))


def _attend(ext, prefill, dims=None, score=None, **kw):
    """A call whose arguments would all do but for kw; tensors are places in a host buffer."""
    buf = ctypes.create_string_buffer(8192)
    at = (ctypes.addressof(buf) + 15) & ~15
    s = dict(softcap=30.0, alibi_slopes=None, first_key=None, prefix_len=None)
    s.update({k: (at + v[1] if isinstance(v, tuple) else v) for k, v in (score or {}).items()})
    args = dict(q=at, k_new=None, v_new=None, k_pool=at + 1024, v_pool=at + 2048, table=at + 3136)
    if prefill:
        args["rows"] = at + 3200
    args.update(positions=at + 3300, sinks=None, window=0, scale=0.125, out=at + 4096,
                workspace=at + 5120, workspace_bytes=0)
    opts = pgd.DecodeOptions(**kw.pop("opts", {}))
    d = dims or _dims()
    table_rows = kw.pop("table_rows", 2)
    given = kw.pop("given", True)
    args.update({k: (at + v[1] if isinstance(v, tuple) else v) for k, v in kw.items()})
    head = [ctypes.byref(d) if dims is not False else None]
    if prefill:
        head.append(table_rows)
    call = ext.pgdx_paged_prefill if prefill else ext.pgdx_paged_decode
    return call(*head, ctypes.byref(pgd.Score(**s)) if given else None, *args.values(),
                ctypes.byref(opts), None)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k_pool=None), dict(v_pool=None), dict(positions=None), dict(out=None),
    dict(table=None), dict(q=("at", 8)), dict(k_pool=("at", 1032)), dict(out=("at", 4098)),
    dict(k_new=("at", 0)), dict(v_new=("at", 0)),             # one of the two alone
    dict(k_new=("at", 4), v_new=("at", 0)),
    dict(scale=float("nan")), dict(scale=float("inf")),
    dict(given=False),
    dict(score=dict(softcap=float("nan"))), dict(score=dict(softcap=float("inf"))),
    dict(score=dict(alibi_slopes=("at", 3))), dict(score=dict(first_key=("at", 2))),
    dict(opts=dict(kernel=-1)), dict(opts=dict(kernel=6)),
])
def test_attention_refuses(ext, prefill, kw):
    assert _attend(ext, prefill, **dict(kw)) == pgd.EINVAL


@pytest.mark.parametrize("prefill", [False, True])
def test_attention_refuses_dims(ext, prefill):
    assert _attend(ext, prefill, dims=False) == pgd.EINVAL
    assert _attend(ext, prefill, dims=_dims(rows=-1)) == pgd.EINVAL
    assert _attend(ext, prefill, dims=_dims(num_q_heads=5)) == pgd.EINVAL
    assert _attend(ext, prefill, dims=_dims(head_dim=96)) == pgd.EUNSUPPORTED
    pages32 = _dims()
    pages32.page_size = 32
    assert _attend(ext, prefill, dims=pages32) == pgd.EUNSUPPORTED
    assert _attend(ext, prefill, dims=_dims(num_pages=2 ** 25)) == pgd.EUNSUPPORTED
    # dense rows without a pool for each
    assert _attend(ext, prefill, dims=_dims(layout=pgd.ROW_MAJOR, num_pages=2),
                   table=None) == pgd.EINVAL
    assert _attend(ext, prefill, dims=_dims(rows=0), q=None, out=None) == pgd.OK


def test_attention_refuses_the_other_calls_kernels(ext):
    for kernel in (pgd.KERNEL_CUDA_CORE, pgd.KERNEL_PREFILL_TILED, pgd.KERNEL_PREFILL_PAIR):
        for prefill in (False, True):
            assert _attend(ext, prefill, opts=dict(kernel=kernel)) == pgd.EUNSUPPORTED
    assert _attend(ext, False, opts=dict(kernel=pgd.KERNEL_PREFILL_UMMA)) == pgd.EINVAL


@pytest.mark.parametrize("prefill", [False, True])
def test_attention_refuses_caps_out_of_range(ext, prefill):
    assert _attend(ext, prefill, score=dict(softcap=1e16)) == pgd.EUNSUPPORTED
    assert _attend(ext, prefill, score=dict(softcap=3e38), scale=1e-30) == pgd.EUNSUPPORTED
    assert _attend(ext, prefill, score=dict(softcap=1e-30), scale=1e10) == pgd.EINVAL
    assert _attend(ext, prefill, score=dict(softcap=3e38), scale=1e30) == pgd.EINVAL


def test_decode_refuses_a_prefix_and_prefill_a_missing_map(ext):
    assert _attend(ext, False, score=dict(prefix_len=("at", 0))) == pgd.EINVAL
    assert _attend(ext, True, score=dict(prefix_len=("at", 2))) == pgd.EINVAL
    assert _attend(ext, True, rows=None) == pgd.EINVAL
    assert _attend(ext, True, table_rows=0) == pgd.EINVAL
    assert _attend(ext, True, table_rows=-3) == pgd.EINVAL


def test_attention_python_checks():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)     # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pgd.paged_decode_attention(b(2, 4, 64), b(4, 2, 64, 64), b(4, 2, 64, 64), i(2, 2), i(2),
                                   num_kv_heads=2, softcap=30.0)
    with pytest.raises(ValueError, match="CUDA"):
        pgd.paged_prefill_attention(b(2, 4, 64), b(4, 2, 64, 64), b(4, 2, 64, 64), i(2, 2), i(2),
                                    i(2), num_kv_heads=2, alibi_slopes=torch.zeros(4))
