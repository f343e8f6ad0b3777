"""Refusals of libpgd_ext at the ends of its arguments' ranges, on the host."""
import ctypes

import pytest
import torch

import paged_gqa_decode_gb300 as pgd


@pytest.fixture(scope="module", autouse=True)
def ext():
    from paged_gqa_decode_gb300 import build
    build.build_library()
    return pgd.load_extension()


def attend(ext, prefill, kernel, **dims):
    """A call with host memory in place of tensors and no workspace: refused, or (on a machine
    with a GPU) found to lack the workspace; nothing is launched."""
    buf = ctypes.create_string_buffer(4096)
    at = (ctypes.addressof(buf) + 15) & ~15
    d = pgd.make_dims(**dict(dict(rows=2, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=4,
                                  max_pages_per_row=2), **dims))
    score = pgd.Score(30.0, None, None, None)
    opts = pgd.DecodeOptions(0, kernel)
    args = [ctypes.byref(d)] + ([2] if prefill else []) + [ctypes.byref(score), at, None, None, at,
                                                           at, at]
    args += ([at] if prefill else []) + [at, None, 0, 0.125, at, at, 0, ctypes.byref(opts), None]
    return (ext.pgdx_paged_prefill if prefill else ext.pgdx_paged_decode)(*args)


@pytest.mark.parametrize("dims", [dict(rows=65536), dict(num_q_heads=65536, num_kv_heads=65536)])
def test_more_than_the_per_token_grid_holds_is_refused(ext, dims):
    assert attend(ext, False, pgd.KERNEL_AUTO, **dims) == pgd.EUNSUPPORTED
    assert attend(ext, False, pgd.KERNEL_TENSOR_CORE, **dims) == pgd.EUNSUPPORTED
    assert attend(ext, True, pgd.KERNEL_TENSOR_CORE, **dims) == pgd.EUNSUPPORTED
    for kernel in (pgd.KERNEL_AUTO, pgd.KERNEL_PREFILL_UMMA):
        assert attend(ext, True, kernel, **dims) in (pgd.ECUDA, pgd.EWORKSPACE)
    fewer = {k: 65535 for k in dims}
    assert attend(ext, False, pgd.KERNEL_AUTO, **fewer) in (pgd.ECUDA, pgd.EWORKSPACE)


def test_a_scaled_base_past_the_range_of_doubles_is_refused():
    for theta, factor in ((1e300, 1e10), (1e10, 1e300)):
        with pytest.raises(pgd.PgdError) as e:
            pgd.Rotary(64, theta, scaling="ntk", factor=factor)
        assert e.value.status == pgd.EINVAL
    assert pgd.Rotary(64, 1e10, scaling="ntk", factor=1e4).plan.turns[0] > 0


def rotate(ext, *, rows, k_at, v_at, k_stride, v_stride, q_out):
    """4 query and 2 kv heads of 64 (rows of 256 and 128 values); places in bytes of one buffer."""
    buf = ctypes.create_string_buffer(1 << 16)
    at = (ctypes.addressof(buf) + 15) & ~15
    d = pgd.make_dims(rows=rows, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=4,
                      max_pages_per_row=2)
    far = at + 40000
    return ext.pgdx_rotary_append(ctypes.byref(d), ctypes.byref(pgd.Rotary(64, 1e4).plan),
                                  far, 256, at + q_out, at + k_at, k_stride, at + v_at, v_stride,
                                  at, 2, None, at, None, at, at, None)


# q_out is 1024 bytes of two tokens; k rows of 128 values: bytes [k_at + 2 i k_stride, + 256)
@pytest.mark.parametrize("rows,k_at,k_stride,q_out,hit", [
    (2, 6144, 128, 2048, False),      # q_out far before k
    (2, 6144, 128, 5136, True),       # reaches k's first row by 16 bytes
    (2, 6144, 128, 5120, False),      # ends where k begins
    (2, 6144, 128, 6640, True),       # k's last 16 bytes
    (2, 6144, 128, 6656, False),      # k ends where it begins
    (2, 6144, 1024, 6400, False),     # in the gap between k's rows, from 6400 to 8192
    (2, 6144, 1024, 7168, False),
    (2, 6144, 1024, 7184, True),      # reaches the second row
    (2, 6144, 1024, 6384, True),      # the first row's end
    (2, 6144, 1024, 8432, True),      # the second row's end
    (2, 6144, 1024, 8448, False),
    (1, 6144, 1024, 6400, False),     # a fused projection of one token: q, k, v in a row
    (3, 0, 128, 512, True),
])
def test_rotary_append_refuses_a_q_out_over_k_or_v(ext, rows, k_at, k_stride, q_out, hit):
    kw = dict(rows=rows, q_out=q_out)
    for call in (dict(k_at=k_at, k_stride=k_stride, v_at=30000, v_stride=128),
                 dict(v_at=k_at, v_stride=k_stride, k_at=30000, k_stride=128)):
        if hit:
            assert rotate(ext, **call, **kw) == pgd.EINVAL
        elif not torch.cuda.is_available():  # (with a device it would be launched)
            assert rotate(ext, **call, **kw) == pgd.ECUDA
