"""Refusals of libpgd_ext at the ends of its arguments' ranges, on the host."""
import ctypes

import pytest

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
