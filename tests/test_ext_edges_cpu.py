"""Refusals of libpgd_ext at the ends of its arguments' ranges, on the host."""
import ctypes

import pytest

import paged_gqa_decode_gb300 as pgd


@pytest.fixture(scope="module", autouse=True)
def ext():
    from paged_gqa_decode_gb300 import build
    build.build_library()
    return pgd.load_extension()


