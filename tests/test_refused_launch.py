"""Large forks and compactions whose cooperative launch is refused, as in a context of fewer SMs
than the device has: what is launched then (on the host, nothing is run), and what comes of it."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import page_side as side

DEV = "cuda:0"
HERE = os.path.dirname(os.path.abspath(__file__))
GRID, CLUSTER = 1, 2  # launches to refuse
DRY = 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from paged_gqa_decode_gb300 import build
    path = str(tmp_path_factory.mktemp("refused") / "librefused.so")
    run = subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", path,
                          os.path.join(HERE, "refused_launch.cu")], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    lib = ctypes.CDLL(path)
    lib.launched.restype = ctypes.c_char_p
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.fork_rows.argtypes = [i32] * 5 + [vp] * 12
    lib.compact_pages.argtypes = [i32] * 6 + [vp] * 13
    return lib


def fork_dry(lib, refused, rows, width):
    lib.refuse(refused, DRY)
    return lib.fork_rows(rows, width, 9, 5, 152, *[None] * 12), lib.launched().decode()


def compact_dry(lib, refused, rows, width):
    lib.refuse(refused, DRY)
    return lib.compact_pages(rows, width, 9, 5, 4, 152, *[None] * 13), lib.launched().decode()


def test_as_it_is_without_a_refusal(lib):
    assert fork_dry(lib, 0, 1000, 25) == (0, "c")
    assert fork_dry(lib, 0, 1000, 50) == (0, "kg")
    assert compact_dry(lib, 0, 1000, 25) == (0, "c")
    assert compact_dry(lib, 0, 1000, 50) == (0, "kg")


def test_a_refused_grid_becomes_a_cluster(lib):
    status, launched = compact_dry(lib, GRID, 1000, 50)
    assert status == 0 and launched == "kc"
    # (the shares' first step is taken back before)
    status, launched = fork_dry(lib, GRID, 1000, 50)
    assert status == 0 and launched == "kkc"


def test_all_refused(lib):
    for run in (fork_dry, compact_dry):
        status, launched = run(lib, GRID | CLUSTER, 1000, 50)
        assert status != 0 and "c" not in launched and "g" not in launched
    assert fork_dry(lib, GRID | CLUSTER, 1000, 50)[1] == "kk"
    assert fork_dry(lib, CLUSTER, 1000, 25)[0] != 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def sms():
    return torch.cuda.get_device_properties(DEV).multi_processor_count


def on_gpu(lib, refused, call, *args):
    """The call's status and the error word it leaves."""
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.refuse(refused, 0)
    torch.cuda.synchronize()
    status = call(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args],
                  err.data_ptr())
    torch.cuda.synchronize()
    return status, err.item()


@pytest.mark.gpu
@pytest.mark.parametrize("requests,beams,hi,grown", [(40, 8, 9000, 300), (500, 8, 900, 200)])
def test_forks_of_a_refused_grid(lib, requests, beams, hi, grown):
    rng = np.random.default_rng(51)
    table, lengths, shares, free, head, pages = side.random_state(rng, requests, beams, hi, grown)
    rows, width = table.shape
    parents = np.arange(rows) // beams * beams + rng.integers(0, beams, rows)
    parents = np.where(rng.random(rows) < 0.05, -1, parents)
    want, error = side.fork_rows(table, lengths, list(parents), None, shares, free, head, pages)
    assert not error and table.size > 40000
    for refused in (0, GRID, GRID | CLUSTER):
        before = dev(table), dev(shares), dev(free)
        t, s, f = (a.clone() for a in before)
        outs = [torch.empty(k, dtype=torch.int32, device=DEV) for k in (rows,) * 4 + (1,)]
        status = on_gpu(lib, refused, lib.fork_rows, rows, width, pages, len(free), sms(), t,
                        dev(lengths), dev(parents), s, f, dev([head]), *outs)
        if refused & CLUSTER:
            assert status[0] != 0
            for a, b in zip((t, s, f), before):
                assert torch.equal(a, b)
            continue
        assert status == (0, 0)
        for got, w in zip((t, s, f, *outs), want):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


@pytest.mark.gpu
def test_compactions_of_a_refused_grid(lib):
    rng = np.random.default_rng(52)
    table, lengths, shares, free, head, pages = side.random_state(rng, 300, 4, 5000, 300, spare=9000)
    rows, width = table.shape
    assert table.size + pages > 60000
    moves = pages // 3
    *want, end = side.compact_pages(table, lengths, shares, free, head, pages, moves)
    need = (pgd.load_extension().pgdx_compact_workspace_bytes(pages) + 3) // 4
    for refused in (0, GRID, GRID | CLUSTER):
        inputs = [dev(a) for a in (table, lengths, shares, free, [head])]
        outs = [torch.full((k,), -9, dtype=torch.int32, device=DEV)
                for k in (table.size, pages, len(free), moves, moves, 1)]
        workspace = torch.empty(need, dtype=torch.int32, device=DEV)
        status = on_gpu(lib, refused, lib.compact_pages, rows, width, pages, len(free), moves, sms(),
                        *inputs, *outs, workspace)
        if refused & CLUSTER:
            assert status[0] != 0 and all(bool((a == -9).all()) for a in outs)
            continue
        assert status == (0, 0)
        for got, w in zip(outs, want + [[end]]):
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(w).reshape(-1))
