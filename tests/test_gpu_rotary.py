"""rotary_append_paged against the plain 64-bit rotation: q, the pools, and
everything that has to stay as it was."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import step_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# A result is x c - y s in fp32, rounded to bf16 once: half a bf16 step (2^-8 of it), plus what
# the fp32 part is off by.  cos and sin: sincospif within 2 ulp (2^-23), the phase held to 2^-32
# turns and 24 bits (2 pi 2^-26), the factor's product and fp32 value 2^-23: under 2^-21 of factor;
# two products and a sum round by 2^-24 each.  So off by at most 2^-20 factor (|x| + |y|).
HALF_STEP, PART = 2.0 ** -8, 2.0 ** -20


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


def f64(t):
    return t.double().cpu().numpy()


def close(got, x, positions, freq, factor, interleaved, what):
    x, got = f64(x), f64(got)
    want = ref.rotate(x, positions, freq, factor, interleaved)
    rd = 2 * len(freq)
    size = np.zeros_like(x)
    if interleaved:
        pair = np.abs(x[..., 0:rd:2]) + np.abs(x[..., 1:rd:2])
        size[..., 0:rd:2] = size[..., 1:rd:2] = pair
    else:
        pair = np.abs(x[..., :rd // 2]) + np.abs(x[..., rd // 2:rd])
        size[..., :rd // 2] = size[..., rd // 2:rd] = pair
    bound = HALF_STEP * np.abs(want) + 2 * PART * abs(factor) * size
    bound[..., rd:] = 0.0
    diff = np.abs(got - want)
    assert np.all(diff <= bound), f"{what}: {np.max(diff - bound)} over its bound"


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=32.0, original=4096.0),
            dict(scaling="banded", factor=8.0, original=8192.0)]


def make(kw, rotary_dim, theta, interleaved):
    freq, factor = ref.frequencies(rotary_dim, theta, **kw)
    names = {"original": "original_positions"}
    rot = pgd.Rotary(rotary_dim, theta, interleaved=interleaved,
                     **{names.get(k, k): v for k, v in kw.items()})
    return rot, freq, factor


POSITIONS = [0, 1, 63, 64, 4095, 65536, 1234567, 2 ** 24 + 1, 2 ** 31 - 1]


@pytest.mark.parametrize("hq,hkv,d,rotary_dim", [
    (14, 2, 64, 64), (14, 2, 64, 16), (64, 8, 64, 48), (32, 8, 128, 128), (32, 8, 128, 64),
    (8, 8, 128, 112), (1, 1, 64, 32), (64, 64, 128, 96), (3, 1, 128, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k.get("scaling", "none"))
def test_slots(hq, hkv, d, rotary_dim, interleaved, kw):
    positions = POSITIONS
    p, pages = len(positions), 3
    rot, freq, factor = make(kw, rotary_dim, 1e4, interleaved)
    q, k, v = normal(1, p, hq, d), normal(2, p, hkv, d), normal(3, p, hkv, d)
    kp, vp = normal(4, pages, hkv, 64, d), normal(5, pages, hkv, 64, d)
    k0, v0, q0 = kp.clone(), vp.clone(), q.clone()
    slots = np.random.default_rng(6).permutation(pages * 64)[:p]
    out = pgd.rotary_append_paged(q, k, v, i32(positions), kp, vp, rotary=rot, slots=i32(slots))
    assert pgd.get_device_error() == pgd.OK
    close(out, q, positions, freq, factor, interleaved, "q")
    assert torch.equal(q, q0)
    pg, at = torch.from_numpy(slots // 64), torch.from_numpy(slots % 64)
    close(kp[pg, :, at], k, positions, freq, factor, interleaved, "k")
    k0[pg, :, at], v0[pg, :, at] = kp[pg, :, at], v
    assert torch.equal(kp, k0) and torch.equal(vp, v0)    # the other slots are untouched


@pytest.mark.parametrize("layout", [pgd.PAGE_MAJOR, pgd.HEAD_MAJOR, pgd.ROW_MAJOR])
def test_layouts_equal_the_append(layout):
    """Rotated k in its slot is what rotating it and appending it gives."""
    r, hq, hkv, d, width = 5, 8, 2, 64, 4
    rot, _, _ = make({}, 32, 1e6, False)
    n = i32([0, 70, 255, 128, -1])
    table = i32(np.arange(20).reshape(5, 4) if layout == pgd.ROW_MAJOR
                else np.random.default_rng(1).permutation(20).reshape(5, 4))
    q, k, v = normal(1, r, hq, d), normal(2, r, hkv, d), normal(3, r, hkv, d)
    kp, vp = normal(4, 20 * hkv * 64 * d), normal(5, 20 * hkv * 64 * d)
    k1, v1, k2, v2 = kp.clone(), vp.clone(), kp.clone(), vp.clone()
    out = torch.full_like(q, 7.0)
    got = pgd.rotary_append_paged(q, k, v, n, kp, vp, rotary=rot, table=table, layout=layout,
                                  q_out=out)
    assert got is out
    assert torch.equal(out[4], torch.full_like(out[4], 7.0))     # inactive: left alone
    pgd.kv_append_paged(pgd.rotary_append_paged(k, k, v, n, k1, v1, rotary=rot, table=table,
                                                layout=layout), v, table, n, k2, v2, layout=layout)
    assert torch.equal(kp, k2) and torch.equal(vp, v2) and torch.equal(vp, v1)
    if layout == pgd.ROW_MAJOR:
        k3, v3 = normal(4, 20 * hkv * 64 * d), normal(5, 20 * hkv * 64 * d)
        pgd.rotary_append_paged(None, k, v, n, k3, v3, rotary=rot, layout=layout,
                                max_pages_per_row=width)
        assert torch.equal(k3, kp) and torch.equal(v3, vp)
    assert pgd.get_device_error() == pgd.OK


def test_views_of_a_fused_projection_and_in_place():
    p, hq, hkv, d = 70, 14, 2, 64
    rot, freq, factor = make(SCALINGS[3], 64, 1.5e5, False)
    qkv = normal(1, p, hq + 2 * hkv, d)
    keep = qkv.clone()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    n = np.arange(1000, 1000 + p)
    kp, vp = normal(2, 2, hkv, 64, d), normal(3, 2, hkv, 64, d)
    slots = i32(np.arange(p) + 5)
    out = pgd.rotary_append_paged(q, k, v, i32(n), kp, vp, rotary=rot, slots=slots)
    assert out.is_contiguous() and torch.equal(qkv, keep)
    close(out, q, n, freq, factor, False, "q")
    kp2, vp2, own = kp.clone().zero_(), vp.clone().zero_(), q.contiguous()
    got = pgd.rotary_append_paged(own, k.contiguous(), v.contiguous(), i32(n), kp2, vp2,
                                  rotary=rot, slots=slots, q_out=own)
    assert got is own and torch.equal(own, out)
    flat = lambda t: t.transpose(1, 2).reshape(-1, hkv, d)[5:5 + p]  # noqa: E731
    assert torch.equal(flat(kp), flat(kp2)) and torch.equal(flat(vp), flat(vp2))
    # one token: its stride does not matter
    one = pgd.rotary_append_paged(q[3:4], k[3:4], v[3:4], i32(n[3:4]), kp, vp, rotary=rot,
                                  slots=slots[3:4])
    assert torch.equal(one, out[3:4])


def test_packed_rows_and_bad_entries():
    rot, freq, factor = make({}, 64, 1e4, True)
    rows = [0, 0, 1, 1, 2, 0, 1, 0]
    n = [5, 6, 64, 200, 0, 64, -3, 2 ** 31 - 1]
    table = i32([[2, 0], [1, 9]])                  # row 1's second page is outside the pool
    q, k, v = normal(1, 8, 4, 64), normal(2, 8, 2, 64), normal(3, 8, 2, 64)
    kp, vp = normal(4, 3, 2, 64, 64), normal(5, 3, 2, 64, 64)
    k0 = kp.clone()
    out = torch.full_like(q, 3.0)
    pgd.rotary_append_paged(q, k, v, i32(n), kp, vp, rotary=rot, table=table, rows=i32(rows),
                            q_out=out)
    assert pgd.get_device_error() == pgd.EDEVICE_BOUNDS
    good = [0, 1, 5]
    close(out[good], q[good], np.array(n)[good], freq, factor, True, "q")
    close(torch.stack([kp[2, :, 5], kp[2, :, 6], kp[0, :, 0]]), k[good], np.array(n)[good], freq,
          factor, True, "k")
    for t in (2, 3, 4, 6, 7):
        assert torch.equal(out[t], torch.full_like(out[t], 3.0)), t
    k0[2, :, 5], k0[2, :, 6], k0[0, :, 0] = kp[2, :, 5], kp[2, :, 6], kp[0, :, 0]
    assert torch.equal(kp, k0)
    pgd.rotary_append_paged(q[:2], k[:2], v[:2], i32([1, 2]), kp, vp, rotary=rot,
                            slots=i32([-1, 3 * 64]), q_out=out[:2])
    assert pgd.get_device_error() == pgd.EDEVICE_BOUNDS
    assert torch.equal(kp, k0)


def test_special_values_pass_through():
    rot, _, _ = make({}, 16, 1e4, False)
    q, k, v = normal(1, 1, 1, 64), normal(2, 1, 1, 64), normal(3, 1, 1, 64)
    q[0, 0, 20], k[0, 0, 30], v[0, 0, 0] = float("nan"), float("inf"), float("-inf")
    kp, vp = normal(4, 1, 1, 64, 64), normal(5, 1, 1, 64, 64)
    out = pgd.rotary_append_paged(q, k, v, i32([9]), kp, vp, rotary=rot, slots=i32([0]))
    assert bool(torch.isnan(out[0, 0, 20])) and torch.isfinite(out[0, 0, :20]).all()
    assert torch.equal(kp[0, 0, 0, 16:], k[0, 0, 16:]) and torch.equal(vp[0, 0, 0], v[0, 0])


def test_graph_replay_and_stream():
    rot, freq, factor = make({}, 128, 1e6, False)
    q, k, v = normal(1, 33, 4, 128), normal(2, 33, 4, 128), normal(3, 33, 4, 128)
    kp, vp = normal(4, 1, 4, 64, 128), normal(5, 1, 4, 64, 128)
    n, slots, out = i32(np.arange(33)), i32(np.arange(33)), torch.empty_like(q)
    pgd.rotary_append_paged(q, k, v, n, kp, vp, rotary=rot, slots=slots, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pgd.rotary_append_paged(q, k, v, n, kp, vp, rotary=rot, slots=slots, q_out=out)
    n.add_(1000)
    graph.replay()
    close(out, q, np.arange(1000, 1033), freq, factor, False, "replayed")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(q)
    pgd.rotary_append_paged(q, k, v, n, kp, vp, rotary=rot, slots=slots, q_out=other, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other, out)


def test_rejects_wrong_tensors():
    rot = pgd.Rotary(64, 1e4)
    q, k = normal(1, 2, 2, 64), normal(2, 2, 2, 64)
    kp = normal(3, 1, 2, 64, 64)
    n = i32([0, 1])
    call = lambda q=q, k=k, v=k, n=n, **kw: pgd.rotary_append_paged(  # noqa: E731
        q, k, v, n, kp, kp.clone(), rotary=rot, **kw)
    with pytest.raises(pgd.PgdError):       # neither slots nor a table
        call()
    with pytest.raises(ValueError):
        call(q=q.float(), slots=n)
    with pytest.raises(ValueError):
        call(q=q.transpose(1, 2), slots=n)
    with pytest.raises(ValueError):
        call(n=n.long(), slots=n)
    with pytest.raises(ValueError):
        call(slots=n, q_out=q[:1])
    with pytest.raises(ValueError):         # one table row per token without rows
        call(table=i32([[0]]))
    with pytest.raises(pgd.PgdError):       # a token stride that is no multiple of 8 values
        call(q=torch.empty(2, 132, device=DEV, dtype=torch.bfloat16)[:, :128].view(2, 2, 64),
             slots=n)
