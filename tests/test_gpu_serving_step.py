"""The step's operators as they are used together: requests of ragged lengths
join, grow and decode over several passes -- pages and slots from lengths,
rotated q and k into the pools, capped (or biased) attention of prompts and
single tokens -- against a plain 64-bit implementation that knows only whole
sequences; eagerly, and with the pass captured into a graph."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_gb300 as pgd
from tests import step_reference as ref
from tests.score_side import DEV, i32

pytestmark = pytest.mark.gpu

# bf16 of rotated q and k: half a step each, 2^-8 of a product's terms (two of them), on top of
# the attention's own error (score_side)
ROTATED = 2 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


class Serving:
    def __init__(self, hq, hkv, d, requests, width, pages, tokens, kw, seed,
                 kernel=pgd.KERNEL_AUTO):
        self.hq, self.hkv, self.d, self.kw, self.kernel = hq, hkv, d, kw, kernel
        self.gen = torch.Generator().manual_seed(seed)
        self.tokens, self.pages = tokens, pages
        self.table = torch.zeros(requests, width, dtype=torch.int32, device=DEV)
        self.lengths = torch.zeros(requests, dtype=torch.int32, device=DEV)
        self.new = torch.zeros(requests, dtype=torch.int32, device=DEV)
        self.free = i32(np.random.default_rng(seed).permutation(pages))
        self.head = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.k_pool = torch.full((pages, hkv, 64, d), float("nan"), device=DEV).bfloat16()
        self.v_pool = self.k_pool.clone()
        self.rotary = pgd.Rotary(d // 2, 1e4, scaling="yarn", factor=8.0,
                                 original_positions=256.0, interleaved=True)
        self.freq = ref.frequencies(d // 2, 1e4, "yarn", 8.0, 256.0)
        self.qkv = torch.zeros(tokens, hq + 2 * hkv, d, device=DEV).bfloat16()
        self.q = torch.empty(tokens, hq, d, device=DEV).bfloat16()
        self.out = torch.empty_like(self.q)
        self.plan = pgd.PagePlan(*(torch.zeros(n, dtype=torch.int32, device=DEV) for n in
                                   (tokens, tokens, tokens, requests + 1, requests, 1)))
        self.prefix = torch.zeros(requests, dtype=torch.int32, device=DEV)
        self.slopes = torch.exp2(-torch.arange(1, hq + 1, device=DEV) * 8.0 / hq)
        dims = pgd.make_dims(rows=tokens, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                             num_pages=pages, max_pages_per_row=width)
        self.work = torch.empty(max(16, pgd.paged_decode_workspace_bytes(dims)),
                                dtype=torch.uint8, device=DEV)
        # what each request has seen, whole sequences in 64 bits
        self.k_seq = [np.zeros((hkv, 0, d)) for _ in range(requests)]
        self.v_seq = [np.zeros((hkv, 0, d)) for _ in range(requests)]

    def enqueue(self):
        hq, hkv = self.hq, self.hkv
        pgd.assign_pages(self.table, self.lengths, self.new, self.free, num_tokens=self.tokens,
                         num_pages=self.pages, free_head=self.head, out=self.plan)
        q, k, v = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:]
        pgd.rotary_append_paged(q, k, v, self.plan.positions, self.k_pool, self.v_pool,
                                rotary=self.rotary, slots=self.plan.slots, q_out=self.q)
        pgd.paged_prefill_attention(
            self.q, self.k_pool, self.v_pool, self.table, self.plan.rows, self.plan.positions,
            None, self.kw.get("window", 0), num_kv_heads=hkv, out=self.out, workspace=self.work,
            softcap=self.kw.get("softcap", 0.0),
            alibi_slopes=self.slopes if self.kw.get("alibi") else None, prefix_len=self.prefix,
            kernel=self.kernel)
        self.lengths.copy_(self.plan.lengths)
        self.head.copy_(self.plan.free_head)

    def feed(self, new):
        self.new.copy_(i32(new))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.gen).bfloat16())
        self.out.fill_(7.0)

    def expect(self, new):
        """Extends the sequences by the pass's tokens; checks the pass's outputs."""
        x = self.qkv.double().cpu().numpy()
        at, rows, positions, q = 0, [], [], []
        for r, t in enumerate(new):
            n0 = self.k_seq[r].shape[1]
            pos = np.arange(n0, n0 + t)
            part = x[at:at + t]
            args = (pos, self.freq[0], self.freq[1], True)
            q.append(ref.rotate(part[:, :self.hq], *args))
            k = ref.rotate(part[:, self.hq:self.hq + self.hkv], *args)
            self.k_seq[r] = np.concatenate([self.k_seq[r], k.transpose(1, 0, 2)], axis=1)
            self.v_seq[r] = np.concatenate(
                [self.v_seq[r], part[:, self.hq + self.hkv:].transpose(1, 0, 2)], axis=1)
            rows += [r] * t
            positions += pos.tolist()
            at += t
        assert pgd.get_device_error() == pgd.OK
        assert self.plan.lengths.tolist() == [s.shape[1] for s in self.k_seq]
        assert self.plan.rows.tolist()[:at] == rows
        assert self.plan.positions.tolist() == positions + [-1] * (self.tokens - at)
        slopes = self.slopes.double().cpu().numpy() if self.kw.get("alibi") else None
        want, mass, size, far = ref.attention(
            np.concatenate(q), self.k_seq, self.v_seq, rows, positions, scale=self.d ** -0.5,
            softcap=self.kw.get("softcap", 0.0), slopes=slopes, window=self.kw.get("window", 0),
            prefix=self.prefix.cpu().numpy())
        got = self.out.double().cpu().numpy()
        weight = (ROTATED + 2 * self.d * 2.0 ** -24) * size + self.kw.get("softcap", 0) * 2.0 ** -20 \
            + far * 2.0 ** -22 + 2.0 ** -14 + 2.0 ** -9
        # (weights off by a few percent: e^(2 w) - 1 in place of 2 w)
        bound = np.expm1(2 * weight) * mass * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want)
        excess = np.abs(got[:at] - want) - bound
        assert excess.max() <= 0, excess.max()
        # on the whole the errors are far below that bound: rms, over all outputs
        rms = np.sqrt(np.mean((got[:at] - want) ** 2) / np.mean(want ** 2))
        assert rms < 0.02, rms
        assert not got[at:].any()


PASSES = [[70, 0, 3, 129], [1, 64, 1, 1], [1, 1, 61, 1], [0, 1, 1, 200], [1, 1, 1, 1]]


@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(alibi=True), dict(softcap=20.0, window=90)])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kernel", [pgd.KERNEL_AUTO, pgd.KERNEL_PREFILL_UMMA])
def test_passes(hq, hkv, d, kw, captured, kernel):
    s = Serving(hq, hkv, d, requests=4, width=8, pages=24, tokens=256, kw=kw, seed=hq,
                kernel=kernel)
    s.prefix.copy_(i32([0, 0, 0, 40]))
    run = s.enqueue
    if captured:
        s.feed([0, 0, 0, 0])
        s.enqueue()                         # (loads the kernels; no tokens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.enqueue()
        run = graph.replay
    for new in PASSES:
        s.feed(new)
        run()
        s.expect(new)


def test_decode_steps_after_a_prompt():
    """The single-token form: assign, rotate and append, then paged_decode_attention."""
    s = Serving(16, 2, 64, requests=3, width=6, pages=12, tokens=200, kw=dict(softcap=25.0), seed=3)
    s.feed([150, 1, 30])
    s.enqueue()
    s.expect([150, 1, 30])
    s.tokens = 3
    plan = pgd.PagePlan(*(t[:n].contiguous() for t, n in zip(s.plan, (3, 3, 3, 4, 3, 1))))
    s.plan, s.qkv, s.q = plan, s.qkv[:3].contiguous(), s.q[:3].contiguous()
    for _ in range(40):                    # across page borders
        s.feed([1, 1, 1])
        pgd.assign_pages(s.table, s.lengths, s.new, s.free, num_tokens=3, num_pages=12,
                         free_head=s.head, out=s.plan)
        pgd.rotary_append_paged(s.qkv[:, :16], s.qkv[:, 16:18], s.qkv[:, 18:], s.plan.positions,
                                s.k_pool, s.v_pool, rotary=s.rotary, table=s.table, q_out=s.q)
        s.out = pgd.paged_decode_attention(s.q, s.k_pool, s.v_pool, s.table, s.plan.positions,
                                           num_kv_heads=2, softcap=25.0)
        s.lengths.copy_(s.plan.lengths)
        s.head.copy_(s.plan.free_head)
        s.expect([1, 1, 1])


def test_a_pool_past_32_bits():
    """Pages whose values lie past 2^31 of the pools (4.7 GB each): appended, decoded, and
    read by a prompt; pools are left uninitialised but for the row's pages."""
    hq, hkv, d, pages = 32, 8, 128, 36000
    k_pool = torch.empty(pages, hkv, 64, d, dtype=torch.bfloat16, device=DEV)
    v_pool = torch.empty_like(k_pool)
    table = i32([[pages - 1, 3, pages - 3]])
    gen = torch.Generator().manual_seed(5)
    n = 170
    x = torch.randn(n, hq + 2 * hkv, d, generator=gen).bfloat16().to(DEV)
    rotary = pgd.Rotary(d, 1e4)
    pos, rows = i32(np.arange(n)), i32(np.zeros(n))
    q = pgd.rotary_append_paged(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, k_pool, v_pool,
                                rotary=rotary, table=table, rows=rows)
    out = pgd.paged_prefill_attention(q, k_pool, v_pool, table, rows, pos, num_kv_heads=hkv,
                                      softcap=30.0)
    one = pgd.paged_decode_attention(q[-1:].contiguous(), k_pool, v_pool, table, i32([n - 1]),
                                     num_kv_heads=hkv, softcap=30.0)
    assert pgd.get_device_error() == pgd.OK
    # the same in a small pool
    small = (torch.empty(4, hkv, 64, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k2, v2 = small
    t2 = i32([[2, 0, 1]])
    q2 = pgd.rotary_append_paged(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, k2, v2,
                                 rotary=rotary, table=t2, rows=rows)
    out2 = pgd.paged_prefill_attention(q2, k2, v2, t2, rows, pos, num_kv_heads=hkv, softcap=30.0)
    one2 = pgd.paged_decode_attention(q2[-1:].contiguous(), k2, v2, t2, i32([n - 1]),
                                      num_kv_heads=hkv, softcap=30.0)
    assert torch.equal(q, q2) and torch.equal(out, out2) and torch.equal(one, one2)
    assert torch.equal(k_pool[pages - 1], k2[2]) and torch.equal(v_pool[pages - 3, :, :42],
                                                                 v2[1, :, :42])


def test_two_calls_at_once():
    """Two steps on two streams, each with tensors of its own, against each alone."""
    def make(seed):
        s = Serving(16, 2, 64, requests=2, width=20, pages=48, tokens=900, kw=dict(softcap=25.0),
                    seed=seed)
        s.feed([500, 380])
        return s
    alone = make(1), make(2)
    for s in alone:
        s.enqueue()
    torch.cuda.synchronize()
    both = make(1), make(2)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s, stream in zip(both, streams):
        with torch.cuda.stream(stream):
            s.enqueue()
    torch.cuda.synchronize()
    assert pgd.get_device_error() == pgd.OK
    for a, b in zip(alone, both):
        assert torch.equal(a.out, b.out) and torch.equal(a.table, b.table)
        b.expect([500, 380])
