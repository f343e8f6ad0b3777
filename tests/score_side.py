"""What the tests of the modified scores share: a paged batch, its plain 64-bit
result, and the bound that a kernel's outputs are held to.

The bound.  Off by relative e_j, a softmax's weights move an output by at most
2 max_j e_j sum_j p_j |v_j| (e_j small).  A weight's error: its score's, in
natural units -- the fp32 products, at most D additions of 2^-24 of scale sum_i
|q_i k_ij| (2^-17 at D = 128; the tensor core may truncate, so twice that); the
cap, 6e-7 relative of a score of at most 0.76 cap in its polynomial and a few
2^-23 of the cap in its other form: under 2^-20 cap; the bias, three roundings:
2^-22 of it -- plus the weight's own: the exponential 2^-22 and its argument's
rounding 2^-23 of it (at most 2^-16 at scores of 2^7), the bf16 head and
residual 2^-16, the sums' additions (a few hundred of 2^-24 in a row) 2^-16:
together under 2^-14.  The tcgen05 prefill rounds each weight to bf16 in the
product with V (half a step, 2^-8 of it), not in the row sums: sum_j p_j |v_j|
times that more.  The result is rounded to bf16 once: 2^-8 of it, or, below 2^-126,
where bf16 values are 2^-133 apart, 2^-134.  A weight below 2^-126 of the
denominator's largest term is no normal fp32 number and may be taken as zero:
2^-126 sum_j |v_j|."""
from __future__ import annotations

import numpy as np
import torch

import paged_gqa_decode_gb300 as pgd
from tests import step_reference as ref

DEV = "cuda:0"


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Paged:
    """Rows of `lengths` cached positions in a shuffled pool (page-major), tables
    padded to `width` entries; pool positions out of use hold NaN."""

    def __init__(self, seed, lengths, hq, hkv, d, width=None, layout=pgd.PAGE_MAJOR, scale_v=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.layout = hq, hkv, d, layout
        self.lengths = np.asarray(lengths)
        need = -(-self.lengths // 64)
        self.width = width or max(1, int(need.max(initial=1)))
        self.pages = int(need.sum()) + 3
        if layout == pgd.ROW_MAJOR:
            self.pages = len(lengths) * self.width
            self.table_np = np.arange(self.pages).reshape(len(lengths), self.width)
        else:
            order = rng.permutation(self.pages)
            self.table_np = np.zeros((len(lengths), self.width), dtype=np.int64)
            at = 0
            for r, k in enumerate(need):
                self.table_np[r, :k] = order[at:at + k]
                at += k
        g = torch.Generator().manual_seed(seed)
        self.k_rows, self.v_rows = [], []
        shape = (self.pages, hkv, 64, d)
        kp, vp = torch.full(shape, float("nan")), torch.full(shape, float("nan"))
        for r, n in enumerate(self.lengths):
            k = torch.randn(hkv, int(n), d, generator=g).bfloat16()
            v = (torch.randn(hkv, int(n), d, generator=g) * scale_v).bfloat16()
            self.k_rows.append(k.double().numpy())
            self.v_rows.append(v.double().numpy())
            for j in range(int(need[r])):
                a, b = 64 * j, min(64 * j + 64, int(n))
                kp[self.table_np[r, j], :, :b - a] = k[:, a:b].float()
                vp[self.table_np[r, j], :, :b - a] = v[:, a:b].float()
        self.k_pool, self.v_pool = self._lay(kp), self._lay(vp)
        self.table = i32(self.table_np)
        self.gen = g

    def _lay(self, pool):
        """Page-major [pages][kv heads][64][D] to the layout under test, bf16 on the GPU."""
        if self.layout == pgd.HEAD_MAJOR:
            pool = pool.transpose(0, 1)
        elif self.layout == pgd.ROW_MAJOR:
            pool = pool.view(len(self.lengths), self.width, self.hkv, 64, self.d).transpose(1, 2)
        return pool.contiguous().bfloat16().to(DEV)

    def write(self, pool, rows, positions, values):
        """Each token's heads at its position, in the layout under test, by plain indexing."""
        for t, (r, n) in enumerate(zip(rows, positions)):
            page = self.table_np[r, n // 64]
            if self.layout == pgd.PAGE_MAJOR:
                pool[page, :, n % 64] = values[t]
            elif self.layout == pgd.HEAD_MAJOR:
                pool[:, page, n % 64] = values[t]
            else:
                pool[r, :, n // 64, n % 64] = values[t]

    def queries(self, tokens):
        return torch.randn(tokens, self.hq, self.d, generator=self.gen).bfloat16().to(DEV)


def check(got, batch, q, rows, positions, *, scale, softcap=0.0, what="", rounded=False, **kw):
    """rounded: the kernel rounds the weights to bf16 (the tcgen05 prefill)."""
    host = lambda t: None if t is None else (  # noqa: E731
        t.double().cpu().numpy() if isinstance(t, torch.Tensor) else np.asarray(t))
    kw = {k: (v if k == "window" else host(v)) for k, v in kw.items()}
    want, mass, size, far = ref.attention(q.double().cpu().numpy(), batch.k_rows, batch.v_rows,
                                          rows, positions, scale=scale, softcap=softcap, **kw)
    d = batch.d
    weight = 2 * d * 2.0 ** -24 * size + softcap * 2.0 ** -20 + far * 2.0 ** -22 + 2.0 ** -14
    if rounded:
        weight = weight + 2.0 ** -9        # (twice the weights' error is taken below)
    bound = (2 * weight * mass) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want) + 2.0 ** -134
    group = batch.hq // batch.hkv
    v_sums = [np.repeat(np.abs(v).sum(axis=1), group, axis=0) for v in batch.v_rows]
    at_row = [r if 0 <= r < len(v_sums) else 0 for r in rows]
    bound = bound + 2.0 ** -126 * np.stack([v_sums[r] for r in at_row])
    g = got.double().cpu().numpy()
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    excess = np.abs(g - want) - bound
    at = np.unravel_index(np.argmax(excess), excess.shape)
    assert excess.max() <= 0, \
        f"{what}: at {at} got {g[at]} for {want[at]}, {excess.max()} over the bound {bound[at]}"
