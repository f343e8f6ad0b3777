"""Measured cases of the serving step's operators: page assignment, rotary
positions written into the paged cache, and decode and prefill attention with
score caps, distance biases and document or prefix masks.

Every case runs in two forms: the plain one (elementary torch operations) and,
with ``own`` set, the framework's kernels through its public entry points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"

# (query heads, kv heads, head_dim) of the framework's workloads
SHAPES = {"qwen": (14, 2, 64), "gptoss": (64, 8, 64), "mistral": (32, 8, 128),
          "square": (8, 8, 128), "pairs": (16, 8, 64)}


def _attention(name, op, shape, **kw):
    case = dict(op=op, shape=shape, softcap=0.0, alibi=False, sinks=False, window=0, docs=0,
                prefix=0)
    case.update(kw)
    return case if name is None else dict(case, name=name)


def listed():
    return [
        # one decode step of a batch: every request gets one token, few get a page
        dict(name="assign_step", op="assign", requests=64, cached_lo=1024, cached_hi=32768, chunk=1,
             prompts=0, tokens=64),
        # a mixed pass: decode steps beside prompt chunks, padded to a fixed token count
        dict(name="assign_mixed", op="assign", requests=500, cached_lo=0, cached_hi=8192, chunk=512,
             prompts=50, tokens=27008),
        # thousands of short requests admitted at once
        dict(name="assign_many", op="assign", requests=4099, cached_lo=0, cached_hi=1000, chunk=61,
             prompts=4099, tokens=131072),
        # the smallest serving step: 4 rows, half layout over the whole head
        dict(name="rotary_step", op="rotary", shape="qwen", tokens=4, interleaved=False,
             rotary_dim=64, scaling="none", fused=False, far=300),
        # one prompt chunk, interleaved pairs over half of the head, far positions
        dict(name="rotary_chunk", op="rotary", shape="mistral", tokens=4096, interleaved=True,
             rotary_dim=64, scaling="linear", fused=False, far=1000000),
        # a long packed prefill out of a fused projection, frequencies stretched for long contexts
        dict(name="rotary_long", op="rotary", shape="gptoss", tokens=16001, interleaved=False,
             rotary_dim=64, scaling="yarn", fused=True, far=131072),
        # a small batch of short contexts with capped scores: latency
        _attention("decode_small", "decode", "qwen", rows=4, lo=1, hi=300, softcap=30.0),
        # a serving batch with capped scores and sinks
        _attention("decode_cap", "decode", "gptoss", rows=64, lo=512, hi=4096, softcap=50.0,
                   sinks=True),
        # long contexts with a distance bias, the longest rows' contexts starting at a document
        _attention("decode_bias", "decode", "mistral", rows=64, lo=1024, hi=16384, alibi=True,
                   docs=11001),
        # one prompt chunk over a long cached prefix, capped scores: too few items to fill the GPU
        _attention("prefill_chunk", "prefill", "mistral", rows=1, lo=8000, hi=8000, chunk=512,
                   softcap=50.0),
        # a packed pass of chunks with capped scores
        _attention("prefill_cap", "prefill", "mistral", rows=8, lo=0, hi=8192, chunk=512,
                   softcap=50.0),
        # prompts with a bidirectional prefix, documents, a distance bias and a window
        _attention("prefill_masks", "prefill", "gptoss", rows=16, lo=0, hi=1500, chunk=400,
                   alibi=True, docs=333, prefix=129, window=1024, sinks=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "rotary", "decode", "prefill"])
    if op == "assign":
        n = _log_uniform(rng, 1, 4000)
        chunk = _log_uniform(rng, 1, max(1, min(2000, 120000 // n)))
        prompts = rng.randint(0, n)
        return dict(op=op, requests=n, cached_lo=0, cached_hi=_log_uniform(rng, 1, 16000),
                    chunk=chunk, prompts=prompts,
                    tokens=n * 1 + prompts * chunk + rng.randint(0, 63))
    if op == "rotary":
        shape = rng.choice(sorted(SHAPES))
        d = SHAPES[shape][2]
        return dict(op=op, shape=shape, tokens=_log_uniform(rng, 1, 15000),
                    interleaved=rng.random() < 0.5, rotary_dim=16 * rng.randint(1, d // 16),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
                    fused=rng.random() < 0.5, far=_log_uniform(rng, 16, 2000000))
    shape = rng.choice(sorted(SHAPES))
    d = SHAPES[shape][2]
    mods = dict(softcap=rng.choice([0.0, 20.0, 30.0, 50.0]), alibi=rng.random() < 0.5,
                sinks=rng.random() < 0.5,
                window=0 if rng.random() < 0.5 else _log_uniform(rng, 1, 4000),
                docs=0 if rng.random() < 0.5 else _log_uniform(rng, 1, 2000))
    if not (mods["softcap"] or mods["alibi"] or mods["docs"]):
        mods["softcap"] = 40.0
    if op == "decode":
        hi = _log_uniform(rng, 1, 12000)
        return _attention(None, op, shape, rows=_log_uniform(rng, 1, 64), lo=rng.randint(1, hi),
                          hi=hi, **mods)
    rows = _log_uniform(rng, 1, 8)
    hi = rng.randint(0, 6000)
    return _attention(None, op, shape, rows=rows, lo=rng.randint(0, hi), hi=hi,
                      chunk=_log_uniform(rng, 8, 500), prefix=rng.choice([0, rng.randint(1, 2000)]),
                      **mods)


# ----------------------------------------------------------------- lengths of a case

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread: their sum is the same for every seed."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _assign_lengths(case):
    n, prompts = case["requests"], case["prompts"]
    cached = _spread(case["cached_lo"], case["cached_hi"], n)
    new = np.ones(n, dtype=np.int64)
    # the prompts' chunks: up to the case's chunk, ragged; the token count always has room for them
    new[:prompts] = 1 + (np.arange(prompts) * 7919) % case["chunk"]
    return cached, new


def _first_keys(docs, positions):
    return positions // docs * docs if docs else np.zeros_like(positions)


def _decode_lengths(case):
    n = _spread(case["lo"], case["hi"], case["rows"]) - 1
    lo = _first_keys(case["docs"], n)
    if case["window"]:
        lo = np.maximum(lo, n - case["window"] + 1)
    return n, np.maximum(lo, 0)


def _prefill_lengths(case):
    """Per row: cached positions and chunk; per token its row, position and visible keys."""
    rows, chunk = case["rows"], case["chunk"]
    cached = _spread(case["lo"], case["hi"], rows)
    chunks = np.maximum(1, chunk - (np.arange(rows) * 37) % (chunk // 4 + 1))
    if rows == 1:
        chunks[:] = chunk
    return cached, chunks


def _prefill_tokens(case, cached, chunks):
    row = np.repeat(np.arange(len(chunks)), chunks)
    start = np.cumsum(chunks) - chunks
    pos = cached[row] + np.arange(len(row)) - start[row]
    prefix = np.minimum(case["prefix"], (cached + chunks)[row])  # only what is in the cache
    first = _first_keys(case["docs"], pos)
    lo = first.copy()
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    hi = np.maximum(pos, prefix - 1)
    return row, pos, first, np.maximum(lo, 0), hi


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _pages(rng, need, width, spare=0):
    """A shuffled pool's pages dealt to rows of `need` pages: table, the pages left, pool size."""
    total = int(need.sum()) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.zeros((len(need), width), dtype=np.int32)
    filled = np.arange(width)[None, :] < need[:, None]
    table[filled] = order[: int(need.sum())]
    return table, order[int(need.sum()):], total


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "assign":
        cached, new = _assign_lengths(case)
        order = rng.permutation(len(cached))
        cached, new = cached[order], new[order]
        have = -(-cached // PAGE)
        need = -(-(cached + new) // PAGE)
        table, free, total = _pages(rng, have, int(need.max()) + 1,
                                    spare=int((need - have).sum()) + 7)
        st.update(table=_i32(table), cached=_i32(cached), new=_i32(new), free=_i32(free),
                  head=_i32([3]), num_pages=total)
        return st
    hq, hkv, d = SHAPES[case["shape"]]
    if case["op"] == "rotary":
        t = case["tokens"]
        positions = rng.integers(0, case["far"] + 1, t)
        pages = -(-t // PAGE) + 3
        if case["fused"]:
            qkv = _normal(g, t, hq + 2 * hkv, d)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            q, k, v = _normal(g, t, hq, d), _normal(g, t, hkv, d), _normal(g, t, hkv, d)
        st.update(q=q, k=k, v=v, positions=_i32(positions),
                  slots=_i32(rng.permutation(pages * PAGE)[:t]),
                  k_pool=torch.zeros(pages, hkv, PAGE, d, device=DEV, dtype=torch.bfloat16),
                  v_pool=torch.zeros(pages, hkv, PAGE, d, device=DEV, dtype=torch.bfloat16),
                  q_out=torch.empty(t, hq, d, device=DEV, dtype=torch.bfloat16))
        return st
    if case["op"] == "decode":
        pos, _ = _decode_lengths(case)
        order = rng.permutation(len(pos))
        pos = pos[order]
        need = pos // PAGE + 1
        first = _first_keys(case["docs"], pos)
        tokens = len(pos)
    else:
        cached, chunks = _prefill_lengths(case)
        order = rng.permutation(len(cached))
        cached, chunks = cached[order], chunks[order]
        row, pos, first, _, _ = _prefill_tokens(case, cached, chunks)
        need = -(-(cached + chunks) // PAGE)
        tokens = len(pos)
        st.update(rows=_i32(row), index=_i32(pos - cached[row]), chunk=int(chunks.max()),
                  prefix=_i32(np.minimum(case["prefix"], cached + chunks))
                  if case["prefix"] else None)
    table, _, total = _pages(rng, need, int(need.max()), spare=int(need.sum()) // 16 + 1)
    st.update(table=_i32(table), positions=_i32(pos),
              first=_i32(first) if case["docs"] else None,
              q=_normal(g, tokens, hq, d),
              k_pool=_normal(g, total, hkv, PAGE, d), v_pool=_normal(g, total, hkv, PAGE, d),
              sinks=_normal(g, hq, dtype=torch.float32) if case["sinks"] else None,
              slopes=torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV,
                                                    dtype=torch.float32) / hq)
              if case["alibi"] else None,
              out=torch.empty(tokens, hq, d, device=DEV, dtype=torch.bfloat16))
    return st


# ----------------------------------------------------------------- plain forms

def _plain_assign(st):
    case, table = st["case"], st["table"]
    cached, new = st["cached"].long(), st["new"].long()
    head, tokens, width = st["head"].long(), case["tokens"], table.shape[1]
    have, need = (cached + PAGE - 1) // PAGE, (cached + new + PAGE - 1) // PAGE
    extra = need - have
    page_end, token_end = torch.cumsum(extra, 0), torch.cumsum(new, 0)
    page_at, starts = page_end - extra, token_end - new
    column = torch.arange(width, device=DEV)[None, :]
    fresh = (column >= have[:, None]) & (column < need[:, None])
    pick = (head + page_at[:, None] + column - have[:, None]).clamp(0, st["free"].numel() - 1)
    table = torch.where(fresh, st["free"][pick], table)
    token = torch.arange(tokens, device=DEV)
    row = torch.searchsorted(token_end, token, right=True).clamp(max=len(cached) - 1)
    used = token < token_end[-1]
    pos = cached[row] + token - starts[row]
    slot = table[row, (pos // PAGE).clamp(0, width - 1)].long() * PAGE + pos % PAGE
    none = torch.full_like(token, -1)
    return {"table": table, "rows": torch.where(used, row, 0 * row).int(),
            "positions": torch.where(used, pos, none).int(),
            "slots": torch.where(used, slot, none).int(),
            "starts": torch.cat([starts, token_end[-1:]]).int(),
            "lengths": (cached + new).int(), "head": (head + page_end[-1:]).int()}


# base, stretch and original context of the measured frequency scalings
THETA, FACTOR, ORIGINAL = 150000.0, 32.0, 4096
BETA_FAST, BETA_SLOW, LOW_BAND, HIGH_BAND = 32.0, 1.0, 1.0, 4.0


def _frequencies(kind, rotary_dim):
    """Radians a position of each pair, in 64 bits, and the factor of cos and sin."""
    i = torch.arange(rotary_dim // 2, device=DEV, dtype=torch.float64)
    theta = THETA * FACTOR ** (rotary_dim / (rotary_dim - 2)) if kind == "ntk" else THETA
    freq = torch.exp(-2.0 * i / rotary_dim * math.log(theta))
    if kind == "linear":
        return freq / FACTOR, 1.0
    if kind == "yarn":
        def pair(turns):
            return rotary_dim * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(THETA))
        low = max(math.floor(pair(BETA_FAST)), 0)
        high = min(math.ceil(pair(BETA_SLOW)), rotary_dim - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return freq * (1 - ramp) + freq / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1.0
    if kind == "banded":
        share = ((ORIGINAL * freq / (2 * math.pi) - LOW_BAND) / (HIGH_BAND - LOW_BAND)).clamp(0, 1)
        return freq * share + freq / FACTOR * (1 - share), 1.0
    return freq, 1.0


def _rotated(x, cos, sin, interleaved, rotary_dim):
    x = x.float()
    part, rest = x[..., :rotary_dim], x[..., rotary_dim:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., : rotary_dim // 2], part[..., rotary_dim // 2:]
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([part, rest], -1).to(torch.bfloat16)


def _plain_rotary(st):
    case = st["case"]
    freq, factor = _frequencies(case["scaling"], case["rotary_dim"])
    angle = st["positions"].double()[:, None, None] * freq
    cos, sin = (torch.cos(angle) * factor).float(), (torch.sin(angle) * factor).float()
    slot = st["slots"].long()
    page, at = slot // PAGE, slot % PAGE
    args = (cos, sin, case["interleaved"], case["rotary_dim"])
    st["k_pool"][page, :, at] = _rotated(st["k"], *args)
    st["v_pool"][page, :, at] = st["v"]
    return {"q": _rotated(st["q"], *args), "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _weights(case, x, seen, distance, slopes, sinks):
    """Softmax weights over the last axis of x [..., heads, queries, keys], in 32 bits."""
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if slopes is not None:
        x = x - slopes * distance
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(st):
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    rows, width = st["table"].shape
    table = st["table"].long()
    k = st["k_pool"][table].permute(0, 2, 1, 3, 4).reshape(rows, hkv, width * PAGE, d).float()
    v = st["v_pool"][table].permute(0, 2, 1, 3, 4).reshape(rows, hkv, width * PAGE, d).float()
    q = st["q"].float().view(rows, hkv, hq // hkv, d)
    x = q @ k.transpose(-1, -2) / math.sqrt(d)
    n = st["positions"].long()[:, None]
    s = torch.arange(width * PAGE, device=DEV)[None, :]
    seen = s <= n
    if case["window"]:
        seen = seen & (s > n - case["window"])
    if st["first"] is not None:
        seen = seen & (s >= st["first"][:, None])
    heads = (1, hkv, hq // hkv, 1)
    slopes = None if st["slopes"] is None else st["slopes"].view(heads)
    sinks = None if st["sinks"] is None else st["sinks"].view(heads)
    w = _weights(case, x, seen[:, None, None], (n - s).abs().float()[:, None, None], slopes, sinks)
    return (w @ v).reshape(rows, hq, d).to(torch.bfloat16)


def _plain_prefill(st):
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    rows, width = st["table"].shape
    table, chunk = st["table"].long(), st["chunk"]
    k = st["k_pool"][table].permute(0, 2, 1, 3, 4).reshape(rows, hkv, 1, width * PAGE, d).float()
    v = st["v_pool"][table].permute(0, 2, 1, 3, 4).reshape(rows, hkv, 1, width * PAGE, d).float()
    row, index = st["rows"].long(), st["index"].long()
    q = torch.zeros(rows, chunk, hq, d, device=DEV)
    q[row, index] = st["q"].float()
    n = torch.full((rows, chunk), -1, device=DEV, dtype=torch.int64)
    n[row, index] = st["positions"].long()
    q = q.view(rows, chunk, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = q @ k.transpose(-1, -2) / math.sqrt(d)
    n = n[:, :, None]
    s = torch.arange(width * PAGE, device=DEV)[None, None, :]
    last = n if st["prefix"] is None else torch.maximum(n, st["prefix"].long()[:, None, None] - 1)
    seen = (s <= last) & (n >= 0)
    if case["window"]:
        seen = seen & (s > n - case["window"])
    if st["first"] is not None:
        first = torch.zeros_like(n)
        first[row, index, 0] = st["first"].long()
        seen = seen & (s >= first)
    heads = (1, hkv, hq // hkv, 1, 1)
    slopes = None if st["slopes"] is None else st["slopes"].view(heads)
    sinks = None if st["sinks"] is None else st["sinks"].view(heads)
    w = _weights(case, x, seen[:, None, None], (n - s).abs().float()[:, None, None], slopes, sinks)
    out = (w @ v).permute(0, 3, 1, 2, 4).reshape(rows, chunk, hq, d)
    return out[row, index].to(torch.bfloat16)


# ----------------------------------------------------------------- the framework's calls

def _own_assign(pgd, st):
    plan = pgd.assign_pages(st["table"], st["cached"], st["new"], st["free"],
                            num_tokens=st["case"]["tokens"], num_pages=st["num_pages"],
                            free_head=st["head"])
    return {"table": st["table"], "rows": plan.rows, "positions": plan.positions,
            "slots": plan.slots, "starts": plan.starts, "lengths": plan.lengths,
            "head": plan.free_head}


def _own_rotary(pgd, st):
    case = st["case"]
    if "rotary" not in st:  # made once by a program, as its weights are
        st["rotary"] = pgd.Rotary(case["rotary_dim"], THETA, interleaved=case["interleaved"],
                                  scaling=case["scaling"], factor=FACTOR,
                                  original_positions=ORIGINAL, beta_fast=BETA_FAST,
                                  beta_slow=BETA_SLOW, low_band=LOW_BAND, high_band=HIGH_BAND)
    q = pgd.rotary_append_paged(st["q"], st["k"], st["v"], st["positions"], st["k_pool"],
                                st["v_pool"], rotary=st["rotary"], slots=st["slots"],
                                q_out=st["q_out"])
    return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _workspace(pgd, st, hq, hkv, d):
    if "workspace" not in st:  # kept by a program beside its pools
        dims = pgd.make_dims(rows=st["q"].shape[0], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                             num_pages=st["k_pool"].shape[0],
                             max_pages_per_row=st["table"].shape[1])
        size = pgd.paged_decode_workspace_bytes(dims)
        st["workspace"] = torch.empty(max(size, 16), device=DEV, dtype=torch.uint8)
    return st["workspace"]


def _own_attention(pgd, st):
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    common = dict(num_kv_heads=hkv, out=st["out"], workspace=_workspace(pgd, st, hq, hkv, d),
                  softcap=case["softcap"], alibi_slopes=st["slopes"], first_key=st["first"])
    if case["op"] == "decode":
        return pgd.paged_decode_attention(st["q"], st["k_pool"], st["v_pool"], st["table"],
                                          st["positions"], st["sinks"], case["window"], **common)
    return pgd.paged_prefill_attention(st["q"], st["k_pool"], st["v_pool"], st["table"],
                                       st["rows"], st["positions"], st["sinks"], case["window"],
                                       prefix_len=st["prefix"], **common)


def run(st):
    op = st["case"]["op"]
    if own:
        import paged_gqa_decode_gb300 as pgd
        if op == "assign":
            return _own_assign(pgd, st)
        if op == "rotary":
            return _own_rotary(pgd, st)
        return _own_attention(pgd, st)
    return {"assign": _plain_assign, "rotary": _plain_rotary, "decode": _plain_decode,
            "prefill": _plain_prefill}[op](st)


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "assign":
        cached, new = _assign_lengths(case)
        pages = int((-(-(cached + new) // PAGE) - -(-cached // PAGE)).sum())
        n = case["requests"]
        # lengths in; a page id in and a table entry out for each new page; the last page in use of
        # each request in; rows, positions and slots of every token, starts and lengths out
        return {"bytes": 4 * (2 * n + 2 * pages + n + 3 * case["tokens"] + 2 * n + 3), "flops": 0}
    hq, hkv, d = SHAPES[case["shape"]]
    if case["op"] == "rotary":
        t = case["tokens"]
        # q, k and v in and out, a position and a slot a token
        return {"bytes": t * (2 * 2 * d * (hq + 2 * hkv) + 8),
                "flops": 3 * t * (hq + hkv) * case["rotary_dim"]}
    if case["op"] == "decode":
        n, lo = _decode_lengths(case)
        keys, tokens = int((n - lo + 1).sum()), len(n)
        cache = keys
        pages = int((n // PAGE - lo // PAGE + 1).sum())
    else:
        cached, chunks = _prefill_lengths(case)
        row, _, _, lo, hi = _prefill_tokens(case, cached, chunks)
        keys, tokens = int((hi - lo + 1).sum()), len(row)
        last = np.zeros(len(chunks), dtype=np.int64)
        np.maximum.at(last, row, hi)
        first = np.full(len(chunks), 1 << 40)
        np.minimum.at(first, row, lo)
        cache = int((last - first + 1).sum())
        pages = int((last // PAGE - first // PAGE + 1).sum())
    # each cached key and value that some token sees once, its page's id, q in and out
    return {"bytes": 4 * hkv * d * cache + 4 * pages + tokens * (4 * hq * d + 4),
            "flops": 4 * hq * d * keys}


# ----------------------------------------------------------------- from the definitions, in 64 bits

def _exact_rotary(st):
    case = st["case"]
    rd, kind = case["rotary_dim"], case["scaling"]
    base = THETA * FACTOR ** (rd / (rd - 2)) if kind == "ntk" else THETA
    omega, factor = [], 1.0
    for j in range(rd // 2):
        w = base ** (-2.0 * j / rd)
        if kind == "linear":
            w = w / FACTOR
        elif kind == "yarn":
            factor = 0.1 * math.log(FACTOR) + 1.0
            def edge(b):
                return rd / 2 * math.log(ORIGINAL / (2 * math.pi * b)) / math.log(THETA)
            a, b = max(math.floor(edge(BETA_FAST)), 0), min(math.ceil(edge(BETA_SLOW)), rd - 1)
            mix = min(max((j - a) / max(b - a, 0.001), 0.0), 1.0)
            w = (1 - mix) * w + mix * w / FACTOR
        elif kind == "banded":
            turns = ORIGINAL * w / (2 * math.pi)
            if turns < LOW_BAND:
                w = w / FACTOR
            elif turns <= HIGH_BAND:
                mix = (turns - LOW_BAND) / (HIGH_BAND - LOW_BAND)
                w = (1 - mix) * w / FACTOR + mix * w
        omega.append(w)
    z = torch.polar(torch.tensor(factor, device=DEV, dtype=torch.float64),
                    st["positions"].double()[:, None] * torch.tensor(omega, device=DEV,
                                                                     dtype=torch.float64))

    def turn(x):
        x = x.double().clone()
        if case["interleaved"]:
            pair = torch.view_as_complex(x[..., :rd].reshape(*x.shape[:-1], rd // 2, 2).contiguous())
            x[..., :rd] = torch.view_as_real(pair * z[:, None]).reshape(*x.shape[:-1], rd)
        else:
            pair = torch.complex(x[..., : rd // 2], x[..., rd // 2: rd]) * z[:, None]
            x[..., : rd // 2], x[..., rd // 2: rd] = pair.real, pair.imag
        return x

    k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
    k, v = turn(st["k"]), st["v"].double()
    hkv, d = k.shape[1:]
    flat = st["slots"].long()
    kt, vt = (p.transpose(1, 2).reshape(-1, hkv, d).clone() for p in (k_pool, v_pool))
    kt[flat], vt[flat] = k, v
    back = (len(k_pool), PAGE, hkv, d)
    return {"q": turn(st["q"]), "k_pool": kt.view(back).transpose(1, 2).contiguous(),
            "v_pool": vt.view(back).transpose(1, 2).contiguous()}


def _exact_attention(st):
    """Row by row, in 64 bits, over the visible keys alone."""
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    group = hq // hkv
    q, pos = st["q"].double(), st["positions"].cpu().numpy().astype(np.int64)
    rows = st["rows"].cpu().numpy() if case["op"] == "prefill" else np.arange(len(pos))
    first = st["first"].cpu().numpy() if st["first"] is not None else np.zeros_like(pos)
    prefix = st["prefix"].cpu().numpy()[rows] if st.get("prefix") is not None \
        else np.zeros_like(pos)
    hi = np.maximum(pos, prefix - 1)
    lo = np.maximum(first, 0)
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    out = torch.zeros_like(q)
    for r in range(st["table"].shape[0]):
        mine = np.nonzero(rows == r)[0]
        if not len(mine):
            continue
        end = int(hi[mine].max()) + 1
        pages = st["table"][r, : -(-end // PAGE)].long()
        keys = st["k_pool"][pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :end]
        values = st["v_pool"][pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :end]
        at = torch.from_numpy(mine).to(DEV)
        s = torch.arange(end, device=DEV)[None]
        n, a, b = (torch.from_numpy(x[mine]).to(DEV)[:, None] for x in (pos, lo, hi))
        hidden = (s < a) | (s > b)
        far = (s - n).abs().double()
        for h in range(hq):
            x = q[at, h] @ keys[h // group].T / math.sqrt(d)
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if st["slopes"] is not None:
                x = x - st["slopes"][h].double() * far
            x = x.masked_fill(hidden, -math.inf)
            total = torch.logsumexp(x, -1)
            if st["sinks"] is not None:
                total = torch.logaddexp(total, st["sinks"][h].double())
            p = torch.exp(x - total[:, None])
            p = torch.where(hidden, torch.zeros_like(p), p)
            out[at, h] = p @ values[h // group]
    return out


def exact(case, seed):
    if case["op"] == "assign":
        return None  # whole numbers: the plain form's are exact
    st = prepare(case, seed)
    return _exact_rotary(st) if case["op"] == "rotary" else _exact_attention(st)
