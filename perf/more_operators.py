"""Measured cases of a cache whose pages are shared: rows forked, reordered and
released over reference-counted pages, pages copied and compacted, and decode
attention that reads a prefix shared by many rows once.

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
PAGE_MAJOR, HEAD_MAJOR = 0, 1

# (query heads, kv heads, head_dim) of the framework's workloads
SHAPES = {"qwen": (14, 2, 64), "gptoss": (64, 8, 64), "mistral": (32, 8, 128),
          "square": (8, 8, 128), "pairs": (16, 8, 64)}


def _fork(name, kind, requests, beams, lo, hi, grown, **kw):
    case = dict(op="fork", kind=kind, requests=requests, beams=beams, lo=lo, hi=hi, grown=grown,
                spare_columns=0)
    case.update(kw)
    return case if name is None else dict(case, name=name)


def _shared(name, shape, groups, beams, lo, hi, own_lo, own_hi, **kw):
    case = dict(op="shared", shape=shape, groups=groups, beams=beams, lo=lo, hi=hi, own_lo=own_lo,
                own_hi=own_hi, alone=0, sinks=False, step=False, layout=PAGE_MAJOR)
    case.update(kw)
    return case if name is None else dict(case, name=name)


def listed():
    return [
        # one step of beam search: 8 requests of 4 beams, survivors stay, the others are replaced
        _fork("fork_beams", "beams", 8, 4, 200, 1500, 77),
        # prompts forked into the samples that continue them, each with a last page of its own
        _fork("fork_samples", "samples", 64, 16, 100, 8000, 0),
        # a large batch: some rows finished, some cut back to an earlier position, most reordered
        _fork("fork_many", "mixed", 512, 8, 500, 8000, 300, spare_columns=5),
        # the last pages of 40 beams in the pools of 12 layers, part of each page in use
        dict(name="copy_tails", op="copy", shape="qwen", layers=12, copies=40, partial=True,
             pages=512, layout=PAGE_MAJOR),
        # whole pages moved in two layers' pools: a pool being defragmented
        dict(name="copy_pages", op="copy", shape="mistral", layers=2, copies=1101, partial=False,
             pages=2405, layout=PAGE_MAJOR),
        # a small pool half in use, its pages moved down
        dict(name="compact_small", op="compact", rows=64, lo=1, hi=4000, beams=4, pages=4097,
             moves=4097),
        # a large pool: a bounded number of moves out of its upper end
        dict(name="compact_large", op="compact", rows=2048, lo=1000, hi=16000, beams=8,
             pages=250007, moves=4096),
        # four beams of one short prompt, their step's keys written first: latency
        _shared("shared_step", "qwen", 1, 4, 300, 300, 1, 40, step=True),
        # beam search in a batch: 16 requests of 4 beams over prompts of their own
        _shared("shared_beams", "mistral", 16, 4, 500, 6000, 1, 200),
        # one system prompt under a serving batch, a few rows without it
        _shared("shared_system", "gptoss", 1, 128, 2048, 2048, 100, 2000, alone=3, sinks=True),
        # many samples of one long document: the prefix is nearly all of the work
        _shared("shared_long", "mistral", 1, 256, 32768, 32768, 16, 1024),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "copy", "compact", "shared", "shared"])
    if op == "fork":
        beams = _log_uniform(rng, 1, 32)
        requests = _log_uniform(rng, 1, 2048 // beams)
        lo = _log_uniform(rng, 1, 4000)
        return _fork(None, rng.choice(["beams", "samples", "mixed"]), requests, beams, lo,
                     lo + rng.randint(0, 4000), rng.randint(0, 300),
                     spare_columns=rng.randint(0, 9))
    if op == "copy":
        shape = rng.choice(sorted(SHAPES))
        copies = _log_uniform(rng, 1, 500)
        return dict(op=op, shape=shape, layers=rng.randint(1, 3), copies=copies,
                    partial=rng.random() < 0.5, pages=2 * copies + rng.randint(0, 300),
                    layout=rng.choice([PAGE_MAJOR, HEAD_MAJOR]))
    if op == "compact":
        rows, lo = _log_uniform(rng, 1, 1300), _log_uniform(rng, 1, 4000)
        hi = lo + rng.randint(0, 8000)
        need = rows * (hi // PAGE + 2)
        return dict(op=op, rows=rows, lo=lo, hi=hi, beams=_log_uniform(rng, 1, 16),
                    pages=max(need, min(250000, int(need * rng.uniform(1, 3)))) + rng.randint(1, 6),
                    moves=_log_uniform(rng, 1, 4096))
    shape = rng.choice(sorted(SHAPES))
    beams = _log_uniform(rng, 1, 100)
    groups = _log_uniform(rng, 1, max(1, 200 // beams))
    lo = _log_uniform(rng, 64, 8000)
    own_lo = _log_uniform(rng, 1, 500)
    return _shared(None, shape, groups, beams, lo, lo + rng.randint(0, 4000), own_lo,
                   own_lo + rng.randint(0, 1000), alone=rng.choice([0, 0, rng.randint(1, 9)]),
                   sinks=rng.random() < 0.5, layout=rng.choice([PAGE_MAJOR, HEAD_MAJOR]))


# ----------------------------------------------------------------- lengths of a case

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread: their sum is the same for every seed."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _fork_lengths(case):
    """Per row: its request, its length, and the pages it shares with the request's other rows."""
    requests, beams = case["requests"], case["beams"]
    prompt = np.repeat(_spread(case["lo"], case["hi"], requests), beams)
    member = np.tile(np.arange(beams), requests)
    if case["kind"] == "samples":
        return np.where(member == 0, prompt, 0), np.zeros_like(prompt), member
    return prompt + case["grown"], prompt // PAGE, member


def _fork_parents(case, lengths, member):
    """Per row: its parent and the positions it keeps (-1: all).  Survivors keep their row."""
    rows = np.arange(len(member))
    first = rows - member
    if case["kind"] == "samples":
        return first, np.full(len(rows), -1)
    # of the beams 0, 1, 2, .. of a request, every third and fourth one is replaced
    replaced = (member % 4) >= 2
    parent = np.where(replaced, rows - member % 4 + (rows // 4) % 2, rows)
    keep = np.full(len(rows), -1)
    if case["kind"] == "mixed":
        parent = np.where(rows % 37 == 5, -1, parent)      # finished
        cut = rows % 11 == 3                                # cut back, some inside a shared page
        keep = np.where(cut, np.maximum(lengths - 1 - (rows * 13) % 400, 0), keep)
    return parent, keep


def _shared_rows(case):
    """Rows per group, shared pages per group, own positions per row (the last one is the step's)."""
    prompts = _spread(case["lo"], case["hi"], case["groups"])
    rows = case["groups"] * case["beams"] + case["alone"]
    pages = prompts // PAGE
    owned = _spread(case["own_lo"], case["own_hi"], rows)
    start = np.zeros(rows, dtype=np.int64)
    start[:case["groups"] * case["beams"]] = np.repeat(pages, case["beams"])
    return pages, start, owned


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _deal(order, at, held_shared, own_pages, leaders, width):
    """A table: row r's first held_shared[r] entries are its leader's, the rest pages of its own
    from order[at..].  Returns the table and the next unused index of order."""
    table = np.zeros((len(own_pages), width), dtype=np.int64)
    columns = np.arange(width)[None, :]
    is_leader = leaders == np.arange(len(leaders))
    total = held_shared + own_pages
    fresh = np.where(is_leader[:, None], columns < total[:, None],
                     (columns >= held_shared[:, None]) & (columns < total[:, None]))
    count = int(fresh.sum())
    table[fresh] = order[at:at + count]
    inherit = ~is_leader[:, None] & (columns < held_shared[:, None])
    table = np.where(inherit, table[leaders], table)
    return table, at + count


def _shares(table, pages, total):
    held = np.bincount(table[np.arange(table.shape[1])[None, :] < pages[:, None]], minlength=total)
    return np.maximum(held - 1, 0)


def _prepare_fork(case, rng, st):
    lengths, common, member = _fork_lengths(case)
    parents, keep = _fork_parents(case, lengths, member)
    rows = np.arange(len(member))
    pages = -(-lengths // PAGE)
    common = np.minimum(common, pages)
    width = int(pages.max()) + case["spare_columns"]
    spare = len(rows) + 9  # a page for every row's copy
    total = int(pages.sum()) + spare
    order = rng.permutation(total)
    table, used = _deal(order, 0, common, pages - common, rows - member, width)
    # the list has room for every page of the pool: its free end starts at `used`
    st.update(table=_i32(table), lengths=_i32(lengths), parents=_i32(parents),
              keep=_i32(np.where(keep < 0, np.iinfo(np.int32).max, keep))
              if case["kind"] == "mixed" else None,
              shares=_i32(_shares(table, pages, total)), free=_i32(order), head=_i32([used]))


def _prepare_copy(case, rng, g, st):
    hq, hkv, d = SHAPES[case["shape"]]
    n = case["copies"]
    order = rng.permutation(case["pages"])
    shape = (case["pages"], hkv, PAGE, d) if case["layout"] == PAGE_MAJOR else \
        (hkv, case["pages"] * PAGE, d)
    counts = 1 + (np.arange(n) * 29) % (PAGE - 1)
    st.update(k_pools=[_normal(g, *shape) for _ in range(case["layers"])],
              v_pools=[_normal(g, *shape) for _ in range(case["layers"])],
              sources=_i32(order[:n]), targets=_i32(order[n:2 * n]),
              counts=_i32(counts) if case["partial"] else None)


def _prepare_compact(case, rng, st):
    lengths = _spread(case["lo"], case["hi"], case["rows"])
    rows = np.arange(case["rows"])
    leaders = rows - rows % case["beams"]
    pages = -(-lengths // PAGE)
    common = np.where(rows == leaders, 0, np.minimum(pages[leaders], pages) // 2)
    width = int(pages.max()) + 1
    # a page that is neither listed as free nor held: the user's own
    order = 1 + rng.permutation(case["pages"] - 1)
    table, used = _deal(order, 0, common, pages - common, leaders, width)
    st.update(table=_i32(table), lengths=_i32(lengths),
              shares=_i32(_shares(table, pages, case["pages"])), free=_i32(order),
              head=_i32([used]))


def _prepare_shared(case, rng, g, st):
    hq, hkv, d = SHAPES[case["shape"]]
    shared, start, owned = _shared_rows(case)
    rows, grouped = len(start), case["groups"] * case["beams"]
    own_pages = -(-owned // PAGE)
    leaders = np.arange(rows)
    leaders[:grouped] -= np.arange(grouped) % case["beams"]
    width = int((start + own_pages).max())
    total = int(shared.sum() + own_pages.sum()) + 3
    order = rng.permutation(total)
    table, _ = _deal(order, 0, start, own_pages, leaders, width)
    if case["layout"] == PAGE_MAJOR:
        shape = (total, hkv, PAGE, d)
    else:
        shape = (hkv, total * PAGE, d)
    st.update(table=_i32(table), positions=_i32(start * PAGE + owned - 1),
              starts=_i32(np.arange(case["groups"] + 1) * case["beams"]), pages=_i32(shared),
              q=_normal(g, rows, hq, d), k_pool=_normal(g, *shape), v_pool=_normal(g, *shape),
              sinks=_normal(g, hq, dtype=torch.float32) if case["sinks"] else None,
              k_new=_normal(g, rows, hkv, d) if case["step"] else None,
              v_new=_normal(g, rows, hkv, d) if case["step"] else None,
              out=torch.empty(rows, hq, d, device=DEV, dtype=torch.bfloat16))


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "fork":
        _prepare_fork(case, rng, st)
    elif case["op"] == "copy":
        _prepare_copy(case, rng, g, st)
    elif case["op"] == "compact":
        _prepare_compact(case, rng, st)
    else:
        _prepare_shared(case, rng, g, st)
    return st


# ----------------------------------------------------------------- plain forms

def _plain_fork(st):
    table, shares, free = st["table"].long(), st["shares"].long(), st["free"]
    lengths, parents, head = st["lengths"].long(), st["parents"].long(), st["head"].long()
    rows, width = table.shape
    index = torch.arange(rows, device=DEV)
    column = torch.arange(width, device=DEV)[None, :]
    parent = parents.clamp(min=0)
    kept = torch.where(parents >= 0, lengths[parent], 0)
    if st["keep"] is not None:
        kept = torch.minimum(kept, st["keep"].long())
    old_pages, new_pages = (lengths + PAGE - 1) // PAGE, (kept + PAGE - 1) // PAGE
    old_held, new_held = column < old_pages[:, None], column < new_pages[:, None]
    moved = torch.where(new_held, table[parent], table)
    ones = torch.ones(1, device=DEV, dtype=torch.int64)
    old, new = table[old_held], moved[new_held]
    holders = shares + 1
    holders = holders.index_add(0, old, -ones.expand(len(old)))
    holders = holders.index_add(0, new, ones.expand(len(new)))
    # pages that nobody holds any more, in the order of the entries that held them
    first = torch.full_like(shares, len(old))
    first.scatter_reduce_(0, old, torch.arange(len(old), device=DEV), "amin")
    gone = old[(holders[old] == 0) & (first[old] == torch.arange(len(old), device=DEV))]
    head = head - len(gone)
    free[head + torch.arange(len(gone), device=DEV)] = gone.int()
    # a last page in part use belongs to one row alone
    has_tail = kept % PAGE != 0
    last = (new_pages - 1).clamp(min=0)
    tail = moved[index, last]
    tails = torch.zeros_like(shares).index_add(0, tail, has_tail.long())
    lowest = torch.full_like(shares, rows)
    lowest.scatter_reduce_(0, torch.where(has_tail, tail, 0),
                           torch.where(has_tail, index, rows), "amin")
    copied = has_tail & ~((tails[tail] == holders[tail]) & (lowest[tail] == index))
    rank = torch.cumsum(copied.long(), 0) - copied.long()
    target = free[(head + rank).clamp(max=len(free) - 1)].long()
    holders = holders.index_add(0, tail, -copied.long())
    st["shares"].copy_((holders - 1).clamp(min=0))
    moved[index, last] = torch.where(copied, target, tail)
    st["table"].copy_(moved)
    none = torch.full_like(tail, -1)
    st["lengths"] = kept.int()
    st["head"] = (head + copied.sum()).int()
    return {"table": st["table"], "shares": st["shares"], "free": st["free"], "head": st["head"],
            "lengths": st["lengths"], "sources": torch.where(copied, tail, none).int(),
            "targets": torch.where(copied, target, none).int(),
            "counts": torch.where(copied, kept % PAGE, 0).int()}


def _pages_view(pool, case):
    """The pool as [pages, kv heads, 64, D]."""
    hq, hkv, d = SHAPES[case["shape"]]
    if case["layout"] == PAGE_MAJOR:
        return pool
    return pool.view(hkv, -1, PAGE, d).transpose(0, 1)


def _plain_copy(st):
    case = st["case"]
    source, target = st["sources"].long(), st["targets"].long()
    for pool in st["k_pools"] + st["v_pools"]:
        pages = _pages_view(pool, case)
        page = pages[source]
        if st["counts"] is not None:
            used = torch.arange(PAGE, device=DEV)[None, :] < st["counts"][:, None]
            page = torch.where(used[:, None, :, None], page, pages[target])
        pages[target] = page
    return {"k": st["k_pools"], "v": st["v_pools"]}


def _plain_compact(st):
    case = st["case"]
    table, shares, lengths = st["table"].long(), st["shares"].long(), st["lengths"].long()
    rows, width = table.shape
    total, limit = case["pages"], case["moves"]
    pages = torch.arange(total, device=DEV)
    used = torch.arange(width, device=DEV)[None, :] < ((lengths + PAGE - 1) // PAGE)[:, None]
    is_free = torch.zeros(total, device=DEV, dtype=torch.bool)
    listed_at = torch.arange(len(st["free"]), device=DEV) >= st["head"]
    is_free[st["free"][listed_at].long()] = True
    held = torch.zeros(total, device=DEV, dtype=torch.bool)
    held[table[used]] = True
    hole = pages[is_free]                       # from the bottom
    top = torch.flip(pages[held], [0])          # from the top
    n = min(len(hole), len(top), limit)
    go = hole[:n] < top[:n]
    moves = torch.where(go, top[:n], -1), torch.where(go, hole[:n], -1)
    sources = torch.full((limit,), -1, device=DEV, dtype=torch.int64)
    targets = torch.full((limit,), -1, device=DEV, dtype=torch.int64)
    sources[:n], targets[:n] = moves
    name = pages.clone()
    name[top[:n][go]] = hole[:n][go]
    new_table = torch.where(used, name[table], table)
    new_shares = shares.clone()
    new_shares[hole[:n][go]] = shares[top[:n][go]]
    new_shares[top[:n][go]] = 0
    is_free[hole[:n][go]] = False
    is_free[top[:n][go]] = True
    free = st["free"].clone()
    free[listed_at] = pages[is_free].int()
    held[top[:n][go]] = False
    held[hole[:n][go]] = True
    end = torch.where(held, pages + 1, 0).amax(0, keepdim=True)
    return {"table": new_table.int(), "shares": new_shares.int(), "free": free,
            "sources": sources.int(), "targets": targets.int(), "end": end.int()}


def _softmax_values(x, v, sinks):
    """Softmax weights over the last axis of x [.., queries, keys], with the sink, times v."""
    top = x.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    return e, total


def _plain_shared(st):
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    group = hq // hkv
    shared, start, owned = _shared_rows(case)
    k_pages, v_pages = _pages_view(st["k_pool"], case), _pages_view(st["v_pool"], case)
    table, n = st["table"].long(), st["positions"].long()
    if st["k_new"] is not None:
        at = table[torch.arange(len(n), device=DEV), n // PAGE]
        k_pages[at, :, n % PAGE] = st["k_new"]
        v_pages[at, :, n % PAGE] = st["v_new"]
    spans = [(g * case["beams"], (g + 1) * case["beams"], int(shared[g]))
             for g in range(case["groups"])]
    if case["alone"]:
        spans.append((case["groups"] * case["beams"], len(start), 0))
    out = []
    for b0, b1, pages in spans:
        rows = b1 - b0
        q = st["q"][b0:b1].float().view(rows, hkv, group, d)
        width = int(-(-owned[b0:b1].max() // PAGE))
        tail = table[b0:b1, pages:pages + width]
        k = k_pages[tail].permute(0, 2, 1, 3, 4).reshape(rows, hkv, width * PAGE, d).float()
        v = v_pages[tail].permute(0, 2, 1, 3, 4).reshape(rows, hkv, width * PAGE, d).float()
        x = q @ k.transpose(-1, -2) / math.sqrt(d)
        s = pages * PAGE + torch.arange(width * PAGE, device=DEV)
        x = torch.where(s <= n[b0:b1, None, None, None], x, -math.inf)
        v = torch.where(s[:, None] <= n[b0:b1, None, None, None], v, 0.0)
        kp = k_pages[table[b0, :pages]].transpose(0, 1).reshape(hkv, pages * PAGE, d).float()
        vp = v_pages[table[b0, :pages]].transpose(0, 1).reshape(hkv, pages * PAGE, d).float()
        flat = q.transpose(0, 1).reshape(hkv, rows * group, d)
        xp = (flat @ kp.transpose(-1, -2) / math.sqrt(d)).view(hkv, rows, group, pages * PAGE)
        sinks = None if st["sinks"] is None else st["sinks"].view(1, hkv, group, 1)
        e, total = _softmax_values(torch.cat([xp.transpose(0, 1), x], -1), None, sinks)
        ep, es = e[..., :pages * PAGE], e[..., pages * PAGE:]
        o = (ep.transpose(0, 1).reshape(hkv, rows * group, -1) @ vp).view(hkv, rows, group, d)
        o = (o.transpose(0, 1) + es @ v) / total
        out.append(o.reshape(rows, hq, d))
    out = torch.cat(out).to(torch.bfloat16)
    if st["k_new"] is None:
        return out
    return {"out": out, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


# ----------------------------------------------------------------- the framework's calls

def _own_fork(pgd, st):
    plan = pgd.fork_rows(st["table"], st["lengths"], st["parents"], st["shares"], st["free"],
                         free_head=st["head"], keep=st["keep"])
    st["lengths"], st["head"] = plan.lengths, plan.free_head
    return {"table": st["table"], "shares": st["shares"], "free": st["free"], "head": st["head"],
            "lengths": plan.lengths, "sources": plan.sources, "targets": plan.targets,
            "counts": plan.counts}


def _own_copy(pgd, st):
    hq, hkv, d = SHAPES[st["case"]["shape"]]
    pgd.copy_pages(st["k_pools"], st["v_pools"], st["sources"], st["targets"], st["counts"],
                   num_kv_heads=hkv, head_dim=d, layout=st["case"]["layout"])
    return {"k": st["k_pools"], "v": st["v_pools"]}


def _own_compact(pgd, st):
    plan = pgd.compact_pages(st["table"], st["lengths"], st["shares"], st["free"],
                             free_head=st["head"], max_moves=st["case"]["moves"])
    return {"table": plan.table, "shares": plan.shares, "free": plan.free_pages,
            "sources": plan.sources, "targets": plan.targets, "end": plan.end}


def _own_shared(pgd, st):
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    if "workspace" not in st:  # kept by a program beside its pools
        rows, width = st["table"].shape
        dims = pgd.make_dims(rows=rows, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                             num_pages=st["k_pool"].numel() // (hkv * PAGE * d),
                             max_pages_per_row=width, layout=case["layout"])
        st["workspace"] = torch.empty(pgd.shared_decode_workspace_bytes(dims, case["groups"]),
                                      device=DEV, dtype=torch.uint8)
    common = dict(num_kv_heads=hkv, layout=case["layout"], out=st["out"],
                  workspace=st["workspace"], group_starts=st["starts"], group_pages=st["pages"])
    if st["k_new"] is None:
        return pgd.paged_decode_attention(st["q"], st["k_pool"], st["v_pool"], st["table"],
                                          st["positions"], st["sinks"], **common)
    out = pgd.paged_decode_step(st["q"], st["k_new"], st["v_new"], st["k_pool"], st["v_pool"],
                                st["table"], st["positions"], st["sinks"], **common)
    return {"out": out, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def run(st):
    op = st["case"]["op"]
    if own:
        import paged_gqa_decode_gb300 as pgd
        return {"fork": _own_fork, "copy": _own_copy, "compact": _own_compact,
                "shared": _own_shared}[op](pgd, st)
    return {"fork": _plain_fork, "copy": _plain_copy, "compact": _plain_compact,
            "shared": _plain_shared}[op](st)


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "fork":
        lengths, _, member = _fork_lengths(case)
        parents, keep = _fork_parents(case, lengths, member)
        n = len(lengths)
        kept = np.where(parents >= 0, lengths[np.maximum(parents, 0)], 0)
        kept = np.where(keep >= 0, np.minimum(kept, keep), kept)
        changed = parents != np.arange(n)
        old, new = -(-lengths // PAGE), -(-kept // PAGE)
        # lengths and parents in; of the rows that change, the old pages and the parent's in, the
        # new entries out and a count in and out for each; lengths, sources, targets, counts out
        entries = int((old + new)[changed].sum())
        return {"bytes": 4 * (2 * n + entries + int(new[changed].sum()) + 2 * entries + 4 * n + 2),
                "flops": 0}
    if case["op"] == "copy":
        hq, hkv, d = SHAPES[case["shape"]]
        n = case["copies"]
        positions = int((1 + (np.arange(n) * 29) % (PAGE - 1)).sum()) if case["partial"] \
            else n * PAGE
        # each position's values read and written, in K and V of each layer
        return {"bytes": 2 * 2 * case["layers"] * positions * hkv * d * 2 + 12 * n, "flops": 0}
    if case["op"] == "compact":
        rows, width = case["rows"], -(-case["hi"] // PAGE) + 1
        # table, lengths, shares and list in; table, shares, list and moves out
        return {"bytes": 4 * (2 * rows * width + rows + 4 * case["pages"] + 2 * case["moves"]),
                "flops": 0}
    hq, hkv, d = SHAPES[case["shape"]]
    shared, start, owned = _shared_rows(case)
    rows = len(start)
    cache = int(shared.sum()) * PAGE + int(owned.sum())
    pages = int(shared.sum()) + int((-(-owned // PAGE)).sum())
    keys = int((start * PAGE + owned).sum())
    extra = 2 * 2 * 2 * hkv * d * rows if case["step"] else 0  # the step's keys and values in, out
    # each group's shared keys and values once, each row's own once, q in and out
    return {"bytes": 4 * hkv * d * cache + 4 * pages + rows * (4 * hq * d + 4) + extra,
            "flops": 4 * hq * d * keys}


# ----------------------------------------------------------------- from the definitions, in 64 bits

def _exact_shared(st):
    """Row by row, in 64 bits, over all the pages that the row's own table entries name."""
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    k_pool, v_pool = st["k_pool"], st["v_pool"]
    if case["layout"] == HEAD_MAJOR:
        k_pool, v_pool = (p.view(hkv, -1, PAGE, d).permute(1, 0, 2, 3) for p in (k_pool, v_pool))
    out = torch.zeros(st["q"].shape, device=DEV, dtype=torch.float64)
    pools = [k_pool.double(), v_pool.double()] if case["step"] else None
    for b, n in enumerate(st["positions"].tolist()):
        pages = st["table"][b, : n // PAGE + 1].long()
        k = k_pool[pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, : n + 1]
        v = v_pool[pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, : n + 1]
        if case["step"]:
            k[:, n], v[:, n] = st["k_new"][b].double(), st["v_new"][b].double()
            for pool, new in zip(pools, (st["k_new"], st["v_new"])):
                pool[pages[n // PAGE], :, n % PAGE] = new[b].double()
        x = torch.einsum("hgd,hnd->hgn", st["q"][b].double().view(hkv, -1, d), k) / d ** 0.5
        total = torch.logsumexp(x, -1)
        if st["sinks"] is not None:
            total = torch.logaddexp(total, st["sinks"].double().view(hkv, -1))
        out[b] = torch.einsum("hgn,hnd->hgd", torch.exp(x - total[..., None]), v).reshape(hq, d)
    return {"out": out, "k_pool": pools[0], "v_pool": pools[1]} if case["step"] else out


def _exact_copy(st):
    """Copy by copy and head by head."""
    case = st["case"]
    hq, hkv, d = SHAPES[case["shape"]]
    counts = [PAGE] * case["copies"] if st["counts"] is None else st["counts"].tolist()
    moves = list(zip(st["sources"].tolist(), st["targets"].tolist(), counts))
    result = {}
    for name, pools in (("k", st["k_pools"]), ("v", st["v_pools"])):
        result[name] = [pool.double() for pool in pools]
        for pool in result[name]:
            tiles = pool.view(-1, PAGE, d)  # of a page and head, in the layout's order
            for source, target, count in moves:
                if case["layout"] == PAGE_MAJOR:
                    a, b = (slice(p * hkv, (p + 1) * hkv) for p in (source, target))
                else:
                    a, b = (slice(p, None, case["pages"]) for p in (source, target))
                tiles[b, :count] = tiles[a, :count]
    return result


def exact(case, seed):
    if case["op"] == "copy":
        return _exact_copy(prepare(case, seed))
    if case["op"] == "shared":
        return _exact_shared(prepare(case, seed))
    return None  # whole numbers: the plain form's are exact
