"""What the tests of shared pages have in common: the plain row-by-row models of
fork_rows and compact_pages, states for them, and the plain 64-bit attention of
rows over their own table entries with the bound its outputs are held to."""
from __future__ import annotations

import numpy as np

PAGE = 64


def pages_of(n):
    return -(-n // PAGE)


def fork_rows(table, lengths, parents, keep, shares, free, head, num_pages):
    """Row by row.  Returns the outputs in the order table, shares, free pages, lengths,
    sources, targets, counts, head, and whether an error is reported."""
    rows, width = table.shape
    old, table = table, table.copy()
    free, error = list(free), False
    lengths, parents = list(lengths), list(parents)
    for r in range(rows):
        if not 0 <= lengths[r] <= PAGE * width:
            lengths[r], error = 0, True
        if not -1 <= parents[r] < rows:
            parents[r], error = -1, True
    bad_head = not 0 <= head <= len(free)
    error |= bad_head
    kept = [0 if q < 0 else lengths[q] if keep is None else min(lengths[q], max(keep[r], 0))
            for r, q in enumerate(parents)]
    children = [parents.count(i) for i in range(rows)]
    holders = {p: int(shares[p]) + 1 for p in range(num_pages)}
    for i in range(rows):
        for e in range(pages_of(lengths[i])):
            p = old[i, e]
            if 0 <= p < num_pages:
                holders[p] -= 1
            elif children[i] != 1 or any(parents[r] == i and pages_of(kept[r]) <= e
                                         for r in range(rows)):
                error = True  # an entry that is counted
    for r in range(rows):
        for e in range(pages_of(kept[r])):
            p = table[r, e] = old[parents[r], e]
            if 0 <= p < num_pages:
                holders[p] += 1
    gone, seen = [], set()
    for i in range(rows):
        for e in range(pages_of(lengths[i])):
            p = old[i, e]
            if 0 <= p < num_pages and holders[p] <= 0 and p not in seen:
                gone.append(p)
                seen.add(p)
                error |= holders[p] < 0
    if not bad_head:
        error |= head < len(gone)
        for k, p in enumerate(gone):
            if head - len(gone) + k >= 0:
                free[head - len(gone) + k] = p
        head = max(head - len(gone), 0)
    tails = {}
    for r in range(rows):
        if kept[r] % PAGE:
            tails.setdefault(table[r, pages_of(kept[r]) - 1], []).append(r)
    out = np.full((3, rows), -1, dtype=np.int64)
    out[2] = 0
    total = dict(holders)
    for r in range(rows):
        if kept[r] % PAGE == 0:
            continue
        e = pages_of(kept[r]) - 1
        p = table[r, e]
        if not 0 <= p < num_pages:
            error, table[r, e] = True, old_entry(old, r, e)
            kept[r] -= kept[r] % PAGE
            continue
        if len(tails[p]) == total[p] and tails[p][0] == r:
            continue
        holders[p] -= 1
        to = -1
        if not bad_head and head < len(free):
            to, head = free[head], head + 1
        if 0 <= to < num_pages:
            out[:, r] = p, to, kept[r] % PAGE
            table[r, e] = to
        else:
            error, table[r, e] = True, old_entry(old, r, e)
            kept[r] -= kept[r] % PAGE
    shares = [max(holders[p] - 1, 0) for p in range(num_pages)]
    return (table, shares, free, kept, *out, head), error


def old_entry(old, r, e):
    """Entries past a row's pages stay as they were."""
    return old[r, e]


def compact_pages(table, lengths, shares, free, head, num_pages, max_moves):
    """The k-th held page from the top to the k-th listed one from the bottom."""
    rows, width = table.shape
    ok = 0 <= head <= len(free) and all(0 <= n <= PAGE * width for n in lengths)
    listed = list(free[head:]) if ok else []
    entries = [table[r, e] for r in range(rows) for e in range(pages_of(lengths[r]))] if ok else []
    ok = ok and all(0 <= p < num_pages for p in listed + entries)
    held = sorted(set(entries)) if ok else []
    ok = ok and len(set(listed)) == len(listed) and not set(listed) & set(held)
    sources, targets = np.full(max_moves, -1), np.full(max_moves, -1)
    table, shares, free = table.copy(), list(shares), list(free)
    if not ok:
        return table, shares, free, sources, targets, None
    name = {}
    for k, (p, q) in enumerate(zip(held[::-1], sorted(listed))):
        if k >= max_moves or q >= p:
            break
        sources[k], targets[k], name[p] = p, q, q
    for r in range(rows):
        for e in range(pages_of(lengths[r])):
            table[r, e] = name.get(table[r, e], table[r, e])
    for p, q in name.items():
        shares[q], shares[p] = shares[p], 0
    free[head:] = sorted((set(listed) - set(name.values())) | set(name))
    end = 1 + max((name.get(p, p) for p in held), default=-1)
    return table, shares, free, sources, targets, end


def random_state(rng, requests, beams, hi, grown, width=None, spare=0, filler=-7):
    """Rows in requests of `beams` that hold the whole pages of a prompt together:
    (table, lengths, shares, free list, head, pages)."""
    rows = requests * beams
    prompt = np.repeat(rng.integers(0, hi + 1, requests), beams)
    lengths = prompt + rng.integers(0, grown + 1, rows)
    need, common = pages_of(lengths), prompt // PAGE
    width = width or int(need.max(initial=0)) + 2
    total = int(need.sum()) + spare + rows
    order = rng.permutation(total)
    table = np.full((rows, width), filler, dtype=np.int64)
    used = 0
    for r in range(rows):
        lead = r - r % beams
        have = 0 if r == lead else int(common[r])
        table[r, :have] = table[lead, :have]
        table[r, have:need[r]] = order[used:used + need[r] - have]
        used += need[r] - have
    shares = np.zeros(total, dtype=np.int64)
    for r in range(rows):
        shares[table[r, :need[r]]] += 1
    return table, lengths, np.maximum(shares - 1, 0), order.copy(), used, total


def attention(q, k_pages, v_pages, table, positions, scale, sinks=None):
    """Decode attention in 64 bits: q [R, Hq, D], pages [pages, Hkv, 64, D], as attend_rows."""
    def row(pages, b, n):
        return np.concatenate(list(pages[table[b, : n // PAGE + 1]]), axis=1)[:, : n + 1]
    return attend_rows(q, [None if n < 0 else (row(k_pages, b, n), row(v_pages, b, n))
                           for b, n in enumerate(positions)], scale, sinks)


def attend_rows(q, rows, scale, sinks=None):
    """Row b's queries over rows[b] = its (keys, values), [Hkv, n, D] each, or None.  Returns the
    result, sum_j p_j |v_j|, max_j scale sum_i |q_i k_ij| and sum_j |v_j|."""
    out, mass, every = (np.zeros(q.shape) for _ in range(3))
    size = np.zeros(q.shape[:2] + (1,))
    for b, kv in enumerate(rows):
        if kv is None:
            continue
        k, v = kv
        group = q.shape[1] // len(k)
        for h in range(q.shape[1]):
            kk, vv = k[h // group], v[h // group]
            x = kk @ q[b, h] * scale
            top = max(x.max(), -np.inf if sinks is None else sinks[h])
            e = np.exp(x - top)
            w = e / (e.sum() + (0 if sinks is None else np.exp(sinks[h] - top)))
            out[b, h], mass[b, h], every[b, h] = w @ vv, w @ np.abs(vv), np.abs(vv).sum(0)
            size[b, h] = (np.abs(kk) @ np.abs(q[b, h])).max() * abs(scale)
    return out, mass, size, every


def bound(want, mass, size, every, d):
    """A weight's relative error: its score's, D fp32 additions that may truncate (2 D 2^-24
    of the size); the argument's rounding, 2^-24 of at most 2^8 in log2 units, 2^-16; the
    exponential and the partials' factors 2^-21; the bf16 head and residual 2^-16; the sums,
    a few hundred additions of 2^-24, 2^-15: under 2^-13.  Weights off by e move an output by at most
    2 e sum_j p_j |v_j|; the products with V add in fp32, within the same.  Then one rounding to
    bf16, 2^-8 of the value (2^-134 where bf16 is denormal), and weights under 2^-126 of the
    largest may be taken as zero."""
    weight = 2 * d * 2.0 ** -24 * size + 2.0 ** -13
    return (2 * weight * mass) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want) + 2.0 ** -134 + \
        2.0 ** -126 * every
