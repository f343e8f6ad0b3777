"""Plain 64-bit implementations, on the host, of the operators of
include/pgd_ext.h, request by request and token by token."""
from __future__ import annotations

import math

import numpy as np

PAGE = 64


def assign_pages(table, cached, new, free, num_tokens, num_pages, head=0):
    """Returns (table, rows, positions, slots, starts, lengths, head, error)."""
    table = table.copy()
    requests, width = table.shape
    rows = np.zeros(num_tokens, dtype=np.int64)
    positions = np.full(num_tokens, -1, dtype=np.int64)
    slots = np.full(num_tokens, -1, dtype=np.int64)
    starts = np.zeros(requests + 1, dtype=np.int64)
    lengths = np.array(cached, dtype=np.int64)
    error = not 0 <= head <= len(free)
    room = 0 if error else len(free) - head
    place = page = taken = 0
    for r in range(requests):
        starts[r] = min(place, num_tokens)
        c, t = int(cached[r]), int(new[r])
        if c < 0 or t < 0 or c + t > width * PAGE:
            error = True
            continue
        have, need = -(-c // PAGE), -(-(c + t) // PAGE)
        extra = need - have
        if (t and place + t > num_tokens) or (extra and page + extra > room):
            error = True
        else:
            for j in range(extra):
                table[r, have + j] = free[head + page + j]
                error |= not 0 <= table[r, have + j] < num_pages
            taken = max(taken, page + extra) if extra else taken
            lengths[r] = c + t
            for i in range(t):
                n = c + i
                p = int(table[r, n // PAGE])
                rows[place + i], positions[place + i] = r, n
                if 0 <= p < num_pages:
                    slots[place + i] = p * PAGE + n % PAGE
                else:
                    error = True
        place += t
        page += extra
    starts[requests] = min(place, num_tokens)
    return table, rows, positions, slots, starts, lengths, head + taken, error


def frequencies(rotary_dim, theta, scaling="none", factor=1.0, original=0.0, beta_fast=32.0,
                beta_slow=1.0, exact_bounds=False, low_band=1.0, high_band=4.0):
    """Radians a position of each pair, and the factor of cos and sin."""
    if scaling == "ntk":
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    out, scale = [], 1.0
    for i in range(rotary_dim // 2):
        f = theta ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            a = rotary_dim * math.log(original / (beta_fast * 2 * math.pi)) / (2 * math.log(theta))
            b = rotary_dim * math.log(original / (beta_slow * 2 * math.pi)) / (2 * math.log(theta))
            if not exact_bounds:
                a, b = math.floor(a), math.ceil(b)
            a, b = max(a, 0), min(b, rotary_dim - 1)
            r = min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
            scale = 0.1 * math.log(factor) + 1.0
        elif scaling == "banded":
            turns = original * f / (2 * math.pi)
            s = min(max((turns - low_band) / (high_band - low_band), 0.0), 1.0)
            f = f * s + f / factor * (1 - s)
        out.append(f)
    return np.array(out, dtype=np.float64), scale


def rotate(x, positions, freq, factor, interleaved):
    """x: float64 [P, heads, D]; the first 2 len(freq) dims of each head rotated."""
    x = np.array(x, dtype=np.float64)
    rd = 2 * len(freq)
    # whole turns dropped in extended precision, so far positions keep their angle
    turns = np.asarray(positions, dtype=np.longdouble)[:, None] * (
        freq.astype(np.longdouble) / (2 * np.pi * np.longdouble(1)))
    angle = ((turns - np.rint(turns)) * 2 * np.pi).astype(np.float64)[:, None, :]
    c, s = factor * np.cos(angle), factor * np.sin(angle)
    a = x[..., 0:rd:2] if interleaved else x[..., : rd // 2]
    b = x[..., 1:rd:2] if interleaved else x[..., rd // 2: rd]
    ra, rb = a * c - b * s, b * c + a * s
    if interleaved:
        x[..., 0:rd:2], x[..., 1:rd:2] = ra, rb
    else:
        x[..., : rd // 2], x[..., rd // 2: rd] = ra, rb
    return x


def visible(n, first=0, window=0, prefix=0):
    """First and last position seen from position n (lo > hi: none)."""
    hi = max(n, prefix - 1)
    lo = max(0, first, n - window + 1 if window > 0 else 0)
    return lo, hi


def attention(q, k_rows, v_rows, rows, positions, *, scale, softcap=0.0, slopes=None, sinks=None,
              first=None, window=0, prefix=None):
    """Token by token: q float64 [P, Hq, D]; k_rows, v_rows: per table row float64
    [Hkv, positions, D].  Returns the outputs and, for bounds on a kernel's error,
    per output sum_j p_j |v_j|, per token and head max_j scale sum_i |q_i k_ij| and
    max_j |bias_j|."""
    tokens, hq, d = q.shape
    out = np.zeros_like(q)
    mass = np.zeros_like(q)
    size = np.zeros((tokens, hq, 1))
    far = np.zeros((tokens, hq, 1))
    for t in range(tokens):
        n, r = int(positions[t]), int(rows[t])
        if n < 0:
            continue
        lo, hi = visible(n, 0 if first is None else int(first[t]), window,
                         0 if prefix is None else int(prefix[r]))
        if lo > hi:
            continue
        k, v = k_rows[r][:, lo:hi + 1], v_rows[r][:, lo:hi + 1]
        group = hq // k.shape[0]
        qt = q[t].reshape(k.shape[0], group, d)
        x = scale * np.einsum("gud,gsd->gus", qt, k)
        s = abs(scale) * np.einsum("gud,gsd->gus", np.abs(qt), np.abs(k))
        if softcap > 0:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            bias = np.asarray(slopes, dtype=np.float64).reshape(k.shape[0], group, 1) * np.abs(
                np.arange(lo, hi + 1) - n)
            x = x - bias
            far[t] = np.abs(bias).max(-1).reshape(hq, 1)
        top = x.max(-1, keepdims=True)
        if sinks is not None:
            sk = np.asarray(sinks, dtype=np.float64).reshape(k.shape[0], group, 1)
            top = np.maximum(top, sk)
        e = np.exp(x - top)
        total = e.sum(-1, keepdims=True)
        if sinks is not None:
            total = total + np.exp(sk - top)
        p = e / total
        out[t] = np.einsum("gus,gsd->gud", p, v).reshape(hq, d)
        mass[t] = np.einsum("gus,gsd->gud", p, np.abs(v)).reshape(hq, d)
        size[t] = s.max(-1).reshape(hq, 1)
    return out, mass, size, far
