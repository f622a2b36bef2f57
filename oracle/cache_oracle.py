"""Float64 definition of the token cache's operators (numpy, one stream at a time).

Shares no code with the library.  Pages are numpy arrays [n_pages, heads,
page_size(, d)], table [n_streams, width], lens [n_streams]; offsets cut the new rows
into streams.  Where a result is compared with 16-bit rows, the functions
also return what a tolerance needs (the sums of absolute terms).
"""
from __future__ import annotations

import math

import numpy as np


def rotary(rotary_dim, base, scaling=None, factor=1.0, context=0):
    """Radians per position of every pair, and the factor on a pair's length."""
    freq, length = [], 1.0
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "ramp":
            def index(turns):
                return rotary_dim * math.log(context / (2 * math.pi * turns)) / (2 * math.log(base))
            a, b = max(math.floor(index(32)), 0), min(math.ceil(index(1)), rotary_dim - 1)
            w = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f = (1 - w) * f + w * f / factor
            length = 1 + 0.1 * math.log(factor)
        freq.append(f)
    return np.array(freq), length


def turn(x, positions, freq, length, interleaved):
    """x [rows, heads, d] turned by positions [rows]."""
    y = np.array(x, np.float64)
    half = len(freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = length * np.cos(positions * freq[i])[:, None], length * np.sin(positions * freq[i])[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def slots(table, page_size, s, lo, hi):
    """(pages, rows) of slots lo .. hi - 1 of stream s."""
    j = np.arange(lo, hi)
    return table[s, j // page_size], j % page_size


def seen(length, n, i, causal, window):
    p = length - n + i
    return [j for j in range(max(0, length)) if (not causal or j <= p) and (window <= 0 or j > p - window)]


def attend(q, k_pages, v_pages, table, lens, offsets, scale, causal=True, window=0):
    """(out, lse, spread, reach): spread = sum of w |v|, reach = the largest sum of |q k| * scale of a row."""
    rows, hq, d = q.shape
    hkv, page = k_pages.shape[1], k_pages.shape[2]
    out, spread = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse, reach = np.full((rows, hq), -np.inf), np.zeros((rows, hq))
    for s in range(len(lens)):
        n = offsets[s + 1] - offsets[s]
        p, x = slots(table, page, s, 0, int(lens[s]))
        for i in range(n):
            js = seen(int(lens[s]), n, i, causal, window)
            if not js:
                continue
            for h in range(hq):
                k = k_pages[p[js], h // (hq // hkv), x[js]].astype(np.float64)
                v = v_pages[p[js], h // (hq // hkv), x[js]].astype(np.float64)
                t = offsets[s] + i
                z = k @ q[t, h].astype(np.float64) * scale
                w = np.exp(z - z.max())
                lse[t, h] = z.max() + math.log(w.sum())
                w /= w.sum()
                out[t, h], spread[t, h] = w @ v, w @ np.abs(v)
                reach[t, h] = (np.abs(k) @ np.abs(q[t, h].astype(np.float64))).max() * scale
    return out, lse, spread, reach


def weigh(q, lse, k_pages, mass, table, lens, offsets, scale, causal=True, window=0, decay=1.0):
    """(mass_out, added, terms): added = the new weights alone, terms = how many of them."""
    hq = q.shape[1]
    hkv, page = k_pages.shape[1], k_pages.shape[2]
    out = mass.astype(np.float64).copy()
    added, terms = np.zeros_like(out), np.zeros_like(out)
    for s in range(len(lens)):
        n = offsets[s + 1] - offsets[s]
        if n == 0:
            continue
        p, x = slots(table, page, s, 0, int(lens[s]))
        for i in range(n):
            js = seen(int(lens[s]), n, i, causal, window)
            for h in range(hq):
                hk = h // (hq // hkv)
                t = offsets[s] + i
                z = k_pages[p[js], hk, x[js]].astype(np.float64) @ q[t, h].astype(np.float64) * scale
                added[p[js], hk, x[js]] += np.exp(z - float(lse[t, h]))
                terms[p[js], hk, x[js]] += 1
        for h in range(hkv):
            out[p, h, x] = decay * mass[p, h, x].astype(np.float64) + added[p, h, x]
    return out, added, terms


def evict(mass, table, lens, page_size, budget, recent):
    """Kept slots per stream and key head, ascending (lists)."""
    kept = []
    for s, length in enumerate(int(x) for x in lens):
        p, x = slots(table, page_size, s, 0, length)
        per_head = []
        for h in range(mass.shape[1]):
            new = set(range(max(0, length - recent), length))
            rest = [j for j in range(length) if j not in new]
            w = {j: mass[p[j], h, x[j]] for j in rest}
            rest.sort(key=lambda j: (0 if np.isnan(w[j]) else 1, 0.0 if np.isnan(w[j]) else -float(w[j]), j))
            per_head.append(sorted(list(new) + rest[:max(0, min(length, budget) - len(new))]))
        kept.append(per_head)
    return kept
