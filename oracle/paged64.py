"""Plain 64-bit statements of the paged cache's calls, in NumPy, one sequence
after the other: test infrastructure only, no code shared with the library."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["decode", "append", "reserve", "fork", "free", "compact"]


def _f64(x):
    return x.detach().double().cpu().numpy() if hasattr(x, "detach") else np.asarray(x, dtype=np.float64)


def decode(q, k_pages, v_pages, table, lens, scale, window=0, sinks=0):
    """(o, lse, weight, reach) in float64: the attention of the newest token of
    each sequence; weight [S, H, d] = sum_j P_j |V_j|, the size of the terms
    behind each output, and reach [S, H] = scale max_j sum |q||K_j|, the size
    of those behind each score."""
    q, kp, vp = _f64(q), _f64(k_pages), _f64(v_pages)
    S, H, d = q.shape
    page, Hkv = kp.shape[2], kp.shape[1]
    o, lse = np.zeros_like(q), np.full((S, H), -np.inf)
    weight, reach = np.zeros_like(q), np.zeros((S, H))
    for s in range(S):
        n = int(lens[s])
        seen = [j for j in range(n) if not window or n - 1 - j < window or j < sinks]
        if not seen:
            continue
        for h in range(H):
            g = h // (H // Hkv)
            k = np.stack([kp[table[s][j // page], g, j % page] for j in seen])
            v = np.stack([vp[table[s][j // page], g, j % page] for j in seen])
            x = scale * (k @ q[s, h])
            m = x.max()
            e = np.exp(x - m)
            lse[s, h] = m + math.log(e.sum())
            p = e / e.sum()
            o[s, h], weight[s, h] = p @ v, p @ np.abs(v)
            reach[s, h] = scale * (np.abs(k) @ np.abs(q[s, h])).max()
    return o, lse, weight, reach


def append(k, v, k_pages, v_pages, table, lens, cu=None):
    """Writes into the given arrays [P, Hkv, page, d]."""
    page = k_pages.shape[2]
    for s in range(len(lens)):
        lo, hi = (cu[s], cu[s + 1]) if cu is not None else (s, s + (lens[s] > 0))
        for t in range(lo, hi):
            pos = lens[s] - (hi - t)
            k_pages[table[s][pos // page], :, pos % page] = k[t]
            v_pages[table[s][pos // page], :, pos % page] = v[t]


def _held(n, page):
    return -(-n // page)


def reserve(refs, table, lens, add, page):
    """Changes the given lists; returns what is missing."""
    P, M = len(refs), len(table[0])
    if any(n < 0 or a < 0 or n + a > M * page for n, a in zip(lens, add)):
        return -1
    want = [(s, i) for s, (n, a) in enumerate(zip(lens, add)) for i in range(_held(n, page), _held(n + a, page))]
    free_pages = [p for p in range(P) if refs[p] == 0]
    if len(want) > len(free_pages):
        return len(want) - len(free_pages)
    for (s, i), p in zip(want, free_pages):
        table[s][i], refs[p] = p, 1
    for s, a in enumerate(add):
        lens[s] += a
    return 0


def fork(pools, refs, table, lens, src, dst, page):
    """pools: arrays [L, P, Hkv, page, d].  Changes everything given; returns what is missing."""
    S, before = len(lens), list(lens)
    if len(set(dst)) < len(dst) or any(not 0 <= x < S for x in list(src) + list(dst)) or any(lens[b] for b in dst):
        return -1
    free_pages = [p for p in range(len(refs)) if refs[p] == 0]
    part = [f for f, a in enumerate(src) if before[a] % page]
    if len(part) > len(free_pages):
        return len(part) - len(free_pages)
    for f, (a, b) in enumerate(zip(src, dst)):
        n = before[a]
        for i in range(n // page):
            table[b][i] = table[a][i]
            refs[table[a][i]] += 1
        if n % page:
            new = free_pages[part.index(f)]
            refs[new] = 1
            for x in pools:
                x[:, new, :, :n % page] = x[:, table[a][n // page], :, :n % page]
            table[b][n // page] = new
        lens[b] = n
    return 0


def free(refs, table, lens, seqs, page):
    for s in seqs:
        for i in range(_held(lens[s], page)):
            refs[table[s][i]] -= 1
            table[s][i] = -1
        lens[s] = 0


def compact(pools, refs, table, lens, page):
    """Returns the number of pages in use."""
    P = len(refs)
    live = sum(r > 0 for r in refs)
    to = dict(zip([p for p in range(live, P) if refs[p] > 0], [p for p in range(live) if refs[p] == 0]))
    for a, b in to.items():
        for x in pools:
            x[:, b] = x[:, a]
        refs[b], refs[a] = refs[a], 0
    for s, n in enumerate(lens):
        for i in range(_held(n, page)):
            table[s][i] = to.get(table[s][i], table[s][i])
    return live
