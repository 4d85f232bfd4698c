"""fp64 reference of the key-value cache of a hybrid model's attention layers: rotary positions,
appending to pages, attention over them, and the page tables.

TEST INFRASTRUCTURE ONLY, like the rest of `oracle/`: it shares no code with the CUDA library.
Everything is written token by token and row by row from the definitions.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, trained_length=0, slow=1.0, fast=32.0):
    """Returns (radians per position of each pair, magnitude)."""
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = np.array([math.pow(base, -2 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "by_parts":
        turns = trained_length / (2 * math.pi / f)
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1
    return f, 1.0


def rotary(x, positions, freq, interleaved=False, magnitude=1.0, transpose=False):
    """x [T, H, D]: the leading 2 * len(freq) channels turned."""
    y = np.array(x, np.float64)
    n = len(freq)
    sign = -1.0 if transpose else 1.0
    for t, p in enumerate(positions):
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            c, s = math.cos(float(p) * freq[i]), sign * math.sin(float(p) * freq[i])
            xa, xb = x[t, :, a].astype(np.float64), x[t, :, b].astype(np.float64)
            y[t, :, a] = magnitude * (xa * c - xb * s)
            y[t, :, b] = magnitude * (xb * c + xa * s)
    return y


def attention(q, k, v, window, scale, softcap=0.0, span=0, slopes=None):
    """One sequence: q [W, H, D], its W last tokens' queries; k, v [len, HK, D].  Returns (o, lse,
    sum of p |v|, largest |s| and largest |scale| sum |q k| of each row): the last two for tolerances."""
    W, H, D = q.shape
    n, HK = k.shape[0], k.shape[1]
    o, a = np.zeros((W, H, D)), np.zeros((W, H, D))
    lse, big, mass = np.full((W, H), -np.inf), np.zeros((W, H)), np.zeros((W, H))
    for w in range(W):
        p = n - W + w
        lo = max(0, p - span + 1) if span else 0
        if p < 0:
            continue
        for h in range(H):
            kh = h // (H // HK)
            keys, vals = k[lo:p + 1, kh], v[lo:p + 1, kh]
            s = scale * (keys @ q[w, h])
            mass[w, h] = (abs(scale) * (np.abs(keys) @ np.abs(q[w, h]))).max()
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s + slopes[h] * (np.arange(lo, p + 1) - p)
            m = s.max()
            e = np.exp(s - m)
            o[w, h] = e @ vals / e.sum()
            a[w, h] = e @ np.abs(vals) / e.sum()
            lse[w, h] = m + math.log(e.sum())
            big[w, h] = np.abs(s).max()
    return o, lse, a, big, mass


def gather(pages, row, n):
    """The first n tokens of a table row."""
    P = pages.shape[1]
    return np.stack([pages[row[j // P], j % P] for j in range(n)]) if n else pages[:0, 0]


def update(table, lens, refs, parent, new_lens, P):
    """Returns (table, lens, refs, kept, [(source, target) copies]); raises ValueError where the
    library refuses."""
    S, width = table.shape
    pages = lambda n: -(-n // P)                                              # noqa: E731
    if any(pages(n) > width for n in list(lens) + list(new_lens)):
        raise ValueError("a row is too long")
    if any(not -1 <= p < S for p in parent):
        raise ValueError("no such parent")
    if any(q >= 0 and refs[q] <= 0 for r in range(S) for q in table[r, :pages(lens[r])]):
        raise ValueError("a row names a free page")
    free = [q for q, r in enumerate(refs) if r == 0]
    count = [int(r) for r in refs]
    for r in range(S):
        for q in table[r, :pages(lens[r])]:
            if q >= 0:
                count[q] -= 1
    kept = [min(lens[p], n) if p >= 0 else 0 for p, n in zip(parent, new_lens)]
    rows = [[int(q) for q in table[p, :k // P]] if p >= 0 else [] for p, k in zip(parent, kept)]
    for r in rows:
        for q in r:
            if q >= 0:
                count[q] += 1
    copies, owner = [], {}
    for i, (p, k, n) in enumerate(zip(parent, kept, new_lens)):
        need = pages(n) - len(rows[i])
        if k % P:
            q = int(table[p, k // P])
            if count[q] == 0 and q not in owner:
                owner[q] = i
                rows[i].append(q)
                need -= 1
            else:
                copies.append((q, i))
        for _ in range(need):
            if not free:
                raise ValueError("not enough free pages")
            rows[i].append(free.pop(0))
            count[rows[i][-1]] = 1
    for q in owner:
        count[q] += 1
    out = np.full((len(rows), width), -1, np.int32)
    for i, r in enumerate(rows):
        out[i, :len(r)] = r
    copies = [(q, rows[i][kept[i] // P]) for q, i in copies]
    return out, np.array(new_lens), np.array(count), np.array(kept, np.int64), copies


def compact(table, lens, refs, P):
    """Returns (table, refs, page_map, moves)."""
    used = [q for q, r in enumerate(refs) if r]
    n = len(used)
    moves = list(zip([q for q in used if q >= n], [q for q in range(n) if refs[q] == 0]))
    where = {q: q for q in used if q < n}
    where.update(moves)
    out = np.full_like(table, -1)
    for r in range(table.shape[0]):
        for j in range(-(-lens[r] // P)):
            if table[r, j] >= 0:
                out[r, j] = where[table[r, j]]
    new_refs = np.zeros_like(refs)
    for q, h in where.items():
        new_refs[h] = refs[q]
    return out, new_refs, np.array([where.get(q, -1) for q in range(len(refs))]), moves
