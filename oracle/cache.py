"""Oracle of the rotary positions and the paged cache: plain fp64 on the CPU.

TEST INFRASTRUCTURE, written from the definitions below; it shares no code
with the CUDA path and never imports the package.  Arrays are numpy fp64
unless they are indices; nothing is rounded to a storage type here.

  rotary   pair (a, b) at position t -> m (a cos - b sin, b cos + a sin),
           angle t * f_i; pairs (i, i + rot/2) or (2i, 2i + 1).
  append   row t of sequence b goes to slot lengths[b] - counts[b] + t.
  decode   softmax over the sequence's slots, grouped query heads.
  evict    keep by (protected, weight, lower slot); the i-th kept row at a
           slot >= m moves to the i-th given-up slot < m.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=0.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "bands":
            turns = original * f / (2.0 * math.pi)
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = (1.0 - g) * f / factor + g * f
        out.append(f)
    return np.array(out)


def rotate(x, positions, f, layout, magnitude=1.0, transpose=False):
    """x: [..., N, d] fp64; positions: [..., N] broadcastable to it."""
    x = np.asarray(x, dtype=np.float64)
    rot = 2 * len(f)
    angle = np.asarray(positions, dtype=np.float64)[..., None] * f
    c, s = np.cos(angle) * magnitude, np.sin(angle) * magnitude
    if transpose:
        s = -s
    y = x.copy()
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2] = a * c - b * s
        y[..., rot // 2: rot] = b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * s
        y[..., 1:rot:2] = b * c + a * s
    return y


def rows(pages, table, n, page):
    """[H, n, d]: the first n slots of the sequence with this row of the table."""
    out = np.empty((pages.shape[1], n, pages.shape[3]), dtype=pages.dtype)
    for j in range(n):
        out[:, j] = pages[table[j // page], :, j % page]
    return out


def decode(q, k, v, scale):
    """q: [Hq, d]; k, v: [H, n, d].  (O [Hq, d], lse [Hq], P [Hq, n])."""
    Hq, d = q.shape
    H, n, _ = k.shape
    G = Hq // H
    o, lse, p = np.zeros((Hq, d)), np.full(Hq, -np.inf), np.zeros((Hq, n))
    for h in range(Hq):
        if n == 0:
            continue
        s = (k[h // G] @ q[h]) * scale
        top = s.max()
        lse[h] = top + math.log(np.exp(s - top).sum())
        p[h] = np.exp(s - lse[h])
        o[h] = p[h] @ v[h // G]
    return o, lse, p


def evict(weights, n, budget, positions=None, protect=None):
    """One (sequence, head): weights [capacity].  Returns (m, moves as a list
    of (source slot, target slot), the kept slots in ascending order)."""
    m = min(n, budget)
    pos = list(range(n)) if positions is None else [int(p) for p in positions[:n]]

    def key(j):
        w = float(weights[j])
        return (0 if protect is not None and pos[j] >= protect else 1, 1 if w != w else 0,
                0.0 if w != w else -w, j)

    kept = sorted(sorted(range(n), key=key)[:m])
    chosen = set(kept)
    sources = [j for j in kept if j >= m]
    targets = [j for j in range(m) if j not in chosen]
    return m, list(zip(sources, targets)), kept
