"""Oracle of the beam rows' attention.

OneLA (paper summary), section 3.3: the children of a beam share their parents'
records by reference. A row attends its request's prompt, then its own
ancestors; the ancestors are found by following the back-pointers, one row and
one head at a time, in float64.

Reading: a row one of whose back-pointers leaves [0, B) (step 0: is negative) is
a dead beam and gives zeros, as does a row that attends nothing.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


def ancestors(bp_parent, level: int, r: int, b: int):
    """[(u, slot)] of the row's tokens, the newest first; None for a dead beam."""
    path, slot = [], b
    B = bp_parent.shape[2] if level else 0
    for u in range(level - 1, -1, -1):
        path.append((u, slot))
        slot = int(bp_parent[u, r, slot])
        if slot < 0 or (u > 0 and slot >= B):
            return None
    return path


def beam_attention(q, prompts, level=0, k_beam=None, v_beam=None, bp_parent=None, scale=None):
    """q [R*B, H, D]; prompts: one (k [len, Hkv, D], v) per request; k_beam, v_beam
    [level, R*B, Hkv, D]; all float64. Returns out [R*B, H, D], and per (row,
    head) the weighted mean of |v| per element and the largest sum of the
    magnitudes of a score's terms (what error bounds are made of)."""
    rows, H, D = q.shape
    R = len(prompts)
    B = rows // R
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros_like(q)
    mean_abs = np.zeros_like(q)
    terms = np.zeros((rows, H))
    for r in range(R):
        k0, v0 = prompts[r]
        Hkv = k0.shape[1]
        for b in range(B):
            path = ancestors(bp_parent, level, r, b) if level else []
            if path is None:
                continue
            row = r * B + b
            k = np.concatenate([k0] + [k_beam[u, r * B + s][None] for u, s in path])
            v = np.concatenate([v0] + [v_beam[u, r * B + s][None] for u, s in path])
            if k.shape[0] == 0:
                continue
            for h in range(H):
                g = h // (H // Hkv)
                x = scale * (k[:, g] @ q[row, h])
                w = np.exp(x - x.max())
                w /= w.sum()
                out[row, h] = w @ v[:, g]
                mean_abs[row, h] = w @ np.abs(v[:, g])
                terms[row, h] = abs(scale) * (np.abs(k[:, g]) @ np.abs(q[row, h])).max()
    return out, mean_abs, terms
