"""fp64 CPU oracle of the attention calls (numpy).

TEST INFRASTRUCTURE ONLY: only tests/ may import this module.  The library
never imports it, and it imports nothing from the library.

Each function is the definition written out: no running maximum, no tiles.
Parity status: pinned by ``tests/test_attention_oracle.py`` (hand-worked
cases, rotations as complex numbers, invariances).
"""

from __future__ import annotations

from typing import Optional, Tuple

import numpy as np


def norm(x: np.ndarray, w: Optional[np.ndarray], eps: float) -> np.ndarray:
    """x [..., D] * w / sqrt(mean(x^2) + eps); w None leaves x alone."""
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x * np.asarray(w, np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def rotate(x: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, neighbours: bool) -> np.ndarray:
    """x [T, H, D]: the first 2 * len(inv_freq) elements of each head turned by pos[t] * inv_freq[p]."""
    x = np.array(x, np.float64)
    half = len(inv_freq)
    a_at = np.arange(half) * 2 if neighbours else np.arange(half)
    b_at = a_at + 1 if neighbours else a_at + half
    angle = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    a, b = x[..., a_at].copy(), x[..., b_at].copy()
    x[..., a_at] = a * np.cos(angle) - b * np.sin(angle)
    x[..., b_at] = b * np.cos(angle) + a * np.sin(angle)
    return x


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, seen: np.ndarray, scale: float,
           ) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """One head: q [R, D], k and v [S, D], seen bool [R, S] -> out [R, D], lse [R], and for error bounds
    sum_j p_ij |v_j| [R, D] and max_j |scale| sum_d |q_id k_jd| over the seen keys [R].
    Unseen keys and values take no part, whatever they hold; a row that sees nothing gives 0 and -inf."""
    R, D = q.shape
    out, lse, weight_abs, score_abs = np.zeros((R, D)), np.full(R, -np.inf), np.zeros((R, D)), np.zeros(R)
    for r in range(R):
        j = np.flatnonzero(seen[r])
        if not len(j):
            continue
        kj, vj = np.asarray(k[j], np.float64), np.asarray(v[j], np.float64)
        qr = np.asarray(q[r], np.float64)
        s = scale * (kj @ qr)
        top = s.max()
        e = np.exp(s - top)
        out[r] = (e / e.sum()) @ vj
        lse[r] = top + np.log(e.sum())
        weight_abs[r] = (e / e.sum()) @ np.abs(vj)
        score_abs[r] = abs(scale) * (np.abs(kj) @ np.abs(qr)).max()
    return out, lse, weight_abs, score_abs
