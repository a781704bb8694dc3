"""CPU oracle of the router's balance loss and its gradient, in float64 (test infrastructure).

Per sequence q (tokens cu[q] .. cu[q+1], n_q of them): f_qe = counts_qe E / (k n_q),
P_qe = mean_t s_te / sum_j s_tj, loss = coef / S' sum_q sum_e f_qe P_qe over the S' sequences that
hold tokens.  The counts are constants of the gradient."""
from __future__ import annotations

import numpy as np


def counts(idx, E, cu):
    out = np.zeros((len(cu) - 1, E), dtype=np.int64)
    for q, (lo, hi) in enumerate(zip(cu, cu[1:])):
        sel = np.asarray(idx[lo:hi]).ravel()
        sel = sel[(sel >= 0) & (sel < E)]
        np.add.at(out[q], sel, 1)
    return out


def _probs(s):
    R = s.sum(axis=1, keepdims=True)
    return np.divide(s, R, out=np.zeros_like(s), where=R != 0), R


def loss(scores, cnt, k, cu, coef):
    """The loss for given counts (so differences of it in the scores hold them fixed)."""
    s = np.asarray(scores, dtype=np.float64)
    E = s.shape[1]
    filled = sum(hi > lo for lo, hi in zip(cu, cu[1:]))
    total = 0.0
    for q, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if hi > lo:
            p, _ = _probs(s[lo:hi])
            total += coef / filled * np.dot(cnt[q] * (E / (k * (hi - lo))), p.mean(axis=0))
    return total


def gradient(scores, cnt, k, cu, coef):
    """dL/ds, and the scale of its terms (w (f + D) / R) that its rounding is measured by."""
    s = np.asarray(scores, dtype=np.float64)
    E = s.shape[1]
    g, scale = np.zeros_like(s), np.zeros_like(s)
    filled = sum(hi > lo for lo, hi in zip(cu, cu[1:]))
    for q, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if hi > lo:
            p, R = _probs(s[lo:hi])
            f = cnt[q] * (E / (k * (hi - lo)))
            D = p @ f
            w = np.divide(coef / (filled * (hi - lo)), R, out=np.zeros_like(R), where=R != 0)
            g[lo:hi] = w * (f - D[:, None])
            scale[lo:hi] = np.abs(w) * (f + D[:, None])
    return g, scale
