"""CPU oracle of MXFP4 (microscaled 4-bit floating point) and of its products, in float64.

TEST INFRASTRUCTURE, under the same rule as the rest of this package.  32 consecutive values along
the last axis share a scale 2^X, X = floor(log2 max|v|) - 2 clamped to [-127, 127] (-127 for a zero
block); a value is held as the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times 2^X with its sign, ties to
the even code, saturating at 6.  A block with a NaN or an infinity stands for NaNs.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(a) -> np.ndarray:
    """X + 127 of every block of 32 along the last axis (255: the block holds a NaN or infinity)."""
    a = np.asarray(a, dtype=np.float64)
    blocks = np.abs(a.reshape(a.shape[:-1] + (-1, 32)))
    amax = blocks.max(axis=-1)
    bad = ~np.isfinite(blocks).all(axis=-1)
    amax = np.where(bad, 1.0, amax)
    X = np.full(amax.shape, -127.0)
    np.floor(np.log2(amax, where=amax > 0, out=np.zeros_like(amax)) - 2, where=amax > 0, out=X)
    # log2 next to a power of two: the defining inequality decides
    X = np.where((amax > 0) & (np.ldexp(4.0, X.astype(int)) > amax), X - 1, X)
    X = np.where((amax > 0) & (np.ldexp(8.0, X.astype(int)) <= amax), X + 1, X)
    return np.where(bad, 255, np.clip(X, -127, 127) + 127).astype(np.int64)


def codes(a) -> np.ndarray:
    """E2M1 codes (0 .. 15) of finite blocks, by comparing with every code's value."""
    a = np.asarray(a, dtype=np.float64)
    X = np.repeat(scale_bytes(a) - 127, 32, axis=-1)
    u = np.abs(np.ldexp(np.where(np.isfinite(a), a, 0.0), -X))
    dist = np.abs(np.minimum(u, 6.0)[..., None] - E2M1)
    best = dist.min(axis=-1, keepdims=True)
    # of two codes at the same distance the even one
    near = dist == best
    c = np.where(near & (np.arange(8) % 2 == 0), np.arange(8), -1).max(axis=-1)
    c = np.where(c >= 0, c, near.argmax(axis=-1))
    return c + np.where(np.signbit(a), 8, 0)


def values(a) -> np.ndarray:
    """The values that a stands for in MXFP4."""
    a = np.asarray(a, dtype=np.float64)
    sb = np.repeat(scale_bytes(a), 32, axis=-1)
    c = codes(a)
    v = np.ldexp(E2M1[c & 7], np.where(sb == 255, 0, sb - 127))
    return np.where(sb == 255, np.nan, np.where(c & 8, -v, v))


def atom_offset(tile: int, row: int, block: int, cols: int) -> int:
    """Byte of the scale of row `row` (0 .. 127) of row tile `tile`, 32-column block `block`."""
    nkb = (cols + 255) // 256
    return ((tile * nkb + block // 8) * 2 + (block // 4) % 2) * 512 + 16 * (row % 32) + 4 * (row // 32) + block % 4


def product(a, b, offsets=None):
    """a [M, K] b^T with b [N, K], or rows of group g times b[g] (rows of no group: zeros).  a and b are
    the values of the operands.  Returns (product, sum of the terms' magnitudes)."""
    if offsets is None:
        return a @ b.T, np.abs(a) @ np.abs(b).T
    c = np.zeros((a.shape[0], b.shape[1]))
    m = np.zeros_like(c)
    for g in range(b.shape[0]):
        r = slice(int(offsets[g]), int(offsets[g + 1]))
        c[r] = a[r] @ b[g].T
        m[r] = np.abs(a[r]) @ np.abs(b[g]).T
    return c, m


def swiglu_columns(c):
    """(gate, linear) columns of a product with interleaved weights (groups of 64 and 64)."""
    v = c.reshape(c.shape[0], -1, 2, 64)
    return v[:, :, 0].reshape(c.shape[0], -1), v[:, :, 1].reshape(c.shape[0], -1)


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def bf16(a) -> np.ndarray:
    """Nearest bf16 values (torch's cast)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


def layer_forward_mxfp4(x, w: dict, b, k: int, eps: float = 1e-6) -> np.ndarray:
    """The layer with MXFP4 routed experts: the forward oracle's steps, the experts' products on the MXFP4
    values of bf16 rows of h, of the weights, and of the activations rounded to bf16."""
    import oracle
    r = oracle.layer_routing(x, w, b, k, eps)
    h, idx = bf16(r["h"]), r["idx"]
    o = np.zeros(idx.shape + (h.shape[1],))
    for e in np.unique(idx):
        t, i = np.nonzero(idx == e)
        w1, w3, w2 = (values(oracle.f64(w[n][e])) for n in ("w1", "w3", "w2"))
        a = values(h[t])
        o[t, i] = values(bf16(silu(a @ w1.T) * (a @ w3.T))) @ w2.T
    y = oracle.up_projection(oracle.combine(r["gates"], o), oracle.f64(w["w_up"]))
    if "ws1" in w:
        x_hat = oracle.rmsnorm(oracle.f64(x), oracle.f64(w["rms_gain"]), eps)
        y = y + oracle.shared_expert(x_hat, oracle.f64(w["ws1"]), oracle.f64(w["ws3"]), oracle.f64(w["ws2"]))
    return y
