"""Float64 definitions of the norm, 8-bit and expert-grouped operators (test
infrastructure only).

Everything is computed from the stored (already rounded) inputs widened to
float64.  The ``*_bound`` functions give the sums of magnitudes that the
tolerances scale with.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
TINY_SCALE = 2.0 ** -126


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


# ---- norm -----------------------------------------------------------------------


def rmsnorm(x64, w64, r64=None, eps=1e-6):
    """(y, h): h = x + r, y = h / sqrt(mean(h^2) + eps) * w."""
    h = x64 if r64 is None else x64 + r64
    u = np.mean(h * h, axis=1, keepdims=True) + eps
    return h / np.sqrt(u) * w64, h


def rmsnorm_grad(dy64, h64, w64, dh64=None, eps=1e-6):
    """(dx, dw, the magnitudes that dx and dw sum)."""
    cols = h64.shape[1]
    u = np.mean(h64 * h64, axis=1, keepdims=True) + eps
    g = dy64 * w64
    dot = np.sum(g * h64, axis=1, keepdims=True)
    mag = np.sum(np.abs(g * h64), axis=1, keepdims=True)
    dx = g / np.sqrt(u) - h64 * dot / (cols * u * np.sqrt(u))
    bound = np.abs(g) / np.sqrt(u) + np.abs(h64) * mag / (cols * u * np.sqrt(u))
    if dh64 is not None:
        dx = dx + dh64
        bound = bound + np.abs(dh64)
    each = dy64 * h64 / np.sqrt(u)
    return dx, each.sum(0), bound, np.abs(each).sum(0)


# ---- 8-bit values with scales ------------------------------------------------------


def row_scales(y64):
    """The scale of each row and 128 columns."""
    out = np.empty((y64.shape[0], blocks(y64.shape[1])))
    for t in range(out.shape[1]):
        part = np.abs(y64[:, t * BLOCK:(t + 1) * BLOCK])
        out[:, t] = np.maximum(part.max(axis=1, initial=0.0) / E4M3_MAX, TINY_SCALE)
    return out


def square_scales(w64):
    """The scale of each 128 x 128 block."""
    out = np.empty((blocks(w64.shape[0]), blocks(w64.shape[1])))
    for i in range(out.shape[0]):
        for t in range(out.shape[1]):
            part = np.abs(w64[i * BLOCK:(i + 1) * BLOCK, t * BLOCK:(t + 1) * BLOCK])
            out[i, t] = max(part.max() / E4M3_MAX, TINY_SCALE)
    return out


def spread(scales, length, axis):
    """One scale per block as one per element along an axis."""
    s = np.repeat(scales, BLOCK, axis=axis)
    return np.take(s, np.arange(length), axis=axis)


def half_step(v64):
    """Half the spacing of e4m3 at |v|: the largest rounding error there."""
    _, e = np.frexp(np.maximum(np.abs(v64), 2.0 ** -10))
    return np.ldexp(1.0, np.maximum(e - 1, -6) - 4)


def gemm_fp8(a64, sa64, b64, sb64):
    """(c, sum of magnitudes) of the block-scaled product; b is n x k."""
    k = a64.shape[1]
    aa = a64 * spread(sa64, k, 1)
    bb = b64 * spread(spread(sb64, b64.shape[0], 0), k, 1)
    return aa @ bb.T, np.abs(aa) @ np.abs(bb).T


# ---- products grouped by expert -------------------------------------------------------


def grouped(a64, w64, offsets, trans_b=False):
    """(c, sum of magnitudes); rows outside every group stay NaN."""
    n = w64.shape[1] if trans_b else w64.shape[2]
    c = np.full((a64.shape[0], n), np.nan)
    s = np.zeros_like(c)
    for g in range(w64.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        w = w64[g].T if trans_b else w64[g]
        c[r] = a64[r] @ w
        s[r] = np.abs(a64[r]) @ np.abs(w)
    return c, s


def grouped_fp8(a64, sa64, b64, sb64, offsets):
    c = np.full((a64.shape[0], b64.shape[1]), np.nan)
    s = np.zeros_like(c)
    for g in range(b64.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        if r.stop > r.start:
            c[r], s[r] = gemm_fp8(a64[r], sa64[r], b64[g], sb64[g])
    return c, s


def wgrad(a64, dc64, offsets):
    groups = len(offsets) - 1
    dw = np.zeros((groups, a64.shape[1], dc64.shape[1]))
    s = np.zeros_like(dw)
    for g in range(groups):
        r = slice(offsets[g], offsets[g + 1])
        dw[g] = a64[r].T @ dc64[r]
        s[g] = np.abs(a64[r]).T @ np.abs(dc64[r])
    return dw, s
