"""Oracle of the operators around a block's matrix products: plain fp64 NumPy, from the formulas.

The norms before and after a block with its gate and residual scale, 8-bit values
with a power-of-two scale for each block of 128 and their products, and the norm
and clipping of many gradients. Shares no code with the HIP path.
"""

from __future__ import annotations

import numpy as np


# --- norms around a block ---------------------------------------------------

def spread(gate, rows: int):
    """A gate row for every row of x: gate (G, H), each for rows / G rows."""
    return np.repeat(gate, rows // gate.shape[0], axis=0)


def block_norm(x, y, w_post, w_pre, gate, post_norm, alpha, scale, eps):
    """(r, h); y, the weights and gate may be None."""
    r = alpha * x
    if y is not None:
        z = y / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + eps) if post_norm else y
        if w_post is not None:
            z = z * w_post
        r = r + scale * (z if gate is None else spread(gate, len(x)) * z)
    h = r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    return r, h if w_pre is None else h * w_pre


def block_norm_backward(x, y, w_post, w_pre, gate, post_norm, alpha, scale, eps, g, dh):
    """dict(dx, dy, dw_post, dw_pre, dgate) for the gradients g of r and dh of h (None: zeros)."""
    ones = np.ones(x.shape[1])
    r, _ = block_norm(x, y, w_post, w_pre, gate, post_norm, alpha, scale, eps)
    dr = np.zeros_like(r) if g is None else g.copy()
    out = {"dw_pre": np.zeros(x.shape[1])}
    if dh is not None:
        rr = 1 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
        n, dn = r * rr, dh * (ones if w_pre is None else w_pre)
        dr = dr + rr * (dn - n * np.mean(dn * n, axis=1, keepdims=True))
        out["dw_pre"] = np.sum(dh * n, axis=0)
    out["dx"] = alpha * dr
    if y is None:
        return out
    ry = 1 / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + eps) if post_norm else 1.0
    u, w = y * ry, ones if w_post is None else w_post
    a = scale * dr
    if gate is not None:
        out["dgate"] = (a * u * w).reshape(len(gate), -1, x.shape[1]).sum(1)
        a = a * spread(gate, len(x))
    out["dw_post"] = np.sum(a * u, axis=0)
    du = a * w
    out["dy"] = ry * (du - u * np.mean(du * u, axis=1, keepdims=True)) if post_norm else du
    return out


# --- 8-bit values -----------------------------------------------------------

def e4m3(v):
    """|v| <= 448 rounded to nearest even on e4m3's grid (steps of 2^-9 below 2^-6); NaN stays."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(v), np.abs(v), 0.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.where(np.isfinite(v), np.rint(v / step) * step, np.nan)


def exponent(largest: float) -> int:
    """The smallest whole e >= -126 with largest <= 448 2^e; 0 for a block of zeros."""
    if largest == 0:
        return 0
    e = -126
    while largest > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantize(x, block_rows: int):
    """(values over their scales on the grid, exponent bytes); columns padded to a multiple of 128."""
    rows, cols = x.shape
    nb, nr = -(-cols // 128), -(-rows // block_rows)
    q, s = np.zeros((rows, nb * 128)), np.zeros((nr, nb), np.uint8)
    for i in range(nr):
        for j in range(nb):
            at = (slice(i * block_rows, min(rows, (i + 1) * block_rows)), slice(j * 128, min(cols, (j + 1) * 128)))
            part = x[at]
            finite = np.abs(part[np.isfinite(part)])
            e = exponent(float(finite.max()) if finite.size else 0.0)
            s[i, j] = e + 127
            q[at] = e4m3(np.where(np.isfinite(part), part, np.nan) * 2.0 ** -e)
    return q, s


def value(q, s):
    """What values and exponent bytes stand for; a scale row for each row or for 128 of them."""
    tall = 1 if s.shape[0] == q.shape[0] else 128
    f = np.exp2(s.astype(np.float64) - 127)
    f = np.repeat(np.repeat(f, tall, axis=0)[:q.shape[0]], 128, axis=1)
    return q * f


def quantize_groups(x, offsets):
    """The transpose by groups: (values (cols, P), bytes, written columns), P = (rows // 128 + groups) * 128."""
    rows, cols = x.shape
    groups = len(offsets) - 1
    p = (rows // 128 + groups) * 128
    q, s = np.full((cols, p), np.nan), np.zeros((cols, p // 128), np.uint8)
    written, at = np.zeros(p, bool), 0
    for e in range(groups):
        part = x[offsets[e]:offsets[e + 1]]
        if not len(part):
            continue
        qe, se = quantize(part.T, 1)
        q[:, at:at + qe.shape[1]], s[:, at // 128:at // 128 + se.shape[1]] = qe, se
        written[at:at + qe.shape[1]] = True
        at += qe.shape[1]
    return q, s, written


# --- gradients together -----------------------------------------------------

def grad_norm(grads):
    return float(np.sqrt(sum(float(np.sum(np.square(g))) for g in grads)))


def clip_factor(norm, max_norm, eps):
    with np.errstate(all="ignore"):
        c = np.float64(max_norm) / (np.float64(norm) + eps)
    return 1.0 if c >= 1 else float(c)
