"""Oracle of the training-step operators: plain fp64 NumPy, from the formulas.

Query/key norm with the position rotation, tokens sorted by expert and back,
and the loss against a teacher's top logits, each with its gradient. Shares no
code with the HIP path.
"""

from __future__ import annotations

import numpy as np


# --- queries and keys -------------------------------------------------------

def _pairs(rope: int, interleaved: bool):
    i = np.arange(rope // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rope // 2)


def rotate(x, cos, sin, interleaved: bool):
    """x (..., D); cos, sin broadcastable to (..., R / 2)."""
    out = np.array(x, dtype=np.float64)
    a, b = _pairs(2 * cos.shape[-1], interleaved)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def norm_rope(x, w, cos, sin, eps, interleaved: bool):
    """x (B, S, H, D), w (D,), cos and sin (B, S, 1, R / 2)."""
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return rotate(n * w, cos, sin, interleaved)


def norm_rope_backward(x, g, w, cos, sin, eps, interleaved: bool):
    """(dx, dw) for the gradient g of norm_rope's output."""
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r
    du = rotate(g, cos, -sin, interleaved)
    dn = du * w
    dx = r * (dn - n * np.mean(dn * n, axis=-1, keepdims=True))
    return dx, np.sum(du * n, axis=tuple(range(x.ndim - 1)))


# --- tokens by expert -------------------------------------------------------

def moe_sort(ids, experts: int):
    """(offsets, slot_of_row, row_of_slot) for ids (T, K), one slot at a time."""
    flat = [int(e) for e in np.asarray(ids).ravel()]
    lists = [[] for _ in range(experts + 1)]
    for s, e in enumerate(flat):
        lists[e if 0 <= e < experts else experts].append(s)
    offsets, slot_of_row, row_of_slot = [0], [], [0] * len(flat)
    for e, slots in enumerate(lists):
        for s in slots:
            row = len(slot_of_row)
            slot_of_row.append(s if e < experts else -1 - s)
            row_of_slot[s] = row if e < experts else -1 - row
        if e < experts:
            offsets.append(len(slot_of_row))
    return (np.array(offsets, np.int32), np.array(slot_of_row, np.int32),
            np.array(row_of_slot, np.int32).reshape(np.shape(ids)))


def moe_dispatch(x, row_of_slot):
    t, k = row_of_slot.shape
    out = np.zeros((t * k, x.shape[1]), dtype=x.dtype)
    for i in range(t):
        for j in range(k):
            if row_of_slot[i, j] >= 0:
                out[row_of_slot[i, j]] = x[i]
    return out


def moe_combine(y, row_of_slot, w=None):
    t, k = row_of_slot.shape
    out = np.zeros((t, y.shape[1]))
    for i in range(t):
        for j in range(k):
            if row_of_slot[i, j] >= 0:
                out[i] += (1.0 if w is None else w[i, j]) * y[row_of_slot[i, j]]
    return out


def moe_combine_backward(g, y, row_of_slot, w):
    t, k = row_of_slot.shape
    dy, dw = np.zeros((t * k, y.shape[1])), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            r = row_of_slot[i, j]
            if r >= 0:
                dy[r] = w[i, j] * g[i]
                dw[i, j] = np.dot(g[i], y[r])
    return dy, dw


# --- distillation -----------------------------------------------------------

def _lse(x):
    if len(x) == 0:
        return -np.inf
    m = np.max(x)
    return m if not np.isfinite(m) else m + np.log(np.sum(np.exp(x - m)))


def _rounding_left(p, scaled, lse, teacher_bf16):
    """What rounding of the teacher's logits (a step of bf16) and of an fp32 logsumexp of them can leave of 1 - sum p."""
    with np.errstate(all="ignore"):
        size = np.abs(scaled)
        each = p * (size * (2.0 ** -7 if teacher_bf16 else 0.0) + 2.0 ** -22 * (size + abs(lse) + 4))
    return np.sum(each[p > 0])


def distill_row(z, ids, t, tau, teacher_lse=None, grad_loss=None, teacher_bf16=False):
    """One row: dict(loss, lse, rest_lse, dlogits, p, p_rest, q) in fp64; z (V,), ids and t (K,).

    teacher_bf16: the teacher's logits were rounded to bf16, which counts where all that is left of 1 - sum p may be
    rounding.
    """
    v = len(z)
    here = [(int(i), float(x)) for i, x in zip(ids, t) if 0 <= i < v]
    empty = {"loss": 0.0, "lse": 0.0, "rest_lse": 0.0, "dlogits": np.zeros(v), "some": False}
    if not here or (teacher_lse is None and all(x == -np.inf for _, x in here)):
        return empty
    with np.errstate(all="ignore"):
        z = np.asarray(z, np.float64) / tau
        tk = np.array([x for _, x in here]) / tau
        log_p = tk - (_lse(tk) if teacher_lse is None else teacher_lse)
        p = np.exp(log_p)
        lse = _lse(z)
        z0 = z - np.max(z)            # log q keeps its digits where z is as large as a type's lowest value
        log_q = z0 - _lse(z0)
        loss = sum(p[i] * (log_p[i] - log_q[j]) for i, (j, _) in enumerate(here) if p[i] != 0)
        q = np.exp(log_q)
        dz = q.copy()
        rest_lse, p_rest = 0.0, 0.0
        if teacher_lse is not None:
            outside = np.ones(v, bool)
            outside[[j for j, _ in here]] = False
            rest_lse, log_q_rest = _lse(z[outside]), _lse(log_q[outside])
            p_rest = max(0.0, 1.0 - p.sum()) if outside.any() else 0.0
            if log_q_rest == -np.inf and 0 < p_rest <= _rounding_left(p, tk, teacher_lse, teacher_bf16):
                p_rest = 0.0
            if p_rest > 0:
                loss += p_rest * (np.log(p_rest) - log_q_rest)
                dz[outside] = (np.exp(log_q_rest) - p_rest) * np.exp(log_q[outside] - log_q_rest)
            else:
                dz *= p.sum()        # what all classes' p add up to, here not 1
        for i, (j, _) in enumerate(here):
            dz[j] -= p[i]
        g = 1.0 if grad_loss is None else grad_loss
    return {"loss": loss, "lse": lse, "rest_lse": rest_lse, "dlogits": dz * g / tau, "p": p, "log_p": log_p, "q": q,
            "p_rest": p_rest, "some": True}
