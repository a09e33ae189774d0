"""ctypes binding of the training-step operators of ``include/ns.h``: argument
marshalling only, under the C entry points' names.

Outputs and inputs are torch tensors on the current GPU, and a call's work goes
to ``stream`` (default: torch's current one) without waiting for it. Tensors
that torch allocated on another stream are the caller's to order and to record
on it, as for any kernel. The calls that need a workspace take one (a uint8 GPU
tensor) or allocate it, and return it for reuse.
"""

from __future__ import annotations

import ctypes
import struct

from . import _lib
from ._lib import NS_BF16, NS_F32, _check, _new_workspace, lib


class ns_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


# The same 40 bytes made in one step: a call's marshalling is as long as a short kernel, so it is kept brief.
_pack_heads = struct.Struct("@Pqqqi4x").pack
_NO_HEADS = _pack_heads(0, 0, 0, 0, 0)
assert len(_NO_HEADS) == ctypes.sizeof(ns_heads)

_torch = None      # imported with the first call
_codes, _int_sizes = {}, {}


def _load_torch():
    global _torch
    import torch
    _codes.update({torch.bfloat16: NS_BF16, torch.float32: NS_F32})
    _int_sizes.update({torch.int32: 4, torch.int64: 8})
    _torch = torch
    return torch


def _c():
    """The loaded library (without the lock once it is there)."""
    return _lib._lib or lib()


def _code(t, name: str) -> int:
    """The ns_dtype of a float tensor."""
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _int_bytes(t, name: str) -> int:
    size = _int_sizes.get(t.dtype)
    if size is None:
        raise TypeError(f"{name} must be int32 or int64, not {t.dtype}")
    return size


def _on_gpu(names: str, tensors) -> int:
    """Checks that all tensors (or None) are on the current GPU; returns its index. Every call's first step."""
    torch = _torch or _load_torch()
    here = None
    for t in tensors:
        if t is None:
            continue
        at = t.get_device()
        if at != here:
            if here is None and at >= 0:
                here = torch.cuda.current_device()
            if at != here:
                name = next(n for n, x in zip(names.split(), tensors) if x is t)
                raise ValueError(f"{name} is on {t.device}, not on the current GPU")
    return here


def _stream(stream, device: int) -> int:
    """The stream's handle; torch's current one on the device by default."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _array(t, name: str, shape, dtype):
    """Checks a contiguous tensor of one shape and dtype; returns its address."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and of shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _floats(t, name: str, shape):
    return _array(t, name, shape, _torch.float32)


def _ints(t, name: str, shape):
    return _array(t, name, shape, _torch.int32)


def _rows(t, name: str, rows: int, cols: int, dtype) -> int:
    """Checks a (rows, cols) tensor whose rows are contiguous; returns its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape ({rows}, {cols}), not {tuple(t.shape)}")
    down, across = t.stride()
    if across != 1 and cols > 1 and rows:
        raise ValueError(f"each row of {name} must be contiguous")
    return down if rows > 1 else max(cols, 1)


def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace, or a new one of ``nbytes()`` (the library checks the size of a given one)."""
    if workspace is None:
        return _new_workspace(nbytes(), device, stream)
    if workspace.dtype is not _torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    return workspace


# ---------------------------------------------------------------------------
# queries and keys
# ---------------------------------------------------------------------------

def _heads(t, name: str, shape, dtype) -> bytes:
    """The ns_heads of a tensor with contiguous heads, checked against the shape and dtype it must have."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must have shape {tuple(shape)} and dtype {dtype}, not {tuple(t.shape)}, {t.dtype}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and t.numel():
        raise ValueError(f"each head of {name} must be contiguous")
    return _pack_heads(t.data_ptr(), st[0] if len(st) == 4 else 0, st[-3], st[-2], shape[-2])


def _head_args(q, k, like, q_weight, k_weight, cos, sin, pos, eps, interleaved):
    """(sizes, heads, the arguments from the weights to the positions) that the two calls share. ``like``: pairs of
    tensors, each shaped like q and k, whose heads follow those of q and k."""
    first = k if q is None else q
    if first is None:
        raise ValueError("q or k is required")
    shape, dtype = first.shape, first.dtype
    code = _code(first, "q or k")
    if len(shape) == 4:
        batch, seq, _, dim = shape
    elif len(shape) == 3:
        batch = 1
        seq, _, dim = shape
    else:
        raise ValueError("q and k must be (batch, seq, heads, head_dim) or (seq, heads, head_dim)")
    if q is not None and k is not None:
        ks = k.shape
        if k.dtype != dtype or ks[:-2] != shape[:-2] or ks[-1] != dim:
            raise ValueError("q and k must share dtype, batch, seq and head_dim")
    heads = []
    for a, b, name in ((q, k, ""), *like):
        for t, of, side in ((a, q, "q"), (b, k, "k")):
            if t is None or of is None:
                if t is not None or of is not None:
                    raise ValueError(f"{name % side} goes with {side}: give both or neither")
                heads.append(_NO_HEADS)
            else:
                heads.append(_heads(t, name % side if name else side, of.shape, dtype))
    w_code, wq, wk = NS_F32, None, None
    if q_weight is not None or k_weight is not None:
        w = k_weight if q_weight is None else q_weight
        w_code = _code(w, "weights")
        if w.shape != (dim,) or not w.is_contiguous() or (q_weight is not None and k_weight is not None and (
                k_weight.dtype != w.dtype or k_weight.shape != (dim,) or not k_weight.is_contiguous())):
            raise ValueError(f"weights must share one dtype and be contiguous of shape ({dim},)")
        wq = None if q_weight is None else q_weight.data_ptr()
        wk = None if k_weight is None else k_weight.data_ptr()
    cos_ptr = sin_ptr = pos_ptr = None
    rows = rope = pos_stride = 0
    pos_bytes = 4
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        table = cos.shape
        if len(table) != 2:
            raise ValueError("cos and sin must be (positions, rope_dim / 2)")
        cos_ptr, sin_ptr = _floats(cos, "cos", table), _floats(sin, "sin", table)
        rows, rope = table[0], 2 * table[1]
    if pos is not None:
        pos_bytes = _int_bytes(pos, "pos")
        if pos.shape == (batch, seq):
            pos_stride = seq
        elif pos.shape != (seq,):
            raise ValueError(f"pos must have shape ({seq},) or ({batch}, {seq}), not {tuple(pos.shape)}")
        if not pos.is_contiguous():
            raise ValueError("pos must be contiguous")
        pos_ptr = pos.data_ptr()
    return (batch, seq, dim, code), heads, (wq, wk, w_code, eps, cos_ptr, sin_ptr, rows, rope, 1 if interleaved else 0,
                                            pos_ptr, pos_bytes, pos_stride)


def ns_qk_norm_rope(q, k, q_out, k_out, q_weight=None, k_weight=None, cos=None, sin=None, pos=None,
                    eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """RMS norm of each head of q and k, its weight and the position rotation (see ns.h).

    q, k: (batch, seq, heads, head_dim) or (seq, heads, head_dim) views with
    contiguous heads, bf16 or f32; k (or q) and its output may be None. cos, sin:
    (positions, rope_dim / 2) f32, or None for no rotation. pos: (seq,) or
    (batch, seq) int32 or int64, or None for 0, 1, ... Outputs may be the inputs.
    """
    device = _on_gpu("q k q_out k_out q_weight k_weight cos sin pos",
                     (q, k, q_out, k_out, q_weight, k_weight, cos, sin, pos))
    sizes, (hq, hk, oq, ok), rest = _head_args(q, k, ((q_out, k_out, "%s_out"),), q_weight, k_weight, cos, sin, pos,
                                               eps, interleaved)
    _check(_c().ns_qk_norm_rope(*sizes, hq, hk, *rest, oq, ok, _stream(stream, device)))


def ns_qk_norm_rope_workspace_bytes(batch: int, seq: int, head_dim: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ns_qk_norm_rope_workspace_bytes(batch, seq, head_dim, ctypes.byref(n)))
    return n.value


def ns_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dq_weight=None, dk_weight=None, q_weight=None,
                             k_weight=None, cos=None, sin=None, pos=None, eps: float = 1e-6,
                             interleaved: bool = False, workspace=None, stream=None):
    """Gradient of ns_qk_norm_rope (see ns.h): q and k are the forward's inputs,
    dq_weight and dk_weight (head_dim) f32 or None. Returns the workspace (None
    if neither weight gradient is wanted and none was given)."""
    device = _on_gpu("q k dq_out dk_out dq dk dq_weight dk_weight q_weight k_weight cos sin pos workspace",
                     (q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, q_weight, k_weight, cos, sin, pos, workspace))
    sizes, (hq, hk, gq, gk, oq, ok), rest = _head_args(q, k, ((dq_out, dk_out, "d%s_out"), (dq, dk, "d%s")), q_weight,
                                                       k_weight, cos, sin, pos, eps, interleaved)
    dim = (sizes[2],)
    wq, wk = _floats(dq_weight, "dq_weight", dim), _floats(dk_weight, "dk_weight", dim)
    if wq or wk:
        workspace = _workspace(workspace, lambda: ns_qk_norm_rope_workspace_bytes(*sizes[:3]),
                               (k if q is None else q).device, stream)
    _check(_c().ns_qk_norm_rope_backward(
        *sizes, hq, hk, gq, gk, *rest, oq, ok, wq, wk, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), _stream(stream, device)))
    return workspace


# ---------------------------------------------------------------------------
# tokens by expert
# ---------------------------------------------------------------------------

def ns_moe_sort_workspace_bytes(tokens: int, top_k: int, num_experts: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ns_moe_sort_workspace_bytes(tokens, top_k, num_experts, ctypes.byref(n)))
    return n.value


def ns_moe_sort(expert_ids, num_experts: int, offsets, slot_of_row, row_of_slot, workspace=None, stream=None):
    """Rows of the tokens' choices sorted by expert (see ns.h).

    expert_ids: (tokens, top_k) int32 or int64 with contiguous choices; ids
    outside [0, num_experts) are dropped. offsets (num_experts + 1),
    slot_of_row (tokens * top_k) and row_of_slot (tokens, top_k): int32 outputs.
    Returns the workspace.
    """
    device = _on_gpu("expert_ids offsets slot_of_row row_of_slot workspace",
                     (expert_ids, offsets, slot_of_row, row_of_slot, workspace))
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be (tokens, top_k)")
    tokens, top_k = expert_ids.shape
    ld = _rows(expert_ids, "expert_ids", tokens, top_k, expert_ids.dtype)
    id_bytes = _int_bytes(expert_ids, "expert_ids")
    workspace = _workspace(workspace, lambda: ns_moe_sort_workspace_bytes(tokens, top_k, num_experts),
                           expert_ids.device, stream)
    _check(_c().ns_moe_sort(
        tokens, top_k, num_experts, expert_ids.data_ptr(), id_bytes, ld,
        _ints(offsets, "offsets", (num_experts + 1,)),
        _ints(slot_of_row, "slot_of_row", (tokens * top_k,)),
        _ints(row_of_slot, "row_of_slot", (tokens, top_k)), workspace.data_ptr(), workspace.numel(),
        _stream(stream, device)))
    return workspace


def _moe_sizes(tok, name: str, row_of_slot):
    """(tokens, top_k, hidden, dtype code, address of the map) of a call on token rows ``tok``."""
    if row_of_slot.dim() != 2:
        raise ValueError("row_of_slot must be (tokens, top_k)")
    if tok.dim() != 2:
        raise ValueError(f"{name} must be (tokens, hidden)")
    tokens, top_k = row_of_slot.shape
    return tokens, top_k, tok.shape[1], _code(tok, name), _ints(row_of_slot, "row_of_slot", row_of_slot.shape)


def ns_moe_dispatch(x, row_of_slot, xs, stream=None) -> None:
    """xs[row_of_slot[t, k]] = x[t] (see ns.h): x (tokens, hidden), xs (tokens * top_k, hidden), rows contiguous."""
    device = _on_gpu("x row_of_slot xs", (x, row_of_slot, xs))
    t, k, h, code, rows = _moe_sizes(x, "x", row_of_slot)
    _check(_c().ns_moe_dispatch(t, k, h, code, x.data_ptr(), _rows(x, "x", t, h, x.dtype), rows, xs.data_ptr(),
                                 _rows(xs, "xs", t * k, h, x.dtype), _stream(stream, device)))


def ns_moe_dispatch_backward(dxs, row_of_slot, dx, stream=None) -> None:
    """dx[t] = sum over k of dxs[row_of_slot[t, k]] (see ns.h)."""
    device = _on_gpu("dxs row_of_slot dx", (dxs, row_of_slot, dx))
    t, k, h, code, rows = _moe_sizes(dx, "dx", row_of_slot)
    _check(_c().ns_moe_dispatch_backward(t, k, h, code, dxs.data_ptr(), _rows(dxs, "dxs", t * k, h, dx.dtype), rows,
                                          dx.data_ptr(), _rows(dx, "dx", t, h, dx.dtype), _stream(stream, device)))


def ns_moe_combine(y, row_of_slot, weights, out, stream=None) -> None:
    """out[t] = sum over k of weights[t, k] * y[row_of_slot[t, k]] (see ns.h); weights (tokens, top_k) f32 or None."""
    device = _on_gpu("y row_of_slot weights out", (y, row_of_slot, weights, out))
    t, k, h, code, rows = _moe_sizes(out, "out", row_of_slot)
    _check(_c().ns_moe_combine(t, k, h, code, y.data_ptr(), _rows(y, "y", t * k, h, out.dtype), rows,
                                _floats(weights, "weights", (t, k)), out.data_ptr(),
                                _rows(out, "out", t, h, out.dtype), _stream(stream, device)))


def ns_moe_combine_backward(dout, y, row_of_slot, weights, dy, dweights, stream=None) -> None:
    """Gradient of ns_moe_combine (see ns.h): dy like y (or y itself), dweights (tokens, top_k) f32."""
    device = _on_gpu("dout y row_of_slot weights dy dweights", (dout, y, row_of_slot, weights, dy, dweights))
    t, k, h, code, rows = _moe_sizes(dout, "dout", row_of_slot)
    _check(_c().ns_moe_combine_backward(
        t, k, h, code, dout.data_ptr(), _rows(dout, "dout", t, h, dout.dtype), y.data_ptr(),
        _rows(y, "y", t * k, h, dout.dtype), rows, _floats(weights, "weights", (t, k)), dy.data_ptr(),
        _rows(dy, "dy", t * k, h, dout.dtype), _floats(dweights, "dweights", (t, k)),
        _stream(stream, device)))


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def _distill_args(logits, ids, teacher, teacher_lse, temperature):
    if logits.dim() != 2 or ids.dim() != 2:
        raise ValueError("logits must be (rows, vocab) and ids (rows, top_k)")
    rows, vocab = logits.shape
    top_k = ids.shape[1]
    ld = _rows(logits, "logits", rows, vocab, logits.dtype)
    if ids.shape[0] != rows or not ids.is_contiguous():
        raise ValueError(f"ids must be contiguous of shape ({rows}, top_k)")
    if teacher.shape != ids.shape or not teacher.is_contiguous():
        raise ValueError("teacher must be contiguous and shaped like ids")
    return (rows, vocab, top_k, _code(logits, "logits"), logits.data_ptr(), ld, ids.data_ptr(),
            _int_bytes(ids, "ids"), teacher.data_ptr(), _code(teacher, "teacher"),
            _floats(teacher_lse, "teacher_lse", (rows,)), float(temperature))


def ns_distill_workspace_bytes(rows: int, vocab: int, top_k: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ns_distill_workspace_bytes(rows, vocab, top_k, ctypes.byref(n)))
    return n.value


def ns_distill_topk(logits, ids, teacher, loss, lse, teacher_lse=None, rest_lse=None, temperature: float = 1.0,
                    grad_loss=None, dlogits=None, workspace=None, stream=None):
    """Loss against a teacher's top logits and, with grad_loss and dlogits, its
    gradient in the same pass (see ns.h).

    logits: (rows, vocab) with contiguous rows; ids (rows, top_k) int32 or int64;
    teacher (rows, top_k) bf16 or f32; loss, lse, rest_lse, teacher_lse,
    grad_loss: (rows,) f32. dlogits may be logits. Returns the workspace.
    """
    device = _on_gpu("logits ids teacher loss lse teacher_lse rest_lse grad_loss dlogits workspace",
                     (logits, ids, teacher, loss, lse, teacher_lse, rest_lse, grad_loss, dlogits, workspace))
    args = _distill_args(logits, ids, teacher, teacher_lse, temperature)
    rows, vocab, top_k = args[:3]
    if (dlogits is None) != (grad_loss is None):
        raise ValueError("dlogits and grad_loss go together")
    if (rest_lse is None) != (teacher_lse is None):
        raise ValueError("rest_lse and teacher_lse go together")
    workspace = _workspace(workspace, lambda: ns_distill_workspace_bytes(rows, vocab, top_k), logits.device, stream)
    one = (rows,)
    _check(_c().ns_distill_topk(
        *args, _floats(grad_loss, "grad_loss", one), _floats(loss, "loss", one),
        _floats(lse, "lse", one), _floats(rest_lse, "rest_lse", one),
        None if dlogits is None else dlogits.data_ptr(),
        0 if dlogits is None else _rows(dlogits, "dlogits", rows, vocab, logits.dtype), workspace.data_ptr(),
        workspace.numel(), _stream(stream, device)))
    return workspace


def ns_distill_topk_backward(logits, ids, teacher, lse, grad_loss, dlogits, teacher_lse=None, rest_lse=None,
                             temperature: float = 1.0, stream=None) -> None:
    """Gradient of ns_distill_topk by itself, from the lse (and rest_lse) it gave (see ns.h)."""
    device = _on_gpu("logits ids teacher lse grad_loss dlogits teacher_lse rest_lse",
                     (logits, ids, teacher, lse, grad_loss, dlogits, teacher_lse, rest_lse))
    args = _distill_args(logits, ids, teacher, teacher_lse, temperature)
    rows, vocab = args[:2]
    if (rest_lse is None) != (teacher_lse is None):
        raise ValueError("rest_lse and teacher_lse go together")
    one = (rows,)
    _check(_c().ns_distill_topk_backward(
        *args, _floats(lse, "lse", one), _floats(rest_lse, "rest_lse", one),
        _floats(grad_loss, "grad_loss", one), dlogits.data_ptr(),
        _rows(dlogits, "dlogits", rows, vocab, logits.dtype), _stream(stream, device)))
