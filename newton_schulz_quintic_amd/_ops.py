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

from ._lib import NS_BF16, NS_F32, _check, _new_workspace, _stream, lib


class ns_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


_codes = None


def _code(t, name: str) -> int:
    """The ns_dtype of a float tensor."""
    global _codes
    if _codes is None:
        import torch
        _codes = {torch.bfloat16: NS_BF16, torch.float32: NS_F32}
    try:
        return _codes[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}") from None


def _int_bytes(t, name: str) -> int:
    import torch
    if t.dtype == torch.int32:
        return 4
    if t.dtype == torch.int64:
        return 8
    raise TypeError(f"{name} must be int32 or int64, not {t.dtype}")


def _on_gpu(**tensors) -> None:
    import torch
    here = None
    for name, t in tensors.items():
        if t is None:
            continue
        at = t.get_device()
        if here is None and at >= 0:
            here = torch.cuda.current_device()
        if at != here:
            raise ValueError(f"{name} is on {t.device}, not on the current GPU")


def _array(t, name: str, shape, dtype: str):
    """Checks a contiguous tensor of one shape and of a dtype named as in torch; returns its address."""
    import torch
    if t is None:
        return None
    if t.dtype != getattr(torch, dtype):
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and of shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t, name: str, rows: int, cols: int, dtype) -> int:
    """Checks a (rows, cols) tensor whose rows are contiguous; returns its row stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must have shape ({rows}, {cols}), not {tuple(t.shape)}")
    if cols > 1 and rows and t.stride(1) != 1:
        raise ValueError(f"each row of {name} must be contiguous")
    return t.stride(0) if rows > 1 else max(cols, 1)


def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace, or a new one of ``nbytes()`` (the library checks the size of a given one)."""
    if workspace is None:
        return _new_workspace(nbytes(), device, stream)
    import torch
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    return workspace


# ---------------------------------------------------------------------------
# queries and keys
# ---------------------------------------------------------------------------

def _heads(t, name: str, like=None) -> ns_heads:
    """A (batch, seq, heads, head_dim) or (seq, heads, head_dim) tensor with contiguous heads."""
    if t.dim() not in (3, 4):
        raise ValueError(f"{name} must be (batch, seq, heads, head_dim) or (seq, heads, head_dim)")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name} must have the shape and dtype of its input: {tuple(like.shape)}, {like.dtype}")
    st = t.stride()
    if t.shape[-1] > 1 and st[-1] != 1 and t.numel():
        raise ValueError(f"each head of {name} must be contiguous")
    return ns_heads(t.data_ptr(), st[0] if t.dim() == 4 else 0, st[-3], st[-2], t.shape[-2])


def _norm_rope_args(q, k, q_weight, k_weight, cos, sin, pos, eps, interleaved):
    """The arguments that the two calls share, up to the positions."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k is required")
    shape = first.shape
    dtype = _code(first, "q" if q is not None else "k")
    none = ns_heads(None, 0, 0, 0, 0)
    hq = none if q is None else _heads(q, "q")
    hk = none if k is None else _heads(k, "k")
    if q is not None and k is not None and (q.dtype != k.dtype or q.dim() != k.dim() or q.shape[:-2] != k.shape[:-2]
                                            or q.shape[-1] != k.shape[-1]):
        raise ValueError("q and k must share dtype, batch, seq and head_dim")
    batch, seq = (shape[0], shape[1]) if len(shape) == 4 else (1, shape[0])
    dim = shape[-1]
    w_code = NS_F32
    weights = [w for w in (q_weight, k_weight) if w is not None]
    if weights:
        w_code = _code(weights[0], "weights")
        for w in weights:
            if w.dtype != weights[0].dtype or w.shape != (dim,) or not w.is_contiguous():
                raise ValueError(f"weights must share one dtype and be contiguous of shape ({dim},)")
    rows = rope = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be (positions, rope_dim / 2)")
        _array(cos, "cos", cos.shape, "float32")
        _array(sin, "sin", cos.shape, "float32")
        rows, rope = cos.shape[0], 2 * cos.shape[1]
    pos_ptr, pos_bytes, pos_stride = None, 4, 0
    if pos is not None:
        pos_bytes = _int_bytes(pos, "pos")
        if not pos.is_contiguous() or tuple(pos.shape) not in ((seq,), (batch, seq)):
            raise ValueError(f"pos must be contiguous of shape ({seq},) or ({batch}, {seq})")
        pos_ptr, pos_stride = pos.data_ptr(), seq if pos.dim() == 2 else 0
    head = (batch, seq, dim, dtype, ctypes.byref(hq), ctypes.byref(hk))
    tail = (None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
            w_code, eps, None if cos is None else cos.data_ptr(), None if sin is None else sin.data_ptr(), rows, rope,
            1 if interleaved else 0, pos_ptr, pos_bytes, pos_stride)
    return head, tail, none


def _pair(a, b, q, k, names, none):
    """The head arguments of two tensors that go with q and k."""
    for x, of, name in ((a, q, names[0]), (b, k, names[1])):
        if (x is None) != (of is None):
            raise ValueError(f"{name} goes with its input: give both or neither")
    return (none if a is None else _heads(a, names[0], q)), (none if b is None else _heads(b, names[1], k))


def ns_qk_norm_rope(q, k, q_out, k_out, q_weight=None, k_weight=None, cos=None, sin=None, pos=None,
                    eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """RMS norm of each head of q and k, its weight and the position rotation (see ns.h).

    q, k: (batch, seq, heads, head_dim) or (seq, heads, head_dim) views with
    contiguous heads, bf16 or f32; k (or q) and its output may be None. cos, sin:
    (positions, rope_dim / 2) f32, or None for no rotation. pos: (seq,) or
    (batch, seq) int32 or int64, or None for 0, 1, ... Outputs may be the inputs.
    """
    _on_gpu(q=q, k=k, q_out=q_out, k_out=k_out, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin, pos=pos)
    head, tail, none = _norm_rope_args(q, k, q_weight, k_weight, cos, sin, pos, eps, interleaved)
    oq, ok = _pair(q_out, k_out, q, k, ("q_out", "k_out"), none)
    _check(lib().ns_qk_norm_rope(*head, *tail, ctypes.byref(oq), ctypes.byref(ok), _stream(stream)))


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
    _on_gpu(q=q, k=k, dq_out=dq_out, dk_out=dk_out, dq=dq, dk=dk, dq_weight=dq_weight, dk_weight=dk_weight,
            q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin, pos=pos, workspace=workspace)
    head, tail, none = _norm_rope_args(q, k, q_weight, k_weight, cos, sin, pos, eps, interleaved)
    gq, gk = _pair(dq_out, dk_out, q, k, ("dq_out", "dk_out"), none)
    oq, ok = _pair(dq, dk, q, k, ("dq", "dk"), none)
    dim = head[2]
    wq, wk = _array(dq_weight, "dq_weight", (dim,), "float32"), _array(dk_weight, "dk_weight", (dim,), "float32")
    if wq or wk:
        workspace = _workspace(workspace, lambda: ns_qk_norm_rope_workspace_bytes(*head[:3]),
                               (q if q is not None else k).device, stream)
    _check(lib().ns_qk_norm_rope_backward(
        *head, ctypes.byref(gq), ctypes.byref(gk), *tail, ctypes.byref(oq), ctypes.byref(ok), wq, wk,
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
        _stream(stream)))
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
    _on_gpu(expert_ids=expert_ids, offsets=offsets, slot_of_row=slot_of_row, row_of_slot=row_of_slot,
            workspace=workspace)
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be (tokens, top_k)")
    tokens, top_k = expert_ids.shape
    ld = _rows(expert_ids, "expert_ids", tokens, top_k, expert_ids.dtype)
    id_bytes = _int_bytes(expert_ids, "expert_ids")
    workspace = _workspace(workspace, lambda: ns_moe_sort_workspace_bytes(tokens, top_k, num_experts),
                           expert_ids.device, stream)
    _check(lib().ns_moe_sort(
        tokens, top_k, num_experts, expert_ids.data_ptr(), id_bytes, ld,
        _array(offsets, "offsets", (num_experts + 1,), "int32"),
        _array(slot_of_row, "slot_of_row", (tokens * top_k,), "int32"),
        _array(row_of_slot, "row_of_slot", (tokens, top_k), "int32"), workspace.data_ptr(), workspace.numel(),
        _stream(stream)))
    return workspace


def _moe_sizes(tok, name: str, row_of_slot):
    """(tokens, top_k, hidden, dtype code, address of the map) of a call on token rows ``tok``."""
    if row_of_slot.dim() != 2:
        raise ValueError("row_of_slot must be (tokens, top_k)")
    if tok.dim() != 2:
        raise ValueError(f"{name} must be (tokens, hidden)")
    tokens, top_k = row_of_slot.shape
    return tokens, top_k, tok.shape[1], _code(tok, name), _array(row_of_slot, "row_of_slot", row_of_slot.shape, "int32")


def ns_moe_dispatch(x, row_of_slot, xs, stream=None) -> None:
    """xs[row_of_slot[t, k]] = x[t] (see ns.h): x (tokens, hidden), xs (tokens * top_k, hidden), rows contiguous."""
    _on_gpu(x=x, row_of_slot=row_of_slot, xs=xs)
    t, k, h, code, rows = _moe_sizes(x, "x", row_of_slot)
    _check(lib().ns_moe_dispatch(t, k, h, code, x.data_ptr(), _rows(x, "x", t, h, x.dtype), rows, xs.data_ptr(),
                                 _rows(xs, "xs", t * k, h, x.dtype), _stream(stream)))


def ns_moe_dispatch_backward(dxs, row_of_slot, dx, stream=None) -> None:
    """dx[t] = sum over k of dxs[row_of_slot[t, k]] (see ns.h)."""
    _on_gpu(dxs=dxs, row_of_slot=row_of_slot, dx=dx)
    t, k, h, code, rows = _moe_sizes(dx, "dx", row_of_slot)
    _check(lib().ns_moe_dispatch_backward(t, k, h, code, dxs.data_ptr(), _rows(dxs, "dxs", t * k, h, dx.dtype), rows,
                                          dx.data_ptr(), _rows(dx, "dx", t, h, dx.dtype), _stream(stream)))


def ns_moe_combine(y, row_of_slot, weights, out, stream=None) -> None:
    """out[t] = sum over k of weights[t, k] * y[row_of_slot[t, k]] (see ns.h); weights (tokens, top_k) f32 or None."""
    _on_gpu(y=y, row_of_slot=row_of_slot, weights=weights, out=out)
    t, k, h, code, rows = _moe_sizes(out, "out", row_of_slot)
    _check(lib().ns_moe_combine(t, k, h, code, y.data_ptr(), _rows(y, "y", t * k, h, out.dtype), rows,
                                _array(weights, "weights", (t, k), "float32"), out.data_ptr(),
                                _rows(out, "out", t, h, out.dtype), _stream(stream)))


def ns_moe_combine_backward(dout, y, row_of_slot, weights, dy, dweights, stream=None) -> None:
    """Gradient of ns_moe_combine (see ns.h): dy like y (or y itself), dweights (tokens, top_k) f32."""
    _on_gpu(dout=dout, y=y, row_of_slot=row_of_slot, weights=weights, dy=dy, dweights=dweights)
    t, k, h, code, rows = _moe_sizes(dout, "dout", row_of_slot)
    _check(lib().ns_moe_combine_backward(
        t, k, h, code, dout.data_ptr(), _rows(dout, "dout", t, h, dout.dtype), y.data_ptr(),
        _rows(y, "y", t * k, h, dout.dtype), rows, _array(weights, "weights", (t, k), "float32"), dy.data_ptr(),
        _rows(dy, "dy", t * k, h, dout.dtype), _array(dweights, "dweights", (t, k), "float32"), _stream(stream)))


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
            _array(teacher_lse, "teacher_lse", (rows,), "float32"), float(temperature))


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
    _on_gpu(logits=logits, ids=ids, teacher=teacher, loss=loss, lse=lse, teacher_lse=teacher_lse, rest_lse=rest_lse,
            grad_loss=grad_loss, dlogits=dlogits, workspace=workspace)
    args = _distill_args(logits, ids, teacher, teacher_lse, temperature)
    rows, vocab, top_k = args[:3]
    if (dlogits is None) != (grad_loss is None):
        raise ValueError("dlogits and grad_loss go together")
    if (rest_lse is None) != (teacher_lse is None):
        raise ValueError("rest_lse and teacher_lse go together")
    workspace = _workspace(workspace, lambda: ns_distill_workspace_bytes(rows, vocab, top_k), logits.device, stream)
    one = (rows,)
    _check(lib().ns_distill_topk(
        *args, _array(grad_loss, "grad_loss", one, "float32"), _array(loss, "loss", one, "float32"),
        _array(lse, "lse", one, "float32"), _array(rest_lse, "rest_lse", one, "float32"),
        None if dlogits is None else dlogits.data_ptr(),
        0 if dlogits is None else _rows(dlogits, "dlogits", rows, vocab, logits.dtype), workspace.data_ptr(),
        workspace.numel(), _stream(stream)))
    return workspace


def ns_distill_topk_backward(logits, ids, teacher, lse, grad_loss, dlogits, teacher_lse=None, rest_lse=None,
                             temperature: float = 1.0, stream=None) -> None:
    """Gradient of ns_distill_topk by itself, from the lse (and rest_lse) it gave (see ns.h)."""
    _on_gpu(logits=logits, ids=ids, teacher=teacher, lse=lse, grad_loss=grad_loss, dlogits=dlogits,
            teacher_lse=teacher_lse, rest_lse=rest_lse)
    args = _distill_args(logits, ids, teacher, teacher_lse, temperature)
    rows, vocab = args[:2]
    if (rest_lse is None) != (teacher_lse is None):
        raise ValueError("rest_lse and teacher_lse go together")
    one = (rows,)
    _check(lib().ns_distill_topk_backward(
        *args, _array(lse, "lse", one, "float32"), _array(rest_lse, "rest_lse", one, "float32"),
        _array(grad_loss, "grad_loss", one, "float32"), dlogits.data_ptr(),
        _rows(dlogits, "dlogits", rows, vocab, logits.dtype), _stream(stream)))
