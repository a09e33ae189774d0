"""Refusals of the training-step operators, checked on the host before anything is enqueued (no GPU needed).

Addresses here are numbers that are never read: every call is refused, or has
nothing to do.
"""

import ctypes

import pytest

import newton_schulz_quintic_amd as nsq
from newton_schulz_quintic_amd import _lib
from newton_schulz_quintic_amd._ops import ns_heads

OK, INVALID, OVERFLOW, WORKSPACE, DTYPE = 0, -1, -5, -7, -8
P = 1 << 20   # an address aligned to anything
BIG = 1 << 30


def _heads(data=P, b=1024, t=256, h=128, n=2):
    return ns_heads(data, b, t, h, n)


QK = dict(batch=2, seq=4, dim=128, dtype=0, q=_heads(), k=_heads(), qw=None, kw=None, wd=1, eps=1e-6, cos=P, sin=P,
          rows=16, rope=128, inter=0, pos=None, pb=4, ps=0, qo=_heads(), ko=_heads())
QK_BAD = [
    (dict(dtype=2), DTYPE), (dict(wd=7), DTYPE), (dict(batch=-1), INVALID), (dict(seq=-1), INVALID),
    (dict(batch=1 << 40, seq=1 << 40), OVERFLOW), (dict(batch=1 << 16, seq=1 << 16), OVERFLOW),
    (dict(dim=0), INVALID), (dict(dim=1025), INVALID), (dict(rope=3), INVALID), (dict(rope=130), INVALID),
    (dict(rope=-2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(inter=2), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(q=_heads(data=None)), INVALID), (dict(q=_heads(data=P + 1)), INVALID), (dict(q=_heads(n=-1)), INVALID),
    (dict(q=_heads(t=-1)), INVALID), (dict(q=_heads(b=1 << 62)), OVERFLOW), (dict(q=_heads(h=1 << 61)), OVERFLOW),
    (dict(q=_heads(n=BIG), qo=_heads(n=BIG)), OVERFLOW), (dict(cos=None), INVALID), (dict(sin=P + 2), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1 << 60), OVERFLOW), (dict(pos=P, pb=2), DTYPE), (dict(pos=P + 2), INVALID),
    (dict(pos=P, ps=-1), INVALID), (dict(qw=P + 1), INVALID), (dict(qo=_heads(n=3)), INVALID), (dict(ko=None), INVALID),
    (dict(qo=_heads(data=None)), INVALID), (dict(ko=_heads(data=P + 1)), INVALID),
]


def _ref(h):
    return None if h is None else ctypes.byref(h)


def _qk_forward(c):
    return _lib.lib().ns_qk_norm_rope(c["batch"], c["seq"], c["dim"], c["dtype"], _ref(c["q"]), _ref(c["k"]), c["qw"],
                                      c["kw"], c["wd"], c["eps"], c["cos"], c["sin"], c["rows"], c["rope"], c["inter"],
                                      c["pos"], c["pb"], c["ps"], _ref(c["qo"]), _ref(c["ko"]), None)


def _qk_backward(c, dqw=P, dkw=P, ws=P, nbytes=1 << 30, dq=_heads(), dk=_heads()):
    return _lib.lib().ns_qk_norm_rope_backward(
        c["batch"], c["seq"], c["dim"], c["dtype"], _ref(c["q"]), _ref(c["k"]), _ref(c["qo"]), _ref(c["ko"]), c["qw"],
        c["kw"], c["wd"], c["eps"], c["cos"], c["sin"], c["rows"], c["rope"], c["inter"], c["pos"], c["pb"], c["ps"],
        _ref(dq), _ref(dk), dqw, dkw, ws, nbytes, None)


@pytest.mark.parametrize("change,status", QK_BAD)
def test_qk_refusals(change, status):
    c = {**QK, **change}
    assert _qk_forward(c) == status and nsq.ns_last_error()
    assert _qk_backward(c) == status and nsq.ns_last_error()


def test_qk_backward_refusals_of_its_own():
    need = nsq.ns_qk_norm_rope_workspace_bytes(2, 4, 128)
    assert need > 0
    assert _qk_backward(QK, ws=None) == WORKSPACE
    assert _qk_backward(QK, nbytes=need - 1) == WORKSPACE
    assert _qk_backward(QK, ws=P + 16) == INVALID
    assert _qk_backward(QK, dqw=P + 2) == INVALID
    assert _qk_backward(QK, dq=_heads(n=1)) == INVALID
    assert _qk_backward(QK, dk=None) == INVALID


@pytest.mark.parametrize("short", [dict(b=0), dict(t=0), dict(h=0), dict(b=127), dict(t=127), dict(h=64)])
def test_qk_outputs_with_overlapping_heads(short):
    for name in ("qo", "ko"):
        assert _qk_forward({**QK, name: _heads(**short)}) == INVALID
    assert _qk_backward(QK, dq=_heads(**short)) == INVALID
    assert _qk_backward(QK, dk=_heads(**short)) == INVALID


def test_qk_nothing_to_do():
    none = _heads(data=None, n=0)
    assert _qk_forward({**QK, "batch": 0}) == OK
    assert _qk_forward({**QK, "q": none, "k": none, "qo": none, "ko": none}) == OK
    assert _qk_backward({**QK, "seq": 0}, dqw=None, dkw=None, ws=None, nbytes=0) == OK


def _moe(name, t=4, k=2, h=64, dtype=0, a=P, a_ld=64, m=P, w=P, b=P, b_ld=64, c=P, c_ld=64, d=P):
    lib = _lib.lib()
    if name == "dispatch":
        return lib.ns_moe_dispatch(t, k, h, dtype, a, a_ld, m, b, b_ld, None)
    if name == "dispatch_backward":
        return lib.ns_moe_dispatch_backward(t, k, h, dtype, a, a_ld, m, b, b_ld, None)
    if name == "combine":
        return lib.ns_moe_combine(t, k, h, dtype, a, a_ld, m, w, b, b_ld, None)
    return lib.ns_moe_combine_backward(t, k, h, dtype, a, a_ld, c, c_ld, m, w, b, b_ld, d, None)


@pytest.mark.parametrize("name", ["dispatch", "dispatch_backward", "combine", "combine_backward"])
def test_moe_row_refusals(name):
    for change, status in [
            (dict(t=-1), INVALID), (dict(k=0), INVALID), (dict(h=-1), INVALID), (dict(dtype=5), DTYPE),
            (dict(t=BIG, k=2), OVERFLOW), (dict(h=1 << 29, a_ld=1 << 29, b_ld=1 << 29, c_ld=1 << 29), OVERFLOW),
            (dict(a_ld=63), INVALID), (dict(b_ld=63), INVALID), (dict(a_ld=1 << 61), OVERFLOW), (dict(a=None), INVALID),
            (dict(b=None), INVALID), (dict(a=P + 1), INVALID), (dict(b=P + 1), INVALID), (dict(m=None), INVALID),
            (dict(m=P + 2), INVALID)]:
        assert _moe(name, **change) == status, change
        assert nsq.ns_last_error()
    assert _moe(name, t=0) == OK
    if name.startswith("dispatch") or name == "combine":
        assert _moe(name, h=0) == OK
    if name == "combine":
        assert _moe(name, w=P + 2) == INVALID
    if name == "combine_backward":
        for change in (dict(w=None), dict(d=None), dict(w=P + 2), dict(d=P + 1), dict(c=None), dict(c_ld=63)):
            assert _moe(name, **change) == INVALID, change


def test_moe_sort_refusals():
    def sort(t=4, k=2, e=8, ids=P, ib=4, ld=2, off=P, slot=P, row=P, ws=P, nbytes=1 << 30):
        return _lib.lib().ns_moe_sort(t, k, e, ids, ib, ld, off, slot, row, ws, nbytes, None)

    need = nsq.ns_moe_sort_workspace_bytes(4, 2, 8)
    for change, status in [
            (dict(t=-1), INVALID), (dict(k=0), INVALID), (dict(e=0), INVALID), (dict(e=1025), INVALID),
            (dict(t=BIG, k=2), OVERFLOW), (dict(ib=2), DTYPE), (dict(ld=1), INVALID), (dict(ld=1 << 62), OVERFLOW),
            (dict(ids=None), INVALID), (dict(off=None), INVALID), (dict(slot=None), INVALID), (dict(row=None), INVALID),
            (dict(ids=P + 4, ib=8), INVALID), (dict(off=P + 2), INVALID), (dict(slot=P + 1), INVALID),
            (dict(ws=None), WORKSPACE), (dict(nbytes=need - 1), WORKSPACE), (dict(ws=P + 8), INVALID)]:
        assert sort(**change) == status, change


def _distill(backward=False, rows=4, v=100, k=3, dtype=0, z=P, ld=100, ids=P, ib=4, t=P, td=1, tl=None, tau=1.0, g=P,
             loss=P, lse=P, rest=None, d=P, dld=100, ws=P, nbytes=1 << 30):
    lib = _lib.lib()
    if backward:
        return lib.ns_distill_topk_backward(rows, v, k, dtype, z, ld, ids, ib, t, td, tl, tau, lse, rest, g, d, dld, None)
    return lib.ns_distill_topk(rows, v, k, dtype, z, ld, ids, ib, t, td, tl, tau, g, loss, lse, rest, d, dld, ws, nbytes,
                               None)


@pytest.mark.parametrize("backward", [False, True])
def test_distill_refusals(backward):
    for change, status in [
            (dict(rows=-1), INVALID), (dict(rows=(1 << 24) + 1), INVALID), (dict(v=0), INVALID),
            (dict(v=(1 << 24) + 1, ld=1 << 25, dld=1 << 25), INVALID), (dict(k=0), INVALID), (dict(k=1025), INVALID),
            (dict(dtype=3), DTYPE), (dict(td=3), DTYPE), (dict(ib=1), DTYPE), (dict(ld=99), INVALID),
            (dict(dld=99), INVALID), (dict(ld=1 << 61), OVERFLOW), (dict(dld=1 << 61), OVERFLOW), (dict(tau=0.0), INVALID),
            (dict(tau=-1.0), INVALID), (dict(tau=float("nan")), INVALID), (dict(tau=float("inf")), INVALID),
            (dict(tau=1e-38), INVALID), (dict(z=None), INVALID), (dict(ids=None), INVALID), (dict(t=None), INVALID),
            (dict(z=P + 1), INVALID), (dict(d=P + 1), INVALID), (dict(ids=P + 2), INVALID), (dict(ids=P + 4, ib=8), INVALID),
            (dict(t=P + 2), INVALID), (dict(tl=P + 2, rest=P), INVALID), (dict(g=P + 2), INVALID), (dict(lse=None), INVALID),
            (dict(lse=P + 2), INVALID), (dict(tl=P), INVALID), (dict(tl=P, rest=P + 1), INVALID), (dict(g=None), INVALID),
            (dict(d=None), INVALID), (dict(d=P, ld=128), INVALID)]:
        assert _distill(backward, **change) == status, change
        assert nsq.ns_last_error()
    assert _distill(backward, rows=0) == OK


def test_distill_workspace():
    need = nsq.ns_distill_workspace_bytes(4, 100, 3)
    assert need > 0
    assert _distill(ws=None) == WORKSPACE and _distill(nbytes=need - 1) == WORKSPACE and _distill(ws=P + 8) == INVALID
    assert _distill(loss=None) == INVALID
    for bad in ((-1, 100, 3), (4, 0, 3), (4, 100, 0)):
        with pytest.raises(nsq.NSError) as e:
            nsq.ns_distill_workspace_bytes(*bad)
        assert e.value.name == "NS_ERR_INVALID_ARG"


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    x = torch.zeros(1, 2, 2, 4)
    with pytest.raises(ValueError, match="q is on cpu"):
        nsq.ns_qk_norm_rope(x, x, x, x)
    m = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on the current GPU"):
        nsq.ns_moe_sort(m, 4, m, m, m)
    with pytest.raises(ValueError, match="not on the current GPU"):
        nsq.ns_moe_combine(x[0, 0], m, None, x[0, 0])
    with pytest.raises(ValueError, match="not on the current GPU"):
        nsq.ns_distill_topk(x[0, 0], m, x[0, 0], x, x)
