"""Refusals of the operators around a block's products, checked on the host before anything is enqueued (no GPU needed).

Addresses here are numbers that are never read: every call is refused, or has
nothing to do.
"""

import ctypes

import pytest

import newton_schulz_quintic_amd as nsq
from newton_schulz_quintic_amd import _lib
from newton_schulz_quintic_amd._ops import ns_rows

OK, INVALID, OVERFLOW, WORKSPACE, DTYPE = 0, -1, -5, -7, -8
P = 1 << 20   # an address aligned to anything
NAN, INF = float("nan"), float("inf")


def _rows(data=P, ld=64):
    return ns_rows(data, ld)


def _ref(h):
    return None if h is None else ctypes.byref(h)


BLOCK = dict(rows=4, hidden=64, rd=0, dtype=0, x=_rows(), y=_rows(), wp=P, wn=P, wd=1, post=1, gate=_rows(), gates=2, gd=0,
             alpha=1.0, scale=1.0, eps=1e-6, xo=_rows(), h=_rows())
BLOCK_BAD = [
    (dict(rd=2), DTYPE), (dict(dtype=3), DTYPE), (dict(dtype=1), DTYPE), (dict(wd=4), DTYPE), (dict(gd=2), DTYPE),
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(hidden=0), INVALID), (dict(hidden=16385), INVALID),
    (dict(post=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(alpha=NAN), INVALID), (dict(scale=INF), INVALID), (dict(x=None), INVALID), (dict(x=_rows(data=None)), INVALID),
    (dict(x=_rows(data=P + 1)), INVALID), (dict(y=_rows(data=P + 1)), INVALID), (dict(x=_rows(ld=63)), INVALID),
    (dict(y=_rows(ld=63)), INVALID), (dict(xo=_rows(ld=63)), INVALID), (dict(h=_rows(ld=-64)), INVALID),
    (dict(gate=_rows(ld=3)), INVALID), (dict(gates=3), INVALID), (dict(gates=0), INVALID), (dict(gates=-2), INVALID),
    (dict(x=_rows(ld=1 << 61)), OVERFLOW), (dict(h=_rows(ld=1 << 61)), OVERFLOW), (dict(wp=P + 2), INVALID),
    (dict(wn=P + 1), INVALID), (dict(post=0), INVALID), (dict(y=None), INVALID), (dict(xo=None, h=None), INVALID),
    (dict(gate=_rows(data=P + 1)), INVALID),
]


def _forward(c):
    return _lib.lib().ns_block_norm(c["rows"], c["hidden"], c["rd"], c["dtype"], _ref(c["x"]), _ref(c["y"]), c["wp"], c["wn"],
                                    c["wd"], c["post"], _ref(c["gate"]), c["gates"], c["gd"], c["alpha"], c["scale"],
                                    c["eps"], _ref(c["xo"]), _ref(c["h"]), None)


def _backward(c, dx=_rows(), dy=_rows(), dwp=P, dwn=P, dg=_rows(), ws=P, nbytes=1 << 30):
    return _lib.lib().ns_block_norm_backward(
        c["rows"], c["hidden"], c["rd"], c["dtype"], _ref(c["x"]), _ref(c["y"]), c["wp"], c["wn"], c["wd"], c["post"],
        _ref(c["gate"]), c["gates"], c["gd"], c["alpha"], c["scale"], c["eps"], _ref(c["xo"]), _ref(c["h"]), _ref(dx),
        _ref(dy), dwp, dwn, _ref(dg), ws, nbytes, None)


@pytest.mark.parametrize("change,status", BLOCK_BAD)
def test_block_norm_refusals(change, status):
    c = {**BLOCK, **change}
    assert _forward(c) == status
    assert nsq.ns_last_error()
    assert _backward(c) == status


def test_block_norm_needs_y():
    no_y = dict(y=None, gate=None, wp=None)
    assert _forward({**BLOCK, **no_y}) == INVALID                                    # x_out without y
    assert _backward({**BLOCK, **no_y, "xo": None}) == INVALID                       # dy without y
    assert _backward({**BLOCK, **no_y, "xo": None}, dy=None) == INVALID              # dpost_weight without y
    assert _backward({**BLOCK, **no_y, "xo": None}, dy=None, dwp=None) == INVALID    # dgate without gate
    assert _backward({**BLOCK, "post": 0, "wp": None}) == INVALID                    # dpost_weight without post_norm


def test_block_norm_backward_refusals():
    need = nsq.ns_block_norm_workspace_bytes(4, 64)
    assert need > 0
    for kw, status in [(dict(ws=None), WORKSPACE), (dict(nbytes=need - 1), WORKSPACE), (dict(ws=P + 8), INVALID),
                       (dict(dx=_rows(data=P + 1)), INVALID), (dict(dy=_rows(ld=60)), INVALID), (dict(dwp=P + 2), INVALID),
                       (dict(dwn=P + 1), INVALID), (dict(dg=_rows(ld=60)), INVALID)]:
        assert _backward(BLOCK, **kw) == status, kw
    for bad in ((-1, 64), (4, 0), (4, 16385), (1 << 31, 64)):
        with pytest.raises(nsq.NSError) as e:
            nsq.ns_block_norm_workspace_bytes(*bad)
        assert e.value.name == "NS_ERR_INVALID_ARG"


def test_block_norm_without_rows():
    none = _rows(data=None)
    c = {**BLOCK, "rows": 0, "x": none, "y": none, "xo": none, "h": none, "gate": none, "gates": 0}
    assert _forward(c) == OK
    assert _backward(c, dx=none, dy=none, dwp=None, dwn=None, dg=None, ws=None, nbytes=0) == OK
    assert _forward({**c, "gates": 1 << 20}) == INVALID


QUANT = dict(batch=1, rows=4, cols=200, dtype=0, x=P, ld=200, xb=0, tall=1, off=None, groups=0, q=P, qld=256, qb=0, s=P, qt=P,
             tld=128, tb=0, st=P)


def _quantize(c):
    return _lib.lib().ns_quantize(c["batch"], c["rows"], c["cols"], c["dtype"], c["x"], c["ld"], c["xb"], c["tall"], c["off"],
                                  c["groups"], c["q"], c["qld"], c["qb"], c["s"], c["qt"], c["tld"], c["tb"], c["st"], None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), DTYPE), (dict(batch=-1), INVALID), (dict(batch=65536, tall=128), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=(1 << 30) + 1), INVALID), (dict(cols=0), INVALID), (dict(cols=(1 << 22) + 1), INVALID), (dict(tall=64), INVALID),
    (dict(batch=2), INVALID), (dict(s=None), INVALID), (dict(q=None), INVALID), (dict(qt=None), INVALID),
    (dict(q=None, s=None, qt=None, st=None), INVALID), (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(ld=-1), INVALID),
    (dict(ld=1 << 61), OVERFLOW), (dict(q=P + 8), INVALID), (dict(qld=255), INVALID), (dict(qld=264), INVALID),
    (dict(qld=240), INVALID), (dict(qld=(1 << 22) + 16), INVALID), (dict(qt=P + 4), INVALID), (dict(tld=112), INVALID),
    (dict(off=P, groups=0), INVALID), (dict(off=P, groups=1025), INVALID), (dict(off=P + 2, groups=3, tld=384), INVALID),
    (dict(off=P, groups=3, tld=256), INVALID), (dict(off=P, groups=1, tall=128), INVALID),
    (dict(batch=2, tall=128, xb=800, qb=1000), INVALID), (dict(batch=2, tall=128, xb=-8), INVALID),
    (dict(rows=128 * 65536, tld=1 << 22), INVALID)])
def test_quantize_refusals(change, status):
    assert _quantize({**QUANT, **change}) == status, change
    assert nsq.ns_last_error()


def test_quantize_nothing_to_do():
    assert _quantize({**QUANT, "rows": 0, "x": None}) == OK
    assert _quantize({**QUANT, "batch": 0, "tall": 128}) == OK
    assert _quantize({**QUANT, "rows": 128 * 65536, "tall": 128, "qt": None, "st": None}) == OVERFLOW


MAT = dict(m=4, n=8, k=256, a=P, lda=256, sa=P, b=P, ldb=256, bb=0, sb=P, tall=128, off=None, groups=0, reduce=0, rows=0, od=0,
           out=P, ldo=8, ob=0, ws=None, nbytes=0)


def _matmul(c):
    return _lib.lib().ns_scaled_matmul(c["m"], c["n"], c["k"], c["a"], c["lda"], c["sa"], c["b"], c["ldb"], c["bb"], c["sb"],
                                       c["tall"], c["off"], c["groups"], c["reduce"], c["rows"], c["od"], c["out"], c["ldo"],
                                       c["ob"], c["ws"], c["nbytes"], None)


@pytest.mark.parametrize("change,status", [
    (dict(od=2), DTYPE), (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-128), INVALID), (dict(k=200), INVALID),
    (dict(k=(1 << 22) + 128), INVALID), (dict(m=(1 << 30) + 1), INVALID), (dict(tall=2), INVALID), (dict(reduce=2), INVALID),
    (dict(reduce=1), INVALID), (dict(off=P), INVALID), (dict(groups=2), INVALID), (dict(off=P + 2, groups=2), INVALID),
    (dict(groups=-1), INVALID), (dict(off=P, groups=1025), INVALID), (dict(out=None), INVALID), (dict(out=P + 1), INVALID),
    (dict(ldo=7), INVALID), (dict(ldo=1 << 62), INVALID), (dict(a=None), INVALID), (dict(a=P + 8), INVALID),
    (dict(b=P + 1), INVALID), (dict(lda=255), INVALID), (dict(ldb=250), INVALID), (dict(lda=(1 << 22) + 16), INVALID),
    (dict(sa=None), INVALID), (dict(sb=None), INVALID), (dict(off=P, groups=2, bb=1000), INVALID), (dict(ws=P + 8, nbytes=1 << 20), INVALID),
    (dict(off=P, groups=2, reduce=1, rows=-1), INVALID), (dict(off=P, groups=2, reduce=1, rows=1000), INVALID)])
def test_scaled_matmul_refusals(change, status):
    assert _matmul({**MAT, **change}) == status, change
    assert nsq.ns_last_error()


def test_scaled_matmul_nothing_to_do_and_workspace():
    assert _matmul({**MAT, "m": 0}) == OK and _matmul({**MAT, "n": 0}) == OK
    need = nsq.ns_scaled_matmul_workspace_bytes(100, 100, 8192)
    assert need > 0 and nsq.ns_scaled_matmul_workspace_bytes(16, 100, 8192) == 0
    c = {**MAT, "m": 100, "n": 100, "k": 8192, "lda": 8192, "ldb": 8192, "ldo": 100}
    assert _matmul(c) == WORKSPACE and _matmul({**c, "ws": P, "nbytes": need - 1}) == WORKSPACE
    for bad in ((-1, 4, 128), (4, 4, 100), (4, 4, 128, 1025)):
        with pytest.raises(nsq.NSError) as e:
            nsq.ns_scaled_matmul_workspace_bytes(*bad)
        assert e.value.name == "NS_ERR_INVALID_ARG"


def _array(kind, *values):
    return (kind * len(values))(*values)


def _list(n=2, counts=(3, 5), grads=(P, P), dtypes=(0, 1), outs=(P + 4096, P + 8192), out_dtypes=(0, 1), momenta=None, norm=P,
          max_norm=1.0, eps=1e-6, beta=0.0, ws=P, nbytes=1 << 20, only_norm=False, sum_sq=None):
    counts, grads, dtypes = _array(ctypes.c_int64, *counts), _array(ctypes.c_void_p, *grads), _array(ctypes.c_int32, *dtypes)
    if only_norm:
        return _lib.lib().ns_grad_norm(n, counts, grads, dtypes, norm, sum_sq, ws, nbytes, None)
    outs = _array(ctypes.c_void_p, *outs) if outs else None
    out_dtypes = _array(ctypes.c_int32, *out_dtypes) if out_dtypes else None
    momenta = _array(ctypes.c_void_p, *momenta) if momenta else None
    return _lib.lib().ns_grad_clip(n, counts, grads, dtypes, momenta, outs, out_dtypes, norm, max_norm, eps, beta, ws, nbytes,
                                   None)


LIST_BAD = [(dict(n=-1), INVALID), (dict(n=(1 << 20) + 1), INVALID), (dict(counts=(3, -1)), INVALID),
            (dict(counts=(3, 1 << 42)), OVERFLOW), (dict(counts=(1 << 41, 1 << 41)), OVERFLOW), (dict(dtypes=(0, 2)), DTYPE),
            (dict(grads=(P, None)), INVALID), (dict(grads=(P + 1, P)), INVALID), (dict(grads=(P, P + 2)), INVALID),
            (dict(ws=None), WORKSPACE), (dict(nbytes=64), WORKSPACE), (dict(ws=P + 8), INVALID), (dict(norm=P + 2), INVALID)]


@pytest.mark.parametrize("change,status", LIST_BAD)
def test_gradient_list_refusals(change, status):
    assert _list(**change) == status and nsq.ns_last_error()
    assert _list(only_norm=True, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(outs=None), INVALID), (dict(out_dtypes=None), INVALID), (dict(out_dtypes=(0, 3)), DTYPE), (dict(outs=(P + 1, P)), INVALID),
    (dict(outs=(P + 4096, None)), INVALID), (dict(beta=0.9), INVALID), (dict(beta=NAN), INVALID), (dict(beta=INF), INVALID),
    (dict(beta=0.9, momenta=(P, P + 2)), INVALID), (dict(beta=0.9, momenta=(P, None)), INVALID), (dict(max_norm=-1.0), INVALID),
    (dict(max_norm=NAN), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=INF), INVALID),
    (dict(outs=(P, P + 8192), out_dtypes=(1, 1)), INVALID)])
def test_grad_clip_refusals(change, status):
    assert _list(**change) == status, change
    assert nsq.ns_last_error()


def test_gradient_list_workspace_and_empty_list():
    assert _list(n=0, ws=None, nbytes=0) == OK
    assert _list(only_norm=True, norm=None) == INVALID and _list(only_norm=True, norm=None, sum_sq=P + 4) == INVALID
    assert nsq.ns_grad_workspace_bytes(97) > nsq.ns_grad_workspace_bytes(96) == nsq.ns_grad_workspace_bytes(0)
    for bad in (-1, (1 << 20) + 1):
        with pytest.raises(nsq.NSError) as e:
            nsq.ns_grad_workspace_bytes(bad)
        assert e.value.name == "NS_ERR_INVALID_ARG"


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8)
    for call in (lambda: nsq.ns_block_norm(x, x, x, x), lambda: nsq.ns_block_norm_backward(x, x, x, x, x, x),
                 lambda: nsq.ns_quantize(x, q, s), lambda: nsq.ns_scaled_matmul(q, s, q, s, x),
                 lambda: nsq.ns_grad_norm([x], torch.zeros(1)), lambda: nsq.ns_grad_clip([x], [x])):
        with pytest.raises(ValueError, match="not on the current GPU"):
            call()
    with pytest.raises(TypeError, match="list of tensors"):
        nsq.ns_grad_clip(3, [])
    with pytest.raises(TypeError, match="must hold tensors"):
        nsq.ns_grad_clip([3], [])
