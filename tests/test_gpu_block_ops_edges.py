"""Operators around a block's products: calls at the edge of what their documentation allows."""

import ctypes

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from newton_schulz_quintic_amd import _lib
from newton_schulz_quintic_amd._ops import ns_rows
from oracle import block_ops as ops
from tests.helpers import log
from tests.test_gpu_scaled import _beside, _bytes, _check, _new8, _offsets, _operand, _out, _same, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
def test_block_norm_backward_without_rows_and_gate(given):
    """No rows, and a gate that is left out by a NULL address, with or without a struct: the sums are zeros."""
    import torch
    log(f"block no rows, no gate {given}")
    none = ctypes.byref(ns_rows(None, 64))
    wp, dwp, dwn = torch.full((64,), 2.0, device="cuda"), torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    status = _lib.lib().ns_block_norm_backward(0, 64, 0, 0, none, none, wp.data_ptr(), None, 1, 1, none if given else None, 1, 0,
                                               1.0, 1.0, 1e-6, none, none, none, none, dwp.data_ptr(), dwn.data_ptr(), none, None,
                                               0, torch.cuda.current_stream().cuda_stream)
    assert status == 0, nsq.ns_last_error()
    torch.cuda.synchronize()
    assert not dwp.any() and not dwn.any()


def test_outputs_that_overlap_are_refused():
    """A batch or groups whose matrices share memory; matrices between each other's rows do not."""
    import torch
    log("overlapping outputs")
    x = torch.zeros(3, 150, 200, device="cuda")
    q, s, qt, st = _new8(3, 150, 256), _bytes(3, 2, 2), _new8(3, 200, 256), _bytes(3, 2, 2)
    off, k = _offsets([0, 2, 4]), 256
    a, sa, b, sb = _new8(4, k), _bytes(4, 2), _new8(8, k), _bytes(8, 2)
    for bad in (lambda: nsq.ns_quantize(x, q[:1].expand(3, 150, 256), s, block_rows=128),
                lambda: nsq.ns_quantize(x, None, None, qt[:1].expand(3, 200, 256), st, block_rows=128),
                lambda: nsq.ns_scaled_matmul(a, sa, b, sb, torch.empty(4, 8, device="cuda").expand(2, 4, 8), offsets=off, reduce=True)):
        with pytest.raises(nsq.NSError, match="overlap"):
            bad()


def test_outputs_between_each_others_rows():
    import torch
    log("interleaved outputs")
    x, x64 = _values(np.random.default_rng(3), 3 * 150, 200, "bf16")
    q, s, qt, st = _new8(150, 3, 256).transpose(0, 1), _bytes(3, 2, 2), _new8(200, 3, 256).transpose(0, 1), _bytes(3, 2, 2)
    nsq.ns_quantize(x.view(3, 150, 200), q, s, qt, st, block_rows=128)
    torch.cuda.synchronize()
    for i in range(3):
        part = x64[150 * i:150 * i + 150]
        for got, ref in zip((q[i], s[i], qt[i], st[i]), ops.quantize(part, 128) + ops.quantize(part.T, 128)):
            _same(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [[3, 100, 228, 228, 290], [128, 130, 300], [129, 129, 300], [300, 300], [257, 258, 258, 259]])
def test_quantize_rows_in_front_of_the_first_group(at, dtype):
    """q and its scales hold every row, whether or not qt is asked for."""
    import torch
    log(f"quantize in front {at} {dtype}")
    rows, groups = 300, len(at) - 1
    p = (rows // 128 + groups) * 128
    x, x64 = _values(np.random.default_rng(at[0]), rows, 200, dtype)
    want = ops.quantize(x64, 1)
    vt, sw, written = ops.quantize_groups(x64, at)
    for turned in (True, False):
        q, s, qt, st = _new8(rows, 256), _bytes(rows, 2), _new8(200, p), _bytes(200, p // 128)
        nsq.ns_quantize(x, q, s, *((qt, st) if turned else ()), offsets=_offsets(at))
        torch.cuda.synchronize()
        _same(q, want[0])
        _same(s, want[1])
        _same(qt, np.where(written & turned, vt, np.nan))
        np.testing.assert_array_equal(st.cpu().numpy(), np.where(written[::128] & turned, sw, 255))


def test_a_gate_without_rows_is_refused():
    import torch
    log("empty gate")
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    none = torch.empty(0, 64, device="cuda")
    for bad in (lambda: nsq.ns_block_norm(x, x, x.clone(), x.clone(), gate=none),
                lambda: nsq.ns_block_norm_backward(x, x, x, x, x.clone(), x.clone(), dgate=none, gate=none),
                lambda: nsq.ns_block_norm_backward(x, x, x, x, x.clone(), x.clone(), dpost_weight=w.clone(), gate=none)):
        with pytest.raises(ValueError, match="gate"):
            bad()


@pytest.mark.parametrize("turned", [False, True])
def test_quantize_groups_without_rows(turned):
    """No row in any group: nothing to write, with or without the transpose."""
    import torch
    log(f"quantize groups no rows {turned}")
    x, q, s = torch.empty(0, 200, device="cuda"), _new8(0, 256), _bytes(0, 2)
    qt, st = _new8(200, 3 * 128), _bytes(200, 3)
    nsq.ns_quantize(x, q, s, *((qt, st) if turned else ()), offsets=_offsets([0, 0, 0, 0]))
    torch.cuda.synchronize()
    assert torch.isnan(qt.float()).all() and (st == 255).all()


def test_groups_of_many_tiles_with_scales_for_each_row():
    """Groups on the 256-tiles, the matrices' rows with scales of their own."""
    import torch
    log("groups many tiles, rows' scales")
    rng = np.random.default_rng(19)
    at = [0, 0, 1, 700, 700, 2300, 2556, 4000]
    rows, n, k = 4100, 3001, 640
    a, sa, a64 = _operand(rng, rows, k, 1)
    b, sb, b64 = _operand(rng, n, k, 1, batch=7)
    out = _out(rows, n, "bfloat16")
    nsq.ns_scaled_matmul(a, sa, b, sb, out, offsets=_offsets(at))
    torch.cuda.synchronize()
    for e in range(7):
        picked = np.unique(np.concatenate([rng.integers(at[e], at[e + 1], 12), [at[e], at[e + 1] - 1]])) if at[e + 1] > at[e] else []
        if len(picked):
            _check(out[torch.from_numpy(picked).cuda()], a64[picked], b64[e], f"group {e}")
    assert torch.isnan(out[4000:].float()).all() and _beside(out)
