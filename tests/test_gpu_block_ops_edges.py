"""Operators around a block's products: calls at the edge of what their documentation allows."""

import ctypes

import pytest

import newton_schulz_quintic_amd as nsq
from newton_schulz_quintic_amd import _lib
from newton_schulz_quintic_amd._ops import ns_rows
from tests.helpers import log

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
