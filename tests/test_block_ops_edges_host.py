"""Operators around a block's products: calls at the edge of what their documentation allows, refused on the host (no GPU needed)."""

import pytest

import newton_schulz_quintic_amd as nsq
from tests.test_block_ops_host import INVALID, MAT, OK, OVERFLOW, P, QUANT, _matmul, _quantize

BATCH = {**QUANT, "batch": 3, "tall": 128, "xb": 800}


@pytest.mark.parametrize("change", [
    dict(qt=None, st=None, qb=0), dict(qt=None, st=None, qb=256 * 3), dict(qt=None, st=None, qld=512, qb=272),
    dict(qt=None, st=None, qld=768, qb=272), dict(q=None, s=None, tb=0), dict(q=None, s=None, tb=199 * 128),
    dict(q=None, s=None, tld=256, tb=128)])
def test_quantize_refuses_matrices_that_overlap(change):
    assert _quantize({**BATCH, **change}) == INVALID
    assert "overlap" in nsq.ns_last_error()


OVER = {**MAT, "k": 512, "lda": 512, "ldb": 512, "off": P, "groups": 3, "reduce": 1, "rows": 200}


@pytest.mark.parametrize("change", [dict(ob=0), dict(ob=31), dict(ldo=16, ob=8), dict(ldo=24, ob=4), dict(ldo=40, ob=36),
                                    dict(ldo=40, ob=84)])
def test_products_over_groups_refuse_outputs_that_overlap(change):
    assert _matmul({**OVER, **change}) == INVALID
    assert "overlap" in nsq.ns_last_error()


def test_overlap_is_found_exactly():
    """Outputs that share a place are refused for that, all others for the next fault, an operand that is NULL."""
    for rows in (1, 2, 5):
        for cols in (8, 9):
            for ld in (cols, 24, 40, 41):
                for stride in (0, 1, 7, 8, 9, 16, 20, 30, 40, 80, 100, 1000):
                    places = [g * stride + i * ld + j for g in range(3) for i in range(rows) for j in range(cols)]
                    assert _matmul({**OVER, "m": rows, "n": cols, "ldo": ld, "ob": stride, "a": None}) == INVALID
                    told = "overlap" if len(set(places)) < len(places) else "a is NULL"
                    assert told in nsq.ns_last_error(), (rows, cols, ld, stride)


def test_quantize_groups_without_rows():
    """Empty tensors have no address; there is nothing to write."""
    assert _quantize({**QUANT, "rows": 0, "x": None, "q": None, "s": None, "qt": None, "st": None, "off": P, "groups": 3}) == OK
    assert _quantize({**QUANT, "rows": 0, "x": None, "off": P, "groups": 3, "tld": 384}) == OK


def test_more_workgroups_than_a_launch_takes():
    """A launch has fewer than 2^32 threads along an axis."""
    top = 1 << 30
    assert _quantize({**QUANT, "rows": top, "cols": 1, "ld": 1, "qt": None, "st": None, "qld": 128}) == OVERFLOW
    few = {**MAT, "k": 128, "lda": 128, "ldb": 128, "tall": 1, "ldo": top}
    assert _matmul({**few, "m": 1, "n": top}) == OVERFLOW and _matmul({**few, "m": 32, "n": top}) == OVERFLOW
    wide = {**few, "m": 2048, "n": 1 << 22, "off": P, "groups": 1024, "od": 1}
    assert _matmul(wide) == OVERFLOW and _matmul({**wide, "od": 0}) == OVERFLOW
