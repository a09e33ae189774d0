"""GPU parity of ns_quantize (exact) and ns_scaled_matmul against the fp64 oracle (oracle/block_ops.py).

Tolerances of the products, per value, with S the sum of |a b| over the reduction (scales included) and U = 2^-24:
 - fp32 outputs: products are exact (4 x 4 significant bits); a sum of n blocks of 128 is added in 4 n matrix instructions
   of 32 products each and, split, in up to 32 parts: under 2 (4 n + 32 + 32) U S, a matrix instruction counted as two
   roundings a step; and half a step of the result.
 - bf16 outputs of the 8-bit matrix instructions: they align a block's products to the largest of them and drop what lies
   below some 2^-13 of it, for each of at most 128 products at most 2^-13 of the largest: a block is off by at most
   128 x 2^-13 = 2^-6 of its largest product. Half a step of bf16 is 2^-8 of the value. (No bound holds relative to the
   value alone: the products of an output may cancel to less than what is dropped of the largest.)
"""

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from oracle import block_ops as ops
from tests.helpers import host_to_f64, log, to_device
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _up(n):
    return -(-n // 128) * 128


def _new8(*shape):
    """e4m3 NaN everywhere, to see what was written."""
    import torch
    return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def _bytes(*shape):
    import torch
    return torch.full(shape, 255, dtype=torch.uint8, device="cuda")


def _np(t):
    import torch
    return t.float().cpu().numpy().astype(np.float64) if t.dtype != torch.uint8 else t.cpu().numpy()


def _same(got, want):
    np.testing.assert_array_equal(np.nan_to_num(_np(got), nan=1e9), np.nan_to_num(want, nan=1e9))


def _values(rng, rows, cols, dtype, kind="normal"):
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    if kind == "spread":      # sizes from below e4m3's exponents to fp32's ends, rows and columns of their own
        x *= np.exp2(rng.integers(-60, 60, (rows, 1)) + rng.integers(-12, 12, (1, cols))).astype(np.float32)
    elif kind == "ties":      # many values halfway between two of e4m3
        x = np.exp2(rng.integers(-12, 8, (rows, cols))).astype(np.float32) * (rng.integers(16, 32, (rows, cols)) / 16).astype(np.float32)
    elif kind == "ends":
        x = np.resize(np.array([0.0, -0.0, 1e-45, -1e-40, 1.2e-38, 3.3e38, -3.4e38, 448.0, 449.0, 464.0, 0.01], np.float32), (rows, cols))
        x = np.where(rng.random((rows, cols)) < 0.7, 0, x).astype(np.float32)
    elif kind == "strange":
        x[rng.random((rows, cols)) < 0.02] = np.nan
        x[rng.random((rows, cols)) < 0.02] = np.inf
        x[rng.random((rows, cols)) < 0.02] = -np.inf
        x[0] = np.nan
    if dtype == "bf16":
        with np.errstate(all="ignore"):
            h = f32_to_bf16_bits(np.clip(x, -3.38e38, 3.38e38) if kind == "ends" else x)
    else:
        h = x
    return to_device(h, dtype), host_to_f64(h, dtype)


@pytest.mark.parametrize("kind", ["normal", "spread", "ties", "ends", "strange"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (128, 128), (129, 257), (20, 1000), (260, 72), (2100, 136)])
def test_quantize(rows, cols, dtype, kind):
    import torch
    log(f"quantize {rows} {cols} {dtype} {kind}")
    x, x64 = _values(np.random.default_rng([rows, cols]), rows, cols, dtype, kind)
    for tall in (1, 128):
        want = ops.quantize(x64, tall) + ops.quantize(x64.T, tall)
        for q_only, t_only in ((False, False), (True, False), (False, True)):
            q, s = _new8(rows, _up(cols)), _bytes(rows if tall == 1 else -(-rows // 128), _up(cols) // 128)
            qt, st = _new8(cols, _up(rows)), _bytes(cols if tall == 1 else -(-cols // 128), _up(rows) // 128)
            nsq.ns_quantize(x, *((None, None) if t_only else (q, s)), *((None, None) if q_only else (qt, st)), block_rows=tall)
            torch.cuda.synchronize()
            if not t_only:
                _same(q, want[0])
                _same(s, want[1])
            if not q_only:
                _same(qt, want[2])
                _same(st, want[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_views_and_batches(dtype):
    """Rows of wider tensors at odd offsets, and matrices one after another."""
    import torch
    log(f"quantize views {dtype}")
    rng = np.random.default_rng(2)
    x, x64 = _values(rng, 150, 301, dtype)
    x, x64 = x[:, 7:207], x64[:, 7:207]
    q8, t8 = _new8(150, 400), _new8(200, 512)
    q, qt, s, st = q8[:, 16:272], t8[:, 128:384], _bytes(150, 2), _bytes(200, 2)
    nsq.ns_quantize(x, q, s, qt, st)
    torch.cuda.synchronize()
    want, wt = ops.quantize(x64, 1), ops.quantize(x64.T, 1)
    _same(q, want[0])
    _same(s, want[1])
    _same(qt, wt[0])
    _same(st, wt[1])
    for t, lo, hi in ((q8, 16, 272), (t8, 128, 384)):
        assert torch.isnan(t[:, :lo].float()).all() and torch.isnan(t[:, hi:].float()).all()
    w, w64 = _values(rng, 3 * 150, 200, dtype)
    q, s, qt, st = _new8(3, 150, 256), _bytes(3, 2, 2), _new8(3, 200, 256), _bytes(3, 2, 2)
    nsq.ns_quantize(w.view(3, 150, 200), q, s, qt, st, block_rows=128)
    torch.cuda.synchronize()
    for i in range(3):
        want, wt = ops.quantize(w64[150 * i:150 * i + 150], 128), ops.quantize(w64[150 * i:150 * i + 150].T, 128)
        for got, ref in ((q[i], want[0]), (s[i], want[1]), (qt[i], wt[0]), (st[i], wt[1])):
            _same(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 7, 8, 9, 14, 15, 63, 121, 125, 134, 135])
def test_quantize_ends_of_rows(cols, dtype):
    """Widths that end inside a lane's eight elements, in rows that other values follow."""
    import torch
    log(f"quantize ends {cols} {dtype}")
    x, x64 = _values(np.random.default_rng(cols), 40, cols + 9, dtype, "strange" if cols == 63 else "normal")
    x, x64 = x[:, :cols], x64[:, :cols]
    for tall in (1, 128):
        want = ops.quantize(x64, tall) + ops.quantize(x64.T, tall)
        q, s = _new8(40, _up(cols)), _bytes(40 if tall == 1 else 1, _up(cols) // 128)
        qt, st = _new8(cols, 128), _bytes(cols if tall == 1 else -(-cols // 128), 1)
        nsq.ns_quantize(x, q, s, qt, st, block_rows=tall)
        torch.cuda.synchronize()
        for got, ref in ((q, want[0]), (s, want[1]), (qt, want[2]), (st, want[3])):
            _same(got, ref)
    q, s = _new8(40, _up(cols)), _bytes(40, _up(cols) // 128)
    nsq.ns_quantize(x, q, s)
    torch.cuda.synchronize()
    want = ops.quantize(x64, 1)
    _same(q, want[0])
    _same(s, want[1])


GROUPS = [[0, 5], [0, 0, 130, 130, 131, 300], [3, 100, 228, 228, 290], [0, 128, 256, 300], [0] * 70 + [300], [0, 0, 0]]


def _offsets(at):
    import torch
    return torch.tensor(at, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("at", GROUPS)
def test_quantize_groups(at):
    """Each group from a whole block on; rows behind the last group in q alone; what is not written stays."""
    import torch
    log(f"quantize groups {at[:6]}")
    rows, groups = 300, len(at) - 1
    p = (rows // 128 + groups) * 128
    x, x64 = _values(np.random.default_rng(5), rows, 200, "bf16")
    q, s, qt, st = _new8(rows, 256), _bytes(rows, 2), _new8(200, p), _bytes(200, p // 128)
    nsq.ns_quantize(x, q, s, qt, st, offsets=_offsets(at))
    torch.cuda.synchronize()
    want = ops.quantize(x64, 1)
    first = at[0]   # rows before the first group have no place either
    _same(q[first:], want[0][first:])
    _same(s[first:], want[1][first:])
    vt, sw, written = ops.quantize_groups(x64, at)
    _same(qt, np.where(written, vt, np.nan))
    np.testing.assert_array_equal(st.cpu().numpy(), np.where(written[::128], sw, 255))


def _operand(rng, rows, k, tall, batch=None, wide=False):
    """e4m3 values of every finite kind, and scales: tensors, and what they stand for in 64 bits."""
    import torch
    lead = () if batch is None else (batch,)
    codes = rng.integers(0, 256, (*lead, rows, k), dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = rng.integers(118, 136, (*lead, rows if tall == 1 else -(-rows // 128), k // 128), dtype=np.uint8)
    if wide:
        t = torch.full((*lead, rows, k + 48), 0x7F, dtype=torch.uint8, device="cuda")
        t[..., 16:16 + k] = torch.from_numpy(codes).cuda()
        t = t[..., 16:16 + k]
    else:
        t = torch.from_numpy(codes).cuda()
    q = t.view(torch.float8_e4m3fn)
    flat = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy().astype(np.float64).reshape(-1, rows, k)
    v = np.stack([ops.value(f, s) for f, s in zip(flat, scales.reshape(len(flat), -1, k // 128))])
    return q, torch.from_numpy(scales).cuda(), v if batch is not None else v[0]


def _check(got, a, b, what):
    """got against a b^T, by the tolerances above."""
    import torch
    want = a @ b.T
    n = a.shape[1] // 128
    size = np.abs(a) @ np.abs(b).T
    if got.dtype == torch.float32:
        tol = 2 * (4 * n + 64) * U * size + U * np.abs(want)
    else:
        largest = sum(np.abs(a[:, None, k:k + 128] * b[None, :, k:k + 128]).max(2) if a.size * b.shape[0] < 3e7 else
                      np.abs(a[:, k:k + 128]).max(1)[:, None] * np.abs(b[:, k:k + 128]).max(1)[None] for k in range(0, a.shape[1], 128))
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -6 * largest
    bad = ~(np.abs(_np(got) - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(_np(got) - want) / (tol + 1e-300)):.3g} x tol"


def _out(rows, cols, dtype, *lead, wide=True):
    import torch
    t = torch.full((*lead, rows, cols + (11 if wide else 0)), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    return t[..., 3:3 + cols] if wide else t


def _beside(out):
    import torch
    b = out._base
    return bool(torch.isnan(b[..., :3].float()).all() and torch.isnan(b[..., 3 + out.shape[-1]:].float()).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k,tall", [
    (1, 1, 128, 1), (1, 130, 256, 128), (16, 64, 384, 128), (17, 300, 640, 1), (32, 7000, 128, 128), (5, 13400, 256, 1),
    (33, 129, 512, 128), (100, 100, 2048, 1), (128, 256, 1152, 128), (300, 70, 4096, 128), (200, 1000, 896, 1),
    (2000, 1700, 128, 128), (1800, 1900, 256, 1)])
def test_products(m, n, k, tall, dtype):
    import torch
    log(f"product {m} {n} {k} {tall} {dtype}")
    rng = np.random.default_rng([m, n, k])
    a, sa, a64 = _operand(rng, m, k, 1, wide=True)
    b, sb, b64 = _operand(rng, n, k, tall, wide=True)
    out = _out(m, n, dtype)
    nsq.ns_scaled_matmul(a, sa, b, sb, out)
    torch.cuda.synchronize()
    _check(out, a64, b64, "product")
    assert _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n", [4000, 4100, 8200, 12300, 16400, 20500, 24600, 28700, 33000])
@pytest.mark.parametrize("m,k", [(1, 1152), (16, 256), (17, 384), (32, 1152)])
def test_products_of_few_rows(m, k, n, dtype):
    """A workgroup takes one to eight blocks of 16 rows of b, by their number."""
    import torch
    log(f"few rows {m} {n} {k} {dtype}")
    rng = np.random.default_rng([m, n, k])
    a, sa, a64 = _operand(rng, m, k, 1)
    b, sb, b64 = _operand(rng, n, k, 128)
    out = _out(m, n, dtype)
    nsq.ns_scaled_matmul(a, sa, b, sb, out)
    torch.cuda.synchronize()
    _check(out, a64, b64, "few rows")
    assert _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", [(20, 500, 7000 // 128 * 128), (16, 1900, 8448), (900, 2950, 8192)])
def test_products_of_long_reductions(m, n, k, dtype):
    """Few rows whose reduction is cut into parts, and a tile for most CUs, cut in two."""
    import torch
    log(f"long {m} {n} {k} {dtype}")
    rng = np.random.default_rng([m, n, k])
    a, sa, a64 = _operand(rng, m, k, 1)
    b, sb, b64 = _operand(rng, n, k, 128)
    out = _out(m, n, dtype)
    nsq.ns_scaled_matmul(a, sa, b, sb, out)
    torch.cuda.synchronize()
    rows = np.unique(rng.integers(0, m, 60))
    _check(out[torch.from_numpy(rows).cuda()], a64[rows], b64, "long")
    assert _beside(out)


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("m,n,k", [(3600, 3500, 128), (3600, 3500, 384), (3584, 3584, 512), (3590, 3599, 640), (3333, 4001, 1152)])
def test_products_of_many_tiles(m, n, k, tall):
    """Calls that run on the 256-tiles: one to several stages, whole and cut tiles. Rows picked for the oracle."""
    import torch
    log(f"many tiles {m} {n} {k} {tall}")
    rng = np.random.default_rng([m, n, k, tall])
    a, sa, a64 = _operand(rng, m, k, 1)
    b, sb, b64 = _operand(rng, n, k, tall)
    out = _out(m, n, "bfloat16")
    nsq.ns_scaled_matmul(a, sa, b, sb, out)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([rng.integers(0, m, 40), [0, 127, 128, 255, 256, m - 1]]))
    _check(out[torch.from_numpy(rows).cuda()], a64[rows], b64, "rows")
    cols = np.unique(np.concatenate([rng.integers(0, n, 40), [0, 127, 128, 255, 256, n - 1]]))
    _check(out[:, torch.from_numpy(cols).cuda()], a64, b64[cols], "columns")
    assert _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("at", GROUPS[1:])
def test_products_by_group(at, dtype):
    """Rows of each group with its own matrix; the rows behind the last group stay as they were."""
    import torch
    log(f"groups {at[:6]} {dtype}")
    rows, groups, n, k = 300, len(at) - 1, 200, 384
    rng = np.random.default_rng(len(at))
    a, sa, a64 = _operand(rng, rows, k, 1)
    for tall in (128, 1):
        b, sb, b64 = _operand(rng, n, k, tall, batch=groups)
        out = _out(rows, n, dtype)
        nsq.ns_scaled_matmul(a, sa, b, sb, out, offsets=_offsets(at))
        torch.cuda.synchronize()
        for e in range(groups):
            if at[e + 1] > at[e]:
                _check(out[at[e]:at[e + 1]], a64[at[e]:at[e + 1]], b64[e], f"group {e}")
        assert torch.isnan(out[:at[0]].float()).all() and torch.isnan(out[at[-1]:].float()).all() and _beside(out)


def test_groups_of_many_tiles():
    """Groups on the 256-tiles: empty ones, one row, many; some rows in none."""
    import torch
    log("groups many tiles")
    rng = np.random.default_rng(9)
    at = [0, 0, 1, 700, 700, 2300, 2556, 4000]
    rows, n, k = 4100, 3000, 640
    a, sa, a64 = _operand(rng, rows, k, 1)
    b, sb, b64 = _operand(rng, n, k, 128, batch=7)
    out = _out(rows, n, "bfloat16")
    nsq.ns_scaled_matmul(a, sa, b, sb, out, offsets=_offsets(at))
    torch.cuda.synchronize()
    for e in range(7):
        picked = np.unique(np.concatenate([rng.integers(at[e], at[e + 1], 12), [at[e], at[e + 1] - 1]])) if at[e + 1] > at[e] else []
        if len(picked):
            _check(out[torch.from_numpy(picked).cuda()], a64[picked], b64[e], f"group {e}")
    assert torch.isnan(out[4000:].float()).all() and _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("at", [g for g in GROUPS[1:] if len(g) < 20])
def test_products_over_groups(at, dtype):
    """A matrix for each group, over its rows; zeros for an empty one."""
    import torch
    log(f"reduce {at[:6]} {dtype}")
    rows, groups = 300, len(at) - 1
    rng = np.random.default_rng(len(at) + 50)
    y, y64 = _values(rng, rows, 70, "bf16")
    x, x64 = _values(rng, rows, 140, "f32")
    p, offsets = (rows // 128 + groups) * 128, _offsets(at)
    yq, ys, xq, xs = _new8(70, p), _bytes(70, p // 128), _new8(140, p), _bytes(140, p // 128)
    nsq.ns_quantize(y, None, None, yq, ys, offsets=offsets)
    nsq.ns_quantize(x, None, None, xq, xs, offsets=offsets)
    out = _out(70, 140, dtype, groups)
    nsq.ns_scaled_matmul(yq, ys, xq, xs, out, offsets=offsets, reduce=True)
    torch.cuda.synchronize()
    for e in range(groups):
        if at[e + 1] == at[e]:
            assert not out[e].any()
            continue
        a = ops.value(*ops.quantize(y64[at[e]:at[e + 1]].T, 1))
        b = ops.value(*ops.quantize(x64[at[e]:at[e + 1]].T, 1))
        _check(out[e], a, b, f"group {e}")
    assert _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("at,n,k", [([0, 1, 1, 2, 2], 300, 7808), ([2, 20, 150, 151], 190, 4096), ([0, 0, 0], 130, 2048),
                                    ([1, 40, 41, 60, 70], 1027, 2176)])
def test_products_by_group_of_long_reductions(at, n, k, dtype):
    """Few rows by group: the reduction is cut into parts, and rows of no group stay as they were."""
    import torch
    log(f"groups long {at} {n} {k} {dtype}")
    rows, groups = max(at[-1], 1) + 3, len(at) - 1
    rng = np.random.default_rng([n, k])
    a, sa, a64 = _operand(rng, rows, k, 1)
    b, sb, b64 = _operand(rng, n, k, 128, batch=groups)
    out = _out(rows, n, dtype)
    assert nsq.ns_scaled_matmul_workspace_bytes(rows, n, k, groups)
    nsq.ns_scaled_matmul(a, sa, b, sb, out, offsets=_offsets(at))
    torch.cuda.synchronize()
    for e in range(groups):
        if at[e + 1] > at[e]:
            _check(out[at[e]:at[e + 1]], a64[at[e]:at[e + 1]], b64[e], f"group {e}")
    assert torch.isnan(out[:at[0]].float()).all() and torch.isnan(out[at[-1]:].float()).all() and _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_products_over_a_long_group(dtype):
    """Groups of very different lengths, whose reductions are cut into parts."""
    import torch
    log(f"reduce long {dtype}")
    at, rows = [0, 100, 100, 7000, 7001], 7100
    rng = np.random.default_rng(51)
    y, y64 = _values(rng, rows, 70, "bf16")
    x, x64 = _values(rng, rows, 140, "bf16")
    p, offsets = (rows // 128 + 4) * 128, _offsets(at)
    yq, ys, xq, xs = _new8(70, p), _bytes(70, p // 128), _new8(140, p), _bytes(140, p // 128)
    nsq.ns_quantize(y, None, None, yq, ys, offsets=offsets)
    nsq.ns_quantize(x, None, None, xq, xs, offsets=offsets)
    out = _out(70, 140, dtype, 4)
    nsq.ns_scaled_matmul(yq, ys, xq, xs, out, offsets=offsets, reduce=True)
    torch.cuda.synchronize()
    for e in range(4):
        if at[e + 1] == at[e]:
            assert not out[e].any()
            continue
        a = ops.value(*ops.quantize(y64[at[e]:at[e + 1]].T, 1))
        b = ops.value(*ops.quantize(x64[at[e]:at[e + 1]].T, 1))
        _check(out[e], a, b, f"group {e}")
    assert _beside(out)


def test_groups_over_many_rows_on_large_tiles():
    """bf16 gradients of many large matrices: the reduction by group on the 256-tiles."""
    import torch
    log("reduce large")
    rng = np.random.default_rng(3)
    at, rows, n, m = [0, 300, 300, 1000, 1129], 1200, 1900, 2000
    y, y64 = _values(rng, rows, m, "bf16")
    x, x64 = _values(rng, rows, n, "bf16")
    p, offsets = (rows // 128 + 4) * 128, _offsets(at)
    yq, ys, xq, xs = _new8(m, p), _bytes(m, p // 128), _new8(n, p), _bytes(n, p // 128)
    nsq.ns_quantize(y, None, None, yq, ys, offsets=offsets)
    nsq.ns_quantize(x, None, None, xq, xs, offsets=offsets)
    out = _out(m, n, "bfloat16", 4)
    nsq.ns_scaled_matmul(yq, ys, xq, xs, out, offsets=offsets, reduce=True)
    torch.cuda.synchronize()
    picked = np.unique(np.concatenate([rng.integers(0, m, 20), [0, 255, 256, m - 1]]))
    for e in range(4):
        if at[e + 1] == at[e]:
            assert not out[e].any()
            continue
        a = ops.value(*ops.quantize(y64[at[e]:at[e + 1], picked].T, 1))
        b = ops.value(*ops.quantize(x64[at[e]:at[e + 1]].T, 1))
        _check(out[e][torch.from_numpy(picked).cuda()], a, b, f"group {e}")
    assert _beside(out)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_what_is_not_finite_stays_in_its_row(dtype):
    import torch
    log(f"nan rows {dtype}")
    rng = np.random.default_rng(8)
    for m, n in ((8, 40), (200, 150)):
        a, sa, _ = _operand(rng, m, 256, 1)
        b, sb, _ = _operand(rng, n, 256, 1)
        a.view(torch.uint8)[3, 130] = 0x7F
        b.view(torch.uint8)[5, 7] = 0xFF
        out = torch.empty(m, n, dtype=getattr(torch, dtype), device="cuda")
        nsq.ns_scaled_matmul(a, sa, b, sb, out)
        torch.cuda.synchronize()
        bad = torch.isnan(out.float())
        assert bad[3].all() and bad[:, 5].all() and bad.sum() == m + n - 1


def test_scales_over_their_range():
    """Exponents far apart: powers of two that cancel, and results at fp32's ends."""
    import torch
    log("scale range")
    one = torch.full((4, 256), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)   # 1.0
    for ea, eb in ((1, 253), (254, 1), (127, 1), (60, 60), (200, 170), (90, 64)):
        want = 256.0 * 2.0 ** (ea + eb - 254)
        sa, sb = (torch.full((4, 2), e, dtype=torch.uint8, device="cuda") for e in (ea, eb))
        for dtype in (torch.float32, torch.bfloat16):
            out = torch.empty(4, 4, dtype=dtype, device="cuda")
            nsq.ns_scaled_matmul(one, sa, one, sb, out)
            torch.cuda.synchronize()
            assert (out.double() == want).all(), (ea, eb, dtype, out[0, 0].item(), want)


def test_same_bits_and_offsets_that_are_wrong():
    """The same inputs give the same bits; offsets out of range or order leave no fault."""
    import torch
    log("bits and wrong offsets")
    rng = np.random.default_rng(4)
    a, sa, _ = _operand(rng, 500, 1024, 1)
    b, sb, _ = _operand(rng, 300, 1024, 128, batch=3)
    out, again = (torch.empty(500, 300, device="cuda") for _ in "ab")
    good = _offsets([0, 100, 400, 500])
    for o in (out, again):
        nsq.ns_scaled_matmul(a, sa, b, sb, o, offsets=good)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    x, _ = _values(rng, 500, 128, "bf16")
    qt, st = _new8(128, 6 * 128), _bytes(128, 6)
    q, s = _new8(500, 128), _bytes(500, 1)
    for wrong in ([0, 600, 700, 800], [-5, 100, 90, 2 ** 31 - 1], [400, 300, 200, 100], [0, 500, 0, 500], [500, 500, 500, 500]):
        nsq.ns_scaled_matmul(a, sa, b, sb, again, offsets=_offsets(wrong))
        nsq.ns_quantize(x, q, s, qt, st, offsets=_offsets(wrong))
        nsq.ns_scaled_matmul(qt, st, qt, st, torch.empty(3, 128, 128, device="cuda"), offsets=_offsets(wrong), reduce=True)
        torch.cuda.synchronize()


def test_refusals_of_the_binding():
    import torch
    log("scaled refusals")
    a, s = _new8(4, 256), _bytes(4, 2)
    b3, s3, o = _new8(2, 8, 256), _bytes(2, 1, 2), torch.empty(4, 8, device="cuda")
    off = _offsets([0, 2, 4])
    x = torch.zeros(4, 200, device="cuda")
    for bad in (lambda: nsq.ns_scaled_matmul(a[:, :200], s, a, s, o), lambda: nsq.ns_scaled_matmul(a, s[:3], a, s, o[:, :4]),
                lambda: nsq.ns_scaled_matmul(a, s, a, s, o), lambda: nsq.ns_scaled_matmul(a, s, b3, s3, o),
                lambda: nsq.ns_scaled_matmul(a, s, a, s, o[:, :4], offsets=off), lambda: nsq.ns_scaled_matmul(a, s, b3, s3, o, offsets=off[:2]),
                lambda: nsq.ns_scaled_matmul(a, s, b3, s3, o, offsets=off, reduce=True), lambda: nsq.ns_scaled_matmul(a, s, a, s, o[:, :4], reduce=True),
                lambda: nsq.ns_quantize(x, a, s[:, :1]), lambda: nsq.ns_quantize(x, a, None), lambda: nsq.ns_quantize(x, None, None),
                lambda: nsq.ns_quantize(x[0], a, s), lambda: nsq.ns_quantize(x, a, s, block_rows=64), lambda: nsq.ns_quantize(x.t(), a, s)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nsq.ns_scaled_matmul(a.view(torch.uint8), s, a, s, o[:, :4]), lambda: nsq.ns_scaled_matmul(a, s.int(), a, s, o[:, :4]),
                lambda: nsq.ns_scaled_matmul(a, s, b3, s3, o, offsets=off.long()), lambda: nsq.ns_quantize(x.half(), a, s),
                lambda: nsq.ns_scaled_matmul(a, s, a, s, o[:, :4].half())):
        with pytest.raises(TypeError):
            bad()
    big = _new8(5, 256 + 8)
    for bad in (lambda: nsq.ns_scaled_matmul(big[:4, 8:], s, a, s, torch.empty(4, 4, device="cuda")),
                lambda: nsq.ns_quantize(torch.zeros(4, 8, 200, device="cuda"), _new8(4, 8, 256), _bytes(4, 8, 2))):
        with pytest.raises(nsq.NSError):
            bad()


def _far(rows, cols, ld, dtype):
    """(rows, cols) of a buffer whose rows lie ld elements apart, NaN in and beside them."""
    import torch
    big = torch.empty((rows - 1) * ld + cols + 16, dtype=dtype, device="cuda")
    t = big.as_strided((rows, cols + 16), (ld, 1)).fill_(float("nan"))
    return t[:, 8:8 + cols], t


def test_offsets_past_32_bits():
    """Rows, matrices and outputs further apart than 2^31 give the bits of those that lie together."""
    import torch
    log("far rows")
    rng = np.random.default_rng(31)
    x, _ = _values(rng, 3, 300, "bf16")
    far, beside = _far(3, 300, 1 << 31, torch.bfloat16)
    far.copy_(x)
    both = []
    for t in (x, far):
        q, s, qt, st = _new8(3, 384), _bytes(3, 3), _new8(300, 128), _bytes(300, 1)
        nsq.ns_quantize(t, q, s, qt, st)
        both.append([t.view(torch.uint8) for t in (q, s, qt, st)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*both))
    del far, beside
    for m, n, k, ld in ((3, 500, 384, 1 << 31), (200, 300, 256, 1 << 24), (3590, 3599, 256, 1 << 20)):
        a, sa, _ = _operand(rng, m, k, 1)
        b, sb, _ = _operand(rng, n, k, 128)
        near = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        far, beside = _far(m, n, ld, torch.bfloat16)
        for out in (near, far):
            nsq.ns_scaled_matmul(a, sa, b, sb, out)
        torch.cuda.synchronize()
        assert torch.equal(near, far), (m, n)
        assert torch.isnan(beside[:, :8].float()).all() and torch.isnan(beside[:, 8 + n:].float()).all()
        del far, beside
    a, sa, _ = _operand(rng, 200, 256, 1)
    b, sb, _ = _operand(rng, 40, 256, 128, batch=2)
    apart = torch.empty((1 << 32) + 40 * 256, dtype=torch.uint8, device="cuda")
    far = apart.as_strided((2, 40, 256), (1 << 32, 256, 1)).view(torch.float8_e4m3fn)
    far.view(torch.uint8).copy_(b.view(torch.uint8))
    outs = [torch.empty(200, 40, device="cuda") for _ in "ab"]
    for o, w in zip(outs, (b, far)):
        nsq.ns_scaled_matmul(a, sa, w, sb, o, offsets=_offsets([0, 70, 200]))
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    del far, apart
    at, p = _offsets([0, 130, 200]), (200 // 128 + 2) * 128
    qt, st = _new8(64, p), _bytes(64, p // 128)
    nsq.ns_quantize(_values(rng, 200, 64, "f32")[0], None, None, qt, st, offsets=at)
    near = torch.empty(2, 64, 64, device="cuda")
    far = torch.empty((1 << 31) + 64 * 64, device="cuda").as_strided((2, 64, 64), (1 << 31, 64, 1))
    for out in (near, far):
        nsq.ns_scaled_matmul(qt, st, qt, st, out, offsets=at, reduce=True)
    torch.cuda.synchronize()
    assert torch.equal(near, far)


def test_operands_of_more_than_2_gib():
    """600000 rows of 4096: the last ones, quantized and multiplied."""
    import torch
    log("many rows")
    m, k, n = 600000, 4096, 24
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(m, k, generator=g, device="cuda", dtype=torch.bfloat16)
    q, s = torch.empty(m, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(m, k // 128, dtype=torch.uint8, device="cuda")
    nsq.ns_quantize(x, q, s)
    b, sb, b64 = _operand(np.random.default_rng(4), n, k, 1)
    out = torch.empty(m, n, device="cuda")
    nsq.ns_scaled_matmul(q, s, b, sb, out)
    torch.cuda.synchronize()
    for lo in (0, 524200, m - 80):
        want = ops.quantize(_np(x[lo:lo + 80]), 1)
        _same(q[lo:lo + 80], want[0])
        _same(s[lo:lo + 80], want[1])
        _check(out[lo:lo + 80], ops.value(*want), b64, f"rows {lo}")
