"""GPU parity of the training-step operators against the fp64 oracle (oracle/train_ops.py).

Tolerances are bounds of the arithmetic, per value. U = 2^-24 is half a step of
fp32; a stored result adds half a step of its type (2^-8 of the value for bf16,
2^-24 for f32). An fp32 sum of n terms along a path of p additions is off by at
most p U times the sum of their absolute values; the kernels' paths are given
where they are used.
"""

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from oracle import train_ops as ops
from tests.helpers import host_to_f64, log, to_device, to_host
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}
PAD = 7   # elements around strided test tensors, to find writes outside them


def _torch_dtype(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def _host(rng, shape, dtype, std=1.0):
    """(array for to_device, its exact values)."""
    x = (rng.standard_normal(shape) * std).astype(np.float32)
    h = f32_to_bf16_bits(x) if dtype == "bf16" else x
    return h, host_to_f64(h, dtype)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype.itemsize < 4 else \
        t.detach().cpu().numpy().astype(np.float64)


def _close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want)) & ~(got == want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.where(bad, np.abs(got - want) / (tol + 1e-300), 0)):.3g} x tol"


# ---------------------------------------------------------------------------
# queries and keys
# ---------------------------------------------------------------------------

def _head_tensor(values, layout, dtype):
    """A device tensor of the (B, S, H, D) values in a memory order, amid a larger NaN buffer."""
    import torch
    b, s, h, d = values.shape
    t = to_device(values, dtype)
    nan = float("nan")
    if layout == "contiguous":
        return t
    if layout == "heads first":
        return torch.full((b, h, s, d), nan, dtype=t.dtype, device="cuda").transpose(1, 2).copy_(t)
    wide = torch.full((b, s, h * d + 2 * PAD), nan, dtype=t.dtype, device="cuda")   # a part of a fused row, odd offset
    view = wide[..., PAD:PAD + h * d].view(b, s, h, d) if (h * d) else wide[..., :0].view(b, s, h, d)
    return view.copy_(t)


def _qk_case(rng, b, s, hq, hk, d, r, dtype, layout, wdtype="f32", positions="far"):
    import torch
    c = {"b": b, "s": s, "d": d, "r": r, "dtype": dtype}
    for name, h in (("q", hq), ("k", hk), ("gq", hq), ("gk", hk)):
        bits, c[name + "64"] = _host(rng, (b, s, h, d), dtype)
        c[name] = _head_tensor(bits, layout, dtype)
    for name in ("wq", "wk"):
        bits, c[name + "64"] = _host(rng, (d,), wdtype)
        c[name] = to_device(bits, wdtype)
    rows = 50
    angle = rng.uniform(-3, 3, (rows, max(r // 2, 1)))
    c["cos"] = torch.from_numpy(np.cos(angle).astype(np.float32)).cuda() if r else None
    c["sin"] = torch.from_numpy(np.sin(angle).astype(np.float32)).cuda() if r else None
    pos = rng.integers(0, rows, (b, s))
    c["pos"] = torch.from_numpy(pos).cuda() if r else None
    if r:
        c["c64"], c["s64"] = (t.cpu().numpy().astype(np.float64)[pos][:, :, None] for t in (c["cos"], c["sin"]))
    else:
        c["c64"] = c["s64"] = np.zeros((b, s, 1, 0))
    return c


def _check_forward(c, got, x64, w64, inter, eps, what):
    """Path of the sum of squares: at most 16 values a lane and 6 exchanges; then mean, eps, square root,
    division (half of their sum reaches r), two products and a rotation: under 24 U of the pair's size."""
    want = ops.norm_rope(x64, w64, c["c64"], c["s64"], eps, inter)
    n = np.abs(x64) / np.sqrt(np.mean(x64 * x64, -1, keepdims=True) + eps) * np.abs(w64)
    size = ops.rotate(n, np.abs(c["c64"]), -np.abs(c["s64"]), inter)      # |a c| + |b s| at a's place
    size = np.maximum(size, ops.rotate(n, np.abs(c["c64"]), np.abs(c["s64"]), inter))
    _close(_f64(got), want, HALF_STEP[c["dtype"]] * np.abs(want) + 24 * U * size, what)


def _check_backward(c, dx, dw, x64, g64, w64, inter, eps, what):
    """As forward, with the second sum's path of 16 values and 6 exchanges, its three products and its mean: under
    48 U of |r| (|dn| + |n| mean|dn n|). dw: a lane's rows in turn (at most 32 here), 6 exchanges, 4 waves, and the
    join of at most 64 partials a lane and 4 exchanges, each term off by 16 U: under 128 U of the sum of |du n|."""
    wx, ww = ops.norm_rope_backward(x64, g64, w64, c["c64"], c["s64"], eps, inter)
    r = 1 / np.sqrt(np.mean(x64 * x64, -1, keepdims=True) + eps)
    n = np.abs(x64) * r
    ag = np.abs(g64)
    ac, as_ = np.abs(c["c64"]), np.abs(c["s64"])
    du = np.maximum(ops.rotate(ag, ac, as_, inter), ops.rotate(ag, ac, -as_, inter))
    dn = du * np.abs(w64)
    size = r * (dn + n * np.mean(dn * n, -1, keepdims=True))
    _close(_f64(dx), wx, HALF_STEP[c["dtype"]] * np.abs(wx) + 48 * U * size, what + " dx")
    if dw is not None:
        _close(_f64(dw), ww, 128 * U * np.sum(du * n, axis=(0, 1, 2)), what + " dw")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,s,hq,hk,d,r,layout", [
    (1, 1, 1, 1, 128, 128, "contiguous"),       # one token, one head
    (2, 1, 32, 8, 128, 128, "fused"),           # decode
    (2, 33, 8, 2, 128, 128, "fused"),
    (1, 70, 5, 3, 64, 64, "heads first"),
    (3, 5, 3, 1, 96, 64, "heads first"),        # partly rotated, groups with idle lanes
    (2, 7, 2, 2, 72, 72, "contiguous"),         # pieces of 4
    (1, 9, 3, 1, 72, 40, "fused"),
    (2, 3, 2, 1, 50, 20, "fused"),              # single elements
    (1, 4, 2, 1, 7, 4, "heads first"),          # an odd head, an odd tail
    (1, 3, 1, 1, 1, 0, "contiguous"),
    (2, 3, 3, 2, 80, 0, "contiguous"),          # no rotation
    (1, 2, 2, 1, 1024, 1024, "contiguous"),     # the longest heads
    (1, 2, 2, 1, 1022, 510, "contiguous"),
    (1, 3, 2, 1, 520, 264, "fused"),            # over 512 and in eighths only
])
def test_qk_norm_rope(b, s, hq, hk, d, r, layout, dtype, inter):
    import torch
    log(f"qk {b} {s} {hq} {hk} {d} {r} {layout} {dtype} {inter}")
    rng = np.random.default_rng([b, s, hq, d, r, inter])
    c = _qk_case(rng, b, s, hq, hk, d, r, dtype, layout)
    empty = lambda h: np.full((b, s, h, d), 0x7FC0, np.uint16) if dtype == "bf16" else np.full((b, s, h, d), np.nan, np.float32)  # noqa: E731
    qo, ko = (_head_tensor(empty(h), layout, dtype) for h in (hq, hk))
    kw = dict(q_weight=c["wq"], k_weight=c["wk"], cos=c["cos"], sin=c["sin"], pos=c["pos"], eps=1e-5, interleaved=inter)
    nsq.ns_qk_norm_rope(c["q"], c["k"], qo, ko, **kw)
    torch.cuda.synchronize()
    _check_forward(c, qo, c["q64"], c["wq64"], inter, 1e-5, "q")
    _check_forward(c, ko, c["k64"], c["wk64"], inter, 1e-5, "k")
    dq, dk = (_head_tensor(empty(h), layout, dtype) for h in (hq, hk))
    dwq, dwk = (torch.full((d,), float("nan"), device="cuda") for _ in "qk")
    nsq.ns_qk_norm_rope_backward(c["q"], c["k"], c["gq"], c["gk"], dq, dk, dq_weight=dwq, dk_weight=dwk, **kw)
    torch.cuda.synchronize()
    _check_backward(c, dq, dwq, c["q64"], c["gq64"], c["wq64"], inter, 1e-5, "q")
    _check_backward(c, dk, dwk, c["k64"], c["gk64"], c["wk64"], inter, 1e-5, "k")
    if layout == "fused":   # nothing outside the heads was written
        for t in (qo, ko, dq, dk):
            assert torch.isnan(t._base.view(b, s, -1)[..., :PAD]).all()
            assert torch.isnan(t._base.view(b, s, -1)[..., -PAD:]).all()


def test_qk_options():
    """One tensor alone, no weights, bf16 weights, positions absent, shared by the batch, of both widths; in place; the
    same bits from another stream, from a second call and in place."""
    import torch
    log("qk options")
    rng = np.random.default_rng(3)
    c = _qk_case(rng, 2, 6, 4, 2, 128, 128, "bf16", "contiguous", wdtype="bf16")
    kw = dict(cos=c["cos"], sin=c["sin"], pos=c["pos"], eps=1e-6)
    qo, ko = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    nsq.ns_qk_norm_rope(c["q"], c["k"], qo, ko, q_weight=c["wq"], k_weight=c["wk"], **kw)
    torch.cuda.synchronize()
    _check_forward(c, qo, c["q64"], c["wq64"], False, 1e-6, "bf16 weights")
    only = torch.empty_like(c["k"])
    nsq.ns_qk_norm_rope(None, c["k"], None, only, k_weight=c["wk"], **kw)
    narrow = torch.empty_like(c["q"])
    nsq.ns_qk_norm_rope(c["q"], None, narrow, None, q_weight=c["wq"], cos=c["cos"], sin=c["sin"], pos=c["pos"].int())
    side = torch.cuda.Stream()
    other = torch.empty_like(c["q"])
    torch.cuda.synchronize()
    nsq.ns_qk_norm_rope(c["q"], None, other, None, q_weight=c["wq"], **kw, stream=side)
    place = c["q"].clone()
    nsq.ns_qk_norm_rope(place, None, place, None, q_weight=c["wq"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(only, ko) and torch.equal(narrow, qo) and torch.equal(other, qo) and torch.equal(place, qo)
    nsq.ns_qk_norm_rope(c["q"], None, qo, None, **kw)
    torch.cuda.synchronize()
    _check_forward(c, qo, c["q64"], np.ones(128), False, 1e-6, "no weights")
    count = dict(c, c64=np.broadcast_to(c["cos"].cpu().numpy()[None, :6, None], (2, 6, 1, 64)).astype(np.float64),
                 s64=np.broadcast_to(c["sin"].cpu().numpy()[None, :6, None], (2, 6, 1, 64)).astype(np.float64))
    for pos in (None, torch.arange(6, device="cuda")):
        nsq.ns_qk_norm_rope(c["q"], None, qo, None, cos=c["cos"], sin=c["sin"], pos=pos)
        torch.cuda.synchronize()
        _check_forward(count, qo, c["q64"], np.ones(128), False, 1e-6, "counted positions")
    three = torch.empty_like(c["q"][0])
    nsq.ns_qk_norm_rope(c["q"][0], None, three, None, cos=c["cos"], sin=c["sin"])
    torch.cuda.synchronize()
    assert torch.equal(three, qo[0])
    # gradients in place of their inputs, and without the weights'
    dq, dwq = torch.empty_like(c["q"]), torch.empty(128, device="cuda")
    nsq.ns_qk_norm_rope_backward(c["q"], None, c["gq"], None, dq, None, dq_weight=dwq, q_weight=c["wq"], **kw)
    g, x = c["gq"].clone(), c["q"].clone()
    assert nsq.ns_qk_norm_rope_backward(c["q"], None, g, None, g, None, q_weight=c["wq"], **kw) is None
    nsq.ns_qk_norm_rope_backward(x, None, c["gq"], None, x, None, q_weight=c["wq"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(g, dq) and torch.equal(x, dq)
    _check_backward(c, dq, dwq, c["q64"], c["gq64"], c["wq64"], False, 1e-6, "bf16 weights")


def test_qk_positions_outside_the_table_and_zero_heads():
    import torch
    log("qk outside")
    x = torch.randn(1, 4, 2, 16, device="cuda")
    cos = torch.ones(3, 4, device="cuda")
    pos = torch.tensor([[0, -1, 3, 2]], device="cuda")
    out = torch.empty_like(x)
    nsq.ns_qk_norm_rope(x, None, out, None, cos=cos, sin=cos, pos=pos)
    torch.cuda.synchronize()
    bad = torch.isnan(out)
    assert bad[0, 1:3, :, :8].all() and not bad[0, [0, 3]].any() and not bad[..., 8:].any()
    zero = torch.zeros(1, 1, 1, 16, device="cuda")
    nsq.ns_qk_norm_rope(zero, None, out[:, :1, :1], None, eps=1e-6)
    dx, dw = torch.full_like(zero, 9.0), torch.full((16,), 9.0, device="cuda")
    nsq.ns_qk_norm_rope_backward(zero, None, torch.ones_like(zero), None, dx, None, dq_weight=dw, eps=1e-6)
    torch.cuda.synchronize()
    assert not out[:, :1, :1].any() and not dw.any()
    assert torch.allclose(dx, torch.full_like(dx, 1e3), rtol=1e-6)   # 1 / sqrt(eps)
    none = x[:, :0]
    nsq.ns_qk_norm_rope_backward(none, None, none, None, none, None, dq_weight=dw.fill_(9.0))
    torch.cuda.synchronize()
    assert not dw.any()   # a sum over no tokens


def test_qk_many_tokens():
    """More tokens than the backward has waves, so that a wave sums several; dw's path: 20000 rows over 4096 waves."""
    import torch
    log("qk many")
    rng = np.random.default_rng(8)
    c = _qk_case(rng, 1, 5000, 3, 1, 64, 64, "f32", "contiguous")
    qo, ko, dq, dk = (torch.empty_like(c[n]) for n in ("q", "k", "q", "k"))
    dwq, dwk = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    kw = dict(q_weight=c["wq"], k_weight=c["wk"], cos=c["cos"], sin=c["sin"], pos=c["pos"])
    nsq.ns_qk_norm_rope(c["q"], c["k"], qo, ko, **kw)
    nsq.ns_qk_norm_rope_backward(c["q"], c["k"], c["gq"], c["gk"], dq, dk, dq_weight=dwq, dk_weight=dwk, **kw)
    torch.cuda.synchronize()
    _check_forward(c, qo, c["q64"], c["wq64"], False, 1e-6, "q")
    _check_backward(c, dq, dwq, c["q64"], c["gq64"], c["wq64"], False, 1e-6, "q")
    _check_backward(c, dk, dwk, c["k64"], c["gk64"], c["wk64"], False, 1e-6, "k")


def test_qk_large_call_gives_the_bits_of_its_parts():
    """A call that moves more than the last-level cache holds (its stores take another path), sequence by sequence."""
    import torch
    log("qk large")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q, g = (torch.randn(9, 2048, 32, 128, device="cuda", generator=gen, dtype=torch.bfloat16) for _ in "qg")
    cos, sin = torch.rand(2048, 64, device="cuda"), torch.rand(2048, 64, device="cuda")
    out, dq = torch.empty_like(q), torch.empty_like(q)
    nsq.ns_qk_norm_rope(q, None, out, None, cos=cos, sin=sin)
    nsq.ns_qk_norm_rope_backward(q, None, g, None, dq, None, cos=cos, sin=sin)
    part, dpart = torch.empty_like(q[:1]), torch.empty_like(q[:1])
    for b in range(9):
        nsq.ns_qk_norm_rope(q[b:b + 1], None, part, None, cos=cos, sin=sin)
        nsq.ns_qk_norm_rope_backward(q[b:b + 1], None, g[b:b + 1], None, dpart, None, cos=cos, sin=sin)
        torch.cuda.synchronize()
        assert torch.equal(part[0], out[b]) and torch.equal(dpart[0], dq[b])


def test_qk_offsets_past_32_bits():
    import torch
    log("qk far")
    far = 2 ** 32 + 64
    buf = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (1, 2, 2, 64), (0, far, 64, 1))
    small = torch.randn(1, 2, 2, 64, device="cuda").bfloat16()
    x.copy_(small)
    want = torch.empty_like(small)
    nsq.ns_qk_norm_rope(small, None, want, None)
    nsq.ns_qk_norm_rope(x, None, x, None)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


# ---------------------------------------------------------------------------
# tokens by expert
# ---------------------------------------------------------------------------

def _sorted(ids, experts):
    import torch
    t, k = ids.shape
    off = torch.full((experts + 1,), -9, dtype=torch.int32, device="cuda")
    slot = torch.full((t * k,), -9, dtype=torch.int32, device="cuda")
    row = torch.full((t, k), -9, dtype=torch.int32, device="cuda")
    nsq.ns_moe_sort(ids, experts, off, slot, row)
    torch.cuda.synchronize()
    return off, slot, row


@pytest.mark.parametrize("t,k,e,kind", [
    (1, 1, 1, "even"), (1, 8, 64, "even"), (0, 4, 8, "even"), (7, 3, 5, "drop"), (64, 1, 2, "one"), (65, 1, 3, "skew"),
    (100, 4, 1024, "even"), (1000, 8, 64, "drop"), (1024, 8, 256, "even"),
    (256, 8, 256, "even"), (257, 8, 256, "even"),           # the largest in one workgroup, and one past it
    (65536, 8, 31, "drop"), (70001, 8, 1024, "skew"), (300007, 7, 33, "drop"),   # runs ranked at once, and longer ones
    (1025, 8, 255, "skew"), (3000, 3, 17, "drop"), (9001, 7, 64, "one"), (20000, 8, 1023, "drop"),
    (40000, 8, 64, "skew"), (5000, 2, 6, "none"),
])
def test_moe_sort(t, k, e, kind):
    import torch
    log(f"sort {t} {k} {e} {kind}")
    rng = np.random.default_rng([t, k, e])
    ids = rng.integers(0, e, (t, k))
    if kind == "drop":
        ids = np.where(rng.random((t, k)) < 0.2, rng.choice([-1, e, e + 5, -2 ** 31, 2 ** 31 - 1], (t, k)), ids)
    elif kind == "one":
        ids[:] = e - 1
    elif kind == "skew":
        ids = np.minimum(ids, rng.integers(0, e, (t, k)) // 4)
    elif kind == "none":
        ids[:] = -1
    want = ops.moe_sort(ids, e)
    wide = torch.full((t, k + 3), -5, dtype=torch.int64, device="cuda")
    wide[:, 1:k + 1] = torch.from_numpy(ids)
    wide[:, 1:k + 1][wide[:, 1:k + 1] == -1] = -2 ** 40   # far outside 32 bits: dropped, not truncated
    for x in (torch.from_numpy(ids.astype(np.int32)).cuda(), wide[:, 1:k + 1]):
        for got, w in zip(_sorted(x, e), want):
            assert np.array_equal(got.cpu().numpy(), w)


def _moe_case(t, k, e, h, dtype, drop, strided):
    import torch
    rng = np.random.default_rng([t, k, e, h])
    ids = np.where(rng.random((t, k)) < drop, -1, rng.integers(0, e, (t, k)))
    if drop and t > 2:
        ids[1] = -1   # a token with nothing left
    c = {"ids": ids, "row": ops.moe_sort(ids, e)[2]}
    c["row_d"] = torch.from_numpy(c["row"]).cuda()
    c["w64"] = rng.standard_normal((t, k)).astype(np.float32).astype(np.float64)
    for name, n in (("x", t), ("y", t * k), ("dout", t), ("dxs", t * k)):
        bits, c[name + "64"] = _host(rng, (n, h), dtype)
        v = to_device(bits, dtype)
        if strided:
            wide = torch.full((n, h + 2 * PAD), float("nan"), dtype=v.dtype, device="cuda")
            v = wide[:, PAD:PAD + h].copy_(v)
        c[name] = v
    w = c["w64"].astype(np.float32)
    dropped = c["row"] < 0
    w[dropped] = np.nan                        # what belongs to dropped slots is not used
    c["w"] = torch.from_numpy(w).cuda()
    c["w64"][dropped] = 0.0
    for name in ("y", "dxs"):
        c[name][torch.from_numpy(~c["row"][dropped]).cuda().long()] = float("nan")
        c[name + "64"][~c["row"][dropped]] = 0.0

    def out(n):
        wide = torch.full((n, h + 2 * PAD), float("nan"), dtype=_torch_dtype(dtype), device="cuda")
        return wide[:, PAD:PAD + h] if strided else wide[:, :h].contiguous()
    c["new"] = out
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k,e,h,drop,strided", [
    (1, 1, 1, 8, 0.0, False), (1, 8, 64, 7168, 0.0, False), (9, 3, 5, 1, 0.3, False), (9, 3, 5, 7, 0.3, True),
    (33, 2, 4, 100, 0.0, True), (17, 8, 16, 1537, 0.2, True), (50, 4, 8, 4096, 0.1, False), (5, 13, 40, 264, 0.2, False),
    (40, 1, 8, 520, 0.5, False), (3, 6, 8, 9000, 1.0, False), (12, 17, 20, 33, 0.1, True),
])
def test_moe_rows(t, k, e, h, drop, strided, dtype):
    """out: k products and additions, under (k + 1) U of their size. dweights: a thread's values in turn (at most
    9000 / 512 rounded up to whole vectors: 24), 6 exchanges and 8 waves: under 40 U of the sum of |g y|."""
    import torch
    log(f"moe rows {t} {k} {e} {h} {drop} {strided} {dtype}")
    c = _moe_case(t, k, e, h, dtype, drop, strided)
    row, half = c["row"], HALF_STEP[dtype]
    xs, out, dy, dx = c["new"](t * k), c["new"](t), c["new"](t * k), c["new"](t)
    dw = torch.full((t, k), float("nan"), device="cuda")
    nsq.ns_moe_dispatch(c["x"], c["row_d"], xs)
    nsq.ns_moe_combine(c["y"], c["row_d"], c["w"], out)
    nsq.ns_moe_combine_backward(c["dout"], c["y"], c["row_d"], c["w"], dy, dw)
    nsq.ns_moe_dispatch_backward(c["dxs"], c["row_d"], dx)
    torch.cuda.synchronize()
    assert np.array_equal(_f64(xs), ops.moe_dispatch(c["x64"], row))
    want = ops.moe_combine(c["y64"], row, c["w64"])
    size = ops.moe_combine(np.abs(c["y64"]), row, np.abs(c["w64"]))
    _close(_f64(out), want, half * np.abs(want) + (k + 1) * U * size, "out")
    want = ops.moe_combine(c["dxs64"], row)
    _close(_f64(dx), want, half * np.abs(want) + (k + 1) * U * ops.moe_combine(np.abs(c["dxs64"]), row), "dx")
    want_y, want_w = ops.moe_combine_backward(c["dout64"], c["y64"], row, c["w64"])
    _close(_f64(dy), want_y, (half + U) * np.abs(want_y), "dy")
    size = ops.moe_combine_backward(np.abs(c["dout64"]), np.abs(c["y64"]), row, c["w64"])[1]
    _close(_f64(dw), want_w, 40 * U * size, "dweights")
    if strided:
        for v in (xs, out, dy, dx):
            assert torch.isnan(v._base[:, :PAD]).all() and torch.isnan(v._base[:, -PAD:]).all()
    ones = c["new"](t)
    nsq.ns_moe_combine(c["dxs"], c["row_d"], None, ones)     # no weights: the dispatch's gradient
    place = c["y"].clone() if not strided else c["y"]
    nsq.ns_moe_combine_backward(c["dout"], place, c["row_d"], c["w"], place, dw)
    torch.cuda.synchronize()
    assert torch.equal(ones, dx) and torch.equal(place, dy)


def test_moe_map_entries_outside_the_rows_are_left_alone():
    import torch
    log("moe bad map")
    x = torch.randn(2, 16, device="cuda")
    row = torch.tensor([[0, 100], [-200, 3]], dtype=torch.int32, device="cuda")
    xs = torch.full((4, 16), 5.0, device="cuda")
    out, dw = torch.empty(2, 16, device="cuda"), torch.empty(2, 2, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    nsq.ns_moe_dispatch(x, row, xs)
    nsq.ns_moe_combine(xs, row, w, out)
    dy = torch.full((4, 16), 5.0, device="cuda")
    nsq.ns_moe_combine_backward(x, xs, row, w, dy, dw)
    torch.cuda.synchronize()
    assert torch.equal(xs[[0, 3]], x) and (xs[1:3] == 5).all() and torch.equal(out, x)
    assert torch.equal(dy[[0, 3]], x) and (dy[1:3] == 5).all() and dw[0, 1] == 0 and dw[1, 0] == 0


@pytest.mark.parametrize("dtype,hidden", [("bf16", 4096), ("f32", 2049)])
def test_moe_large_calls_give_the_bits_of_their_parts(dtype, hidden):
    """Calls that move more than the last-level cache holds (their rows take another path), token range by token range."""
    import torch
    log(f"moe large {dtype} {hidden}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    t, k = 9000, 4
    x, g = (torch.randn(t, hidden, device="cuda", generator=gen).to(_torch_dtype(dtype)) for _ in "xg")
    y = torch.randn(t * k, hidden, device="cuda", generator=gen).to(_torch_dtype(dtype))
    w = torch.rand(t, k, device="cuda", generator=gen)
    row = torch.randperm(t * k, device="cuda", generator=gen).to(torch.int32).view(t, k)
    row[5] = ~row[5]
    xs, dy, out, dx = (torch.empty_like(v) for v in (y, y, x, x))
    dw = torch.empty_like(w)
    nsq.ns_moe_dispatch(x, row, xs)
    nsq.ns_moe_combine(y, row, w, out)
    nsq.ns_moe_dispatch_backward(y, row, dx)
    nsq.ns_moe_combine_backward(g, y, row, w, dy, dw)
    torch.cuda.synchronize()
    kept = (row >= 0)[:, :, None]
    at = torch.where(row >= 0, row, ~row).long()
    assert torch.equal(xs[at], torch.where(kept, x[:, None], torch.zeros_like(x[:1])))
    for a in range(0, t, 1500):
        # the same tokens with their rows brought together
        s, n = slice(a, a + 1500), 1500 * k
        some = torch.arange(n, device="cuda", dtype=torch.int32).view(1500, k)
        some = torch.where(row[s] >= 0, some, ~some)
        ys = y[at[s].reshape(-1)].contiguous()
        o, d, e, f = torch.empty_like(x[s]), torch.empty_like(x[s]), torch.empty_like(ys), torch.empty_like(w[s])
        nsq.ns_moe_combine(ys, some, w[s], o)
        nsq.ns_moe_dispatch_backward(ys, some, d)
        nsq.ns_moe_combine_backward(g[s], ys, some, w[s], e, f)
        torch.cuda.synchronize()
        assert torch.equal(o, out[s]) and torch.equal(d, dx[s]) and torch.equal(f, dw[s])
        assert torch.equal(e, dy[at[s].reshape(-1)])


def test_moe_offsets_past_32_bits():
    import torch
    log("moe far")
    ld = 2 ** 31 + 8
    buf = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(buf, (3, 40), (ld, 1))
    x = torch.randn(3, 40, device="cuda").bfloat16()
    row = torch.tensor([[2], [0], [1]], dtype=torch.int32, device="cuda")
    nsq.ns_moe_dispatch(x, row, far)
    back = torch.empty_like(x)
    nsq.ns_moe_dispatch_backward(far, row, back)
    torch.cuda.synchronize()
    assert torch.equal(far, x[[1, 2, 0]]) and torch.equal(back, x)


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def _distill_case(rng, n, v, k, dtype, tdtype="f32", rest=False, tau=1.0, kind="plain", ld=None):
    import torch
    z = rng.standard_normal((n, v)) * 2
    ids = np.stack([rng.permutation(max(v, k))[:k] for _ in range(n)]) if v <= 4096 else \
        (rng.integers(0, v, (n, 1)) + np.arange(k) * rng.integers(1, v // k, (n, 1))) % v
    if kind == "twice":      # one token in all pairs, few tokens, tokens in several pairs, absent ones
        from_pair = np.where(rng.random((n, k)) < 0.3, rng.integers(0, k, (n, k)), np.arange(k))
        ids = np.take_along_axis(ids, from_pair, 1)
        ids[0] = ids[0, 0] % v
        ids[1] = rng.integers(0, min(v, 40), k)
        ids[2:][rng.random((n - 2, k)) < 0.1] = v
    for i in range(n):
        ok = ids[i] < v
        z[i, ids[i][ok]] += rng.uniform(3, 9, ok.sum())
    t = rng.uniform(3, 9, (n, k))
    if kind == "masked":     # absent pairs, rows without any, the same token twice, masked logits of both sides
        ids[rng.random((n, k)) < 0.3] = -1
        ids[rng.random((n, k)) < 0.1] = v + 3
        if k > 2:
            ids[:, 2] = ids[:, 0]
        if n > 2:
            ids[1] = -7
        t[rng.random((n, k)) < 0.2] = -np.inf
        if n > 4:
            t[3] = -np.inf
        dead = rng.random((n, v)) < 0.3
        for i in range(n):
            dead[i, ids[i][(ids[i] >= 0) & (ids[i] < v)]] = False
        z[dead] = -np.inf
        if n > 2:
            z[1] = np.nan    # not looked at
    if kind == "lowest":     # masks of the type's lowest value
        low = -3.3895313892515355e38 if dtype == "bf16" else -3.4028234663852886e38
        z[rng.random((n, v)) < 0.5] = low
        t[:, k // 2:] = -3.3895313892515355e38
    c = {"tau": tau, "ids": ids, "dtype": dtype}
    bits = f32_to_bf16_bits(z.astype(np.float32)) if dtype == "bf16" else z.astype(np.float32)
    c["z64"] = host_to_f64(bits, dtype)
    c["z"] = to_device(bits, dtype)
    if ld:
        wide = torch.full((n, ld), float("nan"), dtype=c["z"].dtype, device="cuda")
        c["z"] = wide[:, 3:3 + v].copy_(c["z"])
    tb = f32_to_bf16_bits(t.astype(np.float32)) if tdtype == "bf16" else t.astype(np.float32)
    c["t64"], c["t"] = host_to_f64(tb, tdtype), to_device(tb, tdtype)
    c["lse64"] = None
    if rest:
        with np.errstate(all="ignore"):
            inside = np.where((ids >= 0) & (ids < v), c["t64"] / tau, -np.inf)
            lse = np.array([ops._lse(r) if np.isfinite(r).any() else 0.0 for r in inside])
        c["lse64"] = (lse + rng.uniform(0.01, 0.8, n)).astype(np.float32).astype(np.float64)
    c["lse_d"] = None if not rest else torch.from_numpy(c["lse64"].astype(np.float32)).cuda()
    c["g64"] = rng.uniform(0.1, 1, n).astype(np.float32).astype(np.float64)
    c["g"] = torch.from_numpy(c["g64"].astype(np.float32)).cuda()
    c["ids_d"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    return c


def _distill_run(c, form, stream=None, place=False):
    import torch
    n, v = c["z"].shape
    loss, lse, rest = (torch.full((n,), float("nan"), device="cuda") for _ in range(3))
    rest = rest if c["lse_d"] is not None else None
    z = c["z"].clone() if place else c["z"]
    dz = z if place else torch.full((n, c["z"].stride(0) if n > 1 else v), float("nan"), dtype=z.dtype, device="cuda")[:, :v]
    kw = dict(teacher_lse=c["lse_d"], rest_lse=rest, temperature=c["tau"])
    torch.cuda.synchronize()
    if form == "train":
        nsq.ns_distill_topk(z, c["ids_d"], c["t"], loss, lse, grad_loss=c["g"], dlogits=dz, stream=stream, **kw)
    else:
        nsq.ns_distill_topk(z, c["ids_d"], c["t"], loss, lse, stream=stream, **kw)
        nsq.ns_distill_topk_backward(z, c["ids_d"], c["t"], lse, c["g"], dz, stream=stream, **kw)
    torch.cuda.synchronize()
    return loss, lse, rest, dz


def _check_distill(c, got, rows=None):
    """Every exponential is off by 2 U and by 2 U of its argument, and the reference point of q, m, by nothing: with
    E = sum q |z - m| / tau the sum's relative error is under (2 E + 64) U, 64 covering a path of at most 24 additions
    a thread, 6 exchanges, 16 waves and 64 parts' join less what a rescaling adds (2 U each, at most 12 in turn)."""
    loss, lse, rest, dz = got
    tau, half = c["tau"], HALF_STEP[c["dtype"]]
    for i in (range(len(c["z64"])) if rows is None else rows):
        tl = None if c["lse64"] is None else c["lse64"][i]
        w = ops.distill_row(c["z64"][i], c["ids"][i], c["t64"][i], tau, tl, c["g64"][i])
        g = c["g64"][i]
        got_z = _f64(dz[i])
        w["dlogits"][np.abs(w["dlogits"]) < 2.0 ** -126] = 0.0   # neither type holds it as a normal number
        if not w["some"]:
            assert loss[i] == 0 and lse[i] == 0 and not got_z.any()
            continue
        with np.errstate(all="ignore"):
            m = np.max(c["z64"][i])
            arg = np.where(w["q"] > 0, np.abs(c["z64"][i] - m) / tau, 0.0)
            E = np.sum(w["q"] * arg)
            here = [(int(j), float(x)) for j, x in zip(c["ids"][i], c["t64"][i]) if 0 <= j < len(c["z64"][i])]
            at = np.array([j for j, _ in here])
            t = np.array([x for _, x in here])
            targ = np.abs(t - np.max(t)) / tau + (0 if tl is None else abs(tl) + np.max(np.abs(t[np.isfinite(t)]), initial=0) / tau)
            p, log_p = w["p"], w["log_p"]
            used = p > 0
            err_q = (4 * arg[at] + 4 * E + 64) * U                 # of log q
            err_p = np.where(used, (4 * targ + 64) * U, 0)         # of log p, and relative of p (0 is exact)
            diff = np.abs(log_p - (np.log(w["q"][at])))
            tol = np.sum((p * (err_q + err_p + err_p * diff + 64 * U * diff))[used])
            tol_lse = U * (4 * np.abs(m) / tau + 4 * E + 64 + 2 * abs(w["lse"]))
            rest_term, err_others = 0.0, 0.0
            others = 1.0
            if tl is not None:
                outside = np.ones(len(c["z64"][i]), bool)
                outside[at] = False
                if not outside.any():   # no such class
                    assert rest[i] == -np.inf
                else:
                    zr = c["z64"][i][outside]
                    qr = np.exp(w["rest_lse"] - w["lse"])
                    er = np.sum(np.where(zr > -np.inf, w["q"][outside] * np.abs(zr - zr.max()) / tau, 0)) / max(qr, 1e-300)
                    err_rest = (4 * er + 64 + 4 * np.abs(zr.max() - m) / tau + 4 * E) * U
                    dp = np.sum((p * err_p)[used]) + 64 * U            # absolute, of p_r
                    if w["p_rest"] > 0:
                        rest_term = dp * (1 + abs(np.log(w["p_rest"]) - np.log(qr))) + w["p_rest"] * (err_rest + 8 * U)
                        others = 1.0 - w["p_rest"] / qr
                        err_others = (dp + w["p_rest"] * (err_rest + (2 * abs(w["lse"]) + 2 * abs(w["rest_lse"]) + 8) * U)) / qr
                    assert abs(float(rest[i]) - w["rest_lse"]) <= U * (4 * abs(zr.max()) / tau + 4 * er + 64 + 2 * abs(w["rest_lse"]))
        assert abs(float(loss[i]) - w["loss"]) <= tol + rest_term + 4 * U * abs(w["loss"]), (i, float(loss[i]), w["loss"], tol)
        assert abs(float(lse[i]) - w["lse"]) <= tol_lse
        err = (4 * arg + 4 * E + 64 + 2 * abs(w["lse"])) * U       # of q; 2 |lse| U where lse itself was rounded
        size = w["q"] * (err * abs(others) + err_others)
        size[at] = (w["q"] * err)[at]
        for a, b in zip(at, p * err_p):
            size[a] += b
        _close(got_z, w["dlogits"], half * np.abs(w["dlogits"]) * (1 + 2 * U) + g / tau * size + 4 * U * np.abs(w["dlogits"]),
               f"row {i}")


CASES = [
    (1, 1, 1, "plain"), (1, 5, 3, "plain"), (3, 8, 8, "plain"), (2, 1000, 4, "masked"), (5, 4099, 7, "masked"),
    (4, 8195, 20, "masked"), (3, 33333, 64, "masked"), (2, 70001, 130, "plain"), (6, 2048, 1024, "plain"),
    (7, 300, 20, "lowest"),
]


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,k,kind", CASES)
def test_distill_few_rows(n, v, k, kind, dtype, rest, form):
    log(f"distill {n} {v} {k} {kind} {dtype} {rest} {form}")
    rng = np.random.default_rng([n, v, k])
    c = _distill_case(rng, n, v, k, dtype, "bf16" if k % 2 else "f32", rest, 1.5 if n % 2 else 1.0, kind,
                      ld=v + 9 if n > 2 else None)
    _check_distill(c, _distill_run(c, form))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,n,v,k", [("bf16", 2600, 33000, 8), ("f32", 1100, 40001, 8), ("bf16", 2100, 70002, 5),
                                         ("f32", 1030, 70001, 5), ("bf16", 2200, 131072, 5), ("bf16", 9000, 1001, 5)])
def test_distill_rows_over_rounds_and_past_the_cache(dtype, n, v, k, rest):
    """Several rows a workgroup one after the other, and gradients stored past the cache, each row as by itself."""
    import torch
    log(f"distill rounds {dtype} {n} {v} {rest}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(v)
    z = (torch.randn(n, v, device="cuda", generator=gen) * 2).to(_torch_dtype(dtype))
    ids = torch.randint(0, v, (n, 1), device="cuda", generator=gen) + torch.arange(k, device="cuda") * (v // k // 2)
    ids = (ids % v).to(torch.int32)
    ids[::13] = -1
    t, g = torch.randn(n, k, device="cuda", generator=gen) + 4, torch.rand(n, device="cuda", generator=gen)
    tl = torch.logsumexp(t, 1) + 0.3 if rest else None
    rng = np.random.default_rng(v)
    rows = np.unique(np.concatenate([rng.integers(0, n, 4), [0, 1, n - 1]]))
    c = {"tau": 1.0, "dtype": dtype, "z": z, "ids_d": ids, "t": t, "g": g, "lse_d": tl}
    pick = torch.from_numpy(rows).cuda()
    c64 = dict(c, z64=_f64(z[pick]), ids=ids[pick].cpu().numpy(), t64=_f64(t[pick]), g64=_f64(g[pick]),
               lse64=None if tl is None else _f64(tl[pick]))
    for form in ("train", "step"):
        got = _distill_run(c, form)
        _check_distill(c64, tuple(None if x is None else x[pick] for x in got))


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,n,v,k,kind", [
    ("bf16", 257, 500, 5, "masked"), ("f32", 300, 77, 9, "masked"), ("bf16", 260, 20001, 16, "plain"),
    ("f32", 258, 12345, 16, "plain"), ("f32", 256, 20001, 8, "plain"), ("bf16", 256, 66001, 70, "plain"),
    ("bf16", 256, 131072, 64, "plain"), ("f32", 256, 50021, 20, "plain"), ("bf16", 257, 140003, 12, "plain"),
    ("f32", 256, 70001, 12, "plain"), ("bf16", 256, 300, 300, "plain"), ("bf16", 300, 5000, 200, "masked"),
    ("f32", 300, 2000, 700, "plain"), ("bf16", 300, 16385, 100, "masked"), ("f32", 1100, 900, 9, "masked"),
])
def test_distill_many_rows(dtype, n, v, k, kind, rest, form):
    """One workgroup a row, in every form of it: rows held in registers of 256 to 1024 threads, and read twice."""
    log(f"distill {n} {v} {k} {kind} {dtype} {rest} {form}")
    rng = np.random.default_rng([n, v, k])
    c = _distill_case(rng, n, v, k, dtype, "f32", rest, 2.0, kind)
    _check_distill(c, _distill_run(c, form), rows=sorted(set(rng.integers(0, n, 5)) | {0, 1, 3, n - 1}))


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,n,v,k", [
    ("bf16", 4, 5000, 129), ("f32", 4, 40000, 1024), ("bf16", 5, 9001, 128), ("f32", 258, 3000, 300),
    ("bf16", 257, 5000, 1024), ("bf16", 1030, 600, 200), ("f32", 1030, 300, 129), ("bf16", 256, 140003, 500),
])
def test_distill_many_pairs(dtype, n, v, k, rest, form):
    """Pairs that are compared by their tokens' hashes first, tokens in many of them."""
    log(f"distill many pairs {n} {v} {k} {dtype} {rest} {form}")
    rng = np.random.default_rng([n, v, k])
    c = _distill_case(rng, n, v, k, dtype, "f32", rest, 1.5, "twice")
    _check_distill(c, _distill_run(c, form), rows=sorted(set(rng.integers(0, n, 4)) | {0, 1, 2, n - 1}))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,v", [("bf16", 3001), ("f32", 20002), ("bf16", 140011), ("f32", 66001)])
def test_distill_rows_far_from_their_pairs(dtype, v, rest):
    """Rows whose sum does not fit relative to their pairs' largest logit: others far above it, all others far below
    it, masked by infinity or by the lowest value; next to ordinary rows."""
    log(f"distill far rows {dtype} {v} {rest}")
    rng = np.random.default_rng([v, rest])
    c = _distill_case(rng, 270, v, 6, dtype, rest=rest, tau=1.0)
    z = c["z64"].copy()
    top = np.zeros(z.shape, bool)
    np.put_along_axis(top, c["ids"], True, 1)
    z[0] += np.where(top[0], 0.0, 200.0)
    z[1] -= np.where(top[1], 0.0, 300.0)
    z[2] = np.where(top[2], z[2], -np.inf)
    z[2, np.flatnonzero(~top[2])[0]] = 1.0
    z[3] = np.where(top[3], -500.0, z[3])
    low = -3.3895313892515355e38
    z[4] = np.where(top[4], z[4], low)
    z[4, np.flatnonzero(~top[4])[5]] = -1.0
    z[5] += 1000.0
    z[6] -= 3.0e4
    z[7] = low
    bits = f32_to_bf16_bits(z.astype(np.float32)) if dtype == "bf16" else z.astype(np.float32)
    c["z64"], c["z"] = host_to_f64(bits, dtype), to_device(bits, dtype)
    c["g"][8] *= -1
    c["g64"][8] *= -1
    c["g"][9], c["g64"][9] = 0, 0
    for form in ("train", "step"):
        got = _distill_run(c, form)
        g = c["g64"]
        _check_distill(dict(c, g64=np.abs(g)), got[:3] + (_signed(got[3], g),),
                       rows=[r for r in range(12) if r != 9])
        assert not got[3][9].float().abs().any()


def _signed(dz, g):
    import torch
    return dz * torch.from_numpy(np.where(g < 0, -1.0, 1.0)).to(dz)[:, None]


def test_distill_same_bits():
    """In place, on another stream, a second time, and rows by themselves: the same bits (a row's own split apart)."""
    import torch
    log("distill bits")
    rng = np.random.default_rng(0)
    for n, v in ((3, 20000), (300, 9000), (260, 140011)):
        for rest in (False, True):
            c = _distill_case(rng, n, v, 11, "bf16", rest=rest, tau=1.3)
            for form in ("train", "step"):
                want = _distill_run(c, form)
                for got in (_distill_run(c, form), _distill_run(c, form, stream=torch.cuda.Stream()),
                            _distill_run(c, form, place=True)):
                    for a, b in zip(got, want):
                        assert a is b is None or torch.equal(a, b)
            c8 = dict(c, ids_d=c["ids_d"].long())
            for a, b in zip(_distill_run(c8, "train"), _distill_run(c, "train")):
                assert a is b is None or torch.equal(a, b)


def test_distill_nonfinite():
    """What the formulas give: a NaN or +inf logit makes its row NaN, a masked student token that the teacher wants an
    infinite loss, and a row is no other row's business."""
    import torch
    log("distill nonfinite")
    z = torch.zeros(5, 40, device="cuda")
    z[0, 30], z[1, 31], z[2, 5] = float("nan"), float("inf"), float("-inf")
    z[3] = float("-inf")
    ids = torch.tensor([[5, 6]], device="cuda").repeat(5, 1)
    t = torch.zeros(5, 2, device="cuda")
    for n in (5, 300):   # both forms
        zz = torch.zeros(n, 40, device="cuda")
        zz[:5] = z
        loss, lse, dz = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(zz)
        nsq.ns_distill_topk(zz, ids[:1].repeat(n, 1), t[:1].repeat(n, 1), loss, lse,
                            grad_loss=torch.ones(n, device="cuda"), dlogits=dz)
        torch.cuda.synchronize()
        assert torch.isnan(loss[[0, 1, 3]]).all() and loss[2] == float("inf") and torch.isfinite(loss[4:]).all()
        assert torch.isnan(dz[[0, 1, 3]]).any(1).all() and torch.isfinite(dz[[2, 4]]).all()
        assert dz[2, 5] == -0.5


def test_distill_offsets_past_32_bits():
    import torch
    log("distill far")
    ld = 2 ** 31 + 24
    buf = torch.empty(2 * ld + 2048, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (3, 1001), (ld, 1))
    rng = np.random.default_rng(4)
    c = _distill_case(rng, 3, 1001, 5, "bf16")
    z.copy_(c["z"])
    want = _distill_run(c, "train")
    loss, lse = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    nsq.ns_distill_topk(z, c["ids_d"], c["t"], loss, lse, grad_loss=c["g"], dlogits=z)
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(z, want[3])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_graph_replays():
    """Every operator captured into one graph; each replay, on new inputs with eager work between, gives eager's bits."""
    import torch
    log("graph")
    dev = "cuda"
    q, k = (torch.empty(2, 9, h, 64, device=dev, dtype=torch.bfloat16) for h in (4, 2))
    cos = torch.rand(9, 32, device=dev)
    x, y = torch.empty(200, 72, device=dev), torch.empty(400, 72, device=dev)
    big = torch.empty(9000, 8, device=dev, dtype=torch.int32)
    ids = torch.empty(200, 2, device=dev, dtype=torch.int32)
    z, t = torch.empty(4, 9000, device=dev), torch.empty(4, 6, device=dev)
    top = torch.arange(6, device=dev).repeat(4, 1)
    w, g = torch.rand(200, 2, device=dev), torch.rand(4, device=dev)
    i32 = dict(device=dev, dtype=torch.int32)
    outs = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k), torch.empty(64, device=dev),
            torch.empty(64, device=dev), torch.empty(17, **i32), torch.empty(400, **i32), torch.empty(200, 2, **i32),
            torch.empty_like(y), torch.empty_like(x), torch.empty_like(y), torch.empty(200, 2, device=dev),
            torch.empty_like(x), torch.empty(65, **i32), torch.empty(72000, **i32), torch.empty(9000, 8, **i32),
            torch.empty(4, device=dev), torch.empty(4, device=dev), torch.empty_like(z), torch.empty_like(z)]
    ws = [None, None, None, None]

    def step():
        nsq.ns_qk_norm_rope(q, k, outs[0], outs[1], cos=cos, sin=cos)
        ws[0] = nsq.ns_qk_norm_rope_backward(q, k, outs[0], outs[1], outs[2], outs[3], outs[4], outs[5], cos=cos, sin=cos,
                                             workspace=ws[0])
        ws[1] = nsq.ns_moe_sort(ids, 16, outs[6], outs[7], outs[8], workspace=ws[1])
        nsq.ns_moe_dispatch(x, outs[8], outs[9])
        nsq.ns_moe_combine(y, outs[8], w, outs[10])
        nsq.ns_moe_combine_backward(outs[10], y, outs[8], w, outs[11], outs[12])
        nsq.ns_moe_dispatch_backward(outs[11], outs[8], outs[13])
        ws[2] = nsq.ns_moe_sort(big, 64, outs[14], outs[15], outs[16], workspace=ws[2])
        ws[3] = nsq.ns_distill_topk(z, top, t, outs[17], outs[18], grad_loss=g, dlogits=outs[19], workspace=ws[3])
        nsq.ns_distill_topk_backward(z, top, t, outs[18], g, outs[20])

    def fill(seed):
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        for v in (q, k, x, y, z, t):
            v.normal_(generator=gen)
        ids.random_(-1, 16, generator=gen)
        big.random_(-1, 64, generator=gen)

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 5):
        fill(seed)
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in outs]
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), i


def test_binding_checks_shapes():
    import torch
    x = torch.zeros(2, 3, 4, 8, device="cuda")
    row = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    y = torch.zeros(4, 8, device="cuda")
    z, one = torch.zeros(4, 50, device="cuda"), torch.zeros(4, device="cuda")
    ids, t = torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.zeros(4, 3, device="cuda")
    for error, call in [
        (ValueError, lambda: nsq.ns_qk_norm_rope(x, None, x[:1], None)),
        (ValueError, lambda: nsq.ns_qk_norm_rope(x, None, None, None)),
        (ValueError, lambda: nsq.ns_qk_norm_rope(x, x[:, :2], x, x[:, :2])),
        (ValueError, lambda: nsq.ns_qk_norm_rope(x.transpose(2, 3), None, x.transpose(2, 3), None)),
        (TypeError, lambda: nsq.ns_qk_norm_rope(x.half(), None, x.half(), None)),
        (ValueError, lambda: nsq.ns_qk_norm_rope(x, None, x, None, q_weight=y[0, :4])),
        (TypeError, lambda: nsq.ns_qk_norm_rope(x, None, x, None, cos=y.double(), sin=y.double())),
        (ValueError, lambda: nsq.ns_qk_norm_rope(x, None, x, None, cos=y)),
        (ValueError, lambda: nsq.ns_qk_norm_rope(x, None, x, None, cos=y[:, :4].contiguous(), sin=y[:, :4].contiguous(), pos=row)),
        (nsq.NSError, lambda: nsq.ns_qk_norm_rope(x, None, x, None, cos=y, sin=y)),
        (TypeError, lambda: nsq.ns_moe_sort(row.float(), 4, row, row, row)),
        (ValueError, lambda: nsq.ns_moe_sort(row, 4, row[0], row.view(-1), row)),
        (ValueError, lambda: nsq.ns_moe_dispatch(y[:2], row, y[:3])),
        (TypeError, lambda: nsq.ns_moe_dispatch(y[:2], row, y.bfloat16())),
        (TypeError, lambda: nsq.ns_moe_dispatch(y[:2], row.long(), y)),
        (TypeError, lambda: nsq.ns_moe_combine(y, row, row, y[:2])),
        (ValueError, lambda: nsq.ns_moe_combine(y.t().contiguous().t(), row, None, y[:2])),
        (ValueError, lambda: nsq.ns_distill_topk(z, ids[:3], t, one, one)),
        (ValueError, lambda: nsq.ns_distill_topk(z, ids, t[:, :2], one, one)),
        (ValueError, lambda: nsq.ns_distill_topk(z, ids, t, one, one, grad_loss=one)),
        (ValueError, lambda: nsq.ns_distill_topk(z, ids, t, one, one, teacher_lse=one)),
        (TypeError, lambda: nsq.ns_distill_topk(z, ids, t, one.double(), one)),
        (nsq.NSError, lambda: nsq.ns_distill_topk(z, ids, t, one, one, temperature=0.0)),
        (nsq.NSError, lambda: nsq.ns_distill_topk(z, ids, t, one, one, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))),
    ]:
        with pytest.raises(error):
            call()
