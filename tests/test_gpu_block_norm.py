"""GPU parity of ns_block_norm and its gradient against the fp64 oracle (oracle/block_ops.py).

Tolerances count the roundings of the arithmetic, per value. U = 2^-24 is half a step of fp32; a stored result adds half
a step of its type (2^-8 of the value for bf16, 2^-24 for f32). With R = |alpha x| + |scale gate u w| the size of r:
 - a sum of squares has a path of at most 16 values a lane, 6 exchanges and 16 waves: 38 U; with its mean, eps, square
   root and division (half of their sum) ry is off by 24 U, and r by 30 U R (ry, four products, two fma).
 - rr is off by 24 U and by what r's error moves the mean square: 30 U K, K = mean(R^2) rr^2 (1 or more).
 - h = r rr w: 30 U R rr |w| + (24 + 30 K + 3) U |r| rr |w|, under 64 (1 + K) U R rr |w|.
 - backward: every term holds at most three factors of r rr, one mean (38 + 3 U) and six products; with the sizes
   taken over absolute values, R in the place of r, it is off by under 350 (1 + K) U.
 - sums over rows add a path of at most 16 rows a team here, 64 teams a lane and 32 lanes.
"""

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from oracle import block_ops as ops
from tests.helpers import host_to_f64, log, to_device
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}
PAD = 5   # elements around strided test tensors, to find writes outside them


def _values(rng, shape, dtype, std=1.0):
    """(array for to_device, its exact values)."""
    x = (rng.standard_normal(shape) * std).astype(np.float32)
    h = f32_to_bf16_bits(x) if dtype == "bf16" else x
    return h, host_to_f64(h, dtype)


def _tensor(bits, dtype, wide):
    """A device tensor, or rows of a wider one at an odd offset."""
    import torch
    t = to_device(bits, dtype)
    if not wide:
        return t
    big = torch.full((t.shape[0], t.shape[1] + 2 * PAD), float("nan"), dtype=t.dtype, device="cuda")
    return big[:, PAD:PAD + t.shape[1]].copy_(t)


def _clean(t):
    """Nothing was written beside a wide tensor's rows."""
    import torch
    b = t._base
    return b is None or bool(torch.isnan(b[:, :PAD]).all() and torch.isnan(b[:, PAD + t.shape[1]:]).all())


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol) & ~(got == want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.where(bad, np.abs(got - want) / (tol + 1e-300), 0)):.3g} x tol"


def _case(n, h, dtype, res, gates, post, wide=False, wdtype="f32", gdtype="f32", seed=0, y=True):
    rng = np.random.default_rng([n, h, gates or 0, post, seed])
    c = {"n": n, "h": h, "dtype": dtype, "res": res, "post": post, "alpha": 0.75, "scale": -1.25, "eps": 1e-5, "gdtype": gdtype}
    for name, d, std in (("x", res, 2.0), ("y", dtype, 3.0), ("gx", res, 1.0), ("gh", dtype, 1.0)):
        bits, c[name + "64"] = _values(rng, (n, h), d, std)
        c[name] = _tensor(bits, d, wide)
    for name in ("wp", "wn"):
        bits, c[name + "64"] = _values(rng, (h,), wdtype)
        c[name] = to_device(bits, wdtype)
    if not post:
        c["wp"] = c["wp64"] = None
    c["g"] = c["g64"] = None
    if gates is not None:
        bits, c["g64"] = _values(rng, (gates, h), gdtype)
        c["g"] = _tensor(bits, gdtype, wide)
    if not y:
        c["y"] = c["y64"] = c["wp"] = c["wp64"] = None
    return c


def _how(c):
    return dict(post_weight=c["wp"], pre_weight=c["wn"], gate=c["g"], post_norm=c["post"], alpha=c["alpha"], scale=c["scale"],
                eps=c["eps"])


def _sizes(c):
    """(R, u, rr, K, w_pre, gate scale w_post) over absolute values."""
    one = np.ones(c["h"])
    wn, wp = (np.abs(one if c[k] is None else c[k]) for k in ("wn64", "wp64"))
    r, _ = ops.block_norm(c["x64"], c["y64"], c["wp64"], c["wn64"], c["g64"], c["post"], c["alpha"], c["scale"], c["eps"])
    big, u, ry, f = np.abs(c["alpha"] * c["x64"]), 0.0, 1.0, 0.0
    if c["y64"] is not None:
        ry = 1 / np.sqrt(np.mean(c["y64"] ** 2, 1, keepdims=True) + c["eps"]) if c["post"] else 1.0
        u = np.abs(c["y64"]) * ry
        f = np.abs(c["scale"]) * wp * (1.0 if c["g64"] is None else ops.spread(np.abs(c["g64"]), c["n"]))
        big = big + f * u
    rr = 1 / np.sqrt(np.mean(r * r, 1, keepdims=True) + c["eps"])
    return big, u, rr, ry, np.mean(big * big, 1, keepdims=True) * rr * rr, wn, f


def _check_forward(c, x_out, h, what):
    want_r, want_h = ops.block_norm(c["x64"], c["y64"], c["wp64"], c["wn64"], c["g64"], c["post"], c["alpha"], c["scale"], c["eps"])
    big, _, rr, _, k, wn, _ = _sizes(c)
    if x_out is not None:
        _close(_f64(x_out), want_r, HALF_STEP[c["res"]] * np.abs(want_r) + 30 * U * big, what + " x_out")
        assert _clean(x_out)
    if h is not None:
        _close(_f64(h), want_h, HALF_STEP[c["dtype"]] * np.abs(want_h) + 64 * U * (1 + k) * big * rr * wn, what + " h")
        assert _clean(h)


def _check_backward(c, got, g64, gh64, what):
    want = ops.block_norm_backward(c["x64"], c["y64"], c["wp64"], c["wn64"], c["g64"], c["post"], c["alpha"], c["scale"],
                                   c["eps"], g64, gh64)
    big, u, rr, ry, k, wn, f = _sizes(c)
    zero = np.zeros((c["n"], c["h"]))
    ag, ah = (zero if t is None else np.abs(t) for t in (g64, gh64))
    n = big * rr
    dn = ah * wn
    dr = ag + rr * (dn + n * np.mean(dn * n, 1, keepdims=True))
    e = 350 * U * (1 + k)
    rows = (16 + 64 + 32) * U
    if got["dx"] is not None:
        _close(_f64(got["dx"]), want["dx"], HALF_STEP[c["res"]] * np.abs(want["dx"]) + e * abs(c["alpha"]) * dr, what + " dx")
        assert _clean(got["dx"])
    if got.get("dpre") is not None:
        _close(_f64(got["dpre"]), want["dw_pre"], np.sum((e + rows) * ah * n, 0), what + " dpre")
    if c["y64"] is None:
        return
    du = f * dr
    dy = ry * (du + u * np.mean(du * u, 1, keepdims=True)) if c["post"] else du
    if got["dy"] is not None:
        _close(_f64(got["dy"]), want["dy"], HALF_STEP[c["dtype"]] * np.abs(want["dy"]) + e * dy, what + " dy")
        assert _clean(got["dy"])
    wp = np.ones(c["h"]) if c["wp64"] is None else np.abs(c["wp64"])
    gate = 1.0 if c["g64"] is None else ops.spread(np.abs(c["g64"]), c["n"])
    if got.get("dpost") is not None:
        _close(_f64(got["dpost"]), want["dw_post"], np.sum((e + rows) * abs(c["scale"]) * gate * dr * u, 0), what + " dpost")
    if got.get("dgate") is not None:
        tol = ((e + rows) * abs(c["scale"]) * dr * u * wp).reshape(len(c["g64"]), -1, c["h"]).sum(1)
        _close(_f64(got["dgate"]), want["dgate"], HALF_STEP[c["gdtype"]] * np.abs(want["dgate"]) + tol, what + " dgate")
        assert _clean(got["dgate"])


def _like(t):
    import torch
    if t._base is None:
        return torch.full_like(t, float("nan"))
    return torch.full_like(t._base, float("nan"))[:, PAD:PAD + t.shape[1]]


def _backward(c, g=True, gh=True, sums=True, **kw):
    import torch
    dev = dict(device="cuda")
    got = {"dx": _like(c["x"]), "dy": None if c["y"] is None else _like(c["y"])}
    if sums:
        got["dpre"] = torch.full((c["h"],), float("nan"), **dev)
        got["dpost"] = torch.full((c["h"],), float("nan"), **dev) if c["post"] and c["y"] is not None else None
        got["dgate"] = None if c["g"] is None else _like(c["g"])
    nsq.ns_block_norm_backward(c["x"], c["y"], c["gx"] if g else None, c["gh"] if gh else None, got["dx"], got["dy"],
                               dpost_weight=got.get("dpost"), dpre_weight=got.get("dpre"), dgate=got.get("dgate"), **_how(c), **kw)
    torch.cuda.synchronize()
    return got


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("n,h,gates,post,wide", [
    (1, 1, None, True, False), (3, 7, 1, True, True), (5, 8, None, False, False), (4, 9, 2, True, True),
    (2, 130, 2, True, False), (6, 511, 3, True, True), (7, 512, 1, True, False), (5, 1000, 5, True, True),
    (9, 1024, 1, False, False), (4, 1025, 2, True, False), (6, 2047, None, True, True), (3, 4096, 3, True, False),
    (5, 4099, 1, True, True), (2, 8192, 1, True, False), (3, 9001, 3, True, False), (2, 16384, 2, True, False)])
def test_block_norm(n, h, gates, post, wide, dtype, res):
    import torch
    log(f"block norm {n} {h} {gates} {post} {wide} {dtype} {res}")
    c = _case(n, h, dtype, res, gates, post, wide)
    x_out, out = _like(c["x"]), _like(c["y"])
    nsq.ns_block_norm(c["x"], c["y"], x_out, out, **_how(c))
    torch.cuda.synchronize()
    _check_forward(c, x_out, out, "forward")
    _check_backward(c, _backward(c), c["gx64"], c["gh64"], "backward")


@pytest.mark.parametrize("n,h,gates", [(700, 96, 1), (700, 96, 7), (1400, 40, 700), (1500, 64, 1500), (2049, 33, 3),
                                       (1200, 2304, 2), (600, 5000, 1), (520, 4096, 260), (1100, 600, 1100), (12000, 24, 12)])
def test_rows_dealt_to_teams(n, h, gates):
    """Many rows: whole gate rows a team, several teams a gate row, runs that end early."""
    import torch
    log(f"block rows {n} {h} {gates}")
    c = _case(n, h, "bf16", "f32", gates, True, gdtype="bf16" if gates == n else "f32")
    x_out, out = _like(c["x"]), _like(c["y"])
    nsq.ns_block_norm(c["x"], c["y"], x_out, out, **_how(c))
    torch.cuda.synchronize()
    _check_forward(c, x_out, out, "forward")
    _check_backward(c, _backward(c), c["gx64"], c["gh64"], "backward")


@pytest.mark.parametrize("y", [False, True])
def test_parts_left_out(y):
    """The norm in front of the first block, the last block's end, weights and gates of ones, gradients of one output."""
    import torch
    log(f"block parts {y}")
    c = _case(6, 300, "bf16", "f32", 2 if y else None, True, wdtype="bf16", gdtype="bf16", y=y)
    out = torch.empty(6, 300, dtype=torch.bfloat16, device="cuda")
    nsq.ns_block_norm(c["x"], c["y"], None, out, **_how(c))
    _check_forward(c, None, out, "h alone")
    if y:
        x_out = _like(c["x"])
        nsq.ns_block_norm(c["x"], c["y"], x_out, None, **_how(c))
        _check_forward(c, x_out, None, "x_out alone")
        _check_backward(c, _backward(c, gh=False), c["gx64"], None, "no dh")
        _check_backward(c, _backward(c, sums=False), c["gx64"], c["gh64"], "no sums")
    _check_backward(c, _backward(c, g=False), None, c["gh64"], "no dx_out")
    for k in ("wp", "wn", "g"):
        c[k] = c[k + "64"] = None
    nsq.ns_block_norm(c["x"], c["y"], None, out, **_how(c))
    _check_forward(c, None, out, "ones")
    _check_backward(c, _backward(c, g=False), None, c["gh64"], "ones")


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("h", [13, 1537, 4099])
def test_in_place(h, post):
    """Over the inputs, with and without a norm in front of the stores: the bits of separate outputs."""
    import torch
    log(f"block in place {h} {post}")
    c = _case(40, h, "bf16", "bf16", 4, post)
    want = [_like(c["x"]), _like(c["y"])]
    nsq.ns_block_norm(c["x"], c["y"], *want, **_how(c))
    for with_h in (True, False):
        x, y = c["x"].clone(), c["y"].clone()
        nsq.ns_block_norm(x, y, x, y if with_h else None, **_how(c))
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1] if with_h else c["y"])
    sums = _backward(c)
    gx, gh = c["gx"].clone(), c["gh"].clone()
    nsq.ns_block_norm_backward(c["x"], c["y"], gx, gh, gx, gh, **_how(c))
    torch.cuda.synchronize()
    assert torch.equal(gx, sums["dx"]) and torch.equal(gh, sums["dy"])
    x, y = c["x"].clone(), c["y"].clone()
    dgate = _like(c["g"])
    nsq.ns_block_norm_backward(x, y, c["gx"], c["gh"], x, y, dgate=dgate, **_how(c))
    torch.cuda.synchronize()
    assert torch.equal(x, sums["dx"]) and torch.equal(y, sums["dy"]) and torch.equal(dgate, sums["dgate"])


def test_rows_of_zeros_and_what_is_not_finite():
    """A row of zeros has h 0 and finite gradients; infinities and NaN stay in their row."""
    import torch
    log("block odd rows")
    c = _case(6, 200, "bf16", "bf16", None, True)
    x, y = c["x"].clone(), c["y"].clone()
    x[1], y[1] = 0, 0
    x[3, 5], y[4, 7] = float("nan"), float("inf")
    x_out, out = torch.empty_like(x), torch.empty_like(y)
    nsq.ns_block_norm(x, y, x_out, out, **_how(c))
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    nsq.ns_block_norm_backward(x, y, c["gx"], c["gh"], dx, dy, **_how(c))
    torch.cuda.synchronize()
    assert (x_out[1] == 0).all() and (out[1] == 0).all() and torch.isfinite(dx[1]).all() and torch.isfinite(dy[1]).all()
    good = [0, 1, 2, 5]
    for t in (x_out, out, dx, dy):
        assert torch.isfinite(t[good].float()).all()
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[4].float()).any()


def test_no_rows():
    import torch
    log("block no rows")
    z = torch.empty(0, 64, device="cuda")
    nsq.ns_block_norm(z, z, z.clone(), z.clone(), gate=torch.ones(1, 64, device="cuda"))
    for gates in (0, 1, 3):
        dp, dn, g = torch.ones(64, device="cuda"), torch.ones(64, device="cuda"), torch.ones(gates, 64, device="cuda")
        dg = torch.ones_like(g)
        nsq.ns_block_norm_backward(z, z, z, z, z.clone(), z.clone(), dpost_weight=dp, dpre_weight=dn, dgate=dg, gate=g)
        torch.cuda.synchronize()
        assert not dp.any() and not dn.any() and not dg.any()


def test_same_bits_and_other_streams():
    import torch
    log("block bits")
    c = _case(3000, 640, "bf16", "bf16", 3, True)
    first, ws = _backward(c), torch.empty(nsq.ns_block_norm_workspace_bytes(3000, 640), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)   # NaN patterns: a workspace may hold anything
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = _backward(c, workspace=ws, stream=side)
    side.synchronize()
    for k, v in first.items():
        assert torch.equal(v, again[k]), k


def test_refusals_of_the_binding():
    import torch
    log("block refusals")
    x = torch.zeros(4, 64, device="cuda")
    b = x.bfloat16()
    w = torch.ones(64, device="cuda")
    for bad in (lambda: nsq.ns_block_norm(x[0], x, x, x), lambda: nsq.ns_block_norm(x, x[:3], x, x),
                lambda: nsq.ns_block_norm(x, None, x, x), lambda: nsq.ns_block_norm(x, x, None, None),
                lambda: nsq.ns_block_norm(x, x, x, x, pre_weight=w[:5]), lambda: nsq.ns_block_norm(x, x, x, x, post_weight=w.bfloat16(), pre_weight=w),
                lambda: nsq.ns_block_norm(x, x, x.t()[:4], x), lambda: nsq.ns_block_norm(x, x, x[:, ::2], x),
                lambda: nsq.ns_block_norm(x, x, x, x, gate=w), lambda: nsq.ns_block_norm_backward(x, x, None, None, x, x),
                lambda: nsq.ns_block_norm_backward(x, None, x, x, x, None), lambda: nsq.ns_block_norm_backward(x, x, x, x, x, x, dgate=x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        nsq.ns_block_norm(x, b, x, x)
    for bad in (lambda: nsq.ns_block_norm(x, x, x, x, gate=x[:3]), lambda: nsq.ns_block_norm(b, x, b, x),
                lambda: nsq.ns_block_norm(x, x, x, x, post_weight=w, post_norm=False), lambda: nsq.ns_block_norm(x, x, x, x, eps=-1.0)):
        with pytest.raises(nsq.NSError):
            bad()


def test_rows_further_apart_than_32_bits():
    """Every tensor's rows 2^31 elements apart: the bits of a call on rows that lie together."""
    import torch
    log("far rows")
    h = 1000
    c = _case(3, h, "bf16", "bf16", 3, True)
    names = ("x", "y", "gx", "gh", "x_out", "h_out", "dx", "dy")
    big = torch.empty((2 << 31) + 8 * h, dtype=torch.bfloat16, device="cuda").as_strided((3, 8 * h), (1 << 31, 1))
    big.fill_(float("nan"))
    far = {name: big[:, i * h:(i + 1) * h] for i, name in enumerate(names)}
    near = {name: torch.full((3, h), float("nan"), dtype=torch.bfloat16, device="cuda") for name in names}
    sums = []
    for t in (near, far):
        for name in names[:4]:
            t[name].copy_(c[name])
        nsq.ns_block_norm(t["x"], t["y"], t["x_out"], t["h_out"], **_how(c))
        sums.append([torch.empty(h, device="cuda"), torch.empty(h, device="cuda"), torch.empty_like(c["g"])])
        nsq.ns_block_norm_backward(t["x"], t["y"], t["gx"], t["gh"], t["dx"], t["dy"], *sums[-1], **_how(c))
    torch.cuda.synchronize()
    assert all(torch.equal(near[name], far[name]) for name in names)
    assert all(torch.equal(a, b) for a, b in zip(*sums))
