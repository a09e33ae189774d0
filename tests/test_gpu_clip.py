"""GPU parity of ns_grad_norm and ns_grad_clip against the fp64 oracle (oracle/block_ops.py).

Tolerances, U = 2^-24: the sum of squares is added in 64 bits (a path of under 2^12 additions: 2^-41 of it), the norm
rounded once (U). c = max_norm / (norm + eps) adds a sum and a division: 3 U. An output adds two products and a sum: under
6 U (|beta m| + |c g|), and half a step of its type (2^-8 for bf16, U for f32).
"""

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from oracle import block_ops as ops
from tests.helpers import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _list(rng, counts, kinds, std=1.0):
    import torch
    return [torch.from_numpy((rng.standard_normal(n) * std).astype(np.float32)).cuda().to(_dtype(kinds[i % len(kinds)]))
            for i, n in enumerate(counts)]


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _norm(grads, **kw):
    import torch
    norm, sq = torch.full((1,), -1.0, device="cuda"), torch.full((1,), -1.0, device="cuda", dtype=torch.float64)
    nsq.ns_grad_norm(grads, norm, sum_sq=sq, **kw)
    torch.cuda.synchronize()
    return norm, sq


COUNTS = [[1], [0, 5, 0], [2048, 4096, 4097], [3] * 96, [7, 100, 5000] * 40, [70000], [1, 300001, 12], list(range(200)),
          [1 << 20, 999], [0] * 100 + [17], []]


@pytest.mark.parametrize("kinds", [("f32",), ("bf16",), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c, default=0)}")
def test_norm_and_clip(counts, kinds):
    import torch
    log(f"clip {len(counts)} {max(counts, default=0)} {kinds}")
    rng = np.random.default_rng(len(counts))
    grads = _list(rng, counts, kinds)
    norm, sq = _norm(grads)
    want = ops.grad_norm([_f64(g) for g in grads])
    assert abs(norm.item() - want) <= 1.01 * U * want and abs(sq.item() - want * want) <= 2.0 ** -40 * want * want
    for out_kinds in (kinds, ("f32",), ("bf16",)):
        for beta in (0.0, 0.9):
            outs = [torch.full((n,), float("nan"), device="cuda", dtype=_dtype(out_kinds[i % len(out_kinds)])) for i, n in enumerate(counts)]
            momenta = _list(rng, counts, out_kinds) if beta else None
            for max_norm in (0.5 * want, 2.0 * want + 1):
                nsq.ns_grad_clip(grads, outs, norm=norm, max_norm=max_norm, eps=1e-6, momenta=momenta, beta=beta)
                torch.cuda.synchronize()
                c, b = ops.clip_factor(want, np.float32(max_norm), 1e-6), float(np.float32(beta))
                for i, (g, o) in enumerate(zip(grads, outs)):
                    part = c * _f64(g)
                    m = b * _f64(momenta[i]) if beta else 0.0 * part
                    half = 2.0 ** -8 if o.dtype == torch.bfloat16 else U
                    tol = 6 * U * (np.abs(part) + np.abs(m)) + half * np.abs(part + m)
                    assert (np.abs(_f64(o) - part - m) <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_in_place(kind):
    """Over the gradients, and into the momentum: the bits of separate outputs; gradients under the norm stay."""
    import torch
    log(f"clip in place {kind}")
    rng = np.random.default_rng(1)
    counts = [5, 4096, 0, 9001] * 30
    grads, momenta = _list(rng, counts, (kind,)), _list(rng, counts, (kind,))
    norm, _ = _norm(grads)
    how = dict(norm=norm, max_norm=0.25)
    want, sums = [torch.empty_like(g) for g in grads], [torch.empty_like(g) for g in grads]
    nsq.ns_grad_clip(grads, want, **how)
    nsq.ns_grad_clip(grads, sums, momenta=momenta, beta=0.5, **how)
    nsq.ns_grad_clip(grads, momenta, momenta=momenta, beta=0.5, **how)
    kept = [g.clone() for g in grads]
    nsq.ns_grad_clip(grads, grads, **how)
    torch.cuda.synchronize()
    assert all(map(torch.equal, grads, want)) and all(map(torch.equal, momenta, sums))
    again = [g.clone() for g in kept]
    nsq.ns_grad_clip(again, again, norm=norm, max_norm=1e9)
    nsq.ns_grad_clip(again, again)
    torch.cuda.synchronize()
    assert all(map(torch.equal, again, kept))


def test_views_at_odd_addresses():
    """Tensors inside one buffer, at addresses aligned to their elements only; nothing beside them is written."""
    import torch
    log("clip views")
    for kind in ("bf16", "f32"):
        flat = torch.randn(40000, device="cuda").to(_dtype(kind))
        out = torch.full((40000,), 7.0, device="cuda").to(_dtype(kind))
        at = [(1, 3), (11, 4097), (5001, 1), (5003, 8191), (20001, 12000)]
        grads, outs = [flat[a:a + n] for a, n in at], [out[a:a + n] for a, n in at]
        norm, _ = _norm(grads)
        want = ops.grad_norm([_f64(g) for g in grads])
        assert abs(norm.item() - want) <= 1.01 * U * want
        nsq.ns_grad_clip(grads, outs, norm=norm, max_norm=1.0)
        torch.cuda.synchronize()
        mask = torch.ones(40000, dtype=torch.bool, device="cuda")
        for a, n in at:
            mask[a:a + n] = False
        assert (out[mask] == 7).all()
        for g, o in zip(grads, outs):
            part = ops.clip_factor(want, 1.0, 1e-6) * _f64(g)
            assert (np.abs(_f64(o) - part) <= 6 * U * np.abs(part) + (2.0 ** -8 if kind == "bf16" else U) * np.abs(part)).all()


def test_ends_of_the_range():
    """Squares past fp32's ends, zeros, and norms that are not finite."""
    import torch
    log("clip ends")
    for value, n in ((1e30, 1000), (1e-30, 1000), (3e38, 1), (0.0, 50), (1.2e-38, 4)):
        g = [torch.full((n,), value, device="cuda")]
        norm, sq = _norm(g)
        want = float(np.float64(np.float32(value)) * np.sqrt(n))
        assert abs(norm.item() - want) <= 1.01 * U * want
        o = [torch.empty_like(g[0])]
        nsq.ns_grad_clip(g, o, norm=norm, max_norm=1.0, eps=0.0)
        torch.cuda.synchronize()
        c = ops.clip_factor(want, 1.0, 0.0)
        assert np.abs(_f64(o[0]) - c * np.float64(np.float32(value))).max() <= 8 * U * c * value
    for bad in (float("inf"), float("nan")):
        g = [torch.ones(5000, device="cuda"), torch.ones(10, device="cuda")]
        g[0][4321] = bad
        norm, _ = _norm(g)
        assert not np.isfinite(norm.item())
        o = [torch.empty_like(x) for x in g]
        nsq.ns_grad_clip(g, o, norm=norm, max_norm=1.0)
        torch.cuda.synchronize()
        if np.isnan(bad):
            assert torch.isnan(o[0]).all() and torch.isnan(o[1]).all()
        else:
            assert torch.isnan(o[0][4321]) and (o[1] == 0).all()
    norm, sq = _norm([torch.full((2,), 3e38, device="cuda")])   # the norm itself is past fp32
    assert np.isinf(norm.item()) and np.isfinite(sq.item())


def test_same_bits_and_other_streams():
    import torch
    log("clip bits")
    rng = np.random.default_rng(2)
    grads = _list(rng, [12345, 678, 9] * 70, ("bf16", "f32"))
    first = _norm(grads)
    ws = torch.full((nsq.ns_grad_workspace_bytes(len(grads)),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = _norm(grads, workspace=ws, stream=side)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    only = torch.empty((), device="cuda")
    nsq.ns_grad_norm(tuple(grads), only)
    assert only.item() == first[0].item()


def test_large_lists():
    """Past the last-level cache, and a tensor of more than 2^31 bytes."""
    import torch
    log("clip large")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    g = [torch.randn(1_200_000_007, device="cuda", generator=gen, dtype=torch.bfloat16), torch.randn(3001, device="cuda", generator=gen)]
    want = sum((t[i:i + (1 << 27)].double() ** 2).sum().item() for t in g for i in range(0, t.numel(), 1 << 27)) ** 0.5
    norm, _ = _norm(g)
    assert abs(norm.item() - want) <= 1.1 * U * want
    o = [torch.empty_like(t) for t in g]
    nsq.ns_grad_clip(g, o, norm=norm, max_norm=1.0)
    torch.cuda.synchronize()
    c = ops.clip_factor(want, 1.0, 1e-6)
    for t, x in zip(g, o):
        for part in (slice(0, 5000), slice(t.numel() - 5000, t.numel())):
            ref = c * _f64(t[part])
            assert (np.abs(_f64(x[part]) - ref) <= (6 * U + (2.0 ** -8 if x.dtype == torch.bfloat16 else U)) * np.abs(ref)).all()


def test_refusals_of_the_binding():
    import torch
    log("clip refusals")
    x, n = torch.zeros(4, 6, device="cuda"), torch.zeros(1, device="cuda")
    for bad in (lambda: nsq.ns_grad_norm([x.t()], n), lambda: nsq.ns_grad_norm([x], None), lambda: nsq.ns_grad_norm([x], x),
                lambda: nsq.ns_grad_clip([x], []), lambda: nsq.ns_grad_clip([x], [x[:3]]), lambda: nsq.ns_grad_clip([x], [x], norm=n),
                lambda: nsq.ns_grad_clip([x], [x], beta=0.9), lambda: nsq.ns_grad_clip([x], [x], momenta=[x.bfloat16()], beta=0.9),
                lambda: nsq.ns_grad_clip([x], [x.cpu()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nsq.ns_grad_norm([x.half()], n), lambda: nsq.ns_grad_norm([x], n.double()), lambda: nsq.ns_grad_norm(x.numel(), n),
                lambda: nsq.ns_grad_clip([x], [x.int()])):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(nsq.NSError):
        nsq.ns_grad_clip([x], [x], norm=n, max_norm=-1.0)


def test_a_tensor_of_more_than_2_to_the_31():
    """Every value is reached: ones, whose squares are counted exactly, scaled in place by a power of two."""
    import torch
    log("huge tensor")
    n = (1 << 31) + 5001
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    norm, sq = _norm([g])
    assert sq.item() == n and abs(norm.item() - n ** 0.5) <= 1.01 * U * n ** 0.5
    two = torch.full((1,), 2.0, device="cuda")
    nsq.ns_grad_clip([g], [g], norm=two, max_norm=1.0, eps=0.0)
    torch.cuda.synchronize()
    assert (g == 0.5).all()
