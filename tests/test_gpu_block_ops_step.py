"""The operators around a block's products as they are used together: the training-step example with them, gradients
against fp64, captured graphs, and what autograd learns of a call."""

import importlib.util
import os

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from oracle import block_ops as ops
from tests.helpers import log

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_distill_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_distill_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _norm64(x, w):
    import torch
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _plain_loss(m, p, tokens, ids, teacher, teacher_lse, tau, cos, sin):
    """The example's step with its norms in elementary fp64 operations on the CPU."""
    import torch
    b, s = tokens.shape

    def turned(x, w):
        n = _norm64(x, w)
        a, c = n[..., :m.dim // 2], n[..., m.dim // 2:]
        cc, ss = cos[None, :, None], sin[None, :, None]
        return torch.cat((a * cc - c * ss, c * cc + a * ss), -1)

    wa, wo, we, wf, wh = p["norm_weights"]
    x = p["embed"][tokens].reshape(b * s, -1)
    h = _norm64(x, wa)
    q, k, v = ((h @ p[n].t()).view(b, s, -1, m.dim) for n in "qkv")
    q, k = turned(q, p["q_weight"]), turned(k, p["k_weight"])
    k, v = (t.repeat_interleave(q.shape[2] // t.shape[2], dim=2) for t in (k, v))
    score = (q.transpose(1, 2) @ k.transpose(1, 2).transpose(2, 3)) / m.dim ** 0.5
    score = score.masked_fill(torch.ones(s, s, dtype=torch.bool).triu(1), float("-inf"))
    y = (torch.softmax(score, -1) @ v.transpose(1, 2)).transpose(1, 2).reshape(b * s, -1) @ p["o"].t()
    x = x + p["gates"][0] * _norm64(y, wo)
    h = _norm64(x, we)
    top, choice = torch.topk(h @ p["router"].t(), m.top_k, dim=1)
    w = torch.softmax(top, 1)
    y = torch.stack([torch.nn.functional.silu(h @ u.t()) @ d.t() for u, d in zip(p["up"], p["down"])], 1)
    y = (w[:, :, None] * y.gather(1, choice[:, :, None].expand(-1, -1, x.shape[1]))).sum(1)
    z = _norm64(x + p["gates"][1] * _norm64(y, wf), wh) @ p["head"].t() / tau
    lse, rest = torch.logsumexp(z, 1), torch.logsumexp(z.scatter(1, ids, float("-inf")), 1)
    log_p = teacher / tau - teacher_lse[:, None]
    log_p = torch.cat((log_p, torch.log1p(-log_p.exp().sum(1, keepdim=True))), 1)
    log_q = torch.cat((z.gather(1, ids), rest[:, None]), 1) - lse[:, None]
    return (log_p.exp() * (log_p - log_q)).sum(1).mean()


def test_gradients_of_the_step_with_norms():
    """f32 on the GPU against fp64: products of a 64-wide block in fp32 leave about 1e-6 of a gradient's norm, its dozen
    operators in turn some tens of that; the norms after blocks divide by outputs of a tenth."""
    import torch
    log("step gradients with norms")
    ex = _example()
    m = ex.Student(vocab=300, hidden=64, heads=4, kv_heads=2, experts=5, top_k=2, ffn=48, dtype=torch.float32, seed=3, norms=True)
    cos, sin = ex.angles(20, m.dim)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    tokens = torch.randint(0, 300, (2, 20), device="cuda", generator=gen)
    z = torch.randn(40, 300, device="cuda", generator=gen) * 3
    teacher, ids = torch.topk(z, 10, dim=1)
    lse = torch.logsumexp(z / 1.5, 1)
    loss = ex.backward(m, tokens, ids, teacher, lse, 1.5, cos, sin)
    torch.cuda.synchronize()
    single, many = ["embed", "q", "k", "v", "o", "q_weight", "k_weight", "router", "head"], ["up", "down", "norm_weights", "gates"]
    p = {n: getattr(m, n).detach().cpu().double().requires_grad_() for n in single}
    p.update({n: [w.detach().cpu().double().requires_grad_() for w in getattr(m, n)] for n in many})
    want = _plain_loss(m, p, tokens.cpu(), ids.cpu(), teacher.cpu().double(), lse.cpu().double(), 1.5, cos.cpu().double(),
                       sin.cpu().double())
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    pairs = [(n, getattr(m, n), p[n]) for n in single]
    pairs += [(f"{n}[{i}]", g, w) for n in many for i, (g, w) in enumerate(zip(getattr(m, n), p[n]))]
    for name, got, ref in pairs:
        off = (got.grad.cpu().double() - ref.grad).norm() / ref.grad.norm().clamp_min(1e-30)
        assert off <= 1e-4, (name, off.item())


def test_gradients_of_expert_products():
    """Forward and gradients of the example's 8-bit products, from the values that the 8-bit forms stand for."""
    import torch
    log("expert products")
    ex = _example()
    at = [0, 70, 70, 260, 300]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    xs = torch.randn(300, 200, device="cuda", generator=gen, requires_grad=True)
    w = torch.randn(4, 90, 200, device="cuda", generator=gen, requires_grad=True)
    dy = torch.randn(300, 90, device="cuda", generator=gen)
    y = ex.ExpertProducts.apply(xs, w, torch.tensor(at, dtype=torch.int32, device="cuda"))
    y.backward(dy)
    torch.cuda.synchronize()
    f64 = lambda t: t.detach().cpu().numpy().astype(np.float64)  # noqa: E731
    stands = lambda t, tall: ops.value(*ops.quantize(t, tall))[:, :t.shape[1]]  # noqa: E731
    x64, dy64 = f64(xs), f64(dy)
    xq, dq = stands(x64, 1), stands(dy64, 1)
    for e, (a, b) in enumerate(zip(at, at[1:])):
        we = f64(w[e])
        wq, wqt = stands(we, 128), stands(we.T, 128)
        assert np.array_equal(wq.T, wqt)   # one set of scales serves both
        for got, left, right in ((y[a:b], xq[a:b], wq.T), (xs.grad[a:b], dq[a:b], wq)):
            tol = 2 * (4 * 2 + 64) * 2.0 ** -24 * (np.abs(left) @ np.abs(right))
            assert (np.abs(f64(got) - left @ right) <= tol + 2.0 ** -24 * np.abs(left @ right)).all()
        if a == b:
            assert not w.grad[e].any()
            continue
        left, right = stands(dy64[a:b].T, 1), stands(x64[a:b].T, 1).T
        tol = 2 * (4 * 2 + 64) * 2.0 ** -24 * (np.abs(left) @ np.abs(right))
        assert (np.abs(f64(w.grad[e]) - left @ right) <= tol + 2.0 ** -24 * np.abs(left @ right)).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_the_example_runs_with_everything(dtype):
    import torch
    log(f"example {dtype}")
    losses = _example().main(steps=3, dtype=getattr(torch, dtype), quiet=True, norms=True, eight_bit=True, max_norm=0.5)
    assert len(losses) == 3 and np.isfinite(losses).all()


def test_clipped_update_is_the_update_of_clipped_gradients():
    """muon_update with max_norm against torch's own arithmetic on a copy."""
    import torch
    log("clipped update")
    ex = _example()
    for max_norm in (0.3, 1e9):
        a, b = (ex.Student(vocab=50, hidden=64, heads=2, kv_heads=1, experts=2, top_k=1, ffn=48, dtype=torch.float32, seed=5) for _ in "ab")
        gen = torch.Generator(device="cuda")
        gen.manual_seed(2)
        grads = [torch.randn(p.shape, device="cuda", generator=gen) for p in a.muon_matrices() + a.others()]
        for m in (a, b):
            for p, g in zip(m.muon_matrices() + m.others(), grads):
                p.grad = g.clone()
        mus = [[torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)) for w in m.muon_matrices()] for m in (a, b)]
        norm = ex.muon_update(a, mus[0], lr=0.1, max_norm=max_norm)
        total = torch.sqrt(sum((g.double() ** 2).sum() for g in grads))
        c = min(1.0, (max_norm / (total + 1e-6)).item())
        for p in b.muon_matrices() + b.others():
            p.grad.mul_(c)
        assert ex.muon_update(b, mus[1], lr=0.1) is None
        torch.cuda.synchronize()
        assert abs(norm.item() - total.item()) <= 1e-6 * total.item()
        for x, y in zip(mus[0], mus[1]):
            assert torch.allclose(x, y, rtol=1e-5, atol=1e-6)
        for x, y in zip(a.muon_matrices() + a.others(), b.muon_matrices() + b.others()):
            assert torch.allclose(x, y, rtol=1e-3, atol=1e-4)


def test_a_captured_step():
    """Norms, quantization, products, their gradients, norm and clipping (a list of over 96 tensors) as one graph:
    every replay, on inputs of its own, gives the eager bits."""
    import torch
    log("captured step")
    rows, hidden, n, e = 400, 256, 200, 3
    dev = dict(device="cuda")
    b16 = torch.bfloat16
    x, y, gx, gh = (torch.empty(rows, hidden, dtype=b16, **dev) for _ in range(4))
    w = torch.empty(e, n, hidden, dtype=b16, **dev)
    gate, offsets = torch.empty(4, hidden, **dev), torch.empty(e + 1, dtype=torch.int32, **dev)
    small = [torch.empty(50 + i, **dev) for i in range(110)]
    p = (rows // 128 + e) * 128
    new8 = lambda *s: torch.empty(s, dtype=torch.float8_e4m3fn, **dev)  # noqa: E731
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, **dev)  # noqa: E731
    x_out, h, dx, dy = (torch.empty_like(x) for _ in range(4))
    dgate, dpre, dpost = torch.empty_like(gate), torch.empty(hidden, **dev), torch.empty(hidden, **dev)
    q, s, qt, st = new8(rows, hidden), u8(rows, 2), new8(hidden, p), u8(hidden, p // 128)
    wq, ws, wqt, wst = new8(e, n, hidden), u8(e, 2, 2), new8(e, hidden, 256), u8(e, 2, 2)
    out, gq, gs = torch.empty(rows, n, dtype=b16, **dev), new8(rows, 256), u8(rows, 2)
    gt, gst = new8(n, p), u8(n, p // 128)
    back, dw = torch.empty(rows, hidden, dtype=b16, **dev), torch.empty(e, n, hidden, **dev)
    norm, outs = torch.empty(1, **dev), [torch.empty_like(t) for t in small]
    rest = [torch.empty_like(dw)]
    bn_ws = u8(nsq.ns_block_norm_workspace_bytes(rows, hidden))
    mm_ws = u8(max(256, nsq.ns_scaled_matmul_workspace_bytes(n, hidden, p, e)))
    gr_ws = u8(nsq.ns_grad_workspace_bytes(len(small) + 1))

    def step():
        nsq.ns_block_norm(x, y, x_out, h, gate=gate, scale=0.5)
        nsq.ns_quantize(h, q, s, qt, st, offsets=offsets)
        nsq.ns_quantize(w, wq, ws, wqt, wst, block_rows=128)
        nsq.ns_scaled_matmul(q, s, wq, ws, out, offsets=offsets)
        nsq.ns_quantize(out, gq, gs, gt, gst, offsets=offsets)
        nsq.ns_scaled_matmul(gq, gs, wqt, wst, back, offsets=offsets)
        nsq.ns_scaled_matmul(gt, gst, qt, st, dw, offsets=offsets, reduce=True, workspace=mm_ws)
        nsq.ns_block_norm_backward(x, y, gx, back, dx, dy, dpost_weight=dpost, dpre_weight=dpre, dgate=dgate, gate=gate, scale=0.5,
                                   workspace=bn_ws)
        nsq.ns_grad_norm(small + [dw], norm, workspace=gr_ws)
        nsq.ns_grad_clip(small + [dw], outs + rest, norm=norm, max_norm=1.0, workspace=gr_ws)

    def fill(seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        for t in (x, y, gx, gh, w, gate, *small):
            t.copy_(torch.randn(t.shape, generator=gen, **dev))
        cut = torch.randint(0, rows + 1, (e - 1,), generator=gen, **dev).sort()[0]
        offsets.copy_(torch.tensor([0, *cut.tolist(), rows], dtype=torch.int32))
        out.zero_()
        back.zero_()
        qt.view(torch.uint8).zero_()   # what no group has a place in stays
        gt.view(torch.uint8).zero_()
        st.zero_()
        gst.zero_()

    results = [x_out, h, q, s, qt, st, out, back, dw, dx, dy, dpost, dpre, dgate, norm, *outs, *rest]
    bits = lambda t: t.view(torch.uint8) if t.dtype.itemsize == 1 else t  # noqa: E731
    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        fill(seed)
        step()
        torch.cuda.synchronize()
        want = [bits(t).clone() for t in results]
        fill(seed)
        for t in (x_out, dx, dw, norm, *outs):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, ref) in enumerate(zip(results, want)):
            assert torch.equal(bits(t), ref), (seed, i)


def test_every_output_counts_as_written():
    """A tensor's version moves with each call that writes it, and no input's does."""
    import torch
    log("versions")
    new = lambda *s, dtype=torch.float32: torch.zeros(s, device="cuda", dtype=dtype)  # noqa: E731
    u8, f8 = torch.uint8, torch.float8_e4m3fn
    x, y, w, gate = new(4, 128), new(4, 128), new(128), new(2, 128)
    q, s = new(4, 128, dtype=u8).view(f8), new(4, 1, dtype=u8)
    calls = [
        ([x, y, w, w.clone(), gate], [new(4, 128), new(4, 128)],
         lambda i, o: nsq.ns_block_norm(*i[:2], *o, post_weight=i[2], pre_weight=i[3], gate=i[4])),
        ([x, y, x.clone(), y.clone(), gate], [new(4, 128), new(4, 128), new(128), new(128), new(2, 128)],
         lambda i, o: nsq.ns_block_norm_backward(*i[:4], *o, gate=i[4])),
        ([x], [new(4, 128, dtype=u8).view(f8), new(4, 1, dtype=u8), new(128, 128, dtype=u8).view(f8), new(128, 1, dtype=u8)],
         lambda i, o: nsq.ns_quantize(*i, *o)),
        ([q, s], [new(4, 4)], lambda i, o: nsq.ns_scaled_matmul(*i, *i, *o)),
        ([x, y], [new(1), new(1, dtype=torch.float64)], lambda i, o: nsq.ns_grad_norm(i, *o)),
        ([x, y, w, w.clone(), new(1)], [new(4, 128), new(4, 128)],
         lambda i, o: nsq.ns_grad_clip(i[:2], o, norm=i[4], max_norm=1.0, momenta=[x.clone(), y.clone()], beta=0.5)),
    ]
    for n, (ins, outs, call) in enumerate(calls):
        before = [v._version for v in ins + outs]
        call(ins, outs)
        after = [v._version for v in ins + outs]
        assert after[:len(ins)] == before[:len(ins)], n
        assert all(a > b for a, b in zip(after[len(ins):], before[len(ins):])), n
    torch.cuda.synchronize()
