"""The training-step example: its gradients against plain fp64 differentiation, and its loss over steps."""

import importlib.util
import os

import pytest

from tests.helpers import log

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_distill_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_distill_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain_loss(ex, m, p, tokens, ids, teacher, teacher_lse, tau, cos, sin):
    """The example's step in elementary fp64 operations on the CPU; p: its parameters there, by name."""
    import torch
    b, s = tokens.shape

    def turned(x, w):
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, c = n[..., :m.dim // 2], n[..., m.dim // 2:]
        cc, ss = cos[None, :, None], sin[None, :, None]
        return torch.cat((a * cc - c * ss, c * cc + a * ss), -1)

    x = p["embed"][tokens]
    q, k, v = ((x @ p[n].t()).view(b, s, -1, m.dim) for n in "qkv")
    q, k = turned(q, p["q_weight"]), turned(k, p["k_weight"])
    h = q.shape[2]
    k, v = (t.repeat_interleave(h // t.shape[2], dim=2) for t in (k, v))
    score = (q.transpose(1, 2) @ k.transpose(1, 2).transpose(2, 3)) / m.dim ** 0.5
    score = score.masked_fill(torch.ones(s, s, dtype=torch.bool).triu(1), float("-inf"))
    x = (x + (torch.softmax(score, -1) @ v.transpose(1, 2)).transpose(1, 2).reshape(b, s, -1) @ p["o"].t()).reshape(b * s, -1)
    top, choice = torch.topk(x @ p["router"].t(), m.top_k, dim=1)
    w = torch.softmax(top, 1)
    y = torch.stack([torch.nn.functional.silu(x @ u.t()) @ d.t() for u, d in zip(p["up"], p["down"])], 1)
    x = x + (w[:, :, None] * y.gather(1, choice[:, :, None].expand(-1, -1, x.shape[1]))).sum(1)
    z = x @ p["head"].t() / tau
    lse = torch.logsumexp(z, 1)
    rest = torch.logsumexp(z.scatter(1, ids, float("-inf")), 1)
    log_p = teacher / tau - teacher_lse[:, None]
    log_p = torch.cat((log_p, torch.log1p(-log_p.exp().sum(1, keepdim=True))), 1)
    log_q = torch.cat((z.gather(1, ids), rest[:, None]), 1) - lse[:, None]
    return (log_p.exp() * (log_p - log_q)).sum(1).mean()


def test_gradients_of_the_step():
    """f32 on the GPU against fp64: the products of a 256-wide block in fp32 leave about 1e-6 of a gradient's norm, its
    dozen operators in turn at most some tens of that."""
    import torch
    log("step gradients")
    ex = _example()
    m = ex.Student(vocab=300, hidden=64, heads=4, kv_heads=2, experts=5, top_k=2, ffn=48, dtype=torch.float32, seed=3)
    cos, sin = ex.angles(20, m.dim)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    tokens = torch.randint(0, 300, (2, 20), device="cuda", generator=gen)
    z = torch.randn(40, 300, device="cuda", generator=gen) * 3
    teacher, ids = torch.topk(z, 10, dim=1)
    lse = torch.logsumexp(z / 1.5, 1)
    loss = ex.backward(m, tokens, ids, teacher, lse, 1.5, cos, sin)
    torch.cuda.synchronize()
    names = ["embed", "q", "k", "v", "o", "q_weight", "k_weight", "router", "head"]
    p = {n: getattr(m, n).detach().cpu().double().requires_grad_() for n in names}
    for n in ("up", "down"):
        p[n] = [w.detach().cpu().double().requires_grad_() for w in getattr(m, n)]
    want = _plain_loss(ex, m, p, tokens.cpu(), ids.cpu(), teacher.cpu().double(), lse.cpu().double(), 1.5, cos.cpu().double(),
                       sin.cpu().double())
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    pairs = [(n, getattr(m, n), p[n]) for n in names]
    pairs += [(f"{n}[{i}]", g, w) for n in ("up", "down") for i, (g, w) in enumerate(zip(getattr(m, n), p[n]))]
    for name, got, ref in pairs:
        off = (got.grad.cpu().double() - ref.grad).norm() / ref.grad.norm().clamp_min(1e-30)
        assert off <= 1e-4, (name, off.item())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_the_example_trains(dtype):
    import torch
    log(f"example {dtype}")
    losses = _example().main(steps=12, dtype=getattr(torch, dtype), quiet=True)
    assert losses[-1] < 0.7 * losses[0] and all(x == x for x in losses)
