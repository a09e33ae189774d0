"""One training step of a mixture-of-experts student, from a teacher's top logits to the Muon update.

A small transformer block: attention whose queries and keys are normed per head
and rotated (ns_qk_norm_rope), a layer of experts that its tokens are sorted to
and back (ns_moe_sort, ns_moe_dispatch, ns_moe_combine), and a loss against a
teacher's top logits whose gradient comes with it (ns_distill_topk). The matrix
products between are torch's. The gradients go into momentum matrices that
ns_orthogonalize_batched turns into updates, in the order ns_plan gives.

    python examples/moe_distill_step.py [--steps 20] [--dtype bf16|f32]
"""

from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import newton_schulz_quintic_amd as nsq  # noqa: E402


class QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin):
        q_out, k_out = torch.empty_like(q, memory_format=torch.contiguous_format), \
            torch.empty_like(k, memory_format=torch.contiguous_format)
        nsq.ns_qk_norm_rope(q, k, q_out, k_out, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin)
        return q_out, k_out

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cos, sin = ctx.saved_tensors
        dq, dk = torch.empty_like(dq_out, memory_format=torch.contiguous_format), \
            torch.empty_like(dk_out, memory_format=torch.contiguous_format)
        dqw, dkw = torch.empty_like(q_weight), torch.empty_like(k_weight)
        nsq.ns_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dq_weight=dqw, dk_weight=dkw, q_weight=q_weight,
                                     k_weight=k_weight, cos=cos, sin=sin)
        return dq, dk, dqw, dkw, None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_of_slot):
        ctx.save_for_backward(row_of_slot)
        xs = x.new_empty(row_of_slot.numel(), x.shape[1])
        nsq.ns_moe_dispatch(x, row_of_slot, xs)
        return xs

    @staticmethod
    def backward(ctx, dxs):
        row_of_slot, = ctx.saved_tensors
        dx = dxs.new_empty(row_of_slot.shape[0], dxs.shape[1])
        nsq.ns_moe_dispatch_backward(dxs.contiguous(), row_of_slot, dx)
        return dx, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, row_of_slot, weights):
        ctx.save_for_backward(y, row_of_slot, weights)
        out = y.new_empty(row_of_slot.shape[0], y.shape[1])
        nsq.ns_moe_combine(y, row_of_slot, weights, out)
        return out

    @staticmethod
    def backward(ctx, dout):
        y, row_of_slot, weights = ctx.saved_tensors
        dy, dweights = torch.empty_like(y), torch.empty_like(weights)
        nsq.ns_moe_combine_backward(dout.contiguous(), y, row_of_slot, weights, dy, dweights)
        return dy, None, dweights


class Student:
    """The block's parameters; matrices in the step's dtype, norm weights and the router in fp32."""

    def __init__(self, vocab=1000, hidden=256, heads=4, kv_heads=2, experts=8, top_k=2, ffn=128, dtype=torch.bfloat16,
                 seed=0, device="cuda"):
        self.heads, self.kv_heads, self.dim, self.top_k, self.experts = heads, kv_heads, hidden // heads, top_k, experts
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def matrix(*shape, dtype=dtype, std=None):
            w = torch.randn(shape, generator=gen, device=device) * (std or shape[-1] ** -0.5)
            return w.to(dtype).requires_grad_()

        self.embed = matrix(vocab, hidden, std=1.0)
        self.q, self.o = matrix(heads * self.dim, hidden), matrix(hidden, heads * self.dim)
        self.k, self.v = matrix(kv_heads * self.dim, hidden), matrix(kv_heads * self.dim, hidden)
        self.q_weight = torch.ones(self.dim, device=device).requires_grad_()
        self.k_weight = torch.ones(self.dim, device=device).requires_grad_()
        self.router = matrix(experts, hidden, dtype=torch.float32)
        self.up = [matrix(ffn, hidden) for _ in range(experts)]
        self.down = [matrix(hidden, ffn) for _ in range(experts)]
        self.head = matrix(vocab, hidden)

    def muon_matrices(self):
        return [self.q, self.k, self.v, self.o, *self.up, *self.down]

    def others(self):
        return [self.embed, self.q_weight, self.k_weight, self.router, self.head]


def angles(positions: int, dim: int, device="cuda"):
    """cos and sin of every position's angles, computed in fp64."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=device)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * 10000.0 ** (-2.0 * i / dim)
    return a.cos().float(), a.sin().float()


def attention(q, k, v):
    """Causal attention with shared key heads in elementary operations; (batch, seq, heads, dim)."""
    b, s, h, d = q.shape
    k, v = (t.repeat_interleave(h // t.shape[2], dim=2).float().transpose(1, 2).contiguous() for t in (k, v))
    scores = torch.matmul(q.float().transpose(1, 2), k.transpose(2, 3).contiguous()) / d ** 0.5
    later = torch.ones(s, s, dtype=torch.bool, device=q.device).triu(1)
    p = torch.softmax(scores.masked_fill(later, float("-inf")), -1)
    return torch.matmul(p, v).transpose(1, 2).reshape(b, s, h * d).to(q.dtype)


def logits_of(m: Student, tokens, cos, sin):
    b, s = tokens.shape
    x = m.embed[tokens]
    q, k, v = ((x @ w.t()).view(b, s, -1, m.dim) for w in (m.q, m.k, m.v))
    q, k = QkNormRope.apply(q, k, m.q_weight, m.k_weight, cos, sin)
    x = (x + attention(q, k, v) @ m.o.t()).reshape(b * s, -1)
    # the router's choices, sorted by expert
    top, ids = torch.topk(x.float() @ m.router.t(), m.top_k, dim=1)
    offsets = torch.empty(m.experts + 1, dtype=torch.int32, device=x.device)
    slot_of_row = torch.empty(ids.numel(), dtype=torch.int32, device=x.device)
    row_of_slot = torch.empty(ids.shape, dtype=torch.int32, device=x.device)
    nsq.ns_moe_sort(ids, m.experts, offsets, slot_of_row, row_of_slot)
    xs = Dispatch.apply(x, row_of_slot)
    at = offsets.tolist()
    ys = [torch.nn.functional.silu(xs[a:z] @ up.t()) @ down.t() for a, z, up, down in zip(at, at[1:], m.up, m.down)]
    x = x + Combine.apply(torch.cat(ys), row_of_slot, torch.softmax(top, 1))
    return x @ m.head.t()


def backward(m: Student, tokens, ids, teacher, teacher_lse, temperature, cos, sin):
    """Mean loss of the step, with every parameter's gradient left in .grad."""
    z = logits_of(m, tokens, cos, sin)
    n = z.shape[0]
    loss, lse, rest = (torch.empty(n, device=z.device) for _ in range(3))
    grad = torch.full((n,), 1.0 / n, device=z.device)
    dz = torch.empty_like(z)
    nsq.ns_distill_topk(z.detach(), ids, teacher, loss, lse, teacher_lse=teacher_lse, rest_lse=rest,
                        temperature=temperature, grad_loss=grad, dlogits=dz)
    z.backward(dz)
    return loss.mean()


def muon_update(m: Student, momenta, lr: float, beta: float = 0.9):
    """Momentum, its orthogonalization by Newton-Schulz, and the step on every Muon matrix; plain SGD on the rest."""
    weights = m.muon_matrices()
    with torch.no_grad():
        for w, mu in zip(weights, momenta):
            mu.mul_(beta).add_(w.grad)
        updates = [torch.empty_like(mu) for mu in momenta]
        order = nsq.ns_plan([tuple(w.shape) for w in weights])["order"]
        nsq.ns_orthogonalize_batched(momenta, updates, order=order)
        for w, u in zip(weights, updates):
            w.sub_(u, alpha=lr * max(1.0, w.shape[0] / w.shape[1]) ** 0.5)
            w.grad = None
        for p in m.others():
            p.sub_(p.grad, alpha=lr)
            p.grad = None


def main(steps: int = 20, dtype=torch.bfloat16, batch: int = 4, seq: int = 64, top: int = 32, temperature: float = 2.0,
         quiet: bool = False):
    """Trains a student on one teacher's top logits; returns the loss of each step."""
    student, teacher = Student(dtype=dtype, seed=0), Student(dtype=dtype, seed=1)
    cos, sin = angles(seq, student.dim)
    momenta = [torch.zeros_like(w) for w in student.muon_matrices()]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    tokens = torch.randint(0, student.embed.shape[0], (batch, seq), device="cuda", generator=gen)
    with torch.no_grad():   # what a teacher leaves behind: its top logits and its logsumexp
        z = 4.0 * logits_of(teacher, tokens, cos, sin).float()
        values, ids = torch.topk(z, top, dim=1)
        teacher_lse = torch.logsumexp(z / temperature, 1)
    losses = []
    for step in range(steps):
        loss = backward(student, tokens, ids, values, teacher_lse, temperature, cos, sin)
        muon_update(student, momenta, lr=0.02)
        losses.append(loss.item())
        if not quiet:
            print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    main(a.steps, {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype])
