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


class BlockNorm(torch.autograd.Function):
    """(x + scale gate norm(y), its norm), or (x, norm of x) where y is None."""

    @staticmethod
    def forward(ctx, x, y, post_weight, pre_weight, gate, scale):
        h = torch.empty_like(x if y is None else y)
        x_out = None if y is None else torch.empty_like(x)
        ctx.scale = scale
        ctx.save_for_backward(x, y, post_weight, pre_weight, gate)
        nsq.ns_block_norm(x, y, x_out, h, post_weight=post_weight, pre_weight=pre_weight, gate=gate, scale=scale)
        return (x.view_as(x) if y is None else x_out), h

    @staticmethod
    def backward(ctx, dx_out, dh):
        x, y, post_weight, pre_weight, gate = ctx.saved_tensors
        new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        dx, dy, dpost, dpre, dgate = new(x), new(y), new(post_weight), new(pre_weight), new(gate)
        nsq.ns_block_norm_backward(x, y, None if y is None else dx_out.contiguous(), dh.contiguous(), dx, dy,
                                   dpost_weight=dpost, dpre_weight=dpre, dgate=dgate, post_weight=post_weight,
                                   pre_weight=pre_weight, gate=gate, scale=ctx.scale)
        return (dx + dx_out if y is None else dx), dy, dpost, dpre, dgate, None


def eight_bit(shape, rows: int = 1, device="cuda"):
    """Room for the 8-bit form of a (..., rows, cols) tensor: values and scales."""
    *lead, n, cols = shape
    blocks = -(-cols // 128)
    return (torch.empty(*lead, n, 128 * blocks, dtype=torch.float8_e4m3fn, device=device),
            torch.empty(*lead, -(-n // rows), blocks, dtype=torch.uint8, device=device))


class ExpertProducts(torch.autograd.Function):
    """Rows offsets[e] .. offsets[e + 1] of xs times w[e]^T in 8 bits; xs (rows, k), w (experts, n, k)."""

    @staticmethod
    def forward(ctx, xs, w, offsets):
        e, n, k = w.shape
        q, s = eight_bit(xs.shape)
        nsq.ns_quantize(xs, q, s)
        wq, ws = eight_bit(w.shape, 128)
        wqt, wst = eight_bit((e, k, n), 128)
        nsq.ns_quantize(w, wq, ws, wqt, wst, block_rows=128)
        y = xs.new_zeros(xs.shape[0], n)
        nsq.ns_scaled_matmul(q, s, wq, ws, y, offsets=offsets)
        ctx.save_for_backward(xs, wqt, wst, offsets)
        return y

    @staticmethod
    def backward(ctx, dy):
        xs, wqt, wst, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        (rows, n), k, e = dy.shape, xs.shape[1], offsets.numel() - 1
        tall = (rows // 128 + e) * 128
        q, s = eight_bit(dy.shape)
        qt, st = eight_bit((n, tall))
        xt, xst = eight_bit((k, tall))
        nsq.ns_quantize(dy, q, s, qt, st, offsets=offsets)
        nsq.ns_quantize(xs, None, None, xt, xst, offsets=offsets)
        dx = torch.zeros_like(xs)
        nsq.ns_scaled_matmul(q, s, wqt, wst, dx, offsets=offsets)
        dw = torch.empty(e, n, k, dtype=xs.dtype, device=xs.device)
        nsq.ns_scaled_matmul(qt, st, xt, xst, dw, offsets=offsets, reduce=True)
        return dx, dw, None


class Student:
    """The block's parameters; matrices in the step's dtype, norm weights and the router in fp32."""

    def __init__(self, vocab=1000, hidden=256, heads=4, kv_heads=2, experts=8, top_k=2, ffn=128, dtype=torch.bfloat16,
                 seed=0, device="cuda", norms=False, eight_bit=False):
        self.norms, self.eight_bit = norms, eight_bit
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
        if norms:   # before and after the attention and the experts, before the head; a gate per channel after each
            ones = lambda: torch.ones(hidden, device=device).requires_grad_()  # noqa: E731
            self.norm_weights = [ones() for _ in range(5)]
            self.gates = [torch.full((1, hidden), 0.5, device=device).requires_grad_() for _ in range(2)]

    def muon_matrices(self):
        return [self.q, self.k, self.v, self.o, *self.up, *self.down]

    def others(self):
        more = [*self.norm_weights, *self.gates] if self.norms else []
        return [self.embed, self.q_weight, self.k_weight, self.router, self.head, *more]


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


def experts(m: Student, x):
    """The experts' layer of the rows x, sorted by the router's choices and back."""
    top, ids = torch.topk(x.float() @ m.router.t(), m.top_k, dim=1)
    offsets = torch.empty(m.experts + 1, dtype=torch.int32, device=x.device)
    slot_of_row = torch.empty(ids.numel(), dtype=torch.int32, device=x.device)
    row_of_slot = torch.empty(ids.shape, dtype=torch.int32, device=x.device)
    nsq.ns_moe_sort(ids, m.experts, offsets, slot_of_row, row_of_slot)
    xs = Dispatch.apply(x, row_of_slot)
    if m.eight_bit:
        up = torch.nn.functional.silu(ExpertProducts.apply(xs, torch.stack(m.up), offsets))
        ys = ExpertProducts.apply(up, torch.stack(m.down), offsets)
    else:
        at = offsets.tolist()
        ys = torch.cat([torch.nn.functional.silu(xs[a:z] @ up.t()) @ down.t() for a, z, up, down in zip(at, at[1:], m.up, m.down)])
    return Combine.apply(ys, row_of_slot, torch.softmax(top, 1))


def logits_of(m: Student, tokens, cos, sin):
    b, s = tokens.shape
    x = m.embed[tokens].reshape(b * s, -1)
    before_attention, after_attention, before_experts, after_experts, before_head = m.norm_weights if m.norms else 5 * [None]
    h = BlockNorm.apply(x, None, None, before_attention, None, 1.0)[1] if m.norms else x
    q, k, v = ((h @ w.t()).view(b, s, -1, m.dim) for w in (m.q, m.k, m.v))
    q, k = QkNormRope.apply(q, k, m.q_weight, m.k_weight, cos, sin)
    y = (attention(q, k, v) @ m.o.t()).reshape(b * s, -1)
    if not m.norms:
        x = x + y
        return (x + experts(m, x)) @ m.head.t()
    x, h = BlockNorm.apply(x, y, after_attention, before_experts, m.gates[0], 1.0)
    x, h = BlockNorm.apply(x, experts(m, h), after_experts, before_head, m.gates[1], 1.0)
    return h @ m.head.t()


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


def muon_update(m: Student, momenta, lr: float, beta: float = 0.9, max_norm: float | None = None):
    """Momentum, its orthogonalization by Newton-Schulz, and the step on every Muon matrix; plain SGD on the rest.
    With max_norm all gradients are clipped by their common norm; returns that norm (None without)."""
    weights = m.muon_matrices()
    norm = None
    with torch.no_grad():
        if max_norm is not None:
            grads, rest = ([p.grad.contiguous() for p in ps] for ps in (weights, m.others()))
            norm = torch.empty(1, device=grads[0].device)
            workspace = nsq.ns_grad_norm(grads + rest, norm)
            nsq.ns_grad_clip(grads, momenta, norm=norm, max_norm=max_norm, momenta=momenta, beta=beta, workspace=workspace)
            nsq.ns_grad_clip(rest, rest, norm=norm, max_norm=max_norm, workspace=workspace)
            for p, g in zip(m.others(), rest):
                p.grad = g
        else:
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
    return norm


def main(steps: int = 20, dtype=torch.bfloat16, batch: int = 4, seq: int = 64, top: int = 32, temperature: float = 2.0,
         quiet: bool = False, norms: bool = False, eight_bit: bool = False, max_norm: float | None = None):
    """Trains a student on one teacher's top logits; returns the loss of each step."""
    student, teacher = Student(dtype=dtype, seed=0, norms=norms, eight_bit=eight_bit), Student(dtype=dtype, seed=1)
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
        muon_update(student, momenta, lr=0.02, max_norm=max_norm)
        losses.append(loss.item())
        if not quiet:
            print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--norms", action="store_true")
    ap.add_argument("--eight-bit", action="store_true")
    ap.add_argument("--max-norm", type=float)
    a = ap.parse_args()
    main(a.steps, {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype], norms=a.norms, eight_bit=a.eight_bit,
         max_norm=a.max_norm)
