"""GPU tests of the training-step operators' binding: what autograd has to know of a call."""

import pytest

import newton_schulz_quintic_amd as nsq
from tests.helpers import log

pytestmark = pytest.mark.gpu


def _new(*shape, dtype=None):
    import torch
    return torch.zeros(shape, device="cuda", dtype=dtype or torch.float32)


def test_every_output_counts_as_written():
    """A tensor's version moves with each call that writes it, and no input's does."""
    import torch
    log("versions")
    i32 = torch.int32
    q, k, ids = _new(1, 3, 2, 8), _new(1, 3, 1, 8), _new(3, 2, dtype=i32)
    row, x, y = _new(3, 2, dtype=i32), _new(3, 16), _new(6, 16)
    row.copy_(torch.arange(6, device="cuda", dtype=i32).view(3, 2))
    w, z, t, g = _new(3, 2), _new(3, 20), _new(3, 2), _new(3)
    lse, rest = _new(3), _new(3)
    calls = [   # inputs, outputs, call
        ([q, k], [_new(1, 3, 2, 8), _new(1, 3, 1, 8)], lambda i, o: nsq.ns_qk_norm_rope(*i, *o)),
        ([q, k, _new(1, 3, 2, 8), _new(1, 3, 1, 8)], [_new(1, 3, 2, 8), _new(1, 3, 1, 8), _new(8), _new(8)],
         lambda i, o: nsq.ns_qk_norm_rope_backward(*i, *o)),
        ([ids], [_new(5, dtype=i32), _new(6, dtype=i32), _new(3, 2, dtype=i32)], lambda i, o: nsq.ns_moe_sort(i[0], 4, *o)),
        ([x, row], [_new(6, 16)], lambda i, o: nsq.ns_moe_dispatch(*i, *o)),
        ([y, row], [_new(3, 16)], lambda i, o: nsq.ns_moe_dispatch_backward(*i, *o)),
        ([y, row, w], [_new(3, 16)], lambda i, o: nsq.ns_moe_combine(*i, *o)),
        ([x, y, row, w], [_new(6, 16), _new(3, 2)], lambda i, o: nsq.ns_moe_combine_backward(*i, *o)),
        ([z, ids, t], [_new(3), _new(3)], lambda i, o: nsq.ns_distill_topk(*i, *o)),
        ([z, ids, t, g, lse], [_new(3), _new(3), _new(3), _new(3, 20)],
         lambda i, o: nsq.ns_distill_topk(*i[:3], *o[:2], teacher_lse=i[4], rest_lse=o[2], grad_loss=i[3], dlogits=o[3])),
        ([z, ids, t, lse, g, rest], [_new(3, 20)],
         lambda i, o: nsq.ns_distill_topk_backward(*i[:5], *o, teacher_lse=i[3], rest_lse=i[5])),
    ]
    for n, (ins, outs, call) in enumerate(calls):
        before = [v._version for v in ins + outs]
        call(ins, outs)
        after = [v._version for v in ins + outs]
        assert after[:len(ins)] == before[:len(ins)], n
        assert all(a > b for a, b in zip(after[len(ins):], before[len(ins):])), n
    torch.cuda.synchronize()
    with torch.inference_mode():   # tensors without a version
        a, b = _new(1, 3, 2, 8), _new(1, 3, 2, 8)
        nsq.ns_qk_norm_rope(a, None, b, None)
    nsq.ns_qk_norm_rope(q, None, b, None)
    torch.cuda.synchronize()


def test_backward_notices_a_saved_tensor_written_in_place():
    import torch
    log("saved in place")
    x = torch.randn(1, 3, 2, 8, device="cuda", requires_grad=True)
    y = x * 2
    loss = (y * y).sum()                 # saves y
    nsq.ns_qk_norm_rope(y.detach(), None, y.detach(), None)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    z = (torch.randn(4, 30, device="cuda", requires_grad=True) * 1.5).exp()   # saves its output
    ids, t, one = _new(4, 2, dtype=torch.int32), _new(4, 2), _new(4)
    nsq.ns_distill_topk(z.detach(), ids, t, _new(4), _new(4), grad_loss=one, dlogits=z.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()


@pytest.mark.parametrize("dtype", ["int32", "int64"])
def test_positions_shared_by_the_batch_and_in_wider_rows(dtype):
    """(1, seq) for a batch, an expanded row, rows of a wider tensor: the bits of whole (batch, seq) positions."""
    import torch
    log(f"positions {dtype}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    b, s = 3, 7
    q, g = (torch.randn(b, s, 2, 64, device="cuda", generator=gen) for _ in "qg")
    cos, sin = torch.rand(40, 32, device="cuda", generator=gen), torch.rand(40, 32, device="cuda", generator=gen)
    line = torch.randint(0, 40, (1, s), device="cuda", generator=gen).to(getattr(torch, dtype))
    rows = torch.randint(0, 40, (b, s + 5), device="cuda", generator=gen).to(getattr(torch, dtype))
    shared = line.expand(b, s).contiguous()
    for whole, forms in ((shared, [line, line[0], line.expand(b, s)]), (rows[:, 2:2 + s].contiguous(), [rows[:, 2:2 + s]])):
        want, dwant = torch.empty_like(q), torch.empty_like(q)
        nsq.ns_qk_norm_rope(q, None, want, None, cos=cos, sin=sin, pos=whole)
        nsq.ns_qk_norm_rope_backward(q, None, g, None, dwant, None, cos=cos, sin=sin, pos=whole)
        for pos in forms:
            got, dgot = torch.empty_like(q), torch.empty_like(q)
            nsq.ns_qk_norm_rope(q, None, got, None, cos=cos, sin=sin, pos=pos)
            nsq.ns_qk_norm_rope_backward(q, None, g, None, dgot, None, cos=cos, sin=sin, pos=pos)
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(dgot, dwant)
    for bad in (rows[:, ::2][:, :s], line[:, :s - 1], line.expand(b + 1, s), line.t()):
        with pytest.raises(ValueError, match="pos must"):
            nsq.ns_qk_norm_rope(q, None, want, None, cos=cos, sin=sin, pos=bad)
