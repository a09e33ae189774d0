"""Cases that measure the training-step operators around the Newton-Schulz update.

Three operators and their gradients: the per-head norm of queries and keys with
the position rotation (ns_qk_norm_rope), tokens sorted by expert and back
(ns_moe_sort, ns_moe_dispatch, ns_moe_combine), and the loss against a teacher's
top logits (ns_distill_topk). ``run`` computes them in elementary torch
operations while ``own`` is false, and with this package's entry points while it
is true; ``exact`` gives the same outputs from the definitions in 64 bits.

Sizes: the heads are those of the dense-transformer set (hidden 4096, keys and
values 1024: 32 and 8 heads of 128), the experts those of the many-small set
(64 experts, hidden 7168); the others are generic.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _qk(name, do, batch, seq, q_heads, k_heads, head_dim, rope_dim, pairs, dtype, layout, table):
    return {"name": name, "op": "qk", "do": do, "batch": batch, "seq": seq, "q_heads": q_heads, "k_heads": k_heads,
            "head_dim": head_dim, "rope_dim": rope_dim, "pairs": pairs, "dtype": dtype, "layout": layout,
            "table": table}


def _moe(name, do, tokens, top_k, experts, hidden, dtype, dropped):
    return {"name": name, "op": "moe", "do": do, "tokens": tokens, "top_k": top_k, "experts": experts,
            "hidden": hidden, "dtype": dtype, "dropped": dropped}


def _distill(name, do, rows, vocab, top_k, dtype, rest, empty, temperature):
    return {"name": name, "op": "distill", "do": do, "rows": rows, "vocab": vocab, "top_k": top_k, "dtype": dtype,
            "rest": rest, "empty": empty, "temperature": temperature}


def listed():
    return [
        # one new token for each of 16 sequences, far into their contexts: latency
        _qk("qk decode", "forward", 16, 1, 32, 8, 128, 128, "halves", "bf16", "fused", 131072),
        # a training micro-batch, queries and keys read out of the fused projection's output
        _qk("qk train forward", "forward", 4, 4096, 32, 8, 128, 128, "halves", "bf16", "fused", 4096),
        _qk("qk train backward", "backward", 4, 4096, 32, 8, 128, 128, "halves", "bf16", "fused", 4096),
        # heads before tokens, neighbouring pairs, a part of each head rotated, an odd length, all in fp32
        _qk("qk odd step f32", "step", 3, 1027, 12, 3, 96, 64, "neighbours", "f32", "heads first", 2048),
        # eight tokens being decoded: sort, gather and combine are three short launches
        _moe("moe decode", "forward", 8, 8, 64, 7168, "bf16", 0.0),
        # the sort by itself over many experts and a long batch
        _moe("moe sort", "sort", 65536, 8, 256, 0, "bf16", 0.0),
        # a training micro-batch of the many-small set's expert layer, both directions
        _moe("moe train forward", "forward", 8192, 8, 64, 7168, "bf16", 0.0),
        _moe("moe train backward", "backward", 8192, 8, 64, 7168, "bf16", 0.0),
        # odd counts and an odd width in fp32, some slots over capacity and dropped
        _moe("moe ragged step f32", "step", 3001, 3, 17, 1537, "f32", 0.1),
        # a few rows of a long vocabulary: the work has to be split along the row
        _distill("distill few rows", "train", 4, 131072, 32, "bf16", False, 0, 1.0),
        # a training micro-batch: loss and gradient in one call
        _distill("distill train", "train", 4096, 131072, 64, "bf16", False, 0, 2.0),
        # an odd vocabulary in fp32 with the teacher's remaining mass and padded rows; forward, then backward
        _distill("distill odd step f32", "step", 1025, 50021, 20, "f32", True, 100, 1.5),
    ]


def _log(rng, lo, hi):
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return n if n % 1024 else n + 1   # the listed cases have the round sizes


def draw(rng):
    op = rng.choice(["qk", "moe", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "qk":
        k_heads = rng.choice([1, 2, 3, 4, 8])
        q_heads = k_heads * rng.choice([1, 2, 4, 5, 8])
        head_dim = rng.choice([64, 72, 96, 128, 128, 192, 256])
        rope_dim = rng.choice([head_dim, head_dim, head_dim // 2])
        batch = rng.randint(1, 8)
        most = 600_000_000 // (5 * (q_heads + k_heads) * head_dim * _BYTES[dtype] * batch)
        seq = _log(rng, 1, max(1, min(16384, most)))
        layout = rng.choice(["fused", "tokens first", "heads first"])
        c = _qk("", rng.choice(["forward", "backward", "step"]), batch, seq, q_heads, k_heads, head_dim, rope_dim,
                rng.choice(["halves", "halves", "neighbours"]), dtype, layout, rng.choice([16384, 65536]))
    elif op == "moe":
        experts = _log(rng, 4, 384)
        top_k = min(experts, rng.choice([1, 2, 3, 4, 6, 8]))
        hidden = _log(rng, 256, 8192)
        hidden = 64 * (hidden // 128 * 2 + 1) if rng.random() < 0.75 else hidden | 1
        most = 2_500_000_000 // (5 * (top_k + 1) * hidden * _BYTES[dtype])
        c = _moe("", rng.choice(["forward", "backward", "step", "sort"]), _log(rng, 1, min(32768, most)), top_k,
                 experts, hidden, dtype, rng.choice([0.0, 0.0, 0.05]))
        if c["do"] == "sort":
            c["hidden"], c["tokens"] = 0, _log(rng, 1, 65536)
    else:
        vocab = _log(rng, 8192, 200000)
        if rng.random() < 0.7:
            vocab = -(-vocab // 64) * 64
        most = 2_000_000_000 // (4 * vocab * _BYTES[dtype])
        rows = _log(rng, 1, min(8192, most))
        c = _distill("", rng.choice(["forward", "train", "step"]), rows, vocab, _log(rng, 4, 128), dtype,
                     rng.random() < 0.4, rows // 10 if rng.random() < 0.3 else 0, rng.choice([1.0, 1.5, 2.0, 4.0]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"qk": _prepare_qk, "moe": _prepare_moe, "distill": _prepare_distill}[case["op"]](case, gen)


def _randn(gen, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _heads(case, heads, gen):
    """One (batch, seq, heads, head_dim) tensor in the case's memory order."""
    b, s, d, t = case["batch"], case["seq"], case["head_dim"], _DTYPES[case["dtype"]]
    if case["layout"] == "heads first":
        x = torch.empty(b, heads, s, d, dtype=t, device="cuda").transpose(1, 2)
    else:
        x = torch.empty(b, s, heads, d, dtype=t, device="cuda")
    return x if gen is None else x.copy_(torch.randn(b, s, heads, d, generator=gen, device="cuda"))


def _prepare_qk(case, gen):
    b, s, hq, hk, d = case["batch"], case["seq"], case["q_heads"], case["k_heads"], case["head_dim"]
    dtype, half, rows = _DTYPES[case["dtype"]], case["rope_dim"] // 2, case["table"]
    st = {"case": case}
    if case["layout"] == "fused":   # views of one projection's output [q | k | v]
        qkv = _randn(gen, (b, s, (hq + 2 * hk) * d), dtype)
        st["q"] = qkv[..., :hq * d].view(b, s, hq, d)
        st["k"] = qkv[..., hq * d:(hq + hk) * d].view(b, s, hk, d)
    else:
        st["q"], st["k"] = _heads(case, hq, gen), _heads(case, hk, gen)
    st["q_weight"] = 1.0 + _randn(gen, (d,), std=0.1)
    st["k_weight"] = 1.0 + _randn(gen, (d,), std=0.1)
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] \
        * 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
    first = torch.randint(0, rows - s + 1, (b, 1), generator=gen, device="cuda")
    st["pos"] = (first + torch.arange(s, device="cuda")).to(torch.int32)
    st["q_out"], st["k_out"] = _heads(case, hq, None), _heads(case, hk, None)
    if case["do"] != "forward":
        st["dq_out"], st["dk_out"] = _heads(case, hq, gen), _heads(case, hk, gen)
        st["dq"], st["dk"] = _heads(case, hq, None), _heads(case, hk, None)
        st["dq_weight"] = torch.empty(d, device="cuda")
        st["dk_weight"] = torch.empty(d, device="cuda")
    return st


def _prepare_moe(case, gen):
    t, k, e, h, dtype = case["tokens"], case["top_k"], case["experts"], case["hidden"], _DTYPES[case["dtype"]]
    st = {"case": case}
    # router scores with a favourite expert or two, as real ones have
    score = torch.randn(t, e, generator=gen, device="cuda") + _randn(gen, (e,), std=0.7)
    top, ids = torch.topk(score, k, dim=1)
    if case["dropped"]:
        ids = torch.where(torch.rand(t, k, generator=gen, device="cuda") < case["dropped"], -1, ids)
    st["ids"] = ids.to(torch.int32)
    st["weights"] = torch.exp(top) / torch.exp(top).sum(1, keepdim=True)
    st["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
    st["slot_of_row"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
    st["row_of_slot"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
    if case["do"] == "sort":
        return st
    new = lambda rows: torch.empty(rows, h, dtype=dtype, device="cuda")  # noqa: E731
    st["y"] = _randn(gen, (t * k, h), dtype)
    if case["do"] != "backward":
        st["x"] = _randn(gen, (t, h), dtype)
        st["xs"], st["out"] = new(t * k), new(t)
    if case["do"] != "forward":
        st["dout"], st["dxs"] = _randn(gen, (t, h), dtype), _randn(gen, (t * k, h), dtype)
        st["dy"], st["dx"] = new(t * k), new(t)
        st["dweights"] = torch.empty(t, k, device="cuda")
    if case["do"] == "backward":   # the forward pass kept its rows
        st["row_of_slot"] = _sort_plain(st["ids"], e)[2]
    return st


def _prepare_distill(case, gen):
    n, v, k, dtype = case["rows"], case["vocab"], case["top_k"], _DTYPES[case["dtype"]]
    inv = 1.0 / case["temperature"]
    st = {"case": case}
    # distinct tokens in no order; the student's logits stand out at most of them
    first = torch.randint(0, v, (n, 1), generator=gen, device="cuda")
    step = torch.randint(1, max(2, v // k), (n, 1), generator=gen, device="cuda")
    ids = (first + torch.arange(k, device="cuda") * step) % v
    top = 10.0 + 5.0 * torch.rand(n, k, generator=gen, device="cuda").sort(dim=1, descending=True)[0]
    logits = torch.randn(n, v, generator=gen, device="cuda", dtype=dtype) * 2.0
    logits.scatter_add_(1, ids, (top + _randn(gen, (n, k))).to(dtype))
    st["logits"], st["teacher"] = logits, top.to(dtype)
    if case["empty"]:   # padded positions have no teacher
        ids[torch.randperm(n, generator=gen, device="cuda")[:case["empty"]]] = -1
    st["ids"] = ids.to(torch.int32)
    st["teacher_lse"] = None
    if case["rest"]:   # the teacher's logsumexp over its whole vocabulary
        rest = torch.rand(n, generator=gen, device="cuda")
        st["teacher_lse"] = torch.logsumexp(st["teacher"].float() * inv, 1) + 0.01 + 0.5 * rest
    st["grad_loss"] = torch.rand(n, generator=gen, device="cuda") / n
    st["loss"], st["lse"] = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    st["rest_lse"] = torch.empty(n, device="cuda") if case["rest"] else None
    st["dlogits"] = torch.empty_like(logits) if case["do"] != "forward" else None
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return {"qk": _own_qk, "moe": _own_moe, "distill": _own_distill}[case["op"]](state, case["do"])
    return {"qk": _plain_qk, "moe": _plain_moe, "distill": _plain_distill}[case["op"]](state, case["do"])


def _own_qk(st, do):
    import newton_schulz_quintic_amd as nsq
    out, neighbours = {}, st["case"]["pairs"] == "neighbours"
    if do != "backward":
        nsq.ns_qk_norm_rope(st["q"], st["k"], st["q_out"], st["k_out"], q_weight=st["q_weight"],
                            k_weight=st["k_weight"], cos=st["cos"], sin=st["sin"], pos=st["pos"], eps=1e-6,
                            interleaved=neighbours)
        out["q"], out["k"] = st["q_out"], st["k_out"]
    if do != "forward":
        st["workspace"] = nsq.ns_qk_norm_rope_backward(
            st["q"], st["k"], st["dq_out"], st["dk_out"], st["dq"], st["dk"], dq_weight=st["dq_weight"],
            dk_weight=st["dk_weight"], q_weight=st["q_weight"], k_weight=st["k_weight"], cos=st["cos"],
            sin=st["sin"], pos=st["pos"], eps=1e-6, interleaved=neighbours, workspace=st.get("workspace"))
        out["dq"], out["dk"] = st["dq"], st["dk"]
        out["dq_weight"], out["dk_weight"] = st["dq_weight"], st["dk_weight"]
    return out


def _own_moe(st, do):
    import newton_schulz_quintic_amd as nsq
    out = {}
    if do != "backward":
        st["workspace"] = nsq.ns_moe_sort(st["ids"], st["case"]["experts"], st["offsets"], st["slot_of_row"],
                                          st["row_of_slot"], workspace=st.get("workspace"))
        out["offsets"], out["slot_of_row"] = st["offsets"], st["slot_of_row"]
        out["row_of_slot"] = st["row_of_slot"]
    if do in ("forward", "step"):
        nsq.ns_moe_dispatch(st["x"], st["row_of_slot"], st["xs"])
        nsq.ns_moe_combine(st["y"], st["row_of_slot"], st["weights"], st["out"])
        out["xs"], out["out"] = st["xs"], st["out"]
    if do in ("backward", "step"):
        nsq.ns_moe_combine_backward(st["dout"], st["y"], st["row_of_slot"], st["weights"], st["dy"], st["dweights"])
        nsq.ns_moe_dispatch_backward(st["dxs"], st["row_of_slot"], st["dx"])
        out["dy"], out["dweights"], out["dx"] = st["dy"], st["dweights"], st["dx"]
    return out


def _own_distill(st, do):
    import newton_schulz_quintic_amd as nsq
    train = do == "train"
    st["workspace"] = nsq.ns_distill_topk(
        st["logits"], st["ids"], st["teacher"], st["loss"], st["lse"], teacher_lse=st["teacher_lse"],
        rest_lse=st["rest_lse"], temperature=st["case"]["temperature"], grad_loss=st["grad_loss"] if train else None,
        dlogits=st["dlogits"] if train else None, workspace=st.get("workspace"))
    if do == "step":
        nsq.ns_distill_topk_backward(
            st["logits"], st["ids"], st["teacher"], st["lse"], st["grad_loss"], st["dlogits"],
            teacher_lse=st["teacher_lse"], rest_lse=st["rest_lse"], temperature=st["case"]["temperature"])
    out = {"loss": st["loss"], "lse": st["lse"]}
    if st["rest_lse"] is not None:
        out["rest_lse"] = st["rest_lse"]
    if do != "forward":
        out["dlogits"] = st["dlogits"]
    return out


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------

def _rotate(x, cos, sin, neighbours):
    """Rotates the first 2 * cos.shape[-1] values of each head by its token's angles."""
    r = 2 * cos.shape[-1]
    if neighbours:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _qk_forward(x, weight, cos, sin, neighbours):
    x32 = x.float()
    normed = x32 * torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + 1e-6)
    return _rotate(normed * weight, cos, sin, neighbours).to(x.dtype)


def _qk_backward(x, dy, weight, cos, sin, neighbours):
    x32 = x.float()
    scale = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + 1e-6)
    normed = x32 * scale
    du = _rotate(dy.float(), cos, -sin, neighbours)
    dweight = (du * normed).sum((0, 1, 2))
    dn = du * weight
    dx = scale * (dn - normed * (dn * normed).mean(-1, keepdim=True))
    return dx.to(x.dtype), dweight


def _plain_qk(st, do):
    out, neighbours = {}, st["case"]["pairs"] == "neighbours"
    pos = st["pos"].long()
    cos, sin = st["cos"][pos][:, :, None], st["sin"][pos][:, :, None]
    if do != "backward":
        out["q"] = _qk_forward(st["q"], st["q_weight"], cos, sin, neighbours)
        out["k"] = _qk_forward(st["k"], st["k_weight"], cos, sin, neighbours)
    if do != "forward":
        out["dq"], out["dq_weight"] = _qk_backward(st["q"], st["dq_out"], st["q_weight"], cos, sin, neighbours)
        out["dk"], out["dk_weight"] = _qk_backward(st["k"], st["dk_out"], st["k_weight"], cos, sin, neighbours)
    return out


def _sort_plain(ids, experts):
    """Rows by expert, then by slot; dropped slots come last, and both maps hold ~row and ~slot for them."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    sorted_key, slot = torch.sort(key, stable=True)
    row = torch.empty_like(slot)
    row[slot] = torch.arange(slot.numel(), device=slot.device)
    offsets = torch.searchsorted(sorted_key, torch.arange(experts + 1, device=ids.device))
    slot_of_row = torch.where(sorted_key == experts, ~slot, slot)
    row_of_slot = torch.where(key == experts, ~row, row).view(ids.shape)
    return offsets.to(torch.int32), slot_of_row.to(torch.int32), row_of_slot.to(torch.int32)


def _plain_moe(st, do):
    out, row_of_slot = {}, st["row_of_slot"]
    t, k, h = st["case"]["tokens"], st["case"]["top_k"], st["case"]["hidden"]
    if do != "backward":
        out["offsets"], out["slot_of_row"], row_of_slot = _sort_plain(st["ids"], st["case"]["experts"])
        out["row_of_slot"] = row_of_slot
    if do == "sort":
        return out
    kept = row_of_slot >= 0
    row = torch.where(kept, row_of_slot, ~row_of_slot).long().reshape(-1)
    kept3 = kept[:, :, None]
    weights = st["weights"][:, :, None]
    if do in ("forward", "step"):
        copies = torch.where(kept3, st["x"][:, None], torch.zeros((), dtype=st["x"].dtype, device="cuda"))
        out["xs"] = torch.empty_like(st["y"])
        out["xs"][row] = copies.reshape(t * k, h)
        picked = torch.where(kept3, st["y"][row].view(t, k, h).float(), 0.0)
        out["out"] = (picked * weights).sum(1).to(st["y"].dtype)
    if do in ("backward", "step"):
        dout = st["dout"].float()[:, None]
        out["dy"] = torch.empty_like(st["y"])
        out["dy"][row] = torch.where(kept3, dout * weights, 0.0).to(st["y"].dtype).reshape(t * k, h)
        picked = torch.where(kept3, st["y"][row].view(t, k, h).float(), 0.0)
        out["dweights"] = (picked * dout).sum(2)
        out["dx"] = torch.where(kept3, st["dxs"][row].view(t, k, h).float(), 0.0).sum(1).to(st["y"].dtype)
    return out


def _plain_distill(st, do):
    inv = 1.0 / st["case"]["temperature"]
    ids, z = st["ids"].long(), st["logits"].float() * inv
    here = (ids >= 0) & (ids < z.shape[1])
    at = torch.where(here, ids, 0)
    some = here.any(1)
    largest = z.amax(1, keepdim=True)
    e = torch.exp(z - largest)
    total = e.sum(1, keepdim=True)
    lse = largest + torch.log(total)
    log_q = z.gather(1, at) - largest - torch.log(total)
    teacher = torch.where(here, st["teacher"].float() * inv, -math.inf)
    if st["teacher_lse"] is None:
        t_largest = torch.where(some, teacher.amax(1), 0.0)[:, None]
        log_p = teacher - t_largest - torch.log(torch.exp(teacher - t_largest).sum(1, keepdim=True))
    else:
        log_p = teacher - st["teacher_lse"][:, None]
    p = torch.where(here, torch.exp(log_p), 0.0)
    loss = torch.where(here, p * (log_p - log_q), 0.0).sum(1)
    out = {"lse": torch.where(some, lse[:, 0], 0.0)}
    others = 1.0
    if st["teacher_lse"] is not None:
        top = torch.zeros_like(z, dtype=torch.bool).scatter_(1, at, here)
        z_rest = torch.where(top, -math.inf, z)
        rest_largest = z_rest.amax(1, keepdim=True)
        rest_lse = rest_largest + torch.log(torch.exp(z_rest - rest_largest).sum(1, keepdim=True))
        p_rest = (1.0 - p.double().sum(1, keepdim=True)).clamp_min(0.0).float()
        log_q_rest = rest_lse - lse
        loss = loss + (p_rest * (torch.log(p_rest) - log_q_rest))[:, 0]
        others = torch.where(top, 1.0, 1.0 - p_rest * torch.exp(-log_q_rest))
        out["rest_lse"] = torch.where(some, rest_lse[:, 0], 0.0)
    out["loss"] = torch.where(some, loss, 0.0)
    if do != "forward":
        dz = e / total * others
        dz.scatter_add_(1, at, -p)
        scale = torch.where(some, st["grad_loss"] * inv, 0.0)
        out["dlogits"] = (dz * scale[:, None]).to(st["logits"].dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"qk": _exact_qk, "moe": _exact_moe, "distill": _exact_distill}[case["op"]](st, case)


def _turn(x, weight, cos, sin, neighbours):
    """The forward pass with each pair as one complex number."""
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight
    half = cos.shape[-1]
    head = n[..., :2 * half]
    parts = head.unflatten(-1, (half, 2)) if neighbours else head.unflatten(-1, (2, half)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(parts.contiguous()) * torch.complex(cos, sin))
    turned = turned if neighbours else turned.transpose(-1, -2)
    return torch.cat((turned.flatten(-2), n[..., 2 * half:]), -1)


def _exact_qk(st, case):
    out = {}
    rows = st["pos"].long()
    cos, sin = st["cos"].double()[rows].unsqueeze(2), st["sin"].double()[rows].unsqueeze(2)
    for name in ("q", "k"):
        x = st[name].double().requires_grad_(case["do"] != "forward")
        w = st[name + "_weight"].double().requires_grad_(case["do"] != "forward")
        y = _turn(x, w, cos, sin, case["pairs"] == "neighbours")
        if case["do"] != "backward":
            out[name] = y.detach()
        if case["do"] != "forward":
            out["d" + name], out["d" + name + "_weight"] = torch.autograd.grad(y, (x, w), st["d" + name + "_out"].double())
    return out


def _exact_moe(st, case):
    t, k, h, e, do = case["tokens"], case["top_k"], case["hidden"], case["experts"], case["do"]
    if do == "sort":
        return None
    flat = st["ids"].reshape(-1).long().cpu()
    keep = ((flat >= 0) & (flat < e)).nonzero()[:, 0]
    order = keep[torch.argsort(flat[keep] * (t * k) + keep)].cuda()   # the kept slots in row order
    token, n = order // k, order.numel()
    y, w = st["y"][:n].double(), st["weights"].double().reshape(-1)[order]
    out = {"offsets": None, "slot_of_row": None, "row_of_slot": None} if do != "backward" else {}
    if do in ("forward", "step"):
        out["xs"] = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        out["xs"][:n] = st["x"].double()[token]
        out["out"] = torch.zeros(t, h, dtype=torch.float64, device="cuda").index_add_(0, token, y * w[:, None])
    if do in ("backward", "step"):
        g = st["dout"].double()[token]
        out["dy"] = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        out["dy"][:n] = g * w[:, None]
        dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dw[order] = torch.linalg.vecdot(g, y)
        out["dweights"] = dw.view(t, k)
        out["dx"] = torch.zeros(t, h, dtype=torch.float64, device="cuda").index_add_(0, token, st["dxs"][:n].double())
    return out


def _exact_distill(st, case):
    parts = [_exact_rows(st, case, slice(i, i + 256)) for i in range(0, case["rows"], 256)]
    return {key: torch.cat([p[key] for p in parts]) for key in parts[0]}


def _exact_rows(st, case, at):
    """Cross entropy less the teacher's entropy, over the top tokens and, with the teacher's
    logsumexp, one more class that holds all the others; the gradient by differentiation."""
    ids = st["ids"][at].long()
    z = (st["logits"][at].double() / case["temperature"]).requires_grad_(True)
    some = ids[:, 0] >= 0
    ids = ids.clamp_min(0)
    t = st["teacher"][at].double() / case["temperature"]
    lse = torch.logsumexp(z, 1)
    log_q = z.gather(1, ids) - lse[:, None]
    out = {}
    if st["teacher_lse"] is None:
        log_p = t - torch.logsumexp(t, 1, keepdim=True)
    else:
        log_p = t - st["teacher_lse"][at].double()[:, None]
        rest = torch.logsumexp(z.scatter(1, ids, -math.inf), 1)
        out["rest_lse"] = torch.where(some, rest, 0.0).detach()
        log_p = torch.cat((log_p, torch.log1p(-log_p.exp().sum(1, keepdim=True))), 1)
        log_q = torch.cat((log_q, (rest - lse)[:, None]), 1)
    loss = torch.where(some, (log_p.exp() * (log_p - log_q)).sum(1), 0.0)
    if case["do"] != "forward":
        dz, = torch.autograd.grad(loss, z, st["grad_loss"][at].double())
        out["dlogits"] = dz / case["temperature"]
    out["loss"], out["lse"] = loss.detach(), torch.where(some, lse, 0.0).detach()
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size, do = _BYTES[case["dtype"]], case["do"]
    if case["op"] == "qk":
        tokens, heads = case["batch"] * case["seq"], case["q_heads"] + case["k_heads"]
        data = tokens * heads * case["head_dim"] * size
        table = min(tokens, case["table"]) * case["rope_dim"] * 4
        moved = {"forward": 2, "backward": 3, "step": 5}[do] * data + table + 4 * tokens + 16 * case["head_dim"]
        ops = {"forward": 8, "backward": 16, "step": 24}[do] * tokens * heads * case["head_dim"]
        return {"bytes": moved, "flops": ops}
    if case["op"] == "moe":
        slots = case["tokens"] * case["top_k"]
        row, rows = case["tokens"] * case["hidden"] * size, slots * case["hidden"] * size
        moved, ops = 0, 0
        if do != "backward":
            moved += 12 * slots + 4 * (case["experts"] + 1)
        if do in ("forward", "step"):
            moved += 2 * (row + rows) + 4 * slots
            ops += 2 * slots * case["hidden"]
        if do in ("backward", "step"):
            moved += 2 * row + 3 * rows + 12 * slots
            ops += 4 * slots * case["hidden"]
        return {"bytes": moved, "flops": ops}
    rows = case["rows"] - case["empty"]
    read, written = rows * case["vocab"] * size, case["rows"] * case["vocab"] * size
    moved = read + (written if do != "forward" else 0) + (read if do == "step" else 0)
    moved += case["rows"] * (case["top_k"] * (4 + size) + 16)
    return {"bytes": moved, "flops": (3 if do == "forward" else 8) * rows * case["vocab"]}
