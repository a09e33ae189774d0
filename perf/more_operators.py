"""Cases that measure the operators next to a block's matrix products and to the update.

The norms before and after a block with its gate and residual scale
(ns_block_norm), 8-bit matrix products with a scale for each block of 128, dense
and by expert (ns_quantize, ns_scaled_matmul), and the norm and clipping of many
gradients on their way into the momentum (ns_grad_norm, ns_grad_clip). ``run``
computes them in elementary torch operations while ``own`` is false, and with this
package's entry points while it is true; ``exact`` gives the same outputs from the
definitions in 64 bits.

Sizes: hidden, key and feed-forward widths are those of the dense-transformer set
(4096, 1024, 14336), the experts those of the many-small set (64 of 2048 x 7168);
the others are generic.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _grad(name, tensors, sizes, mixed, out, momentum, far):
    return {"name": name, "op": "grad", "tensors": tensors, "sizes": sizes, "mixed": mixed, "out": out,
            "momentum": momentum, "far": far}


def _block(name, do, rows, hidden, dtype, residual, gates, post, alpha, scale):
    return {"name": name, "op": "block", "do": do, "rows": rows, "hidden": hidden, "dtype": dtype, "residual": residual,
            "gates": gates, "post": post, "alpha": alpha, "scale": scale}


def _scaled(name, do, rows, inner, outer, experts, dtype):
    return {"name": name, "op": "scaled", "do": do, "rows": rows, "inner": inner, "outer": outer, "experts": experts,
            "dtype": dtype}


def listed():
    return [
        # norm weights and biases of a small fp32 model: latency
        _grad("clip small", 26, 4096, False, "f32", 0.0, True),
        # four layers' matrices in bf16, clipped on their way into fp32 momentum matrices
        _grad("clip layers", 28, 0, False, "f32", 0.95, True),
        # one new token of each of 16 sequences: latency
        _block("block decode", "forward", 16, 4096, "bf16", "bf16", 1, True, 1.0, 1.0),
        # a training micro-batch, norms on both sides of the block and a gate per channel
        _block("block train forward", "forward", 16384, 4096, "bf16", "bf16", 1, True, 1.0, 0.5),
        _block("block train backward", "backward", 16384, 4096, "bf16", "bf16", 1, True, 1.0, 0.5),
        # an odd width, an fp32 residual stream, a gate per sequence (three of 1027 tokens), both directions
        _block("block odd step", "step", 3081, 1537, "bf16", "f32", 3, True, 0.9, 1.5),
        # 16 tokens through one feed-forward matrix: the weights' bytes
        _scaled("scaled decode", "forward", 16, 4096, 14336, 0, "bf16"),
        # a training micro-batch through the same matrix, and its gradients of input and weight
        _scaled("scaled forward", "forward", 8192, 4096, 14336, 0, "bf16"),
        _scaled("scaled backward", "backward", 8192, 4096, 14336, 0, "bf16"),
        # 8 tokens x 8 choices of 64 experts: a row or two for each expert's matrix
        _scaled("experts decode", "forward", 64, 7168, 2048, 64, "bf16"),
        # a training micro-batch of 8192 tokens x 8 choices
        _scaled("experts forward", "forward", 65536, 7168, 2048, 64, "bf16"),
        # odd counts and widths in fp32, both directions
        _scaled("experts ragged step", "step", 9003, 1537, 520, 17, "f32"),
    ]


def _log(rng, lo, hi):
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))))
    return n if n % 1024 else max(lo, n - 1)   # the listed cases have the round sizes


def draw(rng):
    op = rng.choice(["grad", "block", "scaled", "scaled"])
    if op == "grad":
        tensors = _log(rng, 1, 600)
        most = min(1 << 24, 800_000_000 // tensors)
        c = _grad("", tensors, _log(rng, 16, most), rng.random() < 0.5, rng.choice(["bf16", "f32"]),
                  rng.choice([0.0, 0.9, 0.95]), rng.random() < 0.8)
    elif op == "block":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        residual = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        hidden = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            hidden = 64 * (hidden // 128 * 2 + 1)
        rows = _log(rng, 1, min(32768, 400_000_000 // (8 * hidden * _BYTES[residual]) * 2))
        batch = rng.choice([0, 1, 1, 2, 4, rows])
        rows = -(-rows // batch) * batch if batch else rows
        c = _block("", rng.choice(["forward", "backward", "step"]), rows, hidden, dtype, residual, batch,
                   rng.random() < 0.7, rng.choice([1.0, 0.8]), rng.choice([1.0, 0.25]))
    else:
        experts = rng.choice([0, 0, 0, _log(rng, 2, 128)])
        do = rng.choice(["forward", "forward", "backward", "step", "weights"])
        inner, outer = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.7:
            inner, outer = -(-inner // 64) * 64, 64 * (outer // 128 * 2 + 1)
        if experts:
            outer = min(outer, max(64, 1_000_000_000 // (experts * inner)))
        most = 1_000_000_000_000 // (6 * inner * outer)
        rows = _log(rng, 1, max(1, min(32768, most)))
        c = _scaled("", do, rows, inner, outer, experts, rng.choice(["bf16", "bf16", "f32"]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"grad": _prepare_grad, "block": _prepare_block, "scaled": _prepare_scaled}[case["op"]](case, gen)


def _randn(gen, shape, dtype=torch.float32, std=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(std).to(dtype)


def _counts(case):
    """How many values each tensor of a gradient list holds."""
    if not case["sizes"]:   # the matrices of dense layers: q, k, v, o, gate, up, down
        layer = [4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096] + 3 * [14336 * 4096]
        return [layer[i % 7] for i in range(case["tensors"])]
    return [max(1, case["sizes"] * (1 + i * 7 % 5) // 5 + (i * i) % 3 - 1) for i in range(case["tensors"])]


def _prepare_grad(case, gen):
    counts = _counts(case)
    # each tensor starts at a multiple of 64 values of one flat buffer per type, as flat gradient buffers keep them
    kinds = ["f32" if case["mixed"] and i % 3 == 1 else ("bf16" if case["mixed"] or not case["sizes"] else "f32")
             for i in range(len(counts))]
    flat_of, places = {}, []
    for n, kind in zip(counts, kinds):
        at = flat_of.get(kind, 0)
        places.append((kind, at, n))
        flat_of[kind] = at + -(-n // 64) * 64
    out_of, out_places = 0, []
    for n in counts:
        out_places.append((out_of, n))
        out_of += -(-n // 64) * 64
    st = {"case": case, "flat": {}}
    for kind, size in sorted(flat_of.items()):
        st["flat"][kind] = _randn(gen, (size,), _DTYPES[kind], 0.01 if case["far"] else 1e-6)
    st["grads"] = [st["flat"][kind][at:at + n] for kind, at, n in places]
    st["max_norm"] = 1e-3 if case["far"] else 1e6   # clipped, or left as it is
    st["out"] = torch.zeros(out_of, dtype=_DTYPES[case["out"]], device="cuda")
    st["outs"] = [st["out"][at:at + n] for at, n in out_places]
    st["momenta"] = None
    if case["momentum"]:
        st["momentum"] = _randn(gen, (out_of,), _DTYPES[case["out"]], 0.01)
        st["momenta"] = [st["momentum"][at:at + n] for at, n in out_places]
    st["norm"] = torch.empty(1, device="cuda")
    return st


def _prepare_block(case, gen):
    n, h, b = case["rows"], case["hidden"], case["gates"]
    dtype, residual = _DTYPES[case["dtype"]], _DTYPES[case["residual"]]
    st = {"case": case, "x": _randn(gen, (n, h), residual, 2.0), "y": _randn(gen, (n, h), dtype, 3.0)}
    st["pre_weight"] = 1.0 + _randn(gen, (h,), std=0.1)
    st["post_weight"] = 1.0 + _randn(gen, (h,), std=0.1) if case["post"] else None
    st["gate"] = _randn(gen, (b, h), torch.float32 if b < n else dtype, 0.5) if b else None
    st["x_out"], st["h"] = torch.empty_like(st["x"]), torch.empty_like(st["y"])
    if case["do"] != "forward":
        st["dx_out"], st["dh"] = _randn(gen, (n, h), residual), _randn(gen, (n, h), dtype)
        st["dx"], st["dy"] = torch.empty_like(st["x"]), torch.empty_like(st["y"])
        st["dpre_weight"] = torch.empty(h, device="cuda")
        st["dpost_weight"] = torch.empty(h, device="cuda") if case["post"] else None
        st["dgate"] = torch.empty_like(st["gate"]) if b else None
    return st


def _up(n):
    return -(-n // 128) * 128


def _new8(*shape):
    return torch.empty(shape, dtype=_E4M3, device="cuda")


def _scales(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def _prepare_scaled(case, gen):
    t, k, n, e, do = case["rows"], case["inner"], case["outer"], case["experts"], case["do"]
    dtype = _DTYPES[case["dtype"]]
    st = {"case": case}
    w = _randn(gen, (max(e, 1), n, k), dtype, k ** -0.5)
    if e:   # rows sorted by expert, some favoured, as ns_moe_sort leaves them; the last few were dropped
        score = torch.randn(t, e, generator=gen, device="cuda") + _randn(gen, (e,), std=0.5)
        choice = score.argmax(1)
        choice[:t // 50] = e
        st["offsets"] = torch.searchsorted(choice.sort()[0], torch.arange(e + 1, device="cuda")).to(torch.int32)
    else:
        st["offsets"] = None
        w = w[0]
    lead = (e,) if e else ()
    st["wq"], st["ws"] = _new8(*lead, n, _up(k)), _scales(*lead, _up(n) // 128, _up(k) // 128)
    st["wqt"], st["wst"] = _new8(*lead, k, _up(n)), _scales(*lead, _up(k) // 128, _up(n) // 128)
    if do == "weights":
        st["w"] = w
        return st
    q, s = _quantize_plain(w, 128)
    st["wq"].copy_(q)
    st["ws"].copy_(s)
    # channels of activations differ in size
    spread = torch.exp(_randn(gen, (k,), std=0.7))
    st["x"] = (torch.randn(t, k, generator=gen, device="cuda") * spread).to(dtype)
    if do != "backward":
        st["xq"], st["xs"] = _new8(t, _up(k)), _scales(t, _up(k) // 128)
        st["y"] = torch.zeros(t, n, dtype=dtype, device="cuda")
    if do != "forward":
        q, s = _quantize_plain(w.transpose(-1, -2).contiguous(), 128)
        st["wqt"].copy_(q)
        st["wst"].copy_(s)
        p = (t // 128 + e) * 128 if e else _up(t)   # a place for every expert's rows, each up to a multiple of 128
        st["dy"] = _randn(gen, (t, n), dtype, 1e-3)
        st["dyq"], st["dys"] = _new8(t, _up(n)), _scales(t, _up(n) // 128)
        st["dyqt"], st["dyst"] = _new8(n, p), _scales(n, p // 128)
        st["xqt"], st["xst"] = _new8(k, p), _scales(k, p // 128)
        st["dx"] = torch.zeros(t, k, dtype=dtype, device="cuda")
        st["dw"] = torch.empty(*lead, n, k, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return {"grad": _own_grad, "block": _own_block, "scaled": _own_scaled}[case["op"]](state, case)
    return {"grad": _plain_grad, "block": _plain_block, "scaled": _plain_scaled}[case["op"]](state, case)


def _own_grad(st, case):
    import newton_schulz_quintic_amd as nsq
    st["workspace"] = nsq.ns_grad_norm(st["grads"], st["norm"], workspace=st.get("workspace"))
    nsq.ns_grad_clip(st["grads"], st["outs"], norm=st["norm"], max_norm=st["max_norm"], eps=1e-6,
                     momenta=st["momenta"], beta=case["momentum"], workspace=st["workspace"])
    return {"norm": st["norm"], "out": st["out"]}


def _own_block(st, case):
    import newton_schulz_quintic_amd as nsq
    out = {}
    how = dict(post_weight=st["post_weight"], pre_weight=st["pre_weight"], gate=st["gate"], post_norm=case["post"],
               alpha=case["alpha"], scale=case["scale"], eps=1e-6)
    if case["do"] != "backward":
        nsq.ns_block_norm(st["x"], st["y"], st["x_out"], st["h"], **how)
        out["x_out"], out["h"] = st["x_out"], st["h"]
    if case["do"] != "forward":
        st["workspace"] = nsq.ns_block_norm_backward(
            st["x"], st["y"], st["dx_out"], st["dh"], st["dx"], st["dy"], dpost_weight=st["dpost_weight"],
            dpre_weight=st["dpre_weight"], dgate=st["dgate"], workspace=st.get("workspace"), **how)
        out.update({name: st[name] for name in ("dx", "dy", "dpre_weight", "dpost_weight", "dgate")
                    if st[name] is not None})
    return out


def _own_scaled(st, case):
    import newton_schulz_quintic_amd as nsq
    out, do, offsets = {}, case["do"], st["offsets"]
    if do == "weights":
        nsq.ns_quantize(st["w"], st["wq"], st["ws"], st["wqt"], st["wst"], block_rows=128)
        return {"wq": st["wq"], "ws": st["ws"], "wqt": st["wqt"], "wst": st["wst"]}
    if do != "backward":
        nsq.ns_quantize(st["x"], st["xq"], st["xs"])
        st["workspace"] = nsq.ns_scaled_matmul(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], offsets=offsets,
                                               workspace=st.get("workspace"))
        out.update(xq=st["xq"], xs=st["xs"], y=st["y"])
    if do != "forward":
        nsq.ns_quantize(st["dy"], st["dyq"], st["dys"], st["dyqt"], st["dyst"], offsets=offsets)
        nsq.ns_quantize(st["x"], None, None, st["xqt"], st["xst"], offsets=offsets)
        st["workspace_dx"] = nsq.ns_scaled_matmul(st["dyq"], st["dys"], st["wqt"], st["wst"], st["dx"], offsets=offsets,
                                                  workspace=st.get("workspace_dx"))
        st["workspace_dw"] = nsq.ns_scaled_matmul(st["dyqt"], st["dyst"], st["xqt"], st["xst"], st["dw"],
                                                  offsets=offsets, reduce=offsets is not None,
                                                  workspace=st.get("workspace_dw"))
        out.update(dyq=st["dyq"], dys=st["dys"], dx=st["dx"], dw=st["dw"])
    return out


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------

def _plain_grad(st, case):
    squares = torch.stack([g.float().square().sum() for g in st["grads"]])
    norm = squares.double().sum().sqrt().float().reshape(1)
    c = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    if st["momenta"] is None:
        [o.copy_(g.float() * c) for g, o in zip(st["grads"], st["outs"])]
    else:
        [o.copy_(case["momentum"] * m.float() + c * g.float())
         for g, o, m in zip(st["grads"], st["outs"], st["momenta"])]
    return {"norm": norm, "out": st["out"]}


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def _norm_back(x, r, dn):
    """Gradient of x * r(x) from dn, that of its value."""
    n = x * r
    return r * (dn - n * (dn * n).mean(-1, keepdim=True))


def _plain_block(st, case):
    out = {}
    n, h = st["x"].shape
    x, y = st["x"].float(), st["y"].float()
    ry = _rms(y) if case["post"] else None
    z = y * ry * st["post_weight"] if case["post"] else y
    gate = None
    if st["gate"] is not None:
        gate = st["gate"].float().repeat_interleave(n // case["gates"], 0) if case["gates"] > 1 else st["gate"].float()
    r = case["alpha"] * x + case["scale"] * (z if gate is None else gate * z)
    rr = _rms(r)
    if case["do"] != "backward":
        out["x_out"] = r.to(st["x"].dtype)
        out["h"] = (r * rr * st["pre_weight"]).to(st["y"].dtype)
    if case["do"] != "forward":
        dh = st["dh"].float()
        out["dpre_weight"] = (dh * (r * rr)).sum(0)
        dr = st["dx_out"].float() + _norm_back(r, rr, dh * st["pre_weight"])
        out["dx"] = (case["alpha"] * dr).to(st["x"].dtype)
        dg = case["scale"] * dr
        if gate is not None:
            out["dgate"] = (dg * z).view(case["gates"], -1, h).sum(1).to(st["gate"].dtype)
            dg = dg * gate
        if case["post"]:
            out["dpost_weight"] = (dg * (y * ry)).sum(0)
            dg = _norm_back(y, ry, dg * st["post_weight"])
        out["dy"] = dg.to(st["y"].dtype)
    return out


def _power_of_two(e):
    """2^e in 32 bits for whole e in [-126, 127], exactly (torch's exp2, pow and ldexp round)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantize_plain(x, block_rows):
    """(..., rows, cols) into e4m3 values of whole blocks of 128 columns, zeros behind the last, and the exponents' bytes."""
    rows, cols = x.shape[-2:]
    more = -rows % block_rows
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, more))
    blocks = v.view(*x.shape[:-2], (rows + more) // block_rows, block_rows, -1, 128)
    largest = blocks.abs().amax((-3, -1), keepdim=True)
    m, e = torch.frexp(largest)                       # largest = m 2^e, 0.5 <= m < 1
    power = torch.where(largest > 0, e - 9 + (m > 0.875).int(), 0).clamp(-126, 127)
    q = (blocks * _power_of_two(-power)).to(_E4M3)
    q = q.view(v.shape)[..., :rows, :]
    return q, (power + 127).to(torch.uint8)[..., 0, :, 0]


def _value(q, scales):
    """What e4m3 values with their scales stand for, in 32 bits; scales of single rows or of 128."""
    s = _power_of_two(scales.int() - 127)
    if scales.shape[-2] != q.shape[-2]:
        s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return q.float() * s.repeat_interleave(128, -1)


def _spans(offsets):
    at = offsets.tolist()
    return list(zip(at, at[1:]))


def _plain_scaled(st, case):
    out, do, t, offsets = {}, case["do"], case["rows"], st["offsets"]
    if do == "weights":
        q, s = _quantize_plain(st["w"], 128)
        qt, s_t = _quantize_plain(st["w"].transpose(-1, -2), 128)
        return {"wq": q, "ws": s, "wqt": qt, "wst": s_t}
    spans = _spans(offsets) if offsets is not None else [(0, t)]
    w = _value(st["wq"], st["ws"]).view(len(spans), case["outer"], -1)
    if do != "backward":
        xq, xs = _quantize_plain(st["x"], 1)
        x = _value(xq, xs)
        y = torch.cat([x[a:b] @ m.t() for (a, b), m in zip(spans, w)])
        out["xq"], out["xs"] = xq, xs
        out["y"] = torch.nn.functional.pad(y, (0, 0, 0, t - y.shape[0])).to(st["y"].dtype)
    if do != "forward":
        wt = _value(st["wqt"], st["wst"]).view(len(spans), case["inner"], -1)
        dyq, dys = _quantize_plain(st["dy"], 1)
        dy = _value(dyq, dys)
        dx = torch.cat([dy[a:b] @ m.t() for (a, b), m in zip(spans, wt)])
        out["dyq"], out["dys"] = dyq, dys
        out["dx"] = torch.nn.functional.pad(dx, (0, 0, 0, t - dx.shape[0])).to(st["dx"].dtype)
        # along the tokens, each expert's by itself
        turned = lambda v, a, b: _value(*_quantize_plain(v[a:b].t(), 1))  # noqa: E731
        dw = [turned(st["dy"], a, b) @ turned(st["x"], a, b).t() for a, b in spans]
        out["dw"] = torch.stack(dw) if offsets is not None else dw[0]
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"grad": _exact_grad, "block": _exact_block, "scaled": _exact_scaled}[case["op"]](st, case)


def _exact_grad(st, case):
    # the gaps between the tensors hold random values too, which do not count
    norm = math.sqrt(math.fsum(torch.linalg.vector_norm(g, dtype=torch.float64).item() ** 2 for g in st["grads"]))
    c = min(1.0, st["max_norm"] / (norm + 1e-6))
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for i, (g, o) in enumerate(zip(st["grads"], st["outs"])):
        at = o.storage_offset()
        into = out[at:at + g.numel()]
        into.copy_(g).mul_(c)
        if st["momenta"] is not None:
            into.add_(st["momenta"][i], alpha=case["momentum"])
    return {"norm": torch.tensor([norm], dtype=torch.float64), "out": out}


def _exact_block(st, case):
    n, h = st["x"].shape
    grad = case["do"] != "forward"
    leaf = lambda t: None if t is None else t.double().requires_grad_(grad)  # noqa: E731
    x, y, wp, wn, g = (leaf(st[k]) for k in ("x", "y", "post_weight", "pre_weight", "gate"))
    unit = lambda v: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    z = unit(y) * wp if case["post"] else y
    if g is not None:
        z = (z.view(case["gates"], -1, h) * g[:, None]).view(n, h)
    r = case["alpha"] * x + case["scale"] * z
    hh = unit(r) * wn
    out = {}
    if case["do"] != "backward":
        out["x_out"], out["h"] = r.detach(), hh.detach()
    if grad:
        names = [(k, v) for k, v in (("dx", x), ("dy", y), ("dpre_weight", wn), ("dpost_weight", wp), ("dgate", g))
                 if v is not None]
        grads = torch.autograd.grad([r, hh], [v for _, v in names], [st["dx_out"].double(), st["dh"].double()])
        out.update({k: v for (k, _), v in zip(names, grads)})
    return out


def _exp2(e):
    """2^e in 64 bits for whole e, exactly."""
    return torch.bitwise_left_shift(e.long() + 1023, 52).view(torch.float64)


def _stands_for(x, tall):
    """(values in 64 bits that e4m3 leaves of x's blocks of `tall` x 128, x over its scale)."""
    rows, cols = x.shape
    full = torch.zeros(-(-rows // tall) * tall, _up(cols), dtype=torch.float64, device="cuda")
    full[:rows, :cols] = x
    b = full.unflatten(0, (-1, tall)).unflatten(2, (-1, 128))
    top = b.abs().amax((1, 3), keepdim=True)
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -118) / 448.0))
    e = torch.where(top > 448.0 * _exp2(e), e + 1, torch.where(top <= 448.0 * _exp2(e - 1), e - 1, e))
    e = torch.where(top > 0, e, 0.0)
    unit = b / _exp2(e)
    # e4m3 has three bits behind the first, and steps of 2^-9 below 2^-6
    step = _exp2(torch.frexp(unit.abs().clamp_min(2.0 ** -6))[1] - 4)
    kept = torch.round(unit / step) * step
    back = lambda v: v.flatten(2, 3).flatten(0, 1)[:rows]  # noqa: E731
    return back(kept * _exp2(e)), back(unit)


def _exact_scaled(st, case):
    e, t, k, n, do = case["experts"], case["rows"], case["inner"], case["outer"], case["do"]
    if do == "weights":
        if e:
            return None
        return {"wq": _stands_for(st["w"], 128)[1], "ws": None, "wqt": _stands_for(st["w"].t(), 128)[1], "wst": None}
    edge = st["offsets"].cpu().numpy() if e else [0, t]
    pieces = [slice(int(edge[i]), int(edge[i + 1])) for i in range(max(e, 1))]

    def weight(q, s, i):
        q, s = (q[i], s[i]) if e else (q, s)
        grid = _exp2(s.long() - 127)
        full = torch.kron(grid, torch.ones(128, 128, dtype=torch.float64, device="cuda"))
        return q.double() * full[:q.shape[0]]

    out = {}
    if do != "backward":
        x, unit = _stands_for(st["x"], 1)
        out.update(xq=unit, xs=None, y=torch.zeros(t, n, dtype=torch.float64, device="cuda"))
        for i, p in enumerate(pieces):
            out["y"][p] = x[p] @ weight(st["wq"], st["ws"], i).t()
    if do != "forward":
        dy, unit = _stands_for(st["dy"], 1)
        out.update(dyq=unit, dys=None, dx=torch.zeros(t, k, dtype=torch.float64, device="cuda"),
                   dw=torch.zeros(max(e, 1), n, k, dtype=torch.float64, device="cuda"))
        for i, p in enumerate(pieces):
            out["dx"][p] = dy[p] @ weight(st["wqt"], st["wst"], i).t()
            if p.stop > p.start:
                out["dw"][i] = _stands_for(st["dy"][p].t(), 1)[0] @ _stands_for(st["x"][p].t(), 1)[0].t()
        if not e:
            out["dw"] = out["dw"][0]
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "grad":
        counts = _counts(case)
        kinds = [4 if case["mixed"] and i % 3 == 1 else (2 if case["mixed"] or not case["sizes"] else 4)
                 for i in range(len(counts))]
        grads, total = sum(n * b for n, b in zip(counts, kinds)), sum(counts)
        size = _BYTES[case["out"]]
        # the clipping needs the whole norm, so the gradients are read twice
        return {"bytes": 2 * grads + total * size * (2 if case["momentum"] else 1), "flops": 6 * total}
    if case["op"] == "block":
        n, h, do = case["rows"], case["hidden"], case["do"]
        size, res = _BYTES[case["dtype"]], _BYTES[case["residual"]]
        gate = case["gates"] * h * (4 if case["gates"] < n else size)
        moved = {"forward": 2, "backward": 3, "step": 5}[do] * n * h * (size + res)
        moved += {"forward": 1, "backward": 2, "step": 3}[do] * gate + 16 * h
        return {"bytes": moved, "flops": {"forward": 10, "backward": 25, "step": 35}[do] * n * h}
    t, k, n, e, do, size = (case[key] for key in ("rows", "inner", "outer", "experts", "do", "dtype"))
    size, weights = _BYTES[size], max(e, 1) * k * n
    if do == "weights":
        return {"bytes": weights * (size + 2), "flops": 3 * weights}
    read = k * n
    if e:   # an expert that no row chose is not read; the dropped rows are not multiplied
        t -= t // 50
        read = k * n * e * (1 - (1 - 1 / e) ** t)
    moved, flops = 0, 0
    if do != "backward":
        moved += t * k * (size + 1) + read + t * n * size
        flops += 2 * t * k * n
    if do != "forward":
        moved += t * n * (size + 2) + t * k * (size + 1) + read + t * k * size + 4 * weights
        flops += 4 * t * k * n
    return {"bytes": moved, "flops": flops}
