"""GPU parity of ns_distill_topk's masses and gradients where they take most care: pairs whose mass is not 1, small
remainders, masked others, students far above their pairs, large logits.

Against the fp64 oracle (oracle/train_ops.py), with tolerances as in
test_gpu_train_ops.py: U = 2^-24 is half a step of fp32, a bf16 result adds
2^-8 of the value.
"""

import numpy as np
import pytest

import newton_schulz_quintic_amd as nsq
from oracle import train_ops as ops
from tests.helpers import host_to_f64, log, to_device
from tests.test_gpu_train_ops import HALF_STEP, U, _close, _distill_case, _distill_run, _f64
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _teacher(c, t, lse, tdtype="f32"):
    """Puts teacher logits and logsumexps (rounded to fp32, as the call takes them) into a case."""
    import torch
    tb = f32_to_bf16_bits(t.astype(np.float32)) if tdtype == "bf16" else t.astype(np.float32)
    c["t64"], c["t"], c["tdtype"] = host_to_f64(tb, tdtype), to_device(tb, tdtype), tdtype
    c["lse64"] = lse.astype(np.float32).astype(np.float64)
    c["lse_d"] = torch.from_numpy(lse.astype(np.float32)).cuda()
    return c


def _check(c, got, form, rows, p_steps=None, mass64=False, most=np.inf):
    """With F = P - p_r / q_r the gradient is g / tau (q_j F - sum of j's p). Relative errors: of q, (4 |z - m| / tau + 4 E
    + 64) U as in _check_distill, and 2 |lse| U more where lse was rounded between two calls; of q_r likewise; of p,
    p_steps U if given, else (4 (|t| / tau + |lse_T|) + 64) U, the rounding of fp32 exponents. P and p_r are off by dP, the
    sum of the p's errors (and half a step of their own), which reaches others through F. With mass64 they come from p in
    64 bits and are rounded once: 2^-44 of the exponential, the exponent's roundings, 2^-53 of its parts each (4 of them
    counted), and half a step of p_r. `most`: the largest logsumexp that the second call takes q from."""
    loss, lse, rest, dz = got
    tau, half = c["tau"], HALF_STEP[c["dtype"]]
    for i in rows:
        tl = None if c["lse64"] is None else c["lse64"][i]
        w = ops.distill_row(c["z64"][i], c["ids"][i], c["t64"][i], tau, tl, c["g64"][i],
                            teacher_bf16=c["tdtype"] == "bf16")
        g, z, v = c["g64"][i], c["z64"][i], len(c["z64"][i])
        if not w["some"]:
            assert loss[i] == 0 and lse[i] == 0 and (tl is None or rest[i] == 0) and not dz[i].float().abs().any()
            continue
        here = [(int(j), float(x)) for j, x in zip(c["ids"][i], c["t64"][i]) if 0 <= j < v]
        at = np.array([j for j, _ in here])
        t = np.array([x for _, x in here])
        with np.errstate(all="ignore"):
            q, p, p_rest = w["q"], w["p"], w["p_rest"]
            arg = np.where(q > 0, np.abs(z - np.max(z)) / tau, 0.0)
            E = np.sum(q * arg)
            two = 2 * min(abs(w["lse"]), most) if form == "step" else 0.0
            err_q = (4 * arg + 4 * E + 64 + two) * U
            steps = 4 * (np.abs(t - np.max(t)) / tau if tl is None else np.abs(t) / tau + abs(tl)) + 64
            steps = steps if p_steps is None else p_steps
            err_p = np.where(p > 0, steps * U, 0.0)
            P = p.sum() + p_rest
            dP = np.sum(np.where(p > 0, p * err_p, 0.0)) + 2 * U
            if mass64:
                dP = P * (2.0 ** -44 + 2.0 ** -51 * (np.max(np.abs(t)) / tau + abs(tl))) + U * p_rest
            outside = np.ones(v, bool)
            outside[at] = False
            factor, err_factor = P, dP + 2 * U * P
            err_rest = 0.0
            if tl is None:
                factor, err_factor = 1.0, 0.0
            elif w["rest_lse"] == -np.inf:   # no others, or none with any mass
                assert rest[i] == -np.inf
            elif outside.any():
                zr = z[outside]
                qr = np.exp(w["rest_lse"] - w["lse"])
                er = np.sum(np.where(zr > -np.inf, q[outside] * np.abs(zr - zr.max()) / tau, 0)) / max(qr, 1e-300)
                err_rest = (4 * er + 64 + 4 * np.abs(zr.max() - np.max(z)) / tau + 4 * E
                            + (two + 2 * min(abs(w["rest_lse"]), most) if form == "step" else 0.0)) * U
                if p_rest > 0:
                    factor = 1 - p_rest / qr
                    err_factor = (dP + p_rest * (err_rest + 8 * U)) / qr
                assert abs(float(rest[i]) - w["rest_lse"]) <= U * (4 * abs(zr.max()) / tau + 4 * er + 64 + 2 * abs(w["rest_lse"]))
            size = q * ((err_q + err_rest) * (np.abs(factor) + P * (p_rest > 0)) + err_factor)
            size[at] = (q * (err_q * P + err_factor if p_rest == 0 and tl is not None else err_q))[at]
            for a, b in zip(at, p * err_p):
                size[a] += b
            used = p > 0
            diff = np.abs(w["log_p"] - np.log(q[at]))
            tol = np.sum((p * ((4 * arg[at] + 4 * E + 64) * U + err_p + (err_p + 64 * U) * diff
                               + 2 * U * np.abs(w["log_p"])))[used])
            if p_rest > 0:
                log_qr = w["rest_lse"] - w["lse"]
                tol += dP * (1 + abs(np.log(p_rest) - log_qr)) + p_rest * (err_rest + 8 * U * (1 + abs(np.log(p_rest)) + abs(log_qr)))
        assert abs(float(loss[i]) - w["loss"]) <= tol + 4 * U * abs(w["loss"]), (i, float(loss[i]), w["loss"], tol)
        want = np.where(np.abs(w["dlogits"]) < 2.0 ** -126, 0.0, w["dlogits"])
        _close(_f64(dz[i]), want, half * np.abs(want) + g / tau * size + 8 * U * np.abs(want) + 2.0 ** -126, f"row {i}")


# every form of the kernels: rows split over workgroups, held in 64 .. 1024 threads, too long to hold
FORMS = [(3, 9001, 40), (260, 300, 20), (257, 3001, 300), (256, 33000, 24), (256, 66001, 64), (256, 140003, 16)]


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,k", FORMS)
@pytest.mark.parametrize("kind", ["small logsumexp", "bf16 teacher", "listed twice"])
def test_pairs_whose_mass_passes_one(kind, n, v, k, dtype, form):
    """A logsumexp below the pairs' own, teacher logits rounded to bf16 after it was taken, tokens listed twice."""
    log(f"distill mass {kind} {n} {v} {k} {dtype} {form}")
    rng = np.random.default_rng([n, v, k])
    tau = 1.5
    c = _distill_case(rng, n, v, k, dtype, rest=True, tau=tau)
    t = rng.uniform(3, 14, (n, k))
    lse = np.array([ops._lse(r / tau) for r in t])
    if kind == "small logsumexp":
        lse -= rng.uniform(0.05, 0.8, n)
    elif kind == "bf16 teacher":
        lse += 1e-4
    else:
        c["ids"][:, k // 2:] = c["ids"][:, :k - k // 2]
        t[:, k // 2:] = t[:, :k - k // 2]
        lse = np.array([ops._lse(r[:k // 2] / tau) for r in t]) + 1e-3
        import torch
        c["ids_d"] = torch.from_numpy(c["ids"].astype(np.int32)).cuda()
    _teacher(c, t, lse, "bf16" if kind == "bf16 teacher" else "f32")
    mass = np.exp(c["t64"] / tau - c["lse64"][:, None]).sum(1)
    rows = sorted(set(rng.integers(0, n, 4)) | {0, n - 1, int(np.argmax(mass))})
    assert mass[rows].max() > 1
    _check(c, _distill_run(c, form), form, rows)


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(4, 40), (260, 40), (258, 301), (3, 1), (256, 1024)])
def test_pairs_that_hold_every_token(n, v, dtype, form):
    """No class for the rest, whatever the pairs' mass adds up to."""
    log(f"distill every token {n} {v} {dtype} {form}")
    rng = np.random.default_rng([n, v])
    c = _distill_case(rng, n, v, v, dtype, rest=True, tau=2.0)
    t = rng.uniform(3, 9, (n, v))
    _teacher(c, t, np.array([ops._lse(r / 2.0) for r in t]) + rng.uniform(-0.5, 0.5, n))
    _check(c, _distill_run(c, form), form, sorted(set(rng.integers(0, n, 4)) | {0, n - 1}))


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [1e-2, 1e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("n,v,k", FORMS)
def test_small_tails_keep_their_digits(n, v, k, tail, dtype, form):
    """Little mass left for the rest, and a student that gives it less still: 1 - sum p decides the others' gradient."""
    log(f"distill tail {n} {v} {k} {tail} {dtype} {form}")
    rng = np.random.default_rng([n, v, k])
    tau = 1.5
    c = _distill_case(rng, n, v, k, dtype, rest=True, tau=tau)
    z = c["z64"].copy()
    np.put_along_axis(z, c["ids"], np.take_along_axis(z, c["ids"], 1) + 30.0, 1)
    bits = f32_to_bf16_bits(z.astype(np.float32)) if dtype == "bf16" else z.astype(np.float32)
    c["z64"], c["z"] = host_to_f64(bits, dtype), to_device(bits, dtype)
    t = rng.uniform(3, 14, (n, k)).astype(np.float32).astype(np.float64)
    _teacher(c, t, np.array([ops._lse(r / tau) for r in t]) - np.log1p(-tail))
    _check(c, _distill_run(c, form), form, sorted(set(rng.integers(0, n, 3)) | {0, n - 1}), p_steps=4, mass64=True)


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("dtype,tdtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,v,k", FORMS)
def test_masked_others_and_a_logsumexp_of_the_pairs_alone(n, v, k, dtype, tdtype, form):
    """The student gives every token outside the pairs no mass, and the teacher's logsumexp was taken over the pairs
    alone, in fp32: what its rounding and the teacher logits' leave of 1 - sum p is no mass either. Some rows hold a
    real remainder: their loss is infinite, as the formula says."""
    import torch
    log(f"distill masked others {n} {v} {k} {dtype} {tdtype} {form}")
    rng = np.random.default_rng([n, v, k])
    tau = 1.5
    c = _distill_case(rng, n, v, k, dtype, rest=True, tau=tau)
    z = c["z64"].copy()
    dead = np.ones((n, v), bool)
    np.put_along_axis(dead, c["ids"], False, 1)
    z[dead] = -np.inf
    bits = f32_to_bf16_bits(z.astype(np.float32)) if dtype == "bf16" else z.astype(np.float32)
    c["z64"], c["z"] = host_to_f64(bits, dtype), to_device(bits, dtype)
    t = rng.uniform(3, 14, (n, k)).astype(np.float32)
    scaled = torch.from_numpy(t).cuda() * np.float32(1 / tau)
    lse = torch.logsumexp(scaled, 1).cpu().numpy()
    real = np.arange(n) % 5 == 2
    lse[real] += 0.3
    _teacher(c, t.astype(np.float64), lse, tdtype)
    left = 1 - np.exp(c["t64"] / tau - c["lse64"][:, None]).sum(1)
    if n > 100:
        assert (left[~real] > 0).sum() > 10
    got = _distill_run(c, form)
    loss, dz = _f64(got[0]), _f64(got[3])
    assert np.isposinf(loss[real]).all()
    rows = [i for i in range(n) if not real[i]]
    assert np.isfinite(loss[rows]).all() and np.isfinite(dz[rows]).all() and not dz[rows][dead[rows]].any()
    _check(c, got, form, sorted(set(rng.choice(rows, min(5, len(rows)))) | {rows[0], rows[-1], rows[int(np.argmax(left[rows]))]}))


def test_a_real_remainder_is_kept_where_the_student_gives_it_little_mass():
    """The rule about rounding concerns others without any mass: where they have some, however little, p_r stays."""
    import torch
    log("distill little mass")
    z = torch.full((3, 50), -60.0, device="cuda")
    z[:, :2] = 0
    ids = torch.tensor([[0, 1]] * 3, device="cuda", dtype=torch.int32)
    t = torch.zeros(3, 2, device="cuda")
    lse = torch.full((3,), float(np.log(2.0)) + 2e-7, device="cuda")
    loss, l2, rest = (torch.empty(3, device="cuda") for _ in range(3))
    dz = torch.empty_like(z)
    nsq.ns_distill_topk(z, ids, t, loss, l2, teacher_lse=lse, rest_lse=rest, grad_loss=torch.ones(3, device="cuda"), dlogits=dz)
    torch.cuda.synchronize()
    w = ops.distill_row(z[0].cpu().numpy().astype(np.float64), [0, 1], [0.0, 0.0], 1.0, float(lse[0]))
    assert w["p_rest"] > 0
    assert np.allclose(_f64(dz)[:, 2:], w["dlogits"][2:], rtol=1e-4, atol=0) and np.allclose(_f64(loss), w["loss"], rtol=1e-3)


def _student(c, z, g):
    import torch
    bits = f32_to_bf16_bits(z.astype(np.float32)) if c["dtype"] == "bf16" else z.astype(np.float32)
    c["z64"], c["z"] = host_to_f64(bits, c["dtype"]), to_device(bits, c["dtype"])
    c["g64"] = np.asarray(g, np.float32).astype(np.float64)
    c["g"] = torch.from_numpy(np.asarray(g, np.float32)).cuda()
    c["tdtype"] = "f32"
    return c


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,k", [(3, 9001, 40), (260, 300, 20), (257, 9001, 30), (256, 66001, 64), (256, 140003, 16)])
def test_others_far_above_the_pairs_and_small_loss_gradients(n, v, k, dtype, rest, form):
    """Sums relative to the pairs' logits near 1e30 and loss gradients down to 1e-14: their quotient is below fp32's
    normal numbers, the gradients are not."""
    log(f"distill far above {n} {v} {k} {dtype} {rest} {form}")
    rng = np.random.default_rng([n, v, k])
    c = _distill_case(rng, n, v, k, dtype, rest=rest, tau=1.0)
    z = c["z64"].copy()
    np.put_along_axis(z, c["ids"], np.take_along_axis(z, c["ids"], 1) - rng.uniform(30, 66 - np.log(v), (n, 1)) - 9, 1)
    g = 10.0 ** rng.uniform(-14, -7, n)
    _student(c, z, g)
    _check(c, _distill_run(c, form), form, sorted(set(rng.integers(0, n, 5)) | {0, n - 1, int(np.argmin(g))}))


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [300.0, 3e4, 1e6])
@pytest.mark.parametrize("n,v,k", [(3, 9001, 40), (260, 300, 20), (257, 9001, 30), (256, 140003, 16)])
def test_large_logits(n, v, k, scale, dtype, rest, form):
    """Logits of some `scale` temperatures, many of them tied at the largest value (as bf16 ones are)."""
    log(f"distill large logits {n} {v} {k} {scale} {dtype} {rest} {form}")
    rng = np.random.default_rng([n, v, k])
    tau = float(np.float32(1024.0 / scale))
    c = _distill_case(rng, n, v, k, dtype, rest=rest, tau=tau)
    steps = rng.integers(0, 4, (n, v)) * (rng.random((n, v)) < 0.9) * (rng.random((n, 1)) < 0.8)
    z = rng.uniform(1000, 1400, (n, 1)) - 8.0 * steps
    g = rng.uniform(0.1, 1, n)
    _student(c, z, g)
    t = rng.uniform(3, 9, (n, k)) * tau
    lse = np.array([ops._lse(r.astype(np.float32).astype(np.float64) / tau) for r in t]) + 0.2
    _teacher(c, t, lse)
    if not rest:
        c["lse64"] = c["lse_d"] = None
    _check(c, _distill_run(c, form), form, sorted(set(rng.integers(0, n, 5)) | {0, n - 1}))


@pytest.mark.parametrize("dtype,n,v,k", [
    ("bf16", 3, 262144, 8), ("f32", 3, 262145, 300), ("bf16", 1, 1 << 24, 40),
    ("bf16", 256, 262144, 8), ("bf16", 256, 262144, 300), ("f32", 256, 262144, 1024), ("bf16", 256, 262145, 8),
    ("f32", 256, 262145, 300), ("bf16", 300, 300001, 129), ("bf16", 1030, 262144, 300), ("f32", 1030, 262143, 128),
    ("bf16", 1030, 262145, 300), ("bf16", 1024, 1 << 20, 300), ("bf16", 1025, 786432, 8),
])
def test_vocabularies_around_what_one_workgroup_marks(dtype, n, v, k):
    """With a rest, up to 2^18 tokens are marked in one workgroup's LDS (32 KiB beside up to 37 KiB of pairs) and longer
    rows are split at any row count; both forms, few and many pairs."""
    import torch
    log(f"distill vocabulary {dtype} {n} {v} {k}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(v + n)
    type_ = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    z = torch.randn(n, v, device="cuda", generator=gen, dtype=type_)
    ids = (torch.randint(0, v, (n, 1), device="cuda", generator=gen)
           + torch.arange(k, device="cuda") * (v // k) // 2 * 2 + torch.arange(k, device="cuda") % 2) % v
    ids[:, 0], ids[:, -1] = 0, v - 1
    ids[:, k // 2] = ids[:, k // 2 - 1]                # one token twice
    z.scatter_(1, ids, (torch.rand(n, k, device="cuda", generator=gen) * 6 + 5).to(type_))
    t = torch.rand(n, k, device="cuda", generator=gen) * 6 + 3
    tl = torch.logsumexp(t / 1.5, 1) + 0.01
    g = torch.rand(n, device="cuda", generator=gen) + 0.1
    c = {"tau": 1.5, "dtype": dtype, "tdtype": "f32", "z": z, "ids_d": ids.to(torch.int32), "t": t, "g": g, "lse_d": tl}
    rows = sorted({0, n // 2, n - 1}) if v < 1 << 20 else [n - 1]
    pick = torch.tensor(rows, device="cuda")
    c64 = dict(c, z64=_f64(z[pick]), ids=ids[pick].cpu().numpy(), t64=_f64(t[pick]), g64=_f64(g[pick]), lse64=_f64(tl[pick]))
    for form in ("train", "step"):
        got = _distill_run(c, form)
        _check(c64, tuple(x[pick] for x in got), form, range(len(rows)))


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("below", [0.0, 1.5, 3.0])
@pytest.mark.parametrize("n,v,k", [(3, 9001, 40), (260, 300, 20), (257, 2602, 9), (256, 33001, 24), (256, 140003, 16)])
def test_others_below_the_pairs_over_a_wide_range(n, v, k, below, dtype, form):
    """At a low temperature the others' shares of their class run from 1 down to 1e-40, and the class lies up to 1e-9
    below the pairs: shares of 1e-30 are numbers of either type."""
    log(f"distill wide range {n} {v} {k} {below} {dtype} {form}")
    rng = np.random.default_rng([n, v, k])
    tau = 0.125
    c = _distill_case(rng, n, v, k, dtype, rest=True, tau=tau)
    z = rng.standard_normal((n, v)) * 2 - 8.0 - below
    for i in range(n):
        z[i, c["ids"][i]] = rng.uniform(0, 0.5, k)
    z[:, v - 2:] = z.max(1, keepdims=True) - 9.0 - below     # the last ones, too
    c["ids"] = c["ids"] % (v - 2)
    import torch
    c["ids_d"] = torch.from_numpy(c["ids"].astype(np.int32)).cuda()
    _student(c, z, rng.uniform(0.01, 0.1, n))
    t = rng.uniform(3, 9, (n, k)) * tau
    _teacher(c, t, np.array([ops._lse(r / tau) for r in t]) + rng.uniform(0.01, 0.5, n))
    _check(c, _distill_run(c, form), form, sorted(set(rng.integers(0, n, 5)) | {0, n - 1}))


@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [900.0, 3e3, 1e5, 1e7])
@pytest.mark.parametrize("n,v,k", [(3, 9001, 40), (260, 300, 20), (257, 20003, 300), (5, 140003, 16)])
def test_gradient_alone_where_the_logsumexp_is_large(n, v, k, scale, dtype, rest, place):
    """An fp32 logsumexp of 1e5 is 4e-3 off: from 1024 on the second call sums such rows again, next to ordinary ones."""
    log(f"distill gradient alone {n} {v} {k} {scale} {dtype} {rest} {place}")
    rng = np.random.default_rng([n, v, k])
    tau = float(np.float32(1000.0 / scale))
    c = _distill_case(rng, n, v, k, dtype, rest=rest, tau=tau)
    z = 8.0 * rng.integers(-2, 2, (n, v)) * (rng.random((n, 1)) < 0.7) + rng.choice([-1024.0, 0.0, 1024.0], (n, 1))
    _student(c, z, rng.uniform(0.1, 1, n))
    t = rng.uniform(3, 9, (n, k)) * tau
    _teacher(c, t, np.array([ops._lse(r.astype(np.float32).astype(np.float64) / tau) for r in t]) + 0.2)
    if not rest:
        c["lse64"] = c["lse_d"] = None
    got = _distill_run(c, "step", place=place)
    _check(c, got, "step", sorted(set(rng.integers(0, n, 6)) | {0, n - 1}), most=1024.0)


@pytest.mark.parametrize("form", ["train", "step"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.3, 1.0, 1.7])
@pytest.mark.parametrize("n,v,k", [(4, 5003, 6), (260, 300, 20), (257, 9001, 200)])
def test_rows_masked_whole_by_the_lowest_value(n, v, k, tau, dtype, rest, form):
    """Every logit the type's lowest value, or all but the pairs': the shares are equal, whatever the temperature makes
    of the logsumexp (its quotient by a temperature below 1 is -inf)."""
    log(f"distill lowest rows {n} {v} {k} {tau} {dtype} {rest} {form}")
    rng = np.random.default_rng([n, v, k])
    tau = float(np.float32(tau))
    c = _distill_case(rng, n, v, k, dtype, rest=rest, tau=tau)
    z = c["z64"].copy()
    low = -3.3895313892515355e38 if dtype == "bf16" else -3.4028234663852886e38
    inside = np.zeros((n, v), bool)
    np.put_along_axis(inside, c["ids"], True, 1)
    z[0::3] = low
    z[1::3] = np.where(inside[1::3], z[1::3], low)
    _student(c, z, rng.uniform(0.1, 1, n))
    t = rng.uniform(3, 9, (n, k)) * tau
    _teacher(c, t, np.array([ops._lse(r.astype(np.float32).astype(np.float64) / tau) for r in t]) + 0.2)
    if not rest:
        c["lse64"] = c["lse_d"] = None
    loss, lse, rest_lse, dz = _distill_run(c, form)
    dz, loss = _f64(dz), _f64(loss)
    assert np.isfinite(dz).all()
    for i in (0, 1, 2, 3, n - 1):
        tl = None if not rest else c["lse64"][i]
        w = ops.distill_row(c["z64"][i], c["ids"][i], c["t64"][i], tau, tl, c["g64"][i])
        if i % 3 == 0:   # q is 1 / v: p from fp32 exponents of t / tau up to 9, sums of 9001 equal terms
            size = c["g64"][i] / tau * (1 / v + np.bincount(c["ids"][i], w["p"], v))
            _close(dz[i], w["dlogits"], (HALF_STEP[dtype] + 8 * U) * np.abs(w["dlogits"]) + 256 * U * size, f"row {i}")
            assert abs(loss[i] - w["loss"]) <= 256 * U * (1 + np.log(v))
        elif i % 3 == 1 and rest:   # the others share g p_r / tau equally; their q is 0 in 64 bits, too
            others = -c["g64"][i] / tau * w["p_rest"] / (v - k)
            _close(dz[i][~inside[i]], np.full(v - k, others), (HALF_STEP[dtype] + 256 * U) * abs(others), f"row {i} others")
