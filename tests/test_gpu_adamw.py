"""nvfp4_adamw on the GPU against the 64-bit oracle.

Tolerances, u = 2^-24 (one FP32 rounding). m' = b1 m + (1 - b1) g takes five roundings (two
constants, two products, one sum): 5u (|b1 m| + |(1 - b1) g|) =: dm. v' likewise, with g^2 one
more and no cancellation: 6u v'. sqrt halves that and rounds: 4u; the denominator (constant,
product, eps, sum) 8u; the quotient and its factor (constant, division, product) 4u more, so
the update is off by step/denom * dm + 12u |update|; p (1 - lr wd) and the last sum round four
times: 4u (|p| + |update|). Clipping: a thread's FP32 sum of 32 squares is within 34u, the square
root halves that and the quotient rounds three times: 20u on c, so 21u more on g and 42u on v.
8-bit states: the code has to be one that the rule gives for a value within that distance of the
64-bit one (plus 3u for sqrt and scaling)."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
from helpers import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HP = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _host(t):
    return t.float().cpu().numpy() if t.dtype != torch.uint8 else t.cpu().numpy()


def _at(values, offset, dtype=torch.float32):
    """A GPU tensor holding values that starts `offset` elements into its allocation."""
    buf = torch.zeros((len(values) + offset + 8,), dtype=dtype, device="cuda")
    buf[offset:offset + len(values)] = torch.as_tensor(np.ascontiguousarray(values)).to(dtype).cuda()
    return buf[offset:offset + len(values)]


def _case(n, seed, grad_dtype, eight, offset, decay, w):
    rng = np.random.default_rng(seed)
    p, g = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    g[rng.random(n) < 0.1] = 0
    m = (0.3 * rng.standard_normal(n)).astype(np.float32)
    v = np.square(rng.standard_normal(n)).astype(np.float32)
    v[rng.random(n) < 0.05] = 0
    if n >= 96:
        g[32:64] = m[32:64] = v[32:64] = 0                          # a block with nothing in it
        m[64:96] *= np.float32(2.0) ** rng.integers(-30, 1, 32)     # a block over many binades
        v[64:96] *= np.float32(2.0) ** rng.integers(-60, 1, 32)
    g = _at(g, offset, grad_dtype)
    kw = dict(p=_at(p, offset), grad=g, weight_decay=decay)
    if eight:
        for k, x in (("m", m), ("v", np.sqrt(v))):
            e = oracle.state_scale_exponents(x)
            c = oracle.state_codes(x, e, np.full(n, 32768), k == "v")
            kw[k] = _at(c, offset, torch.uint8)
            kw[k + "_scale"] = _at((e + 127).astype(np.uint8), 0, torch.uint8)
    else:
        kw.update(m=_at(m, offset), v=_at(v, offset))
    if w:
        kw["w_out"] = _at(np.zeros(n, np.float32), offset, torch.bfloat16)
    return nv.AdamWTensor(**kw)


def _state(t, k):
    x = _host(getattr(t, k))
    if t.m.dtype != torch.uint8:
        return x.astype(np.float64)
    r = oracle.state_values(x, _host(getattr(t, k + "_scale")).astype(np.int64) - 127)
    return r if k == "m" else r * r


def _snapshot(t):
    return dict(p=_host(t.p).astype(np.float64), g=_host(t.grad).astype(np.float64), m=_state(t, "m"), v=_state(t, "v"))


def _check(t, old, i, step, clip, clipped, seed, wd):
    b1, b2 = HP["betas"]
    p, m, v = oracle.adamw64(old["p"], old["g"], old["m"], old["v"], HP["lr"], b1, b2, HP["eps"], step, wd, clip)
    more = 21 * U if clipped else 0.0
    dm = (5 * U + more) * (np.abs(b1 * old["m"]) + np.abs((1 - b1) * clip * old["g"])) + 1e-44
    dv = (6 * U + 2 * more) * v + 1e-44
    bc1, bc2 = 1 - b1 ** step, 1 - b2 ** step
    denom = np.sqrt(v / bc2) + HP["eps"]
    upd = HP["lr"] / bc1 * m / denom
    dp = HP["lr"] / bc1 * dm / denom + (12 * U + more) * np.abs(upd) + 4 * U * (np.abs(old["p"]) + np.abs(upd))
    got = _host(t.p_out if t.p_out is not None else t.p).astype(np.float64)
    assert np.all(np.abs(got - p) <= dp), f"p of tensor {i}"
    if t.w_out is not None:
        assert np.array_equal(_host(t.w_out), oracle.round_bf16(got.astype(np.float32)))
    mo, vo = t.m_out if t.m_out is not None else t.m, t.v_out if t.v_out is not None else t.v
    if t.m.dtype != torch.uint8:
        assert np.all(np.abs(_host(mo) - m) <= dm), f"m of tensor {i}"
        assert np.all(np.abs(_host(vo) - v) <= dv), f"v of tensor {i}"
        return
    h = oracle.state_random(len(m), i, step, seed)
    so = {k: getattr(t, k + "_scale_out") if getattr(t, k + "_scale_out") is not None else getattr(t, k + "_scale")
          for k in "mv"}
    for k, x, dx, c in (("m", m, dm, mo), ("v", np.sqrt(v), (3 * U + more) * np.sqrt(v) + 1e-22, vo)):
        e = oracle.state_scale_exponents(x)
        assert np.array_equal(_host(so[k]).astype(np.int64) - 127, e), f"scales of {k}, tensor {i}"
        dx = dx + 3 * U * np.abs(x) + 3 * U * 2.0 ** np.repeat(e, 32)[: len(x)] / 512
        got = _host(c)
        ok = np.zeros(len(x), bool)
        for y in (x - dx, x, x + dx):
            y = np.where(np.sign(y) == np.sign(x), y, 0.0) if k == "v" else y
            want = oracle.state_codes(y, e, h, k == "v" )
            # a value whose own sign is open may come with either sign of zero
            ok |= (want == got) | ((want & 127 == 0) & (got & 127 == 0))
        assert ok.all(), f"codes of {k}, tensor {i}: {np.flatnonzero(~ok)[:5]}"


SIZES = [1, 7, 8, 31, 32, 33, 257, 2048, 8191, 8192, 8193, 20000]


@pytest.mark.parametrize("eight", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16], ids=["g32", "g16"])
@pytest.mark.parametrize("offset", [0, 3], ids=["aligned", "odd"])
@pytest.mark.parametrize("clip", [None, 0.5, 1e6])
def test_step(eight, grad_dtype, offset, clip):
    log(f"adamw eight={eight} {grad_dtype} offset={offset} clip={clip}")
    ts = [_case(n, 40 + i, grad_dtype, eight, offset, 0.1 * (i % 2), i % 3 != 0) for i, n in enumerate(SIZES)]
    plan = nv.AdamWPlan(ts)
    seed = (0xABC << 32) | 0x1234567
    amax = torch.full((len(ts),), -1.0, device="cuda")
    for step in (1, 2, 100):
        old = [_snapshot(t) for t in ts]
        norm = nv.adamw(plan, step=step, max_norm=clip, seed=seed, amax_out=amax, **HP)
        torch.cuda.synchronize()
        c = 1.0
        if clip is not None:
            n64 = np.sqrt(sum(np.square(o["g"]).sum() for o in old))
            assert abs(norm.item() - n64) <= 20 * U * n64
            c = min(1.0, clip / (n64 + 1e-6))
        for i, (t, o) in enumerate(zip(ts, old)):
            _check(t, o, i, step, c, clip is not None, seed, 0.1 * (i % 2))
            stored = t.w_out if t.w_out is not None else t.p
            assert amax[i].item() == np.abs(_host(stored)).max()


@pytest.mark.parametrize("eight", [False, True], ids=["fp32", "8bit"])
def test_outputs_apart_from_inputs(eight):
    """Separate outputs get what the step in place gets, and the inputs stay."""
    log(f"adamw out of place eight={eight}")
    a = [_case(n, 70 + n, torch.float32, eight, 0, 0.1, True) for n in (5, 4097, 9000)]
    b = [_case(n, 70 + n, torch.float32, eight, 0, 0.1, True) for n in (5, 4097, 9000)]
    for t in b:
        t.p_out, t.m_out, t.v_out = torch.zeros_like(t.p), torch.zeros_like(t.m), torch.zeros_like(t.v)
        if eight:
            t.m_scale_out, t.v_scale_out = torch.zeros_like(t.m_scale), torch.zeros_like(t.v_scale)
    keep = [t.p.clone() for t in b]
    for ts in (a, b):
        nv.adamw(nv.AdamWPlan(ts), step=3, max_norm=1.0, seed=5, **HP)
    torch.cuda.synchronize()
    for s, t, k in zip(a, b, keep):
        assert torch.equal(t.p, k) and torch.equal(s.p, t.p_out) and torch.equal(s.w_out, t.w_out)
        for name in ("m", "v") + (("m_scale", "v_scale") if eight else ()):
            assert torch.equal(getattr(s, name), getattr(t, name + "_out")), name


@pytest.mark.parametrize("eight", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e30])
def test_norm_without_a_value_changes_nothing(eight, bad):
    log(f"adamw bad norm eight={eight} {bad}")
    ts = [_case(n, 90 + n, torch.float32, eight, 0, 0.1, True) for n in (100, 8200)]
    ts[1].grad[8195] = bad                                           # 1e30: its square leaves FP32
    names = ("p", "m", "v") + (("m_scale", "v_scale") if eight else ())
    old = [{k: getattr(t, k).clone() for k in names} for t in ts]
    norm = nv.adamw(nv.AdamWPlan(ts), step=2, max_norm=1.0, seed=5, **HP)
    torch.cuda.synchronize()
    assert not np.isfinite(norm.item())
    for t, o in zip(ts, old):
        assert all(torch.equal(getattr(t, k), o[k]) for k in names)
        assert torch.equal(t.w_out, t.p.bfloat16())


def test_bit_reproducible_on_another_stream():
    log("adamw streams")
    got = []
    for stream in (None, torch.cuda.Stream()):
        ts = [_case(n, 110 + n, torch.float32, True, 0, 0.1, True) for n in (333, 30000)]
        plan = nv.AdamWPlan(ts)
        torch.cuda.synchronize()
        norm = nv.adamw(plan, step=9, max_norm=1.0, seed=77, stream=stream, **HP)
        torch.cuda.synchronize()
        got.append([norm] + [x for t in ts for x in (t.p, t.m, t.v, t.m_scale, t.v_scale, t.w_out)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_running_mean_does_not_stall():
    """With no gradient r = sqrt(v) shrinks by sqrt(b2) a step, far less than an E4M3 gap: its
    mean over many elements has to follow. Truncating 16 bits loses at most gap / 2^17 on average
    a step (gap <= r / 8), 400 steps of it below 4e-4 relative; the mean of 65536 elements
    scatters by at most 400 * gap / 2 / 256 / sqrt(400) < 0.3% of r (errors of one step are
    independent, each at most half a gap in deviation). Bound: 1.5% (five deviations)."""
    log("adamw 8-bit decay")
    n, b2, steps = 65536, 0.999, 400
    rng = np.random.default_rng(1)
    r0 = rng.uniform(0.5, 1.0, n)
    e = oracle.state_scale_exponents(r0)
    z = torch.zeros((n,), device="cuda")
    t = nv.AdamWTensor(p=z.clone(), grad=z, m=torch.zeros((n,), dtype=torch.uint8, device="cuda"),
                       v=_at(oracle.state_codes(r0, e, np.full(n, 32768), True), 0, torch.uint8),
                       m_scale=torch.zeros((n // 32,), dtype=torch.uint8, device="cuda"),
                       v_scale=_at((e + 127).astype(np.uint8), 0, torch.uint8))
    before = np.sqrt(_state(t, "v")).mean()
    plan = nv.AdamWPlan([t])
    for step in range(1, steps + 1):
        nv.adamw(plan, lr=1e-3, betas=(0.9, b2), eps=1e-8, step=step, seed=3)
    torch.cuda.synchronize()
    assert abs(np.sqrt(_state(t, "v")).mean() / (before * b2 ** (steps / 2)) - 1) < 0.015
    assert torch.count_nonzero(t.p).item() == 0


def test_refusals():
    t = _case(64, 1, torch.float32, False, 0, 0.1, True)
    with pytest.raises(nv.NVFP4Error, match="at least one"):
        nv.AdamWPlan([])
    with pytest.raises(nv.NVFP4Error, match="grad"):
        nv.AdamWPlan([nv.AdamWTensor(p=t.p, grad=t.grad[:32], m=t.m, v=t.v)])
    with pytest.raises(nv.NVFP4Error, match="grad"):
        nv.AdamWPlan([nv.AdamWTensor(p=t.p, grad=t.grad.half(), m=t.m, v=t.v)])
    with pytest.raises(nv.NVFP4Error, match="m must be"):
        nv.AdamWPlan([nv.AdamWTensor(p=t.p, grad=t.grad, m=t.m.cpu(), v=t.v)])
    with pytest.raises(nv.NVFP4Error, match="contiguous"):
        wide = torch.zeros((128,), device="cuda")
        nv.AdamWPlan([nv.AdamWTensor(p=t.p, grad=wide[::2], m=t.m, v=t.v)])
    with pytest.raises(nv.NVFP4Error, match="v_scale"):
        u = _case(64, 1, torch.float32, True, 0, 0.1, True)
        nv.AdamWPlan([nv.AdamWTensor(p=u.p, grad=u.grad, m=u.m, v=u.v, m_scale=u.m_scale, v_scale=u.v_scale[:1])])
    plan = nv.AdamWPlan([t])
    for kw in (dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0), dict(step=0)):
        with pytest.raises(nv.NVFP4Error, match="out of range"):
            nv.adamw(plan, **{**HP, "step": 1, **kw})
    with pytest.raises(nv.NVFP4Error, match="workspace"):
        nv.adamw(plan, step=1, max_norm=1.0, workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"), **HP)


def test_empty_tensors():
    log("adamw empty")
    z = torch.zeros((0,), device="cuda")
    t = _case(40, 3, torch.float32, False, 0, 0.0, True)
    old = _snapshot(t)
    plan = nv.AdamWPlan([nv.AdamWTensor(p=z, grad=z, m=z, v=z), t, nv.AdamWTensor(p=z, grad=z, m=z, v=z)])
    nv.adamw(plan, step=1, **HP)
    torch.cuda.synchronize()
    _check(t, old, 1, 1, 1.0, False, 0, 0.0)
    norm = nv.adamw(nv.AdamWPlan([nv.AdamWTensor(p=z, grad=z, m=z, v=z)]), step=1, max_norm=1.0, **HP)
    assert norm.item() == 0.0
