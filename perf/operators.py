"""Cases of the layer operators: gemm_act (NVFP4 matrix product with bias, activation and residual),
act_grad (its backward), adamw (one optimizer step over many tensors, 32-bit or 8-bit states) and
moe_tokens (a whole mixture-of-experts layer for a few tokens), each with a plain form in
elementary torch operations on FP32.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---- the cases -------------------------------------------------------------------------------
def listed():
    return [
        # the MLP up-projection of the dense layer (8192 tokens, 5120 -> 20480) with what follows it,
        # and the pre-activation that its backward needs
        dict(name="gemm_act up-projection", op="gemm_act", m=8192, n=20480, k=5120, act="relu2", bias="bf16",
             residual=False, preact=True),
        # the down-projection back into the residual stream
        dict(name="gemm_act down, residual", op="gemm_act", m=8192, n=5120, k=20480, act="none", bias="fp32",
             residual=True, preact=False),
        # the same up-projection while one token is generated
        dict(name="gemm_act one token", op="gemm_act", m=1, n=20480, k=5120, act="gelu", bias="bf16",
             residual=False, preact=False),
        # a short ragged batch on an expert-sized layer whose contraction ends inside a 64-element step
        dict(name="gemm_act ragged", op="gemm_act", m=1003, n=1857, k=2704, act="silu", bias="fp32",
             residual=True, preact=True),
        # backward of the up-projection's activation and bias over the whole batch
        dict(name="act_grad up-projection", op="act_grad", m=8192, n=20480, act="relu2", dy="bf16"),
        # a ragged micro-batch, FP32 gradients, odd width
        dict(name="act_grad ragged", op="act_grad", m=123, n=1857, act="gelu", dy="fp32"),
        # biases and norms of a few layers: many tiny tensors, latency counts
        dict(name="adamw biases", op="adamw", sizes="20480,5120,5120,5120,17,1,20480,5120,5120,5120,333,16",
             state="fp32", grad="fp32", clip=False),
        # the dense layer's weights and biases, FP32 main gradient, clipped by the gradient's norm
        dict(name="adamw layer, 32 bits", op="adamw", sizes="104857600,20480,104857600,5120", state="fp32",
             grad="fp32", clip=True),
        # expert weights and a ragged rest with the states in 8 bits
        dict(name="adamw experts, 8 bits", op="adamw",
             sizes=",".join(["4988928"] * 16 + ["344064", "2688", "1857", "1856", "101", "5120"]), state="8bit",
             grad="fp32", clip=False),
        # the expert layer (128 experts, top 6, 2688 -> 1856) while one token is generated
        dict(name="moe one token", op="moe", t=1, e=128, h=2688, f=1856, k=6, act="relu2", gated=False,
             score="sigmoid"),
        # a few sequences on a small gated expert layer, odd sizes
        dict(name="moe gated, 7 tokens", op="moe", t=7, e=24, h=1040, f=720, k=3, act="silu", gated=True,
             score="softmax"),
        # the expert layer for a batch of 64 sequences: nearly every expert is read
        dict(name="moe 64 tokens", op="moe", t=64, e=128, h=2688, f=1856, k=6, act="relu2", gated=False,
             score="sigmoid"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm_act", "gemm_act", "act_grad", "adamw", "adamw", "moe", "moe"])
    act = rng.choice(["none", "relu2", "gelu", "silu"])
    if op == "gemm_act":
        return dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 16, 10240),
                    k=16 * _log_int(rng, 4, 640), act=act, bias=rng.choice(["none", "bf16", "fp32"]),
                    residual=rng.random() < 0.5, preact=rng.random() < 0.5)
    if op == "act_grad":
        return dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 16, 20480), act=act,
                    dy=rng.choice(["bf16", "fp32"]))
    if op == "adamw":
        total, sizes = _log_int(rng, 10_000, 60_000_000), []
        count = _log_int(rng, 1, 48)
        for _ in range(count):
            sizes.append(max(1, int(total / count * rng.uniform(0.01, 1.9))))
        return dict(op=op, sizes=",".join(str(s) for s in sizes), state=rng.choice(["fp32", "8bit"]),
                    grad=rng.choice(["fp32", "bf16"]), clip=rng.random() < 0.5)
    e = _log_int(rng, 4, 128)
    return dict(op="moe", t=_log_int(rng, 1, 64), e=e, h=16 * _log_int(rng, 8, 168), f=16 * _log_int(rng, 8, 116),
                k=rng.randint(1, min(8, e)), act=rng.choice(["relu2", "gelu", "silu"]), gated=rng.random() < 0.4,
                score=rng.choice(["softmax", "sigmoid"]))


# ---- inputs ----------------------------------------------------------------------------------
_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std)


def _outliers(g, x, frac=1e-3, factor=50.0):
    """Activations: 0.1% of the entries 50 times larger."""
    return torch.where(torch.rand(x.shape, generator=g, device=DEV) < frac, x * factor, x)


def _to_nvfp4(x, groups=1):
    """x [groups*rows, cols] FP32 -> codes, E4M3 scales, one tensor scale per group (1x16 blocks)."""
    rows, cols = x.shape
    amax = x.reshape(groups, -1).abs().amax(1).clamp_min_(1e-30)
    s_dec = amax / 2688.0
    blocks = x.reshape(groups, -1, 16) / s_dec[:, None, None]
    scales = (blocks.abs().amax(2) / 6.0).clamp_(max=448.0).to(torch.float8_e4m3fn)
    y = blocks / scales.float().clamp_min(2.0 ** -9)[:, :, None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(y.abs(), mids, out_int32=True).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    code = code.reshape(rows, cols // 2, 2)
    codes = code[:, :, 0] | (code[:, :, 1] << 4)
    return codes.contiguous(), scales.view(torch.uint8).reshape(rows, cols // 16).contiguous(), s_dec


def _nvfp4_normal(g, rows, cols, std, groups=1, outliers=False):
    x = _randn(g, (rows, cols), std)
    return _to_nvfp4(_outliers(g, x) if outliers else x, groups)


def _sizes(case):
    return [int(s) for s in case["sizes"].split(",")]


def _starts(sizes):
    """First element of each tensor in the flat buffers (multiples of 64), and their length."""
    at, out = 0, []
    for n in sizes:
        out.append(at)
        at += (n + 63) // 64 * 64
    return out, at


LR, B1, B2, EPS, STEP, MAX_NORM = 3e-4, 0.9, 0.95, 1e-8, 100, 1.0


def prepare(case, seed):
    g = _gen(seed)
    op, st = case["op"], {"case": dict(case)}
    if op == "gemm_act":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"] = _nvfp4_normal(g, m, k, 1.0, outliers=True)
        st["b"] = _nvfp4_normal(g, n, k, 0.02)
        bias = _randn(g, (n,), 0.1)
        st["bias"] = {"none": None, "bf16": bias.bfloat16(), "fp32": bias}[case["bias"]]
        st["residual"] = _randn(g, (m, n)).bfloat16() if case["residual"] else None
    elif op == "act_grad":
        m, n = case["m"], case["n"]
        dy = _randn(g, (m, n), 1e-3)
        st["dy"] = dy if case["dy"] == "fp32" else dy.bfloat16()
        st["z"] = _randn(g, (m, n), 1.5).bfloat16()
    elif op == "adamw":
        _prepare_adamw(st, case, g, seed)
    else:
        _prepare_moe(st, case, g)
    if own:
        _handles(st)
    return st


def _prepare_adamw(st, case, g, seed):
    sizes = _sizes(case)
    starts, total = _starts(sizes)
    n_of, at = torch.tensor(sizes, device=DEV), torch.tensor(starts, device=DEV)
    spans = torch.tensor([b - a for a, b in zip(starts, starts[1:] + [total])], device=DEV)
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), spans, output_size=total)
    inside = torch.arange(total, device=DEV) - at[tensor] < n_of[tensor]
    decay = torch.tensor([0.1 if n > 30_000 else 0.0 for n in sizes], device=DEV)   # none on biases and norms
    p = _randn(g, (total,), 0.02) * inside
    grad = _randn(g, (total,), 1e-3) * inside
    grad *= torch.rand(total, generator=g, device=DEV) > 0.05                       # entries no token touched
    m = _randn(g, (total,), 3e-4) * inside
    v = (_randn(g, (total,), 1e-3) * inside).square() * 0.5
    st.update(sizes=sizes, starts=starts, total=total, p=p, decay=decay,
              grad=grad if case["grad"] == "fp32" else grad.bfloat16(), seed=int(seed) % 100003,
              decay_at=decay[tensor], tensor8=tensor[::8].contiguous(),
              group8=((torch.arange(total, device=DEV) - at[tensor]) // 8)[::8].contiguous())
    if case["state"] == "8bit":
        st["m8"], st["r8"] = _nearest8(m), _nearest8(v.sqrt())
    else:
        st["m"], st["v"] = m, v


def _prepare_moe(st, case, g):
    t, e, h, f = case["t"], case["e"], case["h"], case["f"]
    f1 = 2 * f if case["gated"] else f
    st["x"] = _outliers(g, _randn(g, (t, h))).bfloat16()
    st["router"] = _randn(g, (e, h), h ** -0.5).bfloat16()
    st["w1"] = _nvfp4_normal(g, e * f1, h, h ** -0.5, groups=e)
    st["w2"] = _nvfp4_normal(g, e * h, f, f ** -0.5, groups=e)


def _handles(st):
    """What a user's program keeps between calls: the optimizer's plan, the expert layer's handle."""
    import bit_block_scaled_quantize_amd as nv
    c = st["case"]
    if c["op"] == "adamw":
        eight = c["state"] == "8bit"
        like = lambda x: torch.empty_like(x)  # noqa: E731
        st["out"] = {"p": like(st["p"]), "w": torch.zeros(st["total"], dtype=torch.bfloat16, device=DEV)}
        st["out"]["p"].zero_()
        keys = [("m8", 0), ("m8", 1), ("r8", 0), ("r8", 1)] if eight else [("m", None), ("v", None)]
        for key, i in keys:
            src = st[key] if i is None else st[key][i]
            st["out"][key, i] = torch.zeros_like(src)
        entries = []
        for i, (at, n) in enumerate(zip(st["starts"], st["sizes"])):
            cut, cut32 = slice(at, at + n), slice(at // 32, at // 32 + (n + 31) // 32)
            o = st["out"]
            kw = dict(p=st["p"][cut], grad=st["grad"][cut], p_out=o["p"][cut], w_out=o["w"][cut],
                      weight_decay=float(st["decay"][i]))
            if eight:
                kw.update(m=st["m8"][0][cut], m_scale=st["m8"][1][cut32], v=st["r8"][0][cut], v_scale=st["r8"][1][cut32],
                          m_out=o["m8", 0][cut], m_scale_out=o["m8", 1][cut32], v_out=o["r8", 0][cut],
                          v_scale_out=o["r8", 1][cut32])
            else:
                kw.update(m=st["m"][cut], v=st["v"][cut], m_out=o["m", None][cut], v_out=o["v", None][cut])
            entries.append(nv.AdamWTensor(**kw))
        st["plan"] = nv.AdamWPlan(entries)
    elif c["op"] == "moe":
        from bit_block_scaled_quantize_amd.moe import MoETokens
        w1, w2 = _tensor(nv, st["w1"]), _tensor(nv, st["w2"])
        st["layer"] = MoETokens(st["router"], w1, w2, top_k=c["k"], activation=c["act"], gated=c["gated"],
                                score=c["score"])


def _tensor(nv, q):
    codes, scales, gs = q
    return nv.NVFP4Tensor(codes, scales, gs, codes.shape[0], codes.shape[1] * 2)


# ---- one pass --------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "gemm_act":
        return _own_gemm_act(state) if own else _plain_gemm_act(state)
    if op == "act_grad":
        return _own_act_grad(state) if own else _plain_act_grad(state)
    if op == "adamw":
        return _own_adamw(state) if own else _plain_adamw(state)
    return _own_moe(state) if own else _plain_moe(state)


def _own_gemm_act(st):
    import bit_block_scaled_quantize_amd as nv
    c = st["case"]
    a, b = _tensor(nv, st["a"]), _tensor(nv, st["b"])
    z = torch.empty((c["m"], c["n"]), dtype=torch.bfloat16, device=DEV) if c["preact"] else None
    amax = torch.empty((1,), device=DEV)
    d = nv.gemm_act(a, b, bias=st["bias"], activation=c["act"], residual=st["residual"], preact=z, amax_out=amax)
    return {"d": d, "z": z, "amax": amax.view(torch.bfloat16)[1:]}       # a value of D: BF16


def _own_act_grad(st):
    import bit_block_scaled_quantize_amd as nv
    dbias = torch.empty((st["z"].shape[1],), device=DEV)
    dz = nv.act_grad(st["dy"], st["z"], activation=st["case"]["act"], dbias=dbias)
    return {"dz": dz, "dbias": dbias}


def _own_adamw(st):
    import bit_block_scaled_quantize_amd as nv
    clip = st["case"]["clip"]
    norm = torch.empty((1,), device=DEV) if clip else None
    nv.adamw(st["plan"], lr=LR, betas=(B1, B2), eps=EPS, step=STEP, max_norm=MAX_NORM if clip else None,
             norm_out=norm, seed=st["seed"])
    o = st["out"]
    if st["case"]["state"] == "8bit":                             # the values that codes and scales hold
        m = o["m8", 0].view(torch.float8_e4m3fn), o["m8", 1].view(torch.float8_e8m0fnu)
        v = o["r8", 0].view(torch.float8_e4m3fn), o["r8", 1].view(torch.float8_e8m0fnu)
    else:
        m, v = o["m", None], o["v", None]
    return {"p": o["p"], "w": o["w"], "m": m, "v": v, "norm": norm}


def _own_moe(st):
    return st["layer"](st["x"])


def _lut(device):
    v = torch.tensor(_GRID + [-x for x in _GRID], device=device)
    return torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)           # byte -> (low, high) nibble


def _dequantize(codes, scales, gs):
    """FP32 values; gs holds one scale for all rows, or one for each equal run of rows."""
    v = _lut(codes.device)[codes.int()].reshape(*scales.shape, 16)
    v = v * scales.view(torch.float8_e4m3fn).float()[..., None]
    v = v.reshape(gs.numel(), -1) * gs.reshape(-1, 1)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _act(z, kind):
    if kind == "relu2":
        r = z.clamp_min(0.0)
        return r * r
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "relu2":
        return 2.0 * z.clamp_min(0.0)
    if kind == "gelu":
        th = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * 0.7978845608028654 * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain_gemm_act(st):
    c = st["case"]
    z = _dequantize(*st["a"]) @ _dequantize(*st["b"]).t()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    d = _act(z, c["act"])
    if st["residual"] is not None:
        d = d + st["residual"].float()
    d = d.bfloat16()
    return {"d": d, "z": z.bfloat16() if c["preact"] else None, "amax": d.abs().amax().reshape(1)}


def _plain_act_grad(st):
    dz = st["dy"].float() * _act_slope(st["z"].float(), st["case"]["act"])
    return {"dz": dz.bfloat16(), "dbias": dz.sum(0)}


def _scale8(x):
    """The exponent e (per 32 elements) of the smallest power of two with max|x| <= 448 * 2^e."""
    top = x.reshape(-1, 32).abs().amax(1)
    frac, ex = torch.frexp(top)                                   # top = frac * 2^ex, frac in [0.5, 1)
    e = torch.where(frac > 0.875, ex - 8, ex - 9)
    return torch.where(top > 0, e.clamp_min(-117), torch.full_like(e, -127))


def _pow2(e):
    """2^e in FP32 from its bit field (0 for e = -127, the scale of an all-zero block)."""
    return ((e + 127).int() << 23).view(torch.float32)


def _nearest8(x):
    e = _scale8(x)
    y = x.reshape(-1, 32) * _pow2(-e)[:, None]
    return y.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), (e + 127).to(torch.uint8)


def _value8(codes, scales):
    """What codes and scales stand for, in FP32."""
    v = codes.view(torch.float8_e4m3fn).float().reshape(-1, 32)
    return (v * _pow2(scales.int() - 127)[:, None]).reshape(-1)


def _philox_words(group, tensor, step, seed):
    """Philox4x32-10 of counter (group, 0, step, tensor) and key (seed, 0): four words per group."""
    mask = 0xFFFFFFFF
    x0, x1, x2, x3 = group, torch.zeros_like(group), torch.full_like(group, step), tensor
    k0, k1 = seed & mask, (seed >> 32) & mask
    rounds = [((k0 + 0x9E3779B9 * i) & mask, (k1 + 0xBB67AE85 * i) & mask) for i in range(10)]
    for a, b in rounds:
        p, q = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((q >> 32) & mask) ^ x1 ^ a, q & mask, ((p >> 32) & mask) ^ x3 ^ b, p & mask
    return x0, x1, x2, x3


def _halves8(words):
    """The eight 16-bit halves of four words, low half first."""
    w = torch.stack(words, 1)
    return torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1).int()


def _stochastic8(x, rnd, keep_nonzero):
    """x rounded to E4M3 times its block's scale: up where fraction + rnd/65536 reaches one."""
    e = _scale8(x).repeat_interleave(32)
    y = x.abs() * _pow2(-e)
    fine = ((y.view(torch.int32) + (rnd << 4)) & ~0xFFFFF).view(torch.float32)
    low = torch.floor(y * 512.0 + rnd.float() / 65536.0) / 512.0
    q = torch.where(y < 2.0 ** -6, low, fine)
    if keep_nonzero:
        q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
    unit = (e[::32] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return torch.copysign(q, x).to(torch.float8_e4m3fn), unit


def _plain_adamw(st):
    c = st["case"]
    eight = c["state"] == "8bit"
    g, norm = st["grad"].float(), None
    if c["clip"]:
        norm = g.square().sum(dtype=torch.float64).sqrt().float().reshape(1)
        g = g * (MAX_NORM / (norm + 1e-6)).clamp_max(1.0)
    m = _value8(*st["m8"]) if eight else st["m"]
    v = _value8(*st["r8"]).square() if eight else st["v"]
    m = B1 * m + (1.0 - B1) * g
    v = B2 * v + (1.0 - B2) * (g * g)
    denom = v.sqrt() * (1.0 / math.sqrt(1.0 - B2 ** STEP)) + EPS
    p = st["p"] * (1.0 - LR * st["decay_at"]) - (LR / (1.0 - B1 ** STEP)) * (m / denom)
    out = {"p": p, "w": p.bfloat16(), "m": m, "v": v, "norm": norm}
    if eight:
        rnd = _halves8(_philox_words(st["group8"], st["tensor8"], STEP, st["seed"]))
        out["m"] = _stochastic8(m, rnd, False)
        out["v"] = _stochastic8(v.sqrt(), rnd, True)
    return out


def _plain_moe(st):
    c = st["case"]
    t, e, h, f, k = c["t"], c["e"], c["h"], c["f"], c["k"]
    f1 = 2 * f if c["gated"] else f
    x = st["x"].float()
    logits = x @ st["router"].float().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, 1)
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    if t * k < e:                                                 # the chosen experts' weights alone
        pick, rows = ids.reshape(-1), x.repeat_interleave(k, 0)[:, None, :]
        use = w.reshape(-1, 1, 1)
    else:                                                         # every expert on every token
        pick, rows = torch.arange(e, device=x.device), x.expand(e, t, h)
        use = torch.zeros_like(logits).scatter(1, ids, w).t()[:, :, None]
    cut = lambda q, r: _dequantize(q[0].reshape(e, r, -1)[pick], q[1].reshape(e, r, -1)[pick], q[2][pick])  # noqa: E731
    z = torch.bmm(rows, cut(st["w1"], f1).transpose(1, 2))
    a = _act(z[..., :f], c["act"]) * z[..., f:] if c["gated"] else _act(z, c["act"])
    y = torch.bmm(a, cut(st["w2"], h).transpose(1, 2)) * use
    y = y.reshape(t, k, h).sum(1) if t * k < e else y.sum(0)
    return y.bfloat16()


# ---- what a pass cannot do without -----------------------------------------------------------
def _unique(t, e, k):
    """Experts that t tokens reach when each picks k of e."""
    return e * (1.0 - (1.0 - k / e) ** t)


def work(case):
    op = case["op"]
    if op == "gemm_act":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * 9 / 16 + 2 * m * n * (1 + case["residual"] + case["preact"]) + 4 * n,
                "flops": 2 * m * n * k}
    if op == "act_grad":
        mn = case["m"] * case["n"]
        return {"bytes": mn * ((4 if case["dy"] == "fp32" else 2) + 4) + 4 * case["n"], "flops": 4 * mn}
    if op == "adamw":
        n = sum(_sizes(case))
        state = 4 * (1 + 1 / 32) if case["state"] == "8bit" else 16
        return {"bytes": n * ((4 if case["grad"] == "fp32" else 2) + 8 + 2 + state), "flops": 14 * n}
    t, e, h, f, k = case["t"], case["e"], case["h"], case["f"], case["k"]
    mats = (3 if case["gated"] else 2) * h * f
    return {"bytes": _unique(t, e, k) * mats * 9 / 16 + 2 * e * h + 4 * t * h,
            "flops": 2 * t * k * mats + 2 * t * e * h}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _nvfp4_64(q):
    """Values of codes, scales and tensor scales from the bit fields of the two formats."""
    codes, scales, gs = q
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    ex, man = ((nib >> 1) & 3).double(), (nib & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2(ex - 1))
    mag = torch.where(nib > 7, -mag, mag)
    ex, man = (scales >> 3).double(), (scales & 7).double()
    sc = torch.where(ex == 0, man / 512, (1 + man / 8) * torch.exp2(ex - 7))
    rows = codes.shape[0] // gs.numel()
    return mag * sc.repeat_interleave(16, 1) * gs.double().repeat_interleave(rows)[:, None]


def _act_64(z, kind):
    if kind == "relu2":
        return torch.where(z > 0, z * z, torch.zeros_like(z))
    if kind == "gelu":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z / (1 + torch.exp(-2 * u))                        # (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
    return z * torch.sigmoid(z) if kind == "silu" else z


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op = case["op"]
    if op == "gemm_act":
        a, b = _nvfp4_64(st["a"]), _nvfp4_64(st["b"])
        z = a @ b.t()
        if st["bias"] is not None:
            z += st["bias"].double()
        d = _act_64(z, case["act"])
        if st["residual"] is not None:
            d = d + st["residual"].double()
        return {"d": d, "z": z if case["preact"] else None, "amax": None}
    if op == "act_grad":
        z = st["z"].double().requires_grad_(True)
        _act_64(z, case["act"]).backward(st["dy"].double())
        return {"dz": z.grad, "dbias": z.grad.sum(0)}
    if op == "adamw":
        return _exact_adamw(st, case)
    return _exact_moe(st, case)


def _e4m3_64(codes, scales):
    mag, sign = codes & 127, codes >> 7
    ex, man = (mag >> 3).double(), (mag & 7).double()
    v = torch.where(ex == 0, man / 512, (1 + man / 8) * torch.exp2(ex - 7)) * (1 - 2 * sign.double())
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32)


def _random_halves(st):
    """The generator's 16 bits for every element (128 for eight), from its published rounds."""
    u = np.uint64
    low, c = u(0xFFFFFFFF), [st["group8"].cpu().numpy().astype(u), None, None, st["tensor8"].cpu().numpy().astype(u)]
    c[1], c[2] = np.zeros_like(c[0]), np.full_like(c[0], STEP)
    key = [st["seed"] & 0xFFFFFFFF, st["seed"] >> 32]
    for _ in range(10):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> u(32)) ^ c[1] ^ u(key[0]), b & low, (a >> u(32)) ^ c[3] ^ u(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, 1).astype("<u4")
    return torch.from_numpy(words.view("<u2").reshape(-1).astype(np.int32)).to(DEV)


def _rounded_64(x, rnd):
    """x in units of its block's scale on the E4M3 grid, rounded up where the fraction and rnd/65536
    reach one, and the scales."""
    top = x.abs().reshape(-1, 32).amax(1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)).clamp_min(-117)
    unit = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -127)))
    y = x.abs() / unit.repeat_interleave(32)
    gap = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    return torch.floor(y / gap + rnd.double() / 65536) * gap, unit


def _exact_adamw(st, case):
    eight = case["state"] == "8bit"
    g, norm = st["grad"].double(), None
    if case["clip"]:
        norm = g.norm().reshape(1)
        g = g * min(1.0, MAX_NORM / (float(norm) + 1e-6))
    m0 = _e4m3_64(*st["m8"]) if eight else st["m"].double()
    v0 = _e4m3_64(*st["r8"]) ** 2 if eight else st["v"].double()
    m, v = m0 + (1 - B1) * (g - m0), v0 + (1 - B2) * (g * g - v0)
    p0 = st["p"].double()
    step = (m / (1 - B1 ** STEP)) / ((v / (1 - B2 ** STEP)).sqrt() + EPS)
    p = p0 - LR * (step + st["decay_at"].double() * p0)
    if eight:
        rnd = _random_halves(st)
        r = v.sqrt()
        q, q_unit = _rounded_64(r, rnd)
        v = torch.where(r > 0, q.clamp_min(1 / 512), torch.zeros_like(q)), q_unit
        q, q_unit = _rounded_64(m, rnd)
        m = torch.sign(m) * q, q_unit
    return {"p": p, "w": p, "m": m, "v": v, "norm": norm}


def _exact_moe(st, case):
    t, e, h, f, k = (case[x] for x in "tehfk")
    f1 = 2 * f if case["gated"] else f
    x = st["x"].double()
    logits = x @ st["router"].double().t()
    score = logits.sigmoid() if case["score"] == "sigmoid" else (logits - logits.amax(1, keepdim=True)).exp()
    rank = (logits[:, None, :] > logits[:, :, None]).sum(2)
    rank += ((logits[:, None, :] == logits[:, :, None]) & torch.ones(e, e, device=DEV).tril(-1).bool()).sum(2)
    weight = torch.where(rank < k, score, torch.zeros_like(score))
    weight = weight / weight.sum(1, keepdim=True)
    y = torch.zeros(t, h, dtype=torch.float64, device=DEV)
    part = lambda q, i, r: (q[0][i * r:(i + 1) * r], q[1][i * r:(i + 1) * r], q[2][i:i + 1])  # noqa: E731
    for i in range(e):
        rows = (weight[:, i] > 0).nonzero()[:, 0]
        if not rows.numel():
            continue
        z = x[rows] @ _nvfp4_64(part(st["w1"], i, f1)).t()
        a = _act_64(z[:, :f], case["act"]) * z[:, f:] if case["gated"] else _act_64(z, case["act"])
        y[rows] += weight[rows, i, None] * (a @ _nvfp4_64(part(st["w2"], i, h)).t())
    return y
