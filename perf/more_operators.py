"""Cases of the operators around the NVFP4 products in a training step: the root-mean-square norm with
the residual's addition (BF16 and 8-bit outputs) and its gradient, activation checkpoints in 8 bits and
the backward kernels that read them, tokens sorted by expert and back with the routing weights and
gradients, and the softmax cross entropy of a language model's output head without its logits, with
its gradients. Each has a plain form in elementary torch operations on FP32.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
SIGN_MASK = 0x6E04                                # random signs of the Hadamard transform
ALIGN = 64                                        # rows of an expert are padded to a multiple of this


# ---- the cases -------------------------------------------------------------------------------
def listed():
    return [
        # the norm before a layer while one token is generated: latency
        dict(name="norm one token", op="norm", m=1, n=5120, dt="bf16", residual=True, fp8=False, w="fp32"),
        # the norm before the dense layer over a whole batch; its output also in 8 bits, as the checkpoint
        # that the layer's weight gradient reads
        dict(name="norm batch, 8-bit output", op="norm", m=8192, n=5120, dt="bf16", residual=True, fp8=True, w="fp32"),
        # its backward, the residual stream's gradient added
        dict(name="norm gradient", op="norm_grad", m=8192, n=5120, dt="bf16", residual=True, w="fp32"),
        # a ragged micro-batch's activations put away in 8 bits
        dict(name="checkpoint ragged", op="save", m=1003, n=2704, dt="fp32"),
        # the weight gradient's operand (Hadamard transform along tokens, NVFP4) from the 8-bit input
        dict(name="wgrad operand from 8 bits", op="rht8", m=8192, n=5120),
        # backward of the up-projection's activation and bias from the 8-bit pre-activation
        dict(name="act_grad from 8 bits", op="act_grad8", m=8192, n=20480, act="relu2", dy="bf16"),
        # the expert layer (128 experts, top 6, hidden 2688) over a batch: routing to sorted, padded rows
        dict(name="tokens to experts", op="dispatch", t=16384, e=128, k=6, h=2688, dt="bf16", dropped=0.0),
        # back from the experts' FP32 outputs, and both gradients
        dict(name="tokens back, gradients", op="back", t=16384, e=128, k=6, h=2688, dt="fp32", dropped=0.0),
        # a few tokens on a small expert layer, some of them dropped
        dict(name="tokens to experts, few", op="dispatch", t=7, e=24, k=3, h=1040, dt="bf16", dropped=0.2),
        # the loss and gradients of the output head over a training batch
        dict(name="head training", op="head", t=8192, h=5120, v=131072, grad=True, ignored=0.1),
        # evaluation: the loss alone, a vocabulary that ends anywhere
        dict(name="head evaluation", op="head", t=1003, h=2704, v=32003, grad=False, ignored=0.0),
        # one short sequence, half of it a prompt that does not count
        dict(name="head one sequence", op="head", t=333, h=1040, v=50021, grad=True, ignored=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "save", "rht8", "act_grad8", "dispatch", "back", "head", "head"])
    if op in ("norm", "norm_grad"):
        c = dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 16, 8192), dt=rng.choice(["bf16", "fp32"]),
                 residual=rng.random() < 0.7, w=rng.choice(["bf16", "fp32"]))
        return dict(c, fp8=rng.random() < 0.5) if op == "norm" else c
    if op == "save":
        return dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 16, 20480), dt=rng.choice(["bf16", "fp32"]))
    if op == "rht8":
        return dict(op=op, m=16 * _log_int(rng, 1, 512), n=16 * _log_int(rng, 1, 640))
    if op == "act_grad8":
        return dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 16, 20480), act=rng.choice(["relu2", "gelu", "silu"]),
                    dy=rng.choice(["bf16", "fp32"]))
    if op in ("dispatch", "back"):
        e = _log_int(rng, 2, 256)
        return dict(op=op, t=_log_int(rng, 1, 8192), e=e, k=rng.randint(1, min(8, e)), h=16 * _log_int(rng, 4, 256),
                    dt=rng.choice(["bf16", "fp32"]), dropped=rng.choice([0.0, 0.0, 0.1]))
    t, h = _log_int(rng, 1, 8192), 16 * _log_int(rng, 4, 320)
    v = _log_int(rng, 100, 131072)
    return dict(op="head", t=t, h=h, v=v, grad=rng.random() < 0.6, ignored=rng.choice([0.0, 0.1, 0.5]))


# ---- inputs ----------------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std)


def _outliers(g, x, frac=1e-3, factor=50.0):
    """Activations: 0.1% of the entries 50 times larger."""
    return torch.where(torch.rand(x.shape, generator=g, device=DEV) < frac, x * factor, x)


def prepare(case, seed):
    g, op, st = _gen(seed), case["op"], {"case": dict(case)}
    if op in ("norm", "norm_grad"):
        m, n, dt = case["m"], case["n"], _DT[case["dt"]]
        st["x"] = _outliers(g, _randn(g, (m, n))).to(dt)               # a branch's output; backward: the stream itself
        # the stream that it is added to; backward: the stream's own gradient
        st["residual"] = _randn(g, (m, n), 2.0 if op == "norm" else 1e-3).to(dt) if case["residual"] else None
        st["weight"] = (1.0 + _randn(g, (n,), 0.1)).to(_DT[case["w"]])
        if op == "norm_grad":
            st["dy"] = _randn(g, (m, n), 1e-3).to(dt)
    elif op == "save":
        st["x"] = _outliers(g, _randn(g, (case["m"], case["n"]))).to(_DT[case["dt"]])
    elif op == "rht8":
        st["x8"] = _to_fp8(_outliers(g, _randn(g, (case["m"], case["n"]))))
    elif op == "act_grad8":
        m, n = case["m"], case["n"]
        st["dy"] = _randn(g, (m, n), 1e-3).to(_DT[case["dy"]])
        st["z8"] = _to_fp8(_randn(g, (m, n), 1.5))
    elif op in ("dispatch", "back"):
        _prepare_tokens(st, case, g)
    else:
        _prepare_head(st, case, g)
    if own and op == "back":
        import bit_block_scaled_quantize_amd as nv
        st["sort"] = nv.MoESort(*st["plan"], case["t"], case["k"])     # what the forward's moe_sort returned
    return st


def _prepare_tokens(st, case, g):
    t, e, k, h = case["t"], case["e"], case["k"], case["h"]
    # experts of unlike popularity, k different ones a token
    favour = -1.1 * torch.log(1.0 + torch.arange(e, device=DEV))[torch.randperm(e, generator=g, device=DEV)]
    noise = -torch.log(-torch.log(torch.rand((t, e), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)))
    top = torch.topk(favour + noise, k, dim=1)
    ids = top.indices.int()
    if case["dropped"]:                                                # over an expert's capacity: no expert
        ids = torch.where(torch.rand((t, k), generator=g, device=DEV) < case["dropped"], -1, ids).int()
    st["ids"] = ids.contiguous()
    st["weights"] = torch.softmax(top.values.float(), 1).contiguous()
    if case["op"] == "dispatch":
        st["x"] = _outliers(g, _randn(g, (t, h))).to(_DT[case["dt"]])
    else:
        st["plan"] = _plain_sort(st["ids"], e)
        rows = st["plan"][2].numel()
        # the experts' outputs, and the gradients of the sorted inputs
        st["y"] = _randn(g, (rows, h)).to(_DT[case["dt"]])
        st["dxs"] = _randn(g, (rows, h), 1e-3).bfloat16()
        st["dout"] = _randn(g, (t, h), 1e-3).bfloat16()


def _prepare_head(st, case, g):
    t, h, v = case["t"], case["h"], case["v"]
    w = _randn(g, (v, h), 1.5 * h ** -0.5).bfloat16()
    targets = torch.randint(0, v, (t,), generator=g, device=DEV)
    # normed hidden states that lean towards their target, some more than others
    lean = torch.rand((t, 1), generator=g, device=DEV) * 6.0 / 1.5
    x = _randn(g, (t, h)) + lean * w[targets].float()
    st["x"], st["w"] = x.bfloat16(), w
    skip = torch.rand((t,), generator=g, device=DEV) < case["ignored"]
    st["targets"] = torch.where(skip, -100, targets)
    if case["grad"]:
        # the mean over the tokens that count, each with a weight of its own
        st["grad"] = (0.5 + torch.rand((t,), generator=g, device=DEV)) / max(1, t)


# ---- one pass --------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


# the framework's calls
def _own_norm(st):
    import bit_block_scaled_quantize_amd as nv
    x, c = st["x"], st["case"]
    amax = torch.empty((1,), device=DEV)
    h = torch.empty_like(x) if c["residual"] else None
    q = nv.FP8Tensor.empty(c["m"], c["n"], device=DEV) if c["fp8"] else None
    y = nv.rms_norm(x, st["weight"], residual=st["residual"], eps=EPS, residual_out=h, fp8_out=q, amax_out=amax)
    return {"y": y, "h": h, "y8": _views(q) if c["fp8"] else None, "amax": amax.view(torch.bfloat16)[1:]}


def _own_norm_grad(st):
    import bit_block_scaled_quantize_amd as nv
    dw = torch.empty((st["x"].shape[1],), device=DEV)
    dx = nv.rms_norm_grad(st["dy"], st["x"], st["weight"], dresidual=st["residual"], eps=EPS, dweight=dw)
    return {"dx": dx, "dw": dw}


def _own_save(st):
    import bit_block_scaled_quantize_amd as nv
    return _views(nv.fp8_quantize(st["x"]))


def _fp8(nv, q):
    codes, scales = q
    return nv.FP8Tensor(codes, scales, *codes.shape)


def _views(q):
    """The values that codes and scales hold."""
    return q.codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)


def _own_rht8(st):
    import bit_block_scaled_quantize_amd as nv
    q = nv.rht_quantize(_fp8(nv, st["x8"]), SIGN_MASK, "rn")
    return {"values": _e2m1_values(q.codes), "scales": q.scales.view(torch.float8_e4m3fn), "global": q.global_scale}


def _own_act_grad8(st):
    import bit_block_scaled_quantize_amd as nv
    db = torch.empty((st["dy"].shape[1],), device=DEV)
    dz = nv.act_grad(st["dy"], _fp8(nv, st["z8"]), activation=st["case"]["act"], dbias=db)
    return {"dz": dz, "dbias": db}


def _own_dispatch(st):
    import bit_block_scaled_quantize_amd as nv
    sort = nv.moe_sort(st["ids"], st["case"]["e"], align=ALIGN)
    return {"x": nv.moe_gather(st["x"], sort), "offsets": sort.offsets, "row_of": sort.row_of, "pair_of": sort.pair_of}


def _own_back(st):
    import bit_block_scaled_quantize_amd as nv
    s = st["sort"]
    out = nv.moe_combine(st["y"], s, st["weights"])
    dy, dw = nv.moe_combine_grad(st["dout"], st["y"], s, st["weights"])
    return {"out": out, "dy": dy, "dw": dw, "dx": nv.moe_combine(st["dxs"], s)}


def _own_head(st):
    import bit_block_scaled_quantize_amd as nv
    loss, lse = nv.linear_cross_entropy(st["x"], st["w"], st["targets"])
    if not st["case"]["grad"]:
        return {"loss": loss, "lse": lse}
    dx, dw = nv.linear_cross_entropy_grad(st["x"], st["w"], st["targets"], lse, st["grad"])
    return {"loss": loss, "dx": dx, "dw": dw}


# the plain forms
def _pow2(e):
    """2^e in FP32 from its bit field (0 for e = -127, the scale of an all-zero block)."""
    return ((e + 127).int() << 23).view(torch.float32)


def _to_fp8(x):
    """E4M3 codes and an E8M0 scale 2^e per 32 elements of a row: the smallest e >= -117 with
    max|x| <= 448 * 2^e."""
    m, n = x.shape
    blocks = torch.nn.functional.pad(x.float(), (0, -n % 32)).reshape(m, -1, 32)
    top = blocks.abs().amax(2)
    frac, ex = torch.frexp(top)                                       # top = frac * 2^ex, frac in [0.5, 1)
    e = torch.where(frac > 0.875, ex - 8, ex - 9)
    e = torch.where(top > 0, e.clamp_min(-117), torch.full_like(e, -127))
    codes = (blocks * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(m, -1)[:, :n].contiguous(), (e + 127).to(torch.uint8)


def _from_fp8(q):
    codes, scales = q
    v = codes.view(torch.float8_e4m3fn).float()
    return v * _pow2(scales.int() - 127).repeat_interleave(32, 1)[:, :codes.shape[1]]


def _f8(q):
    return q[0].view(torch.float8_e4m3fn), q[1].view(torch.float8_e8m0fnu)


def _plain_norm(st):
    x, r = st["x"], st["residual"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hf = h.float()
    y = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS) * st["weight"].float()
    yb = y.bfloat16()
    return {"y": yb, "h": None if r is None else h, "y8": _f8(_to_fp8(y)) if st["case"]["fp8"] else None,
            "amax": yb.abs().amax().reshape(1)}


def _plain_norm_grad(st):
    h, g, w = st["x"].float(), st["dy"].float(), st["weight"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    u = g * w
    dx = r * (u - h * (r * r) * (u * h).mean(1, keepdim=True))
    if st["residual"] is not None:
        dx = dx + st["residual"].float()
    return {"dx": dx.to(st["x"].dtype), "dw": (g * h * r).sum(0)}


def _plain_save(st):
    return _f8(_to_fp8(st["x"]))


def _hadamard16():
    i = torch.arange(16, device=DEV)
    bits = i[:, None] & i[None, :]
    odd = (bits ^ (bits >> 1) ^ (bits >> 2) ^ (bits >> 3)) & 1
    sign = 1 - 2 * ((SIGN_MASK >> i) & 1)
    return ((1 - 2 * odd) * sign[None, :]).double()


_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e2m1_values(codes):
    """Packed E2M1 codes [r, c/2] as the values [r, c] that they stand for (exact in E4M3)."""
    lut = torch.tensor(_GRID + [-x for x in _GRID], device=codes.device).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).reshape(codes.shape[0], -1).view(torch.float8_e4m3fn)


def _plain_rht8(st):
    x = _from_fp8(st["x8"]).double()
    t, c = x.shape
    y = 0.25 * (_hadamard16() @ x.reshape(t // 16, 16, c).permute(1, 0, 2).reshape(16, -1))
    y = y.reshape(16, t // 16, c).permute(2, 1, 0).float()            # [column, block of tokens, 16]
    amax = y.abs().amax()
    s_enc = torch.where(amax > 0, 2688.0 / amax, torch.ones_like(amax)).clamp_max(3.4028234663852886e38)
    scales = ((y.abs().amax(2) / 6.0) * s_enc).clamp_max(448.0).to(torch.float8_e4m3fn)
    dec = scales.float()
    r = torch.where(dec > 0, (s_enc / dec).clamp_max(3.4028234663852886e38), torch.zeros_like(dec))
    v = y * r[:, :, None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_max(6.0)                 # to nearest, ties to even, in each binade
    return {"values": torch.copysign(q, v).reshape(c, t).to(torch.float8_e4m3fn), "scales": scales,
            "global": torch.where(amax > 0, amax / 2688.0, torch.ones_like(amax)).reshape(1)}


def _act_slope(z, kind):
    if kind == "relu2":
        return 2.0 * z.clamp_min(0.0)
    if kind == "gelu":
        th = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * 0.7978845608028654 * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_act_grad8(st):
    dz = st["dy"].float() * _act_slope(_from_fp8(st["z8"]), st["case"]["act"])
    return {"dz": dz.bfloat16(), "dbias": dz.sum(0)}


def _sorted_rows(t, k, e):
    """Rows that hold t * k pairs of e experts, each expert padded to a multiple of ALIGN."""
    return (t * k + min(e, t * k) * (ALIGN - 1)) // ALIGN * ALIGN


def _plain_sort(ids, e):
    """offsets [e+1] of the experts' padded runs, the row of each pair (-1: dropped), the pair of each row (-1: none)."""
    t, k = ids.shape
    rows = _sorted_rows(t, k, e)
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= e), e, flat)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    first = count.cumsum(0) - count                                   # in the order, without padding
    padded = (count[:e] + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), padded.cumsum(0)])
    kept = key[order]
    row = torch.arange(t * k, device=ids.device) - first[kept] + offsets[kept.clamp_max(e - 1)]
    row = torch.where(kept < e, row, -1).int()
    row_of = torch.empty(t * k, dtype=torch.int32, device=ids.device).scatter_(0, order, row)
    spare = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    spare.scatter_(0, torch.where(row >= 0, row, rows).long(), order.int())
    return offsets, row_of.reshape(t, k), spare[:rows].clone()


def _plain_dispatch(st):
    c = st["case"]
    offsets, row_of, pair_of = _plain_sort(st["ids"], c["e"])
    token = pair_of.clamp_min(0).long() // c["k"]
    x = torch.where(pair_of[:, None] >= 0, st["x"][token], torch.zeros((), dtype=st["x"].dtype, device=DEV))
    return {"x": x, "offsets": offsets, "row_of": row_of, "pair_of": pair_of}


def _plain_back(st):
    _, row_of, pair_of = st["plan"]
    k = row_of.shape[1]
    w = torch.where(row_of >= 0, st["weights"], torch.zeros_like(st["weights"]))
    at = row_of.clamp_min(0).long()
    have = (row_of >= 0).float()
    y = st["y"].float()
    out = (y[at] * w[:, :, None]).sum(1)
    dout = st["dout"].float()
    dw = (y[at] * dout[:, None, :]).sum(2) * have
    wr = torch.where(pair_of >= 0, w.reshape(-1)[pair_of.clamp_min(0).long()], torch.zeros((), device=DEV))
    dy = dout[pair_of.clamp_min(0).long() // k] * wr[:, None]
    dx = (st["dxs"].float()[at] * have[:, :, None]).sum(1)
    return {"out": out.bfloat16(), "dy": dy.bfloat16(), "dw": dw, "dx": dx.bfloat16()}


def _plain_head(st):
    x, w, tg = st["x"].float(), st["w"].float(), st["targets"]
    logits = x @ w.t()
    counts = (tg >= 0) & (tg < w.shape[0])
    at = torch.where(counts, tg, 0)
    top = logits.amax(1, keepdim=True)
    lse = top + torch.exp(logits - top).sum(1, keepdim=True).log()
    loss = torch.where(counts, (lse - logits.gather(1, at[:, None]))[:, 0], torch.zeros_like(lse[:, 0]))
    if not st["case"]["grad"]:
        return {"loss": loss, "lse": lse[:, 0]}
    g = torch.where(counts, st["grad"], torch.zeros_like(st["grad"]))
    p = torch.exp(logits.sub_(lse)).mul_(g[:, None])
    p.scatter_add_(1, at[:, None], -g[:, None])
    return {"loss": loss, "dx": (p @ w).bfloat16(), "dw": (p.t() @ x).bfloat16()}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "save": _plain_save, "rht8": _plain_rht8,
          "act_grad8": _plain_act_grad8, "dispatch": _plain_dispatch, "back": _plain_back, "head": _plain_head}
_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "save": _own_save, "rht8": _own_rht8,
        "act_grad8": _own_act_grad8, "dispatch": _own_dispatch, "back": _own_back, "head": _own_head}


# ---- what a pass cannot do without -----------------------------------------------------------
def _size(dt):
    return 4 if dt == "fp32" else 2


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad", "save", "rht8", "act_grad8"):
        mn = case["m"] * case["n"]
    if op == "norm":
        s = _size(case["dt"])
        return {"bytes": mn * (s + 2 + 2 * s * case["residual"] + 33 / 32 * case["fp8"]) + 4 * case["n"], "flops": 6 * mn}
    if op == "norm_grad":
        return {"bytes": mn * _size(case["dt"]) * (3 + case["residual"]) + 8 * case["n"], "flops": 12 * mn}
    if op == "save":
        return {"bytes": mn * (_size(case["dt"]) + 33 / 32), "flops": 3 * mn}
    if op == "rht8":
        return {"bytes": mn * (33 / 32 + 9 / 16), "flops": 8 * mn}
    if op == "act_grad8":
        return {"bytes": mn * (_size(case["dy"]) + 33 / 32 + 2) + 4 * case["n"], "flops": 4 * mn}
    if op in ("dispatch", "back"):
        t, k, h, s = case["t"], case["k"], case["h"], _size(case["dt"])
        rows, pairs = _sorted_rows(t, k, case["e"]), t * k * (1 - case["dropped"])
        if op == "dispatch":
            return {"bytes": s * h * (t + rows) + 8 * t * k + 4 * rows, "flops": t * k}
        # the experts' outputs once, both gradients of a pair, the tokens' sums and the gradient they come from
        return {"bytes": h * (pairs * (s + 2) + 2 * rows + 6 * t) + 20 * t * k, "flops": 6 * pairs * h}
    t, h, v = case["t"], case["h"], case["v"]
    if not case["grad"]:
        return {"bytes": 2 * h * (t + v) + 16 * t, "flops": 2 * t * h * v}
    # the loss's product, and the backward's three: the logits are not kept
    return {"bytes": 2 * 2 * h * (t + v) + 24 * t, "flops": 8 * t * h * v}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _e4m3_64(codes):
    mag, sign = codes & 127, codes >> 7
    ex, man = (mag >> 3).double(), (mag & 7).double()
    v = torch.where(ex == 0, man / 512, (1 + man / 8) * torch.exp2(ex - 7))
    return v * (1 - 2 * sign.double())


def _fp8_64(q):
    codes, scales = q
    return _e4m3_64(codes) * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :codes.shape[1]]


def _round_fp8_64(x):
    """The nearest E4M3 values of x over its block's power of two, and that power."""
    m, n = x.shape
    pad = torch.zeros((m, (n + 31) // 32 * 32), dtype=torch.float64, device=x.device)
    pad[:, :n] = x
    top = pad.abs().reshape(m, -1, 32).amax(2)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)).clamp_min(-117)
    unit = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -127)))
    y = pad / unit.repeat_interleave(32, 1)
    gap = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(y / gap) * gap)[:, :n], unit


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    return _EXACT[case["op"]](st, case)


def _exact_norm(st, case):
    x, r = st["x"].double(), st["residual"]
    h = x if r is None else x + r.double()
    # the norm is taken of the stream as it is stored
    hs = h if r is None else (st["x"].float() + r.float()).to(st["x"].dtype).double()
    y = hs / torch.sqrt((hs * hs).sum(1, keepdim=True) / case["n"] + EPS) * st["weight"].double()
    return {"y": y, "h": None if r is None else h, "y8": _round_fp8_64(y) if case["fp8"] else None, "amax": None}


def _exact_norm_grad(st, case):
    h = st["x"].double().requires_grad_(True)
    w = st["weight"].double().requires_grad_(True)
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["n"] + EPS) * w
    y.backward(st["dy"].double())
    dx = h.grad if st["residual"] is None else h.grad + st["residual"].double()
    return {"dx": dx, "dw": w.grad}


def _exact_save(st, case):
    return _round_fp8_64(st["x"].double())


def _exact_rht8(st, case):
    x = _fp8_64(st["x8"])
    t, c = x.shape
    u = x.reshape(t // 16, 16, c)
    sign = torch.tensor([-1.0 if (SIGN_MASK >> j) & 1 else 1.0 for j in range(16)], dtype=torch.float64, device=DEV)
    u = u * sign[None, :, None]
    for h in (1, 2, 4, 8):                                            # the butterfly, one bit of the index at a time
        u = u.reshape(t // 16, 16 // (2 * h), 2, h, c)
        u = torch.stack([u[:, :, 0] + u[:, :, 1], u[:, :, 0] - u[:, :, 1]], 2).reshape(t // 16, 16, c)
    y = (u / 4).permute(2, 0, 1).contiguous().float()                 # the format is defined on FP32 values
    amax = y.abs().max()
    if not float(amax):
        return None
    s_enc = torch.tensor(2688.0, device=DEV) / amax
    ts = (y.abs().amax(2) / 6) * s_enc
    gap = torch.exp2(torch.floor(torch.log2(ts.double().clamp_min(2.0 ** -6))) - 3)
    scale = (torch.round(ts.double() / gap) * gap).clamp_max(448)
    r = torch.where(scale > 0, (s_enc / scale.float()), torch.zeros_like(ts))
    v = (y * r[:, :, None]).double()
    grid = torch.tensor(_GRID, dtype=torch.float64, device=DEV)
    mids = (grid[1:] + grid[:-1]) / 2
    a = v.abs()
    # a value on a border goes to the neighbour whose index is even
    low, high = torch.bucketize(a, mids), torch.bucketize(a, mids, right=True)
    at = torch.where((low != high) & (low % 2 == 1), high, low)
    return {"values": torch.sign(v).reshape(c, t) * grid[at].reshape(c, t), "scales": scale, "global": amax.double().reshape(1) / 2688}


def _exact_act_grad8(st, case):
    z = _fp8_64(st["z8"]).requires_grad_(True)
    if case["act"] == "relu2":
        a = torch.where(z > 0, z * z, torch.zeros_like(z))
    elif case["act"] == "gelu":
        a = z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    else:
        a = z * torch.sigmoid(z)
    a.backward(st["dy"].double())
    return {"dz": z.grad, "dbias": z.grad.sum(0)}


def _exact_dispatch(st, case):
    return {"x": _plain_dispatch(st)["x"].double(), "offsets": None, "row_of": None, "pair_of": None}


def _exact_back(st, case):
    t, k, h = case["t"], case["k"], case["h"]
    _, row_of, _ = st["plan"]
    rows, y, dout = st["y"].shape[0], st["y"].double(), st["dout"].double()
    out, dx = torch.zeros((t, h), dtype=torch.float64, device=DEV), torch.zeros((t, h), dtype=torch.float64, device=DEV)
    dy, dw = torch.zeros((rows, h), dtype=torch.float64, device=DEV), torch.zeros((t, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        tok = (row_of[:, j] >= 0).nonzero()[:, 0]
        r, w = row_of[tok, j].long(), st["weights"][tok, j].double()[:, None]
        out[tok] += w * y[r]
        dx[tok] += st["dxs"][r].double()
        dy[r] = w * dout[tok]
        dw[tok, j] = (dout[tok] * y[r]).sum(1)
    return {"out": out, "dy": dy, "dw": dw, "dx": dx}


def _exact_head(st, case):
    t, v = case["t"], case["v"]
    x, w, tg = st["x"].double(), st["w"].double(), st["targets"]
    live = (tg >= 0).nonzero()[:, 0]
    logits = x @ w.t()
    lse = torch.logsumexp(logits, 1)
    loss = torch.zeros(t, dtype=torch.float64, device=DEV)
    loss[live] = lse[live] - logits[live, tg[live]]
    if not case["grad"]:
        return {"loss": loss, "lse": lse}
    p = torch.softmax(logits, 1)
    p[live, tg[live]] -= 1
    p *= torch.where(tg >= 0, st["grad"].double(), torch.zeros(t, dtype=torch.float64, device=DEV))[:, None]
    return {"loss": loss, "dx": p @ w, "dw": p.t() @ x}


_EXACT = {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "save": _exact_save, "rht8": _exact_rht8,
          "act_grad8": _exact_act_grad8, "dispatch": _exact_dispatch, "back": _exact_back, "head": _exact_head}
