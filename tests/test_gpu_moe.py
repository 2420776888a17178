"""nvfp4_moe_tokens on the GPU.

Routing: a logit's FP32 sum of H products is within d = (H / 64 + 8) u sum |x||r| of the 64-bit one
(64 lanes of H / 64 terms, six additions across them); every pick has to lie above every expert left
out up to 2 d, the picks in descending order up to 2 d. Weights, relative: 4 d for the two
exponentials' arguments, (2 |l| + 8) u each for evaluating them, E u for the softmax's sum. y for the
routing that the call reports: oracle.moe64's tolerance."""
import numpy as np
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
import oracle
import workloads
from bit_block_scaled_quantize_amd.moe import MoETokens
from helpers import host, log, to_device_bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _host(t):
    return t.detach().float().cpu().numpy()


def _bf16(shape, seed, std=1.0, outliers=False):
    n = int(np.prod(shape[:-1]))
    bits = (workloads.with_outliers_bf16((n, shape[-1]), seed) if outliers
            else workloads.normal_bf16((n, shape[-1]), seed, std=std))
    return to_device_bf16(bits).reshape(shape)


class Layer:
    def __init__(self, e, h, f, k, seed, router_dtype=torch.bfloat16, **kw):
        self.gated = kw.get("gated", False)
        self.act = kw.get("activation", "relu2")
        f1 = 2 * f if self.gated else f
        self.router = _bf16((e, h), seed, h ** -0.5).to(router_dtype)
        w1, w2 = _bf16((e, f1, h), seed + 1, h ** -0.5), _bf16((e, h, f), seed + 2, f ** -0.5)
        # experts of different magnitude: each has a tensor scale of its own
        w1 = (w1.float() * (0.5 + torch.arange(e, device="cuda")[:, None, None] / e)).bfloat16()
        self.gpu = MoETokens.from_bf16(self.router, w1, w2, k, **kw)
        self.e, self.h, self.f, self.f1, self.k = e, h, f, f1, k
        self.kw = kw

    def weights64(self):
        out = []
        for q, rows in ((self.gpu.weights.w1, self.f1), (self.gpu.weights.w2, self.h)):
            c, s, g = host(q)
            out.append(np.stack([oracle.dequantize(c[i * rows:(i + 1) * rows], s[i * rows:(i + 1) * rows], g[i:i + 1])
                                 for i in range(self.e)]))
        return out

    def run(self, x, **kw):
        t = x.shape[0]
        ids = torch.full((t, self.k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((t, self.k), -1.0, device="cuda")
        y = self.gpu(x, ids_out=ids, weights_out=w, **kw)
        torch.cuda.synchronize()
        return y, ids.cpu().numpy(), w.cpu().numpy()

    def check_routing(self, x, ids, w):
        xh, r = _host(x).astype(np.float64), _host(self.router).astype(np.float64)
        l = xh @ r.T
        d = (self.h / 64 + 8) * U * (np.abs(xh) @ np.abs(r).T)
        sig = self.kw.get("score", "softmax") == "sigmoid"
        for t in range(x.shape[0]):
            pick = ids[t]
            assert len(set(pick)) == self.k and pick.min() >= 0 and pick.max() < self.e
            rest = np.setdiff1d(np.arange(self.e), pick)
            dt = d[t].max()
            if rest.size:
                assert l[t, pick].min() >= l[t, rest].max() - 2 * dt, f"token {t}"
            assert np.all(np.diff(l[t, pick]) <= 2 * dt)
            s = 1 / (1 + np.exp(-l[t])) if sig else np.exp(l[t] - l[t].max()) / np.exp(l[t] - l[t].max()).sum()
            want = s[pick]
            if self.kw.get("renormalize", True):
                want = want / (want.sum() + 1e-20)
            want = want * self.kw.get("routed_scale", 1.0)
            rel = 4 * dt + (4 * np.abs(l[t]).max() + 16 + self.e + self.k) * U
            assert np.all(np.abs(w[t] - want) <= rel * np.abs(want)), f"weights of token {t}"

    def check(self, x, what):
        y, ids, w = self.run(x)
        self.check_routing(x, ids, w)
        w1, w2 = self.weights64()
        want, tol = oracle.moe64(_host(x), ids, w, w1, w2, self.act, self.gated)
        err = np.abs(_host(y) - want)
        assert np.all(err <= tol), f"{what}: {(err > tol).sum()} of {err.size}, first {np.argwhere(err > tol)[0]}"
        assert np.abs(want).max() > 0
        return y


CASES = [
    dict(t=1, e=8, h=256, f=128, k=2),
    dict(t=1, e=1, h=16, f=16, k=1),
    dict(t=3, e=5, h=272, f=80, k=5, activation="gelu", score="sigmoid"),
    dict(t=7, e=24, h=1040, f=720, k=3, activation="silu", gated=True),
    dict(t=8, e=130, h=64, f=48, k=16, activation="silu", gated=True, score="sigmoid", routed_scale=2.5),
    dict(t=9, e=16, h=128, f=1856, k=6, renormalize=False),
    dict(t=16, e=4, h=320, f=96, k=1, activation="none"),
    dict(t=17, e=3, h=336, f=112, k=2, activation="gelu", gated=True, renormalize=False, score="sigmoid"),
    dict(t=33, e=512, h=96, f=64, k=4),
    dict(t=64, e=2, h=192, f=208, k=1, activation="silu"),
    dict(t=64, e=12, h=2688, f=208, k=6, score="sigmoid"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
@pytest.mark.parametrize("router", [torch.bfloat16, torch.float32], ids=["r16", "r32"])
def test_layer(case, router):
    c = dict(case)
    t = c.pop("t")
    log(f"moe {case}")
    layer = Layer(c.pop("e"), c.pop("h"), c.pop("f"), c.pop("k"), 500 + t, router, **c)
    layer.check(_bf16((t, layer.h), 600 + t, outliers=True), str(case))


def test_one_expert_takes_all():
    """Every token of a full batch on the same two experts: four column blocks of one expert."""
    log("moe hot expert")
    for t in (16, 64):
        layer = Layer(6, 128, 96, 2, 700)
        layer.router[:] = 0
        layer.router[4] = 1.0
        layer.router[1] = 0.5
        x = _bf16((t, 128), 701).abs() + 0.5                        # positive sums: experts 4, then 1
        y = layer.check(x, "hot")
        assert np.array_equal(layer.run(x)[1], np.tile([4, 1], (t, 1)))
        assert y.shape == (t, 128)


def test_ties_go_to_the_lowest_expert():
    log("moe ties")
    layer = Layer(200, 64, 32, 7, 720)
    layer.router[:] = layer.router[:1].clone()
    layer.router[150] = 0
    x = _bf16((5, 64), 721)
    x[3] = 0                                                          # every logit 0
    _, ids, w = layer.run(x)
    up = (_host(x) @ _host(layer.router[0])) > 0                       # expert 150's logit is 0
    for t in range(5):
        if t == 3 or up[t]:
            assert list(ids[t]) == list(range(7))
        else:
            assert list(ids[t]) == [150] + list(range(6))
        if t == 3:
            assert np.allclose(w[t], 1 / 7, rtol=1e-6)


def test_a_token_does_not_know_the_others():
    """Bit for bit the same alone, in a batch of 16 and in one of 64, next to non-finite tokens too."""
    log("moe batch")
    for kw in (dict(), dict(gated=True, activation="silu", score="sigmoid")):
        layer = Layer(10, 256, 144, 3, 740, **kw)
        x = _bf16((64, 256), 741, outliers=True)
        y = layer.run(x)[0]
        for i in (0, 5, 63):
            assert torch.equal(layer.run(x[i:i + 1])[0][0], y[i])
        assert torch.equal(layer.run(x[16:32])[0], y[16:32])
        bad = x.clone()
        bad[2, 7] = float("nan")
        bad[9, 100] = float("inf")
        bad[40] = float("-inf")
        z, ids, _ = layer.run(bad)
        keep = [i for i in range(64) if i not in (2, 9, 40)]
        assert torch.equal(z[keep], y[keep])
        assert ids.min() >= 0 and ids.max() < 10
        assert not torch.isfinite(z[[2, 40]]).any()


def test_wide_ranges():
    """Tokens of very different magnitude in one batch, and within a token."""
    log("moe ranges")
    layer = Layer(4, 128, 64, 2, 760, activation="silu")
    x = _bf16((6, 128), 761)
    x = (x.float() * torch.tensor([1e-30, 1e-8, 1.0, 1e4, 1e12, 0.0], device="cuda")[:, None]).bfloat16()
    layer.check(x, "ranges")
    assert torch.count_nonzero(layer.run(x)[0][5]).item() == 0


@pytest.mark.parametrize("t", [2, 20])
def test_strides_and_alignment(t):
    log(f"moe strides {t}")
    layer = Layer(8, 272, 80, 3, 780)
    x = _bf16((t, 272), 781)
    want = layer.run(x)[0]
    for pad, off in ((8, 8), (3, 1)):
        wide = torch.zeros((t, 272 + pad + off), dtype=torch.bfloat16, device="cuda")
        wide[:, off:off + 272] = x
        out = torch.zeros_like(wide)
        got = layer.run(wide[:, off:off + 272], out=out[:, off:off + 272])[0]
        assert torch.equal(got, want)
        out[:, off:off + 272] = 0
        assert torch.count_nonzero(out).item() == 0


def test_streams_and_graph():
    log("moe graph")
    for t in (1, 40):
        layer = Layer(16, 256, 128, 4, 790)
        xs = [_bf16((t, 256), 791 + i) for i in range(3)]
        want = [layer.run(x)[0].clone() for x in xs]
        s = torch.cuda.Stream()
        assert torch.equal(layer.run(xs[0], stream=s)[0], want[0])
        x, out = xs[0].clone(), torch.zeros_like(want[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.gpu(x, out=out)
        for i in (0, 1, 2, 1):
            x.copy_(xs[i])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i])
            assert torch.equal(layer.run(xs[2])[0], want[2])          # eager calls between the replays
        zero = nv.library().nvfp4_moe_workspace_size(layer.gpu.weights.c(), 0)
        assert torch.count_nonzero(layer.gpu.workspace[:zero]).item() == 0


def test_refusals():
    layer = Layer(8, 64, 32, 2, 800)
    w = layer.gpu.weights
    x = _bf16((4, 64), 801)
    for bad in (x.float(), x[:, :48], x.cpu(), x.t(), _bf16((65, 64), 2), x[:1].expand(4, 64)):
        with pytest.raises(nv.NVFP4Error):
            layer.gpu(bad)
    with pytest.raises(nv.NVFP4Error):
        layer.gpu(x, out=torch.zeros((4, 48), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(nv.NVFP4Error):
        layer.gpu(x, ids_out=torch.zeros((4, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(nv.NVFP4Error, match="64"):
        nv.moe_tokens(_bf16((65, 64), 2), w, workspace=layer.gpu.workspace)
    with pytest.raises(nv.NVFP4Error, match="workspace"):
        nv.moe_tokens(x, w, workspace=layer.gpu.workspace[:512])
    for kw in (dict(top_k=9), dict(top_k=0), dict(score="max"), dict(activation="tanh"), dict(gated=True),
               dict(routed_scale=float("nan"))):
        with pytest.raises(nv.NVFP4Error):
            nv.moe_tokens(x, nv.MoEWeights(**{**w.__dict__, **kw}), workspace=layer.gpu.workspace)
    assert layer.gpu(x[:0]).shape == (0, 64)
