"""Host-side refusals of the layer operators' C entries (no GPU: every call fails its checks before
anything is enqueued, or touches host memory alone)."""
import ctypes
import os

import pytest

import bit_block_scaled_quantize_amd as nv

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        pytest.skip("libnvfp4.so not built")
    return nv.library()


def _entry(n=100, **kw):
    f = {k: FAKE for k in ("grad", "p", "p_out", "w_out", "m", "v", "m_out", "v_out", "m_scale", "v_scale",
                           "m_scale_out", "v_scale_out")}
    f.update(kw)
    return nv._CAdamWTensor(n=n, grad_dt=f.pop("grad_dt", 1), weight_decay=0.0, **f)


def _table(lib, entries, state=0, bytes_=None, null=False):
    arr = (nv._CAdamWTensor * len(entries))(*entries)
    size = lib.nvfp4_adamw_table_size(arr, len(entries))
    buf = ctypes.create_string_buffer(max(size, 64))
    chunks = ctypes.c_int64(-1)
    st = lib.nvfp4_adamw_table(arr, len(entries), state, None if null else buf, size if bytes_ is None else bytes_,
                               ctypes.byref(chunks))
    return st, chunks.value, size


def test_adamw_table(lib):
    st, chunks, _ = _table(lib, [_entry(1), _entry(8192), _entry(8193), _entry(0, grad=None, p=None)])
    assert (st, chunks) == (0, 1 + 4 + 5)                             # of 2048 elements
    assert _table(lib, [_entry()], null=True)[0] == INVALID
    assert _table(lib, [_entry()], state=2)[0] == INVALID
    assert _table(lib, [_entry(n=-1)])[0] == INVALID
    assert _table(lib, [_entry(grad_dt=5)])[0] == INVALID
    assert _table(lib, [_entry(p=None)])[0] == INVALID
    assert _table(lib, [_entry(p=FAKE + 2)])[0] == INVALID
    assert _table(lib, [_entry(grad=FAKE + 2)])[0] == INVALID
    assert _table(lib, [_entry(grad=FAKE + 2, grad_dt=0)])[0] == 0
    assert _table(lib, [_entry(m=FAKE + 1)])[0] == INVALID
    assert _table(lib, [_entry(m=FAKE + 1)], state=1)[0] == 0
    assert _table(lib, [_entry(m_scale=None)], state=1)[0] == INVALID
    assert _table(lib, [_entry(m_scale=None)], state=0)[0] == 0
    assert _table(lib, [_entry()], bytes_=8)[0] == INVALID
    assert _table(lib, [_entry(n=1 << 50)])[0] == UNSUPPORTED
    assert lib.nvfp4_adamw_table_size(None, 1) == 0


def test_adamw_validation(lib):
    def call(table=FAKE, count=1, chunks=1, state=0, ws=FAKE, ws_n=8192, norm=None, **hp):
        h = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, max_norm=1.0, seed=0)
        h.update(hp)
        return lib.nvfp4_adamw(table, count, chunks, state, ctypes.byref(nv._CAdamWHyper(**h)), norm, None, ws, ws_n, None)

    assert lib.nvfp4_workspace_size(nv.OP_ADAMW, 0, 0, 0) == 8192
    assert call(table=None) == INVALID
    assert call(table=FAKE + 8) == INVALID
    assert call(count=0) == INVALID
    assert call(chunks=-1) == INVALID
    assert call(state=3) == INVALID
    for hp in (dict(lr=float("inf")), dict(beta1=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-60),
               dict(step=0), dict(max_norm=-1.0), dict(max_norm=float("nan"))):
        assert call(**hp) == INVALID, hp
    assert call(max_norm=0.0, norm=FAKE) == INVALID
    assert call(ws=None) == WORKSPACE
    assert call(ws_n=100) == WORKSPACE
    assert lib.nvfp4_adamw(FAKE, 1, 1, 0, None, None, None, None, 0, None) == INVALID


def _t(rows, cols):
    return ctypes.byref(nv._CTensor(FAKE, FAKE, FAKE, rows, cols))


def test_gemm_act_validation(lib):
    def call(A=_t(64, 128), B=_t(32, 128), D=FAKE, ldd=32, bias=None, bdt=0, act=0, res=None, ldr=0, pre=None, ldp=0,
             amax=None, ws=None, ws_n=0):
        return lib.nvfp4_gemm_act(A, B, D, ldd, bias, bdt, act, res, ldr, pre, ldp, amax, ws, ws_n, None)

    assert call(A=None) == INVALID
    assert call(B=_t(32, 96)) == INVALID
    assert call(A=_t(64, 100), B=_t(32, 100)) == INVALID
    assert call(D=None) == INVALID
    assert call(D=FAKE + 1) == INVALID
    assert call(ldd=31) == INVALID
    assert call(act=4) == INVALID
    assert call(act=-1) == INVALID
    assert call(bias=FAKE, bdt=2) == INVALID
    assert call(bias=FAKE + 2, bdt=1) == INVALID
    assert call(res=FAKE, ldr=31) == INVALID
    assert call(res=FAKE + 1, ldr=32) == INVALID
    assert call(pre=FAKE, ldp=31) == INVALID
    assert call(amax=FAKE + 2) == INVALID
    need = lib.nvfp4_workspace_size(nv.OP_GEMM_ACT, 8192, 5120, 128)
    assert need > 0
    big = dict(A=_t(8192, 128), B=_t(5120, 128), ldd=5120)
    assert call(**big) == WORKSPACE
    assert call(**big, ws=FAKE, ws_n=need - 1) == WORKSPACE
    assert call(**big, ws=FAKE + 16, ws_n=need) == WORKSPACE
    assert call(A=_t(1 << 20, 8192), B=_t(32, 8192)) == UNSUPPORTED


def test_act_grad_validation(lib):
    def call(dy=FAKE, dt=0, M=100, N=32, ldy=32, z=FAKE, ldz=32, act=1, dz=FAKE, lddz=32, dbias=FAKE, acc=0, ws=FAKE,
             ws_n=1 << 20):
        return lib.nvfp4_act_grad(dy, dt, M, N, ldy, z, ldz, act, dz, lddz, dbias, acc, ws, ws_n, None)

    assert call(dy=None) == INVALID
    assert call(z=None) == INVALID
    assert call(dt=2) == INVALID
    assert call(act=7) == INVALID
    assert call(M=-1) == INVALID
    assert call(ldy=31) == INVALID
    assert call(ldz=31) == INVALID
    assert call(lddz=31) == INVALID
    assert call(dz=None, dbias=None) == INVALID
    assert call(dy=FAKE + 2, dt=1) == INVALID
    assert call(dz=FAKE + 1) == INVALID
    assert call(dbias=FAKE + 2) == INVALID
    assert lib.nvfp4_workspace_size(nv.OP_ACT_GRAD, 128, 32, 1) == 0        # one run of rows: no partial sums
    need = lib.nvfp4_workspace_size(nv.OP_ACT_GRAD, 129, 32, 1)
    assert need > 0
    assert call(M=129, ws=None, ws_n=0) == WORKSPACE
    assert call(M=129, ws_n=need - 1) == WORKSPACE
    assert call(M=129, ws=FAKE + 64) == WORKSPACE


def _moe(**kw):
    f = dict(experts=8, hidden=64, ffn=32, top_k=2, router=FAKE, router_dt=0, act=1, gated=0, score=0, renormalize=1,
             routed_scale=1.0)
    w1 = kw.pop("w1", nv._CTensor(FAKE, FAKE, FAKE, 8 * 32, 64))
    w2 = kw.pop("w2", nv._CTensor(FAKE, FAKE, FAKE, 8 * 64, 32))
    f.update(kw)
    return nv._CMoE(w1=w1, w2=w2, **f)


def test_moe_validation(lib):
    def call(moe=None, x=FAKE, tokens=4, ldx=64, y=FAKE, ldy=64, ids=None, wts=None, ws=FAKE, ws_n=1 << 20, **kw):
        m = _moe(**kw)
        return lib.nvfp4_moe_tokens(ctypes.byref(m), x, tokens, ldx, y, ldy, ids, wts, ws, ws_n, None)

    assert lib.nvfp4_moe_tokens(None, FAKE, 1, 64, FAKE, 64, None, None, FAKE, 1 << 20, None) == INVALID
    assert call(tokens=0, x=None, y=None, ws=None) == 0                       # nothing to do
    for kw in (dict(experts=0), dict(hidden=72), dict(ffn=8), dict(top_k=0), dict(top_k=9), dict(router=None),
               dict(router=FAKE + 2, router_dt=1), dict(router_dt=3), dict(act=9), dict(score=2), dict(gated=1),
               dict(routed_scale=float("inf")), dict(w1=nv._CTensor(FAKE, FAKE, FAKE, 256, 48)),
               dict(w2=nv._CTensor(FAKE, FAKE, FAKE, 511, 32)), dict(w1=nv._CTensor(None, FAKE, FAKE, 256, 64)),
               dict(w2=nv._CTensor(FAKE + 8, FAKE, FAKE, 512, 32)), dict(w2=nv._CTensor(FAKE, FAKE + 1, FAKE, 512, 32)),
               dict(x=None), dict(y=None), dict(x=FAKE + 1), dict(ldx=63), dict(ldy=63), dict(tokens=-1),
               dict(ids=FAKE + 2), dict(wts=FAKE + 2)):
        assert call(**kw) == INVALID, kw
    assert call(tokens=65) == UNSUPPORTED
    assert call(experts=513, w1=nv._CTensor(FAKE, FAKE, FAKE, 513 * 32, 64),
                w2=nv._CTensor(FAKE, FAKE, FAKE, 513 * 64, 32)) == UNSUPPORTED
    assert call(experts=32, top_k=17) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 128) == WORKSPACE
    need = [lib.nvfp4_moe_workspace_size(ctypes.byref(_moe()), t) for t in (0, 1, 2, 64)]
    assert need == sorted(need) and 0 < need[0] < need[1]
    assert call(ws_n=need[1]) == WORKSPACE
    assert lib.nvfp4_moe_workspace_size(ctypes.byref(_moe()), 65) == 0
    assert lib.nvfp4_moe_workspace_size(ctypes.byref(_moe(top_k=9)), 1) == 0
