"""Host-side refusals of the C entries for the norm, 8-bit activations, tokens by expert and the output head (no GPU:
every call fails its checks before anything is enqueued)."""
import ctypes
import os

import pytest

import bit_block_scaled_quantize_amd as nv

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        pytest.skip("libnvfp4.so not built")
    return nv.library()


def _fp8(rows=32, cols=64, codes=P, scales=P):
    return ctypes.byref(nv._CFP8Tensor(codes, scales, rows, cols))


def test_fp8(lib):
    q = lambda x=P, dt=0, rows=32, cols=64, ld=64, out=None: lib.nvfp4_fp8_quantize(  # noqa: E731
        x, dt, rows, cols, ld, _fp8() if out is None else out, None)
    assert q(x=None) == q(x=P + 1) == q(dt=2) == q(rows=-1) == q(cols=0) == q(ld=63) == INVALID
    assert q(dt=1, x=P + 2) == INVALID
    assert q(out=_fp8(rows=31)) == q(out=_fp8(codes=None)) == q(out=_fp8(scales=None)) == q(out=_fp8(codes=P + 8)) == INVALID
    assert q(x=None, rows=0, out=_fp8(rows=0, codes=None, scales=None)) == OK
    d = lib.nvfp4_fp8_dequantize
    assert d(None, P, 64, None) == d(_fp8(), None, 64, None) == d(_fp8(), P, 63, None) == d(_fp8(), P + 1, 64, None) == INVALID
    out = lambda rows=64, cols=32: ctypes.byref(nv._CTensor(P, P, P, rows, cols))  # noqa: E731
    r = lambda x=None, rnd=0, seg=None, nseg=1, amax=P, o=None, ws=None, n=0: lib.nvfp4_rht_quantize_fp8(  # noqa: E731
        _fp8() if x is None else x, 1, rnd, 0, 0, seg, nseg, amax, out() if o is None else o, ws, n, None)
    assert r(x=_fp8(rows=24)) == r(x=_fp8(scales=None)) == r(rnd=2) == r(nseg=2) == r(seg=P, nseg=0) == r(o=out(32, 64)) == INVALID
    assert r(amax=None) == r(amax=None, ws=P, n=100) == r(amax=None, ws=P + 8, n=1 << 20) == WORKSPACE
    a = lambda dy=P, dt=0, ldy=64, z=None, act=1, dz=P, lddz=64, db=None, ws=None, n=0: lib.nvfp4_act_grad_fp8(  # noqa: E731
        dy, dt, ldy, _fp8() if z is None else z, act, dz, lddz, db, 0, ws, n, None)
    assert a(dy=None) == a(dt=3) == a(ldy=60) == a(act=0) == a(act=4) == a(lddz=60) == a(dz=None) == a(db=P + 2) == a(z=_fp8(codes=None)) == INVALID
    big = _fp8(rows=5000, cols=64)
    assert a(z=big, db=P) == WORKSPACE


def test_norm(lib):
    def f(x=P, dt=0, rows=4, cols=64, ldx=64, w=P, wdt=1, eps=1e-6, r=None, ldr=64, ro=None, ldro=64, y=P, ldy=64, y8=None, amax=None):
        return lib.nvfp4_rms_norm(x, dt, rows, cols, ldx, w, wdt, eps, r, ldr, ro, ldro, y, ldy, y8, amax, None)
    assert f(x=None) == f(x=P + 1) == f(dt=2) == f(rows=-1) == f(cols=0) == f(ldx=63) == f(w=None) == f(wdt=2) == f(w=P + 2) == INVALID
    assert f(eps=0.0) == f(eps=-1.0) == f(eps=float("nan")) == f(eps=float("inf")) == INVALID
    assert f(y=None) == f(ro=P) == f(r=P, ldr=3) == f(r=P, ro=P, ldro=3) == f(ldy=63) == f(y=P + 1) == f(amax=P + 1) == INVALID
    assert f(y8=_fp8(4, 32)) == f(y8=_fp8(4, 64, codes=None)) == INVALID
    assert f(cols=16385, ldx=16385, ldy=16385) == UNSUPPORTED
    assert f(rows=0, x=None, w=None, y=None) == OK

    def g(dy=P, dydt=0, rows=4, cols=64, lddy=64, h=P, dt=0, ldh=64, w=P, eps=1e-6, dr=None, lddr=64, dx=P, lddx=64, dw=None, ws=None, n=0):
        return lib.nvfp4_rms_norm_grad(dy, dydt, rows, cols, lddy, h, dt, ldh, w, 1, eps, dr, lddr, dx, lddx, dw, 0, ws, n, None)
    assert g(dy=None) == g(dydt=2) == g(h=None) == g(dt=5) == g(dx=None) == g(lddy=1) == g(ldh=1) == g(lddx=1) == g(dr=P, lddr=1) == g(dw=P + 2) == INVALID
    assert g(rows=500, dw=P) == g(rows=500, dw=P, ws=P, n=8) == WORKSPACE


def test_moe_sort(lib):
    rows = lib.nvfp4_moe_sorted_rows
    assert rows(10, 2, 4, 64) == (20 + 4 * 63) // 64 * 64 and rows(1, 1, 128, 64) == 64 and rows(7, 3, 24, 1) == 21 and rows(0, 3, 4, 64) == 0
    assert rows(-1, 1, 1, 1) == rows(1, 0, 1, 1) == rows(1, 1, 0, 1) == rows(1, 1, 1, 0) == rows(1 << 30, 2, 4, 64) == rows(1 << 31, 1, 1, 1) == -1
    assert rows(1 << 30, 1, 1 << 30, 64) == -1

    def s(ids=P, t=10, k=2, e=4, align=64, rows=512, off=P, row_of=P, pair_of=P, ws=None, n=0):
        return lib.nvfp4_moe_sort(ids, t, k, e, align, rows, off, row_of, pair_of, ws, n, None)
    assert s(ids=None) == s(t=-1) == s(k=0) == s(e=0) == s(align=0) == s(rows=255) == s(off=None) == s(row_of=None) == s(pair_of=None) == INVALID
    assert s(off=P + 4) == s(ids=P + 2) == INVALID
    assert s(e=1025, rows=1 << 20) == s(t=1 << 31, rows=1 << 30) == UNSUPPORTED
    assert s(t=4000, rows=9000) == s(t=4000, rows=9000, ws=P, n=4) == WORKSPACE

    def ga(x=P, dt=0, t=10, h=64, ldx=64, pair_of=P, rows=256, k=2, w=None, out=P, ldo=64):
        return lib.nvfp4_moe_gather(x, dt, t, h, ldx, pair_of, rows, k, w, out, ldo, None)
    assert ga(x=None) == ga(dt=2) == ga(h=0) == ga(ldx=1) == ga(pair_of=None) == ga(out=None) == ga(ldo=1) == ga(w=P + 1) == ga(k=0) == INVALID
    assert ga(rows=1 << 31) == ga(rows=1 << 26) == UNSUPPORTED

    def co(y=P, dt=1, rows=256, h=64, ldy=64, row_of=P, t=10, k=2, w=None, out=P, odt=0, ldo=64):
        return lib.nvfp4_moe_combine(y, dt, rows, h, ldy, row_of, t, k, w, out, odt, ldo, None)
    assert co(y=None) == co(dt=2) == co(odt=2) == co(row_of=None) == co(out=None) == co(ldy=1) == co(ldo=1) == co(w=P + 2) == INVALID
    assert co(t=1 << 29) == co(t=1 << 25, h=8192, ldy=8192, ldo=8192) == UNSUPPORTED

    def cg(do=P, odt=0, t=10, h=64, lddo=64, y=P, dt=1, rows=256, ldy=64, row_of=P, pair_of=P, k=2, w=P, dy=P, lddy=64, dw=P):
        return lib.nvfp4_moe_combine_grad(do, odt, t, h, lddo, y, dt, rows, ldy, row_of, pair_of, k, w, dy, lddy, dw, None)
    assert cg(do=None) == cg(y=None) == cg(row_of=None) == cg(pair_of=None) == cg(w=None) == cg(dy=None, dw=None) == cg(lddy=1) == cg(dw=P + 1) == INVALID
    assert cg(t=1 << 25) == cg(rows=1 << 30) == UNSUPPORTED


def test_head(lib):
    def f(x=P, t=8, ldx=64, w=P, v=100, ldw=64, h=64, tg=P, loss=P, lse=P, ws=None, n=0):
        return lib.nvfp4_linear_cross_entropy(x, t, ldx, w, v, ldw, h, tg, loss, lse, ws, n, None)
    assert f(x=None) == f(t=-1) == f(ldx=60) == f(ldx=68) == f(x=P + 8) == f(w=None) == f(v=0) == f(ldw=68) == f(h=24) == f(h=0) == f(tg=None) == INVALID
    assert f(tg=P + 4) == f(loss=None, lse=None) == f(loss=P + 2) == INVALID
    assert f(t=(1 << 21) + 1) == f(ldw=1 << 22) == UNSUPPORTED
    assert f(t=1 << 21, h=8192, ldx=8192, ldw=8192) == f(t=1 << 21, v=1 << 17) == f(v=1 << 30, h=32768, ldx=32768, ldw=32768) == UNSUPPORTED
    assert f() == f(ws=P, n=64) == f(ws=P + 16, n=1 << 30) == WORKSPACE
    assert f(t=0, x=None, tg=None, loss=None, lse=None) == OK

    def g(lse=P, gr=P, dx=P, lddx=64, dw=P, kind=2, lddw=64, ws=None, n=0, t=8):
        return lib.nvfp4_linear_cross_entropy_grad(P, t, 64, P, 100, 64, 64, P, lse, gr, dx, lddx, dw, kind, lddw, ws, n, None)
    assert g(lse=None) == g(gr=None) == g(dx=None, dw=None) == g(lddx=1) == g(lddw=1) == g(kind=3) == g(kind=0, dw=P + 2) == INVALID
    assert g() == g(ws=P, n=100) == WORKSPACE
    for t in (1, 8192):
        assert lib.nvfp4_workspace_size(nv.OP_HEAD_GRAD, t, 131072, 5120) < 2 << 30
    assert lib.nvfp4_workspace_size(nv.OP_HEAD_GRAD, 0, 100, 64) == 0


def test_head_grad_with_the_loss(lib):
    def g(loss=P, lse=P, dx=P, ws=None, n=0):
        return lib.nvfp4_linear_cross_entropy_grad_ex(P, 8, 64, P, 100, 64, 64, P, lse, loss, P, dx, 64, P, 2, 64, ws, n, None)
    assert g(loss=P + 2) == g(lse=None) == g(dx=P + 1) == INVALID
    assert g() == g(loss=None) == g(ws=P, n=100) == WORKSPACE


def test_norm_in_place(lib):
    """An output may be an input only row for row: the same address with unequal strides would overwrite rows that are still to be read."""
    Q, S = 0x20000, 0x30000

    def f(x=P, ldx=64, r=Q, ldr=64, ro=None, ldro=64, y=S, ldy=64, dt=0, rows=4):
        return lib.nvfp4_rms_norm(x, dt, rows, 64, ldx, S, 1, 1e-6, r, ldr, ro, ldro, y, ldy, None, None, None)
    assert f(ro=P, ldro=72) == f(ro=Q, ldro=72) == f(ro=P, ldx=72) == f(ro=Q, ldr=72, dt=1) == INVALID
    assert b"unequal row strides" in lib.nvfp4_last_error()
    assert f(ro=S, y=S) == f(y=P, ldy=72) == f(y=Q, dt=1) == INVALID

    def g(dy=P, lddy=64, h=Q, ldh=64, dr=None, lddr=64, dx=S, lddx=64, dydt=0):
        return lib.nvfp4_rms_norm_grad(dy, dydt, 4, 64, lddy, h, 0, ldh, S, 1, 1e-6, dr, lddr, dx, lddx, None, 0, None, 0, None)
    assert g(dr=S, lddr=72) == g(dx=P, lddx=72) == g(dx=P, dydt=1) == g(dx=Q, ldh=72) == INVALID
    assert b"unequal row strides" in lib.nvfp4_last_error()
