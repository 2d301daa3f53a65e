"""The training-step entry points on a machine without a GPU: arguments are
refused on the host, before any device call. No compute call is made here."""
import ctypes

import pytest

tt = pytest.importorskip("exact_inner_product_b200")

INV, UNS = tt.TT_ERR_INVALID_ARG, tt.TT_ERR_UNSUPPORTED
P = [ctypes.c_void_p(0x1000000 * (i + 1)) for i in range(12)]  # never dereferenced
ODD = ctypes.c_void_p(0x1000002)


def test_layernorm_arguments():
    def call(x=P[0], dt=0, n=4, d=64, w=P[1], bias=P[2], wdt=0, eps=1e-5, y=P[3], mean=P[4], rstd=P[5]):
        return tt._lib.tt_layernorm(x, dt, n, d, w, bias, wdt, eps, y, mean, rstd, None)

    assert call(n=-1) == INV and call(d=0) == INV and call(d=-5) == INV
    assert call(d=tt.TT_MAX_WIDTH + 1) == UNS and call(n=1 << 31) == UNS
    assert call(dt=tt.TT_I8) == INV and call(wdt=7) == INV
    assert call(eps=-1.0) == INV and call(eps=float("nan")) == INV and call(eps=float("inf")) == INV
    assert call(x=None) == INV and call(y=None) == INV
    assert call(x=ODD) == INV and call(y=ODD) == INV and call(w=ODD) == INV and call(mean=ODD) == INV
    assert call(y=P[0]) == INV                                   # in place
    assert call(mean=P[5]) == INV                                # mean is rstd
    assert call(rstd=ctypes.c_void_p(P[0].value + 16)) == INV    # inside x
    assert call(n=0, x=None, y=None) == tt.TT_OK


def test_layernorm_grad_arguments():
    size = ctypes.c_size_t(0)
    assert tt._lib.tt_layernorm_grad_workspace(4, 64, None) == INV
    assert tt._lib.tt_layernorm_grad_workspace(-1, 64, ctypes.byref(size)) == INV
    assert tt._lib.tt_layernorm_grad_workspace(4, 20000, ctypes.byref(size)) == UNS
    assert tt._lib.tt_layernorm_grad_workspace(4, 64, ctypes.byref(size)) == tt.TT_OK
    need = size.value
    assert need >= 2 * 64 * 4

    def call(dy=P[0], x=P[1], dt=0, n=4, d=64, w=P[2], wdt=0, mean=P[3], rstd=P[4], gx=P[5], gw=P[6], gb=P[7], ws=P[8],
             size=need):
        return tt._lib.tt_layernorm_grad(dy, x, dt, n, d, w, wdt, mean, rstd, gx, gw, gb, ws, size, None)

    assert call(n=-1) == INV and call(d=0) == INV and call(d=20000) == UNS
    assert call(dt=9) == INV and call(wdt=tt.TT_I8) == INV
    assert call(dy=None) == INV and call(x=None) == INV and call(mean=None) == INV and call(rstd=None) == INV
    assert call(ws=None) == INV and call(ws=ODD) == INV and call(size=need - 1) == INV
    assert call(gx=ODD) == INV and call(gx=P[1]) == INV and call(gx=P[0]) == INV and call(gw=P[7]) == INV


def test_normalize_grad_arguments():
    def call(dy=P[0], gdt=0, x=P[1], dt=0, n=4, d=64, gx=P[2]):
        return tt._lib.tt_normalize_grad(dy, gdt, x, dt, n, d, gx, None)

    assert call(n=-1) == INV and call(d=0) == INV and call(d=40) == UNS and call(d=528) == UNS and call(n=1 << 31) == UNS
    assert call(dt=tt.TT_I8) == INV and call(gdt=5) == INV
    assert call(dy=None) == INV and call(x=None) == INV and call(gx=None) == INV and call(gx=ODD) == INV
    assert call(gx=P[0]) == INV and call(gx=P[1]) == INV
    assert call(n=0, dy=None, x=None, gx=None) == tt.TT_OK


def _list(kind, values):
    return (kind * max(1, len(values)))(*values)


def test_clip_arguments():
    A, B = 0x1000000, 0x2000000
    size = ctypes.c_size_t(0)
    n2, f2 = _list(ctypes.c_int64, [100, 200]), _list(ctypes.c_int32, [0, 1])
    assert tt._lib.tt_clip_grad_norm_workspace(2, n2, f2, None) == INV
    assert tt._lib.tt_clip_grad_norm_workspace(-1, n2, f2, ctypes.byref(size)) == INV
    assert tt._lib.tt_clip_grad_norm_workspace(2, None, f2, ctypes.byref(size)) == INV
    assert tt._lib.tt_clip_grad_norm_workspace(2, n2, f2, ctypes.byref(size)) == tt.TT_OK
    need = size.value

    def call(count=2, ins=(A, B), n=(100, 200), dt=(0, 1), outs=None, max_norm=1.0, norm=P[5], ws=P[6], size=need):
        outs = None if outs is None else _list(ctypes.c_void_p, outs)
        return tt._lib.tt_clip_grad_norm(count, _list(ctypes.c_void_p, ins), _list(ctypes.c_int64, n),
                                         _list(ctypes.c_int32, dt), outs, max_norm, norm, ws, size, None)

    assert call(count=-1) == INV and call(n=(100, -1)) == INV and call(n=(100, 1 << 42)) == UNS
    assert call(dt=(0, tt.TT_I8)) == INV and call(dt=(0, 9)) == INV
    assert call(max_norm=-1.0) == INV and call(max_norm=float("nan")) == INV
    assert call(norm=None) == INV and call(ws=None) == INV and call(ws=ODD) == INV and call(size=need - 1) == INV
    assert call(ins=(A, None)) == INV and call(ins=(A + 2, B)) == INV and call(ins=(A, B + 1)) == INV
    assert call(ins=(A, A)) == INV                      # one tensor twice, in place
    assert call(ins=(A, A + 396)) == INV                # the last element of the first
    assert call(outs=(A, A)) == INV and call(outs=(B, A)) == INV  # an output over another tensor's input
    assert call(outs=(A + 4, 0x3000000)) == INV         # an output over its own input, shifted
    assert call(norm=ctypes.c_void_p(A + 8)) == INV and call(ws=ctypes.c_void_p(A & ~255)) == INV
    # the norm alone takes the same tensor twice; its other arguments are checked alike
    grad_norm = lambda ins=(A, B), norm=P[5], ws=P[6], size=need: tt._lib.tt_grad_norm(  # noqa: E731
        2, _list(ctypes.c_void_p, ins), n2, f2, norm, ws, size, None)
    assert grad_norm(ins=(None, B)) == INV and grad_norm(norm=None) == INV and grad_norm(size=need - 1) == INV


def test_embedding_arguments():
    def call(table=P[0], dt=0, rows=10, d=64, ids=P[1], id_bytes=8, m=4, scale=1.0, out=P[2], odt=0):
        return tt._lib.tt_embedding(table, dt, rows, d, ids, id_bytes, m, scale, out, odt, None)

    assert call(rows=-1) == INV and call(d=0) == INV and call(m=-1) == INV
    assert call(rows=1 << 31) == UNS and call(d=tt.TT_MAX_WIDTH + 1) == UNS and call(m=1 << 31) == UNS
    assert call(id_bytes=2) == INV and call(scale=float("nan")) == INV and call(scale=float("inf")) == INV
    assert call(dt=tt.TT_I8) == INV and call(odt=8) == INV
    assert call(table=None) == INV and call(ids=None) == INV and call(out=None) == INV
    assert call(table=ODD) == INV and call(out=ODD) == INV and call(ids=ctypes.c_void_p(0x1000004)) == INV
    assert call(out=P[0]) == INV and call(out=ctypes.c_void_p(P[1].value + 16)) == INV
    assert call(m=0, table=None, ids=None, out=None) == tt.TT_OK


def test_embedding_grad_arguments():
    size = ctypes.c_size_t(0)
    assert tt._lib.tt_embedding_grad_workspace(4, 10, 64, None) == INV
    assert tt._lib.tt_embedding_grad_workspace(-4, 10, 64, ctypes.byref(size)) == INV
    assert tt._lib.tt_embedding_grad_workspace(4, 10, 64, ctypes.byref(size)) == tt.TT_OK
    need = size.value

    def dense(ids=P[0], id_bytes=4, m=4, grad=P[1], dt=0, rows=10, d=64, scale=1.0, out=P[2], odt=0, ws=P[3], size=need):
        return tt._lib.tt_embedding_grad(ids, id_bytes, m, grad, dt, rows, d, scale, out, odt, ws, size, None)

    def by_row(ids=P[0], id_bytes=4, m=4, grad=P[1], dt=0, rows=10, d=64, scale=1.0, oids=P[2], out=P[3], odt=0,
               count=P[4], ws=P[5], size=need):
        return tt._lib.tt_embedding_grad_rows(ids, id_bytes, m, grad, dt, rows, d, scale, oids, out, odt, count, ws, size,
                                              None)

    for call in (dense, by_row):
        assert call(rows=-1) == INV and call(rows=1 << 31) == UNS and call(m=-1) == INV and call(m=1 << 31) == UNS
        assert call(d=0) == INV and call(d=20000) == UNS and call(id_bytes=1) == INV and call(scale=float("nan")) == INV
        assert call(dt=tt.TT_I8) == INV and call(odt=tt.TT_I8) == INV
        assert call(ids=None) == INV and call(grad=None) == INV and call(out=None) == INV
        assert call(ids=ODD) == INV and call(grad=ODD) == INV and call(out=ODD) == INV
        assert call(ws=None) == INV and call(ws=ODD) == INV and call(size=need - 1) == INV
        assert call(out=P[1]) == INV and call(ws=P[1]) == INV
    assert by_row(oids=None) == INV and by_row(count=None) == INV and by_row(oids=P[0]) == INV and by_row(count=P[2]) == INV


def test_inbatch_softmax_grad_arguments():
    size = ctypes.c_size_t(0)
    need_of = tt._lib.tt_inbatch_softmax_grad_workspace
    assert need_of(8, 9, 64, 1, 1, None) == INV
    assert need_of(9, 8, 64, 1, 1, ctypes.byref(size)) == INV and need_of(-1, 8, 64, 1, 1, ctypes.byref(size)) == INV
    assert need_of(8, 9, 72, 1, 1, ctypes.byref(size)) == UNS and need_of(8, 9, 48, 1, 1, ctypes.byref(size)) == UNS
    assert need_of(8, 9, 528, 1, 1, ctypes.byref(size)) == UNS
    assert need_of(8, (1 << 28) + 1, 64, 1, 1, ctypes.byref(size)) == UNS
    assert need_of(8, 9, 64, 1, 1, ctypes.byref(size)) == tt.TT_OK
    need = size.value

    def call(u=P[0], v=P[1], dt=tt.TT_BF16, b=8, nc=9, d=64, tau=0.1, logq=P[2], ids=P[3], valid=P[4], lse=P[5], loss=P[6],
             gl=P[7], gm=P[8], gu=P[9], gv=P[10], ws=P[11], size=need):
        return tt._lib.tt_inbatch_softmax_grad(u, v, dt, b, nc, d, tau, logq, ids, valid, lse, loss, gl, gm, gu, gv, ws, size,
                                               None)

    assert call(dt=tt.TT_F32) == UNS and call(dt=7) == INV
    assert call(b=10) == INV and call(b=-1) == INV and call(d=0) == INV and call(d=72) == UNS and call(d=48) == UNS
    assert call(tau=0.0) == INV and call(tau=-1.0) == INV and call(tau=float("nan")) == INV and call(tau=float("inf")) == INV
    assert call(gl=None, gm=None) == INV
    for name in ("u", "v", "lse", "loss", "gu", "gv", "ws"):
        assert call(**{name: None}) == INV, name
    for name in ("u", "v", "ids", "lse", "loss", "gl", "gm", "gu", "gv", "ws", "logq"):
        assert call(**{name: ctypes.c_void_p(0x1000001)}) == INV, name
    assert call(size=need - 1) == INV
    assert call(gu=P[0]) == INV and call(gv=P[1]) == INV and call(gv=P[9]) == INV and call(ws=P[5]) == INV
