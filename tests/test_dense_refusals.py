"""What the linear and gated layers and the optimiser's step refuse, on the host: no call below reaches a GPU."""
import ctypes

import pytest

from activation_sparse_transformer_tcgen05_gb300 import build as tbuild
from activation_sparse_transformer_tcgen05_gb300 import twell as tw

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 40


def at(k):
    return ctypes.c_void_p(k << 20)


@pytest.fixture(scope="module")
def lib():
    tbuild.build()
    return tw.load_library()


def test_linear_forward(lib):
    def call(x=at(1), ldx=64, W=at(2), kn=0, bias=at(3), act=0, res=at(4), ldr=24, M=4, N=24, K=64, pre=at(5), ldp=24, y=at(6),
             ldy=24, ty=0, st=at(7)):
        return lib.twell_linear_fwd(x, ldx, W, kn, bias, act, res, ldr, M, N, K, pre, ldp, y, ldy, ty, st, None)

    assert call(x=None) == call(W=None) == call(y=None) == call(st=None) == INVALID
    assert call(M=-1) == call(N=0) == call(K=0) == call(K=60, ldx=64) == call(kn=2) == call(kn=1, N=23) == INVALID
    assert call(act=5) == call(act=-1) == call(ty=2) == INVALID
    assert call(ldx=56) == call(ldx=68) == call(ldy=23) == call(ldr=23) == call(ldp=23) == INVALID
    odd = ctypes.c_void_p((9 << 20) + 8)
    assert call(x=odd) == call(W=odd) == INVALID
    assert call(y=ctypes.c_void_p((9 << 20) + 1)) == call(y=ctypes.c_void_p((9 << 20) + 2), ty=1) == INVALID
    assert call(bias=ctypes.c_void_p((9 << 20) + 2)) == call(st=ctypes.c_void_p((9 << 20) + 2)) == INVALID
    assert call(y=at(1)) == call(y=at(2)) == call(pre=at(1)) == call(pre=at(6)) == call(pre=at(4)) == INVALID
    assert call(M=2 ** 30 + 1) == call(N=2 ** 30 + 8, ldy=2 ** 31, ldr=2 ** 31, ldp=2 ** 31) == UNSUPPORTED
    assert call(M=0, x=None, y=None) == OK


def test_linear_backward(lib):
    need = lib.twell_linear_bwd_workspace_bytes(100, 24, 64)
    assert need >= 100 * 64 * 2 + 4 * 24 * 4
    assert lib.twell_linear_bwd_workspace_bytes(-1, 24, 64) == lib.twell_linear_bwd_workspace_bytes(4, 24, 60) == 0
    assert lib.twell_linear_bwd_workspace_bytes(2 ** 30 + 1, 24, 64) == 0

    def call(dy=at(1), ldg=24, x=at(2), ldx=64, W=at(3), kn=0, act=1, pre=at(4), ldp=24, M=100, N=24, K=64, dx=at(5), ldd=64,
             dW=at(6), tw_=0, acc=0, db=at(7), ws=at(8), n=need, st=at(9)):
        return lib.twell_linear_bwd(dy, ldg, x, ldx, W, kn, act, pre, ldp, M, N, K, dx, ldd, dW, tw_, acc, db, ws, n, st, None)

    assert call(dy=None) == call(x=None) == call(W=None) == call(pre=None) == call(st=None) == INVALID
    assert call(dx=None, dW=None, db=None) == call(acc=1) == call(tw_=2) == call(K=60) == call(act=7) == INVALID
    assert call(ldg=23) == call(ldx=60) == call(ldp=23) == call(ldd=63) == INVALID
    assert call(dx=at(1)) == call(dW=at(2)) == call(dW=at(5)) == call(dx=at(4)) == INVALID
    assert call(dW=ctypes.c_void_p((9 << 20) + 8)) == call(db=ctypes.c_void_p((9 << 20) + 2)) == INVALID
    assert call(ws=None) == call(n=need - 1) == WORKSPACE and call(ws=ctypes.c_void_p((9 << 20) + 128)) == INVALID
    assert call(N=2 ** 30 + 8) == UNSUPPORTED


def test_gated_forward(lib):
    def call(x=at(1), Wg=at(2), Wu=at(3), b=at(4), Wd=at(5), act=1, res=at(6), M=4, d=64, F=24, g=at(7), u=at(8), h=at(9),
             y=at(10), st=at(11)):
        return lib.twell_dense_gated_ffn_fwd(x, Wg, Wu, b, Wd, act, res, M, d, F, g, u, h, y, st, None)

    assert call(x=None) == call(Wg=None) == call(Wu=None) == call(Wd=None) == call(h=None) == call(y=None) == INVALID
    assert call(st=None) == call(g=None) == call(u=None) == call(act=9) == INVALID
    assert call(M=-1) == call(d=60) == call(F=20) == call(F=0) == INVALID
    assert call(x=ctypes.c_void_p((12 << 20) + 8)) == call(h=ctypes.c_void_p((12 << 20) + 2)) == INVALID
    assert call(b=ctypes.c_void_p((12 << 20) + 2)) == INVALID
    assert call(h=at(1)) == call(y=at(1)) == call(h=at(10)) == call(g=at(8)) == call(u=at(9)) == call(res=at(9)) == INVALID
    assert call(F=2 ** 30 + 8) == UNSUPPORTED
    assert call(M=0, x=None, h=None) == OK


def test_gated_backward(lib):
    need = lib.twell_dense_gated_bwd_workspace_bytes(100, 64, 24)
    assert need >= 2 * 100 * 24 * 2 + 4 * 24 * 4
    assert lib.twell_dense_gated_bwd_workspace_bytes(4, 60, 24) == lib.twell_dense_gated_bwd_workspace_bytes(-4, 64, 24) == 0

    def call(x=at(1), Wg=at(2), Wu=at(3), Wd=at(4), act=1, g=at(5), u=at(6), h=at(7), dy=at(8), M=100, d=64, F=24, dx=at(9),
             dWg=at(10), dWu=at(11), dWd=at(12), tw_=0, acc=0, db=at(13), ws=at(14), n=need, st=at(15)):
        return lib.twell_dense_gated_ffn_bwd(x, Wg, Wu, Wd, act, g, u, h, dy, 0.0, M, d, F, dx, dWg, dWu, dWd, tw_, acc, db, ws, n,
                                             st, None)

    assert call(x=None) == call(Wg=None) == call(Wd=None) == call(g=None) == call(u=None) == call(h=None) == INVALID
    assert call(dy=None) == call(st=None) == call(dWu=None) == call(acc=1) == call(tw_=3) == call(act=-1) == INVALID
    assert call(dx=None, dWg=None, dWu=None, dWd=None, db=None) == INVALID
    assert call(dx=at(8)) == call(dWg=at(7)) == call(dWg=at(11)) == call(dx=at(12)) == INVALID
    assert call(dWd=ctypes.c_void_p((16 << 20) + 8)) == INVALID
    assert call(ws=None) == call(n=need - 1) == WORKSPACE and call(ws=ctypes.c_void_p((16 << 20) + 64)) == INVALID
    assert call(M=2 ** 30 + 1) == UNSUPPORTED


class _List:
    """A list of one tensor with chosen fields."""

    def __init__(self, n=1, bits=32, p=1 << 20, g=2 << 20, m=3 << 20, v=4 << 20, ms=5 << 20, vs=6 << 20, copy=7 << 20, numel=100,
                 pt=1, gt=1, count=1):
        def addr(k):
            return (ctypes.c_void_p * count)(*[k] * count)

        self.keep = [addr(p), addr(g), addr(m), addr(v), addr(ms), addr(vs), addr(copy), (ctypes.c_int64 * count)(*[numel] * count),
                     (ctypes.c_int32 * count)(*[pt] * count), (ctypes.c_int32 * count)(*[gt] * count)]
        self.struct = tw._TwellAdamWList(n, bits, *[ctypes.addressof(k) for k in self.keep])

    @property
    def ref(self):
        return ctypes.byref(self.struct)


def test_adamw(lib):
    def call(lr=at(10), step=at(11), b1=0.9, b2=0.99, eps=1e-8, wd=0.1, norm=at(12), most=1.0, **kw):
        return lib.twell_adamw(_List(**kw).ref, lr, step, b1, b2, eps, wd, norm, most, 0, None)

    nan = float("nan")
    assert lib.twell_adamw(None, at(10), at(11), 0.9, 0.99, 1e-8, 0.1, None, 1.0, 0, None) == INVALID
    assert call(lr=None) == call(step=None) == call(b1=1.0) == call(b2=-0.1) == call(b1=nan) == INVALID
    assert call(eps=0.0) == call(eps=nan) == call(eps=1e-46) == call(wd=-1.0) == call(wd=float("inf")) == INVALID
    assert call(most=-1.0) == call(most=nan) == call(n=-1) == call(bits=16) == call(numel=-1) == INVALID
    assert call(pt=2) == call(gt=-1) == call(p=0) == call(g=0) == call(m=0) == call(v=0) == INVALID
    assert call(p=(1 << 20) + 2) == call(g=(1 << 20) + 1) == call(m=(1 << 20) + 2) == call(copy=(1 << 20) + 1) == INVALID
    assert call(pt=0) == INVALID  # a copy of a bf16 parameter
    assert call(bits=8, ms=0) == call(bits=8, vs=(1 << 20) + 2) == INVALID
    assert call(m=4 << 20) == call(g=1 << 20) == call(copy=1 << 20) == call(v=1 << 20) == INVALID
    assert call(numel=1 << 60) == call(n=32769, count=32769) == UNSUPPORTED
    assert call(n=0) == OK


def test_adamw_values(lib):
    def call(numel=100, out=20 << 20, type_=0, n=1, **kw):
        lst = _List(**{"bits": 8, **kw})
        keep = [(ctypes.c_void_p * 1)(out), (ctypes.c_int64 * 1)(numel), (ctypes.c_int32 * 1)(type_)]
        o = tw._TwellTensorList(n, None, *[ctypes.addressof(k) for k in keep])
        return lib.twell_adamw_values(lst.ref, ctypes.byref(o), ctypes.byref(o), None)

    assert call(bits=32) == call(n=2) == call(type_=2) == call(out=0) == call(out=(20 << 20) + 1) == INVALID
    assert call(out=(20 << 20) + 2, type_=1) == INVALID
    lst = _List(bits=8)
    assert lib.twell_adamw_values(lst.ref, None, None, None) == INVALID
