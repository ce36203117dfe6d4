"""Host-side refusals of the residual norms, the gradient clip and the 8-bit linear: nothing
reaches a device (the addresses are never dereferenced)."""
import ctypes

import pytest

from bit_ternary_qat_b200 import _lib, build

FAKE = 1 << 20
ODD = FAKE + 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


FWD = dict(X=FAKE, x_dt=1, Y=FAKE, y_dt=1, T=8, K=64, post=1, g_post=None, eps_post=1e-6, kind=0, gate=None,
           alpha=1.0, beta=1.0, g_pre=None, eps_pre=1e-6, Xout=FAKE, r_post=FAKE, r_pre=FAKE, H=None, Xq=FAKE, sx=FAKE,
           Xdq=None, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), 1), (dict(Y=None), 1), (dict(Xout=None), 1), (dict(x_dt=2), 1), (dict(y_dt=-1), 1),
    (dict(x_dt=1, y_dt=0), 1), (dict(T=0), 1), (dict(K=0), 1), (dict(T=1 << 31), 2), (dict(K=16416), 2),
    (dict(r_post=None), 1), (dict(r_pre=None), 1), (dict(sx=None), 1), (dict(post=0, g_post=FAKE), 1),
    (dict(kind=5, gate=FAKE), 1), (dict(kind=-1), 1), (dict(kind=2), 1), (dict(gate=FAKE), 1), (dict(alpha=NAN), 1),
    (dict(beta=INF), 1), (dict(eps_post=-1.0), 1), (dict(eps_pre=NAN), 1), (dict(eps_pre=INF), 1), (dict(H=FAKE), 1),
    (dict(Xq=None, sx=None, Xdq=FAKE), 1), (dict(Xq=None, sx=None, g_pre=FAKE), 1), (dict(K=40), 2), (dict(K=33), 2),
    (dict(X=ODD), 3), (dict(Y=ODD), 3), (dict(Xq=ODD), 3), (dict(kind=2, gate=ODD), 3), (dict(g_pre=ODD), 3)])
def test_forward(L, kw, status):
    assert _lib.status("bitlinear_residual_norm", *dict(FWD, **kw).values()) == status
    assert len(_lib.last_error()) > 0


BWD = dict(dXout=FAKE, dH=FAKE, Xout=FAKE, x_dt=1, Y=FAKE, y_dt=1, T=8, K=64, post=1, g_post=None, r_post=FAKE, kind=0,
           gate=None, alpha=1.0, beta=1.0, g_pre=None, r_pre=FAKE, dX=FAKE, dY=FAKE, dg_post=None, dg_pre=None,
           dgate=None, ws=None, ws_bytes=0, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dXout=None, dH=None), 1), (dict(Xout=None), 1), (dict(Y=None), 1), (dict(r_post=None), 1),
    (dict(r_pre=None), 1), (dict(dX=None), 1), (dict(dY=None), 1), (dict(T=0), 1), (dict(K=16385), 2),
    (dict(x_dt=1, y_dt=0), 1), (dict(post=0, dg_post=FAKE), 1), (dict(post=0, g_post=FAKE), 1),
    (dict(dH=None, dg_pre=FAKE), 1), (dict(dgate=FAKE), 1), (dict(kind=2), 1), (dict(dg_pre=FAKE), 1),
    (dict(dg_pre=FAKE, ws=FAKE, ws_bytes=64), 4), (dict(dg_post=FAKE, ws=ODD, ws_bytes=1 << 30), 3),
    (dict(kind=1, gate=FAKE, dgate=FAKE), 1), (dict(dX=ODD), 3), (dict(alpha=INF), 1)])
def test_backward(L, kw, status):
    assert _lib.status("bitlinear_residual_norm_backward", *dict(BWD, **kw).values()) == status
    assert len(_lib.last_error()) > 0


@pytest.mark.parametrize("K", [1, 2, 3, 7, 8, 32, 1000, 4096, 16384])
def test_one_workspace_suffices(L, K):
    """Three gains' partial sums of 148 blocks and the scalar gate's fit the layer's workspace."""
    assert L.bitlinear_workspace_bytes(1, 16, K) >= 148 * (8 + 12 * K)
    assert L.bitlinear_workspace_bytes(1, 1, 1) >= 8 * 1184


def grads(ptrs=(FAKE,), numel=(10,), types=(0,), out=None, count=None, max_norm=1.0, norm=FAKE, coef=FAKE, ws=FAKE,
          ws_bytes=1 << 20, clip=False, null=False):
    n = len(ptrs)
    P = (_lib.P * n)(*ptrs)
    O = (_lib.P * n)(*(ptrs if out is None else out))
    lists = [None if null else P] + ([O] if clip else []) + [(_lib.I64 * n)(*numel), (_lib.INT * n)(*types)]
    return _lib.status("bitlinear_clip_grads" if clip else "bitlinear_grad_norm", *lists, n if count is None else count,
                       max_norm, norm, coef, ws, ws_bytes, None)


def test_grads(L):
    for kw, status in ((dict(null=True), 1), (dict(ptrs=(None,)), 1), (dict(numel=(-1,)), 1), (dict(types=(3,)), 1),
                       (dict(count=-1), 1), (dict(max_norm=NAN), 1), (dict(max_norm=INF), 1), (dict(norm=None), 1),
                       (dict(coef=None), 1), (dict(norm=FAKE + 2), 3), (dict(ws=None), 1), (dict(ws=ODD), 3),
                       (dict(ws_bytes=64), 4), (dict(ptrs=(FAKE + 2,)), 3), (dict(ptrs=(FAKE + 1,), types=(1,)), 3),
                       (dict(numel=((1 << 40) + 1,)), 1), (dict(ptrs=(FAKE, FAKE), numel=(1 << 40, 1), types=(0, 0)), 2)):
        for clip in (False, True):
            assert grads(clip=clip, **kw) == status, (kw, clip)
            assert len(_lib.last_error()) > 0
    assert grads(clip=True, out=(None,)) == 1
    assert grads(clip=True, out=(FAKE + 2,)) == 3


def test_optimizer_step_coef(L):
    names = ["W", "dW", "m", "v", "N", "K", "lr", "b1", "b2", "eps", "wd", "coef", "step", "wq", "wbf", "pk", "gamma",
             "ws", "ws_bytes", "st"]
    ok = [FAKE, FAKE, FAKE, FAKE, 16, 32, 1e-3, 0.9, 0.95, 1e-6, 0.01, FAKE, FAKE, None, None, None, None, FAKE,
          1 << 20, None]
    for kw, status in ((dict(coef=None), 1), (dict(coef=FAKE + 2), 3), (dict(step=None), 1), (dict(b1=1.0), 1),
                       (dict(lr=NAN), 1), (dict(wq=FAKE), 1), (dict(ws_bytes=64), 4), (dict(K=48), 2), (dict(W=ODD), 3)):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        assert _lib.status("bitlinear_optimizer_step_coef", *a) == status, kw


@pytest.mark.parametrize("kw,status", [
    (dict(W=None), 1), (dict(gamma=None), 1), (dict(N=0), 1), (dict(N=24), 2), (dict(K=40), 2), (dict(wq=ODD), 3)])
def test_quant_weight_int8(L, kw, status):
    a = dict(W=FAKE, N=16, K=32, wq=None, wbf=None, gamma=FAKE, st=None)
    assert _lib.status("bitlinear_quant_weight_int8", *dict(a, **kw).values()) == status


@pytest.mark.parametrize("kw,status", [
    (dict(xq=None), 1), (dict(sx=None), 1), (dict(wq=None), 1), (dict(gamma=None), 1), (dict(Y=None), 1),
    (dict(T=0), 1), (dict(T=1 << 31), 2), (dict(N=40), 2), (dict(K=48), 2), (dict(K=1 << 17), 2), (dict(dt=2), 1),
    (dict(Y=ODD), 3), (dict(acc=ODD), 3), (dict(xq=ODD), 3)])
def test_linear_int8(L, kw, status):
    a = dict(xq=FAKE, sx=FAKE, T=4, K=64, wq=FAKE, gamma=FAKE, N=32, Y=FAKE, dt=1, acc=None, st=None)
    assert _lib.status("bitlinear_linear_int8", *dict(a, **kw).values()) == status
    assert len(_lib.last_error()) > 0
