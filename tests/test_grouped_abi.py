"""CPU tests of the ragged 16-bit products' entry points: host-only refusals."""
from gemm_qmm_nbits_amd import qmm as Q

FAKE = 0x1000


def mm(**kw):
    a = dict(X=FAKE, type=Q.QMM_BF16, R=100, K=64, N=48, E=3, off=FAKE, W=FAKE, bias=None, Y=FAKE, yt=Q.QMM_BF16)
    a.update(kw)
    return Q.lib().qmm_validate_grouped_mm(*a.values())


def grad(**kw):
    a = dict(dY=FAKE, X=FAKE, type=Q.QMM_F16, R=100, K=64, N=48, E=3, off=FAKE, W=FAKE, dX=FAKE, dxt=Q.QMM_F16,
             dW=FAKE, db=FAKE, dwt=Q.QMM_F32)
    a.update(kw)
    return Q.lib().qmm_validate_grouped_mm_grad(*a.values())


def test_common_refusals():
    for f in (mm, grad):
        assert f() == 0
        assert f(type=Q.QMM_F32) == -2 and f(type=9) == -2
        for k in ("R", "K", "N", "E"):
            assert f(**{k: -1}) == -5
        for k in ("K", "N", "E"):
            assert f(**{k: 0}) == -5
        assert f(R=(1 << 24) + 1) == -5 and f(K=(1 << 20) + 1) == -5 and f(N=(1 << 20) + 1) == -5
        assert f(E=65536) == -5
        assert f(E=65535, K=1 << 20, N=1 << 20) == -5      # more tiles than one launch has
        assert f(off=None) == -1 and f(off=FAKE + 2) == -6
        assert f(X=FAKE + 1) == -6 and f(W=FAKE + 1) == -6
        assert f(X=FAKE + 2) == 0


def test_mm_refusals():
    assert mm(yt=3) == -2
    assert mm(X=None) == -1 and mm(W=None) == -1 and mm(Y=None) == -1
    assert mm(Y=FAKE + 2, yt=Q.QMM_F32) == -6 and mm(bias=FAKE + 2, yt=Q.QMM_F32) == -6
    assert mm(R=0, X=None, off=None, W=None, Y=None) == 0


def test_grad_refusals():
    assert grad(dxt=3) == -2 and grad(dwt=-1) == -2
    assert grad(dX=None, dxt=3) == 0 and grad(dW=None, db=None, dwt=-1) == 0
    assert grad(dY=None) == -1
    assert grad(W=None) == -1 and grad(W=None, dX=None) == 0
    assert grad(X=None) == -1 and grad(X=None, dW=None) == 0
    assert grad(dW=FAKE + 2) == -6 and grad(db=FAKE + 2) == -6 and grad(dX=FAKE + 2) == 0
    assert grad(dX=None, dW=None, db=None, dY=None, off=None) == 0
    assert grad(R=0, dY=None, X=None, W=None) == 0         # dW is still written (zeros)
    assert grad(R=0, dY=None, X=None, W=None, off=None) == -1
    assert grad(R=0, dY=None, X=None, W=None, off=None, dW=None, db=None) == 0
