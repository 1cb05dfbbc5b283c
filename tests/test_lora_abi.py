"""CPU tests of the adapters' entry points: workspace sizes and host-only refusals."""
import pytest

from gemm_qmm_nbits_amd import qmm as Q

FAKE = 0x1000  # aligned, never dereferenced by the validators


def w(A=FAKE, B=FAKE, scale=FAKE):
    return Q.qmm_lora_weights(A, B, scale)


def add(**kw):
    a = dict(X=FAKE, type=Q.QMM_BF16, M=100, K=64, N=48, r=8, L=3, ids=FAKE, w=w(), base=FAKE, bt=Q.QMM_F32, Y=FAKE,
             yt=Q.QMM_BF16, T=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return Q.lib().qmm_validate_lora_add(*a.values())


def grad(**kw):
    a = dict(dY=FAKE, X=FAKE, type=Q.QMM_F16, M=100, K=64, N=48, r=8, L=3, ids=FAKE, w=w(), T=FAKE, base=None, bt=9,
             dX=FAKE, dxt=Q.QMM_F16, dA=FAKE, dB=FAKE, gt=Q.QMM_F32, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return Q.lib().qmm_validate_lora_grad(*a.values())


@pytest.mark.parametrize("f", [add, grad])
def test_common_refusals(f):
    assert f() == 0
    assert f(type=Q.QMM_F32) == -2 and f(type=7) == -2
    for k in ("M", "K", "N", "r", "L"):
        assert f(**{k: -1}) == -5
    for k in ("K", "N", "r", "L"):
        assert f(**{k: 0}) == -5
    assert f(M=(1 << 24) + 1) == -5 and f(K=(1 << 21) + 1) == -5 and f(N=(1 << 21) + 1) == -5 and f(r=513) == -5 and f(L=32769) == -5
    assert f(ids=None) == -1
    assert f(ids=FAKE + 2) == -6
    assert f(w=w(B=None)) == -1
    assert f(w=w(A=FAKE + 1)) == -6 and f(w=w(scale=FAKE + 2)) == -6
    assert f(w=w(scale=None)) == 0
    assert f(ws=None) == -7 and f(wsb=10) == -7
    assert f(ws=FAKE + 128) == -6
    assert f(base=FAKE, bt=5) == -2
    assert f(base=FAKE + 2, bt=Q.QMM_F32) == -6 and f(base=FAKE + 2, bt=Q.QMM_F16) == 0


def test_add_refusals():
    assert add(yt=4) == -2
    assert add(base=None, bt=77) == 0                     # no base: its type is not read
    assert add(X=None) == -1 and add(Y=None) == -1 and add(w=w(A=None)) == -1
    assert add(Y=FAKE + 2, yt=Q.QMM_F32) == -6 and add(Y=FAKE + 2) == 0 and add(X=FAKE + 1) == -6
    assert add(T=FAKE + 2) == -6
    assert add(M=0, X=None, ids=None, Y=None, ws=None, wsb=0) == 0
    need = Q.lib().qmm_lora_add_workspace_bytes(100, 64, 48, 8, 3)
    assert need > 0 and add(wsb=need) == 0 and add(wsb=need - 1) == -7


def test_grad_refusals():
    assert grad(dxt=4) == -2 and grad(gt=-1) == -2
    assert grad(dX=None, dxt=4) == 0                      # not wanted: its type is not read
    assert grad(dA=None, dB=None, gt=-1) == 0
    assert grad(dY=None) == -1
    assert grad(X=None) == -1                             # dA reads X
    assert grad(X=None, dA=None) == 0                     # T is given
    assert grad(X=None, dA=None, T=None) == -1            # T has to be computed again
    assert grad(w=w(A=None)) == -1 and grad(w=w(A=None), dX=None) == 0
    # no rows: dA and dB are still written (zeros), so the workspace is needed
    assert grad(M=0, dY=None, X=None, ids=None) == 0
    assert grad(M=0, dY=None, X=None, ids=None, ws=None) == -7
    assert grad(M=0, dY=None, X=None, ids=None, dA=None, dB=None, ws=None) == 0
    need = Q.lib().qmm_lora_grad_workspace_bytes(100, 64, 48, 8, 3)
    assert need > 0 and grad(wsb=need) == 0 and grad(wsb=need - 1) == -7


def test_workspace_of_refused_sizes_is_zero():
    L = Q.lib()
    assert L.qmm_lora_add_workspace_bytes(0, 64, 48, 8, 3) == 0
    for bad in ((-1, 64, 48, 8, 3), (4, 0, 48, 8, 3), (4, 64, 48, 0, 3), (4, 64, 48, 8, 0)):
        assert L.qmm_lora_add_workspace_bytes(*bad) == 0
        assert L.qmm_lora_grad_workspace_bytes(*bad) == 0


def test_binding_refuses_wrong_tensors():
    """The binding checks shapes, types and devices before a pointer leaves it."""
    import torch

    X = torch.zeros(4, 16, dtype=torch.float16)
    A, B = torch.zeros(2, 8, 16, dtype=torch.float16), torch.zeros(2, 5, 8, dtype=torch.float16)
    ids = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        Q.qmm_lora_add(X.float(), A, B, ids)
    with pytest.raises(ValueError):
        Q.qmm_lora_add(X, A[0], B, ids)
    if not torch.cuda.is_available():
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            Q.qmm_lora_add(X, A, B, ids)              # host tensors
