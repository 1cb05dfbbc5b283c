"""CPU tests of the low-bit input gradients' entry points: workspace and host-only refusals."""
from gemm_qmm_nbits_amd import qmm as Q

FAKE = 0x1000


def nbits(**kw):
    a = dict(dY=FAKE, dyt=Q.QMM_BF16, M=100, K=256, N=48, W=FAKE, bits=4, block=64, scales=FAKE, zp=FAKE,
             zk=Q.QMM_ZP_PACKED, dX=FAKE, dxt=Q.QMM_BF16, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return Q.lib().qmm_validate_nbits_dgrad(*a.values())


def codebook(**kw):
    a = dict(dY=FAKE, dyt=Q.QMM_BF16, M=100, K=256, N=48, W=FAKE, block=64, absmax=FAKE, cb=FAKE, dX=FAKE,
             dxt=Q.QMM_BF16, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return Q.lib().qmm_validate_codebook4_dgrad(*a.values())


def test_common_refusals():
    for f in (nbits, codebook):
        assert f() == 0
        assert f(dyt=9) == -2 and f(dxt=-1) == -2
        assert f(dyt=Q.QMM_F32) == 0 and f(dxt=Q.QMM_F32) == 0
        for b in (8, 48, 512, 0, -64):
            assert f(block=b) == -4
        for b in (16, 32, 128, 256):
            assert f(block=b) == 0
        for k in ("M", "K", "N"):
            assert f(**{k: -1}) == -5
        assert f(K=0) == -5 and f(N=0) == -5
        assert f(K=(1 << 20) + 1) == -5 and f(N=(1 << 20) + 1) == -5 and f(M=(1 << 24) + 1) == -5
        assert f(dY=None) == -1 and f(W=None) == -1 and f(dX=None) == -1
        assert f(W=FAKE + 2) == -6 and f(dY=FAKE + 1) == -6 and f(dX=FAKE + 2, dxt=Q.QMM_F32) == -6
        assert f(dY=FAKE + 2) == 0
        assert f(M=0, dY=None, W=None, dX=None, ws=None, wsb=0) == 0
        assert f(ws=None) == -7 and f(wsb=100) == -7 and f(ws=FAKE + 128) == -6
        need = Q.lib().qmm_dgrad_workspace_bytes(100, 256, 48)
        assert f(wsb=need) == 0 and f(wsb=need - 1) == -7


def test_format_refusals():
    for b in (1, 5, 6, 16):
        assert nbits(bits=b) == -3
    for b in (2, 3, 4, 8):
        assert nbits(bits=b) == 0
    assert nbits(bits=3, block=16) == -4
    assert nbits(zk=9) == -8
    assert nbits(zp=None) == -1 and nbits(zp=None, zk=Q.QMM_ZP_UNIFORM) == 0 and nbits(zp=None, zk=Q.QMM_ZP_NONE) == 0
    assert nbits(scales=None) == -1 and nbits(scales=FAKE + 1) == -6
    assert nbits(zp=FAKE + 1, zk=Q.QMM_ZP_F16) == -6 and nbits(zp=FAKE + 1) == 0
    assert codebook(absmax=None) == -1 and codebook(cb=None) == -1 and codebook(absmax=FAKE + 2) == -6


def test_workspace():
    """fp16 rows of N rounded up to 64 and the row scales at least; none for refused sizes."""
    q = Q.lib().qmm_dgrad_workspace_bytes
    assert q(0, 256, 48) == 0 and q(4, 0, 48) == 0 and q(-1, 256, 48) == 0
    for M, K, N in ((1, 256, 48), (2048, 5120, 7680), (16, 4096, 14336), (300, 77, 51)):
        a16 = -(-M * (-(-N // 64) * 64) * 2 // 256) * 256
        rs = -(-M * 4 // 256) * 256
        extra = q(M, K, N) - a16 - rs
        assert extra >= 0 and extra % (M * K * 4) == 0        # whole partial sums


def test_binding_refuses_short_or_wrong_side_tensors():
    """A scale, zero-point or codebook tensor of too few bytes (fewer elements, or smaller ones)."""
    import pytest
    import torch

    ok = torch.zeros(16, dtype=torch.float32)
    assert Q._sized(ok, "codebook", 16, 4, -1) == ok.data_ptr()
    with pytest.raises(TypeError):
        Q._sized(ok.half(), "codebook", 16, 4, -1)
    with pytest.raises(ValueError):
        Q._sized(ok[:15], "codebook", 16, 4, -1)
    with pytest.raises(ValueError):
        Q._sized(ok, "codebook", 16, 4, 0)             # host memory for a device call
    with pytest.raises(ValueError):
        Q._sized(torch.zeros(32)[::2], "codebook", 16, 4, -1)
