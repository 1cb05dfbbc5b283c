"""CPU tests of the entry points of the input gradients with unrounded operands: workspace, host-only
refusals, and the bf16 pieces by which they hold a weight."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q

FAKE = 0x1000


def nbits(**kw):
    a = dict(dY=FAKE, dyt=Q.QMM_BF16, M=100, K=256, N=48, W=FAKE, bits=4, block=64, scales=FAKE, zp=FAKE,
             zk=Q.QMM_ZP_PACKED, dX=FAKE, dxt=Q.QMM_F32, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return Q.lib().qmm_validate_nbits_dgrad_f32(*a.values())


def codebook(**kw):
    a = dict(dY=FAKE, dyt=Q.QMM_BF16, M=100, K=256, N=48, W=FAKE, block=64, absmax=FAKE, cb=FAKE, dX=FAKE,
             dxt=Q.QMM_F32, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return Q.lib().qmm_validate_codebook4_dgrad_f32(*a.values())


def test_refusals():
    for f in (nbits, codebook):
        assert f() == 0
        assert f(dyt=9) == -2 and f(dxt=-1) == -2
        assert f(block=48) == -4 and f(block=512) == -4
        for k in ("M", "K", "N"):
            assert f(**{k: -1}) == -5
        assert f(K=0) == -5 and f(N=0) == -5 and f(K=(1 << 20) + 1) == -5 and f(M=(1 << 24) + 1) == -5
        assert f(dY=None) == -1 and f(W=None) == -1 and f(dX=None) == -1
        assert f(W=FAKE + 2) == -6 and f(dY=FAKE + 1) == -6 and f(dX=FAKE + 2) == -6
        assert f(M=0, dY=None, W=None, dX=None, ws=None, wsb=0) == 0
        assert f(ws=None) == -7 and f(ws=FAKE + 128) == -6
        for ty in (Q.QMM_F32, Q.QMM_F16, Q.QMM_BF16):
            need = Q.lib().qmm_dgrad_f32_workspace_bytes(ty, 100, 256, 48)
            assert f(dyt=ty, wsb=need) == 0 and f(dyt=ty, wsb=need - 1) == -7
    assert nbits(bits=5) == -3 and nbits(bits=3, block=16) == -4 and nbits(zk=9) == -8
    assert nbits(zp=None) == -1 and nbits(scales=None) == -1 and codebook(absmax=None) == -1


def test_workspace():
    """Planes of rows of N rounded up to 64, and whole partial sums behind them."""
    q = Q.lib().qmm_dgrad_f32_workspace_bytes
    assert q(Q.QMM_BF16, 0, 256, 48) == 0 and q(Q.QMM_BF16, 4, 0, 48) == 0 and q(9, 4, 256, 48) == 0
    for M, K, N in ((1, 256, 48), (2048, 5120, 7680), (16, 4096, 14336), (300, 77, 51)):
        for ty, planes in ((Q.QMM_BF16, 1), (Q.QMM_F16, 2), (Q.QMM_F32, 3)):
            rows = -(-M * planes * (-(-N // 64) * 64) * 2 // 256) * 256
            extra = q(ty, M, K, N) - rows
            assert extra >= 0 and extra % (M * K * 4) == 0


def pieces(w, n):
    """The truncations of fp32 values to bf16, as the kernels take them."""
    w = np.asarray(w, np.float32)
    x, out = w.copy(), []
    for _ in range(n):
        top = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.append(top)
        left = (x - top).astype(np.float64)
        x = (w.astype(np.float64) * 2.0 ** -40 + left).astype(np.float32)
    return out


@pytest.mark.parametrize("n,top", [(2, 31), (3, None)])
def test_pieces_hold_the_weights(n, top):
    """Two pieces hold a scale times a difference of 5 bits, three any fp32 value, but for 2^-38; no piece
    of a weight other than 0 is 0, and all have its sign."""
    rng = np.random.default_rng(3)
    if top:
        s = np.exp(rng.uniform(-16, 10, 100000)).astype(np.float16).astype(np.float32)
        w = rng.integers(-top, top + 1, s.size).astype(np.float32) * s
    else:
        w = (rng.standard_normal(100000) * np.exp(rng.uniform(-40, 40, 100000))).astype(np.float32)
    w = w[w != 0]
    p = pieces(w, n)
    total = sum(v.astype(np.float64) for v in p)
    assert np.abs(total / w - 1).max() <= 2.0 ** -38
    for v in p:
        assert v.all() and np.array_equal(np.sign(v), np.sign(w))


@pytest.mark.parametrize("f32", [False, True])
def test_binding_refuses_formats_by_status(f32):
    """The statuses of qmm_nbits for bits and blocks, before any shape is computed from them."""
    import torch

    dY, W = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.uint8)
    s = torch.ones(32 * 16, dtype=torch.float16)
    for block in (0, -64, 8, 48, 512):
        with pytest.raises(Q.QmmError) as e:
            Q.qmm_nbits_dgrad(dY, W, s, 128, 4, block, f32=f32)
        assert e.value.status == -4
        with pytest.raises(Q.QmmError) as e:
            Q.qmm_codebook4_dgrad(dY, W, s.float(), torch.ones(16), 128, block, f32=f32)
        assert e.value.status == -4
    for bits, block, status in ((5, 64, -3), (0, 64, -3), (3, 16, -4)):
        with pytest.raises(Q.QmmError) as e:
            Q.qmm_nbits_dgrad(dY, W, s, 128, bits, block, f32=f32)
        assert e.value.status == status
