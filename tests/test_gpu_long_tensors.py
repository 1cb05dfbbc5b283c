"""GPU: tensors of more than 2^31 elements (or packed bytes) of the adapters, the low-bit input
gradient and the 16-bit expert products: sampled rows and columns, the last ones among them, against
fp64 on the device."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q

from gpu_util import assert_elementwise, gamma, host_f64, say, torch

pytestmark = pytest.mark.gpu

M, WIDE = 70000, 40960          # M * WIDE = 2.87e9


def randn(*shape, seed=0, scale=1.0):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return t.randn(*shape, dtype=t.bfloat16, device="cuda", generator=g).mul_(scale)


def sample(n, k=24):
    """Indices over the whole range, its ends among them, and those around n / 2."""
    t = torch()
    i = np.unique(np.concatenate([np.linspace(0, n - 1, k).astype(np.int64), [n - 2, n // 2, n // 2 + 1]]))
    i = i[(i >= 0) & (i < n)]
    return t.from_numpy(i).cuda()


def product(a, b):
    """a . b and |a| . |b| in fp64."""
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


def close(got, ref, lim, n, out, label):
    say(f"  {label}")
    assert_elementwise(host_f64(got), host_f64(ref), gamma(n) * host_f64(lim), out, label)


def test_grouped_rows():
    """Outputs and output gradients past 2^31 elements."""
    t = torch()
    K, E = 32, 3
    off_h = [0, 30000, 30001, M]
    off = t.tensor(off_h, dtype=t.int32, device="cuda")
    X, W = randn(M, K, seed=1), randn(E, WIDE, K, seed=2)
    rows = sample(M)
    expert = t.bucketize(rows, t.tensor(off_h[1:], device="cuda"), right=True)
    Y = Q.qmoe_grouped_mm(X, off, W)
    for r, e in zip(rows.tolist(), expert.tolist()):
        ref, lim = product(X[r:r + 1], W[e].t())
        close(Y[r:r + 1], ref, lim, K + 4, "bf16", f"Y row {r}")
    del Y
    dY = randn(M, WIDE, seed=3)
    dX, dW, db = Q.qmoe_grouped_mm_grad(dY, X, off, W, dw_dtype=t.float32, need_dbias=True)
    for r, e in zip(rows.tolist(), expert.tolist()):
        ref, lim = product(dY[r:r + 1], W[e])
        close(dX[r:r + 1], ref, lim, WIDE + 4, "bf16", f"dX row {r}")
    cols = sample(WIDE, 8)
    for e in range(E):
        part = dY[off_h[e]:off_h[e + 1]][:, cols]
        x = X[off_h[e]:off_h[e + 1]]
        ref, lim = product(part.t(), x)
        close(dW[e][cols], ref, lim, M + 4, "f32", f"dW {e}")
        close(db[e][cols], part.double().sum(0), part.double().abs().sum(0), M + 36, "f32", f"dbias {e}")


def test_grouped_weights():
    """Weights and weight gradients past 2^31 elements, two rows per expert."""
    t = torch()
    E, N, K = 70, 8192, 4096
    off = t.arange(E + 1, dtype=t.int32, device="cuda") * 2
    X, W, dY = randn(2 * E, K, seed=4), randn(E, N, K, seed=5), randn(2 * E, N, seed=6)
    Y = Q.qmoe_grouped_mm(X, off, W)
    dX, dW, _ = Q.qmoe_grouped_mm_grad(dY, X, off, W)
    for e in (0, 35, 63, 64, 69):
        x, g = X[2 * e:2 * e + 2], dY[2 * e:2 * e + 2]
        close(Y[2 * e:2 * e + 2], *product(x, W[e].t()), K + 4, "bf16", f"Y {e}")
        close(dX[2 * e:2 * e + 2], *product(g, W[e]), N + 4, "bf16", f"dX {e}")
        cols = sample(N, 64)
        close(dW[e][cols], *product(g[:, cols].t(), x), 6, "bf16", f"dW {e}")


@pytest.mark.parametrize("K,N", [(64, WIDE), (WIDE, 64)])
def test_adapters(K, N):
    """lora_add in place on a base, then the gradients; either side past 2^31 elements."""
    t = torch()
    r, L = 8, 3
    g = t.Generator(device="cuda").manual_seed(7)
    ids = t.randint(-1, L, (M,), dtype=t.int32, device="cuda", generator=g)
    X, A, B = randn(M, K, seed=8), randn(L, r, K, seed=9, scale=0.125), randn(L, N, r, seed=10)
    rows = sample(M)
    Y = randn(M, N, seed=11)
    base = Y[rows].clone()
    T = t.empty(M, r, device="cuda")
    Q.qmm_lora_add(X, A, B, ids, base=Y, out=Y, T=T)
    for i, (m, a) in enumerate(zip(rows.tolist(), ids[rows].tolist())):
        b = base[i:i + 1].double()
        if a < 0:
            assert bool((Y[m] == base[i]).all()) and not bool(T[m].any())
            continue
        tr, tl = product(X[m:m + 1], A[a].t())
        close(T[m:m + 1], tr, tl, K + 8, "f32", f"T row {m}")
        ref = tr @ B[a].double().t() + b
        lim = tl @ B[a].double().abs().t() + b.abs()
        close(Y[m:m + 1], ref, lim, K + r + 60, "bf16", f"Y row {m}")
    dY = Y                                       # any values do
    dX, dA, dB = Q.qmm_lora_grad(dY, X, A, B, ids, T=T)
    for m, a in zip(rows.tolist(), ids[rows].tolist()):
        if a < 0:
            assert not bool(dX[m].any())
            continue
        d, dl = product(dY[m:m + 1], B[a])
        close(dX[m:m + 1], d @ A[a].double(), dl @ A[a].double().abs(), N + r + 60, "bf16", f"dX row {m}")
    cols, kcols = sample(N, 8), sample(K, 8)
    for a in range(L):
        mine = (ids == a).nonzero()[:, 0]
        close(dB[a][cols], *product(dY[mine][:, cols].t(), T[mine]), M + 60, "f32", f"dB {a}")
        d = t.zeros(mine.numel(), r, dtype=t.float64, device="cuda")
        dl = t.zeros_like(d)
        for c in range(0, N, 4096):              # (in pieces: fp64 of a whole side would be 20 GB)
            part = dY[:, c:c + 4096][mine].double()
            d += part @ B[a][c:c + 4096].double()
            dl += part.abs() @ B[a][c:c + 4096].double().abs()
        x = X[:, kcols][mine].double()
        close(dA[a][:, kcols], d.t() @ x, dl.t() @ x.abs(), M + N + 60, "f32", f"dA {a}")


@pytest.mark.parametrize("m,K,N", [(M, WIDE, 64), (2, 8192, 600000)])
def test_dgrad(m, K, N):
    """Outputs past 2^31 elements, and packed 4-bit weights past 2^31 bytes.  dY is fp16 (read in
    place); weights (q - 8) * scale rounded to fp16, as the forward matrix-core paths round them."""
    t = torch()
    block = 64
    g = t.Generator(device="cuda").manual_seed(12)
    W = t.randint(0, 256, (N, K // block, block // 2), dtype=t.uint8, device="cuda", generator=g)
    scales = (t.rand(N, K // block, device="cuda", generator=g) * 0.01 + 0.001).half()
    dY = randn(m, N, seed=13).half()
    dX = Q.qmm_nbits_dgrad(dY, W, scales, K, 4, block)
    cols = sample(K, 16)
    byte = W.view(N, K // 2)[:, cols // 2].int()
    q = t.where(cols % 2 == 0, byte & 15, byte >> 4)
    w = ((q - 8).float() * scales[:, cols // block].float()).half()
    rows = sample(m)
    close(dX[rows][:, cols], *product(dY[rows], w), N + 70, "f16", f"dX {m} {K} {N}")
