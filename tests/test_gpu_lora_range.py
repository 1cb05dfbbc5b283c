"""GPU: adapters whose ranks differ by many powers of two, and infinities in weights, rows and t, against
the formula in fp64."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q
from oracle import adapters_oracle as AO

from gpu_util import assert_elementwise, dev, gamma, host_bits, host_f64, say, torch

pytestmark = pytest.mark.gpu

DT = {"f16": "float16", "bf16": "bfloat16"}


def put(x, ty):
    t = torch()
    return t.from_numpy(np.ascontiguousarray(x)).to(getattr(t, DT[ty])).cuda()


def graded(rows, wide, r, L, seed):
    """Rows v [rows, wide] and weights w [L, r, wide] whose products of rank j lie near 2^(19 - 42 j / r):
    rank j reads column j alone."""
    rng = np.random.default_rng(seed)
    grade = -np.arange(r) / max(1, r - 1)
    v = np.zeros((rows, wide))
    v[:, :r] = rng.uniform(1, 2, (rows, r)) * 2.0 ** (13 + 27 * grade)
    w = np.zeros((L, r, wide))
    w[:, np.arange(r), np.arange(r)] = rng.uniform(1, 2, (L, r)) * 2.0 ** (5 + 14 * grade)
    return v, w


def stepped(wide, r, L, seed):
    """Weights [L, wide, r] that are zero for the ranks below column % r: each rank leads some columns."""
    w = np.random.default_rng(seed).uniform(0.5, 1, (L, wide, r)) * np.sign(np.random.default_rng(seed + 1).standard_normal((L, wide, r)))
    return w * (np.arange(r)[None, :] >= (np.arange(wide) % r)[:, None])


# few rows in one tile, in 16-row parts, sorted rows; ranks of every piece layout (8, 16, 32, 64, more);
# an output below 64 columns
@pytest.mark.parametrize("M,r,wide", [(1, 8, 130), (9, 2, 256), (40, 12, 192), (200, 8, 130), (200, 24, 256), (9, 30, 100),
                                      (50, 48, 192), (300, 64, 200), (90, 100, 320), (30, 130, 256), (40, 8, 40)])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_small_ranks_beside_large_ones(M, r, wide, ty):
    t = torch()
    L, other = 3, 160
    ids_h = np.random.default_rng(M).integers(-1, L, M).astype(np.int32)
    ids = dev(ids_h)
    # forward: graded T, stepped B
    v, w = graded(M, other, r, L, seed=M + r)
    X, A, B = put(v, ty), put(w, ty), put(stepped(wide, r, L, seed=r), ty)
    say(f"  M={M} r={r} {wide} {ty}")
    y = Q.qmm_lora_add(X, A, B, ids, out_dtype=t.float32)
    x, a, b = host_f64(X), host_f64(A), host_f64(B)
    assert_elementwise(host_f64(y), AO.lora_add(x, a, b, ids_h),
                       gamma(other + r + 40) * AO.lora_add(np.abs(x), np.abs(a), np.abs(b), ids_h), "f32", "Y")
    # gradient: graded dT (dY B), stepped A
    dY, B = X, put(np.swapaxes(w, 1, 2), ty)
    A = put(np.swapaxes(stepped(wide, r, L, seed=r + 7), 1, 2), ty)
    X = put(np.random.default_rng(3).standard_normal((M, wide)), ty)
    dX, _, _ = Q.qmm_lora_grad(dY, X, A, B, ids, dx_dtype=t.float32, need=(True, False, False))
    g, x, a, b = host_f64(dY), host_f64(X), host_f64(A), host_f64(B)
    assert_elementwise(host_f64(dX), AO.lora_grad(g, x, a, b, ids_h)[0],
                       gamma(other + r + 60) * AO.lora_grad(np.abs(g), np.abs(x), np.abs(a), np.abs(b), ids_h)[0],
                       "f32", "dX")


def formula(tv, B, ids, base):
    """base + t B_a^T in fp64 with its infinities and NaN; tv: t after the scale, as fp32 holds it."""
    out = base.copy()
    with np.errstate(invalid="ignore"):
        for m, a in enumerate(ids):
            if 0 <= a < B.shape[0]:
                out[m] += (tv[m][None, :] * B[a]).sum(1)
    return out


def same(got, want, label):
    assert np.array_equal(np.isnan(got), np.isnan(want)), label + ": NaN"
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf]), label + ": infinities"


@pytest.mark.parametrize("M,N,r", [(7, 128, 8), (7, 130, 16), (40, 192, 32), (200, 128, 8), (200, 130, 12), (300, 256, 64),
                                   (90, 128, 100), (20, 40, 8)])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_infinite_weights(M, N, r, ty):
    """An infinite element of B (or A in the gradient) gives its column infinities of t's sign, in the
    rows of its adapter only, also where t has few bits (1, 0.5: its later pieces are empty)."""
    t = torch()
    L, K = 3, 96
    ids_h = (np.arange(M) % (L + 1)).astype(np.int32)          # one group without an adapter
    rng = np.random.default_rng(r)
    x = np.zeros((M, K))
    x[:, :r % K or K] = rng.choice([1.0, -0.5, 3.0], (M, r % K or K))
    a = np.zeros((L, r, K))
    a[:, np.arange(r), np.arange(r) % K] = 1.0                  # t are sums of few such values
    b = rng.choice([0.25, -1.5, 2.0], (L, N, r))
    b[1, 5, r - 1] = np.inf
    b[1, N - 1, 0] = -np.inf
    X, A, B, ids, base = put(x, ty), put(a, ty), put(b, ty), dev(ids_h), t.ones(M, N, device="cuda")
    y = Q.qmm_lora_add(X, A, B, ids, base=base, out_dtype=t.float32)
    T = AO.lora_t(x, a, ids_h)
    want = formula(T, b, ids_h, np.ones((M, N)))
    assert np.isinf(want).any()
    same(host_f64(y), want, "Y")
    # the gradient of the mirrored problem: dT = dY B with B = a^T, dX = dT A with A = b^T
    dY, Bt, At = X, put(np.swapaxes(a, 1, 2), ty), put(np.swapaxes(b, 1, 2), ty)
    dX, _, _ = Q.qmm_lora_grad(dY, t.zeros(M, N, dtype=X.dtype, device="cuda"), At, Bt, ids, base=base,
                               dx_dtype=t.float32, need=(True, False, False))
    same(host_f64(dX), want, "dX")


@pytest.mark.parametrize("M,N", [(6, 128), (30, 192), (200, 130), (6, 40)])
@pytest.mark.parametrize("r", [8, 16, 40])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_infinite_t(M, N, r, ty):
    """One rank of t overflows (scale 3e38): the others, far beyond fp16's range, stay finite, so a column
    is infinite with its own sign, or NaN where its weight is zero; rows of other adapters keep their
    bits."""
    t = torch()
    L, K = 2, 64
    ids_h = (np.arange(M) % L).astype(np.int32)
    rng = np.random.default_rng(r)
    x = np.zeros((M, K))
    x[:, 0], x[:, 1:r] = 2.0, 0.0625
    a = np.zeros((L, r, K))
    a[:, np.arange(r), np.arange(r)] = 1.0
    b = rng.choice([-1.0, 0.5, 0.0], (L, N, r))
    X, A, B, ids = put(x, ty), put(a, ty), put(b, ty), dev(ids_h)
    scale = np.array([3e38, 2.0], np.float32)
    y = Q.qmm_lora_add(X, A, B, ids, scale=dev(scale), out_dtype=t.float32)
    with np.errstate(over="ignore"):
        tv = (x[:, :r] * scale.astype(np.float64)[ids_h][:, None]).astype(np.float32).astype(np.float64)
    tv[np.abs(tv) > 3.4028236e38] = np.inf
    want = formula(tv, b, ids_h, np.zeros((M, N)))
    assert np.isinf(tv[0, 0]) and np.isfinite(tv[0, 1]) and tv[0, 1] > 65504
    # sums of the finite ranks may themselves pass the fp32 range: compared where rank 0 decides
    same(host_f64(y)[ids_h == 0], want[ids_h == 0], "Y")
    clean = Q.qmm_lora_add(X, A, B, ids, scale=dev(np.array([1.0, 2.0], np.float32)), out_dtype=t.float32)
    assert np.array_equal(host_bits(y)[ids_h == 1], host_bits(clean)[ids_h == 1])
