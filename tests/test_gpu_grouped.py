"""GPU parity of the ragged 16-bit expert products (qmoe_grouped_mm and its gradients) against
the fp64 oracle."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q
from oracle import adapters_oracle as AO

from gpu_util import assert_elementwise, dev, gamma, host_bits, host_f64, say, torch

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def tt(name):
    return getattr(torch(), DT[name])


class Problem:
    def __init__(self, counts, K, N, ty, seed, extra=0, offset=0, out="f32"):
        """counts: rows of each expert; `extra` rows behind the last expert's."""
        t = torch()
        rng = np.random.default_rng(seed)
        self.E, self.K, self.N, self.ty = len(counts), K, N, ty
        self.off_h = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.R = int(self.off_h[-1]) + extra

        def put(x, dtype):
            flat = t.zeros(x.size + offset, dtype=dtype, device="cuda")
            v = flat[offset:].view(x.shape)
            v.copy_(t.from_numpy(x))
            return v

        self.X = put(rng.standard_normal((self.R, K)), tt(ty))
        self.dY = put(rng.standard_normal((self.R, N)) * 0.1, tt(ty))
        self.W = put(rng.standard_normal((self.E, N, K)) / np.sqrt(K), tt(ty))
        self.bias = put(rng.standard_normal((self.E, N)), tt(out))
        self.offsets = dev(self.off_h)


def check(p, out, dx, dw, label=""):
    """Forward with and without bias, then all three gradients."""
    t = torch()
    say(f"  {label} rows={np.diff(p.off_h).tolist()[:12]} K={p.K} N={p.N} {p.ty} -> {out} {dx} {dw}")
    X, W, dY, b = host_f64(p.X), host_f64(p.W), host_f64(p.dY), host_f64(p.bias.to(tt(out)))
    owned = int(p.off_h[-1])
    lim = AO.grouped_mm(np.abs(X), p.off_h, np.abs(W), np.abs(b))
    for bias in (None, p.bias.to(tt(out))):
        y = t.full((p.R, p.N), 7.0, dtype=tt(out), device="cuda")
        Q.qmoe_grouped_mm(p.X, p.offsets, p.W, bias=bias, out=y)
        ref = AO.grouped_mm(X, p.off_h, W, None if bias is None else b)
        assert_elementwise(host_f64(y)[:owned], ref[:owned], gamma(p.K + 4) * lim[:owned], out, label + " Y")
        assert bool((y[owned:] == 7.0).all())          # rows of no expert stay
    dXt = t.full((p.R, p.K), 7.0, dtype=tt(dx), device="cuda")
    dX, dW, db = Q.qmoe_grouped_mm_grad(p.dY, p.X, p.offsets, p.W, dX=dXt, dw_dtype=tt(dw), need_dbias=True)
    ref = AO.grouped_mm_grad(dY, X, p.off_h, W)
    lim = AO.grouped_mm_grad(np.abs(dY), np.abs(X), p.off_h, np.abs(W))
    assert_elementwise(host_f64(dX)[:owned], ref[0][:owned], gamma(p.N + 4) * lim[0][:owned], dx, label + " dX")
    assert bool((dX[owned:] == 7.0).all())
    assert_elementwise(host_f64(dW), ref[1], gamma(p.R + 4) * lim[1], dw, label + " dW")
    assert_elementwise(host_f64(db), ref[2], gamma(p.R + 36) * lim[2], dw, label + " dbias")
    empty = np.diff(p.off_h) == 0
    assert not host_f64(dW)[empty].any() and not host_f64(db)[empty].any()


# rows of each expert, K, N: a single row; empty experts first, last and between; tile borders of
# every tile height (64, 128, 256 rows) and one off them; contraction and output sizes on, below
# and past the stages (32) and tiles; sizes that are no multiple of 8 (the element loads)
SHAPES = [
    ([1], 32, 32), ([1], 1, 1), ([0, 1, 0], 40, 24), ([0, 0, 0], 64, 64), ([2, 3, 1, 0, 5], 72, 136),
    ([64], 128, 128), ([65, 63], 96, 129), ([3, 0, 70, 1], 77, 51), ([128, 127, 129], 160, 264),
    ([256], 256, 256), ([257, 255], 104, 520), ([300, 0, 700], 200, 272), ([600], 33, 300), ([1000], 520, 1),
    ([1] * 70 + [0] * 5 + [9], 64, 40),
]


@pytest.mark.parametrize("counts,K,N", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_shapes(counts, K, N, ty):
    check(Problem(counts, K, N, ty, seed=K + N, extra=3, out=ty), ty, ty, "f32")


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [20, 150, 400])
def test_types(out, ty, rows):
    check(Problem([rows, 0, rows + 7], 136, 88, ty, seed=5, out=out), out, out, out)


@pytest.mark.parametrize("rows", [20, 150, 400])
def test_misaligned(rows):
    """Tensors one element past an aligned address: the element loads."""
    p = Problem([rows, 5], 136, 88, "bf16", seed=7, offset=1, out="bf16")
    assert p.X.data_ptr() % 16 != 0
    check(p, "bf16", "bf16", "f32")


# every tile height of the rule on the rows and tiles: 64 (few tiles, or few rows), 128 x 128, 128 x
# 256 and 256 x 256, whole and with a few rows over
@pytest.mark.parametrize("counts,K,N", [([17] * 32, 2880, 5760), ([200, 10, 0, 500], 2048, 1536), ([800], 2600, 2608),
                                        ([60] * 24, 1032, 1544), ([1030, 3, 517, 900], 2904, 3000), ([800], 2601, 2603),
                                        ([60] * 24, 1033, 1545), ([1500, 1, 900], 2901, 3001)])
def test_layer_sizes(counts, K, N):
    """The expert layers' own sizes, a few rows per expert and skewed ones."""
    check(Problem(counts, K, N, "bf16", seed=11, out="bf16"), "bf16", "bf16", "bf16")


@pytest.mark.parametrize("rows", [10, 150, 400])
def test_neighbours_do_not_leak(rows):
    """NaN and inf in one expert's rows, in its weights and in the rows of no expert reach no other
    expert's results."""
    t = torch()
    p = Problem([rows, rows + 3, rows + 1], 72, 104, "f16", seed=13, extra=40, out="f16")
    clean = [host_bits(Q.qmoe_grouped_mm(p.X, p.offsets, p.W)).copy()]
    clean += [host_bits(v).copy() for v in Q.qmoe_grouped_mm_grad(p.dY, p.X, p.offsets, p.W, need_dbias=True)]
    a, b, c = (int(v) for v in p.off_h[1:])
    for v in (p.X, p.dY):
        v[a:b] = float("nan")
        v[c:] = float("inf")
    p.W[1] = float("inf")
    got = [host_bits(Q.qmoe_grouped_mm(p.X, p.offsets, p.W))]
    got += [host_bits(v) for v in Q.qmoe_grouped_mm_grad(p.dY, p.X, p.offsets, p.W, need_dbias=True)]
    for i in (0, 1):
        assert np.array_equal(got[i][:a], clean[i][:a]) and np.array_equal(got[i][b:c], clean[i][b:c])
    for i in (2, 3):
        assert np.array_equal(got[i][[0, 2]], clean[i][[0, 2]])
    t.cuda.synchronize()


def test_offsets_out_of_range_are_clamped():
    """Offsets below 0 and past R: the rows inside are computed, nothing outside is touched."""
    t = torch()
    p = Problem([30, 20], 64, 48, "bf16", seed=17, out="bf16")
    want = host_bits(Q.qmoe_grouped_mm(p.X, p.offsets, p.W)).copy()
    wild = dev(np.array([-5, 30, 1 << 30], np.int32))
    assert np.array_equal(host_bits(Q.qmoe_grouped_mm(p.X, wild, p.W)), want)
    dW = Q.qmoe_grouped_mm_grad(p.dY, p.X, p.offsets, p.W)[1]
    dW2 = Q.qmoe_grouped_mm_grad(p.dY, p.X, wild, p.W)[1]
    assert np.array_equal(host_bits(dW), host_bits(dW2))
    backwards = dev(np.array([0, 40, 20], np.int32))       # expert 1 ends before it begins: empty
    _, dW3, db3 = Q.qmoe_grouped_mm_grad(p.dY, p.X, backwards, p.W, need_dbias=True)
    assert not bool(dW3[1].any()) and not bool(db3[1].any())
    t.cuda.synchronize()


def test_no_rows():
    t = torch()
    p = Problem([0, 0], 64, 48, "f16", seed=19, out="f16")
    assert Q.qmoe_grouped_mm(p.X, p.offsets, p.W).shape == (0, 48)
    dW = t.full((2, 48, 64), 3.0, dtype=t.float32, device="cuda")
    db = t.full((2, 48), 3.0, dtype=t.float32, device="cuda")
    dX, dW, db = Q.qmoe_grouped_mm_grad(p.dY, p.X, p.offsets, p.W, dW=dW, dbias=db)
    assert dX.shape == (0, 64) and not bool(dW.any()) and not bool(db.any())


def test_training_step_repeats_and_graph():
    """Router offsets -> forward -> gradients, as a layer runs: repeated, on another stream, and
    captured with the offsets and inputs changed between replays."""
    t = torch()
    p = Problem([100, 0, 37, 163], 136, 200, "bf16", seed=23, out="bf16")

    def step(o):
        Q.qmoe_grouped_mm(p.X, p.offsets, p.W, bias=p.bias, out=o[0])
        Q.qmoe_grouped_mm_grad(o[0], p.X, p.offsets, p.W, dX=o[1], dW=o[2], dbias=o[3])
        return o

    def outs():
        return [t.empty(p.R, 200, dtype=t.bfloat16, device="cuda"), t.empty(p.R, 136, dtype=t.bfloat16, device="cuda"),
                t.empty(4, 200, 136, device="cuda"), t.empty(4, 200, device="cuda")]

    ref = [host_bits(v).copy() for v in step(outs())]
    for _ in range(4):
        for v, want in zip(step(outs()), ref):
            assert np.array_equal(host_bits(v), want)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        o = step(outs())
    side.synchronize()
    for v, want in zip(o, ref):
        assert np.array_equal(host_bits(v), want)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step(o)
    x0 = p.X.clone()
    for k, offs in enumerate(([0, 100, 100, 137, 300], [0, 0, 300, 300, 300], [0, 1, 2, 3, 300], [0, 100, 100, 137, 300])):
        p.X.copy_(x0 * (k + 1))
        p.offsets.copy_(dev(np.array(offs, np.int32)))
        g.replay()
        t.cuda.synchronize()
        got = [host_bits(v).copy() for v in o]
        for v, want in zip(got, step(outs())):
            assert np.array_equal(v, host_bits(want)), k


def test_refusals():
    t = torch()
    p = Problem([4, 4], 64, 32, "f16", seed=29, out="f16")
    with pytest.raises(TypeError):
        Q.qmoe_grouped_mm(p.X.float(), p.offsets, p.W)
    with pytest.raises(TypeError):
        Q.qmoe_grouped_mm(p.X, p.offsets, p.W.bfloat16())
    with pytest.raises(ValueError):
        Q.qmoe_grouped_mm(p.X, p.offsets[:-1], p.W)
    with pytest.raises(ValueError):
        Q.qmoe_grouped_mm(p.X[:, :63], p.offsets, p.W)
    with pytest.raises(TypeError):
        Q.qmoe_grouped_mm(p.X, p.offsets, p.W, bias=p.bias, out_dtype=t.float32)
    with pytest.raises(ValueError):
        Q.qmoe_grouped_mm_grad(p.dY[:4], p.X, p.offsets, p.W)
