"""GPU parity of the input gradients with unrounded operands (f32=True) against the fp64 oracle: the
only roundings are the fp32 sums' and the output's."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import inputs as gen
from gemm_qmm_nbits_amd import qmm as Q
from oracle import adapters_oracle as AO
from oracle import qmm_oracle as O

from gpu_util import (TOL, ZP_KIND, assert_elementwise, dev, dev_act, gamma, host_bits, host_f64, oracle_zp_kind, say,
                      torch)

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}
PLANES = {"bf16": 1, "f16": 2, "f32": 3}


def tt(name):
    return getattr(torch(), DT[name])


def weights(p):
    return O.dequant_nbits(p["W"], p["bits"], p["K"], p["block"], p["scales"], p["zp"],
                           oracle_zp_kind(O, p["zp_mode"])).astype(np.float64)


def compare(y, g, dy_type, w, out, label):
    """g: dY and w: the weights [N, K], in fp64.  A sum has at most planes x 3 products per row of W
    (the planes of dY times the pieces of a weight) and 64 split sums; pieces have the sign of their
    value and add up to it but for 2^-38."""
    N = w.shape[0]
    terms = PLANES[dy_type] * 3 * (N + 64) + 70
    got, ref = host_f64(y), g @ w
    assert_elementwise(got, ref, gamma(terms) * (np.abs(g) @ np.abs(w)), out, label)
    err = O.rel_l2(got, ref)
    say(f"  {label}: relL2 = {err:.2e}")
    assert err <= TOL[out], err


def run(p, dY, out, **kw):
    z = dev(p["zp"]) if p["zp"] is not None else None
    return Q.qmm_nbits_dgrad(dY, dev(p["W"]), dev(p["scales"]), p["K"], p["bits"], p["block"], z,
                             ZP_KIND[p["zp_mode"]], 0.0, out_dtype=tt(out), f32=True, **kw)


def problem(M, K, N, bits, block, zp, dy_type, seed):
    p = gen.nbits_problem(1, K, N, bits, block, seed=seed, zp=zp)
    dY = dev_act(gen.activations(np.random.default_rng(seed + 1), (M, N), dy_type), dy_type)
    return p, dY


# one row, the borders of the tile heights, split and whole contractions, odd sizes (padded planes)
@pytest.mark.parametrize("M,K,N", [(1, 256, 64), (1, 70, 33), (3, 1, 1), (16, 1024, 304), (65, 264, 97), (129, 515, 136),
                                   (300, 1030, 96), (260, 128, 1000)])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_sizes(M, K, N, bits):
    p, dY = problem(M, K, N, bits, 32, "packed", "bf16", seed=M + K + bits)
    compare(run(p, dY, "f32"), host_f64(dY), "bf16", weights(p), "f32", f"M={M} K={K} N={N} u{bits}")


@pytest.mark.parametrize("zp", ["none", "f16"])
@pytest.mark.parametrize("bits,block", [(2, 16), (3, 128), (4, 64), (8, 32)])
@pytest.mark.parametrize("M", [5, 90, 150])
def test_formats(bits, block, zp, M):
    p, dY = problem(M, 300, 120, bits, block, zp, "bf16", seed=100 + bits + block)
    compare(run(p, dY, "f32"), host_f64(dY), "bf16", weights(p), "f32", f"u{bits} block={block} zp={zp} M={M}")


@pytest.mark.parametrize("uniform", [1.5, -0.3, -14.0, 40.0])
@pytest.mark.parametrize("M", [40, 150])
def test_uniform_zero_point(uniform, M):
    """Constants that two pieces hold (halves, q - z within 5 bits) and that they do not."""
    p = gen.nbits_problem(1, 256, 96, 2, 64, seed=7, zp="f16_uniform", uniform_zp=uniform)
    dY = dev_act(gen.activations(np.random.default_rng(8), (M, 96), "bf16"), "bf16")
    y = Q.qmm_nbits_dgrad(dY, dev(p["W"]), dev(p["scales"]), 256, 2, 64, None, Q.QMM_ZP_UNIFORM, p["uniform_zp"],
                          out_dtype=tt("f32"), f32=True)
    compare(y, host_f64(dY), "bf16", weights(p), "f32", f"uniform {uniform}")


@pytest.mark.parametrize("dy_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M", [20, 200])
def test_types(dy_type, out, M):
    p, dY = problem(M, 200, 104, 4, 32, "packed", dy_type, seed=31)
    compare(run(p, dY, out), host_f64(dY), dy_type, weights(p), out, f"{dy_type} -> {out}")


@pytest.mark.parametrize("scale", [1.0, 1e-6, 1e-25])
@pytest.mark.parametrize("M,K,N,block", [(1, 512, 130, 64), (16, 4096, 256, 64), (100, 250, 99, 16), (300, 640, 72, 128)])
def test_codebook(M, K, N, block, scale):
    """Weights of any magnitude: absmax far below what fp16 holds."""
    p = gen.codebook_problem(1, K, N, seed=41 + M, block=block)
    am = (p["absmax"] * np.float32(scale)).astype(np.float32)
    dY = dev_act(gen.activations(np.random.default_rng(43), (M, N), "bf16"), "bf16")
    w = O.dequant_codebook4(p["W"], K, block, am, p["codebook"]).astype(np.float64)
    y = Q.qmm_codebook4_dgrad(dY, dev(p["W"]), dev(am), dev(p["codebook"]), K, block, out_dtype=tt("f32"), f32=True)
    compare(y, host_f64(dY), "bf16", w, "f32", f"codebook M={M} absmax x {scale}")


@pytest.mark.parametrize("M,N", [(40, 40), (100, 100), (300, 304)])
def test_one_hot_rows_read_the_weights_out(M, N):
    """dY = one-hot rows: dX are the fp32 weights, bit for bit, whatever the format and tile."""
    t = torch()
    eye = t.eye(M, N, dtype=t.bfloat16, device="cuda")
    for bits, zp in ((4, "packed"), (8, "packed"), (4, "f16"), (2, "none")):
        p, _ = problem(1, 333, N, bits, 32, zp, "bf16", seed=51)
        want = weights(p)[:M].astype(np.float32)
        assert np.array_equal(run(p, eye, "f32").cpu().numpy()[:min(M, N)], want), (bits, zp)
    p = gen.codebook_problem(1, 333, N, seed=52, block=64)
    y = Q.qmm_codebook4_dgrad(eye, dev(p["W"]), dev(p["absmax"]), dev(p["codebook"]), 333, 64, out_dtype=t.float32,
                              f32=True)
    want = O.dequant_codebook4(p["W"], 333, 64, p["absmax"], p["codebook"])[:M]
    assert np.array_equal(y.cpu().numpy()[:min(M, N)], want)


@pytest.mark.parametrize("dy_type", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 80, 200])
def test_small_gradients_beside_large_ones(dy_type, M):
    """Gradients 2^-60 of their row's largest keep their bits in the columns whose weights are zero at
    the large ones (code 8 of 4 bits without a zero point)."""
    t = torch()
    K, N = 128, 64
    p = gen.nbits_problem(1, K, N, 4, 32, seed=61, zp="none")
    W = np.array(p["W"]).reshape(N, -1)
    W[: N // 2, :] = (W[: N // 2, :] & 0xF0) | 0x08           # even columns
    p["W"] = W.reshape(np.array(p["W"]).shape)
    g = np.random.default_rng(62).standard_normal((M, N))
    g[:, N // 2:] *= 2.0 ** -60
    dY = t.from_numpy(g).to(tt(dy_type)).cuda()
    compare(run(p, dY, "f32"), host_f64(dY), dy_type, weights(p), "f32", f"{dy_type} M={M}")


@pytest.mark.parametrize("dy_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [4, 100, 300])
def test_infinities(dy_type, M):
    """An infinite gradient gives what the formula gives: infinite with the weights' signs, NaN where a
    weight is zero; other rows keep their bits."""
    t = torch()
    p, dY = problem(M, 264, 136, 4, 64, "none", dy_type, seed=71)
    clean = host_bits(run(p, dY, "f32")).copy()
    dY[1, 5] = float("inf")
    dY[3, 7] = -float("inf")
    dY[2, 9] = float("nan")
    got = run(p, dY, "f32")
    w, g = weights(p), host_f64(dY)
    for m in (1, 3):
        with np.errstate(invalid="ignore"):
            want = (g[m][:, None] * w).sum(0)
        assert np.array_equal(host_f64(got)[m], want, equal_nan=True), m
        assert np.isinf(want).any() and np.isnan(want).any()
    assert bool(t.isnan(got[2]).all())
    keep = [m for m in range(M) if m not in (1, 2, 3)]
    assert np.array_equal(host_bits(got)[keep], clean[keep])
    # an infinite scale: no finite value in its block of columns (fma(q, s, -(z s)) is NaN there, as in
    # the forward product), and the other columns as they were
    p, dY = problem(M, 264, 136, 4, 64, "none", dy_type, seed=73)
    clean = host_bits(run(p, dY, "f32")).copy()
    s = np.array(p["scales"])
    s.reshape(136, -1)[3, 1] = np.float16(np.inf).view(np.uint16)
    p["scales"] = s
    dY[0, 3] = 0.0
    y = run(p, dY, "f32")
    assert not np.isfinite(host_f64(y)[:, 64:128]).any()
    assert np.array_equal(np.delete(host_bits(y), np.arange(64, 128), axis=1)[1:],
                          np.delete(clean, np.arange(64, 128), axis=1)[1:])


@pytest.mark.parametrize("dy_type", ["bf16", "f16"])
def test_misaligned(dy_type):
    """dY one element past an aligned address: through its planes, the same results."""
    t = torch()
    p, dY = problem(70, 264, 136, 4, 64, "packed", dy_type, seed=77)
    flat = t.zeros(dY.numel() + 1, dtype=dY.dtype, device="cuda")
    odd = flat[1:].view(dY.shape)
    odd.copy_(dY)
    compare(run(p, odd, "f32"), host_f64(dY), dy_type, weights(p), "f32", f"misaligned {dy_type}")


def test_gradient_of_the_forward_product():
    """<dY, qmm_nbits(X)> = <dX, X> and differences of the forward product along one coordinate, with
    the forward path of up to 8 rows, whose operands are not rounded either."""
    t = torch()
    M, K, N = 8, 320, 144
    p, dY = problem(M, K, N, 4, 32, "packed", "bf16", seed=81)
    dx, g, w = host_f64(run(p, dY, "f32")), host_f64(dY), weights(p)
    fwd = lambda x: host_f64(Q.qmm_nbits(x, dev(p["W"]), dev(p["scales"]), K, 4, 32, dev(p["zp"]), Q.QMM_ZP_PACKED,  # noqa: E731
                                         out_dtype=t.float32))
    x = t.from_numpy(np.random.default_rng(82).standard_normal((M, K)).astype(np.float32)).cuda()
    lim = (np.abs(g) @ np.abs(w) * np.abs(host_f64(x))).sum()
    # fp32 sums on both sides; the forward path adds z s sums of a block apart: twice the terms
    assert abs((g * fwd(x)).sum() - (dx * host_f64(x)).sum()) <= gamma(2 * K + 3 * (N + 64) + 100) * 4 * lim
    for m, k in ((0, 0), (5, 31), (7, 319)):
        e = t.zeros_like(x)
        e[m, k] = 1.0
        d = (g * (fwd(e) - fwd(t.zeros_like(x)))).sum()
        z = 15.0 * O.f16_bits_to_f64(np.asarray(p["scales"])).reshape(N, -1)[:, k // 32]
        assert abs(d - dx[m, k]) <= gamma(2 * K + 3 * (N + 64) + 100) * (np.abs(g[m]) @ (np.abs(w[:, k]) + z))


@pytest.mark.parametrize("M", [8, 96])
def test_fine_tuning_step(M):
    """Adapters' input gradient on an fp32 base from the frozen weights, to fp32 accuracy."""
    t = torch()
    K, N, r, L = 256, 192, 8, 3
    p, dY = problem(M, K, N, 4, 64, "packed", "bf16", seed=91)
    rng = np.random.default_rng(92)
    X = t.from_numpy(rng.standard_normal((M, K))).bfloat16().cuda()
    A = t.from_numpy(rng.standard_normal((L, r, K)) / 16).bfloat16().cuda()
    B = t.from_numpy(rng.standard_normal((L, N, r)) * 0.3).bfloat16().cuda()
    ids = dev(rng.integers(-1, L, M).astype(np.int32))
    base = run(p, dY, "f32")
    dX, _, _ = Q.qmm_lora_grad(dY, X, A, B, ids, base=base, dx_dtype=t.float32)
    g = host_f64(dY)
    ref = AO.lora_grad(g, host_f64(X), host_f64(A), host_f64(B), ids.cpu().numpy(), base=g @ weights(p))[0]
    assert O.rel_l2(host_f64(dX), ref) <= 1e-5


def test_repeats_streams_and_graph():
    t = torch()
    for M, ty in ((8, "bf16"), (300, "f16")):
        p, g = problem(M, 512, 640, 4, 64, "packed", ty, seed=95)
        W, s, z = dev(p["W"]), dev(p["scales"]), dev(p["zp"])
        need = Q.lib().qmm_dgrad_f32_workspace_bytes(Q.dtype_code(g), M, 512, 640)
        ws = t.empty(need, dtype=t.uint8, device="cuda")

        def step(out):
            return Q.qmm_nbits_dgrad(g, W, s, 512, 4, 64, z, Q.QMM_ZP_PACKED, out=out, workspace=ws, f32=True)

        out = t.empty(M, 512, dtype=t.bfloat16, device="cuda")
        ref = host_bits(step(out)).copy()
        for _ in range(5):
            assert np.array_equal(host_bits(step(out)), ref)
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            step(out)
        side.synchronize()
        assert np.array_equal(host_bits(out), ref)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            step(out)
        g0 = g.clone()
        for k in range(4):
            g.copy_(g0 * (k + 1))
            graph.replay()
            t.cuda.synchronize()
            got = host_bits(out).copy()
            assert np.array_equal(got, host_bits(step(t.empty_like(out)))), k


def test_refusals():
    t = torch()
    p, dY = problem(4, 64, 32, 4, 32, "packed", "f16", seed=97)
    W, s, z = dev(p["W"]), dev(p["scales"]), dev(p["zp"])
    with pytest.raises(ValueError):
        Q.qmm_nbits_dgrad(dY[:, :31].contiguous(), W, s, 64, 4, 32, z, Q.QMM_ZP_PACKED, f32=True)
    with pytest.raises(Q.QmmError) as e:
        Q.qmm_nbits_dgrad(dY, W, s, 64, 4, 32, z, Q.QMM_ZP_PACKED, f32=True,
                          workspace=t.empty(64, dtype=t.uint8, device="cuda"))
    assert e.value.status == -7
    assert Q.qmm_nbits_dgrad(dY[:0], W, s, 64, 4, 32, z, Q.QMM_ZP_PACKED, f32=True).shape == (0, 64)
