"""GPU parity of the input gradients of low-bit projections against the fp64 oracle: with the
declared operand roundings (elementwise bound) and without them (relative L2)."""
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


def tt(name):
    return getattr(torch(), DT[name])


def weights(p):
    return O.dequant_nbits(p["W"], p["bits"], p["K"], p["block"], p["scales"], p["zp"],
                           oracle_zp_kind(O, p["zp_mode"])).astype(np.float64)


def compare(y, dy, dy_type, w, out, label):
    """dy: stored activations; w: exact weights [N, K] in fp64."""
    g = O.activations_f64(dy, dy_type)
    gm = g if dy_type == "f16" else O._round_operand(g, "f16")
    wm = O._round_operand(w, "f16")
    N = w.shape[0]
    got = host_f64(y)
    assert_elementwise(got, gm @ wm, gamma(N + 70) * (np.abs(gm) @ np.abs(wm)), out, label)
    err = O.rel_l2(got, g @ w)
    say(f"  {label}: relL2(exact) = {err:.2e}")
    # operands rounded to fp16: 2^-11 each at most, random in sign; 16-bit outputs their own
    assert err <= max(TOL["f16"], TOL[out]), err


def run_nbits(p, dy, dy_type, out, **kw):
    z = dev(p["zp"]) if p["zp"] is not None else None
    return Q.qmm_nbits_dgrad(dev_act(dy, dy_type), dev(p["W"]), dev(p["scales"]), p["K"], p["bits"], p["block"], z,
                             ZP_KIND[p["zp_mode"]], 0.0, out_dtype=tt(out), **kw)


def problem(M, K, N, bits, block, zp, dy_type, seed):
    p = gen.nbits_problem(1, K, N, bits, block, seed=seed, zp=zp)
    dy = gen.activations(np.random.default_rng(seed + 1), (M, N), dy_type)
    return p, dy


# one row, a few, the borders of the tile heights (64, 128) and past them; sizes on, below and past
# the stages (32 rows of W) and column tiles (128, 256); odd K (a ragged last block) and odd N
SIZES = [(1, 256, 64), (1, 70, 33), (3, 1, 1), (16, 1024, 300), (64, 512, 256), (65, 264, 97), (128, 320, 160),
         (129, 515, 130), (300, 1030, 96), (260, 128, 1000)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_sizes(M, K, N, bits):
    p, dy = problem(M, K, N, bits, 32, "packed", "bf16", seed=M + K + bits)
    compare(run_nbits(p, dy, "bf16", "f32"), dy, "bf16", weights(p), "f32", f"M={M} K={K} N={N} u{bits}")


@pytest.mark.parametrize("zp", ["none", "packed", "f16"])
@pytest.mark.parametrize("bits,block", [(2, 16), (2, 64), (3, 32), (3, 128), (4, 16), (4, 256), (8, 16), (8, 128)])
@pytest.mark.parametrize("M", [5, 150])
def test_formats(bits, block, zp, M):
    p, dy = problem(M, 300, 120, bits, block, zp, "f16", seed=100 + bits + block)
    compare(run_nbits(p, dy, "f16", "f16"), dy, "f16", weights(p), "f16", f"u{bits} block={block} zp={zp} M={M}")


@pytest.mark.parametrize("uniform", [1.5, -0.3])
def test_uniform_zero_point(uniform):
    """A scalar zero point: one that takes the single-fma dequantization and one that does not."""
    p = gen.nbits_problem(1, 256, 96, 2, 64, seed=7, zp="f16_uniform", uniform_zp=uniform)
    dy = gen.activations(np.random.default_rng(8), (40, 96), "bf16")
    y = Q.qmm_nbits_dgrad(dev_act(dy, "bf16"), dev(p["W"]), dev(p["scales"]), 256, 2, 64, None, Q.QMM_ZP_UNIFORM,
                          p["uniform_zp"], out_dtype=tt("f32"))
    compare(y, dy, "bf16", weights(p), "f32", f"uniform {uniform}")


@pytest.mark.parametrize("dy_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M", [20, 200])
def test_types(dy_type, out, M):
    p, dy = problem(M, 200, 104, 4, 32, "packed", dy_type, seed=31)
    compare(run_nbits(p, dy, dy_type, out), dy, dy_type, weights(p), out, f"{dy_type} -> {out}")


@pytest.mark.parametrize("M,K,N,block", [(1, 512, 130, 64), (16, 4096, 256, 64), (100, 250, 99, 16), (300, 640, 72, 128)])
@pytest.mark.parametrize("dy_type", ["bf16", "f16"])
def test_codebook(M, K, N, block, dy_type):
    p = gen.codebook_problem(1, K, N, seed=41 + M, block=block)
    dy = gen.activations(np.random.default_rng(43), (M, N), dy_type)
    w = O.dequant_codebook4(p["W"], K, block, p["absmax"], p["codebook"]).astype(np.float64)
    y = Q.qmm_codebook4_dgrad(dev_act(dy, dy_type), dev(p["W"]), dev(p["absmax"]), dev(p["codebook"]), K, block,
                              out_dtype=tt(dy_type))
    compare(y, dy, dy_type, w, dy_type, f"codebook M={M}")


def test_one_hot_rows_read_the_weights_out():
    """dY = one-hot rows: dX are the fp16 weights, bit for bit, whatever the tile."""
    t = torch()
    for M, N in ((40, 40), (100, 100), (300, 300)):
        p, _ = problem(1, 333, N, 4, 32, "packed", "f16", seed=51)
        eye = np.eye(M, N).astype(np.float16).view(np.uint16)
        y = run_nbits(p, eye, "f16", "f16")
        want = O.to_f16(weights(p)[:M])
        assert np.array_equal(y.cpu().numpy()[:min(M, N)], want)
    t.cuda.synchronize()


def test_small_gradients_keep_their_bits():
    """bf16 gradients far below fp16's range: the row's power of two brings them in."""
    p, dy = problem(6, 256, 64, 4, 64, "packed", "bf16", seed=61)
    tiny = (host_f64(dev_act(dy, "bf16")) * 2.0 ** -100)
    tiny = torch().from_numpy(tiny).to(torch().bfloat16)
    y = Q.qmm_nbits_dgrad(tiny.cuda(), dev(p["W"]), dev(p["scales"]), 256, 4, 64, dev(p["zp"]), Q.QMM_ZP_PACKED,
                          out_dtype=tt("f32"))
    full = run_nbits(p, dy, "bf16", "f32")
    assert np.array_equal(host_f64(y) * 2.0 ** 100, host_f64(full))


@pytest.mark.parametrize("M", [4, 100, 300])
def test_bad_rows_stay_in_their_rows(M):
    p, dy = problem(M, 264, 136, 4, 64, "packed", "f16", seed=71)
    clean = host_bits(run_nbits(p, dy, "f16", "f16")).copy()
    bad = dy.copy()
    bad[1] = np.float16(np.nan).view(np.uint16)
    bad[3] = np.float16(np.inf).view(np.uint16)
    y = host_bits(run_nbits(p, bad, "f16", "f16"))
    keep = [m for m in range(M) if m not in (1, 3)]
    assert np.array_equal(y[keep], clean[keep])


def test_gradient_of_the_forward_product():
    """<dY, qmm_nbits(X)> = <qmm_nbits_dgrad(dY), X>, and differences of the forward product along
    one coordinate: the two directions read the same weights."""
    t = torch()
    M, K, N = 24, 320, 144
    p, dy = problem(M, K, N, 4, 32, "packed", "f16", seed=81)
    g = dev_act(dy, "f16")
    dx = host_f64(run_nbits(p, dy, "f16", "f32"))
    gh = host_f64(g)
    w16 = O._round_operand(weights(p), "f16")
    fwd = lambda x: host_f64(Q.qmm_nbits(x, dev(p["W"]), dev(p["scales"]), K, 4, 32, dev(p["zp"]), Q.QMM_ZP_PACKED,  # noqa: E731
                                         out_dtype=t.float32))
    x = t.from_numpy(np.random.default_rng(82).standard_normal((M, K))).half().cuda()
    lim = gamma(K + N + 100) * (np.abs(gh) @ np.abs(w16) * np.abs(host_f64(x))).sum()
    assert abs((gh * fwd(x)).sum() - (dx * host_f64(x)).sum()) <= lim
    zero = t.zeros_like(x)
    for m, k in ((0, 0), (5, 31), (23, 319)):
        e = zero.clone()
        e[m, k] = 1.0
        d = (gh * (fwd(e) - fwd(zero))).sum()
        assert abs(d - dx[m, k]) <= gamma(K + N + 100) * (np.abs(gh[m]) @ np.abs(w16[:, k])) + 1e-12


def test_fine_tuning_step():
    """The operators as a fine-tuning step uses them: projection, adapters, then the gradients of
    both down to the input."""
    t = torch()
    M, K, N, r, L = 96, 256, 192, 8, 3
    p, dy = problem(M, K, N, 4, 64, "packed", "bf16", seed=91)
    rng = np.random.default_rng(92)
    X = t.from_numpy(rng.standard_normal((M, K))).bfloat16().cuda()
    A = t.from_numpy(rng.standard_normal((L, r, K)) / 16).bfloat16().cuda()
    B = t.from_numpy(rng.standard_normal((L, N, r)) * 0.3).bfloat16().cuda()
    ids = dev(rng.integers(-1, L, M).astype(np.int32))
    T = t.empty(M, r, device="cuda")
    W, s, z = dev(p["W"]), dev(p["scales"]), dev(p["zp"])
    base = Q.qmm_nbits(X, W, s, K, 4, 64, z, Q.QMM_ZP_PACKED, out_dtype=t.float32)
    y = Q.qmm_lora_add(X, A, B, ids, base=base, T=T)
    dY = dev_act(dy, "bf16")
    dbase = Q.qmm_nbits_dgrad(dY, W, s, K, 4, 64, z, Q.QMM_ZP_PACKED, out_dtype=t.float32)
    dX, dA, dB = Q.qmm_lora_grad(dY, X, A, B, ids, T=T, base=dbase)
    w = weights(p)
    x, a, b, g, i = host_f64(X), host_f64(A), host_f64(B), host_f64(dY), ids.cpu().numpy()
    assert O.rel_l2(host_f64(y), AO.lora_add(x, a, b, i, base=x @ w.T)) <= 2.0 ** -8
    ref = AO.lora_grad(g, x, a, b, i, base=g @ w)
    assert O.rel_l2(host_f64(dX), ref[0]) <= 2.0 ** -8
    for got, want in ((dA, ref[1]), (dB, ref[2])):
        assert O.rel_l2(host_f64(got), want) <= 1e-5


def test_repeats_and_graph():
    t = torch()
    for M in (8, 300):
        p, dy = problem(M, 512, 640, 4, 64, "packed", "bf16", seed=95)
        W, s, z, g = dev(p["W"]), dev(p["scales"]), dev(p["zp"]), dev_act(dy, "bf16")
        ws = t.empty(Q.lib().qmm_dgrad_workspace_bytes(M, 512, 640), dtype=t.uint8, device="cuda")

        def step(out):
            return Q.qmm_nbits_dgrad(g, W, s, 512, 4, 64, z, Q.QMM_ZP_PACKED, out=out, workspace=ws)

        out = t.empty(M, 512, dtype=t.bfloat16, device="cuda")
        ref = host_bits(step(out)).copy()
        for _ in range(5):
            assert np.array_equal(host_bits(step(out)), ref)
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
    p, dy = problem(4, 64, 32, 4, 32, "packed", "f16", seed=97)
    g, W, s, z = dev_act(dy, "f16"), dev(p["W"]), dev(p["scales"]), dev(p["zp"])
    with pytest.raises(ValueError):
        Q.qmm_nbits_dgrad(g[:, :31].contiguous(), W, s, 64, 4, 32, z, Q.QMM_ZP_PACKED)
    with pytest.raises(ValueError):
        Q.qmm_nbits_dgrad(g, W, s, 128, 4, 32, z, Q.QMM_ZP_PACKED)
    with pytest.raises(ValueError):
        Q.qmm_nbits_dgrad(g, W, s[:3], 64, 4, 32, z, Q.QMM_ZP_PACKED)
    with pytest.raises(TypeError):
        Q.qmm_nbits_dgrad(g, W, s.float(), 64, 4, 32, z, Q.QMM_ZP_PACKED)
    with pytest.raises(TypeError):
        Q.qmm_nbits_dgrad(g, W, s, 64, 4, 32, z, Q.QMM_ZP_F16)
    am, cb = t.ones(32 * 2, device="cuda"), t.ones(16, device="cuda")
    for args in ((am.half(), cb), (am, cb.half())):
        with pytest.raises(TypeError):
            Q.qmm_codebook4_dgrad(g, W, *args, 64, 32)
    with pytest.raises(Q.QmmError) as e:
        Q.qmm_nbits_dgrad(g, W, s, 64, 4, 32, z, Q.QMM_ZP_PACKED, workspace=t.empty(64, dtype=t.uint8, device="cuda"))
    assert e.value.status == -7
