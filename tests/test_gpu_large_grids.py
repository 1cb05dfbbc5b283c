"""GPU: calls inside the documented sizes whose work-groups times threads pass 2^32, the limit of a
launch's first dimension."""
import pytest

from gemm_qmm_nbits_amd import qmm as Q

from gpu_util import assert_elementwise, gamma, host_f64, say, torch

pytestmark = pytest.mark.gpu


def test_many_narrow_experts():
    """4096 experts of 1 x 2^20: the weight gradient has 2^25 tiles of 256 threads."""
    t = torch()
    E, N, K = 4096, 1, 1 << 20
    g = t.Generator(device="cuda").manual_seed(1)
    counts = t.zeros(E, dtype=t.int64)
    used = {0: 3, 2047: 2, 2048: 1, 4095: 2}
    for e, n in used.items():
        counts[e] = n
    off = t.cat([t.zeros(1, dtype=t.int64), counts.cumsum(0)]).int().cuda()
    R = int(off[-1])
    X = t.randn(R, K, device="cuda", generator=g).half()
    dY = t.randn(R, N, device="cuda", generator=g).half()
    W = t.empty(E, N, K, dtype=t.float16, device="cuda").normal_(generator=g)
    say("  grouped_mm")
    Y = Q.qmoe_grouped_mm(X, off, W, out_dtype=t.float32)
    say("  grouped_mm_grad")
    dX, dW, db = Q.qmoe_grouped_mm_grad(dY, X, off, W, dx_dtype=t.float32, need_dbias=True)
    t.cuda.synchronize()
    r = 0
    for e, n in used.items():
        x, d, w = X[r:r + n].double(), dY[r:r + n].double(), W[e].double()
        for got, ref, lim, terms, out in (
                (Y[r:r + n], x @ w.t(), x.abs() @ w.abs().t(), K + 4, "f32"),
                (dX[r:r + n], d @ w, d.abs() @ w.abs(), N + 4, "f32"),
                (dW[e], d.t() @ x, d.abs().t() @ x.abs(), n + 4, "f16"),
                (db[e], d.sum(0), d.abs().sum(0), n + 36, "f16")):
            assert_elementwise(host_f64(got), host_f64(ref), gamma(terms) * host_f64(lim), out, f"expert {e}")
        r += n
    empty = [i for i in range(E) if i not in used]
    for lo in range(0, len(empty), 512):
        assert not bool(dW[empty[lo:lo + 512]].any())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dy_type", ["float32", "bfloat16"])
def test_most_rows(dy_type, f32):
    """2^24 rows, the most that an input gradient takes: the cast has a work-group per row."""
    t = torch()
    M, K, N, block = 1 << 24, 16, 9, 16
    g = t.Generator(device="cuda").manual_seed(2)
    W = t.randint(0, 256, (N, 1, block // 2), dtype=t.uint8, device="cuda", generator=g)
    scales = (t.rand(N, 1, device="cuda", generator=g) + 0.5).half()
    dY = t.randn(M, N, device="cuda", generator=g).to(getattr(t, dy_type))
    say(f"  {dy_type} f32={f32}")
    dX = Q.qmm_nbits_dgrad(dY, W, scales, K, 4, block, out_dtype=t.float32, f32=f32)
    rows = t.tensor([0, 1, 255, 256, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, M - 257, M - 1], device="cuda")
    q = t.stack([W[:, 0] & 15, W[:, 0] >> 4], 2).reshape(N, block)
    w = (q.float() - 8) * scales.float()
    d = dY[rows].double()
    if not f32:                                      # fp16 operands
        w = w.half().float()
    ref, lim = d @ w.double(), d.abs() @ w.double().abs()
    # fp16 operands: fp32 dY is rounded to 11 bits
    own = 2.0 ** -11 if dy_type == "float32" and not f32 else 0.0
    assert_elementwise(host_f64(dX[rows]), host_f64(ref), (gamma(9 * 73 + 70) + own) * host_f64(lim), "f32", dy_type)
