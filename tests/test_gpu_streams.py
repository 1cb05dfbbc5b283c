"""GPU: calls on a given stream while the current one is busy.  Memory that work queued on the current
stream still uses is not written by the call, and an output that such work still reads is not written
by the next call."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import inputs as gen
from gemm_qmm_nbits_amd import qmm as Q

from gpu_util import dev, dev_act, host_bits, torch

pytestmark = pytest.mark.gpu


def busy():
    """Some milliseconds of work on the current stream."""
    t = torch()
    a = t.ones(4096, 4096, device="cuda")
    for _ in range(40):
        a = a @ a * 0.0 + 1.0
    return a


def entries():
    """name -> (call(stream) -> outputs, bytes of the memory it takes)."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(1)

    def randn(*shape, dtype=t.bfloat16):
        return t.randn(*shape, device="cuda", generator=g).to(dtype)

    M, K, N, r, L, E = 300, 512, 640, 16, 3, 4
    X, dY, A, B = randn(M, K), randn(M, N), randn(L, r, K), randn(L, N, r)
    ids = t.randint(0, L, (M,), dtype=t.int32, device="cuda", generator=g)
    W, off = randn(E, N, K), dev(np.array([0, 100, 100, 180, 300], np.int32))
    p = gen.nbits_problem(1, K, N, 4, 64, seed=5, zp="packed")
    Wq, s, z = dev(p["W"]), dev(p["scales"]), dev(p["zp"])
    c = gen.codebook_problem(1, K, N, seed=6, block=64)
    Wc, am, cb = dev(c["W"]), dev(c["absmax"]), dev(c["codebook"])
    q = Q.lib()
    return {
        "lora_add": (lambda st: [Q.qmm_lora_add(X, A, B, ids, stream=st)],
                     [M * N * 2, q.qmm_lora_add_workspace_bytes(M, K, N, r, L)]),
        "lora_grad": (lambda st: Q.qmm_lora_grad(dY, X, A, B, ids, stream=st),
                      [M * K * 2, L * r * K * 4, L * N * r * 4, q.qmm_lora_grad_workspace_bytes(M, K, N, r, L)]),
        "nbits_dgrad": (lambda st: [Q.qmm_nbits_dgrad(dY, Wq, s, K, 4, 64, z, Q.QMM_ZP_PACKED, stream=st)],
                        [M * K * 2, q.qmm_dgrad_workspace_bytes(M, K, N)]),
        "nbits_dgrad_f32": (lambda st: [Q.qmm_nbits_dgrad(dY, Wq, s, K, 4, 64, z, Q.QMM_ZP_PACKED, stream=st,
                                                          f32=True)],
                            [M * K * 2, q.qmm_dgrad_f32_workspace_bytes(Q.QMM_BF16, M, K, N)]),
        "codebook4_dgrad": (lambda st: [Q.qmm_codebook4_dgrad(dY, Wc, am, cb, K, 64, stream=st)],
                            [M * K * 2, q.qmm_dgrad_workspace_bytes(M, K, N)]),
        "grouped_mm": (lambda st: [Q.qmoe_grouped_mm(X, off, W, stream=st)], [M * N * 2]),
        "grouped_mm_grad": (lambda st: Q.qmoe_grouped_mm_grad(dY, X, off, W, need_dbias=True, stream=st),
                            [M * K * 2, E * N * K * 2, E * N * 2]),
        "nbits": (lambda st: [Q.qmm_nbits(X, Wq, s, K, 4, 64, z, Q.QMM_ZP_PACKED, stream=st)],
                  [M * N * 2, q.qmm_nbits_workspace_bytes(M, K, N, Q.QMM_BF16)]),
    }


NAMES = ["lora_add", "lora_grad", "nbits_dgrad", "nbits_dgrad_f32", "codebook4_dgrad", "grouped_mm", "grouped_mm_grad",
         "nbits"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_queued_work_is_left_alone(name):
    """Freed tensors of the sizes that the call takes, which queued work has yet to read."""
    t = torch()
    call, sizes = entries()[name]
    side = t.cuda.Stream()
    want = [host_bits(v).copy() for v in call(None)]
    t.cuda.synchronize()
    victims = [t.full((n,), 77, dtype=t.uint8, device="cuda") for n in sizes for _ in range(2)]
    copies = [t.zeros_like(v) for v in victims]
    t.cuda.synchronize()
    keep = busy()
    for c, v in zip(copies, victims):
        c.copy_(v)
    del v, victims
    got = call(side)
    side.synchronize()
    got = [host_bits(v).copy() for v in got]
    t.cuda.synchronize()
    assert all(bool((c == 77).all()) for c in copies)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    del keep


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_queued_work_reads_are_left_alone(name):
    """An output freed while the current stream has yet to read it: the next call does not write it."""
    t = torch()
    call, _ = entries()[name]
    side = t.cuda.Stream()
    want = [host_bits(v).copy() for v in call(None)]
    t.cuda.synchronize()
    first = list(call(side))
    t.cuda.current_stream().wait_stream(side)
    keep = busy()
    copies = [v.clone() for v in first]
    where = {v.data_ptr() for v in first}
    first.clear()
    second = call(side)
    for v in second:
        assert v.data_ptr() not in where
        with t.cuda.stream(side):
            v.zero_()
    t.cuda.synchronize()
    assert all(np.array_equal(host_bits(c), b) for c, b in zip(copies, want))
    del keep


def test_a_stream_of_the_tensors_device_is_needed():
    class Other:
        device_index, cuda_stream = 7, 0

    with pytest.raises(ValueError):
        Q._handle(Other, 0)


@pytest.mark.parametrize("name", NAMES[:-1])
def test_captured_on_a_forked_stream(name):
    """A call on a given stream that a captured one forked: its memory is the graph's, and replays repeat
    the call's results."""
    t = torch()
    call, _ = entries()[name]
    want = [host_bits(v).copy() for v in call(None)]
    side = t.cuda.Stream()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        side.wait_stream(t.cuda.current_stream())
        outs = list(call(side))
        t.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for v in outs:
            v.zero_()
        graph.replay()
        t.cuda.synchronize()
        assert all(np.array_equal(host_bits(v), b) for v, b in zip(outs, want))
        call(None)


@pytest.mark.parametrize("M,K,r", [(40, 96, 300), (12, 8200, 64), (300, 128, 512)])
@pytest.mark.parametrize("ty", ["float16", "bfloat16"])
def test_captured_adapters_of_high_rank(M, K, r, ty):
    """Forms whose shared memory passes 32 KB (its limit is raised per call) captured, the first call of
    their shape included, and replayed between eager calls."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(M)
    N, L = 192, 2

    def randn(*shape):
        return t.randn(*shape, device="cuda", generator=g).to(getattr(t, ty))

    X, dY, A, B = randn(M, K), randn(M, N), randn(L, r, K), randn(L, N, r)
    ids = t.randint(-1, L, (M,), dtype=t.int32, device="cuda", generator=g)
    outs = [t.empty_like(dY), t.empty_like(X), t.empty(L, r, K, device="cuda"), t.empty(L, N, r, device="cuda")]

    def step(o):
        Q.qmm_lora_add(X, A, B, ids, out=o[0])
        Q.qmm_lora_grad(dY, X, A, B, ids, dX=o[1], dA=o[2], dB=o[3])
        return o

    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(outs)
    x0 = X.clone()
    for k in range(3):
        X.copy_(x0 * (k + 1))
        graph.replay()
        t.cuda.synchronize()
        got = [host_bits(v).copy() for v in outs]
        for a, b in zip(got, step([t.empty_like(v) for v in outs])):
            assert np.array_equal(a, host_bits(b)), k
