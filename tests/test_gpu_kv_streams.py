"""GPU: the cache's calls on a given stream while the current one is busy, two of them at once, and pools
past 32 bits of bytes and elements."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q

from gpu_util import dev, host_bits, torch

pytestmark = pytest.mark.gpu


def busy():
    """Some milliseconds of work on the current stream."""
    t = torch()
    a = t.ones(4096, 4096, device="cuda")
    for _ in range(40):
        a = a @ a * 0.0 + 1.0
    return a


def problem(B, L, q, heads=8, kv=2, D=128, bits=4, group=64, page=16, seed=0):
    """A filled cache, and the arguments of an attention call over it."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    width = -(-L // page)
    cache = Q.qkv_cache_new(B * width, kv, D, bits=bits, group=group, page=page)
    K, V = (t.randn(B * width * page, kv, D, device="cuda", generator=g).to(t.bfloat16) for _ in range(2))
    slots = t.arange(B * width * page, dtype=t.int32, device="cuda")
    Q.qkv_cache_store(K, V, slots, cache)
    a = dict(cache=cache, table=t.randperm(B * width, device="cuda", generator=g).to(t.int32).view(B, width),
             kv_len=t.full((B,), L, dtype=t.int32, device="cuda"))
    if q > 1:
        a.update(cu_q=t.arange(0, B * q + 1, q, dtype=t.int32, device="cuda"), max_q=q)
    x = t.randn(B * q, heads, D, device="cuda", generator=g).to(t.bfloat16)
    return x, a, slots


# sequences, tokens, queries, tokens expected: decode in many parts, a few queries, a chunk for the kernel of many rows
SHAPES = {"decode": (2, 3000, 1, None), "few": (3, 500, 7, None), "chunk": (3, 2100, 300, 1 << 20)}


def entries():
    """name -> (call(stream) -> outputs, bytes of the memory it takes)."""
    t = torch()
    r = {}
    for name, (B, L, q, much) in SHAPES.items():
        x, a, slots = problem(B, L, q)
        a["max_kv"] = much or a["table"].shape[1] * 16
        ws = Q.lib().qkv_attention_workspace_bytes(B * q, 8, 2, 128, B, q, a["max_kv"], 0)
        r[name] = (lambda st, x=x, a=a: list(Q.qkv_attention(x, need_lse=True, stream=st, **a)),
                   [x.numel() * 2, B * q * 8 * 4, max(ws, 1)])
    n = slots.numel()
    r["load"] = (lambda st: list(Q.qkv_cache_load(a["cache"], slots, out_dtype=t.bfloat16, stream=st)), [n * 2 * 128 * 2])
    return r


NAMES = [*SHAPES, "load"]


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
def test_captured_on_a_forked_stream(name):
    """A call on a given stream that a captured one forked: its memory is the graph's, and replays repeat
    the call's results, with eager calls between them."""
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
        other = call(None)
        t.cuda.synchronize()
        assert all(np.array_equal(host_bits(v), b) for v, b in zip(outs, want))
        assert all(np.array_equal(host_bits(v), b) for v, b in zip(other, want))


def test_calls_at_once():
    """Every kernel, each call on a stream of its own, the same cache read by two of them."""
    t = torch()
    calls = [call for call, _ in entries().values()] * 2
    want = [[host_bits(v).copy() for v in call(None)] for call in calls]
    streams = [t.cuda.Stream() for _ in calls]
    t.cuda.synchronize()
    for _ in range(3):
        got = [call(st) for call, st in zip(calls, streams)]
        t.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(np.array_equal(host_bits(v), b) for v, b in zip(g, w))


def test_a_decode_loop_on_a_stream():
    """Store of the new tokens, attention, load, token after token on one stream, the current one busy: as a
    program without streams."""
    t = torch()
    B, heads, kv, D, page, steps = 3, 8, 2, 64, 16, 5
    g = t.Generator(device="cuda").manual_seed(3)
    width = 8
    table = t.randperm(B * width, device="cuda", generator=g).to(t.int32).view(B, width)
    x = t.randn(steps, B, heads + 2 * kv, D, device="cuda", generator=g).to(t.bfloat16)
    lens = [t.tensor([15 + s, 30 + s, 63 + s], dtype=t.int32, device="cuda") for s in range(steps)]
    at = [(n - 1).long() for n in lens]
    slots = [(table.gather(1, (i // page).view(-1, 1)).view(-1) * page + i % page).int() for i in at]
    side = t.cuda.Stream()
    t.cuda.synchronize()

    def run(st):
        cache = Q.qkv_cache_new(B * width, kv, D, group=32, page=page, stream=st)
        outs = []
        for s in range(steps):
            qkv = x[s]
            Q.qkv_cache_store(qkv[:, heads:heads + kv], qkv[:, heads + kv:], slots[s], cache, stream=st)
            outs.append(Q.qkv_attention(qkv[:, :heads], cache, table, lens[s], stream=st))
            outs += list(Q.qkv_cache_load(cache, slots[s], out_dtype=t.bfloat16, stream=st))
        (t.cuda.current_stream() if st is None else st).synchronize()
        return [host_bits(v).copy() for v in outs]

    want = run(None)
    keep = busy()
    got = run(side)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    t.cuda.synchronize()
    del keep


@pytest.mark.parametrize("new", [1, 40])
def test_pools_past_32_bits(new):
    """Pages at the end of pools whose codes pass 2^34 bytes and parameters 2^31."""
    t = torch()
    D, bits, group, kv, heads, page = 256, 8, 32, 8, 16, 1024
    pages = 8300  # of 2 MiB codes and 256 KiB parameters
    cache = Q.qkv_cache_new(pages, kv, D, bits=bits, group=group, page=page)
    assert cache["k"].numel() > 1 << 34 and cache["k_params"].numel() > 1 << 30
    assert cache["k_params"].numel() * cache["k_params"].element_size() > 1 << 31
    rng = np.random.default_rng(7)
    L = 1200
    small = Q.qkv_cache_new(2, kv, D, bits=bits, group=group, page=page)
    K, V = (t.from_numpy(rng.standard_normal((L, kv, D)).astype(np.float32)).cuda() for _ in range(2))
    tok = np.arange(L)
    far = np.array([pages - 1, 4100], np.int32)
    Q.qkv_cache_store(K, V, dev((far[tok // page].astype(np.int64) * page + tok % page).astype(np.int32)), cache)
    Q.qkv_cache_store(K, V, dev(tok.astype(np.int32)), small)
    for w in ("k", "v", "k_params", "v_params"):
        assert t.equal(cache[w][[pages - 1, 4100]], small[w])
    slots = (far[tok // page].astype(np.int64) * page + tok % page).astype(np.int32)
    got = Q.qkv_cache_load(cache, dev(slots), out_dtype=t.bfloat16)
    want = Q.qkv_cache_load(small, dev(tok.astype(np.int32)), out_dtype=t.bfloat16)
    assert all(t.equal(a, b) for a, b in zip(got, want))
    x = t.from_numpy(rng.standard_normal((new, heads, D))).to(t.bfloat16).cuda()
    a = dict(kv_len=dev(np.array([L], np.int32)), cu_q=dev(np.array([0, new], np.int32)), need_lse=True)
    for much in (None, 1 << 30):
        got = Q.qkv_attention(x, cache, dev(far[None]), max_kv=much, **a)
        want = Q.qkv_attention(x, small, dev(np.array([[0, 1]], np.int32)), max_kv=much, **a)
        assert all(np.array_equal(host_bits(p), host_bits(q)) for p, q in zip(got, want))
    del cache
    t.cuda.synchronize()
    t.cuda.empty_cache()


def test_many_tokens_at_once():
    """A store of 2^20 tokens, the most, whose slots repeat; more are refused."""
    t = torch()
    T, n, D = 1 << 20, 1 << 18, 64
    cache = Q.qkv_cache_new(n // 64, 1, D, page=64)
    rng = np.random.default_rng(9)
    slots = rng.integers(0, n, T).astype(np.int32)
    K = t.randn(T, 1, D, device="cuda").to(t.bfloat16)
    V = K * 2
    Q.qkv_cache_store(K, V, dev(slots), cache)
    last = np.full(n, -1)
    last[slots] = np.arange(T)  # (assignments in order: the last stays)
    held = np.nonzero(last >= 0)[0][:: 97]
    once = Q.qkv_cache_new(len(held) // 64 + 1, 1, D, page=64)
    mine = np.arange(len(held), dtype=np.int32)
    rows = t.from_numpy(last[held]).cuda()
    Q.qkv_cache_store(K[rows], V[rows], dev(mine), once)
    a = Q.qkv_cache_load(cache, dev(held.astype(np.int32)))
    b = Q.qkv_cache_load(once, dev(mine))
    assert all(t.equal(x, y) for x, y in zip(a, b))
    more = t.zeros(T + 1, 1, D, dtype=t.bfloat16, device="cuda")
    with pytest.raises(Q.QmmError):
        Q.qkv_cache_store(more, more, t.zeros(T + 1, dtype=t.int32, device="cuda"), cache)
    t.cuda.synchronize()
