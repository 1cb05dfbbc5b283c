"""GPU parity of the low-bit key/value cache's store and load against the fp64 oracle: codes, scales and
offsets bit for bit, values to the rounding of their type."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q
from oracle import kv_oracle as KO

from gpu_util import assert_elementwise, dev, host_bits, host_f64, say, torch

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}
FORMATS = [(4, 64, 32), (4, 64, 64), (4, 128, 32), (4, 128, 64), (4, 128, 128), (4, 256, 32), (4, 256, 128),
           (8, 64, 32), (8, 64, 64), (8, 128, 64), (8, 128, 128), (8, 256, 32), (8, 256, 64)]


def tt(name):
    return getattr(torch(), DT[name])


def host(cache):
    """The cache's content as the oracle's dict."""
    c = dict(bits=cache["bits"], group=cache["group"])
    for w in ("k", "v"):
        c[w] = cache[w].cpu().numpy().copy()
        c[w + "_params"] = cache[w + "_params"].cpu().numpy().copy()
    return c


def same(a, b):
    for w in ("k", "v"):
        assert np.array_equal(a[w], b[w]), w
        x, y = a[w + "_params"], b[w + "_params"]
        assert np.array_equal(np.isnan(x), np.isnan(y))
        assert np.array_equal(np.nan_to_num(x.astype(np.float32), nan=0.0), np.nan_to_num(y.astype(np.float32), nan=0.0))


def rows(T, H, D, ty, seed, std=1.0):
    t = torch()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, D)) * std + rng.standard_normal((1, H, D)) * 2.0
    return t.from_numpy(x).to(tt(ty)).cuda()


def check_store(K, V, slots, cache, label=""):
    """The call against the oracle, started from the cache's present content."""
    want = host(cache)
    KO.store(host_f64(K), host_f64(V), slots, want)
    Q.qkv_cache_store(K, V, dev(np.asarray(slots, np.int32)), cache)
    same(host(cache), want)
    return want


@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_store_and_load(bits, D, group, ty):
    say(f"store bits={bits} D={D} group={group} {ty}")
    H, page, T = 3, 16, 11
    cache = Q.qkv_cache_new(4, H, D, bits=bits, group=group, page=page)
    slots = [5, 63, 0, 16, 17, -1, 64, 31, 32, 1 << 30, 40]
    want = check_store(rows(T, H, D, ty, 1), rows(T, H, D, ty, 2), slots, cache)
    for out in ("f32", "f16", "bf16"):
        K, V = Q.qkv_cache_load(cache, dev(np.array(slots + [7], np.int32)), out_dtype=tt(out))
        for got, ref in zip((K, V), KO.load(want, slots + [7])):
            # fp32(c s + o) is rounded once, then to the type
            assert_elementwise(host_f64(got), ref, 2.0 ** -24 * np.abs(ref), out, f"load {out}")


@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (1, 10, 64), (2, 8, 256), (33, 5, 32), (65, 2, 16), (300, 1, 128),
                                      (1030, 1, 16)])
def test_sizes(T, H, page):
    """One row to several work-groups, several tokens to a work-group (from 513 tokens on), odd head counts."""
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 2
    cache = Q.qkv_cache_new(pages, H, 64, bits=4, group=32, page=page)
    slots = rng.permutation(pages * page)[:T]
    slots[rng.random(T) < 0.05] = -1
    check_store(rows(T, H, 64, "bf16", 3), rows(T, H, 64, "bf16", 4), slots, cache)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_strides(ty, shift):
    """Keys and values as slices of a fused projection, at element offsets on and off 16 bytes, and heads first."""
    t = torch()
    T, H, D = 9, 4, 128
    fused = rows(1, 1, T * (5 * H * D + shift) + 8, ty, 5).view(-1)[8:].view(T, 5 * H * D + shift)
    K = fused[:, shift:shift + H * D].view(T, H, D) if shift == 0 else \
        fused[:, shift:shift + H * D].unflatten(1, (H, D))
    V = fused[:, shift + 2 * H * D:shift + 3 * H * D].unflatten(1, (H, D))
    cache = Q.qkv_cache_new(2, H, D, bits=8, group=64, page=16)
    check_store(K, V, list(range(3, 12)), cache)
    Kt, Vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (K, V))     # [heads][T][D] in memory
    check_store(Kt, Vt, list(range(13, 22)), cache)
    check_store(K[:1].expand(T, H, D), V[:, :1].expand(T, H, D), list(range(22, 31)), cache)   # strides of 0
    t.cuda.synchronize()


@pytest.mark.parametrize("T", [8, 64, 700, 5000])
def test_one_slot_twice(T):
    """Of tokens with one slot the last is stored, however far apart they are."""
    rng = np.random.default_rng(T)
    cache = Q.qkv_cache_new(8, 1, 64, bits=4, group=64, page=16)
    slots = rng.integers(-1, 100, T)
    K, V = rows(T, 1, 64, "f16", 6), rows(T, 1, 64, "f16", 7)
    want = host(cache)
    last = {int(s): i for i, s in enumerate(slots) if s >= 0}
    order = sorted(last.values())
    KO.store(host_f64(K)[order], host_f64(V)[order], slots[order], want)
    for _ in range(3):
        Q.qkv_cache_store(K, V, dev(slots.astype(np.int32)), cache)
        same(host(cache), want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
def test_values_at_borders(bits, ty):
    """Halves between codes (to the even one), values next to them, groups of one value, of tiny ranges, of the
    types' largest values, signed zeros."""
    t = torch()
    rng = np.random.default_rng(bits)
    top = 2 ** bits - 1
    x = np.zeros((12, 1, 64))
    x[0, 0, :32] = np.resize(np.arange(top + 1), 32) + 0.0
    x[0, 0, 0], x[0, 0, 1] = 0.0, top
    x[0, 0, 2:32] = rng.integers(0, top, 30) + 0.5                       # halves at scale 1
    x[1] = x[0] * 0.25 - 3.0
    x[2] = np.where(rng.random((1, 64)) < 0.5, 1.0, -1.0) * 1e-6
    x[3] = 7.0
    x[4] = rng.standard_normal((1, 64)) * 6e4
    x[5] = rng.standard_normal((1, 64)) * 1e38
    x[6, 0, ::2] = -0.0
    x[7] = rng.standard_normal((1, 64)) * 2.0 ** -14
    x[8] = 1000.0 + rng.standard_normal((1, 64)) * 0.25
    x[9, 0, 3] = 1e-30
    x[10] = rng.integers(-3, 4, (1, 64)) * 2.0 ** -24
    x[11] = (rng.integers(0, 2 * top, (1, 64)) + 0.5) * 0.01
    x[11, 0, ::32] = 0.0
    x[11, 0, 1::32] = 0.01 * 2 * top
    K = t.from_numpy(x).to(tt(ty))
    K = t.where(t.isfinite(K), K, t.full_like(K, t.finfo(K.dtype).max)).cuda()
    if ty == "f32":                                                       # fp32 neighbours of the halves
        K[0, 0, 34:64] = t.nextafter(K[0, 0, 2:32], t.tensor(float("inf"), device="cuda"))
        K[0, 0, 32], K[0, 0, 33] = 0.0, top
    cache = Q.qkv_cache_new(1, 1, 64, bits=bits, group=32, page=16)
    check_store(K, K.flip(0).contiguous(), list(range(12)), cache)


def test_not_finite():
    """A group with a NaN or an infinity reads as NaN; its neighbours and other rows as ever."""
    t = torch()
    K, V = rows(6, 2, 128, "bf16", 8), rows(6, 2, 128, "bf16", 9)
    K[1, 0, 70], K[2, 1, 0], V[3, 0, 127] = float("nan"), float("inf"), -float("inf")
    cache = Q.qkv_cache_new(1, 2, 128, bits=4, group=32, page=16)
    want = check_store(K, V, [0, 1, 2, 3, 4, 5], cache)
    k, v = Q.qkv_cache_load(cache, dev(np.arange(6, dtype=np.int32)))
    for got, ref in zip((k, v), KO.load(want, range(6))):
        assert np.array_equal(np.isnan(host_f64(got)), np.isnan(ref))
    assert int(t.isnan(k).sum()) == 64 and int(t.isnan(v).sum()) == 32


def test_load_parts():
    """Keys or values alone, into given tensors, misaligned ones among them."""
    t = torch()
    cache = Q.qkv_cache_new(2, 3, 128, bits=4, group=64, page=16)
    want = check_store(rows(20, 3, 128, "f16", 10), rows(20, 3, 128, "f16", 11), list(range(20)), cache)
    slots = dev(np.array([4, 19, -7, 0], np.int32))
    k, v = Q.qkv_cache_load(cache, slots, need=(True, False))
    assert v is None
    _, v2 = Q.qkv_cache_load(cache, slots, need=(False, True), out_dtype=t.bfloat16)
    ref = KO.load(want, [4, 19, -7, 0])
    assert_elementwise(host_f64(k), ref[0], 2.0 ** -24 * np.abs(ref[0]), "f32")
    assert_elementwise(host_f64(v2), ref[1], 2.0 ** -24 * np.abs(ref[1]), "bf16")
    for ty in ("f32", "f16"):
        flat = t.full((4 * 3 * 128 + 2,), 9.0, dtype=tt(ty), device="cuda")
        out = flat[1:-1].view(4, 3, 128)
        Q.qkv_cache_load(cache, slots, K=out, need=(True, False))
        assert_elementwise(host_f64(out), ref[0], 2.0 ** -24 * np.abs(ref[0]), ty)
        assert float(flat[0]) == 9.0 and float(flat[-1]) == 9.0


def test_no_tokens():
    t = torch()
    cache = Q.qkv_cache_new(1, 2, 64, page=16)
    e = t.empty(0, 2, 64, device="cuda")
    none = t.empty(0, dtype=t.int32, device="cuda")
    Q.qkv_cache_store(e, e, none, cache)
    k, v = Q.qkv_cache_load(cache, none)
    assert k.shape == v.shape == (0, 2, 64)


def test_graph_and_stream():
    """Store then load, on another stream and captured, with inputs and slots changed between replays."""
    t = torch()
    cache = Q.qkv_cache_new(4, 2, 128, bits=4, group=64, page=16)
    K, V = rows(40, 2, 128, "bf16", 12), rows(40, 2, 128, "bf16", 13)
    slots = dev(np.arange(40, dtype=np.int32))
    out = [t.empty(40, 2, 128, device="cuda") for _ in range(2)]

    def step():
        Q.qkv_cache_store(K, V, slots, cache)
        Q.qkv_cache_load(cache, slots, K=out[0], V=out[1])

    step()
    ref = [host_bits(x).copy() for x in out]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    k2 = Q.qkv_cache_load(cache, slots, stream=side)
    side.synchronize()
    assert all(np.array_equal(host_bits(a), b) for a, b in zip(k2, ref))
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step()
    for k in range(4):
        K.copy_(rows(40, 2, 128, "bf16", 20 + k))
        slots.copy_(dev(np.random.default_rng(k).permutation(64)[:40].astype(np.int32)))
        g.replay()
        t.cuda.synchronize()
        got = [host_bits(x).copy() for x in out]
        step()
        assert all(np.array_equal(a, host_bits(b)) for a, b in zip(got, out)), k
        want = KO.load(host(cache), slots.cpu().numpy())
        assert_elementwise(host_f64(out[0]), want[0], 2.0 ** -24 * np.abs(want[0]), "f32")


def test_refusals():
    t = torch()
    cache = Q.qkv_cache_new(2, 2, 64, page=16)
    K = rows(4, 2, 64, "f16", 14)
    slots = dev(np.arange(4, dtype=np.int32))
    with pytest.raises(ValueError):
        Q.qkv_cache_store(K, K[:3], slots, cache)
    with pytest.raises(ValueError):
        Q.qkv_cache_store(K, K.float(), slots, cache)
    with pytest.raises(ValueError):
        Q.qkv_cache_store(K[:, :1], K[:, :1], slots, cache)
    with pytest.raises(ValueError):
        Q.qkv_cache_store(K.transpose(1, 2), K.transpose(1, 2), slots, cache)
    with pytest.raises(TypeError):
        Q.qkv_cache_store(K, K, slots.long(), cache)
    with pytest.raises(TypeError):
        Q.qkv_cache_store(K.double(), K.double(), slots, cache)
    with pytest.raises(ValueError):
        Q.qkv_cache_store(K, K, slots[:3], cache)
    with pytest.raises(ValueError):
        Q.qkv_cache_store(K.cpu(), K.cpu(), slots, cache)
    with pytest.raises(ValueError):
        Q.qkv_cache_load(dict(cache, v=cache["v"][:1]), slots)
    with pytest.raises(TypeError):
        Q.qkv_cache_load(dict(cache, k_params=cache["k_params"].bfloat16()), slots)
    with pytest.raises(Q.QmmError):
        Q.qkv_cache_load(dict(cache, group=16), slots)
    with pytest.raises(Q.QmmError):
        Q.qkv_cache_load(dict(cache, bits=2), slots)
    with pytest.raises(Q.QmmError):
        Q.qkv_cache_new(2, 2, 64, bits=3)
    with pytest.raises(Q.QmmError):
        Q.qkv_cache_new(2, 2, 64, group=128)
    t.cuda.synchronize()
