"""Operators of fine-tuning and serving low-rank adapters and experts on low-bit weights.

Five operators, each as a user's program calls it:

  lora_add      Y = base + s_a (X A_a^T) B_a^T, every row m with the adapter a = ids[m] of its
                request (none: Y = base), next to the projection whose fp32 output is `base`
  lora_grad     the gradients of lora_add: dX = base + s_a (dY B_a) A_a,
                dA_a = s_a sum_m (dY B_a)^T X, dB_a = s_a sum_m dY^T (X A_a^T)
  dgrad         dX = dY . dequant(W): the input gradient of a frozen low-bit projection
                (blockwise affine codes or a 16-entry codebook)
  grouped       Y[r] = X[r] W_e^T + bias_e, rows grouped by expert, 16-bit weights
  grouped_grad  the gradients of `grouped`: dX = dY W_e, dW_e = dY_e^T X_e, dbias_e = sum dY_e

`own` False computes them in elementary torch operations in 32 bits, True through the
framework's entry points.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one request at a phi4 qkv projection: latency only
        dict(name="lora_add_m1", op="lora_add", M=1, K=5120, N=7680, r=16, L=8, type="bf16", base="f32", out="bf16",
             order="mixed", none=0.0),
        # a decode batch of 32 requests over 64 loaded adapters, some requests without one
        dict(name="lora_add_m32", op="lora_add", M=32, K=5120, N=5120, r=16, L=64, type="f16", base="f32", out="f16",
             order="mixed", none=0.1),
        # chunked prefill of a few requests mixed with decode rows, odd sizes
        dict(name="lora_add_m333", op="lora_add", M=333, K=2880, N=5755, r=24, L=5, type="bf16", base="bf16",
             out="bf16", order="runs", none=0.1),
        # a long prefill batch of eight requests at the gate_up projection
        dict(name="lora_add_m4096", op="lora_add", M=4096, K=5120, N=35840, r=32, L=8, type="bf16", base="f32",
             out="bf16", order="runs", none=0.0),
        # a small fine-tuning step at a 4096 -> 1024 projection
        dict(name="lora_grad_m500", op="lora_grad", M=500, K=4096, N=1024, r=8, L=3, type="f16", base="f32",
             out="f16", order="runs", none=0.0),
        # one adapter's fine-tuning step of 8192 tokens at a square projection
        dict(name="lora_grad_m8192", op="lora_grad", M=8192, K=5120, N=5120, r=16, L=1, type="bf16", base="f32",
             out="bf16", order="runs", none=0.0),
        # codebook weights (4096 -> 14336), a few tokens: the weights are what is read
        dict(name="dgrad_cb_m16", op="dgrad", fmt="codebook", M=16, K=4096, N=14336, bits=4, block=64, zp="none",
             type="bf16", out="bf16"),
        # 4-bit phi4 qkv projection, a training batch of 2048 tokens
        dict(name="dgrad_u4_m2048", op="dgrad", fmt="affine", M=2048, K=5120, N=7680, bits=4, block=64, zp="packed",
             type="bf16", out="bf16"),
        # one 8-token decode step of a 128-expert top-8 layer with 16-bit experts
        dict(name="grouped_t8", op="grouped", T=8, k=8, E=128, K=2048, N=1536, type="f16", out="f16", bias=False,
             skew=0.0),
        # 1024 tokens of a 32-expert top-4 layer's fc1, skewed routing
        dict(name="grouped_t1024", op="grouped", T=1024, k=4, E=32, K=2880, N=5760, type="bf16", out="bf16",
             bias=True, skew=1.0),
        # the backward pass of a 128-expert layer's fc2 for 256 tokens: some experts have no row
        dict(name="grouped_grad_t256", op="grouped_grad", T=256, k=8, E=128, K=768, N=2048, type="f16", out="f16",
             bias=False, skew=1.0),
        # the backward pass of fc1 for 2048 tokens of the 32-expert layer
        dict(name="grouped_grad_t2048", op="grouped_grad", T=2048, k=4, E=32, K=2880, N=5760, type="bf16",
             out="f32", bias=True, skew=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora_add", "lora_grad", "dgrad", "grouped", "grouped_grad"])
    ty = rng.choice(["f16", "bf16"])
    step = rng.choice([1, 8, 64])  # odd sizes, aligned ones, whole tiles

    def size(lo, hi):
        return max(step, _log(rng, lo, hi) // step * step)

    if op in ("lora_add", "lora_grad"):
        M = _log(rng, 1, 8192)
        return dict(op=op, M=M, K=size(256, 8192), N=size(256, 8192), r=rng.choice([1, 4, 8, 16, 24, 32, 64, 100]),
                    L=_log(rng, 1, 96), type=ty, base=rng.choice(["f32", ty]), out=ty,
                    order=rng.choice(["mixed", "runs"]), none=rng.choice([0.0, 0.1, 0.5]))
    if op == "dgrad":
        fmt = rng.choice(["affine", "affine", "codebook"])
        bits = 4 if fmt == "codebook" else rng.choice([2, 3, 4, 8])
        return dict(op=op, fmt=fmt, M=_log(rng, 1, 2048), K=size(256, 8192), N=size(256, 8192), bits=bits,
                    block=rng.choice([32, 64, 128]), zp="none" if fmt == "codebook" else rng.choice(
                        ["none", "packed", "f16", "uniform"]), type=ty, out="bf16")
    E = rng.choice([1, 4, 8, 32, 64, 128])
    return dict(op=op, T=_log(rng, 1, 2048), k=rng.randint(1, min(E, 4)), E=E, K=size(128, 2048), N=size(128, 2048),
                type=ty, out=rng.choice(["f32", ty]), bias=rng.choice([True, False]),
                skew=rng.choice([0.0, 1.0]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ids(case, g):
    """Adapter of each row: runs of a request's tokens, or every row another request's."""
    M, L = case["M"], case["L"]
    if case["order"] == "mixed":
        ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
        none = torch.rand(M, generator=g, device="cuda") < case["none"]
    else:
        cuts = torch.sort(torch.randint(0, M + 1, (max(L, 2) - 1,), generator=g, device="cuda")).values
        run = torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)
        perm = torch.randperm(max(L, 2), generator=g, device="cuda")
        ids = (perm[run] % L).to(torch.int32)
        none = (torch.rand(max(L, 2), generator=g, device="cuda") < case["none"])[run]
    return torch.where(none, torch.full_like(ids, -1), ids)


def _routing(case, g):
    """Rows of each expert as offsets [E + 1], from top-k routing with a popularity term."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, generator=g, device="cuda") - case["skew"] * torch.log1p(
        torch.arange(E, device="cuda", dtype=torch.float32))
    chosen = torch.topk(logits, k, dim=1).indices.reshape(-1)
    counts = torch.zeros(E, device="cuda", dtype=torch.int64).index_add_(
        0, chosen, torch.ones_like(chosen))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)
    return offsets, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    ty = TYPES[case["type"]]

    def randn(*shape, std=1.0, dtype=ty):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case, type=ty, out=TYPES[case["out"]])
    op = case["op"]
    if op in ("lora_add", "lora_grad"):
        M, K, N, r, L = (case[x] for x in ("M", "K", "N", "r", "L"))
        s["ids"] = _ids(case, g)
        s["most"] = max(1, int(torch.bincount(s["ids"].long() + 1, minlength=L + 1)[1:].max()))
        s["X"] = randn(M, K)
        s["A"] = randn(L, r, K, std=K ** -0.5)
        s["B"] = randn(L, N, r, std=0.1)
        s["scale"] = torch.rand(L, generator=g, device="cuda") * 1.5 + 0.5
        if op == "lora_add":
            s["base"] = randn(M, N, dtype=TYPES[case["base"]])
        else:
            s["dY"] = randn(M, N, std=0.05)
            s["T"] = _forward_t(s)
            s["base"] = randn(M, K, std=0.1, dtype=TYPES[case["base"]])
    elif op == "dgrad":
        M, K, N, bits, block = (case[x] for x in ("M", "K", "N", "bits", "block"))
        nblk = -(-K // block)
        s["dY"] = randn(M, N, std=0.05)
        s["W"] = torch.randint(0, 256, (N, nblk, block * bits // 8), generator=g, device="cuda", dtype=torch.uint8)
        if case["fmt"] == "codebook":
            s["absmax"] = torch.rand(N, nblk, generator=g, device="cuda") * 0.09 + 0.01
            s["codebook"] = torch.sort(torch.rand(16, generator=g, device="cuda") * 2 - 1).values
        else:
            s["scales"] = (torch.rand(N, nblk, generator=g, device="cuda") * 0.015 + 0.005).to(torch.float16)
            s["zp"], s["uniform"] = None, 0.0
            if case["zp"] == "packed":
                s["zp"] = torch.randint(0, 256, (N, -(-nblk * bits // 8)), generator=g, device="cuda",
                                        dtype=torch.uint8)
            elif case["zp"] == "f16":
                top = 8.0 if bits == 8 else float(2 ** bits - 1)
                s["zp"] = (torch.rand(N, nblk, generator=g, device="cuda") * top).to(torch.float16)
            elif case["zp"] == "uniform":
                s["uniform"] = 1.5
    else:
        E, K, N = case["E"], case["K"], case["N"]
        s["offsets"], s["most"] = _routing(case, g)
        R = case["T"] * case["k"]
        s["X"] = randn(R, K)
        s["W"] = randn(E, N, K, std=K ** -0.5)
        if op == "grouped":
            s["bias"] = randn(E, N, dtype=s["out"]) if case["bias"] else None
        else:
            s["dY"] = randn(R, N, std=0.05)
    return s


def _forward_t(s):
    """X A^T of every row in 32 bits, which a training program keeps from its forward pass."""
    T = torch.zeros(s["X"].shape[0], s["A"].shape[1], device="cuda")
    for a in range(s["A"].shape[0]):
        rows = torch.nonzero(s["ids"] == a)[:, 0]
        T[rows] = (s["X"][rows].double() @ s["A"][a].double().T).float()
    return T


# ---------------------------------------------------------------------------
# the operators in elementary operations, in 32 bits
# ---------------------------------------------------------------------------

def _slots(group, most):
    """Place of every row in a [groups, most] table: its group, its rank in the group."""
    order = torch.sort(group, stable=True).indices
    sorted_group = group[order]
    first = torch.searchsorted(sorted_group, sorted_group)
    rank = torch.empty_like(group)
    rank[order] = torch.arange(group.numel(), device=group.device) - first
    return group * most + rank


def _spread(x, slot, groups, most):
    """Rows of x at their places of a zero [groups, most, ...] table, in 32 bits; rows of no
    group share one place behind it."""
    t = torch.zeros(groups * most + 1, x.shape[1], device=x.device)
    t[slot] = x.float()
    return t[:-1].view(groups, most, x.shape[1])


def _plain_lora_add(s):
    L, most = s["A"].shape[0], s["most"]
    ids = s["ids"].long()
    has = (ids >= 0).float()[:, None]
    slot = torch.where(ids < 0, L * most, _slots(torch.where(ids < 0, L, ids), most))
    x = _spread(s["X"], slot, L, most)
    t = torch.matmul(x, s["A"].float().transpose(1, 2).contiguous())
    d = torch.matmul(t, s["B"].float().transpose(1, 2).contiguous()) * s["scale"][:, None, None]
    d = torch.cat([d.reshape(L * most, -1), d.new_zeros(1, d.shape[2])])[slot]
    return (s["base"].float() + has * d).to(s["out"])


def _plain_lora_grad(s):
    L, most = s["A"].shape[0], s["most"]
    ids = s["ids"].long()
    has = (ids >= 0).float()[:, None]
    slot = torch.where(ids < 0, L * most, _slots(torch.where(ids < 0, L, ids), most))
    x = _spread(s["X"], slot, L, most)
    dy = _spread(s["dY"], slot, L, most)
    t = _spread(s["T"], slot, L, most)
    sc = s["scale"][:, None, None]
    dt = torch.matmul(dy, s["B"].float()) * sc
    da = torch.matmul(dt.transpose(1, 2).contiguous(), x)
    db = torch.matmul(dy.transpose(1, 2).contiguous(), t) * sc
    dx = torch.matmul(dt, s["A"].float())
    dx = torch.cat([dx.reshape(L * most, -1), dx.new_zeros(1, dx.shape[2])])[slot]
    return (s["base"].float() + has * dx).to(s["out"]), da, db


def _codes(W, bits, K):
    """Codes [N][K] of packed weights: the `bits`-wide fields of each block's bit stream."""
    N, nblk, nbytes = W.shape
    if bits == 8:
        return W.view(torch.int8).reshape(N, -1)[:, :K].float()
    stream = (W[..., None] >> torch.arange(8, device=W.device, dtype=torch.uint8)) & 1
    fields = stream.reshape(N, -1, bits).float()
    weight = 2.0 ** torch.arange(bits, device=W.device)
    return (fields * weight).sum(-1)[:, :K]


def _plain_dgrad(s):
    c = s["case"]
    K, bits, block = c["K"], c["bits"], c["block"]
    q = _codes(s["W"], bits, K)
    blk = torch.arange(K, device="cuda") // block
    if c["fmt"] == "codebook":
        w = s["codebook"][q.long()] * s["absmax"][:, blk]
    else:
        nblk = s["scales"].shape[1]
        if c["zp"] == "packed" and bits == 8:
            z = s["zp"].view(torch.int8).float()[:, :nblk]
        elif c["zp"] == "packed":
            stream = (s["zp"][..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
            fields = stream.reshape(stream.shape[0], -1)[:, :nblk * bits].reshape(-1, nblk, bits).float()
            z = (fields * 2.0 ** torch.arange(bits, device="cuda")).sum(-1)
        elif c["zp"] == "f16":
            z = s["zp"].float()
        else:
            mid = 0.0 if bits == 8 else float(2 ** (bits - 1))
            z = torch.full((1, nblk), s["uniform"] if c["zp"] == "uniform" else mid, device="cuda")
        w = (q - z[:, blk]) * s["scales"].float()[:, blk]
    return torch.matmul(s["dY"].float(), w).to(s["out"])


def _groups(offsets, R):
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(R, device="cuda", dtype=torch.int32), right=True)


def _plain_grouped(s):
    E, most = s["W"].shape[0], s["most"]
    e = _groups(s["offsets"], s["X"].shape[0])
    slot = _slots(e, most)
    y = torch.matmul(_spread(s["X"], slot, E, most), s["W"].float().transpose(1, 2).contiguous())
    y = y.reshape(E * most, -1)[slot]
    if s["bias"] is not None:
        y = y + s["bias"].float()[e]
    return y.to(s["out"])


def _plain_grouped_grad(s):
    E, most = s["W"].shape[0], s["most"]
    e = _groups(s["offsets"], s["X"].shape[0])
    slot = _slots(e, most)
    dy = _spread(s["dY"], slot, E, most)
    x = _spread(s["X"], slot, E, most)
    dx = torch.matmul(dy, s["W"].float()).reshape(E * most, -1)[slot]
    dw = torch.matmul(dy.transpose(1, 2).contiguous(), x)
    out = [dx.to(s["type"]), dw.to(s["out"])]
    if s["case"]["bias"]:
        out.append(dy.sum(1).to(s["out"]))
    return out


# ---------------------------------------------------------------------------
# the operators through the framework
# ---------------------------------------------------------------------------

def _own(s):
    from gemm_qmm_nbits_amd import qmm as Q

    c = s["case"]
    op = c["op"]
    if op == "lora_add":
        return Q.qmm_lora_add(s["X"], s["A"], s["B"], s["ids"], scale=s["scale"], base=s["base"], out_dtype=s["out"])
    if op == "lora_grad":
        return Q.qmm_lora_grad(s["dY"], s["X"], s["A"], s["B"], s["ids"], scale=s["scale"], T=s["T"], base=s["base"],
                               dx_dtype=s["out"], grad_dtype=torch.float32)
    if op == "dgrad":
        if c["fmt"] == "codebook":
            return Q.qmm_codebook4_dgrad(s["dY"], s["W"], s["absmax"], s["codebook"], c["K"], c["block"],
                                         out_dtype=s["out"], f32=True)
        kind = {"none": Q.QMM_ZP_NONE, "packed": Q.QMM_ZP_PACKED, "f16": Q.QMM_ZP_F16,
                "uniform": Q.QMM_ZP_UNIFORM}[c["zp"]]
        return Q.qmm_nbits_dgrad(s["dY"], s["W"], s["scales"], c["K"], c["bits"], c["block"], s["zp"], kind,
                                 s["uniform"], out_dtype=s["out"], f32=True)
    if op == "grouped":
        return Q.qmoe_grouped_mm(s["X"], s["offsets"], s["W"], bias=s["bias"], out_dtype=s["out"])
    dx, dw, db = Q.qmoe_grouped_mm_grad(s["dY"], s["X"], s["offsets"], s["W"], dw_dtype=s["out"],
                                        need_dbias=c["bias"])
    return [dx, dw, db] if c["bias"] else [dx, dw]


def run(s):
    if own:
        return _own(s)
    return {"lora_add": _plain_lora_add, "lora_grad": _plain_lora_grad, "dgrad": _plain_dgrad,
            "grouped": _plain_grouped, "grouped_grad": _plain_grouped_grad}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _used(L, M):
    """Adapters (or experts) that M rows use, of L: what is expected of even choices."""
    return L * (1.0 - (1.0 - 1.0 / L) ** M) if L > 1 else 1.0


def work(case):
    c, size = case, {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] in ("lora_add", "lora_grad"):
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        rows = M * (1.0 - c["none"])
        adapters = _used(c["L"], rows) * r * (K + N) * 2 if rows else 0.0
        if c["op"] == "lora_add":
            io = rows * K * 2 + M * N * (size[c["base"]] + size[c["out"]]) + 4 * M
            return {"bytes": io + adapters, "flops": 2.0 * rows * r * (K + N)}
        io = rows * (K + N) * 2 + rows * r * 4 + M * K * (size[c["base"]] + size[c["out"]]) + 4 * M
        return {"bytes": io + adapters + c["L"] * r * (K + N) * 4, "flops": 4.0 * rows * r * (K + N)}
    if c["op"] == "dgrad":
        M, K, N = c["M"], c["K"], c["N"]
        nblk = -(-K // c["block"])
        w = N * nblk * (c["block"] * c["bits"] / 8 + (4 if c["fmt"] == "codebook" else 2))
        w += N * nblk * {"packed": c["bits"] / 8, "f16": 2}.get(c["zp"], 0)
        return {"bytes": w + M * N * 2 + M * K * size[c["out"]], "flops": 2.0 * M * N * K}
    R, E, K, N = c["T"] * c["k"], c["E"], c["K"], c["N"]
    w = _used(E, R) * N * K * 2
    if c["op"] == "grouped":
        return {"bytes": R * K * 2 + w + R * N * size[c["out"]], "flops": 2.0 * R * K * N}
    return {"bytes": R * (2 * K + N) * 2 + w + E * N * K * size[c["out"]], "flops": 4.0 * R * K * N}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    if op in ("lora_add", "lora_grad"):
        ids = s["ids"].tolist()
        out = s["base"].to(f).clone()
        da = torch.zeros(s["A"].shape, dtype=f, device="cuda")
        db = torch.zeros(s["B"].shape, dtype=f, device="cuda")
        for a in sorted(set(i for i in ids if i >= 0)):
            rows = torch.tensor([m for m, i in enumerate(ids) if i == a], device="cuda")
            A, B, sc = s["A"][a].to(f), s["B"][a].to(f), float(s["scale"][a])
            x = s["X"][rows].to(f)
            if op == "lora_add":
                out[rows] += sc * ((x @ A.T) @ B.T)
            else:
                dy = s["dY"][rows].to(f)
                out[rows] += sc * ((dy @ B) @ A)
                da[a] = sc * ((dy @ B).T @ x)
                db[a] = sc * (dy.T @ s["T"][rows].to(f))
        return out if op == "lora_add" else (out, da, db)
    if op == "dgrad":
        return s["dY"].to(f) @ _exact_weights(case, s)
    offsets = s["offsets"].tolist()
    E, K, N, R = case["E"], case["K"], case["N"], s["X"].shape[0]
    if op == "grouped":
        y = torch.zeros(R, N, dtype=f, device="cuda")
        for e in range(E):
            i, j = offsets[e], offsets[e + 1]
            y[i:j] = s["X"][i:j].to(f) @ s["W"][e].to(f).T
            if case["bias"]:
                y[i:j] += s["bias"][e].to(f)
        return y
    dx = torch.zeros(R, K, dtype=f, device="cuda")
    dw = torch.zeros(E, N, K, dtype=f, device="cuda")
    dbias = torch.zeros(E, N, dtype=f, device="cuda")
    for e in range(E):
        i, j = offsets[e], offsets[e + 1]
        dy = s["dY"][i:j].to(f)
        dx[i:j] = dy @ s["W"][e].to(f)
        dw[e] = dy.T @ s["X"][i:j].to(f)
        dbias[e] = dy.sum(0)
    return [dx, dw, dbias] if case["bias"] else [dx, dw]


def _exact_weights(case, s):
    """The weights [N][K] in 64 bits: code j of a block is the field at bit j * bits of its
    bytes read as one little-endian number."""
    N, nblk, nbytes = s["W"].shape
    bits, block, K = case["bits"], case["block"], case["K"]

    def fields(rows, count):
        """The first `count` fields of each row of bytes."""
        padded = torch.cat([rows.to(torch.int64), rows.new_zeros(rows.shape[0], 1).to(torch.int64)], 1)
        at = torch.arange(count, device="cuda") * bits
        two = padded[:, at // 8] + 256 * padded[:, at // 8 + 1]
        v = torch.remainder(torch.div(two, 2 ** (at % 8), rounding_mode="floor"), 2 ** bits)
        return torch.where(v >= 128, v - 256, v) if bits == 8 else v

    q = fields(s["W"].reshape(N * nblk, nbytes), block).reshape(N, nblk, block)
    if case["fmt"] == "codebook":
        w = s["codebook"].double()[q] * s["absmax"].double()[:, :, None]
    else:
        z = {"none": 0.0 if bits == 8 else 2.0 ** (bits - 1), "uniform": s["uniform"]}.get(case["zp"])
        if case["zp"] == "packed":
            z = fields(s["zp"], nblk).double()[:, :, None]
        elif case["zp"] == "f16":
            z = s["zp"].double()[:, :, None]
        w = (q.double() - z) * s["scales"].double()[:, :, None]
    return w.reshape(N, nblk * block)[:, :K]
