"""The 16-bit operators around the quantised expert layer, as measured cases: ragged products grouped by
expert, the dense product with its epilogue, and the layer norm, each with its backward pass.

``own`` false: the plain forms, in elementary FP32 torch operations.  ``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
#: no drawn case costs more than the largest listed ones
MOST_FLOPS = 8.5e11
MOST_BYTES = 1.6e9


def listed():
    return [
        # one rank of four holds 64 of 256 experts; a decode step of 16 tokens sends it 32 rows for the up projection
        dict(name="grouped_decode", op="grouped", dtype="bf16", E=64, M=32, K=5120, N=2560, skew=0.5),
        # the same rank's down projection in a long prefill, every expert busy and some much busier
        dict(name="grouped_prefill", op="grouped", dtype="bf16", E=64, M=32768, K=2560, N=5120, skew=0.5),
        # a fine-tuning step over 32 experts: both gradients of the up projection
        dict(name="grouped_backward", op="grouped_backward", dtype="bf16", E=32, M=8192, K=5120, N=2560, skew=0.6),
        # a small FP16 layer with odd sizes; the skew leaves experts without a row
        dict(name="grouped_backward_odd", op="grouped_backward", dtype="fp16", E=13, M=1531, K=520, N=776, skew=2.5),
        # one token through the dense layers' down projection, added to the residual stream
        dict(name="linear_token", op="linear", dtype="bf16", M=1, K=20480, N=5120, act="none", bias=False,
             residual=True, save_z=False),
        # a prefill batch through the dense up projection, pre-activation kept for the backward pass
        dict(name="linear_prefill", op="linear", dtype="bf16", M=4096, K=5120, N=20480, act="gelu", bias=True,
             residual=False, save_z=True),
        # backward of a square projection with a SiLU and a bias
        dict(name="linear_backward", op="linear_backward", dtype="bf16", M=4096, K=5120, N=5120, act="silu", bias=True),
        # backward of a small FP16 projection with odd sizes
        dict(name="linear_backward_odd", op="linear_backward", dtype="fp16", M=333, K=1032, N=584, act="gelu_tanh",
             bias=True),
        # the RMS norm of a decode step's 16 tokens: launch latency
        dict(name="norm_decode", op="norm", dtype="bf16", rows=16, cols=5120, rms=True, affine=True),
        # an FP32 layer norm of odd width over a long batch
        dict(name="norm_odd", op="norm", dtype="fp32", rows=8191, cols=2571, rms=False, affine=True),
        # backward of a small FP16 layer norm
        dict(name="norm_backward_small", op="norm_backward", dtype="fp16", rows=129, cols=1000, rms=False, affine=True),
        # backward of the layer norm over a training batch of 32768 tokens
        dict(name="norm_backward", op="norm_backward", dtype="bf16", rows=32768, cols=5120, rms=False, affine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grouped", "grouped", "grouped_backward", "linear", "linear", "linear_backward", "norm",
                     "norm_backward"))
    while True:
        if op.startswith("norm"):
            c = dict(op=op, dtype=rng.choice(("bf16", "fp16", "fp32")), rows=_log(rng, 1, 32768),
                     cols=_log(rng, 64, 20480), rms=rng.random() < 0.5, affine=rng.random() < 0.8)
        else:
            c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp16")))
            if op.startswith("grouped"):
                c.update(E=_log(rng, 1, 64), M=_log(rng, 1, 32768))
            else:
                c.update(M=_log(rng, 1, 32768))
            # rows of 16-bit operands are multiples of 16 bytes
            c.update(K=8 * _log(rng, 8, 2560), N=8 * _log(rng, 8, 2560))
            if op.startswith("grouped"):
                c.update(skew=rng.choice((0.0, 0.4, 0.8, 1.5)))
            else:
                c.update(act=rng.choice(ACTS), bias=rng.random() < 0.6)
                if op == "linear":
                    c.update(residual=rng.random() < 0.5, save_z=rng.random() < 0.3)
        w = work(c)
        if w["flops"] > MOST_FLOPS or w["bytes"] > MOST_BYTES:
            continue
        if "E" in c:
            # the plain form pads every expert to the busiest one's rows
            padded = c["E"] * max(_counts(c))
            if padded * c["K"] * c["N"] > 2e12 or padded * (c["K"] + c["N"]) > 4e9:
                continue
        return c


def _counts(case):
    """Rows per expert in descending order: shares proportional to (rank + 1)^-skew, rounded down, the rest one
    each to the first half of the experts (so some may have none)."""
    E, M = case["E"], case["M"]
    share = [(r + 1.0) ** -case["skew"] for r in range(E)]
    total = sum(share)
    counts = [int(M * s / total) for s in share]
    rest = M - sum(counts)
    for r in range(rest):
        counts[r % (E - E // 2)] += 1
    return counts


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, b = case["rows"] * case["cols"], {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        stats = 4 * case["rows"] * (1 if case["rms"] else 2)
        vecs = 4 * case["cols"] * ((1 if case["rms"] else 2) if case["affine"] else 0)
        if op == "norm":
            return {"bytes": 2 * n * b + stats + vecs, "flops": 8 * n}
        gamma = 4 * case["cols"] if case["affine"] else 0
        return {"bytes": 3 * n * b + stats + gamma + vecs, "flops": 16 * n}
    M, K, N = case["M"], case["K"], case["N"]
    mm = 2 * M * K * N
    if op.startswith("grouped"):
        busy = sum(1 for c in _counts(case) if c)
        idx = 4 * (case["E"] + 1)
        if op == "grouped":
            return {"bytes": 2 * (M * K + M * N + busy * N * K) + idx, "flops": mm}
        return {"bytes": 2 * (2 * M * K + M * N + (busy + case["E"]) * N * K) + idx, "flops": 2 * mm}
    if op == "linear":
        outs = 1 + (1 if case["residual"] else 0) + (1 if case["save_z"] else 0)
        return {"bytes": 2 * (M * K + N * K + outs * M * N) + (4 * N if case["bias"] else 0), "flops": mm}
    ins = 2 if case["act"] != "none" else 1
    return {"bytes": 2 * (2 * M * K + 2 * N * K + ins * M * N) + (4 * N if case["bias"] else 0), "flops": 2 * mm}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    s = {"case": dict(case)}
    op = case["op"]
    if op.startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        # a residual stream of RMS about 3, a few channels twenty times the others
        chan = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        s["x"] = (torch.randn((rows, cols), generator=g, device="cuda") * 3.0 * chan + 0.3).to(dt)
        s["gamma"] = s["beta"] = None
        if case["affine"]:
            s["gamma"] = 1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")
            if not case["rms"]:
                s["beta"] = 0.1 * torch.randn(cols, generator=g, device="cuda")
        s["eps"] = 1e-5
        if op == "norm_backward":
            s["dy"] = rand(rows, cols)
            # the statistics the forward pass saved
            x = s["x"].double()
            mean = x.mean(1, keepdim=True) if not case["rms"] else 0.0
            s["rstd"] = torch.rsqrt((x - mean).square().mean(1) + s["eps"]).float()
            s["mean"] = mean[:, 0].float() if not case["rms"] else None
        return s
    M, K, N = case["M"], case["K"], case["N"]
    s["x"] = rand(M, K)
    if op.startswith("grouped"):
        E = case["E"]
        counts = _counts(case)
        random.Random(seed).shuffle(counts)
        s["counts"] = counts
        s["rows_max"] = max(counts)
        offs = [0]
        for c in counts:
            offs.append(offs[-1] + c)
        s["offsets"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((E, N, K), dtype=dt, device="cuda")
        for e in range(E):
            s["w"][e] = rand(N, K, scale=K ** -0.5)
        if op == "grouped_backward":
            s["dy"] = rand(M, N)
        return s
    s["w"] = rand(N, K, scale=K ** -0.5)
    s["bias"] = 0.5 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
    if op == "linear":
        s["residual"] = rand(M, N, scale=3.0) if case["residual"] else None
    else:
        s["dy"] = rand(M, N)
        s["z"] = rand(M, N) if case["act"] != "none" else None
    return s


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _padded(t, s):
    """The rows of each expert as a batch [E, rows_max, ...], zeros behind them, and the rows' places in it."""
    off = s["offsets"].long()
    row = torch.arange(t.shape[0], device=t.device)
    e = torch.bucketize(row, off[1:], right=True)
    place = e * s["rows_max"] + row - off[e]
    batch = torch.zeros((len(s["counts"]) * s["rows_max"], t.shape[1]), device=t.device)
    batch[place] = t.float()
    return batch.view(len(s["counts"]), s["rows_max"], t.shape[1]), place


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    dt = s["x"].dtype
    if own:
        import nvfp4_quantized_moe_group_b200 as moe
        if op == "grouped":
            return moe.grouped_mm(s["x"], s["w"], s["offsets"])
        if op == "grouped_backward":
            return moe.grouped_mm_backward(s["dy"], s["x"], s["w"], s["offsets"])
        if op == "linear":
            return moe.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"],
                              save_z=case["save_z"])
        if op == "linear_backward":
            return moe.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], act=case["act"], bias=case["bias"])
        if op == "norm":
            return moe.layer_norm(s["x"], s["gamma"], s["beta"], eps=s["eps"], rms=case["rms"], stats=True)
        return moe.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], rms=case["rms"])
    if op == "grouped":
        xb, place = _padded(s["x"], s)
        return torch.bmm(xb, s["w"].float().transpose(1, 2)).flatten(0, 1)[place].to(dt)
    if op == "grouped_backward":
        xb, place = _padded(s["x"], s)
        db, _ = _padded(s["dy"], s)
        return torch.bmm(db, s["w"].float()).flatten(0, 1)[place].to(dt), torch.bmm(db.transpose(1, 2), xb).to(dt)
    x = s["x"].float()
    if op == "linear":
        z = x @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return (y.to(dt), z.to(dt)) if case["save_z"] else y.to(dt)
    if op == "linear_backward":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"].float(), case["act"])
        return (dz @ s["w"].float()).to(dt), (dz.t() @ x).to(dt), dz.sum(0) if case["bias"] else None
    if op == "norm":
        mean = x.mean(1, keepdim=True) if not case["rms"] else None
        c = x - mean if mean is not None else x
        rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + s["eps"])
        y = c * rstd
        if s["gamma"] is not None:
            y = y * s["gamma"]
        if s["beta"] is not None:
            y = y + s["beta"]
        return y.to(dt), mean[:, 0] if mean is not None else None, rstd[:, 0]
    dy, r = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None] if s["mean"] is not None else x) * r
    g = dy * s["gamma"] if s["gamma"] is not None else dy
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    affine = s["gamma"] is not None
    return ((dx * r).to(dt), (dy * xh).sum(0) if affine else None,
            dy.sum(0) if affine and s["mean"] is not None else None)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f8 = torch.float64
    X = s["x"].to(f8)
    if op.startswith("grouped"):
        M, K, N, E = case["M"], case["K"], case["N"], case["E"]
        begin = 0
        y = torch.empty((M, N), dtype=f8, device="cuda")
        dx = torch.empty((M, K), dtype=f8, device="cuda")
        dw = []
        for e, c in enumerate(s["counts"]):
            rows = slice(begin, begin + c)
            W = s["w"][e].to(f8)
            if op == "grouped":
                y[rows] = torch.einsum("mk,nk->mn", X[rows], W)
            else:
                D = s["dy"][rows].to(f8)
                dx[rows] = torch.einsum("mn,nk->mk", D, W)
                dw.append(torch.einsum("mn,mk->nk", D, X[rows]))
            begin += c
        return y if op == "grouped" else (dx, torch.stack(dw))
    if op.startswith("linear"):
        W = s["w"].to(f8)
        act = case["act"]

        def f(z):
            if act == "relu":
                return z.clamp(min=0)
            if act == "silu":
                return z * torch.sigmoid(z)
            if act == "gelu":
                return z * torch.special.ndtr(z)
            if act == "gelu_tanh":
                return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            return z

        if op == "linear":
            z = torch.einsum("mk,nk->mn", X, W)
            if s["bias"] is not None:
                z += s["bias"].to(f8)
            y = f(z)
            if s["residual"] is not None:
                y = y + s["residual"].to(f8)
            return (y, z) if case["save_z"] else y
        dz = s["dy"].to(f8)
        if act != "none":
            z = s["z"].to(f8).requires_grad_(True)
            dz, = torch.autograd.grad(f(z), z, dz)
        return (torch.einsum("mn,nk->mk", dz, W), torch.einsum("mn,mk->nk", dz, X),
                dz.sum(0) if case["bias"] else None)
    G = s["gamma"].to(f8) if s["gamma"] is not None else torch.ones(case["cols"], dtype=f8, device="cuda")
    if op == "norm":
        mean = X.mean(1) if not case["rms"] else None
        var = X.var(1, unbiased=False) if mean is not None else X.square().mean(1)
        rstd = (var + s["eps"]).rsqrt()
        y = (X if mean is None else X - mean[:, None]) * rstd[:, None] * G
        if s["beta"] is not None:
            y = y + s["beta"].to(f8)
        return y, mean, rstd
    D, R = s["dy"].to(f8), s["rstd"].to(f8)[:, None]
    H = (X if s["mean"] is None else X - s["mean"].to(f8)[:, None]) * R
    A = D * G
    back = A * case["cols"] - H * (A * H).sum(1, keepdim=True)
    if s["mean"] is not None:
        back = back - A.sum(1, keepdim=True)
    affine = s["gamma"] is not None
    return (back * R / case["cols"], (D * H).sum(0) if affine else None,
            D.sum(0) if affine and s["mean"] is not None else None)
