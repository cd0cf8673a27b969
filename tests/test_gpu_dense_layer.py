"""The 16-bit operators together, as a layer uses them: norm, router, experts' products over the routed rows,
combine, dense product with the residual stream, and the backward pass through all of it, against an
FP64 computation of the same layer with the same routing.

Tolerance.  Each 16-bit rounding perturbs a tensor by at most 2^-8 of its norm; the maps between are random
matrices and activations with slopes below 1.13, which pass a perturbation on at about the scale of the
signal.  Forward takes 8 roundings on the longest path, backward 8 more: relative Frobenius error below
12 * 2^-8 and 24 * 2^-8."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def rel(got, want):
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    return float((g - w).norm() / w.norm())


class Layer:
    """E SwiGLU experts behind a router, an output projection, the residual stream."""

    def __init__(self, E=12, topk=3, H=256, I=136, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.cfg = moe.make_cfg(E, 1, 1, topk, H, 128, 1.0)
        bf = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).bfloat16().cuda()  # noqa: E731
        self.gate, self.up, self.down = bf(E, I, H), bf(E, I, H), bf(E, H, I)
        self.wo = bf(H, H)
        self.bo = (0.1 * torch.randn(H, generator=g)).cuda()
        self.gamma = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
        self.router = (torch.randn((E, H), generator=g) * 0.3).cuda()

    def forward(self, x0):
        c, T = self.cfg, x0.shape[0]
        s = {"x0": x0}
        s["x"], _, s["rstd"] = moe.layer_norm(x0, self.gamma, rms=True, stats=True)
        idx, s["wts"] = moe.route(c, s["x"], self.router)
        flat = idx.view(-1).long()
        order = torch.argsort(flat, stable=True)
        s["idx"], s["order"], s["token"] = idx, order, order // c.topk
        s["off"] = torch.zeros(c.E + 1, dtype=torch.int32, device="cuda")
        s["off"][1:] = torch.cumsum((flat[:, None] == torch.arange(c.E, device="cuda")).sum(0), 0)
        s["xs"] = s["x"][s["token"]].contiguous()
        s["g"] = moe.grouped_mm(s["xs"], self.gate, s["off"])
        s["u"] = moe.grouped_mm(s["xs"], self.up, s["off"])
        s["h"] = (torch.nn.functional.silu(s["g"].float()) * s["u"].float()).bfloat16()
        s["y"] = moe.grouped_mm(s["h"], self.down, s["off"])
        s["w"] = s["wts"].view(-1)[order]
        pos = torch.empty_like(order)
        pos[order] = torch.arange(order.numel(), device="cuda")
        s["o"] = moe.ep_combine(s["y"].float() * s["w"][:, None], pos.int(), T, c.topk)
        return moe.linear(s["o"], self.wo, bias=self.bo, residual=x0), s

    def backward(self, dout, s):
        do, dwo, dbo = moe.linear_backward(dout, s["o"], self.wo, bias=True)
        dy = (do[s["token"]].float() * s["w"][:, None]).bfloat16()
        dh, ddown = moe.grouped_mm_backward(dy, s["h"], self.down, s["off"])
        g, u, d = s["g"].float(), s["u"].float(), dh.float()
        sg = torch.sigmoid(g)
        dg = (d * u * sg * (1 + g * (1 - sg))).bfloat16()
        du = (d * g * sg).bfloat16()
        dxs, dgate = moe.grouped_mm_backward(dg, s["xs"], self.gate, s["off"])
        dxs2, dup = moe.grouped_mm_backward(du, s["xs"], self.up, s["off"])
        dx = torch.zeros((s["x0"].shape), device="cuda").index_add_(0, s["token"], dxs.float() + dxs2.float())
        dx0, dgamma, _ = moe.layer_norm_backward(dx.bfloat16(), s["x0"], self.gamma, None, s["rstd"], rms=True)
        return {"x0": dx0 + dout, "gamma": dgamma, "gate": dgate, "up": dup, "down": ddown, "wo": dwo, "bo": dbo}

    def reference(self, x0, dout, idx, wts):
        leaf = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
        p = {n: leaf(getattr(self, n)) for n in ("gamma", "gate", "up", "down", "wo", "bo")}
        p["x0"] = leaf(x0)
        x = p["x0"] * torch.rsqrt(p["x0"].square().mean(1, keepdim=True) + 1e-5) * p["gamma"]
        out = torch.zeros_like(x)
        idx, wts = idx.cpu().long(), wts.double().cpu()
        for j in range(self.cfg.topk):
            e = idx[:, j]
            gu = [torch.einsum("th,tih->ti", x, p[n][e]) for n in ("gate", "up")]
            out = out + wts[:, j, None] * torch.einsum("ti,thi->th", torch.nn.functional.silu(gu[0]) * gu[1],
                                                       p["down"][e])
        final = out @ p["wo"].t() + p["bo"] + p["x0"]
        final.backward(dout.double().cpu())
        return final, {n: t.grad for n, t in p.items()}


@pytest.mark.parametrize("T", [1, 7, 150, 700])
def test_layer_forward_and_backward(T):
    layer = Layer(seed=T)
    gen = torch.Generator().manual_seed(T)
    x0 = (torch.randn((T, 256), generator=gen) * 2).bfloat16().cuda()
    dout = torch.randn((T, 256), generator=gen).bfloat16().cuda()
    out, s = layer.forward(x0)
    grads = layer.backward(dout, s)
    want, want_grads = layer.reference(x0, dout, s["idx"], s["wts"])
    assert rel(out, want) < 12 * 2.0 ** -8
    for n, g in grads.items():
        if want_grads[n].norm() > 0:
            assert rel(g, want_grads[n]) < 24 * 2.0 ** -8, n
    # experts no token went to have no gradient
    used = torch.zeros(layer.cfg.E, dtype=torch.bool)
    used[s["idx"].cpu().view(-1).long()] = True
    for n in ("gate", "up", "down"):
        assert (grads[n][~used.cuda()] == 0).all()


def test_layer_in_a_graph():
    """The library's calls of the forward and backward pass captured once and replayed on new rows."""
    layer = Layer(seed=3)
    x0 = torch.randn((90, 256), device="cuda").bfloat16()
    dout = torch.randn((90, 256), device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.backward(dout, layer.forward(x0)[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, s = layer.forward(x0)
        grads = layer.backward(dout, s)
    for seed in (1, 2):
        torch.manual_seed(seed)
        x0.copy_(torch.randn((90, 256), device="cuda"))
        dout.copy_(torch.randn((90, 256), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want_out, want_s = layer.forward(x0)
        want = layer.backward(dout, want_s)
        assert torch.equal(out, want_out)
        for n in ("gate", "up", "down", "wo", "bo"):
            assert torch.equal(grads[n], want[n]), n
        # index_add_ adds a token's rows in no fixed order
        assert rel(grads["x0"], want["x0"]) < 2.0 ** -8 and rel(grads["gamma"], want["gamma"]) < 2.0 ** -8


def test_two_streams_at_once():
    """Calls with workspaces of their own run beside each other."""
    layer = Layer(seed=4, E=8, H=512, I=264)
    xs = [torch.randn((300, 512), device="cuda").bfloat16() for _ in range(2)]
    offs = [torch.tensor([0, 10, 10, 60, 100, 180, 200, 299, 300], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 100, 140, 141, 150, 160, 240, 250, 290], dtype=torch.int32, device="cuda")]
    dys = [torch.randn((300, 264), device="cuda").bfloat16() for _ in range(2)]

    def work(i):
        y = torch.zeros((300, 264), dtype=torch.bfloat16, device="cuda")
        dx = torch.zeros((300, 512), dtype=torch.bfloat16, device="cuda")
        moe.grouped_mm(xs[i], layer.gate, offs[i], out=y)
        _, dw = moe.grouped_mm_backward(dys[i], xs[i], layer.gate, offs[i], dx=dx)
        z, m, r = moe.layer_norm(xs[i], stats=True)
        db = moe.linear_backward(dys[i], xs[i], layer.gate[0], z=y, act="gelu", bias=True)
        return [y, dx, dw, z, *moe.layer_norm_backward(xs[i], z, None, m, r, need_params=True), *db]

    alone = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(work(i))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_host_threads():
    """Calls from two host threads, each on a stream of its own."""
    import threading
    w = torch.randn((6, 264, 512), device="cuda").bfloat16()
    x = torch.randn((400, 512), device="cuda").bfloat16()
    dy = torch.randn((400, 264), device="cuda").bfloat16()
    o = torch.tensor([0, 3, 90, 90, 300, 301, 400], dtype=torch.int32, device="cuda")

    def work():
        y, (dx, dw) = moe.grouped_mm(x, w, o), moe.grouped_mm_backward(dy, x, w, o)
        z, m, r = moe.layer_norm(x, stats=True)
        return [y, dx, dw, z, moe.linear(x[:5], w[0]), *moe.linear_backward(dy, x, w[0], z=y, act="silu", bias=True),
                *moe.layer_norm_backward(x, z, None, m, r, need_params=True)]

    want = work()
    torch.cuda.synchronize()
    errors = []

    def run():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(40):
                    got = work()
                s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        except BaseException as e:      # noqa: BLE001  reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements (a row's offset passes 32 bits): sampled rows against FP64."""
    torch.cuda.empty_cache()
    M, K, N = (1 << 20) + 5, 64, 4104                     # y: 4.3e9 elements
    x = torch.randn((M, K), device="cuda").bfloat16()
    w = torch.randn((N, K), device="cuda").bfloat16()
    y = moe.linear(x, w)
    rows = torch.tensor([0, 1, 523264, 523265, M // 2, M - 2, M - 1], device="cuda")
    want = x[rows].double() @ w.double().t()
    assert rel(y[rows], want) < 2.0 ** -8
    dx, dw, db = moe.linear_backward(y, x, w, bias=True)
    assert rel(dx[rows], y[rows].double() @ w.double()) < 2.0 ** -8
    cols = torch.arange(0, N, 700, device="cuda")
    yc = y[:, cols].double()
    assert rel(dw[cols], yc.t() @ x.double()) < 2.0 ** -8
    # FP32 sums of 2^20 terms in blocks: relative to the column's magnitude
    assert float(((db[cols] - yc.sum(0)).abs() / yc.abs().sum(0)).max()) < 2.0 ** -18
    del x, w, y, dx, dw, yc
    E, N, K = 40, 8192, 8192                              # w, dw: 2.7e9 elements
    torch.cuda.empty_cache()
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = torch.randn((N, K), device="cuda") * K ** -0.5
    counts = [5] * E
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    x = torch.randn((5 * E, K), device="cuda").bfloat16()
    y = moe.grouped_mm(x, w, off)
    dx, dw = moe.grouped_mm_backward(y, x, w, off)
    for e in (0, 31, 32, E - 1):
        r = slice(5 * e, 5 * e + 5)
        assert rel(y[r], x[r].double() @ w[e].double().t()) < 2.0 ** -8
        assert rel(dx[r], y[r].double() @ w[e].double()) < 2.0 ** -8
        assert rel(dw[e], y[r].double().t() @ x[r].double()) < 2.0 ** -8
    del w, dw
    torch.cuda.empty_cache()
    x = torch.randn((80001, 28671), device="cuda", dtype=torch.bfloat16)          # 2.3e9 elements
    y, m, r = moe.layer_norm(x, stats=True)
    dx, dg, db = moe.layer_norm_backward(y, x, None, m, r, need_params=True)
    rows = torch.tensor([0, 74899, 74900, 80000], device="cuda")
    X = x[rows].double()
    c = X - X.mean(1, keepdim=True)
    want = c * torch.rsqrt(c.square().mean(1, keepdim=True) + 1e-5)
    assert rel(y[rows], want) < 2.0 ** -8
    # the gradient along xh itself nearly vanishes: bounded by the rounding of its terms
    assert float(dx[rows].abs().max()) < 2.0 ** -5
