"""One workspace sized for the most rows serves calls of fewer, with the bits of a call that has its own, and no call
writes behind a workspace of exactly its size."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def guarded(n):
    return torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")


def serves(size, most, rows, call):
    """call(rows, ws) -> tensors; size(rows) -> bytes"""
    shared = guarded(size(most))
    for m in rows:
        want = call(m, None)
        exact = guarded(size(m))
        for ws, n in ((exact, size(m)), (shared, size(most))):
            got = call(m, ws[:n])
            assert all(torch.equal(a, b) for a, b in zip(got, want)), m
            assert (ws[n:] == 0xA5).all(), m


ROWS = [1, 17, 100, 290, 297, 600, 1100, 2500]


@pytest.mark.parametrize("K,N", [(16008, 264), (16008, 520), (20480, 1024), (264, 136)])
def test_linear(K, N):
    x, w = torch.randn((2500, K), device="cuda").bfloat16(), (torch.randn((N, K), device="cuda") * 0.02).bfloat16()
    dy = torch.randn((2500, N), device="cuda").bfloat16()
    z = torch.randn((2500, N), device="cuda").bfloat16()
    serves(lambda m: moe.linear_workspace_bytes(m, K, N), 2500, ROWS, lambda m, ws: [moe.linear(x[:m], w, act="silu", ws=ws)])
    serves(lambda m: moe.linear_backward_workspace_bytes(m, K, N), 2500, ROWS,
           lambda m, ws: moe.linear_backward(dy[:m], x[:m], w, z=z[:m], act="gelu", bias=True, ws=ws))
    # a long reduction of dx
    wt = w.t().contiguous()
    serves(lambda m: moe.linear_backward_workspace_bytes(m, N, K), 2500, ROWS,
           lambda m, ws: moe.linear_backward(x[:m], dy[:m], wt, bias=True, ws=ws))


def test_grouped():
    K, N = 264, 136
    x, dy, w = (torch.randn(s, device="cuda").bfloat16() for s in ((5000, K), (5000, N), (2, N, K)))

    def call(m, ws):
        o = torch.tensor([0, m // 3, m], dtype=torch.int32, device="cuda")
        return moe.grouped_mm_backward(dy[:m], x[:m], w, o, ws=ws)

    serves(lambda m: moe.grouped_mm_backward_workspace_bytes(m, K, 2, N), 5000, ROWS + [5000], call)


@pytest.mark.parametrize("cols", [96, 1001, 5120, 9000, 20001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm(cols, dtype):
    x, dy = torch.randn((2500, cols), device="cuda").to(dtype), torch.randn((2500, cols), device="cuda").to(dtype)
    g = torch.randn(cols, device="cuda")
    _, mean, rstd = moe.layer_norm(x, g, stats=True)
    serves(lambda m: moe.layer_norm_backward_workspace_bytes(m, cols), 2500, ROWS + [147, 148, 296, 304],
           lambda m, ws: moe.layer_norm_backward(dy[:m], x[:m], g, mean[:m], rstd[:m], ws=ws))
