"""Workspaces of the 16-bit operators serve fewer rows than they were sized for (no GPU needed): the sizes never fall as
the rows grow, and the calls accept the larger workspace."""
import random

import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from tests.test_dense_arguments import NO_DEVICE, grouped_backward, lib, linear, linear_backward, norm_backward  # noqa: F401

ROWS = [0, 1, 2, 7, 8, 9, 33, 64, 100, 147, 148, 149, 200, 295, 296, 297, 400, 600, 1000, 1024, 1500, 2368, 2369, 4096, 5000,
        9472, 18944, 18945, 32768, 10 ** 6, (1 << 25) - 1]
SHAPES = [(8, 8), (64, 128), (264, 264), (40, 16008), (16008, 264), (16008, 520), (5120, 5120), (20480, 5120), (5120, 20480),
          (1032, 584), (72, 1000), (524288, 8)]


def sizes(K, N, E):
    rng = random.Random(K * 7 + N)
    rows = sorted(ROWS + [rng.randrange(1, 20000) for _ in range(60)])
    rows = [m for m in rows if m * max(K, N) < 1 << 40]
    yield "linear", [moe.linear_workspace_bytes(m, K, N) for m in rows], rows
    yield "linear_backward", [moe.linear_backward_workspace_bytes(m, K, N) for m in rows], rows
    yield "grouped_mm_backward", [moe.grouped_mm_backward_workspace_bytes(m, K, E, N) for m in rows], rows
    cols = min(max(1, K + N % 7), 28672)
    yield "layer_norm_backward", [moe.layer_norm_backward_workspace_bytes(m, cols) for m in rows], rows


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("E", [1, 2, 40])
def test_sizes_never_fall_with_more_rows(lib, K, N, E):  # noqa: F811
    for name, v, rows in sizes(K, N, E):
        assert v[0] > 0
        for i in range(1, len(v)):
            assert v[i] >= v[i - 1], (name, rows[i - 1], v[i - 1], rows[i], v[i])


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder device pointers: host-only checks, no GPU")
def test_calls_take_a_workspace_for_more_rows(lib):  # noqa: F811
    for K, N in SHAPES:
        most = 8192
        for m in (1, 100, 200, 297, 400, 600, 1000, 5000):
            kw = dict(M=m, K=K, N=N)
            assert linear(lib, ws_bytes=moe.linear_workspace_bytes(most, K, N), **kw) in NO_DEVICE
            assert linear_backward(lib, ws_bytes=moe.linear_backward_workspace_bytes(most, K, N), **kw) in NO_DEVICE
            n = moe.grouped_mm_backward_workspace_bytes(most, K, 2, N)
            assert grouped_backward(lib, ws_bytes=n, E=2, **kw) in NO_DEVICE
            cols = min(K, 28672)
            assert norm_backward(lib, ws_bytes=moe.layer_norm_backward_workspace_bytes(most, cols), rows=m,
                                 cols=cols) in NO_DEVICE


def test_parts_stay_within_a_tile_a_pair(lib):  # noqa: F811
    """The parts add at most 74 tiles of 256 x 256 FP32 values to a product (19.4 MB)."""
    for K, N in SHAPES:
        for m in ROWS:
            if m * max(K, N) < 1 << 40:
                assert moe.linear_workspace_bytes(m, K, N) <= 74 * 65536 * 4 + 4096
                assert moe.grouped_mm_backward_workspace_bytes(m, K, 3, N) <= 74 * 65536 * 4 + 8192
