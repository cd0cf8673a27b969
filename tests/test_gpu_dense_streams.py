"""Calls on a stream that is not the current one take no memory that the current stream may still be working on, and their
outputs may be used on the current stream and dropped at once."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu

ROWS, COLS = 2048, 2048


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def calls():
    """name -> call(stream), with operands that are there already"""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((ROWS, COLS), generator=gen).bfloat16().cuda()
    w = (torch.randn((2, COLS, COLS), generator=gen) * 0.02).bfloat16().cuda()
    o = torch.tensor([0, 100, ROWS], dtype=torch.int32, device="cuda")
    _, mean, rstd = moe.layer_norm(x, stats=True)
    w0 = w[0].contiguous()
    return {"linear": lambda s: list(moe.linear(x, w0, act="silu", save_z=True, stream=s)),
            "linear_backward": lambda s: list(moe.linear_backward(x, x, w0, z=x, act="relu", bias=True, stream=s)),
            "grouped_mm": lambda s: [moe.grouped_mm(x, w, o, stream=s)],
            "grouped_mm_backward": lambda s: list(moe.grouped_mm_backward(x, x, w, o, stream=s)),
            "layer_norm": lambda s: list(moe.layer_norm(x, stats=True, stream=s)),
            "layer_norm_backward": lambda s: list(moe.layer_norm_backward(x, x, None, mean, rstd, need_params=True,
                                                                          stream=s))}


NAMES = ["linear", "linear_backward", "grouped_mm", "grouped_mm_backward", "layer_norm", "layer_norm_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_the_current_stream_still_uses(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None)
    for _ in range(4):
        src = [torch.full((ROWS, COLS), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
        dst = torch.empty((6, ROWS, COLS), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)           # the current stream: about 10 ms, then the copies
        for i in range(6):
            dst[i].copy_(src[i])
        del src                                 # given back with the copies still to run
        got = call(side)                        # the side stream starts at once
        side.synchronize()
        torch.cuda.synchronize()
        assert (dst == 3).all()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_used_on_the_current_stream_and_dropped(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    kept = []
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(5_000_000)
        kept.append([t.clone() for t in got])   # still to run when the outputs are dropped
        del got
        with torch.cuda.stream(side):           # work of the side stream that would take the blocks
            junk = [torch.full((ROWS, COLS), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(6)]
            del junk
    torch.cuda.synchronize()
    for got in kept:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
