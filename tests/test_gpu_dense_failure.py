"""Failure detection of the 16-bit products without a GPU fault: one CTA of each product kernel brings in no operands
(the call's test hook), so the waits for them run out after a 5 ms limit.  A caller sees NVFP4MOE_ERR_TIMEOUT soon after
the limit, and the next call on the same workspace gives the clean call's bits."""
import threading
import time

import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _defaults():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()
    yield
    moe.product_debug()


def rand(seed, *shape, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16().cuda()


def offsets(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def case_few_rows():                     # single CTAs, a tile's reduction shared by a cluster
    x, w = rand(1, 3, 5120), rand(2, 512, 5120, scale=0.01)
    ws = torch.zeros(moe.linear_workspace_bytes(3, 5120, 512), dtype=torch.uint8, device="cuda")
    return ws, lambda: [moe.linear(x, w, act="silu", ws=ws)]


def case_many_columns():                 # single CTAs, several tiles each
    x, w = rand(3, 40, 64), rand(4, 40960, 64, scale=0.1)
    ws = torch.zeros(moe.linear_workspace_bytes(40, 64, 40960), dtype=torch.uint8, device="cuda")
    return ws, lambda: [moe.linear(x, w, ws=ws)]


def case_pairs():                        # pairs, several tiles each
    x, w = rand(5, 2048, 640), rand(6, 5120, 640, scale=0.04)
    ws = torch.zeros(moe.linear_workspace_bytes(2048, 640, 5120), dtype=torch.uint8, device="cuda")
    return ws, lambda: list(moe.linear(x, w, act="gelu", save_z=True, ws=ws))


def case_parts():                        # pairs that share a tile's reduction, then a join
    x, w = rand(7, 600, 16008), rand(8, 264, 16008, scale=0.01)
    ws = torch.zeros(moe.linear_workspace_bytes(600, 16008, 264), dtype=torch.uint8, device="cuda")
    return ws, lambda: [moe.linear(x, w, ws=ws)]


def case_grouped():
    x, w, o = rand(9, 900, 256), rand(10, 5, 520, 256, scale=0.06), offsets(0, 300, 300, 310, 800, 900)
    ws = torch.zeros(moe.grouped_mm_workspace_bytes(5), dtype=torch.uint8, device="cuda")
    return ws, lambda: [moe.grouped_mm(x, w, o, ws=ws)]


def case_grouped_backward():
    x, w, dy, o = rand(11, 900, 256), rand(12, 5, 520, 256), rand(13, 900, 520), offsets(0, 300, 300, 310, 800, 900)
    ws = torch.zeros(moe.grouped_mm_backward_workspace_bytes(900, 256, 5, 520), dtype=torch.uint8, device="cuda")
    return ws, lambda: list(moe.grouped_mm_backward(dy, x, w, o, ws=ws))


def case_linear_backward():              # dw in parts
    x, w, dy = rand(14, 4000, 264), rand(15, 136, 264), rand(16, 4000, 136)
    ws = torch.zeros(moe.linear_backward_workspace_bytes(4000, 264, 136), dtype=torch.uint8, device="cuda")
    return ws, lambda: list(moe.linear_backward(dy, x, w, z=dy, act="silu", bias=True, ws=ws))


CASES = [case_few_rows, case_many_columns, case_pairs, case_parts, case_grouped, case_grouped_backward,
         case_linear_backward]


@pytest.mark.parametrize("cta", [1, 2, 3])
@pytest.mark.parametrize("case", CASES, ids=lambda c: c.__name__[5:])
def test_a_wait_that_runs_out_is_reported(case, cta):
    ws, call = case()
    want = [t.clone() for t in call()]
    assert moe.status_read(ws) == moe.OK
    torch.cuda.synchronize()
    moe.product_debug(wait_limit_us=5000, inject_skip_loads=cta)
    t0 = time.perf_counter()
    call()
    status = moe.status_read(ws)
    elapsed = time.perf_counter() - t0
    moe.product_debug()
    assert status == moe.ERR_TIMEOUT
    assert elapsed < 0.5, f"the call took {elapsed:.2f} s: the 5 ms limit was not applied to every wait"
    for _ in range(2):
        got = call()
        assert moe.status_read(ws) == moe.OK and moe.last_device_status() == moe.OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("case", CASES, ids=lambda c: c.__name__[5:])
def test_a_short_limit_on_a_normal_call(case):
    """200 ms is far above every wait of these calls: no timeout, the same bits."""
    ws, call = case()
    want = [t.clone() for t in call()]
    moe.product_debug(wait_limit_us=200_000)
    got = call()
    assert moe.status_read(ws) == moe.OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_setting_belongs_to_its_host_thread():
    ws, call = case_pairs()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    moe.product_debug(wait_limit_us=5000, inject_skip_loads=1)
    seen = []

    def other():
        with torch.cuda.stream(torch.cuda.Stream()):
            seen.append([t.clone() for t in call()])
            seen.append(moe.status_read(ws))

    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert seen[1] == moe.OK and all(torch.equal(a, b) for a, b in zip(seen[0], want))
