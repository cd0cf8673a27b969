"""Layer norm backward of wide rows from two host threads: the shared-memory limit of a kernel belongs to the
device, not to the thread that set it, so one thread's narrower call must not take it from another's wider one."""
import threading

import numpy as np
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from oracle import dense
from tests.test_gpu_norm import E, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.lib()


def case(cols, dtype):
    gen = torch.Generator().manual_seed(cols)
    x, dy = torch.randn((5, cols), generator=gen).to(dtype), torch.randn((5, cols), generator=gen).to(dtype)
    gamma = 1 + 0.2 * torch.randn(cols, generator=gen)
    X, D, G = f64(x), f64(dy), f64(gamma)
    r = torch.rsqrt(x.float().square().mean(1) + 1e-5)
    DX, DG, _ = dense.layer_norm_backward(D, X, G, None, f64(r), rms=True)
    XH, GG = X * f64(r)[:, None], D * G
    eg = 4 * np.abs(GG) + np.abs(XH) * 58 * np.abs(GG * XH).mean(1, keepdims=True)
    bounds = f64(r)[:, None] * E * eg, 13 * E * np.abs(D * XH).sum(0)
    args = (dy.cuda(), x.cuda(), gamma.cuda(), None, r.cuda())

    def run():
        dx, dg, _ = moe.layer_norm_backward(*args, rms=True)
        check(dx, DX, bounds[0], (cols, "dx"))
        check(dg, DG, bounds[1], (cols, "dgamma"))

    return run


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wide,narrow", [(28672, 17000), (28671, 16389)])
def test_two_threads_with_rows_of_different_widths(wide, narrow, dtype):
    runs = {"wide": case(wide, dtype), "narrow": case(narrow, dtype)}
    # the calls alternate between the threads: wide, narrow, wide, ...
    turns = {"wide": threading.Semaphore(1), "narrow": threading.Semaphore(0)}
    other = {"wide": "narrow", "narrow": "wide"}
    errors = []

    def work(name):
        for _ in range(3):
            turns[name].acquire()
            try:
                runs[name]()
            except BaseException as e:      # noqa: BLE001  reported by the main thread
                errors.append((name, e))
            turns[other[name]].release()

    threads = [threading.Thread(target=work, args=(n,)) for n in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_two_threads_at_once():
    runs = [case(28672, torch.bfloat16), case(20008, torch.bfloat16)]
    errors = []

    def work(run):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    run()
        except BaseException as e:      # noqa: BLE001  reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(r,)) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
