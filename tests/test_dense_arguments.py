"""Argument checking of the 16-bit products and the layer norm on a machine without a GPU: every C-ABI call
returns its documented status before any CUDA call, and the binding rejects tensors of the wrong
type, shape, layout or device.  The placeholder pointers are never dereferenced; the module is
skipped where a GPU is present, since a call that passed its checks would launch on them."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from nvfp4_quantized_moe_group_b200 import build as build_mod

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder device pointers: host-only checks, no GPU")

A = 1 << 20                       # a 256-byte aligned placeholder address
MIS = A + 8                       # 8-byte aligned, not 16
BIG = 1 << 40
NO_DEVICE = (moe.ERR_DEVICE, moe.ERR_CUDA)
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return moe.lib()


def grouped(lib, **kw):
    a = dict(dtype=BF16, x=A, M=16, K=64, w=A, E=4, N=128, offsets=A, y=A, ws=A, ws_bytes=BIG)
    a.update(kw)
    return lib.nvfp4moe_grouped_mm(a["dtype"], a["x"], a["M"], a["K"], a["w"], a["E"], a["N"], a["offsets"], a["y"],
                                   a["ws"], a["ws_bytes"], None)


def grouped_backward(lib, **kw):
    a = dict(dtype=BF16, dy=A, x=A, w=A, M=16, K=64, E=4, N=128, offsets=A, dx=A, dw=A, dw_dtype=BF16, ws=A,
             ws_bytes=BIG)
    a.update(kw)
    return lib.nvfp4moe_grouped_mm_backward(a["dtype"], a["dy"], a["x"], a["w"], a["M"], a["K"], a["E"], a["N"],
                                            a["offsets"], a["dx"], a["dw"], a["dw_dtype"], a["ws"], a["ws_bytes"],
                                            None)


def linear(lib, **kw):
    a = dict(dtype=BF16, x=A, M=16, K=64, w=A, N=128, bias=None, act=0, residual=None, z=None, y=A, ws=A, ws_bytes=BIG)
    a.update(kw)
    return lib.nvfp4moe_linear(a["dtype"], a["x"], a["M"], a["K"], a["w"], a["N"], a["bias"], a["act"], a["residual"],
                               a["z"], a["y"], a["ws"], a["ws_bytes"], None)


def linear_backward(lib, **kw):
    a = dict(dtype=BF16, dy=A, x=A, w=A, z=None, M=16, K=64, N=128, act=0, dx=A, dw=A, dw_dtype=BF16, db=None, ws=A,
             ws_bytes=BIG)
    a.update(kw)
    return lib.nvfp4moe_linear_backward(a["dtype"], a["dy"], a["x"], a["w"], a["z"], a["M"], a["K"], a["N"], a["act"],
                                        a["dx"], a["dw"], a["dw_dtype"], a["db"], a["ws"], a["ws_bytes"], None)


def norm(lib, **kw):
    a = dict(dtype=BF16, x=A, rows=4, cols=100, gamma=A, beta=A, eps=1e-5, rms=0, y=A, mean=A, rstd=A)
    a.update(kw)
    return lib.nvfp4moe_layer_norm(a["dtype"], a["x"], a["rows"], a["cols"], a["gamma"], a["beta"], a["eps"], a["rms"],
                                   a["y"], a["mean"], a["rstd"], None)


def norm_backward(lib, **kw):
    a = dict(dtype=BF16, dy=A, x=A, rows=4, cols=100, gamma=A, mean=A, rstd=A, rms=0, dx=A, dgamma=A, dbeta=A, ws=A,
             ws_bytes=BIG)
    a.update(kw)
    return lib.nvfp4moe_layer_norm_backward(a["dtype"], a["dy"], a["x"], a["rows"], a["cols"], a["gamma"], a["mean"],
                                            a["rstd"], a["rms"], a["dx"], a["dgamma"], a["dbeta"], a["ws"],
                                            a["ws_bytes"], None)


SHAPES = [dict(K=0), dict(K=63), dict(K=12), dict(N=0), dict(N=4), dict(N=130), dict(K=(1 << 19) + 8),
          dict(N=(1 << 19) + 8), dict(M=-1), dict(M=1 << 25), dict(M=(1 << 25) - 1, K=(1 << 15) + 8)]


@pytest.mark.parametrize("call", [grouped, grouped_backward, linear, linear_backward])
@pytest.mark.parametrize("kw", SHAPES)
def test_product_shapes(lib, call, kw):
    assert call(lib, **kw) == moe.ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=1025), dict(E=-3), dict(E=1024, K=1 << 15, N=1 << 15)])
def test_group_limits(lib, kw):
    assert grouped(lib, **kw) == moe.ERR_SHAPE and grouped_backward(lib, **kw) == moe.ERR_SHAPE


def test_product_types_and_pointers(lib):
    for call in (grouped, grouped_backward, linear, linear_backward):
        assert call(lib, dtype=FP32) == moe.ERR_ARG and call(lib, dtype=-1) == moe.ERR_ARG
        assert call(lib, ws=None) == moe.ERR_ARG and call(lib, ws=A + 16) == moe.ERR_ARG
        assert call(lib, ws_bytes=255) == moe.ERR_WORKSPACE
        assert call(lib, x=MIS) == moe.ERR_ARG and call(lib, w=MIS) == moe.ERR_ARG
        assert call(lib) in NO_DEVICE
    for call in (grouped, linear):
        for name in ("x", "w", "y"):
            assert call(lib, **{name: None}) == moe.ERR_ARG
        assert call(lib, y=MIS) == moe.ERR_ARG
    for call in (grouped, grouped_backward):
        assert call(lib, offsets=None) == moe.ERR_ARG and call(lib, offsets=A + 2) == moe.ERR_ARG
    for call in (grouped_backward, linear_backward):
        assert call(lib, dw_dtype=FP16) == moe.ERR_ARG and call(lib, dtype=FP16, dw_dtype=BF16) == moe.ERR_ARG
        assert call(lib, dw_dtype=FP32) in NO_DEVICE
        assert call(lib, dw_dtype=7, dw=None) in NO_DEVICE           # no dw, no type of it
        assert call(lib, dx=None, dw=None) == moe.ERR_ARG
        assert call(lib, dy=None) == moe.ERR_ARG and call(lib, dy=MIS) == moe.ERR_ARG
        assert call(lib, dx=MIS) == moe.ERR_ARG and call(lib, dw=MIS) == moe.ERR_ARG
        assert call(lib, x=None) == moe.ERR_ARG and call(lib, x=None, dw=None) in NO_DEVICE
        assert call(lib, w=None) == moe.ERR_ARG and call(lib, w=None, dx=None) in NO_DEVICE
    for name in ("bias", "residual", "z"):
        assert linear(lib, **{name: MIS}) == moe.ERR_ARG and linear(lib, **{name: A}) in NO_DEVICE
    for act in (-1, 5):
        assert linear(lib, act=act) == moe.ERR_ARG and linear_backward(lib, act=act) == moe.ERR_ARG
    assert linear_backward(lib, act=2) == moe.ERR_ARG                 # an activation needs z
    assert linear_backward(lib, act=2, z=A) in NO_DEVICE
    assert linear_backward(lib, dx=None, dw=None, db=A) in NO_DEVICE
    assert linear_backward(lib, db=A + 2) == moe.ERR_ARG


def test_parts_need_their_workspace(lib):
    """Calls whose reduction is shared by several pairs refuse the workspace of those without."""
    need = moe.grouped_mm_backward_workspace_bytes(1 << 20, 64, 1, 128)
    kw = dict(M=1 << 20, K=64, E=1, N=128)
    assert grouped_backward(lib, ws_bytes=need - 1, **kw) == moe.ERR_WORKSPACE
    assert grouped_backward(lib, ws_bytes=need, **kw) in NO_DEVICE
    kw = dict(M=600, K=16008, N=264)
    need = moe.linear_workspace_bytes(600, 16008, 264)
    assert need > 9 * 4 * 600 * 264
    assert linear(lib, ws_bytes=need - 1, **kw) == moe.ERR_WORKSPACE and linear(lib, ws_bytes=need, **kw) in NO_DEVICE
    kw = dict(M=520, K=40, N=16008)
    need = moe.linear_backward_workspace_bytes(520, 40, 16008)
    assert linear_backward(lib, ws_bytes=need - 1, **kw) == moe.ERR_WORKSPACE
    assert linear_backward(lib, ws_bytes=need, **kw) in NO_DEVICE


def test_no_rows_need_no_row_pointers(lib):
    assert grouped(lib, M=0, x=None, y=None) in NO_DEVICE
    assert linear(lib, M=0, x=None, y=None) in NO_DEVICE
    assert grouped_backward(lib, M=0, x=None, dy=None, w=None) in NO_DEVICE
    assert linear_backward(lib, M=0, x=None, dy=None, w=None, act=2) in NO_DEVICE
    assert norm(lib, rows=0, x=None, y=None) in NO_DEVICE
    assert norm_backward(lib, rows=0, x=None, dy=None, dx=None, mean=None, rstd=None) in NO_DEVICE


def test_norm_arguments(lib):
    for call in (norm, norm_backward):
        assert call(lib, dtype=3) == moe.ERR_ARG and call(lib, dtype=-1) == moe.ERR_ARG
        for kw in (dict(cols=0), dict(cols=28673), dict(rows=-1), dict(rows=1 << 31)):
            assert call(lib, **kw) == moe.ERR_SHAPE
        assert call(lib, x=None) == moe.ERR_ARG and call(lib, x=MIS) == moe.ERR_ARG
        assert call(lib, gamma=A + 2) == moe.ERR_ARG and call(lib, mean=A + 2) == moe.ERR_ARG
        assert call(lib, gamma=A + 4) in NO_DEVICE
        assert call(lib) in NO_DEVICE and call(lib, cols=28672, dtype=FP32) in NO_DEVICE
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == moe.ERR_ARG
    assert norm(lib, y=None) == moe.ERR_ARG and norm(lib, y=MIS) == moe.ERR_ARG
    assert norm(lib, rms=1) == moe.ERR_ARG and norm(lib, rms=1, beta=None) in NO_DEVICE
    assert norm(lib, gamma=None, beta=None, mean=None, rstd=None) in NO_DEVICE
    for name in ("dy", "dx", "rstd", "mean"):
        assert norm_backward(lib, **{name: None}) == moe.ERR_ARG
    assert norm_backward(lib, rms=1) == moe.ERR_ARG
    assert norm_backward(lib, rms=1, mean=None) == moe.ERR_ARG        # dbeta with rms
    assert norm_backward(lib, rms=1, mean=None, dbeta=None) in NO_DEVICE
    assert norm_backward(lib, ws=None) == moe.ERR_ARG and norm_backward(lib, ws=A + 64) == moe.ERR_ARG
    need = moe.layer_norm_backward_workspace_bytes(4, 100)
    assert norm_backward(lib, ws_bytes=need - 1) == moe.ERR_WORKSPACE
    assert norm_backward(lib, ws=None, ws_bytes=0, dgamma=None, dbeta=None) in NO_DEVICE


def test_workspace_sizes(lib):
    assert moe.grouped_mm_workspace_bytes(0) == 0 and moe.grouped_mm_workspace_bytes(1025) == 0
    assert 256 < moe.grouped_mm_workspace_bytes(1) <= moe.grouped_mm_workspace_bytes(1024) < 1 << 20
    # backward: parts of dw where few tiles have many rows
    assert moe.grouped_mm_backward_workspace_bytes(64, 64, 4, 128) == moe.grouped_mm_workspace_bytes(4)
    assert moe.grouped_mm_backward_workspace_bytes(1 << 20, 64, 1, 128) >= 2 * 4 * 64 * 128
    assert moe.grouped_mm_backward_workspace_bytes((1 << 25) - 1, 256, 74, 256) < 1 << 27
    assert moe.grouped_mm_backward_workspace_bytes(0, 64, 0, 128) == 0
    assert moe.grouped_mm_backward_workspace_bytes(1 << 25, 64, 1, 128) == 0
    assert moe.linear_workspace_bytes(16, 64, 128) >= 256 and moe.linear_workspace_bytes(16, 65, 128) == 0
    assert moe.linear_backward_workspace_bytes(1000, 64, 128) >= 1000 * 128 * 2
    assert moe.linear_backward_workspace_bytes(-1, 64, 128) == 0
    assert moe.layer_norm_backward_workspace_bytes(5, 0) == 0 and moe.layer_norm_backward_workspace_bytes(5, 28673) == 0
    assert moe.layer_norm_backward_workspace_bytes(0, 7) >= 56
    # sized for the grid of any element type, for every count of rows
    for cols in (1, 255, 256, 1000, 1024, 2048, 5111, 5120, 8192, 9000, 16384, 20000, 28672):
        last = 0
        for rows in (1, 16, 296, 297, 1000, 10 ** 6):
            n = moe.layer_norm_backward_workspace_bytes(rows, cols)
            assert n >= 8 * cols and n <= 300 * 8 * cols + 256
            last = n
        assert last >= 100 * 8 * cols


def _raises(err, match, fn, *args, **kw):
    with pytest.raises(err, match=match):
        fn(*args, **kw)


def test_binding_products():
    x, w, o = torch.zeros((6, 64)).bfloat16(), torch.zeros((4, 32, 64)).bfloat16(), torch.zeros(5, dtype=torch.int32)
    f = moe.grouped_mm
    _raises(TypeError, "x must be a tensor of one of", f, x.float(), w, o)
    _raises(TypeError, "x must be a 2-D tensor", f, x[0], w, o)
    _raises(TypeError, "w must be a 3-D tensor", f, x, w[0], o)
    _raises(TypeError, r"w must have shape \(4, 32, 64\)", f, x, torch.zeros((4, 32, 72)).bfloat16(), o)
    _raises(TypeError, "w must be torch.bfloat16", f, x, w.half(), o)
    _raises(TypeError, r"offsets must have shape \(5,\)", f, x, w, o[:4])
    _raises(TypeError, "offsets must be torch.int32", f, x, w, o.long())
    _raises(TypeError, "x must be contiguous", f, torch.zeros((6, 128)).bfloat16()[:, ::2], w, o)
    _raises(TypeError, r"out must have shape \(6, 32\)", f, x, w, o, out=torch.zeros((6, 31)).bfloat16())
    _raises(TypeError, "must be a CUDA tensor", f, x, w, o)
    dy = torch.zeros((6, 32)).bfloat16()
    f = moe.grouped_mm_backward
    _raises(TypeError, r"x must have shape \(6, 64\)", f, dy, x[:5], w, o)
    _raises(TypeError, "dw_dtype must be", f, dy, x, w, o, dw_dtype=torch.float16)
    _raises(TypeError, "dw_dtype must be", f, dy, x, w, o, dw=torch.zeros((4, 32, 64)).half())
    _raises(TypeError, r"dw must have shape", f, dy, x, w, o, dw=torch.zeros((4, 32, 63)))
    _raises(TypeError, "must be a CUDA tensor", f, dy, x, w, o)
    f = moe.linear
    _raises(ValueError, "act must be one of", f, x, w[0], act="swish")
    _raises(TypeError, "bias must be torch.float32", f, x, w[0], bias=torch.zeros(32).bfloat16())
    _raises(TypeError, r"residual must have shape \(6, 32\)", f, x, w[0], residual=x)
    _raises(TypeError, "must be a CUDA tensor", f, x, w[0])
    f = moe.linear_backward
    _raises(ValueError, "needs the pre-activation z", f, dy, x, w[0], act="gelu")
    _raises(TypeError, r"z must have shape \(6, 32\)", f, dy, x, w[0], z=x, act="gelu")
    _raises(TypeError, "must be a CUDA tensor", f, dy, x, w[0])


def test_binding_norm():
    x, g = torch.zeros((6, 33)), torch.ones(33)
    f = moe.layer_norm
    _raises(TypeError, "x must be a tensor of one of", f, x.double())
    _raises(TypeError, r"gamma must have shape \(33,\)", f, x, g[:32])
    _raises(TypeError, "beta must be torch.float32", f, x, g, g.half())
    _raises(TypeError, "out must be torch.float32", f, x, g, out=x.half())
    _raises(TypeError, "x must be contiguous", f, x.t())
    _raises(TypeError, "must be a CUDA tensor", f, x, g)
    f, s = moe.layer_norm_backward, torch.ones(6)
    _raises(ValueError, "needs the mean", f, x, x, g, None, s)
    _raises(TypeError, r"rstd must have shape \(6,\)", f, x, x, g, s, s[:5])
    _raises(TypeError, "x must be torch.float32", f, x, x.half(), g, s, s)
    _raises(TypeError, "must be a CUDA tensor", f, x, x, g, s, s)
