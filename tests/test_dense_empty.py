"""Batches without rows at the C ABI (no GPU needed): a gradient without elements may be NULL."""
import pytest
import torch

import nvfp4_quantized_moe_group_b200 as moe
from tests.test_dense_arguments import NO_DEVICE, grouped_backward, lib, linear_backward  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder device pointers: host-only checks, no GPU")


def test_nothing_to_write_without_rows(lib):  # noqa: F811
    for call in (grouped_backward, linear_backward):
        assert call(lib, M=0, dy=None, x=None, dx=None, dw=None) in NO_DEVICE
        assert call(lib, M=1, dx=None, dw=None) == moe.ERR_ARG
