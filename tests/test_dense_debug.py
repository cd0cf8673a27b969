"""Arguments of the product calls' debugging aids (no GPU needed)."""
import pytest

import nvfp4_quantized_moe_group_b200 as moe
from nvfp4_quantized_moe_group_b200 import build as build_mod


def test_product_debug_arguments():
    build_mod.build()
    moe.product_debug(wait_limit_us=1, inject_skip_loads=7)
    moe.product_debug(wait_limit_us=(1 << 32) - 1)
    with pytest.raises(moe.NvFp4MoeError) as e:
        moe.product_debug(inject_skip_loads=-1)
    assert e.value.status == moe.ERR_ARG
    moe.product_debug()
