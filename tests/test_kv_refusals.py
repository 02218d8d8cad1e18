"""Calls of the key-value cache's operators that their arithmetic could not serve are refused; CPU only."""
import numpy as np
import pytest

import moe_expert_execution_amd as M
from tests.test_kv_abi import attend, cache, check


@pytest.mark.parametrize("scale", [2.0 ** 127 * 1.01, -2.4e38, float(np.finfo(np.float32).max)])
def test_scales_beyond_base_2(scale):
    """The logits are in base 2: scale * log2(e) has to be finite in fp32."""
    check(M.ft_kv_attend, cache(), attend(scale=scale), 0, msg="scale must be finite")


@pytest.mark.parametrize("scale", [2.0 ** 127, -2.0 ** 127, 0.0, 1e-45])
def test_other_scales_are_accepted(scale):
    check(M.ft_kv_attend, cache(), attend(scale=scale), 0, msg="workspace is null")
