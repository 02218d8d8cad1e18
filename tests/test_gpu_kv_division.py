"""ft_kv_attend with each number of teams: two to a compute unit, one, fewer, on either side of the rules' borders and where the
launch has room for more than the lengths take (tests/kv_division.py; tests/test_kv_division.py counts the teams)."""
import numpy as np
import pytest

import moe_expert_execution_amd as M
from moe_expert_execution_amd.tensors import Workspace
from tests.gpu_util import cuda
from tests.kv_division import CALLS, width
from tests.test_gpu_kv_attend import make
from tests.test_gpu_kv_steps import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", CALLS)
def test_every_token_once(name):
    cuda()
    fmt, D, heads, g, P, lens, _ = CALLS[name]
    call, bits = run(fmt, D, heads, g, P, lens)
    assert call.table.shape[1] == width(P, lens)
    np.testing.assert_array_equal(call.run(times=3), bits)


@pytest.mark.parametrize("name", CALLS)
def test_against_the_definition(name):
    """Random keys and queries; equal bits call after call, and over one workspace in a row with a call of fewer teams."""
    cuda()
    fmt, D, heads, g, P, lens, _ = CALLS[name]
    a = make(fmt, D, heads, g, P, lens, seed=230, wide=True)
    assert a.table.shape[1] == width(P, lens)
    got = a.check()
    small = make(fmt, D, 1, g, P, [1500, 2], seed=231, wide=True)
    want = small.run()
    ws = Workspace(max(M.ft_kv_attend_workspace(c.cache.struct(), c.hq, c.B) for c in (a, small)))
    for _ in range(3):
        np.testing.assert_array_equal(a.run(ws), got)
        np.testing.assert_array_equal(small.run(ws), want)
    ws.close()
