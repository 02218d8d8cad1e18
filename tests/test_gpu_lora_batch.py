"""What a token's result may depend on: not on the values of the tokens beside it."""
import numpy as np
import pytest

from tests.resident_util import Pool, mixed_ids
from tests.test_gpu_lora import Expert, Project, x_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T", [5, 40, 64, 130, 700])
def test_other_tokens_values_do_not_reach_a_row(fmt, T):
    """The same rows and adapters among other tokens of other sizes: the same bits, streamed and in the tiles."""
    d, f, R, count = 512, 384, 32, 6
    ex, pr = Expert(fmt, d, f, R, T, seed=81), Project(fmt, d, f, R, T, seed=81)
    pds = [Pool(count, R, d, f, 811).device(), Pool(count, R, d, f, 812).device(), Pool(count, R, f, d, 813).device()]
    ids = mixed_ids(T, count, 81, run=3)
    kept = np.arange(T) % 3 == 1
    for op, K, pools in ((ex, d, pds), (pr, f, pds[2])):
        x, other = x_of(T, K, 0), x_of(T, K, 1)
        other = np.where(kept[:, None], x, other ^ np.uint16(0x8100))      # (another sign, a quarter or four times the size)
        a, b = op(x, pools, ids), op(other, pools, ids)
        np.testing.assert_array_equal(a[kept], b[kept])
        assert (a[~kept] != b[~kept]).any()
