"""The values and bounds of tests/kv_codes.py show a step left out or taken twice (planted in the reference); CPU only."""
import numpy as np
import pytest

from tests.kv_codes import LONG, long_row, lost


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1025, 5000, 9000, 20011])
def test_every_step_would_show(D, n):
    """The bounds are tight enough (computed here, on the host, with the step left out of the reference)."""
    assert not lost(n, D, 32)


@pytest.mark.parametrize("D,g", [(64, 4), (128, 4), (256, 12)])
def test_random_values_show_an_absent_step(D, g):
    rng = np.random.default_rng(D)
    q, k, v = rng.standard_normal((g, D)), rng.standard_normal((LONG, D)), rng.standard_normal((LONG, D))
    out, bound = long_row(q, k, v, D ** -0.5)
    for step in rng.integers(0, LONG // 32, 20):
        wrong, _ = long_row(q, k, v, D ** -0.5, drop=slice(32 * step, 32 * step + 32))
        assert (np.abs(wrong - out) > 2 * bound).any(), step   # (twice: the kernel's own error may hide one)
