"""ft_kv_attend over values up to the format's largest: the result is a mean of them, so it is finite, however many add up."""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.kv_util import Cache, attend_reference, random_table
from tests.resident_util import assert_within
from tests.test_gpu_kv_attend import Attend, extra

from oracle import formats as OF

pytestmark = pytest.mark.gpu

LARGEST = {"bf16": 0x7F7F, "e4m3": 0x7E}
SIGN = {"bf16": 0x8000, "e4m3": 0x80}


@pytest.mark.parametrize("fmt,D", [(f, d) for f in ("bf16", "e4m3") for d in (64, 128, 256)])
@pytest.mark.parametrize("g", [2, 12])
@pytest.mark.parametrize("n,wide,window", [(1, False, 0), (2, False, 0), (300, False, 0), (300, True, 0), (5000, True, 0),
                                           (900, True, 200)])
def test_largest_values(fmt, D, g, n, wide, window):
    """All of one sign, of either sign at random, and one such value among ordinary ones; equal logits, ordinary ones, and
    with sinks."""
    cuda()
    P = 32
    lens = [n] * 3
    table, pages = random_table(lens, P, 1, 210, extra(wide, P))
    cache = Cache(fmt, pages, P, 1, D, 210)
    rng = np.random.default_rng([210, n, D])
    for b in range(3):
        slots = table[b, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        if b < 2:
            v = np.full((n, D), LARGEST[fmt])
            if b:
                v |= np.where(rng.random((n, D)) < 0.5, SIGN[fmt], 0)
            cache.write("v", slots, 0, v)
        else:
            cache.write("v", slots[n // 2:n // 2 + 1], 0, np.full((1, D), LARGEST[fmt]))
    cache.upload()
    for q_scale, sinks in ((0.0, None), (1.0, None), (0.0, np.linspace(-3, 9, g).astype(np.float32))):
        call = Attend(cache, table, lens, g, window=window, sinks=sinks, q_scale=q_scale, seed=210)
        out = OF.bf16_to_f64(call.run())
        ref, bound = attend_reference(cache, call.q.reshape(3, g, D), table, lens, call.scale, window, sinks)
        assert np.isfinite(out).all()
        assert_within(out, ref, bound, f"q {q_scale}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("g", [2, 12])
@pytest.mark.parametrize("n,wide", [(2, False), (300, False), (5000, True)])
def test_smallest_values(D, g, n, wide):
    """Values of 2^-116 to 2^-112, near the least normal number: their mean has an error of bf16's step and of the least fp32
    number a token, and is not zero."""
    cuda()
    P = 32
    table, pages = random_table([n], P, 1, 211, extra(wide, P))
    cache = Cache("bf16", pages, P, 1, D, 211)
    rng = np.random.default_rng([211, n, D])
    slots = table[0, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
    cache.write("v", slots, 0, (rng.integers(11, 16, (n, D)) << 7) | rng.integers(0, 128, (n, D)))
    cache.upload()
    for q_scale in (0.0, 1.0):
        call = Attend(cache, table, [n], g, q_scale=q_scale, seed=211)
        out = OF.bf16_to_f64(call.run())
        ref, bound = attend_reference(cache, call.q.reshape(1, g, D), table, [n], call.scale)
        # the definition's bound carries 1e-37 for outputs near zero; here it is 2^-149 of each scaled product and sum
        assert_within(out, ref, bound - 1e-37 + 2.0 ** -149 * 64 * n, f"q {q_scale}")
