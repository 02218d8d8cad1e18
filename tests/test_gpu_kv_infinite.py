"""Infinite values in the cache give ft_kv_attend's formula: a positive weight times infinity is infinity of the value's
sign, whatever bits the weight has."""
import numpy as np
import pytest

from oracle import formats as OF
from tests.gpu_util import cuda
from tests.kv_util import Cache, attend_row, random_table
from tests.resident_util import assert_within
from tests.test_gpu_kv_attend import Attend, extra

pytestmark = pytest.mark.gpu

INF, MINUS_INF = 0x7F80, 0xFF80
# Logits of the infinite tokens below a largest of 0 (bf16, so exact): the rest of the weight after its nearest bf16 is
# zero for the first, and negative for some and positive for others of the following.
LOGITS = [0.0, -0.25, -0.5, -0.75, -1.0, -1.5, -2.0, -3.0, -5.0, -7.25, -11.0, -20.0, -33.0, -47.0]


def rests():
    p = np.exp2(np.array(LOGITS, np.float32) * np.float32(1.4426950408889634))
    return p - OF.bf16_to_f64(bf16(p))


def bf16(x):
    import synth
    return synth.f32_to_bf16(np.asarray(x, np.float32))


def test_the_logits_leave_rests_of_every_sign():
    r = rests()
    assert r[0] == 0 and (r < 0).sum() >= 4 and (r > 0).sum() >= 4


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 2, 8, 12])
@pytest.mark.parametrize("n,wide", [(1, False), (1, True), (40, False), (300, False), (300, True), (2500, True)])
def test_infinite_values(D, g, n, wide):
    """A request per logit and place of its infinite token: in the first step, in the last and between, before and behind
    the largest logit, so that it is also rescaled, in another wave's part and in another team's.  Dimension 1 has
    a positive, 2 a negative infinity, 3 one of each sign; the others are finite."""
    cuda()
    P = 16
    places = sorted({0, n // 3, n - 1})
    cases = [(a, t) for a in LOGITS for t in places if n > 1 or a == 0.0]
    lens = [n] * len(cases)
    table, pages = random_table(lens, P, 1, 200, extra(wide, P))
    cache = Cache("bf16", pages, P, 1, D, 200)
    for b, (a, t) in enumerate(cases):
        slots = table[b, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        top = (t + n // 2) % n                                 # the largest logit's place
        k = np.zeros((n, D), np.uint16)
        logits = np.full(n, -60.0)
        logits[t], logits[top] = a, 0.0
        k[:, 0] = bf16(logits)
        cache.write("k", slots, 0, k)
        v = cache.read("v", slots, 0)
        v = bf16(v)
        v[t, 1], v[t, 2], v[t, 3] = INF, MINUS_INF, INF
        v[top if top != t else t, 3] = MINUS_INF if top != t else 0x7FC0
        cache.write("v", slots, 0, v)
    cache.upload()
    call = Attend(cache, table, lens, g, seed=200)
    call.scale = 1.0
    call.q[:] = 0
    call.q[:, ::D] = 0x3F80                                    # s_t = k_t[0] in every head
    out = OF.bf16_to_f64(call.run())
    assert np.isposinf(out[:, :, 1]).all(), [cases[b] for b in np.nonzero(~np.isposinf(out[:, :, 1]).all(1))[0]]
    assert np.isneginf(out[:, :, 2]).all()
    assert np.isnan(out[:, :, 3]).all()
    finite = [0] + list(range(4, D))
    for b in range(len(cases)):
        slots = table[b, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        q = OF.bf16_to_f64(call.q[b].reshape(g, D))
        ref, bound = attend_row(q, cache.read("k", slots, 0), cache.read("v", slots, 0)[:, finite], 1.0)
        assert_within(out[b][:, finite], ref, bound, str(cases[b]))


@pytest.mark.parametrize("g", [4, 16])
@pytest.mark.parametrize("n,wide", [(33, False), (3000, True)])
def test_infinite_values_beside_sinks_and_windows(g, n, wide):
    """Equal logits (weights of exactly 1), a sink above them and a window: an infinity inside it counts, one before it does
    not."""
    cuda()
    P, D = 16, 128
    table, pages = random_table([n, n], P, 1, 201, extra(wide, P))
    cache = Cache("bf16", pages, P, 1, D, 201)
    at = lambda b, t: [int(table[b, t // P]) * P + t % P]  # noqa: E731
    for b, t in ((0, n - 1), (1, n - 21)):
        v = bf16(cache.read("v", at(b, t), 0))
        v[0, 7] = MINUS_INF
        cache.write("v", at(b, t), 0, v)
    cache.upload()
    sinks = np.linspace(-2, 8, g).astype(np.float32)
    for window in (0, 20):
        call = Attend(cache, table, [n, n], g, window=window, sinks=sinks, seed=201)
        call.q[:] = 0
        out = OF.bf16_to_f64(call.run())
        assert np.isneginf(out[0, :, 7]).all()
        assert (np.isfinite if window else np.isneginf)(out[1, :, 7]).all()
        assert np.isfinite(np.delete(out, 7, axis=2)).all()
