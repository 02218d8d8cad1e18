"""Every token of a long request counts in ft_kv_attend, once: equal logits over values that tell where a token lies, so that a
step left out or taken twice at a cut, by a wave or in a join shows in its own dimension."""
import numpy as np
import pytest

from oracle import formats as OF
from tests.gpu_util import cuda
from tests.kv_codes import LONG, expected, long_row, positions_code
from tests.kv_util import Cache, random_table
from tests.resident_util import assert_within
from tests.test_gpu_kv_attend import Attend, make

pytestmark = pytest.mark.gpu

ONE = {"bf16": 0x3F80, "e4m3": 0x38}
FORMS = [(f, D) for f in ("bf16", "e4m3") for D in (64, 128, 256)]


def run(fmt, D, heads, g, P, lens, window=0, extra_pages=None, seed=220):
    """All tokens' keys random, queries zero; value codes of units of 32 and of 1 in alternate requests."""
    extra_width = 1 + 1024 // P if extra_pages is None else extra_pages
    table, pages = random_table(lens, P, 2, seed, extra_width)
    cache = Cache(fmt, pages, P, heads, D, seed)
    want = []
    for b, n in enumerate(lens):
        v = positions_code(n, D, (32, 1)[b % 2])
        slots = table[b, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        for h in range(heads):
            cache.write("v", slots, h, np.where(np.roll(v, h, axis=1) > 0, ONE[fmt], 0))
        want.append(v[max(0, n - window) if window else 0:])
    cache.upload()
    call = Attend(cache, table, lens, heads * g, window=window, q_scale=0.0, seed=seed)
    bits = call.run()
    out = OF.bf16_to_f64(bits).reshape(len(lens), heads, g, D)
    for b, n in enumerate(lens):
        for h in range(heads):
            s = 1.0 if fmt == "bf16" else float(cache.scales["v"][h])
            if n == 0:
                assert (out[b, h] == 0).all()
                continue
            ref, bound = expected(np.roll(want[b], h, axis=1), s)
            assert_within(out[b, h], np.broadcast_to(ref, (g, D)), np.broadcast_to(bound, (g, D)), f"request {b} head {h}")
    return call, bits


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("g", [4, 12])
@pytest.mark.parametrize("lens", [[20011], [20011, 5003], [3, 9000, 1, 0, 40], [700] * 30, [1025], [32 * 31] * 3 + [4097]])
def test_every_token_once(fmt, D, g, lens):
    cuda()
    run(fmt, D, 2, g, 64, lens)


@pytest.mark.parametrize("fmt,D", FORMS)
def test_every_token_once_at_every_length_of_a_cut(fmt, D):
    """One more token each: cuts, waves' shares and runs of the join fall elsewhere."""
    cuda()
    for n in list(range(1024, 1100, 5)) + [1536, 2048, 2999, 3105, 6143, 8193, 12288, 16385]:
        run(fmt, D, 1, 2, 16, [n])


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("window", [1500, 5000])
def test_every_token_of_a_window_once(fmt, D, window):
    cuda()
    run(fmt, D, 2, 3, 32, [20011, 4990, 100, 1501], window=window)


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("g", [1, 16])
def test_every_token_of_whole_items_once(fmt, D, g):
    """Tables of 64 pages of 16: a workgroup an item, of four waves or of two."""
    cuda()
    lens = [1024, 1023, 993, 992, 512, 33, 32, 31, 1]
    run(fmt, D, 2, g, 16, lens, extra_pages=0)
    run(fmt, D, 12, g, 16, [256, 255, 225, 224, 96, 33, 32, 1] * 9, extra_pages=0)


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("g", [4, 12])
def test_a_long_request_within_the_bound_of_its_own_sums(fmt, D, g):
    """Random logits and values, every output within the bound of sums in the kernel's order, which no absent step would meet
    (tests/test_kv_codes.py)."""
    cuda()
    a = make(fmt, D, 2, g, 64, [LONG], seed=7)
    out = OF.bf16_to_f64(a.run())[0].reshape(2, g, D)
    q = OF.bf16_to_f64(a.q[0]).reshape(2, g, D)
    slots = a.table[0, np.arange(LONG) // 64].astype(np.int64) * 64 + np.arange(LONG) % 64
    for h in range(2):
        ref, bound = long_row(q[h], a.cache.read("k", slots, h), a.cache.read("v", slots, h), a.scale)
        assert_within(out[h], ref, bound, f"head {h}")
