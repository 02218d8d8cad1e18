"""ft_kv_attend against its definition in 64 bits, within a bound derived for every output (tests/kv_util.py)."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from moe_expert_execution_amd.tensors import Workspace
from oracle import formats as OF
from tests.gpu_util import cuda, dev
from tests.kv_util import Cache, attend_reference, attend_row, random_table, stream
from tests.resident_util import assert_within

pytestmark = pytest.mark.gpu

FORMS = [(f, D) for f in ("bf16", "e4m3") for D in (64, 128, 256)]


class Attend:
    def __init__(self, cache, table, lens, hq, window=0, sinks=None, q_scale=1.0, seed=0, gap=0):
        rng = np.random.default_rng([seed, hq, len(lens)])
        self.cache, self.table, self.lens, self.hq = cache, table, np.asarray(lens, np.int64), hq
        self.window, self.sinks = window, sinks
        self.B, self.D = len(lens), cache.D
        self.row = hq * self.D + gap
        self.q = synth.f32_to_bf16((q_scale * rng.standard_normal((self.B, self.row))).astype(np.float32))
        self.scale = self.D ** -0.5

    def args(self):
        self.keep = [dev(self.q.view(np.int16)), dev(self.table), dev(self.lens.astype(np.int32))]
        self.sk = dev(self.sinks) if self.sinks is not None else None
        # rows behind the last request, to be left as they were
        self.out = torch.full((self.B + 2, self.row), 0x5A5A, dtype=torch.int16, device="cuda")
        return M.kv_attend(self.B, self.hq, self.table.shape[1], self.scale, self.keep[0].data_ptr(), self.row,
                           self.keep[1].data_ptr(), self.keep[2].data_ptr(), self.out.data_ptr(), self.row, self.window,
                           self.sk.data_ptr() if self.sk is not None else 0)

    def bits(self):
        return self.out.cpu().numpy().view(np.uint16)

    def run(self, ws=None, times=1, around=lambda call: call()):
        c = self.cache.struct()
        own = ws is None
        ws = ws or Workspace(M.ft_kv_attend_workspace(c, self.hq, max(self.B, 1)))
        a = self.args()
        torch.cuda.synchronize()
        for _ in range(times):
            around(lambda: M.ft_kv_attend(c, a, ws.handle, stream()))
        torch.cuda.synchronize()
        if own:
            ws.close()
        out = self.bits()
        assert (out[self.B:] == 0x5A5A).all() and (out[:, self.hq * self.D:] == 0x5A5A).all()
        return out[:self.B, :self.hq * self.D].reshape(self.B, self.hq, self.D)

    def check(self, raw=None, ws=None, what="", **kw):
        got = self.run(ws, **kw)
        q = self.q[:, :self.hq * self.D].reshape(self.B, self.hq, self.D)
        ref, bound = attend_reference(self.cache, q, self.table, self.lens, self.scale, self.window, self.sinks, raw)
        assert_within(OF.bf16_to_f64(got), ref, bound, what)
        return got


# A table for more than 1,024 tokens a request: the work is divided and cut; without, a workgroup takes a whole item.
WIDE = [False, True]


def extra(wide, P):
    return 1 + 1024 // P if wide else 2


def make(fmt, D, hkv, g, P, lens, seed=0, spare=3, wide=False, **kw):
    table, pages = random_table(lens, P, spare, seed, extra(wide, P))
    return Attend(Cache(fmt, pages, P, hkv, D, seed), table, lens, hkv * g, seed=seed, **kw)


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("g", [1, 3, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("wide", WIDE)
def test_head_groups(fmt, D, g, wide):
    cuda()
    make(fmt, D, 2, g, 16, [1, 0, 77, 300], seed=g, wide=wide).check()
    if wide:                                                  # cut and joined
        make(fmt, D, 1, g, 16, [2500], seed=g).check()


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("wide", WIDE)
def test_lengths(fmt, D, P, wide):
    """Lengths round every border: a block, a step, a team's steps, a page."""
    cuda()
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]
    make(fmt, D, 1, 4, P, lens, seed=P, wide=wide).check()
    make(fmt, D, 3, 12, P, lens[::-1], seed=P + 1, wide=wide).check()


@pytest.mark.parametrize("n", [1007, 1008, 1009, 1023, 1024, 1025, 1040])
def test_either_side_of_whole_items(n):
    """Tables of 64 and 65 pages: the longest whole items and the shortest that are cut."""
    cuda()
    for fmt, D in (("bf16", 128), ("e4m3", 256)):
        a = make(fmt, D, 2, 6, 16, [n, 3, 0, n // 2], seed=n)
        a.table = a.table[:, :max(64, -(-n // 16))].copy()
        a.check()


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("lens", [[20011], [3, 9000, 1, 0, 40], [700] * 30])
def test_work_split_and_joined(fmt, D, lens):
    """Long requests over many workgroups, alone and beside short ones; equal inputs give equal bits, call after call."""
    cuda()
    a = make(fmt, D, 2, 8, 64, lens, seed=7, gap=8)
    got = a.check()
    np.testing.assert_array_equal(a.run(times=3), got)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("e4m3", 64), ("bf16", 256)])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 4096])
def test_windows_and_sinks(fmt, D, window):
    cuda()
    lens = [0, 1, 2, 31, 32, 33, 64, 99, 100, 101, 132, 1000]
    rng = np.random.default_rng(window)
    for g in (5, 10):
        sinks = (3 * rng.standard_normal(2 * g)).astype(np.float32)
        make(fmt, D, 2, g, 32, lens, seed=8, window=window, sinks=sinks).check()
        make(fmt, D, 2, g, 32, lens, seed=9, window=window).check()


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("g", [1, 7, 12])
def test_many_short_items(fmt, D, g):
    """12 KV heads of 63 to 65 requests: either side of the number from which short items take two waves, by their
    table's width (8 steps) or their window."""
    cuda()
    rng = np.random.default_rng(g)
    for B in (63, 64, 65):
        lens = rng.permutation(np.r_[[0, 1, 31, 32, 33, 64, 65, 96, 97, 255, 256], rng.integers(0, 257, B - 11)])
        a = make(fmt, D, 12, g, 16, lens, seed=B)
        a.table = a.table[:, :16].copy()
        a.check()
    sinks = (3 * rng.standard_normal(12 * g)).astype(np.float32)
    make(fmt, D, 12, g, 32, 2 * lens, seed=9, window=127, sinks=sinks, gap=8).check()


def test_extreme_sinks():
    """A sink far above every logit, and of minus infinity (no term)."""
    cuda()
    lens = [0, 5, 900]
    for wide in WIDE:
        for s in (80.0, -np.inf, -3.0e38):
            make("bf16", 128, 1, 4, 16, lens, seed=10, sinks=np.full(4, s, np.float32), wide=wide).check()
        # an infinite sink takes everything, as the formula's limit; a NaN one is NaN in its own head
        for lens in ([0, 5, 900], [3000, 2, 1]):
            got = make("bf16", 128, 1, 4, 16, lens, seed=10, sinks=np.array([np.inf, 0, np.nan, 1], np.float32),
                       wide=wide).run()
            out = OF.bf16_to_f64(got)
            assert (out[:, 0] == 0).all() and np.isfinite(out[:, [1, 3]]).all()
            assert all(np.isnan(out[b, 2]).all() for b in range(3) if lens[b])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_peaked_and_flat_logits(fmt):
    """Logits of hundreds (one token takes it all) and of zero (a plain mean)."""
    cuda()
    for q_scale in (60.0, 0.0, 1e-3):
        make(fmt, 128, 2, 4, 16, [1, 50, 2500], seed=11, q_scale=q_scale).check()
        make(fmt, 128, 2, 4, 16, [1, 50, 700], seed=11, q_scale=q_scale).check()


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("wide", WIDE)
def test_what_lies_beside_the_visible_tokens(fmt, D, wide):
    """NaN in the cache everywhere but in the visible tokens: the rest of the last page, pages of others, and tokens
    before a window reach nothing."""
    cuda()
    P = 64
    lens = [1, 15, 33, 64, 65, 200, 0, 350]
    for window in (0, 40):
        table, pages = random_table(lens, P, 2, 12, extra(wide, P))
        cache = Cache(fmt, pages, P, 2, D, 12, fill="nan")
        rng = np.random.default_rng(12)
        for b, n in enumerate(lens):
            t = np.arange(max(0, n - window) if window else 0, n)
            slots = table[b, t // P].astype(np.int64) * P + t % P
            for w in "kv":
                for h in range(2):
                    x = rng.standard_normal((len(t), D)).astype(np.float32)
                    val = synth.f32_to_bf16(x) if fmt == "bf16" else rng.integers(0, 0x7E, (len(t), D))
                    cache.write(w, slots, h, val)
        cache.upload()
        for g in (4, 16):
            Attend(cache, table, lens, 2 * g, window, seed=12).check()


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("wide", WIDE)
def test_pages_outside_the_pool_are_left_out(fmt, D, wide):
    cuda()
    for P in (16, 32):
        lens = [40, 100, 16, 48]
        table, pages = random_table(lens, P, 1, 13, extra(wide, P))
        table[0, 0] = -1
        table[1, 1] = pages
        table[1, 2] = 2 ** 31 - 1
        table[2, 0] = -2 ** 31                               # the whole of a short request
        table[3, :] = -7
        cache = Cache(fmt, pages, P, 2, D, 13)
        for sinks in (None, np.ones(8, np.float32)):
            got = Attend(cache, table, lens, 8, sinks=sinks, seed=13).check()
            assert (got[2:] == 0).all()


@pytest.mark.parametrize("full", [32, 1200])
def test_lengths_out_of_range(full):
    cuda()
    table, pages = random_table([32, full, 32], 16, 1, 14, extra_width=0)
    cache = Cache("bf16", pages, 16, 1, 128, 14)
    Attend(cache, table, [-5, 2 ** 31 - 1, -2 ** 31], 4, seed=14).check()
    Attend(cache, table, [-5, full + 1, 2 ** 31 - 16], 4, seed=14).run()


@pytest.mark.parametrize("wide", WIDE)
def test_infinite_and_nan_values(wide):
    """What the formula gives: a NaN key or value makes its heads NaN, an infinite value at a probability above zero
    infinite, and a key of minus infinity has no share."""
    cuda()
    P, D = 16, 64
    table, pages = random_table([20, 20, 20, 20], P, 0, 15, extra(wide, P))
    cache = Cache("bf16", pages, P, 1, D, 15)
    slot = lambda b, t: int(table[b, t // P]) * P + t % P  # noqa: E731
    kn = np.full((1, D), 0x7FC0)
    cache.write("k", [slot(0, 3)], 0, kn)
    v1 = np.full((1, D), 0x3F80)
    v1[0, 5] = 0x7F80
    cache.write("v", [slot(1, 17)], 0, v1)
    k2 = np.zeros((1, D), np.uint16)
    k2[0, 0] = 0xFF80
    cache.write("k", [slot(2, 0)], 0, k2)
    cache.upload()
    a = Attend(cache, table, [20] * 4, 2, seed=15)
    a.q[:, ::D] = 0x3F80                                       # (q's first element is 1 in every head)
    out = OF.bf16_to_f64(a.run())
    assert np.isnan(out[0]).all()
    assert np.isposinf(out[1, :, 5]).all() and np.isfinite(np.delete(out[1], 5, axis=1)).all()
    t = np.arange(1, 20)
    ref_k = cache.read("k", [slot(2, int(i)) for i in t], 0)
    ref_v = cache.read("v", [slot(2, int(i)) for i in t], 0)
    ref, bound = attend_row(OF.bf16_to_f64(a.q[2].reshape(2, D)), ref_k, ref_v, a.scale)
    assert_within(out[2], ref, bound)
    assert np.isfinite(out[3]).all()


def test_shared_pages():
    """Requests with a common prefix name the same pages."""
    cuda()
    lens = [100, 130, 96]
    table, pages = random_table(lens, 32, 2, 16)
    table[1, :3] = table[0, :3]
    table[2, :3] = table[0, :3]
    Attend(Cache("bf16", pages, 32, 2, 128, 16), table, lens, 8, seed=16).check()


def test_many_requests():
    cuda()
    rng = np.random.default_rng(17)
    for B in (255, 256, 257, 1000):
        make("bf16", 64, 1, 2, 16, rng.integers(0, 40, B).tolist(), seed=17).check()
    make("e4m3", 64, 1, 1, 16, [3] * 4096, seed=18).check()
    # lists and sums of more than 64 KiB of LDS, items that are cut
    for fmt, g in (("bf16", 16), ("e4m3", 8)):
        make(fmt, 256, 1, g, 16, [2] * 3000 + [1500, 0] + [40] * 1094, seed=19).check()


def test_pages_beyond_32_bits():
    """Pages a GiB apart give what the same pages side by side give."""
    cuda()
    stride, P = 1 << 30, 32
    table, pages = random_table([150, 33], P, 0, 19)
    small = Cache("bf16", pages, P, 1, 128, 19)
    a = Attend(small, table, [150, 33], 4, seed=19)
    want = a.run()
    pool = {w: torch.zeros(pages * stride, dtype=torch.uint8, device="cuda") for w in "kv"}
    for w in "kv":
        for i in range(pages):
            pool[w][i * stride:i * stride + small.page] = small.dev[w][i * small.page:(i + 1) * small.page]
    small.dev, small.stride = pool, stride
    np.testing.assert_array_equal(a.run(), want)


def test_other_stream_and_workspaces():
    """Two calls at once on two streams, each with a workspace of its own."""
    cuda()
    calls = [make("bf16", 128, 2, 8, 16, [5000, 30, 900], seed=20 + i) for i in range(2)]
    want = [c.check() for c in calls]
    ws = [Workspace(M.ft_kv_attend_workspace(c.cache.struct(), c.hq, c.B)) for c in calls]
    args = [c.args() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, a, w, s in zip(calls, args, ws, streams):
            M.ft_kv_attend(c.cache.struct(), a, w.handle, s.cuda_stream)
    torch.cuda.synchronize()
    for c, r in zip(calls, want):
        np.testing.assert_array_equal(c.bits()[:c.B, :c.hq * c.D].reshape(r.shape), r)
    for w in ws:
        w.close()


def test_one_workspace_of_the_stated_size_serves_all():
    """Calls of many shapes in a row over one workspace: the counters are zero again after each."""
    cuda()
    big = make("bf16", 256, 1, 16, 16, [4000], seed=30)
    ws = Workspace(M.ft_kv_attend_workspace(big.cache.struct(), 16, 1))
    for i, (fmt, D, hkv, g, lens) in enumerate([("bf16", 256, 1, 16, [4000]), ("e4m3", 64, 4, 2, [1, 9999]),
                                                ("bf16", 128, 2, 8, [30] * 50), ("bf16", 256, 1, 16, [4000, 3])]):
        make(fmt, D, hkv, g, 16, lens, seed=31 + i).check(ws=ws, what=f"call {i}")
    ws.close()


def test_small_workspace_refused():
    cuda()
    a = make("bf16", 128, 2, 8, 16, [50], seed=40)
    need = M.ft_kv_attend_workspace(a.cache.struct(), a.hq, 1)
    ws = Workspace(need - 1)
    with pytest.raises(M.FtError, match="workspace holds"):
        M.ft_kv_attend(a.cache.struct(), a.args(), ws.handle, stream())
    ws.close()


@pytest.mark.parametrize("width", [40, 80])
def test_captured(width):
    """A captured call follows lengths, tables and cache contents as they are at each replay; whole items and cut ones."""
    cuda()
    P = 16
    rng = np.random.default_rng(50)
    table = rng.permutation(5 * width).reshape(5, width).astype(np.int32)
    cache = Cache("bf16", 5 * width, P, 2, 128, 50)
    a = Attend(cache, table, [1] * 5, 16, seed=50)
    ws = Workspace(M.ft_kv_attend_workspace(cache.struct(), 16, 5))
    args = a.args()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.ft_kv_attend(cache.struct(), args, ws.handle, stream())
    full = P * width
    for lens in ([0, 0, 0, 0, 0], [1, 2, 3, 4, 5], [full, 0, 17, 33, 600], [0, 0, full, 0, 0], [100] * 5):
        a.lens = np.array(lens)
        a.keep[2].copy_(torch.from_numpy(np.array(lens, np.int32)))
        a.out.fill_(0x5A5A)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = a.bits()[:5].reshape(5, 16, 128)
        ref, bound = attend_reference(cache, a.q.reshape(5, 16, 128), table, lens, a.scale)
        assert_within(OF.bf16_to_f64(got), ref, bound, str(lens))
        eager = Attend(cache, table, lens, 16, seed=50)
        np.testing.assert_array_equal(eager.run(), got)
    ws.close()
