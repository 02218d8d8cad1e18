"""ft_kv_append against its definition: types, head sizes, rotation, strides, padding, and what it leaves alone."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from oracle import formats as OF
from tests.gpu_util import cuda, dev
from tests.kv_util import Cache, E4M3, bf16_bound, e4m3_bound, rope, stream

pytestmark = pytest.mark.gpu


class Call:
    """Tokens of an append: one projection's rows [T, (q + 2 kv) heads, D] with `gap` elements between rows."""

    def __init__(self, cache, T, hq, rot, slots, pos, positions=512, gap=0, seed=0, scale=1.0):
        rng = np.random.default_rng([seed, T, hq, rot])
        D, hkv = cache.D, cache.heads
        row = (hq + 2 * hkv) * D + gap
        self.bits = synth.f32_to_bf16((scale * rng.standard_normal((T, row))).astype(np.float32))
        self.cache, self.T, self.hq, self.rot, self.row = cache, T, hq, rot, row
        ang = rng.uniform(-np.pi, np.pi, (positions, max(rot // 2, 1)))
        self.cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.slots, self.pos = np.asarray(slots, np.int64), np.asarray(pos, np.int64)

    def args(self, in_place=False):
        T, hq, D, hkv = self.T, self.hq, self.cache.D, self.cache.heads
        self.x = dev(self.bits.view(np.int16))
        self.q = torch.full((T, hq * D), 0x4321, dtype=torch.int16, device="cuda")
        self.keep = [dev(self.slots.astype(np.int32)), dev(self.pos.astype(np.int32)), dev(self.cos_sin)]
        p = self.x.data_ptr()
        out, out_stride = (p, self.row) if in_place else (self.q.data_ptr(), hq * D)
        return M.kv_append(T, p + 2 * hq * D, self.row, p + 2 * (hq + hkv) * D, self.row, self.keep[0].data_ptr(),
                           self.keep[1].data_ptr() if self.rot else 0, self.rot, len(self.cos_sin) if self.rot else 0,
                           self.keep[2].data_ptr() if self.rot else 0, hq, p if hq else 0, self.row, out if hq else 0,
                           out_stride)

    def run(self, in_place=False, around=lambda call: call()):
        """`around` makes the call: for what happens beside it."""
        a, T, hq, D = self.args(in_place), self.T, self.hq, self.cache.D
        c = self.cache.struct()
        torch.cuda.synchronize()
        around(lambda: M.ft_kv_append(c, a, stream()))
        torch.cuda.synchronize()
        q = self.x.cpu().numpy()[:, :hq * D] if in_place else self.q.cpu().numpy()
        return q.view(np.uint16).reshape(T, hq, D)

    def check(self, in_place=False, **kw):
        c, T, hq, D, hkv = self.cache, self.T, self.hq, self.cache.D, self.cache.heads
        q = self.run(in_place, **kw)
        x = OF.bf16_to_f64(self.bits[:, :(hq + 2 * hkv) * D]).reshape(T, hq + 2 * hkv, D)
        live = (self.slots >= 0) & (self.slots < c.pages * c.P)
        if self.rot:
            live &= (self.pos >= 0) & (self.pos < len(self.cos_sin))
        on = np.nonzero(live)[0]
        turned, err = rope(x[on, :hq + hkv], self.pos[on], self.cos_sin, self.rot)
        # queries: rotated and rounded, padding's left as they were
        got = OF.bf16_to_f64(q[on])
        assert (np.abs(got - turned[:, :hq]) <= bf16_bound(turned[:, :hq], err[:, :hq])).all()
        was = self.bits[:, :hq * D].reshape(T, hq, D) if in_place else np.full_like(q, 0x4321)
        np.testing.assert_array_equal(q[~live], was[~live])
        # the caches: every new token's element, and every other byte as it was
        for w, val, e in (("k", turned[:, hq:], err[:, hq:]), ("v", x[on, hq + hkv:], np.zeros((len(on), hkv, D)))):
            raw, want = c.dev[w].cpu().numpy(), c.host[w].copy()
            for h in range(hkv):
                off = c.offsets(w, self.slots[on], h)
                if c.fmt == "bf16":
                    got = OF.bf16_to_f64(raw[off].astype(np.uint16) | raw[off + 1].astype(np.uint16) << 8)
                    assert (np.abs(got - val[:, h]) <= bf16_bound(val[:, h], e[:, h])).all(), (w, h)
                    want[off], want[off + 1] = raw[off], raw[off + 1]
                else:
                    v, b = e4m3_bound(val[:, h], e[:, h], float(c.scales[w][h]))
                    assert (np.abs(E4M3[raw[off]] - v) <= b).all(), (w, h)
                    want[off] = raw[off]
            np.testing.assert_array_equal(raw, want, err_msg=f"{w}: bytes beside the new tokens")


FORMS = [(f, D) for f in ("bf16", "e4m3") for D in (64, 128, 256)]


@pytest.mark.parametrize("fmt,D", FORMS)
@pytest.mark.parametrize("T,hq,hkv,P,rot,gap", [(1, 4, 1, 16, 64, 0), (1, 0, 2, 256, 0, 0), (15, 3, 3, 16, 16, 8),
                                                (16, 8, 1, 32, 32, 0), (17, 2, 2, 64, 48, 24), (100, 5, 5, 128, 64, 0),
                                                (333, 16, 2, 16, 0, 0), (1500, 7, 7, 64, 64, 8)])
def test_shapes(fmt, D, T, hq, hkv, P, rot, gap):
    """Scattered slots of a decode batch (up to 100 tokens) and runs of a prompt that begin anywhere."""
    cuda()
    rng = np.random.default_rng([T, D])
    pages = max(2, -(-2 * T // P) + 1)
    cache = Cache(fmt, pages, P, hkv, D, T, gap=16 * (T % 3))
    if T <= 100:
        slots = rng.permutation(pages * P)[:T]
    else:
        slots = (np.arange(T) + 5) % (pages * P)
    call = Call(cache, T, hq, rot, slots, rng.integers(0, 512, T), gap=gap, seed=D)
    call.check()


@pytest.mark.parametrize("fmt,D", FORMS)
def test_whole_head_rotates_in_place(fmt, D):
    cuda()
    cache = Cache(fmt, 5, 16, 2, D, 3)
    Call(cache, 40, 4, D, np.random.default_rng(1).permutation(80)[:40], np.arange(40), seed=1).check(in_place=True)


@pytest.mark.parametrize("fmt,D", FORMS)
def test_padding_is_left_alone(fmt, D):
    """Slots and positions outside their ranges, the first and last of a tile and a whole tile among them."""
    cuda()
    T = 70
    rng = np.random.default_rng(2)
    cache = Cache(fmt, 6, 16, 2, D, 4)
    slots, pos = rng.permutation(96)[:T].astype(np.int64), rng.integers(0, 512, T)
    slots[[0, 15, 33]] = [-1, 96, -2 ** 31]
    slots[48:64] = -1
    slots[69] = 2 ** 31 - 1
    pos[[2, 20, 21, 22]] = [-1, 512, 2 ** 31 - 1, -2 ** 31]
    Call(cache, T, 3, 32, slots, pos, seed=2).check()
    cache = Cache(fmt, 6, 16, 2, D, 4)
    Call(cache, T, 3, 0, slots, pos, seed=3).check()             # without rotation positions do not matter


def test_e4m3_rounding_and_saturation():
    """Exact codes: ties to even, subnormals, values beyond the largest, infinities and NaN."""
    cuda()
    cache = Cache("e4m3", 4, 16, 1, 64, 5)
    cache.scales = {w: np.array([0.25], np.float32) for w in "kv"}
    cache.upload()
    vals = np.array([0, -0.0, 1, -1, 448, -448, 449, 1e6, -1e30, np.inf, -np.inf, np.nan, 2.0 ** -9, 2.0 ** -10,
                     2.0 ** -11, 3 * 2.0 ** -10, 17, 19, 18, 18.5, 21, 23, 0.1, 464, 456, 240, 232, 2.0 ** -6, 2.0 ** -7,
                     1.0625, 1.1875, 1.3125], np.float32)
    call = Call(cache, 1, 0, 0, [9], [0])
    call.bits = synth.f32_to_bf16(np.tile(vals * 0.25, 4)[None, :128])
    vals = (OF.bf16_to_f64(call.bits[0, :32]) * 4).astype(np.float32)     # (bf16 holds some of them rounded)
    want = torch.from_numpy(np.clip(vals, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    call.run()
    for w in "kv":
        raw = cache.dev[w].cpu().numpy()[cache.offsets(w, [9], 0)][0]
        nan = np.isnan(np.tile(vals, 2))
        np.testing.assert_array_equal(raw[~nan], np.tile(want, 2)[~nan])
        assert ((raw[nan] & 0x7F) == 0x7F).all()


def test_special_values_in_bf16():
    cuda()
    cache = Cache("bf16", 2, 16, 1, 64, 6)
    call = Call(cache, 2, 1, 0, [0, 31], [0, 0])
    call.bits[:, ::5] = [[0x7F80], [0xFF80]]
    call.bits[:, 1::7] = 0x7FC1
    call.bits[:, 2::9] = 0x8000
    q = call.run()
    np.testing.assert_array_equal(q.reshape(2, 64), call.bits[:, :64])
    for w, first in (("k", 64), ("v", 128)):
        raw = cache.dev[w].cpu().numpy()
        off = cache.offsets(w, [0, 31], 0)
        np.testing.assert_array_equal(raw[off].astype(np.uint16) | raw[off + 1].astype(np.uint16) << 8,
                                      call.bits[:, first:first + 64])


def test_pages_beyond_32_bits():
    """Pages a GiB apart: byte offsets beyond 2^32."""
    cuda()
    stride = 1 << 30
    pool = {w: torch.zeros(6 * stride, dtype=torch.uint8, device="cuda") for w in "kv"}
    small = Cache("bf16", 6, 16, 2, 128, 7)
    call = Call(small, 96, 0, 0, np.random.default_rng(3).permutation(96), np.zeros(96))
    call.run()
    big = M.kv_cache(6, 16, 2, 128, "bf16", pool["k"].data_ptr(), pool["v"].data_ptr(), page_stride=stride)
    D = 128
    p = call.x.data_ptr()
    M.ft_kv_append(big, M.kv_append(96, p, call.row, p + 2 * 2 * D, call.row, call.keep[0].data_ptr()), stream())
    torch.cuda.synchronize()
    for w in "kv":
        got = torch.stack([pool[w][i * stride:i * stride + small.page] for i in range(6)])
        assert torch.equal(got, small.dev[w].view(6, small.page))
        assert int(pool[w].count_nonzero()) == int(got.count_nonzero())


@pytest.mark.parametrize("fmt,D,hq,hkv,rot", [("bf16", 128, 40, 4, 128), ("e4m3", 128, 40, 4, 128), ("bf16", 128, 40, 4, 32),
                                              ("bf16", 64, 90, 3, 64), ("e4m3", 64, 90, 3, 0), ("bf16", 256, 20, 2, 256),
                                              ("e4m3", 256, 20, 2, 64), ("bf16", 128, 41, 3, 128), ("e4m3", 64, 90, 4, 64)])
def test_calls_that_stream(fmt, D, hq, hkv, rot):
    """Rows of more than the L2s hold: other loads and stores, the same results; in place too."""
    cuda()
    T = 4001
    assert T * (2 * hq + 2 * hkv) * D * 2 > 32 << 20
    cache = Cache(fmt, 64, 64, hkv, D, 8)
    rng = np.random.default_rng(8)
    slots, pos = (np.arange(T) + 30) % 4096, rng.integers(0, 512, T)
    slots[::501] = -1
    call = Call(cache, T, hq, rot, slots, pos, seed=8)
    call.check(in_place=rot == D)
