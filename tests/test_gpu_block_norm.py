"""ft_block_norm against its definition in 64 bits, within a bound derived for every output (tests/kv_util.py)."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from oracle import formats as OF
from tests.gpu_util import cuda, dev
from tests.kv_util import norm_reference, stream
from tests.resident_util import assert_within

pytestmark = pytest.mark.gpu


class Norm:
    def __init__(self, T, d, block=True, residual=True, post=True, pre=True, want_sum=True, kind="none", sigmoid=False,
                 scale=1.0, offset=0.0, eps=1e-6, gap=0, seed=0, size=1.0):
        rng = np.random.default_rng([seed, T, d])
        bf = lambda *s, mul=1.0, add=0.0: synth.f32_to_bf16(  # noqa: E731
            (mul * rng.standard_normal(s) + add).astype(np.float32))
        self.T, self.d, self.row = T, d, d + gap
        self.block = bf(T, self.row, mul=size) if block else None
        self.residual = bf(T, self.row, mul=2 * size) if residual else None
        self.post = bf(d, mul=0.3, add=1 - offset) if post else None
        self.pre = bf(d, mul=0.3, add=1 - offset) if pre else None
        shape = {"none": None, "channel": (d,), "token": (T,), "full": (T, self.row)}[kind]
        self.gate = bf(*shape) if shape else None
        self.want_sum, self.kind, self.sigmoid = want_sum, kind, sigmoid
        self.scale, self.offset, self.eps = scale, offset, eps

    def args(self, alias=()):
        up = lambda a: dev(a.view(np.int16)) if a is not None else None  # noqa: E731
        p = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
        self.t = {k: up(getattr(self, k)) for k in ("block", "residual", "post", "pre", "gate")}
        new = lambda: torch.full((self.T + 1, self.row), 0x5A5A, dtype=torch.int16, device="cuda")  # noqa: E731
        self.sum = self.t[alias[0]] if alias and alias[0] else new() if self.want_sum else None
        self.normed = self.t[alias[1]] if len(alias) > 1 and alias[1] else new() if self.pre is not None else None
        s = self.row
        return M.block_norm(self.T, self.d, self.eps, p(self.t["block"]), p(self.t["residual"]), p(self.t["post"]),
                            p(self.t["pre"]), p(self.t["gate"]), self.kind, self.sigmoid, p(self.sum), p(self.normed),
                            self.scale, self.offset, s, s, s, s, s)

    def result(self, t):
        a = t.cpu().numpy().view(np.uint16)
        if len(a) > self.T:
            assert (a[self.T:] == 0x5A5A).all()
            assert (a[:, self.d:] == 0x5A5A).all()
        return OF.bf16_to_f64(a[:self.T, :self.d])

    def reference(self):
        cut = lambda a: OF.bf16_to_f64(a[..., :self.d]) if a is not None else None  # noqa: E731
        gate = None if self.gate is None else OF.bf16_to_f64(self.gate if self.kind == "token" else
                                                             self.gate[..., :self.d])
        f32 = lambda v: float(np.float32(v))  # noqa: E731
        return norm_reference(cut(self.block), cut(self.residual), cut(self.post), cut(self.pre), gate, self.kind,
                              self.sigmoid, f32(self.scale), f32(self.offset), f32(self.eps))

    def check(self, alias=()):
        M.ft_block_norm(self.args(alias), stream())
        torch.cuda.synchronize()
        (s, sb), (n, nb) = self.reference()
        if self.sum is not None:
            assert_within(self.result(self.sum), s, sb, "sum")
        if self.normed is not None:
            assert_within(self.result(self.normed), n, nb, "normed")


@pytest.mark.parametrize("d", [8, 16, 64, 120, 128, 136, 512, 520, 1024, 2048, 2056, 4096, 7168, 8192, 8200, 20000, 32768])
@pytest.mark.parametrize("T", [1, 2, 33])
def test_widths(T, d):
    cuda()
    Norm(T, d, kind="full", sigmoid=True, scale=0.75, gap=8, seed=d).check()


@pytest.mark.parametrize("T", [1, 15, 16, 17, 64, 1000, 20001])
def test_tokens(T):
    cuda()
    Norm(T, 128, kind="token").check()
    if T <= 1000:
        Norm(T, 2048, kind="channel").check()


@pytest.mark.parametrize("kind,sigmoid", [("none", False), ("channel", False), ("channel", True), ("token", False),
                                          ("token", True), ("full", False), ("full", True)])
@pytest.mark.parametrize("post,residual", [(False, True), (True, True), (True, False), (False, False)])
def test_forms(kind, sigmoid, post, residual):
    cuda()
    for d in (96, 640, 2048):
        Norm(5, d, post=post, residual=residual, kind=kind, sigmoid=sigmoid, scale=-1.5, offset=1.0, seed=1).check()
        Norm(5, d, post=post, residual=residual, kind=kind, sigmoid=sigmoid, want_sum=False, seed=2).check()
        Norm(5, d, post=post, residual=residual, kind=kind, sigmoid=sigmoid, pre=False, seed=3).check()


def test_norm_alone():
    """Without a block: the norm of a scaled residual."""
    cuda()
    for d in (64, 4096, 16384):
        Norm(7, d, block=False, post=False, scale=1.0, want_sum=False, seed=4).check()
        Norm(7, d, block=False, post=False, scale=2.5, seed=5).check()


@pytest.mark.parametrize("alias", [("residual",), ("block",), ("residual", "block"), ("block", "residual"),
                                   (None, "block"), (None, "residual")])
@pytest.mark.parametrize("T,d", [(3, 64), (9, 2048), (5, 9000)])
def test_in_place(alias, T, d):
    cuda()
    Norm(T, d, kind="full", scale=0.5, seed=6).check(alias)


def test_small_and_large_values():
    """eps carries rows of zeros and of tiny values; large ones stay finite up to the stated size."""
    cuda()
    for size in (0.0, 1e-30, 1e-4, 1e10, 2.0 ** 50):
        Norm(4, 1024, size=size, kind="channel", seed=7).check()
    Norm(4, 1024, size=1e-3, eps=0.0, seed=8).check()


def test_zero_rows_without_eps_are_nan_and_only_those():
    cuda()
    n = Norm(3, 256, post=False, eps=0.0, seed=9)
    n.block[1] = 0
    n.residual[1] = 0
    M.ft_block_norm(n.args(), stream())
    torch.cuda.synchronize()
    s, m = n.result(n.sum), n.result(n.normed)
    assert (s[1] == 0).all() and np.isnan(m[1]).all() and np.isfinite(m[[0, 2]]).all()


def test_nan_stays_in_its_row():
    cuda()
    n = Norm(40, 64, kind="full", seed=10)
    n.block[17, 5] = 0x7FC0
    n.residual[3, 9] = 0x7F80
    M.ft_block_norm(n.args(), stream())
    torch.cuda.synchronize()
    s, m = n.result(n.sum), n.result(n.normed)
    ok = np.delete(np.arange(40), [3, 17])
    assert np.isfinite(s[ok]).all() and np.isfinite(m[ok]).all()
    assert np.isnan(s[17]).all() and np.isnan(m[17]).all()
    assert np.isinf(s[3, 9]) and np.isfinite(np.delete(s[3], 9)).all()


def test_captured_and_on_another_stream():
    cuda()
    n = Norm(20, 2048, kind="token", seed=11)
    a = n.args()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.ft_block_norm(a, stream())
    other = torch.cuda.Stream()
    want = None
    for i in range(3):
        n.block = n.block.copy()
        n.block[:, i] = 0x4000
        n.t["block"].copy_(dev(n.block.view(np.int16)))
        n.sum.fill_(0x5A5A)
        n.normed.fill_(0x5A5A)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        (s, sb), (m, mb) = n.reference()
        assert_within(n.result(n.sum), s, sb)
        assert_within(n.result(n.normed), m, mb)
        want = n.sum.clone(), n.normed.clone()
        M.ft_block_norm(a, other.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(n.sum, want[0]) and torch.equal(n.normed, want[1])


@pytest.mark.parametrize("T,d,kind", [(70000, 64, "token"), (40000, 128, "full"), (9000, 512, "none"), (3000, 2048, "full"),
                                      (1025, 4096, "channel"), (1500, 7168, "none"), (700, 16384, "full")])
def test_calls_that_stream(T, d, kind):
    """More than the L2s hold, in every division of a row over threads; in place too."""
    cuda()
    n = Norm(T, d, kind=kind, seed=12)
    n.check()
    if T <= 3000:
        Norm(T, d, kind=kind, seed=13).check(("residual", "block"))


@pytest.mark.parametrize("T", [1023, 1024, 1025])
@pytest.mark.parametrize("d", [520, 2048, 2304, 4104, 8192])
def test_few_and_many_rows(T, d):
    cuda()
    Norm(T, d, kind="token", sigmoid=True, scale=0.5, seed=14).check()
