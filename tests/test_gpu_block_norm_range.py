"""ft_block_norm over rows of every size that bf16 has, where a plain sum of squares leaves fp32's range, with no eps or one
of the squares' size."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from oracle import formats as OF
from tests.gpu_util import cuda
from tests.kv_util import stream
from tests.resident_util import assert_within
from tests.test_gpu_block_norm import Norm

pytestmark = pytest.mark.gpu

SIZES = [2.0 ** e for e in (-130, -124, -100, -70, -64, -55, -50, -45, -30, 0, 50, 58, 64, 80, 110, 122)]


class Rows(Norm):
    """Row t of block and residual is of size sizes[t % len(sizes)]."""

    def __init__(self, T, d, sizes=SIZES, **kw):
        super().__init__(T, d, **kw)
        f = np.array(sizes)[np.arange(T) % len(sizes)][:, None]
        for name in ("block", "residual"):
            if getattr(self, name) is not None:
                setattr(self, name, synth.f32_to_bf16((OF.bf16_to_f64(getattr(self, name)) * f).astype(np.float32)))


# a thread per 8, a wave, a workgroup with a unit a thread or two, and the widest
WIDTHS = [8, 64, 120, 512, 2048, 4096, 8192, 20000, 32768]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -126, 2.0 ** -110, 2.0 ** -99, 1e-6])
def test_rows_of_every_size(d, eps):
    cuda()
    T = 2 * len(SIZES) + 1
    Rows(T, d, eps=eps, seed=1).check()                                        # both norms
    Rows(T, d, eps=eps, post=False, seed=2).check()                            # the sum of two of one size
    Rows(T, d, eps=eps, block=False, post=False, want_sum=False, seed=3).check()
    Rows(T, d, eps=eps, residual=False, kind="channel", seed=4).check()        # a norm of a norm


@pytest.mark.parametrize("d", [64, 2048, 4104, 8192])
def test_many_rows_of_every_size(d):
    """More rows than a thread a unit is taken for, in place."""
    cuda()
    Rows(1040, d, eps=0.0, post=False, seed=5).check(("residual", "block"))
    Rows(1040, d, eps=0.0, seed=6).check()


@pytest.mark.parametrize("d", [16, 256, 4096])
def test_one_large_value_among_small_ones(d):
    """Its square alone leaves the range; the small ones' share of the row stays theirs."""
    cuda()
    for large, rest in ((2.0 ** 100, 2.0 ** 20), (2.0 ** -60, 2.0 ** -120), (2.0 ** 127, 1.0)):
        n = Norm(5, d, block=False, post=False, want_sum=False, eps=0.0, size=rest / 2, seed=7)
        n.residual[:, 3] = synth.f32_to_bf16(np.full(5, large, np.float32))
        n.check()


@pytest.mark.parametrize("d", [64, 2048])
def test_infinities_and_nan_beside_rows_of_every_size(d):
    """An infinite value's row is 0 but for itself, NaN; a NaN's row is NaN; the other rows are as they were."""
    cuda()
    T = len(SIZES)
    n = Rows(T, d, eps=0.0, block=False, post=False, want_sum=False, seed=8)
    n.residual[4, 1] = 0x7F80
    n.residual[9, 2] = 0x7FC0
    M.ft_block_norm(n.args(), stream())
    torch.cuda.synchronize()
    got = n.result(n.normed)
    assert np.isnan(got[4, 1]) and (np.delete(got[4], 1) == 0).all() and np.isnan(got[9]).all()
    n.residual[4, 1], n.residual[9, 2] = 0x3F80, 0x3F80
    keep = np.delete(np.arange(T), [4, 9])
    ref, bound = n.reference()[1]
    assert_within(got[keep], ref[keep], bound[keep])
