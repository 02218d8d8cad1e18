"""The hand-over from gate/up to down inside ft_moe_layer's one-launch form (up to 16 tokens), its two rare parts forced
from the host by variables that a workspace reads when it is created."""
import numpy as np
import pytest
import torch

import synth
from oracle import formats as OF
from tests.gpu_util import cuda
from tests.resident_util import config
from tests.test_gpu_moe_layer import Layer, check

pytestmark = pytest.mark.gpu


def layer_with(monkeypatch, name, value, cfg, max_tokens, recs):
    cuda()
    monkeypatch.setenv(name, value)
    layer = Layer(cfg, max_tokens, recs)
    monkeypatch.delenv(name)
    return layer


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T", [1, 5, 16])
@pytest.mark.parametrize("d,f,E,k,whole", [(2048, 768, 16, 8, True), (8192, 128, 8, 2, False)])
def test_wait_that_runs_out_leaves_nan(monkeypatch, fmt, T, d, f, E, k, whole):
    """The lower half of the workgroups gives up its wait at once (FTMOE_LAYER_WAIT_POLLS=0).  Where row panels have
    several splits (d = 2,048: the lower half holds some of each panel's) y is NaN everywhere, whoever adds the
    splits; with one split, in the lower panels alone, and the others have the ordinary bits.  Every kernel ends, and
    the workspace serves other calls."""
    cfg = config(fmt, d, f, E, k, seed=41)
    recs = synth.bank(cfg)
    ordinary = Layer(cfg, 40, recs)
    low = layer_with(monkeypatch, "FTMOE_LAYER_WAIT_POLLS", "0", cfg, 40, recs)
    for i in range(3):                       # (h of the call before lies in the workspace)
        x = synth.tokens(cfg, T, T, i)
        ids, w, y = low(x)
        oids, ow, oy = ordinary(x)
        np.testing.assert_array_equal(ids, oids)
        np.testing.assert_array_equal(w, ow)
        assert np.isfinite(OF.bf16_to_f64(oy)).all()
        nan = np.isnan(OF.bf16_to_f64(y))
        if whole:
            assert nan.all()
        else:
            np.testing.assert_array_equal(nan, np.broadcast_to(np.arange(d) < d // 2, (T, d)))
            np.testing.assert_array_equal(y[~nan], oy[~nan])
    check(low, synth.tokens(cfg, 40, 0), what="three launches over the same workspace")


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
@pytest.mark.parametrize("d,f,E,k", [(2048, 768, 16, 8), (256, 640, 8, 2), (8192, 128, 8, 2)])
def test_waiting_workgroups_do_the_work_of_absent_ones(monkeypatch, fmt, T, d, f, E, k):
    """Odd workgroups draw no gate/up number when they start (FTMOE_LAYER_ABSENT): half of the numbers, whose counters
    nobody else draws from at first, are found and done by workgroups that wait, and each of those loads its first down
    weights again.  The bits are those of the ordinary call; MXFP4 from 32 routes on has two row panels."""
    cfg = config(fmt, d, f, E, k, seed=42)
    recs = synth.bank(cfg)
    ordinary = Layer(cfg, T, recs)
    absent = layer_with(monkeypatch, "FTMOE_LAYER_ABSENT", "1", cfg, T, recs)
    for i in range(3):
        x = synth.tokens(cfg, T, T, i)
        base = synth.tokens(cfg, T, T, i, 1) if i else None
        if i == 0:
            check(ordinary, x, base, f"{fmt} T={T}")
        for got, want in zip(absent(x, base), ordinary(x, base)):
            np.testing.assert_array_equal(got, want)
