"""ft_moe_layer at the borders of its launches' rules, one token's own path, and ties, NaN and infinities in routing."""
import numpy as np
import pytest
import torch

import synth
from oracle import formats as OF
from tests.gpu_util import dev_u16
from tests.resident_util import bits, config
from tests.test_gpu_moe_layer import Layer, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("d,f,E,k", [(256, 384, 6, 3), (640, 128, 65, 16), (128, 256, 255, 2), (2048, 256, 130, 9), (256, 128, 1, 1)])
def test_borders(fmt, d, f, E, k):
    """One and two operands of tokens, one and two row panels of down, one to four logits a lane, experts that are
    no multiple of four."""
    cfg = config(fmt, d, f, E, k, seed=31)
    layer = Layer(cfg, 64)
    for T in (1, 3, 4, 8, 15, 16, 17, 31, 63):
        check(layer, synth.tokens(cfg, T, T), synth.tokens(cfg, T, T, 1) if T % 2 else None,
              f"{fmt} d={d} f={f} E={E} k={k} T={T}")


@pytest.mark.parametrize("E,k", [(8, 3), (100, 8), (256, 16)])
def test_one_token_routes_as_in_a_batch(E, k):
    """A token alone is selected in another launch than a batch's: the same ids and weights, ties to the lower
    expert (-0 equals +0), NaN logits last, +inf logits first."""
    cfg = config("bf16", 256, 128, E, k, seed=32)
    layer = Layer(cfg, 8)
    x = synth.tokens(cfg, 8, 0).copy()
    wr = layer.wr.copy()
    wr[:, E - 1] = wr[:, 1]                  # two equal logits everywhere
    wr[0, E // 2] = 0x7F80                   # +inf or -inf by the sign of x[0], NaN where it is zero
    x[0, 0], x[1, 0], x[2, 0] = 0x3F80, 0xBF80, 0x0000
    x[3] = 0                                 # all equal: a NaN and zeros
    x[4] = 0x8000
    x[5, 7] = 0x7FC0                         # every logit NaN
    layer.wrd = dev_u16(wr)
    ids, w, _ = layer(x)
    for t in range(8):
        one_ids, one_w, _ = layer(x[t:t + 1])
        np.testing.assert_array_equal(one_ids[0], ids[t])
        np.testing.assert_array_equal(one_w[0], w[t])
        assert ((ids[t] >= 0) & (ids[t] < E)).all() and len(set(ids[t])) == k
    mid = E // 2
    assert ids[0, 0] == mid and mid not in ids[1]
    zeros = [e for e in range(E) if e != mid][:k]
    for t in (3, 4):
        assert list(ids[t]) == zeros
        np.testing.assert_allclose(w[t], 1.0 / k, rtol=1e-6)
    assert list(ids[5]) == list(range(k)) and np.isnan(w[5]).all()
    for t in (6, 7):                         # x[0] is an ordinary value: the equal pair stays in order
        pair = [int(e) for e in ids[t] if e in (1, E - 1)]
        assert pair in ([], [1], [1, E - 1])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_one_token_in_a_graph_and_in_place(fmt):
    """Two captured one-token calls that share a stream and a workspace, the second reading the first's y as base."""
    cfg = config(fmt, 512, 256, 40, 6, seed=33)
    layer, eager = Layer(cfg, 1), Layer(cfg, 1)
    xd = dev_u16(synth.tokens(cfg, 1, 0))
    y0, o1, o2 = dev_u16(synth.tokens(cfg, 1, 1)), layer.outputs(1), layer.outputs(1)
    o2 = (o2[0], o2[1], o1[2])

    def both():
        layer.enqueue(xd, o1, base=y0)
        layer.enqueue(xd, o2, base=o1[2])

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        both()
    for i in range(2, 6):
        x = synth.tokens(cfg, 1, i)
        xd.copy_(dev_u16(x))
        g.replay()
        torch.cuda.synchronize()
        first = eager(x, synth.tokens(cfg, 1, 1))
        second = eager(x, first[2])
        np.testing.assert_array_equal(o2[0].cpu().numpy(), second[0])
        np.testing.assert_array_equal(bits(o2[2]), second[2])


def test_records_further_apart_than_their_size():
    """A stride past the record, garbage in between."""
    cfg = config("fp8", 256, 128, 5, 2, seed=34)
    layer = Layer(cfg, 20)
    S = layer.records.shape[1]
    wide = torch.full((5, S + 4096 + (-S) % 16), 255, dtype=torch.uint8, device="cuda")
    wide[:, :S] = layer.rec[:, :S]
    want = {T: layer(synth.tokens(cfg, T, T)) for T in (1, 20)}
    layer.rec = wide
    for T, ref in want.items():
        for a, b in zip(layer(synth.tokens(cfg, T, T)), ref):
            np.testing.assert_array_equal(a, b)
    assert np.isfinite(OF.bf16_to_f64(want[20][2])).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
def test_two_and_three_launches_in_one_graph(fmt):
    """Calls of 17, 64, 16 and 2 tokens captured one after the other over one workspace, in both of its forms."""
    cfg = config(fmt, 640, 384, 24, 4, seed=35)
    layer, eager = Layer(cfg, 64), Layer(cfg, 64)
    Ts = (17, 64, 16, 2)
    xds, outs = [dev_u16(synth.tokens(cfg, T, T)) for T in Ts], [layer.outputs(T) for T in Ts]

    def all_four():
        for xd, out in zip(xds, outs):
            layer.enqueue(xd, out)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        all_four()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        all_four()
    for i in range(1, 5):
        xs = [synth.tokens(cfg, T, T, i) for T in Ts]
        for xd, x in zip(xds, xs):
            xd.copy_(dev_u16(x))
        g.replay()
        torch.cuda.synchronize()
        for x, out in zip(xs, outs):
            ids, w, y = eager(x)
            np.testing.assert_array_equal(out[0].cpu().numpy(), ids)
            np.testing.assert_array_equal(out[1].cpu().numpy(), w)
            np.testing.assert_array_equal(bits(out[2]), y)
