"""ft_moe_layer (a whole layer for a few tokens over resident records) against the fp64 layer."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from oracle import formats as OF
from tests.gpu_util import cuda, dev, dev_u16
from tests.resident_util import HALF, assert_within, bits, config, layer_with_bound, padded

pytestmark = pytest.mark.gpu


class Layer:
    """One layer's records and router on the device, its workspace, and a call."""

    def __init__(self, cfg, max_tokens, records=None):
        from moe_expert_execution_amd.tensors import Workspace
        cuda()
        self.cfg = cfg
        self.records = synth.bank(cfg) if records is None else records
        self.rec = dev(padded(self.records))
        self.wr = synth.router(cfg, 0)
        self.wrd = dev_u16(self.wr)
        self.shape = M.shape(1, cfg.E, cfg.k, cfg.d, cfg.f, cfg.fmt)
        self.ws = Workspace(M.ft_moe_layer_workspace(self.shape, max_tokens))

    def outputs(self, T):
        c = self.cfg
        return (torch.full((T, c.k), -7, dtype=torch.int32, device="cuda"), torch.full((T, c.k), -7.0, device="cuda"),
                torch.full((T, c.d), -7, dtype=torch.int16, device="cuda"))

    def enqueue(self, xd, out, base=None, stream=None, T=None):
        ids, w, y = out
        s = (stream or torch.cuda.current_stream()).cuda_stream
        M.ft_moe_layer(self.shape, xd.data_ptr(), self.wrd.data_ptr(), self.rec.data_ptr(), self.rec.shape[1],
                       xd.shape[0] if T is None else T, 0 if base is None else base.data_ptr(), ids.data_ptr(),
                       w.data_ptr(), y.data_ptr(), self.ws.handle, s)

    def __call__(self, x, base=None):
        out = self.outputs(len(x))
        self.enqueue(dev_u16(x), out, None if base is None else dev_u16(base))
        torch.cuda.synchronize()
        return out[0].cpu().numpy(), out[1].cpu().numpy(), bits(out[2])


def check(layer, x, base=None, what=""):
    ids, w, y = layer(x, base)
    rid, rw, ref, bound, gap = layer_with_bound(x, layer.wr, layer.records, layer.cfg, base)
    assert gap > 1e-12, "inputs with a near tie decide nothing"
    np.testing.assert_array_equal(ids, rid)
    np.testing.assert_allclose(w, rw, rtol=1e-6, atol=0)
    assert_within(OF.bf16_to_f64(y), ref, bound, what)
    return ids, w, y


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("d,f,E,k", [(256, 128, 8, 2), (384, 256, 7, 7), (1152, 640, 40, 5), (2048, 768, 128, 8),
                                     (128, 128, 256, 16), (4224, 128, 3, 1)])
def test_layer_parity(fmt, d, f, E, k):
    cfg = config(fmt, d, f, E, k, seed=3)
    layer = Layer(cfg, 64)
    for T in (1, 2, 9, 32, 33, 64) if E < 128 else (1, 40):
        x = synth.tokens(cfg, T, T)
        base = synth.tokens(cfg, T, T, 1) if T % 2 else None
        check(layer, x, base, f"{fmt} d={d} f={f} E={E} k={k} T={T}")


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
def test_every_token_on_one_expert(fmt):
    """64 tokens and one expert: two full tiles of routes; 33: a second tile of one route."""
    cfg = config(fmt, 256, 256, 1, 1, seed=4)
    layer = Layer(cfg, 64)
    for T in (33, 64):
        check(layer, synth.tokens(cfg, T, T), what=f"{fmt} T={T}")


def test_large_shapes():
    """The size limits of a record: d = 32,768 (1,024 row panels) and f = 8,192."""
    for d, f in ((32768, 128), (128, 8192)):
        cfg = config("mxfp4", d, f, 4, 2, seed=5)
        layer = Layer(cfg, 3)
        check(layer, synth.tokens(cfg, 3, 0), what=f"d={d} f={f}")


def test_same_inputs_same_bits_and_rows_of_a_batch():
    """Equal inputs give equal bits, call after call."""
    cfg = config("bf16", 2048, 768, 128, 8, seed=6)
    layer = Layer(cfg, 64)
    x = synth.tokens(cfg, 64, 0)
    first = layer(x)
    for _ in range(5):
        again = layer(x)
        for a, b in zip(first, again):
            np.testing.assert_array_equal(a, b)


def test_outputs_stop_at_the_last_token():
    """Rows behind the last token stay as they were; T = 0 writes nothing."""
    cfg = config("bf16", 256, 128, 8, 2, seed=7)
    layer = Layer(cfg, 8)
    x = dev_u16(synth.tokens(cfg, 8, 0))
    out = layer.outputs(8)
    layer.enqueue(x, out, T=0)
    torch.cuda.synchronize()
    assert all((o == -7).all() for o in out)
    layer.enqueue(x, out, T=5)
    torch.cuda.synchronize()
    assert all((o[5:] == -7).all() for o in out)
    assert (out[0][:5] >= 0).all()


def test_base_in_place():
    cfg = config("bf16", 256, 128, 8, 2, seed=8)
    layer = Layer(cfg, 40)
    x, base = synth.tokens(cfg, 40, 0), synth.tokens(cfg, 40, 1)
    _, _, y = layer(x, base)
    out = layer.outputs(40)
    out[2].copy_(dev_u16(base))
    layer.enqueue(dev_u16(x), out, base=out[2])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(out[2]), y)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_token_stays_in_its_row(bad):
    """A token with a NaN or an infinity: every other row as without it, and valid ids everywhere."""
    cfg = config("bf16", 256, 128, 8, 2, seed=9)
    layer = Layer(cfg, 40)
    x = synth.tokens(cfg, 40, 0)
    clean = layer(x)
    x2 = x.copy()
    x2[17, 100] = synth.f32_to_bf16(np.array([np.inf], np.float32))[0] if np.isinf(bad) else 0x7FC0
    if bad == -np.inf:
        x2[17, 100] = 0xFF80
    got = layer(x2)
    rows = np.arange(40) != 17
    for a, b in zip(clean, got):
        np.testing.assert_array_equal(a[rows], b[rows])
    assert ((got[0][17] >= 0) & (got[0][17] < 8)).all() and len(set(got[0][17])) == 2


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_non_finite_expert_stays_with_its_tokens(fmt):
    """An expert whose weights hold NaN changes only the tokens routed to it."""
    cfg = config(fmt, 256, 256, 8, 2, seed=10)
    recs = synth.bank(cfg)
    layer = Layer(cfg, 64, recs)
    x = synth.tokens(cfg, 64, 0)
    ids, _, clean = layer(x)
    bad = recs.copy()
    codes = bad[3, :3 * cfg.d * cfg.f * (2 if fmt == "bf16" else 1)]
    codes[:] = 0x7F if fmt == "fp8" else 0xFF
    _, _, y = Layer(cfg, 64, bad)(x)
    hit = (ids == 3).any(axis=1)
    assert hit.any() and not hit.all()
    np.testing.assert_array_equal(y[~hit], clean[~hit])
    assert np.isnan(OF.bf16_to_f64(y[hit])).all()


def test_captured_graph_replays():
    """A captured call, replayed with new inputs between eager calls of another workspace."""
    cfg = config("bf16", 1152, 640, 40, 5, seed=11)
    layer, eager = Layer(cfg, 64), Layer(cfg, 64)
    T = 13
    xd = dev_u16(synth.tokens(cfg, T, 0))
    out = layer.outputs(T)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        layer.enqueue(xd, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        layer.enqueue(xd, out)
    for i in range(1, 5):
        x = synth.tokens(cfg, T, i)
        xd.copy_(dev_u16(x))
        graph.replay()
        torch.cuda.synchronize()
        ids, w, y = eager(x)
        np.testing.assert_array_equal(out[0].cpu().numpy(), ids)
        np.testing.assert_array_equal(out[1].cpu().numpy(), w)
        np.testing.assert_array_equal(bits(out[2]), y)


def test_two_streams_two_workspaces():
    """Calls on two streams at once, each with a workspace of its own."""
    cfg = config("bf16", 2048, 768, 128, 8, seed=12)
    layers = [Layer(cfg, 64), Layer(cfg, 64)]
    xs = [synth.tokens(cfg, 64, i) for i in range(2)]
    want = [l(x) for l, x in zip(layers, xs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    xd = [dev_u16(x) for x in xs]
    outs = [l.outputs(64) for l in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            layers[i].enqueue(xd[i], outs[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        np.testing.assert_array_equal(outs[i][0].cpu().numpy(), want[i][0])
        np.testing.assert_array_equal(bits(outs[i][2]), want[i][2])


def test_one_workspace_serves_other_shapes_in_turn():
    cfg1, cfg2 = config("bf16", 2048, 768, 128, 8, seed=13), config("mxfp4", 384, 256, 7, 3, seed=13)
    a, b = Layer(cfg1, 64), Layer(cfg2, 64)
    b.ws = a.ws
    for T in (64, 1, 7):
        check(a, synth.tokens(cfg1, T, T), what=f"a T={T}")
        check(b, synth.tokens(cfg2, T, T), what=f"b T={T}")


def test_refusals_with_a_workspace():
    cfg = config("bf16", 256, 128, 8, 2, seed=14)
    layer = Layer(cfg, 4)
    x = dev_u16(synth.tokens(cfg, 64, 0))
    out = layer.outputs(64)
    with pytest.raises(M.FtError, match="workspace holds"):
        layer.enqueue(x, out)
    torch.cuda.synchronize()
    assert all((o == -7).all() for o in out)
    h = layer.ws.handle
    args = [layer.shape, x.data_ptr(), layer.wrd.data_ptr(), layer.rec.data_ptr(), layer.rec.shape[1], 4, 0,
            out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), h, 0]
    for i, v, msg in ((1, x.data_ptr() + 2, "aligned"), (4, 16, "record_stride"), (4, layer.rec.shape[1] + 8, "multiple of 16"),
                      (9, out[2].data_ptr() + 1, "misaligned"), (10, 0, "workspace is null")):
        bad = list(args)
        bad[i] = v
        with pytest.raises(M.FtError, match=msg) as err:
            M.ft_moe_layer(*bad)
        assert err.value.status == M.FT_ERR_ARG
    torch.cuda.synchronize()
    assert all((o == -7).all() for o in out)


@pytest.mark.parametrize("T", [1, 5, 16])
def test_one_launch_experts_share_the_card(T):
    """Few-token calls on three streams at once, with a large product on a fourth: workgroups of each call start
    late or after others wait, and every call gives the bits it gives alone."""
    cfg = config("bf16", 2048, 768, 128, 8, seed=15)
    recs = synth.bank(cfg)
    layers = [Layer(cfg, T, recs) for _ in range(3)]
    xs = [synth.tokens(cfg, T, 20 + i) for i in range(3)]
    want = [l(x) for l, x in zip(layers, xs)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    xd = [dev_u16(x) for x in xs]
    outs = [l.outputs(T) for l in layers]
    m = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for i in range(30):
        for j in range(3):
            layers[j].enqueue(xd[j], outs[j], stream=streams[j])
        if i % 10 == 0:
            with torch.cuda.stream(streams[3]):
                m = (m @ m).clamp(-1, 1)
    torch.cuda.synchronize()
    for j in range(3):
        for got, ref in zip((outs[j][0].cpu().numpy(), outs[j][1].cpu().numpy(), bits(outs[j][2])), want[j]):
            np.testing.assert_array_equal(got, ref)
