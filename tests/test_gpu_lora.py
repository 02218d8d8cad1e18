"""ft_lora_project and ft_lora_expert against fp64, and a layer step of ft_moe_layer beside a shared expert."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from oracle import formats as OF
from tests.gpu_util import cuda, dev, dev_u16
from tests.resident_util import (Pool, assert_within, bits, config, expert_with_bound, layer_with_bound, mixed_ids,
                                 padded, project_with_bound)

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "fp8", "mxfp4"]


class Project:
    """A resident matrix W [n x K]: the down matrix of a record (rows d = n, K = f)."""

    def __init__(self, fmt, n, K, max_rank, max_tokens, seed=0):
        from moe_expert_execution_amd.tensors import Workspace
        cuda()
        cfg = config(fmt, n, K, 1, 1, seed)
        rec = synth.bank(cfg)[0]
        self.W = OF.decode_record(rec, fmt, n, K)[2]                # [K x n]
        cb = n * K * {"bf16": 4, "fp8": 2, "mxfp4": 1}[fmt] // 2
        sb = {"bf16": 0, "fp8": 4 * (n // 128) * (K // 128), "mxfp4": n * K // 32}[fmt]
        self.codes, self.scales = dev(rec[2 * cb:3 * cb].copy()), dev(np.append(rec[3 * cb + 2 * sb:3 * cb + 3 * sb], np.uint8(0)))
        self.m = M.matrix(n, K, fmt, self.codes.data_ptr(), self.scales.data_ptr())
        self.n, self.K = n, K
        self.ws = Workspace(M.ft_lora_project_workspace(self.m, max_rank, max_tokens))

    def enqueue(self, pool, xd, idd, y, base=None, T=None, stream=None):
        s = (stream or torch.cuda.current_stream()).cuda_stream
        M.ft_lora_project(self.m, pool.struct if pool is not None else None, xd.data_ptr(),
                          idd.data_ptr() if idd is not None else 0, xd.shape[0] if T is None else T,
                          base.data_ptr() if base is not None else 0, y.data_ptr(), self.ws.handle, s)

    def __call__(self, x, pool=None, ids=None, base=None):
        y = torch.full((len(x), self.n), -7, dtype=torch.int16, device="cuda")
        keep = (dev_u16(x), dev(ids) if ids is not None else None, dev_u16(base) if base is not None else None)
        self.enqueue(pool, keep[0], keep[1], y, keep[2])
        torch.cuda.synchronize()
        return bits(y)


class Expert:
    def __init__(self, fmt, d, f, max_rank, max_tokens, seed=0):
        from moe_expert_execution_amd.tensors import Workspace
        cuda()
        cfg = config(fmt, d, f, 1, 1, seed)
        rec = synth.bank(cfg)
        self.mats = OF.decode_record(rec[0], fmt, d, f)
        self.rec = dev(padded(rec))
        self.shape = M.shape(1, 1, 1, d, f, fmt)
        self.cfg, self.d = cfg, d
        self.ws = Workspace(M.ft_lora_expert_workspace(self.shape, max_rank, max_tokens))

    def enqueue(self, pools, xd, idd, y, base=None, T=None, stream=None):
        s = (stream or torch.cuda.current_stream()).cuda_stream
        p = [q.struct if q is not None else None for q in pools]
        M.ft_lora_expert(self.shape, self.rec.data_ptr(), *p, xd.data_ptr(), idd.data_ptr() if idd is not None else 0,
                         xd.shape[0] if T is None else T, base.data_ptr() if base is not None else 0, y.data_ptr(),
                         self.ws.handle, s)

    def __call__(self, x, pools=(None, None, None), ids=None, base=None):
        y = torch.full((len(x), self.d), -7, dtype=torch.int16, device="cuda")
        keep = (dev_u16(x), dev(ids) if ids is not None else None, dev_u16(base) if base is not None else None)
        self.enqueue(pools, keep[0], keep[1], y, keep[2])
        torch.cuda.synchronize()
        return bits(y)


def x_of(T, K, *tag):
    return synth.tokens(config("bf16", K, 128, 1, 1), T, *tag)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,K,count,R", [(256, 128, 3, 16), (384, 1152, 7, 48), (128, 4224, 33, 128), (2048, 2048, 6, 64)])
def test_project_parity(fmt, n, K, count, R):
    pr = Project(fmt, n, K, R, 200, seed=2)
    pool = Pool(count, R, K, n, 2)
    pd = pool.device()
    for T in (1, 2, 31, 33, 64, 65, 200):
        x, ids = x_of(T, K, T), mixed_ids(T, count, 2, run=1 if T <= 64 else 9)
        base = x_of(T, n, T, 1) if T % 2 else None
        ref, bound = project_with_bound(x, pr.W, pool, ids, base)
        assert_within(OF.bf16_to_f64(pr(x, pd, ids, base)), ref, bound, f"{fmt} n={n} K={K} T={T}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,f,count,R", [(256, 128, 3, 16), (384, 256, 5, 32), (1152, 640, 9, 128)])
def test_expert_parity(fmt, d, f, count, R):
    ex = Expert(fmt, d, f, R, 300, seed=3)
    pools = [Pool(count, R, d, f, 31), Pool(count, 16, d, f, 32), Pool(count, R, f, d, 33)]
    pds = [p.device() for p in pools]
    for T, use in ((1, (0, 1, 2)), (5, (0,)), (33, (1, 2)), (64, (0, 1, 2)), (65, (2,)), (300, (0, 1, 2))):
        x, ids = x_of(T, d, T), mixed_ids(T, count, 3, run=1 if T <= 64 else 40)
        base = x_of(T, d, T, 1) if T % 2 else None
        ps = [pools[i] if i in use else None for i in range(3)]
        ref, bound = expert_with_bound(x, ex.mats, ps, ids, base)
        got = ex(x, [pds[i] if i in use else None for i in range(3)], ids, base)
        assert_within(OF.bf16_to_f64(got), ref, bound, f"{fmt} d={d} f={f} T={T} pools={use}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [700, 1500, 4096])
def test_prompt_lengths(fmt, T):
    """Long batches of a few requests of ragged lengths, and one whose adapters change with every token."""
    d, f, count, R = 512, 384, 4, 32
    ex, pr = Expert(fmt, d, f, R, T, seed=4), Project(fmt, d, f, R, T, seed=4)
    pools = [Pool(count, R, d, f, 41), Pool(count, R, d, f, 42), Pool(count, R, f, d, 43)]
    pds = [p.device() for p in pools]
    x, xf, base = x_of(T, d, T), x_of(T, f, T), x_of(T, d, T, 1)
    for run in (300, 1):
        ids = mixed_ids(T, count, 4, run=run)
        ref, bound = expert_with_bound(x, ex.mats, pools, ids, base)
        assert_within(OF.bf16_to_f64(ex(x, pds, ids, base)), ref, bound, f"expert {fmt} T={T} run={run}")
        ref, bound = project_with_bound(xf, pr.W, pools[2], ids)
        assert_within(OF.bf16_to_f64(pr(xf, pds[2], ids)), ref, bound, f"project {fmt} T={T} run={run}")


@pytest.mark.parametrize("T", [3, 64, 600])
def test_without_adapters(T):
    """No pool, an empty pool, and a pool that no token names: the same bits."""
    K, n = 384, 256
    pr = Project("bf16", n, K, 16, T, seed=5)
    x = x_of(T, K, 0)
    plain = pr(x)
    ref, bound = project_with_bound(x, pr.W, None, None)
    assert_within(OF.bf16_to_f64(plain), ref, bound)
    pd = Pool(2, 16, K, n, 5).device()
    np.testing.assert_array_equal(pr(x, pd, np.full(T, -1, np.int32)), plain)
    pd.struct.count = 0
    np.testing.assert_array_equal(pr(x, pd, np.zeros(T, np.int32)), plain)


@pytest.mark.parametrize("T", [40, 600])
def test_non_finite_adapter_stays_with_its_requests(T):
    """NaN and infinities of one adapter, and of one token, reach no other row."""
    d, f = 256, 256
    ex = Expert("bf16", d, f, 32, T, seed=6)
    pools = [Pool(3, 32, d, f, 61), Pool(3, 32, d, f, 62), Pool(3, 32, f, d, 63)]
    x, ids = x_of(T, d, 0), mixed_ids(T, 3, 6, run=3)
    clean = ex(x, [p.device() for p in pools], ids)
    for p in pools:
        p.a[0, 0, ::2] = 0x7F80
        p.b[0, ::3, 0] = 0x7FC0
    got = ex(x, [p.device() for p in pools], ids)
    hit = ids == 0
    assert hit.any() and not hit.all()
    np.testing.assert_array_equal(got[~hit], clean[~hit])
    assert not np.isfinite(OF.bf16_to_f64(got[hit])).any()
    x2 = x.copy()
    x2[7, 3] = 0x7FC0
    got = ex(x2, (None, None, None))
    rows = np.arange(T) != 7
    np.testing.assert_array_equal(got[rows], ex(x)[rows])
    assert np.isnan(OF.bf16_to_f64(got[7])).all()


@pytest.mark.parametrize("T", [20, 64, 700])
def test_same_bits_rows_behind_and_base_in_place(T):
    d, f, R = 512, 256, 32
    ex = Expert("mxfp4", d, f, R, T, seed=7)
    pds = [Pool(4, R, d, f, 71).device(), Pool(4, R, d, f, 72).device(), Pool(4, R, f, d, 73).device()]
    x, base, ids = x_of(T, d, 0), x_of(T, d, 1), mixed_ids(T, 4, 7, run=20)
    want = ex(x, pds, ids, base)
    xd, idd = dev_u16(x), dev(ids)
    y = dev_u16(base)
    for _ in range(3):
        np.testing.assert_array_equal(ex(x, pds, ids, base), want)
    ex.enqueue(pds, xd, idd, y, base=y)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y), want)
    y = dev_u16(base)
    ex.enqueue(pds, xd, idd, y, T=0)
    ex.enqueue(pds, xd, idd, y, base=y, T=T - 3)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y)[T - 3:], base[T - 3:])


def test_graph_and_second_stream():
    """A captured expert call and eager calls on another stream with a workspace of their own."""
    d, f, R = 512, 384, 32
    for T in (9, 500):
        a, b = Expert("bf16", d, f, R, T, seed=8), Expert("bf16", d, f, R, T, seed=8)
        pds = [Pool(4, R, d, f, 81).device(), Pool(4, R, d, f, 82).device(), Pool(4, R, f, d, 83).device()]
        ids = mixed_ids(T, 4, 8, run=10)
        xd, idd = dev_u16(x_of(T, d, 0)), dev(ids)
        y = torch.empty(T, d, dtype=torch.int16, device="cuda")
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            a.enqueue(pds, xd, idd, y)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            a.enqueue(pds, xd, idd, y)
        for i in range(1, 4):
            x = x_of(T, d, i)
            xd.copy_(dev_u16(x))
            g.replay()
            want = b(x, pds, ids)
            torch.cuda.synchronize()
            np.testing.assert_array_equal(bits(y), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_layer_step_with_shared_expert(fmt):
    """A decode step as it is used: the shared expert with the requests' adapters adds to the residual, the
    routed layer adds to that, one stream and one workspace, eagerly and as a captured graph."""
    from moe_expert_execution_amd.tensors import Workspace
    d, f, E, k, T, R = 512, 256, 16, 4, 11, 32
    cfg = config(fmt, d, f, E, k, seed=9)
    recs, wr = synth.bank(cfg), synth.router(cfg, 0)
    ex = Expert(fmt, d, 384, R, T, seed=10)
    pools = [Pool(4, R, d, 384, 91), Pool(4, R, d, 384, 92), Pool(4, R, 384, d, 93)]
    pds = [p.device() for p in pools]
    shape = M.shape(1, E, k, d, f, fmt)
    ws = Workspace(max(M.ft_moe_layer_workspace(shape, T), M.ft_lora_expert_workspace(ex.shape, R, T)))
    ex.ws = ws
    rec, wrd = dev(padded(recs)), dev_u16(wr)
    ids = mixed_ids(T, 4, 9)
    idd = dev(ids)
    xd = dev_u16(x_of(T, d, 0))
    resd = dev_u16(x_of(T, d, 1))
    rid = torch.empty(T, k, dtype=torch.int32, device="cuda")
    rw = torch.empty(T, k, device="cuda")
    y = torch.empty(T, d, dtype=torch.int16, device="cuda")

    def step():
        s = torch.cuda.current_stream()
        ex.enqueue(pds, xd, idd, y, base=resd, stream=s)
        M.ft_moe_layer(shape, xd.data_ptr(), wrd.data_ptr(), rec.data_ptr(), rec.shape[1], T, y.data_ptr(),
                       rid.data_ptr(), rw.data_ptr(), y.data_ptr(), ws.handle, s.cuda_stream)

    def check(x, res):
        shared, ds = expert_with_bound(x, ex.mats, pools, ids, res)
        oid, ow, routed, dr, gap = layer_with_bound(x, wr, recs, cfg)
        assert gap > 1e-12
        np.testing.assert_array_equal(rid.cpu().numpy(), oid)
        np.testing.assert_allclose(rw.cpu().numpy(), ow, rtol=1e-6)
        # dr holds the rounding of the routed part alone; the sum's is another half step
        assert_within(OF.bf16_to_f64(bits(y)), shared + routed, ds + dr + 2.0 ** -8 * (np.abs(shared + routed) + ds + dr))

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    check(x_of(T, d, 0), x_of(T, d, 1))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step()
    for i in range(2, 5):
        x, res = x_of(T, d, i), x_of(T, d, i, 1)
        xd.copy_(dev_u16(x))
        resd.copy_(dev_u16(res))
        g.replay()
        torch.cuda.synchronize()
        check(x, res)


def test_refusals_on_the_device():
    pr = Project("bf16", 256, 256, 16, 4, seed=11)
    pd = Pool(2, 16, 256, 256, 11).device()
    x = dev_u16(x_of(600, 256, 0))
    idd = dev(np.zeros(600, np.int32))
    y = torch.full((600, 256), -7, dtype=torch.int16, device="cuda")
    with pytest.raises(M.FtError, match="workspace holds"):
        pr.enqueue(pd, x, idd, y)
    with pytest.raises(M.FtError, match="adapter is null"):
        pr.enqueue(pd, x, None, y, T=2)
    from moe_expert_execution_amd.tensors import LoraPool
    with pytest.raises(ValueError):
        LoraPool(pd.a, pd.b, pd.rank.cpu(), pd.scale)
    with pytest.raises(ValueError):
        LoraPool(pd.a, pd.b[:, :, :8], pd.rank, pd.scale)
    torch.cuda.synchronize()
    assert (y == -7).all()
