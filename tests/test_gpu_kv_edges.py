"""The key-value cache's and the block norm's calls beside other work: after an error that the program left behind, in two
captured graphs at once, replayed between eager calls, and over memory that interleaves layers."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
from moe_expert_execution_amd.tensors import KvPool, Workspace
from oracle import formats as OF
from tests.gpu_util import cuda
from tests.kv_util import Cache, Plan, attend_reference, plan_reference, random_table, stream
from tests.resident_util import assert_within
from tests.test_gpu_block_norm import Norm
from tests.test_gpu_kv_append import Call
from tests.test_gpu_kv_attend import Attend, make
from tests.test_gpu_kv_plan import random_batch
from tests.test_gpu_stale_error import with_stale_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [7, 900])
def test_plan_after_a_stale_error(B):
    cuda()
    b, ws = random_batch(B, 16, 8, 3 * B, 0, 5), Workspace(16)
    p = Plan(**b)
    with_stale_error(lambda: M.ft_kv_plan(p.struct, ws.handle, stream()))
    torch.cuda.synchronize()
    got, want = p.host(), plan_reference(**b)
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    ws.close()


def test_the_others_after_a_stale_error():
    cuda()
    Call(Cache("bf16", 4, 16, 2, 64, 1), 20, 3, 32, np.arange(20), np.arange(20), seed=1).check(around=with_stale_error)
    for lens in ([5, 40], [3000]):
        make("bf16", 64, 2, 4, 16, lens, seed=2).check(around=with_stale_error)
    for d in (64, 4096):
        n = Norm(5, d, seed=3)
        args = n.args()
        torch.cuda.synchronize()
        with_stale_error(lambda: M.ft_block_norm(args, stream()))
        torch.cuda.synchronize()
        (s, sb), (m, mb) = n.reference()
        assert_within(n.result(n.sum), s, sb)
        assert_within(n.result(n.normed), m, mb)


def test_two_graphs_at_once():
    """Attentions that are cut and joined, captured over a workspace each, replayed on two streams at the same time, with
    the program's own work between the replays."""
    cuda()
    calls = [make("bf16", 128, 2, 8, 16, [6000, 70, 2500], seed=60), make("e4m3", 256, 1, 4, 32, [9000], seed=61)]
    want = [c.check() for c in calls]
    ws = [Workspace(M.ft_kv_attend_workspace(c.cache.struct(), c.hq, c.B)) for c in calls]
    args, graphs, streams = [c.args() for c in calls], [], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for c, a, w in zip(calls, args, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                M.ft_kv_attend(c.cache.struct(), a, w.handle, stream())
        graphs.append(g)
    x = torch.randn(512, 512, device="cuda")
    for _ in range(5):
        for c in calls:
            c.out.fill_(0x5A5A)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        x = torch.tanh(x @ x)
        torch.cuda.synchronize()
        for c, r in zip(calls, want):
            np.testing.assert_array_equal(c.bits()[:c.B, :c.hq * c.D].reshape(r.shape), r)
    for w in ws:
        w.close()


def test_one_workspace_for_the_plan_and_the_attention():
    """Their arrival counters are the same words, zero again after each call."""
    cuda()
    ws = Workspace(M.ft_kv_attend_workspace(make("bf16", 128, 1, 16, 16, [4000], seed=70).cache.struct(), 16, 4))
    for i in range(4):
        b = random_batch(3000, 16, 5, 9000, 0, 70 + i)
        p = Plan(in_place=True, **b)
        M.ft_kv_plan(p.struct, ws.handle, stream())
        make("bf16", 128, 1, 16, 16, [4000, 9, 700], seed=71 + i).check(ws=ws)
        got, want = p.host(), plan_reference(**b)
        for k in want:
            np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    ws.close()


def test_layers_interleaved_in_one_allocation():
    """Pages of two layers, keys and values of each, one after the other: a page_stride of four pages."""
    cuda()
    lens = [100, 37, 0, 300]
    table, pages = random_table(lens, 16, 1, 80)
    layers = [Cache("bf16", pages, 16, 2, 64, 80 + i) for i in range(2)]
    size = layers[0].page
    pool = torch.zeros(pages, 4, size, dtype=torch.uint8, device="cuda")
    for i, c in enumerate(layers):
        for j, w in enumerate("kv"):
            pool[:, 2 * i + j] = c.dev[w].view(pages, size)
    for i, c in enumerate(layers):
        a = Attend(c, table, lens, 8, seed=80)
        want = a.check()
        struct = M.kv_cache(pages, 16, 2, 64, "bf16", pool.data_ptr() + 2 * i * size, pool.data_ptr() + (2 * i + 1) * size,
                            page_stride=4 * size)
        ws = Workspace(M.ft_kv_attend_workspace(struct, 8, 4))
        M.ft_kv_attend(struct, a.args(), ws.handle, stream())
        torch.cuda.synchronize()
        np.testing.assert_array_equal(a.bits()[:4].reshape(want.shape), want)
        ws.close()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pool_of_tensors(fmt):
    """A KvPool that was appended to holds what attention reads from a cache with the same bytes."""
    cuda()
    small = Cache(fmt, 12, 32, 2, 128, 90)
    pool = KvPool(12, 32, 2, 128, fmt, *([small.dev_scales[w] for w in "kv"] if fmt == "e4m3" else []))
    call = Call(small, 300, 0, 0, np.random.default_rng(90).permutation(384)[:300], np.zeros(300), seed=90)
    call.run()
    for w, t in (("k", pool.k), ("v", pool.v)):
        t.view(torch.uint8).view(-1).copy_(small.dev[w])
    table = np.array([[3, 1, 2, 0], [9, 11, 4, 5]], np.int32)
    a = Attend(small, table, [128, 70], 16, seed=90)
    ws = Workspace(M.ft_kv_attend_workspace(pool.struct, 16, 2))
    M.ft_kv_attend(pool.struct, a.args(), ws.handle, stream())
    torch.cuda.synchronize()
    raw = {w: small.dev[w].cpu().numpy() for w in "kv"}
    ref, bound = attend_reference(small, a.q.reshape(2, 16, 128), table, [128, 70], a.scale, raw=raw)
    assert_within(OF.bf16_to_f64(a.bits()[:2].reshape(2, 16, 128)), ref, bound)
    with pytest.raises(ValueError):
        KvPool(2, 16, 1, 64, "e4m3")
    ws.close()
