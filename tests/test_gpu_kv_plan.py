"""ft_kv_plan against its definition, integers equal: shapes of batches, shortage, ended requests, values out of range,
in place, captured."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
from moe_expert_execution_amd.tensors import Workspace
from tests.gpu_util import cuda
from tests.kv_util import Plan, plan_reference, stream

pytestmark = pytest.mark.gpu


def random_batch(B, P, width, tokens, row_tokens, seed, ended=0.1, idle=0.1, free=None):
    rng = np.random.default_rng([seed, B, P, width, tokens])
    room = width * P
    context = rng.integers(0, max(1, room - room // 4), B)
    most = row_tokens if row_tokens else max(1, min(2 * tokens // max(B, 1), room // 4 + 1))
    add = rng.integers(1, most + 1, B)
    add[rng.random(B) < idle] = 0
    add[rng.random(B) < ended] = rng.choice([-1, -7, -2 ** 31])
    have = -(-context // P)
    lacks = int((-(-(context + np.maximum(add, 0)) // P) - have).sum())
    free = lacks + 3 if free is None else int(lacks * free)
    pages = max(1, int(have.sum()) + free)
    ids = rng.permutation(pages)
    table = np.full((B, width), -5, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    stack = np.full(pages, -3, np.int64)
    stack[:free] = ids[at:at + free]
    return dict(context=context, add=add, table=table, free_pages=stack, free_count=free, pages=pages, P=P,
                tokens=tokens, row_tokens=row_tokens)


def compare(batch, in_place=False, what=""):
    ws = Workspace(16)
    p = Plan(in_place=in_place, **batch)
    M.ft_kv_plan(p.struct, ws.handle, stream())
    torch.cuda.synchronize()
    got, want = p.host(), plan_reference(**batch)
    for k in ("counts", "kv_len", "start", "slot", "pos", "table", "free"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=f"{what} {k}")
    ws.close()
    return want


SHAPES = [(1, 16, 1, 1, 1), (1, 16, 4, 40, 0), (2, 256, 3, 600, 0), (63, 16, 40, 63, 1), (64, 32, 9, 64, 1),
          (65, 64, 5, 200, 3), (257, 16, 7, 1000, 0), (1023, 128, 6, 5000, 0), (1024, 16, 3, 1024, 1),
          (1025, 32, 11, 9000, 0), (3000, 16, 5, 24001, 8), (4096, 16, 4, 4096, 1), (4095, 64, 3, 65535, 0),
          (4096, 16, 9, 65535, 0)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("free", [None, 0.5, 0.0])
@pytest.mark.parametrize("B,P,width,tokens,row_tokens", SHAPES)
def test_batches(B, P, width, tokens, row_tokens, free, in_place):
    cuda()
    compare(random_batch(B, P, width, tokens, row_tokens, 1, free=free), in_place)


@pytest.mark.parametrize("B,tokens,row_tokens", [(64, 4032, 0), (64, 4033, 0), (256, 16128, 0), (256, 16129, 0), (256, 256, 1),
                                                 (512, 512, 1), (513, 3000, 0), (2048, 2048, 1), (2049, 9000, 0), (7, 65535, 0)])
def test_borders_of_the_workgroups(B, tokens, row_tokens):
    """Either side of the sizes at which a call takes other workgroups."""
    cuda()
    for in_place in (False, True):
        compare(random_batch(B, 16, 12, tokens, row_tokens, B, free=0.6), in_place)


@pytest.mark.parametrize("ended,idle", [(1.0, 0.0), (0.0, 1.0), (0.9, 0.5), (0.0, 0.0)])
def test_ended_and_idle(ended, idle):
    cuda()
    for B, tokens, rows in ((1, 5, 0), (100, 100, 1), (2000, 20000, 0)):
        compare(random_batch(B, 16, 20, tokens, rows, 2, ended, idle, free=0.7), True)


def test_refusals_for_room_and_rows():
    """Requests that pass the table's width, the packed rows or their padded rows are refused; the others are served."""
    cuda()
    base = dict(table=np.array([[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, 5, 6], [7, -1, -1, -1]]),
                free_pages=np.r_[8:20, np.full(8, -1)], free_count=12, pages=20, P=16)
    ctx = [20, 5, 64, 16]
    w = compare(dict(context=ctx, add=[50, 60, 0, 48], tokens=200, row_tokens=0, **base))
    assert w["counts"][3] == 2 and w["kv_len"].tolist() == [20, 5, 64, 64]
    w = compare(dict(context=ctx, add=[10, 30, 1, 48], tokens=41, row_tokens=0, **base))
    assert w["kv_len"].tolist() == [30, 35, 64, 16] and w["start"].tolist() == [0, 10, 40, 41, 41]
    w = compare(dict(context=ctx, add=[2, 3, 0, 4], tokens=15, row_tokens=3, **base))
    assert w["kv_len"].tolist() == [22, 8, 64, 16] and w["counts"][3] == 1
    compare(dict(context=ctx, add=[2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1], tokens=0, row_tokens=0, **base))


def test_values_out_of_range():
    """Contexts and counts outside their ranges are clamped; ids outside the pool give slot -1 and reach no memory."""
    cuda()
    base = dict(table=np.array([[0, 99], [-4, 2], [2 ** 31 - 1, 3]]), pages=6, P=16, tokens=12, row_tokens=4)
    compare(dict(context=[-5, 17, 40], add=[2, 2, -1], free_pages=np.arange(6), free_count=2, **base))
    compare(dict(context=[2 ** 31 - 1, 30, 15], add=[0, 3, 4], free_pages=[77, -1, 4, 5, 0, 1], free_count=900, **base))
    compare(dict(context=[-2 ** 31, 1, 1], add=[4, -1, 1], free_pages=np.arange(6), free_count=-3, **base))
    # a table that names pages twice returns more than the list can hold: it keeps `pages` of them
    table = np.tile(np.arange(4), (5, 1))
    compare(dict(context=[64] * 5, add=[-1] * 5, table=table, free_pages=np.arange(4), free_count=3, pages=4, P=16,
                 tokens=5, row_tokens=1))


def test_decode_loop_in_place_captured():
    """Steps of a captured decode batch: lengths, the free list and the count advance in place over replays, as the
    definition applied step by step."""
    cuda()
    B, P, width, pages = 37, 16, 6, 120
    rng = np.random.default_rng(3)
    b = random_batch(B, P, width, B, 1, 4, ended=0.0, idle=0.0)
    b["pages"] = max(pages, b["pages"])
    b["free_pages"] = np.r_[b["free_pages"], np.full(b["pages"] - len(b["free_pages"]), -1)]
    p, ws = Plan(in_place=True, **b), Workspace(16)
    state = {k: np.array(b[k]) for k in ("context", "table", "free_pages")}
    count = b["free_count"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.ft_kv_plan(p.struct, ws.handle, stream())
    for step in range(60):
        add = rng.choice([1, 1, 1, 1, 0, -1], B)
        p.add.copy_(torch.from_numpy(add.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        got = p.host()
        want = plan_reference(state["context"], add, state["table"], state["free_pages"], count, b["pages"], P, B, 1)
        for k in ("counts", "kv_len", "start", "slot", "pos", "table", "free"):
            np.testing.assert_array_equal(got[k], want[k], err_msg=f"step {step} {k}")
        state = {"context": want["kv_len"], "table": want["table"], "free_pages": state["free_pages"].copy()}
        count = int(want["counts"][2])
        state["free_pages"][:count] = want["free"]
        # pages are owned once
        own = np.concatenate([want["table"][r, :-(-int(n) // P)] for r, n in enumerate(want["kv_len"])] + [want["free"]])
        assert len(set(own.tolist())) == len(own)
    ws.close()
