"""The shrink launch with two slots (of 16 ranks of a projection) to a workgroup, which prompts take whose x exceeds
the L2s: odd numbers of slots, gate and up sharing a workgroup, pools of other ranks and counts, one pool alone."""
import numpy as np
import pytest

from oracle import formats as OF
from tests.resident_util import Pool, assert_within, expert_with_bound, mixed_ids, project_with_bound
from tests.test_gpu_lora import Expert, Project, x_of

pytestmark = pytest.mark.gpu

T = 2750
# n, K, count, rank
PROJECTS = [(256, 7168, 5, 48), (384, 7168, 3, 128)]
# d, f, (count, rank) of gate, up and down; None without the pool
EXPERTS = [(7168, 128, (5, 48), (3, 16), (4, 32)), (7168, 128, (3, 16), (5, 64), None), (7168, 256, (70, 48), None, (2, 16)),
           (7168, 128, None, (4, 48), None)]


@pytest.mark.parametrize("n,K,count,R", PROJECTS)
def test_project(n, K, count, R):
    pr = Project("bf16", n, K, R, T, seed=71)
    pool = Pool(count, R, K, n, 71)
    x, base = x_of(T, K, 0), x_of(T, n, 1)
    for run in (1, 500):
        ids = mixed_ids(T, count, 71, run=run)
        ref, bound = project_with_bound(x, pr.W, pool, ids, base)
        assert_within(OF.bf16_to_f64(pr(x, pool.device(), ids, base)), ref, bound, f"n={n} R={R} run={run}")


@pytest.mark.parametrize("d,f,gate,up,down", EXPERTS)
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_expert(fmt, d, f, gate, up, down):
    made = [Pool(p[0], p[1], *((f, d) if i == 2 else (d, f)), 72 + i) if p else None
            for i, p in enumerate((gate, up, down))]
    ex = Expert(fmt, d, f, max(p.max_rank for p in made if p), T, seed=72)
    x, base = x_of(T, d, 0), x_of(T, d, 1)
    for run in (1, 500):
        ids = mixed_ids(T, max(p.count for p in made if p), 72, run=run)
        ref, bound = expert_with_bound(x, ex.mats, made, ids, base)
        got = ex(x, [p.device() if p else None for p in made], ids, base)
        assert_within(OF.bf16_to_f64(got), ref, bound, f"{fmt} {gate} {up} {down} run={run}")


def test_non_finite_adapter_stays_with_its_requests():
    n, K, count, R = 256, 7168, 3, 48
    pr = Project("bf16", n, K, R, T, seed=73)
    pool = Pool(count, R, K, n, 73)
    x, ids = x_of(T, K, 0), mixed_ids(T, count, 73, run=7)
    clean = pr(x, pool.device(), ids)
    pool.a[0, 0, ::2] = 0x7F80
    pool.b[0, :, 0] = 0x7FC0
    got = pr(x, pool.device(), ids)
    hit = ids == 0
    np.testing.assert_array_equal(got[~hit], clean[~hit])
    assert not np.isfinite(OF.bf16_to_f64(got[hit])).any()
