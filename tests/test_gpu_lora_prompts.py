"""ft_lora_project and ft_lora_expert at prompt lengths on both sizes of GEMM tiles, and calls that leave them:
wide ranges of block scales, large pools, outputs off the 16-byte grid."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
from oracle import formats as OF
from tests.gpu_util import dev, dev_u16
from tests.resident_util import Pool, assert_within, bits, expert_with_bound, mixed_ids, project_with_bound
from tests.test_gpu_lora import FMTS, Expert, Project, x_of

pytestmark = pytest.mark.gpu


# A tile is 128 x 256, or 64 x 128 while those are fewer than the 256 compute units.  Full tiles with 1, 52 and 92
# rows in the last one and with half a tile of columns; half tiles with one row, and with all of theirs.
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,K,count,R,T", [(4096, 128, 3, 16, 2049), (4096, 384, 5, 48, 2100), (4096, 128, 4, 128, 2140),
                                           (1152, 128, 4, 32, 6600), (1152, 640, 9, 128, 513), (4096, 2048, 6, 64, 192)])
def test_project_tiles(fmt, n, K, count, R, T):
    pr = Project(fmt, n, K, R, T, seed=21)
    pool = Pool(count, R, K, n, 21)
    x, base = x_of(T, K, T), x_of(T, n, T, 1)
    for run in (1, 500):
        ids = mixed_ids(T, count, 21, run=run)
        ref, bound = project_with_bound(x, pr.W, pool, ids, base)
        assert_within(OF.bf16_to_f64(pr(x, pool.device(), ids, base)), ref, bound, f"{fmt} n={n} K={K} T={T} run={run}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,f,T", [(128, 1024, 4100), (2048, 128, 4100), (640, 384, 777)])
def test_expert_tiles(fmt, d, f, T):
    """Gate/up on full tiles, down on full tiles, both on half ones; all pools, and one or two of them."""
    count, R = 4, 48
    ex = Expert(fmt, d, f, R, T, seed=22)
    pools = [Pool(count, R, d, f, 221), Pool(count, 16, d, f, 222), Pool(count, R, f, d, 223)]
    x, base, ids = x_of(T, d, T), x_of(T, d, T, 1), mixed_ids(T, count, 22, run=200)
    for use in ((0, 1, 2), (1,), (0, 2)):
        ps = [pools[i] if i in use else None for i in range(3)]
        ref, bound = expert_with_bound(x, ex.mats, ps, ids, base)
        got = ex(x, [p.device() if p is not None else None for p in ps], ids, base)
        assert_within(OF.bf16_to_f64(got), ref, bound, f"{fmt} d={d} f={f} T={T} pools={use}")


@pytest.mark.parametrize("n,T", [(4096, 2100), (512, 2100)])
def test_tiles_without_adapters_and_in_place(n, T):
    """No pool and a pool that no token names give the same bits; base in place; rows behind are left."""
    K = 256
    pr = Project("fp8", n, K, 32, T, seed=23)
    x, base, ids = x_of(T, K, 0), x_of(T, n, 1), mixed_ids(T, 4, 23, run=90)
    pd = Pool(4, 32, K, n, 23).device()
    plain = pr(x, None, None, base)
    np.testing.assert_array_equal(pr(x, pd, np.full(T, -1, np.int32), base), plain)
    want = pr(x, pd, ids, base)
    xd, idd = dev_u16(x), dev(ids)
    y = dev_u16(base)
    pr.enqueue(pd, xd, idd, y, base=y)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y), want)
    y = dev_u16(base)
    pr.enqueue(pd, xd, idd, y, base=y, T=T - 3)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y)[:T - 3], want[:T - 3])
    np.testing.assert_array_equal(bits(y)[T - 3:], base[T - 3:])


@pytest.mark.parametrize("n", [4096, 512])
def test_tiles_keep_non_finite_values_apart(n):
    """One adapter's NaN and infinities, and one token's, reach no other row of a tile."""
    K, T = 256, 2100
    pr = Project("bf16", n, K, 32, T, seed=24)
    pool = Pool(3, 32, K, n, 24)
    x, ids = x_of(T, K, 0), mixed_ids(T, 3, 24, run=3)
    clean = pr(x, pool.device(), ids)
    x[7, 3] = 0x7FC0
    pool.a[0, 0, ::2] = 0x7F80
    pool.b[0, :, 0] = 0x7FC0
    got = pr(x, pool.device(), ids)
    hit = ids == 0
    hit[7] = True
    np.testing.assert_array_equal(got[~hit], clean[~hit])
    assert not np.isfinite(OF.bf16_to_f64(got[hit])).any()


def test_expert_tiles_in_a_graph():
    """A captured call over full and half tiles, replayed with new tokens and other adapters."""
    d, f, R, T = 512, 1024, 32, 4100
    a, b = Expert("bf16", d, f, R, T, seed=25), Expert("bf16", d, f, R, T, seed=25)
    pds = [Pool(4, R, d, f, 251).device(), Pool(4, R, d, f, 252).device(), Pool(4, R, f, d, 253).device()]
    xd, idd = dev_u16(x_of(T, d, 0)), dev(mixed_ids(T, 4, 0, run=90))
    y = torch.empty(T, d, dtype=torch.int16, device="cuda")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        a.enqueue(pds, xd, idd, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        a.enqueue(pds, xd, idd, y)
    for i in range(1, 4):
        x, ids = x_of(T, d, i), mixed_ids(T, 4, i, run=[90, 1, 4000][i - 1])
        xd.copy_(dev_u16(x))
        idd.copy_(dev(ids))
        g.replay()
        want = b(x, pds, ids)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(y), want)


@pytest.mark.parametrize("T", [3, 48, 2100])
def test_block_scales_of_any_size(T):
    """FP8 blocks along K whose scales rise and fall by up to 2^130, zeros and subnormals among them."""
    n, K = 512, 1152
    pr = Project("fp8", n, K, 16, T, seed=26)
    blocks = np.array([0.0, 2.0 ** -100, 2.0 ** 30, 2.0 ** -90, 2.0 ** -126, -2.0 ** 40, 2.0 ** -130, 0.0, 2.0 ** 10])
    rows = np.array([1.0, 2.0 ** -60, 2.0 ** 20, -1.0])          # the first two of a pair of row blocks fall, then rise
    scale = np.float32(np.outer(rows, blocks)).astype(np.float32)
    scale[3] = scale[3, ::-1]
    old = pr.scales.cpu().numpy()[:-1].view(np.float32).reshape(n // 128, K // 128)
    # the matrix's own scales are replaced: decoded weights scale with them
    W = pr.W / np.repeat(np.repeat(old.astype(np.float64), 128, 0), 128, 1).T
    W = W * np.repeat(np.repeat(scale.astype(np.float64), 128, 0), 128, 1).T
    pr.scales.copy_(dev(np.append(scale.view(np.uint8).ravel(), np.uint8(0))))
    x = x_of(T, K, T)
    for rows_on in (slice(None), slice(128, 384), slice(0, 128)):        # columns of x that are not zero
        xs = np.zeros_like(x)
        xs[:, rows_on] = x[:, rows_on]
        ref, bound = project_with_bound(xs, W, None, None)
        # numbers below the smallest normal one may be flushed; the tiles take a zero or subnormal scale as 2^-126
        # times one of the row's others (the codes are at most 448 = 1.75 2^8)
        ax = np.abs(OF.bf16_to_f64(xs)).sum(1)[:, None]
        slack = 2.0 ** -110 + 2.0 ** -117 * ax * np.repeat(np.abs(scale.astype(np.float64)).max(1), 128)
        assert_within(OF.bf16_to_f64(pr(xs)), ref, bound + slack, f"T={T} {rows_on}")


@pytest.mark.parametrize("T", [1, 33, 64, 2100])
def test_large_pools(T):
    """More adapters in the pool than one wave looks up, and more in a tile than it has room for pairs of."""
    n, K, count, R = 512, 384, 97, 16
    pr = Project("bf16", n, K, R, T, seed=27)
    pool = Pool(count, R, K, n, 27)
    x, ids = x_of(T, K, T), mixed_ids(T, count, 27)
    ref, bound = project_with_bound(x, pr.W, pool, ids)
    assert_within(OF.bf16_to_f64(pr(x, pool.device(), ids)), ref, bound, f"T={T}")


@pytest.mark.parametrize("T", [2, 40, 1100])
def test_two_wide_pools_of_many_adapters(T):
    """Both matrices' v at the largest rank beside the waves' sums: more than 64 KiB of shared memory."""
    d, f, count, R = 256, 512, 9, 128
    ex = Expert("bf16", d, f, R, T, seed=28)
    pools = [Pool(count, R, d, f, 281), Pool(count, R, d, f, 282), Pool(count, R, f, d, 283)]
    x, ids = x_of(T, d, T), mixed_ids(T, count, 28)
    ref, bound = expert_with_bound(x, ex.mats, pools, ids)
    assert_within(OF.bf16_to_f64(ex(x, [p.device() for p in pools], ids)), ref, bound, f"T={T}")


@pytest.mark.parametrize("T", [5, 2100])
def test_outputs_off_the_16_byte_grid(T):
    """y and base at any multiple of two bytes."""
    n, K, R = 512, 256, 32
    pr = Project("mxfp4", n, K, R, T, seed=29)
    pool = Pool(4, R, K, n, 29)
    x, base, ids = x_of(T, K, 0), x_of(T, n, 1), mixed_ids(T, 4, 29, run=90)
    ref, bound = project_with_bound(x, pr.W, pool, ids, base)
    room = torch.full((T * n + 8,), -7, dtype=torch.int16, device="cuda")
    y = room[1:T * n + 1].view(T, n)
    src = torch.empty(T * n + 8, dtype=torch.int16, device="cuda")[3:T * n + 3].view(T, n)
    src.copy_(dev_u16(base))
    pr.enqueue(pool.device(), dev_u16(x), dev(ids), y, base=src)
    torch.cuda.synchronize()
    assert_within(OF.bf16_to_f64(bits(y)), ref, bound, f"T={T}")
    assert room[0] == -7 and (room[T * n + 1:] == -7).all()


def test_prompts_on_two_streams():
    """Calls on two streams at once, each with a workspace of its own, and the same pools."""
    d, f, R, T = 512, 384, 32, 1500
    exs = [Expert("fp8", d, f, R, T, seed=30) for _ in range(2)]
    pds = [Pool(4, R, d, f, 301).device(), Pool(4, R, d, f, 302).device(), Pool(4, R, f, d, 303).device()]
    ids = mixed_ids(T, 4, 30, run=70)
    xs = [x_of(T, d, i) for i in range(2)]
    want = [e(x, pds, ids) for e, x in zip(exs, xs)]
    xd, idd = [dev_u16(x) for x in xs], dev(ids)
    ys = [torch.empty(T, d, dtype=torch.int16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            exs[i].enqueue(pds, xd[i], idd, ys[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        np.testing.assert_array_equal(bits(ys[i]), want[i])


@pytest.mark.parametrize("off", [0, 1])
def test_most_tokens(off):
    """The largest call, through the tiles and, with y off the 16-byte grid, through the few-token kernel."""
    n, K, R, T = 128, 128, 16, 65535
    pr = Project("bf16", n, K, R, T, seed=32)
    pool = Pool(5, R, K, n, 32)
    x, ids = x_of(T, K, 0), mixed_ids(T, 5, 32, run=3000)
    ref, bound = project_with_bound(x, pr.W, pool, ids)
    y = torch.full((T * n + 8,), -7, dtype=torch.int16, device="cuda")
    pr.enqueue(pool.device(), dev_u16(x), dev(ids), y[off:])
    torch.cuda.synchronize()
    assert_within(OF.bf16_to_f64(bits(y[off:off + T * n].view(T, n))), ref, bound)
    assert (y[:off] == -7).all() and (y[off + T * n:] == -7).all()
    with pytest.raises(M.FtError, match="T must be"):
        pr.enqueue(pool.device(), dev_u16(x), dev(ids), y, T=T + 1)
