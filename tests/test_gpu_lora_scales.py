"""Block-FP8 matrices whose scales are zero, tiny, or fall steeply along K, on the few-token kernels and both sizes of
GEMM tiles."""
import numpy as np
import pytest

from oracle import formats as OF
from tests.gpu_util import dev
from tests.resident_util import assert_within, project_with_bound
from tests.test_gpu_lora import Project, x_of

pytestmark = pytest.mark.gpu


def project_with_scales(n, scales, T, seed):
    """A matrix [n x 128 len(scales)] whose block (i, j) has the scale scales[j], and its fp64 values."""
    K = 128 * len(scales)
    pr = Project("fp8", n, K, 16, T, seed=seed)
    new = np.tile(np.float32(scales), (n // 128, 1))
    old = pr.scales.cpu().numpy()[:-1].view(np.float32).reshape(n // 128, K // 128)
    wide = lambda s: np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1).T
    pr.scales.copy_(dev(np.append(new.view(np.uint8).ravel(), np.uint8(0))))
    return pr, pr.W / wide(old) * wide(new)


def scaled(x, e):
    """bf16 x times 2^e."""
    return (np.ldexp(OF.bf16_to_f64(x), e).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


# 3 and 48 tokens stream, 2,100 go through half tiles at n = 512 and full ones at 4,096
CASES = [(512, 3), (512, 48), (512, 2100), (4096, 2100)]


@pytest.mark.parametrize("n,T", CASES)
@pytest.mark.parametrize("scales", [[0.0, 0.5, 0.25], [0.5, 0.0, 0.25], [0.5, 0.25, -0.0], [0.0, 0.0, 0.0]])
def test_a_zero_scale_adds_nothing(n, T, scales):
    """Tokens that meet only blocks of zero scale: exactly zero, however large they are.  With the others: their sum
    alone."""
    pr, W = project_with_scales(n, scales, T, 51)
    x = x_of(T, 384, T)
    zero = np.repeat(np.array(scales) == 0, 128)
    xs = np.where(zero, scaled(x, 40), 0).astype(np.uint16)
    np.testing.assert_array_equal(OF.bf16_to_f64(pr(xs)), 0.0)
    xs = np.where(zero, scaled(x, 40), x).astype(np.uint16)
    ref, bound = project_with_bound(xs, W, None, None)
    assert_within(OF.bf16_to_f64(pr(xs)), ref, bound, f"n={n} T={T}")


@pytest.mark.parametrize("n,T", CASES)
@pytest.mark.parametrize("tiny", [2.0 ** -126, 2.0 ** -128, 2.0 ** -140, 2.0 ** -149])
def test_tiny_scales_beside_ordinary_ones(n, T, tiny):
    """A block 2^125 and more below another: its products, or nothing in their place, never more."""
    pr, W = project_with_scales(n, [0.5, tiny, 0.5], T, 52)
    xs = x_of(T, 384, T).copy()
    xs[:, :128] = xs[:, 256:] = 0
    ref, bound = project_with_bound(xs, W, None, None)
    # dropped products are off by themselves; numbers below the smallest normal one may be flushed
    most = np.abs(OF.bf16_to_f64(xs)) @ np.abs(W)
    assert_within(OF.bf16_to_f64(pr(xs)), ref, bound + most + 2.0 ** -126, f"n={n} T={T}")


@pytest.mark.parametrize("n,T", CASES)
@pytest.mark.parametrize("fall", [20, 50, 59, 100])
def test_large_tokens_where_scales_fall(n, T, fall):
    """Tokens of 2^70 on block scales that fall, and rise again, along K: sums that fit fp32 are finite and right."""
    pr, W = project_with_scales(n, [1.0, 2.0 ** -fall, 2.0 ** -fall, 0.5, 2.0 ** -fall], T, 53)
    x = scaled(x_of(T, 640, T), 70)
    ref, bound = project_with_bound(x, W, None, None)
    assert_within(OF.bf16_to_f64(pr(x)), ref, bound, f"n={n} T={T}")
