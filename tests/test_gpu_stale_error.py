"""An error that an earlier HIP call of the program left behind is not the resident operators' own."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from tests.gpu_util import dev, dev_u16
from tests.resident_util import Pool, config, mixed_ids
from tests.test_gpu_lora import Expert, Project, x_of
from tests.test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu


def with_stale_error(call):
    """The call right after a failed one of the HIP runtime that the library uses."""
    hip = M.lib()                            # (its dependencies' symbols are found through it)
    assert hip.hipSetDevice(9999) != 0
    try:
        return call()
    finally:
        hip.hipGetLastError()


@pytest.mark.parametrize("T", [1, 9, 40])
def test_layer(T):
    cfg = config("bf16", 256, 128, 8, 2, seed=61)
    layer = Layer(cfg, T)
    x = synth.tokens(cfg, T, 0)
    want = layer(x)
    xd, out = dev_u16(x), layer.outputs(T)
    torch.cuda.synchronize()
    with_stale_error(lambda: layer.enqueue(xd, out))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out[0].cpu().numpy(), want[0])
    np.testing.assert_array_equal(out[2].cpu().numpy().view(np.uint16), want[2])


@pytest.mark.parametrize("T", [2, 40, 700])
def test_adapters(T):
    """The streaming kernels with the adapters inside, behind a shrink launch, and the GEMM tiles."""
    d, f, R, count = 512, 384, 32, 20
    ex, pr = Expert("bf16", d, f, R, T, seed=62), Project("bf16", d, f, R, T, seed=62)
    pds = [Pool(count, R, d, f, 621).device(), Pool(count, R, d, f, 622).device(), Pool(count, R, f, d, 623).device()]
    ids = mixed_ids(T, count, 62)
    for op, x, pools, n in ((ex, x_of(T, d, 0), pds, d), (pr, x_of(T, f, 0), pds[2], d)):
        want = op(x, pools, ids)
        xd, idd, y = dev_u16(x), dev(ids), torch.full((T, n), -7, dtype=torch.int16, device="cuda")
        torch.cuda.synchronize()
        with_stale_error(lambda: op.enqueue(pools, xd, idd, y))
        torch.cuda.synchronize()
        np.testing.assert_array_equal(y.cpu().numpy().view(np.uint16), want)
