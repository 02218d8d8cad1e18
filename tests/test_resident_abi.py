"""The resident-weight operators' refusals and size queries, before any device work."""
import ctypes

import pytest

import moe_expert_execution_amd as M


def refused(fn, *args):
    with pytest.raises(M.FtError) as e:
        fn(*args)
    return e.value


GOOD = dict(E=8, k=2, d=256, f=128, fmt="bf16")


def layer_shape(**kw):
    s = dict(GOOD, **kw)
    return M.shape(1, s["E"], s["k"], s["d"], s["f"], s["fmt"])


@pytest.mark.parametrize("kw,msg", [(dict(E=257), "256"), (dict(E=0), "256"), (dict(k=0), "top_k"), (dict(k=9), "top_k"),
                                    (dict(E=32, k=17), "top_k"), (dict(d=100), "128"), (dict(f=0), "128"),
                                    (dict(fmt=9), "fmt"), (dict(d=65536), "128")])
def test_layer_shapes_refused(kw, msg):
    e = refused(M.ft_moe_layer, layer_shape(**kw), 16, 16, 16, 1 << 20, 1, 0, 16, 16, 16, 16, 0)
    assert e.status == M.FT_ERR_ARG and msg in str(e)
    assert M.ft_moe_layer_workspace(layer_shape(**kw), 4) == 0


def test_layer_arguments_refused():
    s = layer_shape()
    S = M.ft_record_bytes(s)
    good = [s, 16, 16, 16, S, 4, 0, 16, 16, 16, 0, 0]
    for i, v, msg in ((5, 65, "T must"), (5, -1, "T must"), (1, 0, "null"), (2, 0, "null"), (3, 0, "null"), (7, 0, "null"),
                      (8, 0, "null"), (9, 0, "null"), (4, S - 16, "record_stride"), (4, S + 8, "record_stride"),
                      (1, 24, "aligned"), (3, 8, "aligned"), (6, 17, "misaligned"), (10, 0, "workspace is null")):
        bad = list(good)
        bad[i] = v
        e = refused(M.ft_moe_layer, *bad)
        assert e.status == M.FT_ERR_ARG and msg in str(e), (i, v, str(e))
    M.ft_moe_layer(s, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)          # T = 0: nothing to do


def test_layer_workspace_grows_with_tokens():
    s = M.shape(1, 128, 8, 2048, 768, "bf16")
    sizes = [M.ft_moe_layer_workspace(s, t) for t in range(1, 65)]
    assert all(b >= a > 0 for a, b in zip(sizes, sizes[1:]))
    assert M.ft_moe_layer_workspace(s, 0) == 0 and M.ft_moe_layer_workspace(s, 65) == 0


def test_workspace_refused():
    assert refused(M.ft_workspace_create, 0).status == M.FT_ERR_ARG
    assert M.lib().ft_workspace_create(16, None) == M.FT_ERR_ARG
    M.ft_workspace_destroy(0)
