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


def test_new_structs_match_header(tmp_path):
    import os
    import subprocess
    from tests.test_abi import HEADER
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "ftmoe.h"', 'int main(void) {']
    structs = {"ft_lora": M.FtLora, "ft_matrix": M.FtMatrix}
    for cname, py in structs.items():
        src.append(f'printf("%zu\\n", sizeof({cname}));')
        src += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    c, exe = tmp_path / "l.c", tmp_path / "l"
    c.write_text("\n".join(src + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(c), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for py in structs.values():
        want += [ctypes.sizeof(py)] + [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want


def pool(**kw):
    p = dict(count=2, max_rank=16, rank=16, scale=16, a=16, b=16, **{})
    p.update(kw)
    return M.FtLora(p["count"], p["max_rank"], p["rank"], p["scale"], p["a"], p["b"])


@pytest.mark.parametrize("kw,msg", [(dict(count=-1), "count"), (dict(max_rank=0), "max_rank"), (dict(max_rank=24), "max_rank"),
                                    (dict(max_rank=144), "max_rank"), (dict(rank=0), "null"), (dict(scale=0), "null"),
                                    (dict(a=0), "null"), (dict(b=0), "null"), (dict(a=8), "aligned"), (dict(b=24), "aligned"),
                                    (dict(rank=18), "aligned")])
def test_pools_refused(kw, msg):
    m = M.matrix(256, 256, "bf16", 16)
    e = refused(M.ft_lora_project, m, pool(**kw), 16, 16, 4, 0, 16, 0, 0)
    assert e.status == M.FT_ERR_ARG and msg in str(e)
    s = layer_shape()
    for i, name in enumerate(("gate", "up", "down")):
        pools = [None, None, None]
        pools[i] = pool(**kw)
        e = refused(M.ft_lora_expert, s, 16, *pools, 16, 16, 4, 0, 16, 0, 0)
        assert e.status == M.FT_ERR_ARG and msg in str(e) and name in str(e)


def test_lora_arguments_refused():
    m = M.matrix(256, 256, "fp8", 16, 16)
    good = [m, pool(), 16, 16, 4, 0, 16, 0, 0]
    for i, v, msg in ((0, M.matrix(200, 256, "bf16", 16), "multiples of 128"), (0, M.matrix(256, 0, "bf16", 16), "multiples of 128"),
                      (0, M.matrix(256, 65536, "bf16", 16), "multiples of 128"), (0, M.matrix(256, 256, 5, 16), "fmt"),
                      (0, M.matrix(256, 256, "fp8", 16), "null"), (0, M.matrix(256, 256, "fp8", 16, 18), "aligned"),
                      (0, M.matrix(256, 256, "fp8", 8, 16), "aligned"), (2, 0, "null"), (2, 8, "aligned"), (3, 0, "adapter"),
                      (3, 18, "aligned"), (4, 65536, "T must"), (4, -1, "T must"), (5, 1, "misaligned"), (6, 0, "null"),
                      (6, 17, "misaligned"), (7, 0, "workspace is null")):
        bad = list(good)
        bad[i] = v
        e = refused(M.ft_lora_project, *bad)
        assert e.status == M.FT_ERR_ARG and msg in str(e), (i, v, str(e))
    M.ft_lora_project(m, None, 0, 0, 0, 0, 0, 0, 0)
    s = layer_shape()
    for args, msg in (((s, 0, None, None, None, 16, 0, 4, 0, 16, 0, 0), "null"), ((s, 8, None, None, None, 16, 0, 4, 0, 16, 0, 0), "aligned"),
                      ((layer_shape(d=100), 16, None, None, None, 16, 0, 4, 0, 16, 0, 0), "128"),
                      ((s, 16, None, None, None, 16, 0, 70000, 0, 16, 0, 0), "T must"),
                      ((s, 16, None, None, None, 16, 0, 4, 0, 16, 0, 0), "workspace is null")):
        e = refused(M.ft_lora_expert, *args)
        assert e.status == M.FT_ERR_ARG and msg in str(e), msg


def test_lora_workspace_covers_fewer_tokens():
    """A workspace for max_tokens serves every smaller call: the queries never shrink as tokens grow."""
    for n, K in ((128, 128), (2048, 2048), (7168, 2048)):
        m = M.matrix(n, K, "bf16", 16)
        sizes = [M.ft_lora_project_workspace(m, 64, t) for t in list(range(1, 400)) + [1024, 8192, 65535]]
        assert all(b >= a > 0 for a, b in zip(sizes, sizes[1:]))
    s = M.shape(1, 1, 1, 2048, 768, "bf16")
    sizes = [M.ft_lora_expert_workspace(s, 16, t) for t in list(range(1, 400)) + [1024, 8192, 65535]]
    assert all(b >= a > 0 for a, b in zip(sizes, sizes[1:]))
    assert M.ft_lora_expert_workspace(s, 8, 4) == 0 and M.ft_lora_expert_workspace(s, 16, 0) == 0
    assert M.ft_lora_project_workspace(M.matrix(100, 128, "bf16", 16), 16, 4) == 0


@pytest.mark.parametrize("rank", [0, 16, 128])
def test_lora_workspace_at_every_tile_border(rank):
    """The same where the second tile of tokens takes a call's splits away (more row panels, or long K), and the
    fewest tokens of a tile are queried right after the most of the one before."""
    tokens = [1, 2, 31, 32, 33, 34, 63, 64, 65, 66, 96, 97, 128, 129, 1024, 1025]
    for n in (256, 384, 1024, 2048, 4096, 4224, 8192, 32768):
        for K in (128, 1024, 2048, 4096, 8192, 32768):
            m = M.matrix(n, K, "bf16", 16)
            sizes = [M.ft_lora_project_workspace(m, rank, t) for t in tokens]
            assert sizes == sorted(sizes) and sizes[0] > 0, (n, K, dict(zip(tokens, sizes)))
            if K <= 8192 and n <= 8192:
                s = M.shape(1, 1, 1, n, K, "bf16")
                sizes = [M.ft_lora_expert_workspace(s, rank, t) for t in tokens]
                assert sizes == sorted(sizes) and sizes[0] > 0, (n, K, dict(zip(tokens, sizes)))
