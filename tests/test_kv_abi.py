"""The key-value cache's and the block norm's refusals and size queries, before any device work."""
import ctypes
import os
import subprocess

import pytest

import moe_expert_execution_amd as M
from tests.test_abi import HEADER

NAN, INF = float("nan"), float("inf")


def refused(fn, *args):
    with pytest.raises(M.FtError) as e:
        fn(*args)
    return e.value


def check(fn, *args, msg):
    e = refused(fn, *args)
    assert e.status == M.FT_ERR_ARG and msg in str(e), str(e)


def cache(**kw):
    c = dict(pages=4, page_tokens=16, kv_heads=2, head_dim=128, fmt="bf16", k=16, v=16)
    c.update(kw)
    return M.kv_cache(**c)


BAD_CACHES = [(dict(pages=0), "pages"), (dict(pages=2 ** 27), "pages"), (dict(page_tokens=8), "page_tokens"),
              (dict(page_tokens=48), "page_tokens"), (dict(page_tokens=512), "page_tokens"),
              (dict(kv_heads=0), "kv_heads"), (dict(kv_heads=1025), "kv_heads"), (dict(head_dim=96), "head_dim"),
              (dict(head_dim=512), "head_dim"), (dict(fmt=2), "fmt"), (dict(page_stride=8191), "page_stride"),
              (dict(page_stride=8192 - 16), "page_stride"), (dict(page_stride=8200), "page_stride"),
              (dict(page_stride=2 ** 62), "page_stride")]
BAD_POINTERS = [(dict(k=0), "null"), (dict(v=0), "null"), (dict(k=8), "aligned"), (dict(v=24), "aligned"),
                (dict(k_scale=16), "no scales"), (dict(fmt="e4m3"), "needs k_scale"),
                (dict(fmt="e4m3", k_scale=16), "needs k_scale"), (dict(fmt="e4m3", k_scale=16, v_scale=18), "4-byte")]


def append(**kw):
    a = dict(tokens=3, k=16, k_stride=256, v=16, v_stride=256, slot=16, pos=16, rot=64, positions=10, cos_sin=16,
             q_heads=4, q=16, q_stride=512, q_out=16, q_out_stride=512)
    a.update(kw)
    return M.kv_append(**a)


def attend(**kw):
    a = dict(requests=3, q_heads=4, width=5, scale=0.1, q=16, q_stride=512, table=16, kv_len=16, out=32,
             out_stride=512)
    a.update(kw)
    return M.kv_attend(**a)


@pytest.mark.parametrize("kw,msg", BAD_CACHES + BAD_POINTERS)
def test_caches_refused(kw, msg):
    check(M.ft_kv_append, cache(**kw), append(), msg=msg)
    check(M.ft_kv_attend, cache(**kw), attend(), 0, msg=msg)
    if (kw, msg) in BAD_CACHES:
        assert M.ft_kv_attend_workspace(cache(**kw), 4, 3) == 0


@pytest.mark.parametrize("kw,msg", [
    (dict(tokens=-1), "tokens"), (dict(tokens=65536), "tokens"), (dict(q_heads=-1), "q_heads"),
    (dict(q_heads=1025), "q_heads"), (dict(rot=8), "rot"), (dict(rot=-16), "rot"), (dict(rot=144), "rot"),
    (dict(positions=0), "positions"), (dict(k=0), "null pointer: k"), (dict(v=0), "null pointer: v"),
    (dict(q=0), "null pointer: q"), (dict(q_out=0), "null pointer: q_out"), (dict(k=8), "aligned"),
    (dict(q_out=24), "aligned"), (dict(k_stride=248), "stride"), (dict(v_stride=260), "stride"),
    (dict(q_stride=504), "stride"), (dict(q_out_stride=-512), "stride"), (dict(k_stride=2 ** 41), "stride"),
    (dict(q_stride=520), "equal stride"), (dict(q_heads=0), "must be NULL"), (dict(slot=0), "slot"),
    (dict(slot=18), "slot"), (dict(pos=0), "pos"), (dict(cos_sin=0), "cos_sin"), (dict(cos_sin=8), "cos_sin")])
def test_appends_refused(kw, msg):
    check(M.ft_kv_append, cache(), append(**kw), msg=msg)


def test_streams_refused():
    for s in (1, 2):                                 # hipStreamLegacy, hipStreamPerThread
        check(M.ft_kv_append, cache(), append(), s, msg="hipStreamLegacy")
        check(M.ft_block_norm, norm(), s, msg="hipStreamLegacy")


@pytest.mark.parametrize("kw,msg", [
    (dict(requests=-1), "requests"), (dict(requests=4097), "requests"), (dict(q_heads=3), "q_heads"),
    (dict(q_heads=0), "q_heads"), (dict(q_heads=1026), "q_heads"), (dict(width=0), "width"),
    (dict(width=131073), "width"), (dict(window=-1), "window"), (dict(scale=NAN), "scale"), (dict(scale=INF), "scale"),
    (dict(q=0), "null pointer: q"), (dict(out=0), "null pointer: out"), (dict(q=8), "aligned"),
    (dict(out_stride=504), "stride"), (dict(q_stride=516), "stride"), (dict(table=0), "table"),
    (dict(out=16), "out must not be q"), (dict(kv_len=0), "kv_len"), (dict(kv_len=18), "misaligned"), (dict(sinks=17), "misaligned"),
    (dict(), "workspace is null")])
def test_attends_refused(kw, msg):
    check(M.ft_kv_attend, cache(), attend(**kw), 0, msg=msg)


def test_attends_of_too_many_tokens_refused():
    c = cache(page_tokens=256, kv_heads=2, page_stride=2 ** 20)
    for requests, q_heads, width in ((4096, 32, 16385), (2048, 34, 16385), (256, 2, 65537 * 4)):
        a = attend(requests=requests, q_heads=q_heads, width=min(width, 131072), q_stride=8192, out_stride=8192)
        if width <= 131072:
            check(M.ft_kv_attend, c, a, 0, msg="2^35")
    a = attend(requests=4096, q_heads=32, width=16384, q_stride=8192, out_stride=8192)
    check(M.ft_kv_attend, c, a, 0, msg="workspace is null")


def test_reserved_fields_refused():
    c, a = cache(), attend()
    c.reserved = 1
    check(M.ft_kv_attend, c, attend(), 0, msg="reserved")
    a.reserved = 1
    check(M.ft_kv_attend, cache(), a, 0, msg="reserved")


def test_attend_workspace():
    one = M.ft_kv_attend_workspace(cache(), 2, 1)
    assert 0 < one < M.ft_kv_attend_workspace(cache(), 32, 1) <= 64 << 20
    assert M.ft_kv_attend_workspace(cache(), 32, 1) == M.ft_kv_attend_workspace(cache(), 64, 4096)
    for q_heads, requests in ((3, 1), (0, 1), (1026, 1), (2, 0), (2, 4097)):
        assert M.ft_kv_attend_workspace(cache(), q_heads, requests) == 0
    assert M.ft_kv_attend_workspace(cache(k=0, v=0), 2, 1) == one         # sizes alone


def batch(**kw):
    b = dict(requests=2, pages=8, page_tokens=16, width=4, tokens=4, row_tokens=0, **{k: 16 for k in (
        "context", "add", "table", "free_pages", "free_count", "kv_len", "start", "slot", "pos", "counts")})
    b.update(kw)
    return M.kv_batch(**b)


@pytest.mark.parametrize("kw,msg", [
    (dict(requests=-1), "requests"), (dict(requests=4097), "requests"), (dict(pages=0), "pages"),
    (dict(page_tokens=24), "page_tokens"), (dict(width=0), "width"), (dict(width=131073), "width"),
    (dict(tokens=-1), "tokens"), (dict(tokens=65536), "tokens"), (dict(row_tokens=-1), "row_tokens"),
    (dict(row_tokens=3), "row_tokens"), (dict(row_tokens=2 ** 31 - 1), "row_tokens"), (dict(context=18), "misaligned"),
    (dict(counts=17), "misaligned"), (dict(), "workspace is null")] +
    [({k: 0}, "null pointer") for k in ("context", "add", "table", "free_pages", "free_count", "kv_len", "start", "slot",
                                        "pos", "counts")])
def test_plans_refused(kw, msg):
    check(M.ft_kv_plan, batch(**kw), 0, msg=msg)


def norm(**kw):
    a = dict(T=2, d=64, eps=1e-6, block=16, residual=32, pre_w=16, sum=16, normed=48)
    a.update(kw)
    return M.block_norm(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "T must"), (dict(T=2 ** 24 + 1), "T must"), (dict(d=0), "d must"), (dict(d=60), "d must"),
    (dict(d=32776), "d must"), (dict(T=2 ** 19 + 1, d=32768), "T * d must"),
    (dict(T=2 ** 24, d=1032), "T * d must"), (dict(gate_kind=4), "gate_kind"), (dict(gate_kind=0x10), "gate_kind"),
    (dict(gate_kind=-1), "gate_kind"), (dict(gate_kind=0x21), "gate_kind"), (dict(eps=-1.0), "eps"),
    (dict(eps=NAN), "eps"), (dict(eps=INF), "eps"), (dict(residual_scale=NAN), "finite"),
    (dict(weight_offset=INF), "finite"), (dict(block=0, post_w=16), "need block"),
    (dict(block=0, gate=16, gate_kind="full"), "need block"), (dict(normed=0), "belong together"),
    (dict(pre_w=0), "belong together"), (dict(gate=16), "do not agree"), (dict(gate_kind="token"), "do not agree"),
    (dict(block=0, residual=0), "block and residual"), (dict(sum=0, normed=0, pre_w=0), "sum and normed"),
    (dict(post_w=8), "aligned"), (dict(pre_w=24), "aligned"), (dict(gate=17, gate_kind="token"), "misaligned gate"),
    (dict(gate=18, gate_kind="channel"), "misaligned gate"), (dict(block=8), "aligned"),
    (dict(residual_stride=56), "stride"), (dict(sum_stride=68), "stride"), (dict(normed_stride=-64), "stride"),
    (dict(gate=16, gate_kind="full", gate_stride=32), "stride"), (dict(block_stride=72), "needs its stride"),
    (dict(residual=48, residual_stride=128), "needs its stride"), (dict(sum=48, normed=48), "must differ")])
def test_norms_refused(kw, msg):
    check(M.ft_block_norm, norm(**kw), msg=msg)


def test_nothing_to_do():
    """No tokens or requests: accepted without looking at pointers."""
    M.ft_kv_append(cache(), append(tokens=0, k=0, v=0, slot=0))
    M.ft_kv_attend(cache(), attend(requests=0, q=0, table=0), 0)
    M.ft_kv_plan(batch(requests=0, context=0), 0)
    M.ft_block_norm(norm(T=0, block=0, residual=0))


def test_null_descriptors_refused():
    lib = M.lib()
    c = cache()
    assert lib.ft_kv_plan(None, None, None) == M.FT_ERR_ARG
    assert lib.ft_kv_append(None, ctypes.byref(append()), None) == M.FT_ERR_ARG
    assert lib.ft_kv_append(ctypes.byref(c), None, None) == M.FT_ERR_ARG
    assert lib.ft_kv_attend(ctypes.byref(c), None, None, None) == M.FT_ERR_ARG
    assert lib.ft_kv_attend_workspace(None, 1, 1) == 0
    assert lib.ft_block_norm(None, None) == M.FT_ERR_ARG


def test_structs_match_header(tmp_path):
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "ftmoe.h"', 'int main(void) {']
    structs = {"ft_kv_cache": M.FtKvCache, "ft_kv_batch": M.FtKvBatch, "ft_append": M.FtAppend,
               "ft_attend": M.FtAttend, "ft_norm": M.FtNorm}
    want = []
    for cname, py in structs.items():
        src.append(f'printf("%zu\\n", sizeof({cname}));')
        src += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
        want += [ctypes.sizeof(py)] + [getattr(py, f).offset for f, _ in py._fields_]
    c, exe = tmp_path / "l.c", tmp_path / "l"
    c.write_text("\n".join(src + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(c), "-o", str(exe)])
    assert [int(v) for v in subprocess.check_output([str(exe)], text=True).split()] == want
