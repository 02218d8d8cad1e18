"""A decoder layer as a program runs it: plan, norm, projection, append, attend, projection, norm and the
mixture-of-experts layer, for prompts once and then for decoding steps, eager and as one captured graph.  Each stage is
compared with its definition in 64 bits on the stage's own inputs; the captured steps with the eager ones bit for bit."""
import numpy as np
import pytest
import torch

import moe_expert_execution_amd as M
import synth
from moe_expert_execution_amd.tensors import Workspace
from oracle import formats as OF
from tests.gpu_util import cuda, dev
from tests.kv_util import Cache, attend_reference, bf16_bound, e4m3_bound, norm_reference, plan_reference, rope, stream
from tests.resident_util import assert_within, bits, config, layer_with_bound, padded, project_with_bound

pytestmark = pytest.mark.gpu

HQ, HKV, D, P, ROT, d = 8, 2, 64, 16, 32, 512
ROW = (HQ + 2 * HKV) * D
EPS, GROWTH = 1e-5, 0.5


def panels(w):
    """bf16 [n, K] row-major -> the record's panel order."""
    n, K = w.shape
    return np.ascontiguousarray(w.view(np.uint16).reshape(n // 32, 32, K // 16, 2, 8).transpose(0, 2, 3, 1, 4))


class Layer:
    """The weights of one decoder layer, its cache and its page bookkeeping for B requests."""

    def __init__(self, B, fmt, width=6, seed=1):
        rng = np.random.default_rng(seed)
        bf = lambda *s, mul=1.0, add=0.0: synth.f32_to_bf16(  # noqa: E731
            (mul * rng.standard_normal(s) + add).astype(np.float32))
        self.B, self.fmt, self.width, self.pages = B, fmt, width, B * width - 3
        self.cfg = config("bf16", d, 128, 8, 2, seed=seed)
        self.records = synth.bank(self.cfg)
        self.router = synth.router(self.cfg, 0)
        self.w = {"qkv": bf(ROW, d, mul=0.06), "out": bf(d, HQ * D, mul=0.06), "in_norm": bf(d, mul=0.1, add=1.0),
                  "post": bf(d, mul=0.1, add=1.0), "pre": bf(d, mul=0.1, add=1.0)}
        ang = rng.uniform(-3, 3, (width * P, ROT // 2))
        self.cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.cache = Cache(fmt, self.pages, P, HKV, D, seed)
        i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
        self.free, self.table = i32(rng.permutation(self.pages)), i32(np.full((B, width), -1))
        self.len, self.counts = i32(np.zeros(B)), i32([0, 0, self.pages, 0])
        self.dev = {k: dev(panels(v).view(np.int16)) if k in ("qkv", "out") else dev(v.view(np.int16))
                    for k, v in self.w.items()}
        self.dev.update(records=dev(padded(self.records)), router=dev(self.router.view(np.int16)), cos_sin=dev(self.cos_sin))
        self.m = {"qkv": M.matrix(ROW, d, "bf16", self.dev["qkv"].data_ptr()),
                  "out": M.matrix(d, HQ * D, "bf16", self.dev["out"].data_ptr())}
        self.shape = M.shape(1, 8, 2, d, 128, "bf16")

    def buffers(self, T, row_tokens):
        """One step's arrays and descriptors: T token rows."""
        z = lambda *s, t=torch.int16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        b = {"x": z(T, d), "add": z(self.B, t=torch.int32), "start": z(self.B + 1, t=torch.int32),
             "slot": z(T, t=torch.int32), "pos": z(T, t=torch.int32), "h": z(T, d), "qkv": z(T, ROW), "q": z(T, HQ * D),
             "att": z(T, HQ * D), "o": z(T, d), "sum": z(T, d), "normed": z(T, d), "y": z(T, d),
             "ids": z(T, 2, t=torch.int32), "wt": z(T, 2, t=torch.float32)}
        p = {k: v.data_ptr() for k, v in b.items()}
        c = self.cache.struct()
        s = {"plan": M.kv_batch(self.B, self.pages, P, self.width, T, row_tokens, self.len.data_ptr(), p["add"],
                                self.table.data_ptr(), self.free.data_ptr(), self.counts.data_ptr() + 8,
                                self.len.data_ptr(), p["start"], p["slot"], p["pos"], self.counts.data_ptr()),
             "in": M.block_norm(T, d, EPS, residual=p["x"], pre_w=self.dev["in_norm"].data_ptr(), normed=p["h"]),
             "append": M.kv_append(T, p["qkv"] + 2 * HQ * D, ROW, p["qkv"] + 2 * (HQ + HKV) * D, ROW, p["slot"],
                                   p["pos"], ROT, len(self.cos_sin), self.dev["cos_sin"].data_ptr(), HQ, p["qkv"], ROW,
                                   p["q"], HQ * D),
             "attend": M.kv_attend(self.B, HQ, self.width, D ** -0.5, p["q"], HQ * D, self.table.data_ptr(),
                                   self.len.data_ptr(), p["att"], HQ * D),
             "mid": M.block_norm(T, d, EPS, block=p["o"], residual=p["x"], post_w=self.dev["post"].data_ptr(),
                                 pre_w=self.dev["pre"].data_ptr(), sum=p["sum"], normed=p["normed"],
                                 residual_scale=GROWTH)}
        need = max(M.ft_kv_attend_workspace(c, HQ, self.B), M.ft_moe_layer_workspace(self.shape, min(T, 64)),
                   M.ft_lora_project_workspace(self.m["qkv"], 0, T), M.ft_lora_project_workspace(self.m["out"], 0, T))
        return b, p, c, s, Workspace(need)

    def enqueue(self, step, decode=True):
        b, p, c, s, ws = step
        st, T = stream(), b["x"].shape[0]
        M.ft_kv_plan(s["plan"], ws.handle, st)
        M.ft_block_norm(s["in"], st)
        M.ft_lora_project(self.m["qkv"], None, p["h"], 0, T, 0, p["qkv"], ws.handle, st)
        M.ft_kv_append(c, s["append"], st)
        if decode:
            M.ft_kv_attend(c, s["attend"], ws.handle, st)
            M.ft_lora_project(self.m["out"], None, p["att"], 0, T, 0, p["o"], ws.handle, st)
            M.ft_block_norm(s["mid"], st)
            M.ft_moe_layer(self.shape, p["normed"], self.dev["router"].data_ptr(), self.dev["records"].data_ptr(),
                           self.dev["records"].shape[1], T, p["sum"], p["ids"], p["wt"], p["y"], ws.handle, st)

    def state(self):
        torch.cuda.synchronize()
        n = int(self.counts[2])
        return {"ctx": self.len.cpu().numpy().copy(), "table": self.table.cpu().numpy().copy(),
                "free": self.free.cpu().numpy().copy(), "count": n,
                "raw": {w: self.cache.dev[w].cpu().numpy().copy() for w in "kv"}}


def check_step(L, before, add, step, row_tokens, decode=True):
    """Every stage of a step that has run, from its own inputs."""
    b = step[0]
    after = L.state()
    h = {k: v.cpu().numpy() for k, v in b.items()}
    f = {k: OF.bf16_to_f64(bits(b[k])) for k in ("x", "h", "qkv", "q", "att", "o", "sum", "normed", "y")}
    T = len(h["x"])
    want = plan_reference(before["ctx"], add, before["table"], before["free"], before["count"], L.pages, P, T, row_tokens)
    for k, got in (("slot", h["slot"]), ("pos", h["pos"]), ("start", h["start"]), ("kv_len", after["ctx"]),
                   ("table", after["table"]), ("counts", L.counts.cpu().numpy())):
        np.testing.assert_array_equal(got, want[k], err_msg=k)
    w = {k: OF.bf16_to_f64(v) for k, v in L.w.items()}
    eps = float(np.float32(EPS))
    _, (n, nb) = norm_reference(None, f["x"], None, w["in_norm"], None, "none", False, 1.0, 0.0, eps)
    assert_within(f["h"], n, nb, "norm before the block")
    assert_within(f["qkv"], *project_with_bound(bits(b["h"]), w["qkv"].T, None, None), "projection")
    on = np.nonzero(h["slot"] >= 0)[0]
    x = f["qkv"].reshape(T, HQ + 2 * HKV, D)[on]
    turned, err = rope(x[:, :HQ + HKV], h["pos"][on], L.cos_sin, ROT)
    assert_within(f["q"].reshape(T, HQ, D)[on], turned[:, :HQ], bf16_bound(turned[:, :HQ], err[:, :HQ]), "queries")
    for which, val, e in (("k", turned[:, HQ:], err[:, HQ:]), ("v", x[:, HQ + HKV:], np.zeros((len(on), HKV, D)))):
        for g in range(HKV):
            got = L.cache.read(which, h["slot"][on], g, after["raw"][which])
            if L.fmt == "bf16":
                assert_within(got, val[:, g], bf16_bound(val[:, g], e[:, g]), which)
            else:
                s = float(L.cache.scales[which][g])
                v, bound = e4m3_bound(val[:, g], e[:, g], s)
                assert_within(got / s, v, bound * (1 + 1e-12), which)
    if not decode:
        return after
    out, bound = attend_reference(L.cache, bits(b["q"]).reshape(T, HQ, D)[:L.B], after["table"], after["ctx"], D ** -0.5,
                                  raw=after["raw"])
    assert_within(f["att"].reshape(T, HQ, D)[:L.B], out, bound, "attention")
    assert_within(f["o"], *project_with_bound(bits(b["att"]), w["out"].T, None, None), "output projection")
    (s, sb), (n, nb) = norm_reference(f["o"], f["x"], w["post"], w["pre"], None, "none", False, GROWTH, 0.0, eps)
    assert_within(f["sum"], s, sb, "residual")
    assert_within(f["normed"], n, nb, "norm after the block")
    ids, wt, y, yb, gap = layer_with_bound(bits(b["normed"]), L.router, L.records, L.cfg, bits(b["sum"]))
    np.testing.assert_array_equal(h["ids"], ids)
    assert_within(f["y"], y, yb, "experts")
    return after


def rows(rng, T):
    return dev(synth.f32_to_bf16(rng.standard_normal((T, d)).astype(np.float32)).view(np.int16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_prompts_then_decoding(fmt):
    cuda()
    B, steps = 5, 12
    eager, graphed = Layer(B, fmt), Layer(B, fmt)
    rng = np.random.default_rng(9)
    # prompts of ragged lengths into the empty cache, one of them empty, with padding rows behind
    lengths = np.array([17, 1, 0, 40, 16], np.int32)
    x = rows(rng, 80)
    before = eager.state()
    for L in (eager, graphed):
        step = L.buffers(80, 0)
        step[0]["x"].copy_(x)
        step[0]["add"].copy_(torch.from_numpy(lengths))
        L.enqueue(step, decode=False)
        after = L.state()
        if L is eager:
            check_step(L, before, lengths, step, 0, decode=False)
            before = after
    # decoding: one row a request; requests pause, end and start over
    se, sg = eager.buffers(B, 1), graphed.buffers(B, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.enqueue(sg)
    for i in range(steps):
        add = rng.choice([1, 1, 1, 1, 1, 0, -1], B).astype(np.int32)
        x = rows(rng, B)
        for step in (se, sg):
            step[0]["x"].copy_(x)
            step[0]["add"].copy_(torch.from_numpy(add))
        eager.enqueue(se)
        torch.cuda.synchronize()
        g.replay()
        before = check_step(eager, before, add, se, 1)
        for k in se[0]:
            assert torch.equal(se[0][k], sg[0][k]), (i, k)
        for u, v in ((eager.table, graphed.table), (eager.len, graphed.len), (eager.counts, graphed.counts),
                     (eager.cache.dev["k"], graphed.cache.dev["k"]), (eager.cache.dev["v"], graphed.cache.dev["v"])):
            assert torch.equal(u, v), i
