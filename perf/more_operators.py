"""Cases of the operators around a resident layer: what is timed, on which inputs, and what the outputs are.

Four operators of a decoder layer, beside the resident weights' (see include/ftmoe.h):

  plan     block tables and slot maps of a paged key-value cache from the requests' lengths (ft_kv_plan):
           pages are taken from a free list, pages of ended requests return to it, and every new token gets
           its cache slot and position.
  append   the new tokens' keys and values into their slots, rotated by their positions, and the rotated
           queries (ft_kv_append).
  attend   attention of one new token per request over its pages (ft_kv_attend).
  norm     the norms after one block and before the next, with the block's gate and the residual scale
           (ft_block_norm).

`listed()` gives the timed cases, `draw(rng)` others of the same ranges, `prepare(case, seed)` the inputs,
`run(state)` one call, `work(case)` the bytes and operations it cannot do without and `exact(case, seed)`
its outputs in 64 bits.  With `own` false `run` is the plain form in elementary torch operations in 32
bits; with `own` true it calls the library.

Layout of a cache page, per KV head and block of 16 tokens (see ft_kv_cache): 16-byte units; a unit of keys
is ck = 16 / size consecutive dimensions of one token, unit (dim / ck) * 16 + token % 16; a unit of values is
tu tokens of cv dimensions each (cv = 8, or 4 where the head has 64), unit (token % 16 / tu) * (D / cv) + dim / cv.
"""
import math
import zlib

import numpy as np
import torch

own = False


# ---- cases ----------------------------------------------------------------------------------------

def _plan(name, B, P, width, tokens, rows, release, short):
    """rows: tokens per request of a padded call (0: packed, ragged); release: share of requests that end;
    short: the free list runs out before the last request."""
    return {"name": name, "op": "plan", "B": B, "P": P, "width": width, "tokens": tokens, "rows": rows,
            "release": release, "short": short}


def _append(name, fmt, D, hq, hkv, T, requests, P, rot):
    return {"name": name, "op": "append", "fmt": fmt, "D": D, "hq": hq, "hkv": hkv, "T": T, "requests": requests,
            "P": P, "rot": rot}


def _attend(name, fmt, D, hq, hkv, B, L, ragged, P, window, sinks):
    return {"name": name, "op": "attend", "fmt": fmt, "D": D, "hq": hq, "hkv": hkv, "B": B, "L": L,
            "ragged": ragged, "P": P, "window": window, "sinks": sinks}


def _norm(name, T, d, post, gate, sigmoid, scale):
    return {"name": name, "op": "norm", "T": T, "d": d, "post": post, "gate": gate, "sigmoid": sigmoid,
            "scale": scale}


def listed():
    return [
        # a decode step of 64 requests: one token each, now and then a new page, a few requests end
        _plan("plan_decode_b64", 64, 16, 512, 64, 1, 0.06, False),
        # a packed step of prompts and decoding requests; the free list does not hold them all
        _plan("plan_mixed_b1000", 1000, 64, 256, 16384, 0, 0.1, True),
        # the new tokens of a small decode batch
        _append("append_bf16_t16", "bf16", 128, 32, 4, 16, 16, 16, 128),
        # a prefill chunk of a few ragged prompts
        _append("append_bf16_t8192", "bf16", 128, 32, 8, 8192, 5, 64, 128),
        # an odd chunk into an 8-bit cache of wide heads, a quarter of each rotated
        _append("append_e4m3_t777", "e4m3", 256, 16, 2, 777, 9, 32, 64),
        # one request a few words in: nothing but latency
        _attend("attend_bf16_l37", "bf16", 128, 32, 4, 1, 37, False, 16, 0, False),
        # one request with a long context: split over its length
        _attend("attend_bf16_l131072", "bf16", 128, 32, 4, 1, 131072, False, 64, 0, False),
        # a decode batch of ragged contexts, padded with an empty row
        _attend("attend_bf16_b64", "bf16", 128, 64, 8, 64, 8192, True, 16, 0, False),
        # a smaller batch of long ragged contexts in an 8-bit cache of wide heads
        _attend("attend_e4m3_b13", "e4m3", 256, 16, 2, 13, 65536, True, 128, 0, False),
        # a sliding window with sinks over narrow heads
        _attend("attend_window_b100", "bf16", 64, 64, 8, 100, 5000, True, 32, 128, True),
        # one token between two blocks of the decode configuration's width
        _norm("norm_t1", 1, 2048, False, "none", False, 1.0),
        # a prefill chunk at the widest configuration: both norms, a gate of every element, a scaled residual
        _norm("norm_t4096", 4096, 7168, True, "full", True, 0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "attend", "attend", "attend", "norm"))
    P = rng.choice((16, 32, 64, 128, 256))
    if op == "plan":
        B = _log_int(rng, 1, 4096)
        rows = rng.choice((0, 0, 1, rng.randint(2, 8)))
        tokens = B * rows if rows else _log_int(rng, B, 16384)
        width = _log_int(rng, max(4, 2048 // P), 65536 // P)
        while B * width > 1024 * 1024:
            width = width * 2 // 3
        return {"op": op, "B": B, "P": P, "width": width, "tokens": tokens, "rows": rows,
                "release": rng.choice((0.0, 0.05, 0.5)), "short": rng.random() < 0.4}
    if op == "norm":
        d = 8 * _log_int(rng, 8, 896)
        T = _log_int(rng, 1, min(262144, 4096 * 7168 // d))
        return {"op": op, "T": T, "d": d, "post": rng.random() < 0.5,
                "gate": rng.choice(("none", "channel", "token", "full")), "sigmoid": rng.random() < 0.3,
                "scale": rng.choice((1.0, 0.5, 1.25))}
    fmt = rng.choice(("bf16", "bf16", "e4m3"))
    D = rng.choice((64, 128, 128, 256))
    hkv = rng.choice((1, 2, 3, 4, 8, 16))
    hq = hkv * rng.choice((1, 2, 3, 4, 5, 6, 8, 12, 16))
    if op == "append":
        T = _log_int(rng, 1, 8192)
        while T * (2 * hq + 3 * hkv) * D > 8192 * 88 * 128:
            T = T * 2 // 3
        T = max(1, T)
        return {"op": op, "fmt": fmt, "D": D, "hq": hq, "hkv": hkv, "T": T, "requests": _log_int(rng, 1, T), "P": P,
                "rot": rng.choice([r for r in (0, 32, 64, 128, 256) if r <= D])}
    B = _log_int(rng, 1, 256)
    L = _log_int(rng, 1, 131072)
    ragged = rng.random() < 0.7
    while B * L * hq * D > (64 if ragged else 16) * 8192 * 64 * 128:
        L = L * 2 // 3
    while B * L * hkv * D > (64 if ragged else 16) * 8192 * 8 * 128:
        L = L * 2 // 3
    return {"op": op, "fmt": fmt, "D": D, "hq": hq, "hkv": hkv, "B": B, "L": max(1, L), "ragged": ragged, "P": P,
            "window": rng.choice((0, 0, 0, _log_int(rng, 1, 8192))), "sinks": rng.random() < 0.3}


# ---- inputs ---------------------------------------------------------------------------------------

def _shape_rng(case):
    """Lengths belong to the case, not to the seed."""
    return np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))


def _lengths(case):
    """Context lengths of an attend case: all L, or ragged (spread over their logarithm, one of L, and from
    eight requests on an empty row at the end, the padding of a batch)."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return np.full(B, L, np.int64)
    r = _shape_rng(case)
    n = np.exp(r.uniform(math.log(max(1.0, L / 64)), math.log(L + 1.0), B)).astype(np.int64).clip(1, L)
    n[r.integers(0, B)] = L
    if B >= 8:
        n[B - 1] = 0
    return n


def _visible(case):
    n = _lengths(case)
    return np.minimum(n, case["window"]) if case["window"] else n


def _parts(total, n, rng):
    """total as n parts of at least one each."""
    cuts = np.sort(rng.choice(np.arange(1, total), size=n - 1, replace=False)) if n > 1 else np.zeros(0, np.int64)
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int64)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _esize(fmt):
    return 2 if fmt == "bf16" else 1


def _pool(fmt, pages, page_elems, heads, gen):
    """Cache pages of normal values; 8-bit ones as codes with a scale per head."""
    x = torch.randn(pages, heads, page_elems // heads, device="cuda", generator=gen, dtype=torch.float32)
    if fmt == "bf16":
        return x.to(torch.bfloat16).view(pages, page_elems), None
    scale = (0.5 + torch.rand(heads, device="cuda", generator=gen)) * (4.5 / 448)
    x = (x / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.view(pages, page_elems), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 23)
    rng = np.random.default_rng([seed, 31])
    return {"plan": _prepare_plan, "append": _prepare_append, "attend": _prepare_attend,
            "norm": _prepare_norm}[case["op"]](case, rng, gen)


def _prepare_plan(c, rng, gen):
    B, P, width, rows, tokens = c["B"], c["P"], c["width"], c["rows"], c["tokens"]
    r = _shape_rng(c)
    room = width * P
    # contexts of any length; packed calls hold some prompts (no context yet, many new tokens) among
    # requests that decode; a few rows are idle
    ctx = np.exp(r.uniform(0, math.log(room - room // 4), B)).astype(np.int64)
    if rows:
        add = r.integers(1, rows + 1, B)
    else:
        add = np.ones(B, np.int64)
        left = int(tokens * 0.95) - B
        prompts = r.permutation(B)[:max(1, B // 20)]
        if left > len(prompts):
            add[prompts] += _parts(left, len(prompts), r)
            ctx[prompts] = np.where(r.random(len(prompts)) < 0.7, 0, ctx[prompts])
    add[r.random(B) < 0.03] = 0
    add[r.random(B) < c["release"]] = -1
    have = (ctx + P - 1) // P
    need = np.where(add > 0, np.where(ctx + add <= room, (ctx + add + P - 1) // P - have, 0), 0)
    released = int(have[add < 0].sum())
    free = int(need.sum()) + 64
    if c["short"]:
        free = max(1, int(need.sum() * 0.9) - released)
    pages = int(have.sum()) + free
    ids = rng.permutation(pages).astype(np.int64)
    table = np.full((B, width), -1, np.int64)
    first = np.concatenate([[0], np.cumsum(have)])
    j = np.arange(width)[None, :]
    src = first[:-1, None] + j
    table = np.where(j < have[:, None], ids[np.minimum(src, pages - 1)], -1)
    listed_free = np.full(pages, -1, np.int64)
    listed_free[:free] = ids[first[-1]:]
    new = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": c, "pages": pages, "ctx": _int(ctx), "add": _int(add), "table": _int(table),
            "free": _int(listed_free), "free_count": _int(np.array([free])), "len": new(B), "start": new(B + 1),
            "slot": new(tokens), "pos": new(tokens), "counts": new(4)}


def _prepare_append(c, rng, gen):
    T, P, D, hq, hkv, fmt = c["T"], c["P"], c["D"], c["hq"], c["hkv"], c["fmt"]
    r = _shape_rng(c)
    n = _parts(T, c["requests"], r)
    ctx = np.where(r.random(len(n)) < 0.3, 0, np.exp(r.uniform(0, math.log(32768), len(n))).astype(np.int64))
    pos = np.concatenate([a + np.arange(b) for a, b in zip(ctx, n)])
    which = np.repeat(np.arange(len(n)), n)
    block = pos // P
    # every (request, page) pair gets a page of its own
    key = which * (1 << 20) + block
    u, inv = np.unique(key, return_inverse=True)
    pages = len(u) + 3
    ids = rng.permutation(pages)[:len(u)]
    slot = ids[inv] * P + pos % P
    pad = max(1, T // 50) if T >= 8 else 0
    if pad:                                           # the call's last tokens are padding
        slot[T - pad:] = -1
        pos[T - pad:] = -1
    k, ks = _pool(fmt, pages, hkv * P * D, hkv, gen)
    v, vs = _pool(fmt, pages, hkv * P * D, hkv, gen)
    rows = (hq + 2 * hkv) * D
    rot = c["rot"]
    table = None
    if rot:
        far = 65536 // 4 if T < 64 else 65536
        far = max(far, int(pos.max()) + 1)
        inv_freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        ang = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * inv_freq[None, :]
        table = torch.cat([torch.cos(ang), torch.sin(ang)], dim=1).float()
    return {"case": c, "pages": pages, "qkv": torch.randn(T, rows, device="cuda", generator=gen).to(torch.bfloat16),
            "slot": _int(slot), "pos": _int(pos), "k": k, "v": v, "k_scale": ks, "v_scale": vs, "cos_sin": table,
            "q_out": torch.zeros(T, hq * D, device="cuda", dtype=torch.bfloat16)}


def _prepare_attend(c, rng, gen):
    B, P, D, hq, hkv, fmt = c["B"], c["P"], c["D"], c["hq"], c["hkv"], c["fmt"]
    n = _lengths(c)
    have = (n + P - 1) // P
    width = int(have.max()) + 1
    pages = int(have.sum()) + 2
    ids = rng.permutation(pages)
    first = np.concatenate([[0], np.cumsum(have)])
    j = np.arange(width)[None, :]
    table = np.where(j < have[:, None], ids[np.minimum(first[:-1, None] + j, pages - 1)], -1)
    k, ks = _pool(fmt, pages, hkv * P * D, hkv, gen)
    v, vs = _pool(fmt, pages, hkv * P * D, hkv, gen)
    rows = (hq + 2 * hkv) * D
    # queries as a projection leaves them: the first heads of a wider row
    qkv = (torch.randn(B, rows, device="cuda", generator=gen) * 1.5).to(torch.bfloat16)
    sinks = torch.randn(hq, device="cuda", generator=gen) if c["sinks"] else None
    return {"case": c, "pages": pages, "qkv": qkv, "k": k, "v": v, "k_scale": ks, "v_scale": vs,
            "table": _int(table), "len": _int(n), "sinks": sinks,
            "out": torch.empty(B, hq * D, device="cuda", dtype=torch.bfloat16)}


def _prepare_norm(c, rng, gen):
    T, d = c["T"], c["d"]

    def bf(*s, mul=1.0, add=0.0):
        return (torch.randn(*s, device="cuda", generator=gen) * mul + add).to(torch.bfloat16)

    gate = {"none": None, "channel": (d,), "token": (T,), "full": (T, d)}[c["gate"]]
    return {"case": c, "block": bf(T, d, mul=0.7), "residual": bf(T, d, mul=3.0),
            "post": bf(d, mul=0.1, add=1.0) if c["post"] else None, "pre": bf(d, mul=0.1, add=1.0),
            "gate": bf(*gate) if gate else None, "sum": torch.empty(T, d, device="cuda", dtype=torch.bfloat16),
            "normed": torch.empty(T, d, device="cuda", dtype=torch.bfloat16)}


# ---- one pass -------------------------------------------------------------------------------------

EPS = 1e-6


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attend": _own_attend, "norm": _own_norm}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend, "norm": _plain_norm}[op](state)


_spaces = []


def _workspace(nbytes):
    """The program's one workspace: every call runs on one stream."""
    from moe_expert_execution_amd.tensors import Workspace
    if not _spaces or _spaces[-1].nbytes < nbytes:
        _spaces.append(Workspace(max(nbytes, 1 << 20)))
    return _spaces[-1].handle


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_plan(st):
    import moe_expert_execution_amd as M
    c = st["case"]
    if "batch" not in st:
        st["batch"] = M.kv_batch(
            requests=c["B"], pages=st["pages"], page_tokens=c["P"], width=c["width"], tokens=c["tokens"],
            row_tokens=c["rows"], context=st["ctx"].data_ptr(), add=st["add"].data_ptr(),
            table=st["table"].data_ptr(), free_pages=st["free"].data_ptr(), free_count=st["free_count"].data_ptr(),
            kv_len=st["len"].data_ptr(), start=st["start"].data_ptr(), slot=st["slot"].data_ptr(),
            pos=st["pos"].data_ptr(), counts=st["counts"].data_ptr())
    M.ft_kv_plan(st["batch"], _workspace(1), _stream())
    return {k: st[k] for k in ("table", "free", "len", "start", "slot", "pos", "counts")}


def _cache(st):
    import moe_expert_execution_amd as M
    c = st["case"]
    return M.kv_cache(pages=st["pages"], page_tokens=c["P"], kv_heads=c["hkv"], head_dim=c["D"], fmt=c["fmt"],
                      k=st["k"].data_ptr(), v=st["v"].data_ptr(), k_scale=_ptr(st["k_scale"]),
                      v_scale=_ptr(st["v_scale"]))


def _own_append(st):
    import moe_expert_execution_amd as M
    c = st["case"]
    if "cache" not in st:
        st["cache"] = _cache(st)
        q = st["qkv"].data_ptr()
        rows = st["qkv"].shape[1]
        rot = c["rot"]
        st["args"] = M.kv_append(
            tokens=c["T"], q_heads=c["hq"] if rot else 0, rot=rot, positions=st["cos_sin"].shape[0] if rot else 0,
            q=q if rot else 0, q_stride=rows, k=q + 2 * c["hq"] * c["D"], k_stride=rows,
            v=q + 2 * (c["hq"] + c["hkv"]) * c["D"], v_stride=rows, slot=st["slot"].data_ptr(),
            pos=st["pos"].data_ptr(), cos_sin=_ptr(st["cos_sin"]), q_out=st["q_out"].data_ptr() if rot else 0,
            q_out_stride=c["hq"] * c["D"])
    M.ft_kv_append(st["cache"], st["args"], _stream())
    return {"k": st["k"], "v": st["v"], "q": st["q_out"]}


def _own_attend(st):
    import moe_expert_execution_amd as M
    c = st["case"]
    if "cache" not in st:
        st["cache"] = _cache(st)
        st["args"] = M.kv_attend(
            requests=c["B"], q_heads=c["hq"], width=st["table"].shape[1], window=c["window"],
            scale=c["D"] ** -0.5, q=st["qkv"].data_ptr(), q_stride=st["qkv"].shape[1], table=st["table"].data_ptr(),
            kv_len=st["len"].data_ptr(), sinks=_ptr(st["sinks"]), out=st["out"].data_ptr(),
            out_stride=c["hq"] * c["D"])
        st["need"] = M.ft_kv_attend_workspace(st["cache"], c["hq"], c["B"])
    M.ft_kv_attend(st["cache"], st["args"], _workspace(st["need"]), _stream())
    return {"out": st["out"]}


def _own_norm(st):
    import moe_expert_execution_amd as M
    c = st["case"]
    if "args" not in st:
        d = c["d"]
        st["args"] = M.block_norm(
            T=c["T"], d=d, gate_kind=c["gate"], sigmoid=c["sigmoid"], eps=EPS, residual_scale=c["scale"],
            block=st["block"].data_ptr(), residual=st["residual"].data_ptr(), post_w=_ptr(st["post"]),
            pre_w=st["pre"].data_ptr(), gate=_ptr(st["gate"]), sum=st["sum"].data_ptr(),
            normed=st["normed"].data_ptr())
    M.ft_block_norm(st["args"], _stream())
    return {"sum": st["sum"], "normed": st["normed"]}


def _plain_plan(st):
    c = st["case"]
    B, P, width, tokens, rows = c["B"], c["P"], c["width"], c["tokens"], c["rows"]
    ctx, add, table, free = (st[k].long() for k in ("ctx", "add", "table", "free"))
    F = st["free_count"].long()[0]
    cap = free.shape[0]
    dev = table.device
    ctx = ctx.clamp(0, width * P)
    n = add.clamp(0, tokens + 1)
    have = (ctx + P - 1) // P
    if rows:
        start = torch.arange(B + 1, device=dev) * rows
        fits = n <= rows
    else:
        start = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(n, 0)]).clamp(max=tokens)
        fits = torch.cumsum(n, 0) <= tokens
    fits = fits & (ctx + n <= width * P)
    out = add < 0
    want = torch.where(fits & ~out, (ctx + n + P - 1) // P - have, 0)
    upto = torch.cumsum(want, 0)
    back = torch.where(out, have, 0)
    R = back.sum()
    ok = fits & ~out & ((want == 0) | (upto <= F + R))
    taken = torch.where(ok, want, 0).sum()
    j = torch.arange(width, device=dev)[None, :]
    # the stack: the free list, then the released pages in the order of their rows
    rel = out[:, None] & (j < have[:, None])
    place = torch.where(rel, F + (torch.cumsum(back, 0) - back)[:, None] + j, cap + B * width)
    stack = torch.cat([free, torch.full((B * width + 1,), -1, dtype=torch.long, device=dev)])
    stack = stack.scatter(0, place.reshape(-1), table.reshape(-1))
    top = F + R - 1
    fresh = ok[:, None] & (j >= have[:, None]) & (j < (have + want)[:, None])
    at = (top - (upto - want)[:, None] - (j - have[:, None])).clamp(0, cap + B * width)
    table = torch.where(fresh, stack[at], table)
    left = F + R - taken
    i = torch.arange(cap, device=dev)
    free = torch.where(i < left, stack[:cap], free)
    length = torch.where(out, 0, torch.where(ok, ctx + n, ctx))
    t = torch.arange(tokens, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=B - 1)
    k = t - start[b]
    live = ok[b] & (k >= 0) & (k < n[b])
    pos = torch.where(live, ctx[b] + k, -1)
    page = table[b, (pos.clamp(min=0) // P)]
    slot = torch.where(live & (page >= 0) & (page < st["pages"]), page * P + pos % P, -1)
    refused = (~out & ~ok & (n > 0)).sum()
    counts = torch.stack([live.sum(), taken, left, refused])
    got = {"table": table, "free": free, "len": length, "start": start, "slot": slot, "pos": pos, "counts": counts}
    return {k: v.int() for k, v in got.items()}


def _sizes(c):
    """Elements of a key unit, dimensions and tokens of a value unit."""
    e = _esize(c["fmt"])
    cv = 4 if c["D"] == 64 else 8
    return 16 // e, cv, 16 // (e * cv)


def _rotate(x, pos, cos_sin, rot):
    """x [T, heads, D] fp32: the first rot dimensions in pairs (i, i + rot / 2)."""
    h = rot // 2
    cs = cos_sin[pos.clamp(min=0).long()][:, None, :]
    a, b = x[..., :h], x[..., h:rot]
    return torch.cat([a * cs[..., :h] - b * cs[..., h:], b * cs[..., :h] + a * cs[..., h:], x[..., rot:]], dim=-1)


def _plain_append(st):
    c = st["case"]
    T, P, D, hq, hkv, fmt, rot = c["T"], c["P"], c["D"], c["hq"], c["hkv"], c["fmt"], c["rot"]
    x = st["qkv"].view(T, hq + 2 * hkv, D).float()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if rot:
        q, k = _rotate(q, st["pos"], st["cos_sin"], rot), _rotate(k, st["pos"], st["cos_sin"], rot)
    on = st["slot"] >= 0
    ck, cv, tu = _sizes(c)
    s = st["slot"].long().clamp(min=0)
    page, off = (s // P)[:, None, None], (s % P)[:, None, None]
    h = torch.arange(hkv, device=x.device)[None, :, None]
    dim = torch.arange(D, device=x.device)[None, None, :]
    base = ((page * hkv + h) * (P // 16) + off // 16) * (16 * D)
    r = off % 16
    ki = base + ((dim // ck) * 16 + r) * ck + dim % ck
    vi = base + ((r // tu) * (D // cv) + dim // cv) * (tu * cv) + (r % tu) * cv + dim % cv

    def put(pool, at, val, scale):
        if fmt == "bf16":
            pool.view(torch.int16).view(-1)[at[on]] = val.to(torch.bfloat16).view(torch.int16)[on]
        else:
            val = (val / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            pool.view(torch.uint8).view(-1)[at[on]] = val.view(torch.uint8)[on]

    put(st["k"], ki, k.contiguous(), st["k_scale"])
    put(st["v"], vi, v.contiguous(), st["v_scale"])
    if rot:
        st["q_out"][on] = q.reshape(T, hq * D).to(torch.bfloat16)[on]
    return {"k": st["k"], "v": st["v"], "q": st["q_out"]}


def _gathered(st, which, table):
    """Keys or values of every request's table [B, hkv, width * P, D] in fp32."""
    c = st["case"]
    D, hkv, P = c["D"], c["hkv"], c["P"]
    ck, cv, tu = _sizes(c)
    pool = st[which]
    raw = pool.view(torch.int16 if c["fmt"] == "bf16" else torch.uint8)[table]
    x = raw.view(pool.dtype).float()
    B, W = table.shape
    if which == "k":
        x = x.view(B, W, hkv, P // 16, D // ck, 16, ck).permute(0, 2, 1, 3, 5, 4, 6)
    else:
        x = x.view(B, W, hkv, P // 16, 16 // tu, D // cv, tu, cv).permute(0, 2, 1, 3, 4, 6, 5, 7)
    x = x.reshape(B, hkv, W * P, D)
    scale = st[which + "_scale"]
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attend(st):
    c = st["case"]
    B, D, hq, hkv = c["B"], c["D"], c["hq"], c["hkv"]
    table = st["table"].long().clamp(min=0)
    q = st["qkv"][:, :hq * D].float().reshape(B, hkv, hq // hkv, D)
    k = _gathered(st, "k", table)
    s = (q @ k.transpose(2, 3).contiguous()) * (D ** -0.5)
    del k
    n = st["len"].long()[:, None]
    t = torch.arange(s.shape[-1], device=s.device)[None, :]
    on = t < n
    if c["window"]:
        on = on & (t >= n - c["window"])
    on = on[:, None, None, :]
    s = torch.where(on, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    sink = None
    if st["sinks"] is not None:
        sink = st["sinks"].view(1, hkv, hq // hkv, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(s - m)
    del s
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - m)
    o = p @ _gathered(st, "v", table)
    o = torch.where(total > 0, o / total, 0.0)
    return {"out": o.reshape(B, hq * D).to(torch.bfloat16)}


def _plain_norm(st):
    c = st["case"]
    b, r = st["block"].float(), st["residual"].float()
    u = b
    if st["post"] is not None:
        u = b * torch.rsqrt(b.square().mean(-1, keepdim=True) + EPS) * st["post"].float()
    if st["gate"] is not None:
        g = st["gate"].float()
        g = torch.sigmoid(g) if c["sigmoid"] else g
        u = u * (g[:, None] if c["gate"] == "token" else g)
    s = c["scale"] * r + u
    n = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * st["pre"].float()
    return {"sum": s.to(torch.bfloat16), "normed": n.to(torch.bfloat16)}


# ---- what a pass cannot do without ------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "plan":
        # per request two lengths in, two numbers out and its share of the pages; per token a slot and a position
        return {"bytes": 4 * (4 * c["B"] + 2 * c["tokens"] + 2 * (c["tokens"] // c["P"] + 1)), "flops": 0}
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        gate = {"none": 0, "channel": d, "token": T, "full": T * d}[c["gate"]]
        return {"bytes": 2 * (4 * T * d + (2 if c["post"] else 1) * d + gate), "flops": (12 if c["post"] else 7) * T * d}
    D, hq, hkv = c["D"], c["hq"], c["hkv"]
    e = _esize(c["fmt"])
    if c["op"] == "append":
        T, rot = c["T"], c["rot"]
        moved = 2 * 2 * hkv * D + 2 * e * hkv * D + (4 * hq * D + 4 * rot if rot else 0) + 8
        return {"bytes": T * moved, "flops": 3 * T * (hq + hkv) * rot}
    seen = int(_visible(c).sum())
    return {"bytes": 2 * e * seen * hkv * D + 4 * c["B"] * hq * D + 4 * (seen // c["P"] + 2 * c["B"]),
            "flops": 4 * seen * hq * D}


# ---- the definition in 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend, "norm": _exact_norm}[case["op"]](st)


def _exact_plan(st):
    """The definition request by request."""
    c = st["case"]
    P, width, tokens, rows = c["P"], c["width"], c["tokens"], c["rows"]
    ctx, add, table, free = (st[k].cpu().numpy().astype(np.int64) for k in ("ctx", "add", "table", "free"))
    F = int(st["free_count"].item())
    stack = list(free[:F])
    length = np.zeros(c["B"], np.int64)
    start = np.zeros(c["B"] + 1, np.int64)
    slot, pos = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int64)
    for b in range(c["B"]):
        if add[b] < 0:
            stack.extend(table[b, :-(-ctx[b] // P)])
    placed = taken = refused = at = asked = 0
    room = len(stack)
    for b in range(c["B"]):
        n, k = max(int(add[b]), 0), int(ctx[b])
        start[b] = b * rows if rows else min(at, tokens)
        fits = k + n <= width * P and (n <= rows if rows else at + n <= tokens)
        at += n
        if add[b] < 0:
            continue
        have, then = -(-k // P), -(-(k + n) // P)
        want = then - have if fits else 0
        asked += want
        length[b] = k
        if not fits or (want and asked > room):
            refused += n > 0
            continue
        for j in range(have, then):
            table[b, j] = stack.pop()
        taken += want
        length[b] = k + n
        for i in range(n):
            p = k + i
            pos[start[b] + i] = p
            slot[start[b] + i] = table[b, p // P] * P + p % P
        placed += n
    start[c["B"]] = c["B"] * rows if rows else min(at, tokens)
    free[:len(stack)] = stack
    counts = np.array([placed, taken, len(stack), refused])
    got = {"table": table, "free": free, "len": length, "start": start, "slot": slot, "pos": pos, "counts": counts}
    return {k: torch.from_numpy(np.asarray(v).astype(np.int32)) for k, v in got.items()}


def _e4m3_values(device):
    """Value of every code: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    half = [math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10) for e in range(16) for m in range(8)]
    half[127] = float("nan")
    return torch.tensor(half + [-v for v in half], dtype=torch.float64, device=device)


def _values64(c, pool):
    if c["fmt"] == "bf16":
        return pool.double()
    return _e4m3_values(pool.device)[pool.view(torch.uint8).int()]


def _place(c, slot, head, dim, which):
    """Element of a pool that holds dimension `dim` of the token at `slot`."""
    D, P, e = c["D"], c["P"], _esize(c["fmt"])
    page, inside = slot // P, slot % P
    block = page * (c["hkv"] * P * D) + head * (P * D) + inside // 16 * (16 * D)
    tok = inside % 16
    if which == "k":
        per = 16 // e
        unit, rest = dim // per * 16 + tok, dim % per
    else:
        dims = 8 if D > 64 else 4
        group = 16 // e // dims
        per = 16 // e
        unit, rest = tok // group * (D // dims) + dim // dims, tok % group * dims + dim % dims
    return block + unit * per + rest


def _exact_append(st):
    c = st["case"]
    D, hq, hkv, rot = c["D"], c["hq"], c["hkv"], c["rot"]
    on = torch.nonzero(st["slot"] >= 0)[:, 0]
    x = st["qkv"].double().view(c["T"], hq + 2 * hkv, D)[on]
    if rot:
        cs = st["cos_sin"].double()[st["pos"][on].long()]
        # the pair (i, i + rot/2) as a complex number times cos + i sin
        z = torch.complex(x[:, :hq + hkv, :rot // 2].contiguous(), x[:, :hq + hkv, rot // 2:rot].contiguous())
        z = z * torch.complex(cs[:, :rot // 2].contiguous(), cs[:, rot // 2:].contiguous())[:, None, :]
        x = x.clone()
        x[:, :hq + hkv, :rot // 2] = z.real
        x[:, :hq + hkv, rot // 2:rot] = z.imag
    slot = st["slot"][on].long()[:, None, None]
    head = torch.arange(hkv, device=x.device)[None, :, None]
    dim = torch.arange(D, device=x.device)[None, None, :]
    out = {}
    for which, first in (("k", hq), ("v", hq + hkv)):
        pool = _values64(c, st[which]).reshape(-1)
        val = x[:, first:first + hkv]
        if c["fmt"] == "e4m3":
            val = (val / st[which + "_scale"].double()[None, :, None]).clamp(-448, 448)
        pool[_place(c, slot, head, dim, which)] = val
        out[which] = pool.view(st[which].shape)
    q = torch.zeros(c["T"], hq * D, dtype=torch.float64, device=x.device)
    if rot:
        q[on] = x[:, :hq].reshape(len(on), hq * D)
    out["q"] = q
    return out


def _exact_attend(st):
    c = st["case"]
    D, hq, hkv, P = c["D"], c["hq"], c["hkv"], c["P"]
    out = torch.zeros(c["B"], hq * D, dtype=torch.float64, device=st["k"].device)
    dev = out.device
    head = torch.arange(hkv, device=dev)[:, None, None]
    dim = torch.arange(D, device=dev)[None, None, :]
    flat = {w: st[w].view(torch.int16 if c["fmt"] == "bf16" else torch.uint8).reshape(-1) for w in "kv"}
    values = _e4m3_values(dev)
    q = st["qkv"].double()

    def read(which, slots):
        raw = flat[which][_place(c, slots[None, :, None], head, dim, which)]
        if c["fmt"] == "bf16":
            return raw.view(torch.bfloat16).double()
        return values[raw.int()] * st[which + "_scale"].double()[:, None, None]

    for b, n in enumerate(st["len"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == lo:
            continue
        t = torch.arange(lo, n, device=dev)
        slots = st["table"][b].long()[t // P] * P + t % P
        qb = q[b, :hq * D].view(hkv, hq // hkv, D)
        s = torch.matmul(qb, read("k", slots).transpose(1, 2).contiguous()) / math.sqrt(D)
        if st["sinks"] is not None:
            s = torch.cat([s, st["sinks"].double().view(hkv, hq // hkv, 1)], dim=2)
        w = torch.softmax(s, dim=2)[:, :, :n - lo].contiguous()
        out[b] = torch.matmul(w, read("v", slots)).reshape(-1)
    return {"out": out}


def _exact_norm(st):
    c = st["case"]
    b, r = st["block"].double(), st["residual"].double()
    d = c["d"]
    if st["post"] is not None:
        b = st["post"].double() * b / torch.sqrt((b * b).sum(1, keepdim=True) / d + EPS)
    if st["gate"] is not None:
        g = st["gate"].double()
        if c["sigmoid"]:
            g = 1.0 / (1.0 + torch.exp(-g))
        b = b * (g.view(-1, 1) if c["gate"] == "token" else g)
    s = r * c["scale"] + b
    return {"sum": s, "normed": st["pre"].double() * s / torch.sqrt((s * s).sum(1, keepdim=True) / d + EPS)}
