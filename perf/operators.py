"""Cases of the resident-weight operators: what is timed, on which inputs, and what the outputs are.

Three operators, over weights that stay in device memory in the library's record format (panel-ordered
bf16, block-FP8 or MXFP4; see include/ftmoe.h):

  moe      a whole mixture-of-experts layer for a few tokens: top-k routing, the routed experts' SwiGLU
           FFN and the weighted combine (ft_moe_layer).
  project  one shared projection with the low-rank adapters of many requests beside it
           (ft_lora_project): y = base + x W + scale_a (x A_a) B_a, a = the token's adapter.
  expert   a shared expert's SwiGLU FFN with low-rank adapters beside its three projections
           (ft_lora_expert).

`listed()` gives the timed cases, `draw(rng)` others of the same ranges, `prepare(case, seed)` the inputs,
`run(state)` one call, `work(case)` the bytes and operations it cannot do without and `exact(case, seed)`
its outputs in 64 bits.  With `own` false `run` is the plain form in elementary torch operations in 32
bits; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

_CHUNK = {"bf16": 8, "fp8": 16, "mxfp4": 32}          # elements of a 16-byte chunk along K
_FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ----------------------------------------------------------------------------------------

def _moe(name, fmt, d, f, E, k, T, base):
    return {"name": name, "op": "moe", "fmt": fmt, "d": d, "f": f, "E": E, "k": k, "T": T, "base": base}


def _project(name, fmt, K, n, T, requests, adapters, rank, base):
    return {"name": name, "op": "project", "fmt": fmt, "d": K, "n": n, "T": T, "requests": requests,
            "adapters": adapters, "rank": rank, "base": base}


def _expert(name, fmt, d, f, T, requests, adapters, rank, base):
    return {"name": name, "op": "expert", "fmt": fmt, "d": d, "f": f, "T": T, "requests": requests,
            "adapters": adapters, "rank": rank, "base": base}


def listed():
    return [
        # the tiny configuration's layer for one token: nothing but latency
        _moe("moe_tiny_t1", "bf16", 256, 128, 8, 2, 1, False),
        # one decoding request on the bf16 decode configuration's layer
        _moe("moe_bf16_t1", "bf16", 2048, 768, 128, 8, 1, True),
        # a batch of sixteen decoding requests on the same layer: most experts serve one token
        _moe("moe_bf16_t16", "bf16", 2048, 768, 128, 8, 16, True),
        # a speculative run of five tokens on the block-FP8 configuration's layer
        _moe("moe_fp8_t5", "fp8", 4096, 2048, 256, 8, 5, False),
        # a full decode batch on the MXFP4 configuration's layer: nearly every expert is read
        _moe("moe_mxfp4_t64", "mxfp4", 7168, 2048, 256, 8, 64, False),
        # one token of one request through a square projection of the decode configuration's width
        _project("project_bf16_t1", "bf16", 2048, 2048, 1, 1, 4, 16, False),
        # a decode batch of many requests, each with its own choice of 32 adapters of mixed ranks
        _project("project_fp8_t64", "fp8", 4096, 4096, 64, 64, 32, 64, False),
        # a prefill chunk: eleven requests of ragged lengths, adapters of up to 32 ranks
        _project("project_bf16_t8192", "bf16", 2048, 2048, 8192, 11, 8, 32, True),
        # the shared expert of the decode configuration's size for a small decode batch
        _expert("expert_bf16_t7", "bf16", 2048, 768, 7, 7, 8, 16, True),
        # the block-FP8 expert for a decode batch of many adapters
        _expert("expert_fp8_t64", "fp8", 4096, 2048, 64, 64, 32, 32, False),
        # a short, odd prompt chunk: too long for a matrix-vector shape, too short to fill the card by rows
        _expert("expert_bf16_t777", "bf16", 2048, 768, 777, 5, 8, 16, True),
        # the MXFP4 configuration's prefill chunk through its expert, a few long requests
        _expert("expert_mxfp4_t4096", "mxfp4", 7168, 2048, 4096, 6, 8, 16, False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_128(rng, lo, hi):
    return 128 * _log_int(rng, lo // 128, hi // 128)


def _matrix_bytes(fmt, rows, K):
    if fmt == "bf16":
        return 2 * rows * K
    if fmt == "fp8":
        return rows * K + 4 * (rows // 128) * (K // 128)
    return rows * K // 2 + rows * K // 32


def draw(rng):
    op = rng.choice(("moe", "moe", "project", "expert"))
    fmt = rng.choice(("bf16", "fp8", "mxfp4"))
    base = rng.random() < 0.5
    d = _log_128(rng, 256, 7168)
    if op == "moe":
        f = _log_128(rng, 128, 2048)
        E = _log_int(rng, 4, 256)
        T = _log_int(rng, 1, 64)
        while E * 3 * _matrix_bytes(fmt, f, d) > 6 * 2 ** 30:
            E = E * 2 // 3
        return {"op": op, "fmt": fmt, "d": d, "f": f, "E": E, "k": rng.randint(1, min(8, E)), "T": T, "base": base}
    T = _log_int(rng, 1, 8192)
    requests = _log_int(rng, 1, min(T, 64))
    adapters = _log_int(rng, 1, 32)
    rank = 16 * rng.choice((1, 2, 3, 4, 8))
    if op == "project":
        n = _log_128(rng, 256, 7168)
        while T * n * d > 4096 * 7168 * 2048:
            T //= 2
        c = {"op": op, "fmt": fmt, "d": d, "n": n}
    else:
        f = _log_128(rng, 128, 2048)
        while T * f * d > 4096 * 7168 * 2048:
            T //= 2
        c = {"op": op, "fmt": fmt, "d": d, "f": f}
    c.update(T=T, requests=min(requests, T), adapters=adapters, rank=rank, base=base)
    return c


# ---- inputs ---------------------------------------------------------------------------------------

def _panels(rows_bytes, unit):
    """Row-major bytes [..., rows, row_bytes] -> the record's panel order, flattened over rows."""
    *lead, rows, rb = rows_bytes.shape
    n = len(lead)
    a = rows_bytes.reshape(*lead, rows // 32, 32, rb // (2 * unit), 2, unit)
    return a.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).reshape(*lead, rows * rb)


def _make_matrix(fmt, rows, K, gen):
    """Random weights ~ N(0, 0.02) in one format: (code bytes, scale bytes), as a record holds them."""
    dev = "cuda"
    if fmt == "bf16":
        w = (torch.randn(rows, K, device=dev, generator=gen) * 0.02).to(torch.bfloat16)
        return _panels(w.view(torch.uint8), 16), None
    if fmt == "fp8":
        w = (torch.randn(rows, K, device=dev, generator=gen) * 0.02).reshape(rows // 128, 128, K // 128, 128)
        s = w.abs().amax(dim=(1, 3), keepdim=True) / 448.0
        c = (w / s).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(rows, K).view(torch.uint8)
        return _panels(c, 16), s.reshape(-1).contiguous().view(torch.uint8)
    # random codes; block scales as the largest of 32 normal draws would set them (mostly 2^-7 .. 2^-5 of
    # the largest code)
    c = torch.randint(0, 256, (rows, K // 2), device=dev, dtype=torch.uint8, generator=gen)
    amax = 0.02 * (2.0 + 0.45 * torch.randn(rows, K // 32, device=dev, generator=gen)).clamp(1.0, 4.0)
    e = (torch.floor(torch.log2(amax)) - 2 + 127).to(torch.uint8)
    return _panels(c, 16), _panels(e, 1)


def _make_record(fmt, d, f, gen):
    parts, scales = [], []
    for rows, K in ((f, d), (f, d), (d, f)):
        c, s = _make_matrix(fmt, rows, K, gen)
        parts.append(c)
        if s is not None:
            scales.append(s)
    return torch.cat(parts + scales)


def _make_lora(count, rank, K, n, gen, ranks):
    return {"a": (torch.randn(count, rank, K, device="cuda", generator=gen) * 0.02).to(torch.bfloat16),
            "b": (torch.randn(count, n, rank, device="cuda", generator=gen) * 0.02).to(torch.bfloat16),
            "rank": ranks, "scale": 0.5 + torch.rand(count, device="cuda", generator=gen)}


def _adapter_ids(case, rng):
    """Each request has one adapter, or (about one in eight) none; its tokens are contiguous."""
    T, n = case["T"], case["requests"]
    cuts = np.sort(rng.choice(np.arange(1, T), size=n - 1, replace=False)) if n > 1 else np.zeros(0, np.int64)
    lengths = np.diff(np.concatenate([[0], cuts, [T]])).astype(np.int64)
    ids = np.where(rng.random(n) < 0.125, -1, rng.integers(0, case["adapters"], n))
    return torch.from_numpy(np.repeat(ids, lengths).astype(np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    rng = np.random.default_rng([seed, 29])
    T, d, fmt = case["T"], case["d"], case["fmt"]
    out = case["n"] if case["op"] == "project" else d
    st = {"case": case, "x": torch.randn(T, d, device="cuda", generator=gen).to(torch.bfloat16),
          "base": torch.randn(T, out, device="cuda", generator=gen).to(torch.bfloat16) if case["base"] else None}
    if case["op"] == "moe":
        f, E = case["f"], case["E"]
        S = 3 * _matrix_bytes(fmt, f, d)
        P = (S + 255) // 256 * 256
        recs = torch.zeros(E, P, device="cuda", dtype=torch.uint8)
        for e in range(E):
            recs[e, :S] = _make_record(fmt, d, f, gen)
        st["records"] = recs
        st["router"] = (torch.randn(d, E, device="cuda", generator=gen) * 0.02).to(torch.bfloat16)
    else:
        count, rank = case["adapters"], case["rank"]
        ranks = torch.from_numpy(rng.integers(max(1, rank // 4), rank + 1, count).astype(np.int32)).cuda()
        st["adapter"] = _adapter_ids(case, rng)
        if case["op"] == "project":
            st["codes"], st["scales"] = _make_matrix(fmt, out, d, gen)
            st["lora"] = _make_lora(count, rank, d, out, gen, ranks)
        else:
            f = case["f"]
            st["record"] = _make_record(fmt, d, f, gen)
            st["gate"] = _make_lora(count, rank, d, f, gen, ranks)
            st["up"] = _make_lora(count, rank, d, f, gen, ranks)
            st["down"] = _make_lora(count, rank, f, d, gen, ranks)
    if own:
        _keep(st)
    return st


def _keep(st):
    """What a program that uses the library keeps between calls: the shape, the workspace, output buffers
    and the adapter tables' descriptions."""
    import moe_expert_execution_amd as M
    from moe_expert_execution_amd.tensors import LoraPool, Workspace
    c = st["case"]
    T = c["T"]
    if c["op"] == "moe":
        st["shape"] = M.shape(1, c["E"], c["k"], c["d"], c["f"], c["fmt"])
        st["ws"] = Workspace(M.ft_moe_layer_workspace(st["shape"], T))
        st["ids"] = torch.empty(T, c["k"], device="cuda", dtype=torch.int32)
        st["w"] = torch.empty(T, c["k"], device="cuda")
        st["y"] = torch.empty(T, c["d"], device="cuda", dtype=torch.bfloat16)
        return

    def pool(p):
        return LoraPool(p["a"], p["b"], p["rank"], p["scale"])

    if c["op"] == "project":
        st["matrix"] = M.matrix(c["n"], c["d"], c["fmt"], st["codes"].data_ptr(),
                                st["scales"].data_ptr() if st["scales"] is not None else 0)
        st["pool"] = pool(st["lora"])
        st["ws"] = Workspace(M.ft_lora_project_workspace(st["matrix"], c["rank"], T))
        st["y"] = torch.empty(T, c["n"], device="cuda", dtype=torch.bfloat16)
    else:
        st["shape"] = M.shape(1, 1, 1, c["d"], c["f"], c["fmt"])
        st["pools"] = [pool(st[p]) for p in ("gate", "up", "down")]
        st["ws"] = Workspace(M.ft_lora_expert_workspace(st["shape"], c["rank"], T))
        st["y"] = torch.empty(T, c["d"], device="cuda", dtype=torch.bfloat16)


# ---- one pass -------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"moe": _plain_moe, "project": _plain_project, "expert": _plain_expert}[op](state)


def _own(st, op):
    import moe_expert_execution_amd as M
    T = st["case"]["T"]
    stream = torch.cuda.current_stream().cuda_stream
    base = st["base"].data_ptr() if st["base"] is not None else 0
    if op == "moe":
        M.ft_moe_layer(st["shape"], st["x"].data_ptr(), st["router"].data_ptr(), st["records"].data_ptr(),
                       st["records"].shape[1], T, base, st["ids"].data_ptr(), st["w"].data_ptr(),
                       st["y"].data_ptr(), st["ws"].handle, stream)
        return {"y": st["y"], "ids": st["ids"], "w": st["w"]}
    if op == "project":
        M.ft_lora_project(st["matrix"], st["pool"].struct, st["x"].data_ptr(), st["adapter"].data_ptr(), T, base,
                          st["y"].data_ptr(), st["ws"].handle, stream)
    else:
        g, u, dn = (p.struct for p in st["pools"])
        M.ft_lora_expert(st["shape"], st["record"].data_ptr(), g, u, dn, st["x"].data_ptr(),
                         st["adapter"].data_ptr(), T, base, st["y"].data_ptr(), st["ws"].handle, stream)
    return {"y": st["y"]}


def _rows(phys, rows, row_bytes, unit):
    """Panel order -> row-major bytes [rows, row_bytes]."""
    a = phys.reshape(rows // 32, row_bytes // (2 * unit), 2, 32, unit)
    return a.permute(0, 3, 1, 2, 4).reshape(rows, row_bytes)


def _fp4_pairs(device):
    t = torch.tensor(_FP4 + tuple(-v for v in _FP4), device=device)
    b = torch.arange(256, device=device)
    return torch.stack([t[b % 16], t[b // 16]], dim=1)


def _decode(fmt, rows, K, codes, scales, pairs):
    """One matrix [rows, K] in fp32 from its code and scale bytes."""
    if fmt == "bf16":
        return _rows(codes, rows, 2 * K, 16).view(torch.bfloat16).float()
    if fmt == "fp8":
        w = _rows(codes, rows, K, 16).view(torch.float8_e4m3fn).float().view(rows // 128, 128, K // 128, 128)
        return (w * scales.view(torch.float32).view(rows // 128, 1, K // 128, 1)).view(rows, K)
    w = pairs.index_select(0, _rows(codes, rows, K // 2, 16).reshape(-1).int()).view(rows, K // 32, 32)
    s = torch.exp2(_rows(scales, rows, K // 32, 1).float() - 127.0)
    return (w * s.view(rows, K // 32, 1)).view(rows, K)


def _decode_record(fmt, d, f, rec, pairs):
    """WgT [f, d], WuT [f, d], WdT [d, f] of one record, in fp32."""
    cb = d * f * 16 // (8 * _CHUNK[fmt]) * 8
    sb = {"bf16": 0, "fp8": 4 * (d // 128) * (f // 128), "mxfp4": d * f // 32}[fmt]
    out = []
    for i, (rows, K) in enumerate(((f, d), (f, d), (d, f))):
        s = rec[3 * cb + i * sb:3 * cb + (i + 1) * sb]
        out.append(_decode(fmt, rows, K, rec[i * cb:(i + 1) * cb], s, pairs))
    return out


def _swiglu(g, u):
    return g * torch.sigmoid(g) * u


def _plain_moe(st):
    c = st["case"]
    T, d, f, E, k, fmt = c["T"], c["d"], c["f"], c["E"], c["k"], c["fmt"]
    # logits in 64 bits: an expert next to the k-th place is decided by their last digits
    z = st["x"].double() @ st["router"].double()
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    ids = order[:, :k].contiguous()
    w = torch.softmax(zs[:, :k], dim=1).float()
    x = st["x"].float()
    pairs = _fp4_pairs(x.device)
    y = torch.zeros(T, d, device=x.device)
    if T * k < E:
        for r in range(T * k):
            t, j = divmod(r, k)
            rec = st["records"].index_select(0, ids[t, j:j + 1])[0]
            wg, wu, wd = _decode_record(fmt, d, f, rec, pairs)
            xt = x[t:t + 1]
            y[t] += w[t, j] * (_swiglu(xt @ wg.T, xt @ wu.T) @ wd.T)[0]
    else:
        for e in range(E):
            we = torch.where(ids == e, w, 0.0).sum(1, keepdim=True)
            wg, wu, wd = _decode_record(fmt, d, f, st["records"][e], pairs)
            y += torch.where(we != 0, we * (_swiglu(x @ wg.T, x @ wu.T) @ wd.T), 0.0)
    if st["base"] is not None:
        y = y + st["base"].float()
    return {"y": y.to(torch.bfloat16), "ids": ids.int(), "w": w}


def _plain_lora(p, x, adapter):
    """scale_a (x A_a) B_a of every row's adapter (0 where it has none), in fp32."""
    count, R, _ = p["a"].shape
    live = torch.arange(R, device=x.device)[None, :] < p["rank"][:, None]
    out = torch.zeros(x.shape[0], p["b"].shape[1], device=x.device)
    if x.shape[0] <= 128:
        on = adapter >= 0
        i = adapter.clamp(min=0).long()
        v = (p["a"][i].float() @ x[:, :, None])[:, :, 0]
        v = torch.where(live[i], v, 0.0) * p["scale"][i][:, None]
        y = (p["b"][i].float() @ v[:, :, None])[:, :, 0]
        return torch.where(on[:, None], y, out)
    for a in range(count):
        v = torch.where(live[a], x @ p["a"][a].float().T, 0.0) * p["scale"][a]
        out = torch.where((adapter == a)[:, None], v @ p["b"][a].float().T, out)
    return out


def _plain_project(st):
    c = st["case"]
    x = st["x"].float()
    w = _decode(c["fmt"], c["n"], c["d"], st["codes"], st["scales"], _fp4_pairs(x.device))
    y = x @ w.T + _plain_lora(st["lora"], x, st["adapter"])
    if st["base"] is not None:
        y = y + st["base"].float()
    return {"y": y.to(torch.bfloat16)}


def _plain_expert(st):
    c = st["case"]
    x = st["x"].float()
    wg, wu, wd = _decode_record(c["fmt"], c["d"], c["f"], st["record"], _fp4_pairs(x.device))
    g = x @ wg.T + _plain_lora(st["gate"], x, st["adapter"])
    u = x @ wu.T + _plain_lora(st["up"], x, st["adapter"])
    h = _swiglu(g, u)
    y = h @ wd.T + _plain_lora(st["down"], h, st["adapter"])
    if st["base"] is not None:
        y = y + st["base"].float()
    return {"y": y.to(torch.bfloat16)}


# ---- what a pass cannot do without ------------------------------------------------------------------

def _distinct(n, draws, per_draw=1):
    """Expected number of distinct values among `draws` draws of `per_draw` of n."""
    return n * (1.0 - (1.0 - per_draw / n) ** draws)


def work(case):
    c = case
    T, d, fmt = c["T"], c["d"], c["fmt"]
    out = c["n"] if c["op"] == "project" else d
    rows = 2 * T * d + 2 * T * out * (2 if c["base"] else 1)       # x, y and the addend
    if c["op"] == "moe":
        f, E, k = c["f"], c["E"], c["k"]
        rec = 3 * _matrix_bytes(fmt, f, d)
        return {"bytes": int(_distinct(E, T, k) * rec + 2 * d * E + rows + 8 * T * k),
                "flops": 2 * T * d * E + 6 * T * k * d * f}
    used = _distinct(c["adapters"], c["requests"] * 0.875)
    r = 0.625 * c["rank"]                                           # mean rank of an adapter
    if c["op"] == "project":
        n = c["n"]
        return {"bytes": int(_matrix_bytes(fmt, n, d) + rows + 4 * T + used * r * (d + n) * 2),
                "flops": int(2 * T * d * n + 1.75 * T * r * (d + n))}
    f = c["f"]
    return {"bytes": int(3 * _matrix_bytes(fmt, f, d) + rows + 4 * T + used * r * 3 * (d + f) * 2),
            "flops": int(6 * T * d * f + 1.75 * T * r * 3 * (d + f))}


# ---- the definition in 64 bits ----------------------------------------------------------------------

def _table64(fmt, device):
    """Value of every code: e4m3 (sign, 4 exponent bits of bias 7, 3 mantissa bits) or e2m1 (bias 1, 1 bit)."""
    n, eb, mb, bias = (256, 4, 3, 7) if fmt == "fp8" else (16, 2, 1, 1)
    vals = []
    for code in range(n):
        m = code & ((1 << mb) - 1)
        e = (code >> mb) & ((1 << eb) - 1)
        v = math.ldexp(m, 1 - bias - mb) if e == 0 else math.ldexp((1 << mb) + m, e - bias - mb)
        vals.append(-v if code >> (eb + mb) else v)
    if fmt == "fp8":
        vals[0x7F] = vals[0xFF] = float("nan")
    return torch.tensor(vals, dtype=torch.float64, device=device)


def _matrix64(fmt, rows, K, codes, scales):
    """One matrix [rows, K] in fp64: element (r, c) is looked up where the format's definition puts it."""
    dev = codes.device
    epc = _CHUNK[fmt]
    r = torch.arange(rows, device=dev)[:, None]
    col = torch.arange(K, device=dev)[None, :]

    def place(units_per_row, unit_index):
        return (r // 32) * (32 * units_per_row) + (unit_index // 2) * 64 + (unit_index % 2) * 32 + r % 32

    unit = place(K // epc, col // epc)
    if fmt == "bf16":
        bits = codes.view(torch.int16)[unit * 8 + col % 8]
        return bits.view(torch.bfloat16).double()
    table = _table64(fmt, dev)
    if fmt == "fp8":
        s = scales.view(torch.float32).double()[(r // 128) * (K // 128) + col // 128]
        return table[codes[unit * 16 + col % 16].int()] * s
    byte = codes[unit * 16 + (col % 32) // 2].int()
    code = torch.where(col % 2 == 0, byte & 15, byte >> 4)
    e = scales[place(K // 32, col // 32)].int()
    return torch.ldexp(table[code], e - 127)


def _record64(fmt, d, f, rec):
    bits = {"bf16": 16, "fp8": 8, "mxfp4": 4}[fmt]
    cb = d * f * bits // 8
    sb = {"bf16": 0, "fp8": d * f // 4096, "mxfp4": d * f // 32}[fmt]
    return [_matrix64(fmt, *((f, d) if i < 2 else (d, f)), rec[i * cb:(i + 1) * cb].contiguous(),
                      rec[3 * cb + i * sb:3 * cb + (i + 1) * sb].clone()) for i in range(3)]


def _ffn64(x, mats, lora=None):
    wg, wu, wd = mats
    add = lora if lora is not None else (lambda name, v: 0.0)
    g = x @ wg.T + add("gate", x)
    u = x @ wu.T + add("up", x)
    h = g / (1.0 + torch.exp(-g)) * u
    return h @ wd.T + add("down", h)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    x = st["x"].double()
    y = torch.zeros(c["T"], c["n"] if c["op"] == "project" else c["d"], dtype=torch.float64, device=x.device)
    if st["base"] is not None:
        y = y + st["base"].double()
    if c["op"] == "moe":
        z = x @ st["router"].double()
        order = np.argsort(-z.cpu().numpy(), axis=1, kind="stable")[:, :c["k"]]
        ids = torch.from_numpy(order.copy()).to(x.device)
        top = z.gather(1, ids)
        w = torch.exp(top - top[:, :1])
        w = w / w.sum(1, keepdim=True)
        for e in np.unique(order):
            tt, jj = np.nonzero(order == e)
            tt, jj = torch.from_numpy(tt).to(x.device), torch.from_numpy(jj).to(x.device)
            y[tt] += w[tt, jj][:, None] * _ffn64(x[tt], _record64(c["fmt"], c["d"], c["f"], st["records"][int(e)]))
        return {"y": y, "ids": ids.int(), "w": w}
    adapter = st["adapter"].cpu().numpy()

    def lora(p, v):
        out = torch.zeros(v.shape[0], p["b"].shape[1], dtype=torch.float64, device=v.device)
        for a in np.unique(adapter[adapter >= 0]):
            tt = torch.from_numpy(np.nonzero(adapter == a)[0]).to(v.device)
            r = int(p["rank"][int(a)])
            down = v[tt] @ p["a"][int(a), :r].double().T
            out[tt] = float(p["scale"][int(a)]) * (down @ p["b"][int(a), :, :r].double().T)
        return out

    if c["op"] == "project":
        return {"y": y + x @ _matrix64(c["fmt"], c["n"], c["d"], st["codes"], st["scales"]).T + lora(st["lora"], x)}
    mats = _record64(c["fmt"], c["d"], c["f"], st["record"])
    return {"y": y + _ffn64(x, mats, lambda name, v: lora(st[name], v))}
