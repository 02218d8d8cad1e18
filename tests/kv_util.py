"""Shared helpers of the key-value cache and block norm tests: the definitions in plain NumPy with 64 bits, and a bound
of the kernel's error for every output."""
import numpy as np
import torch

import moe_expert_execution_amd as M
from oracle import formats as OF
from tests.gpu_util import dev
from tests.resident_util import HALF, gamma

ESIZE = {"bf16": 2, "e4m3": 1}


# ---- the cache's layout, element by element ------------------------------------------------------

def place(fmt, D, which, tok, dim):
    """Byte inside a head's 16-token block of dimension `dim` of its token `tok`."""
    e = ESIZE[fmt]
    if which == "k":
        ck = 16 // e
        return (dim // ck * 16 + tok) * 16 + dim % ck * e
    cv = 4 if D == 64 else 8
    tu = 16 // (cv * e)
    return (tok // tu * (D // cv) + dim // cv) * 16 + (tok % tu * cv + dim % cv) * e


class Cache:
    """A cache on the device with random contents; host copies of its bytes."""

    def __init__(self, fmt, pages, P, heads, D, seed=0, gap=0, fill="normal"):
        rng = np.random.default_rng([seed, pages, P, heads, D])
        self.fmt, self.pages, self.P, self.heads, self.D = fmt, pages, P, heads, D
        e = ESIZE[fmt]
        self.page = heads * P * D * e
        self.stride = self.page + gap
        self.scales = None
        if fmt == "e4m3":
            self.scales = {w: rng.uniform(0.005, 0.02, heads).astype(np.float32) for w in "kv"}
        self.host = {}
        for w in "kv":
            n = pages * self.stride
            if fill == "nan":
                raw = np.full(n, 0xFF, np.uint8)                  # bf16 0xFFFF and e4m3 0xFF are NaN
            elif fmt == "bf16":
                raw = OF_bf16(rng.standard_normal(n // 2).astype(np.float32)).view(np.uint8)
            else:
                raw = rng.integers(0, 256, n).astype(np.uint8)
                raw[(raw & 0x7F) == 0x7F] = 0x15
            self.host[w] = np.ascontiguousarray(raw)
        self.upload()

    def upload(self):
        self.dev = {w: dev(self.host[w]) for w in "kv"}
        self.dev_scales = {w: dev(self.scales[w]) for w in "kv"} if self.scales else None

    def struct(self):
        s = self.dev_scales
        return M.kv_cache(self.pages, self.P, self.heads, self.D, self.fmt, self.dev["k"].data_ptr(),
                          self.dev["v"].data_ptr(), s["k"].data_ptr() if s else 0, s["v"].data_ptr() if s else 0,
                          self.stride)

    def offsets(self, which, slots, head):
        """Byte offsets [n, D] of the slots' elements."""
        slots = np.asarray(slots, np.int64)[:, None]
        dim = np.arange(self.D)[None, :]
        page, inside = slots // self.P, slots % self.P
        e = ESIZE[self.fmt]
        return (page * self.stride + head * self.P * self.D * e + inside // 16 * 16 * self.D * e +
                place(self.fmt, self.D, which, inside % 16, dim))

    def read(self, which, slots, head, raw=None):
        """Values [n, D] of the slots, in fp64."""
        raw = self.host[which] if raw is None else raw
        off = self.offsets(which, slots, head)
        if self.fmt == "bf16":
            bits = raw[off].astype(np.uint16) | raw[off + 1].astype(np.uint16) << 8
            return OF.bf16_to_f64(bits)
        return E4M3[raw[off]] * float(self.scales[which][head])

    def write(self, which, slots, head, values):
        """bf16 bits or e4m3 codes [n, D] into the host copy (then upload())."""
        off = self.offsets(which, slots, head)
        if self.fmt == "bf16":
            v = np.asarray(values, np.uint16)
            self.host[which][off] = (v & 255).astype(np.uint8)
            self.host[which][off + 1] = (v >> 8).astype(np.uint8)
        else:
            self.host[which][off] = np.asarray(values, np.uint8)


def OF_bf16(a):
    import synth
    return synth.f32_to_bf16(a)


def _e4m3():
    c = np.arange(256)
    m, e = (c & 7).astype(np.float64), (c >> 3) & 15
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c > 127, -v, v)


E4M3 = _e4m3()


# ---- attention ------------------------------------------------------------------------------------

def attend_row(q, k, v, scale, sinks=None):
    """q [g, D], k, v [n, D] in fp64 -> out [g, D] and the bound of |kernel - out|, its bf16 rounding included.

    A logit's error: fp32 sums of D products, then three roundings of its own size (scale, base 2, the subtraction of
    the maximum), each 2^-24 of |s| or |s - m|; exp2 is within 2^-22.  A probability's relative error is that; it is
    kept to 2^-16 for the product with v; sums over n tokens are fp32, rescaled at most n times."""
    g, D = q.shape
    n = len(k)
    if n == 0:
        return np.zeros((g, D)), np.zeros((g, D))
    s = scale * (q @ k.T)
    m = s.max(1, keepdims=True)
    if sinks is not None:
        m = np.maximum(m, sinks[:, None])
    w = np.exp(s - m)
    total = w.sum(1, keepdims=True)
    if sinks is not None:
        total = total + np.exp(sinks[:, None] - m)
    out = (w @ v) / total
    u = HALF["fp32"]
    ds = abs(scale) * gamma(D) * (np.abs(q) @ np.abs(k).T) + 4 * u * (np.abs(s) + np.abs(s - m)) + 4 * u * np.abs(m)
    e = ds + 2.0 ** -21
    num = (w * (e + 2.0 ** -16 + gamma(2 * n))) @ np.abs(v) / total
    den = np.abs(out) * ((w * e).sum(1, keepdims=True) / total + gamma(2 * n))
    err = 1.05 * (num + den) + 2.0 ** -20 * np.abs(out)
    return out, err + HALF["bf16"] * (np.abs(out) + err) + 1e-37


def attend_reference(cache, q_bits, table, lens, scale, window=0, sinks=None, raw=None):
    """q_bits [B, Hq, D] bf16 -> out, bound [B, Hq, D]."""
    B, Hq, D = q_bits.shape
    g = Hq // cache.heads
    q = OF.bf16_to_f64(q_bits)
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    room = table.shape[1] * cache.P
    for b in range(B):
        n = min(max(int(lens[b]), 0), room)
        t = np.arange(max(0, n - window) if window else 0, n)
        page = table[b, t // cache.P].astype(np.int64)
        ok = (page >= 0) & (page < cache.pages)
        slots = (page * cache.P + t % cache.P)[ok]
        for h in range(cache.heads):
            k = cache.read("k", slots, h, None if raw is None else raw["k"])
            v = cache.read("v", slots, h, None if raw is None else raw["v"])
            r = slice(h * g, (h + 1) * g)
            out[b, r], bound[b, r] = attend_row(q[b, r], k, v, scale, None if sinks is None else
                                                sinks[r].astype(np.float64))
    return out, bound


def random_table(lens, P, spare, seed, extra_width=2, pages=None):
    """A table of distinct shuffled pages for the lengths; entries past them are garbage ids."""
    rng = np.random.default_rng([seed, len(lens), P])
    have = [-(-max(int(n), 0) // P) for n in lens]
    pages = sum(have) + spare if pages is None else pages
    ids = rng.permutation(pages)[:sum(have)]
    width = max(max(have), 1) + extra_width
    table = rng.choice(np.array([-1, -2 ** 31, 2 ** 31 - 1, pages, 10 ** 6], np.int64), size=(len(lens), width))
    at = 0
    for b, k in enumerate(have):
        table[b, :k] = ids[at:at + k]
        at += k
    return table.astype(np.int32), pages


# ---- the plan ---------------------------------------------------------------------------------------

def plan_reference(context, add, table, free_pages, free_count, pages, P, tokens, row_tokens):
    """The definition request by request; integers."""
    B, width = table.shape
    table, free_pages = np.array(table, np.int64), np.array(free_pages, np.int64)
    room = width * P
    F = min(max(int(free_count), 0), pages)
    ctx = [min(max(int(c), 0), room) for c in context]
    stack = list(free_pages[:F])
    for b in range(B):
        if add[b] < 0:
            stack += [int(table[b, j]) for j in range(-(-ctx[b] // P))]
    size, counted, at = len(stack), 0, 0
    kv_len, start = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    slot, pos = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int64)
    served_tokens = taken = refused = 0
    for b in range(B):
        n = max(int(add[b]), 0)
        start[b] = b * row_tokens if row_tokens else min(at, tokens)
        fits = (n <= row_tokens if row_tokens else at + n <= tokens) and ctx[b] + n <= room
        at += n
        if add[b] < 0:
            continue
        kv_len[b] = ctx[b]
        have = -(-ctx[b] // P)
        lacks = -(-(ctx[b] + n) // P) - have if fits else 0
        counted += lacks
        if not fits or (lacks > 0 and counted > size):
            refused += n > 0
            continue
        for j in range(lacks):
            table[b, have + j] = stack.pop()
        taken += lacks
        served_tokens += n
        kv_len[b] = ctx[b] + n
        for i in range(n):
            p = ctx[b] + i
            page = table[b, p // P]
            pos[start[b] + i] = p
            if 0 <= page < pages:
                slot[start[b] + i] = page * P + p % P
    start[B] = B * row_tokens if row_tokens else min(at, tokens)
    left = min(len(stack), pages)
    free_pages[:left] = stack[:left]
    return {"table": table, "free": free_pages[:left], "kv_len": kv_len, "start": start, "slot": slot, "pos": pos,
            "counts": np.array([served_tokens, taken, left, refused])}


class Plan:
    """The device arrays of an ft_kv_batch."""

    def __init__(self, context, add, table, free_pages, free_count, pages, P, tokens, row_tokens, in_place=False):
        i32 = lambda a: dev(np.ascontiguousarray(np.asarray(a).astype(np.int32)))  # noqa: E731
        B, self.width = table.shape
        self.B, self.tokens = B, tokens
        self.context, self.add, self.table, self.free = i32(context), i32(add), i32(table), i32(free_pages)
        self.counts = i32([0, 0, free_count, 0])
        self.kv_len = self.context if in_place else i32(np.full(B, -9))
        self.start, self.slot, self.pos = i32(np.full(B + 1, -9)), i32(np.full(max(tokens, 1), -9)), \
            i32(np.full(max(tokens, 1), -9))
        self.free_count = self.counts[2:3] if in_place else i32([free_count])
        self.struct = M.kv_batch(B, pages, P, self.width, tokens, row_tokens, self.context.data_ptr(),
                                 self.add.data_ptr(), self.table.data_ptr(), self.free.data_ptr(),
                                 self.free_count.data_ptr(), self.kv_len.data_ptr(), self.start.data_ptr(),
                                 self.slot.data_ptr(), self.pos.data_ptr(), self.counts.data_ptr())

    def host(self):
        h = {"table": self.table, "free": self.free, "kv_len": self.kv_len, "start": self.start,
             "slot": self.slot[:self.tokens], "pos": self.pos[:self.tokens], "counts": self.counts}
        h = {k: v.cpu().numpy().astype(np.int64) for k, v in h.items()}
        h["free"] = h["free"][:h["counts"][2]]
        return h


# ---- append -----------------------------------------------------------------------------------------

def rope(x, pos, cos_sin, rot):
    """x [T, H, D] fp64 -> rotated, and a bound of the fp32 arithmetic's error."""
    y = x.copy()
    err = np.zeros_like(x)
    if rot:
        h = rot // 2
        cs = cos_sin[pos].astype(np.float64)[:, None, :]
        c, s = cs[..., :h], cs[..., h:]
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * c - b * s, b * c + a * s
        err[..., :h] = np.abs(a * c) + np.abs(b * s)
        err[..., h:rot] = np.abs(b * c) + np.abs(a * s)
        err *= 3 * HALF["fp32"]
    return y, err


def bf16_bound(y, err):
    return err + HALF["bf16"] * (np.abs(y) + err) + 2.0 ** -134          # (half a step of the smallest bf16)


def e4m3_bound(y, err, scale):
    """Of the code's value against clamp(y / scale): the division's rounding, then half a step of e4m3 (2^-4 of the
    value, 2^-10 among its subnormals)."""
    v = np.clip(y / scale, -448, 448)
    d = err / scale + HALF["fp32"] * np.abs(y / scale)
    return v, d + 2.0 ** -4 * (np.abs(v) + d) + 2.0 ** -10


# ---- norms ------------------------------------------------------------------------------------------

def norm_reference(block, residual, post, pre, gate, kind, sigmoid, scale, offset, eps):
    """fp64 values of bf16 inputs -> (sum, bound), (normed, bound).  Relative errors: fp32 sums of squares (gamma(d)),
    the root, the product with a few roundings (2^-21 together), a sigmoid within 2^-19."""
    d = (block if block is not None else residual).shape[1]
    small = 2.0 ** -21 + (2.0 ** -19 if sigmoid else 0.0)
    s = err = 0.0
    if block is not None:
        u, ue = block, 0.0
        if post is not None:
            u = block / np.sqrt((block ** 2).mean(1, keepdims=True) + eps) * (offset + post)
            ue = gamma(d) + 2.0 ** -21
            # (the weight's own sum is rounded)
            ue = ue * np.abs(u) + HALF["fp32"] * np.abs(u)
        if kind != "none":
            g = 1 / (1 + np.exp(-gate)) if sigmoid else gate
            g = g[:, None] if kind == "token" else g
            u, ue = u * g, ue * np.abs(g)
        s, err = u, ue + small * np.abs(u)
    if residual is not None:
        r = scale * residual
        s = s + r
        err = err + 2 * HALF["fp32"] * (np.abs(r) + np.abs(s))
    n = nb = None
    if pre is not None:
        root = np.sqrt((s ** 2).mean(1, keepdims=True) + eps)
        n = s / root * (offset + pre)
        # the root's relative error: its own sums', and the sum's error by Cauchy and Schwarz
        es = np.sqrt((np.broadcast_to(err, s.shape) ** 2).mean(1, keepdims=True)) / root
        nb = (err / root) * np.abs(offset + pre) + np.abs(n) * (es + gamma(d) + 2.0 ** -20)
        nb = nb * 1.01 + 1e-37
        nb = nb + HALF["bf16"] * (np.abs(n) + nb)
    err = err * 1.01 + 1e-37
    return (s, err + HALF["bf16"] * (np.abs(s) + err)), (n, nb)


def stream():
    return torch.cuda.current_stream().cuda_stream
