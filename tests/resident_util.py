"""Shared helpers of the resident-weight operator tests: records on the device, and the fp64 layer with a
rounding bound for every output."""
import numpy as np
import torch

import synth
from oracle import formats as OF, moe as OM, route as OR
from synth.configs import MoEConfig

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}        # a rounding is off by at most half a step


def config(fmt, d, f, E, k, seed=0):
    return MoEConfig("case", 9, layers=1, d=d, E=E, k=k, f=f, fmt=fmt, slots=1, bp_mbps=1, bh_mbps=1, seed=seed)


def padded(records, multiple=256):
    n, S = records.shape
    out = np.zeros((n, (S + multiple - 1) // multiple * multiple), np.uint8)
    out[:, :S] = records
    return out


def gamma(n):
    """Relative bound of a sum of n products in fp32, whatever its order (n 2^-24, and as much again for the
    matrix core's own rounding of partial products' sums)."""
    return 2 * (n + 8) * HALF["fp32"]


def ffn_bound(x, mats, lora=None, h_step=2.0 ** -16):
    """fp64 FFN of rows x and a bound of the kernel's error before its last rounding: fp32 sums, h kept to a
    relative `h_step`, exp and reciprocal within 2^-20.  `lora(name, v)` -> (term, bound of its error, and the
    product of absolute values)."""
    Wg, Wu, Wd = mats
    g, u = x @ Wg, x @ Wu
    dg, du = gamma(len(Wg)) * (np.abs(x) @ np.abs(Wg)), gamma(len(Wu)) * (np.abs(x) @ np.abs(Wu))
    if lora is not None:
        for name, v, dv in (("gate", g, dg), ("up", u, du)):
            t, b = lora(name, x, 0.0)
            v += t
            dv += b
    with np.errstate(over="ignore"):
        h = OM.silu(g) * u
    s = np.abs(OM.silu(g))
    dh = 1.1 * dg * (np.abs(u) + du) + s * du + (h_step + 2.0 ** -19) * np.abs(h)
    y = h @ Wd
    dy = dh @ np.abs(Wd) + gamma(len(Wd)) * ((np.abs(h) + dh) @ np.abs(Wd))
    if lora is not None:
        t, b = lora("down", h, dh)
        y += t
        dy += b
    return y, dy


def layer_with_bound(x_bf16, wr, records, cfg, base=None):
    """ids, w, y [T x d] of the layer in fp64, and the bound of |kernel - y| (its bf16 rounding included)."""
    ids, w, gap = OR.route(x_bf16, wr, cfg.k)
    x = OF.bf16_to_f64(x_bf16)
    T, k = ids.shape
    w64 = w.astype(np.float64)
    y = np.zeros((T, cfg.d))
    dy = np.zeros((T, cfg.d))
    mag = np.zeros((T, cfg.d))
    for e in np.unique(ids):
        tt, jj = np.nonzero(ids == e)
        v, dv = ffn_bound(x[tt], OF.decode_record(records[e], cfg.fmt, cfg.d, cfg.f))
        y[tt] += w64[tt, jj][:, None] * v
        dy[tt] += w64[tt, jj][:, None] * (dv + 1e-6 * np.abs(v))
        mag[tt] += w64[tt, jj][:, None] * np.abs(v)
    if base is not None:
        y += OF.bf16_to_f64(base)
        mag += np.abs(OF.bf16_to_f64(base))
    dy += gamma(k + 8) * mag
    return ids, w, y, dy + HALF["bf16"] * (np.abs(y) + dy), gap


def assert_within(got, ref, bound, what=""):
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    over = err - bound
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what}: at {i}: got {got[i]}, want {ref[i]} within {bound[i]:.3e}, off by {err[i]:.3e}"


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


class Pool:
    """A random adapter pool of a projection [n x K]: mixed ranks (none, one, odd ones, the whole), and garbage
    (NaN) past an adapter's ranks, as a slot that an earlier adapter used may hold."""

    def __init__(self, count, max_rank, K, n, seed, ranks=None, garbage=True):
        rng = np.random.default_rng([seed, K, n])
        odd = [max_rank, 1, 0, max_rank - 1, max(1, max_rank // 2 + 1), 16]
        self.rank = np.array([odd[i % len(odd)] for i in range(count)] if ranks is None else ranks, np.int32)
        self.scale = rng.uniform(-2, 2, count).astype(np.float32)
        self.a = synth.f32_to_bf16(0.05 * rng.standard_normal((count, max_rank, K)))
        self.b = synth.f32_to_bf16(0.05 * rng.standard_normal((count, n, max_rank)))
        if garbage:
            for i, r in enumerate(self.rank):
                r = min(max(r, 0), max_rank)
                self.a[i, r:] = 0x7FC0
                self.b[i, :, r:] = 0xFF80
        self.count, self.max_rank = count, max_rank

    def device(self):
        from moe_expert_execution_amd.tensors import LoraPool
        from tests.gpu_util import dev
        return LoraPool(dev(self.a.view(np.int16)).view(torch.bfloat16), dev(self.b.view(np.int16)).view(torch.bfloat16),
                        dev(self.rank), dev(self.scale))

    def term(self, x, dx, ids):
        """s_a (x A_a) B_a of rows x (fp64) and a bound of the kernel's error, given one of x's."""
        n = self.b.shape[1]
        y, dy = np.zeros((len(x), n)), np.zeros((len(x), n))
        dx = np.broadcast_to(dx, x.shape)
        for a in np.unique(ids):
            if a < 0 or a >= self.count:
                continue
            r = min(max(int(self.rank[a]), 0), self.max_rank)
            if r == 0:
                continue
            t = ids == a
            A, B = OF.bf16_to_f64(self.a[a, :r]).T, OF.bf16_to_f64(self.b[a, :, :r]).T
            s = float(self.scale[a])
            v = s * (x[t] @ A)
            dv = abs(s) * ((dx[t] + gamma(len(A)) * (np.abs(x[t]) + dx[t])) @ np.abs(A)) + 2.0 ** -16 * np.abs(v)
            y[t] = v @ B
            dy[t] = dv @ np.abs(B) + gamma(r) * ((np.abs(v) + dv) @ np.abs(B))
        return y, dy


def final_bound(y, dy, base=None):
    """The bound with the addend and the bf16 rounding of y."""
    if base is not None:
        y = y + OF.bf16_to_f64(base)
    dy = dy + 2.0 ** -20 * (np.abs(y) + dy)
    return y, dy + HALF["bf16"] * (np.abs(y) + dy)


def project_with_bound(x_bf16, W, pool, ids, base=None):
    """W: fp64 [K x n]."""
    x = OF.bf16_to_f64(x_bf16)
    y, dy = x @ W, gamma(len(W)) * (np.abs(x) @ np.abs(W))
    if pool is not None:
        t, b = pool.term(x, 0.0, ids)
        y, dy = y + t, dy + b
    return final_bound(y, dy, base)


def expert_with_bound(x_bf16, mats, pools, ids, base=None):
    """pools: gate, up, down (or None each).  Up to 64 tokens h keeps 16 bits, above that bf16's 8."""
    def lora(name, v, dv):
        p = pools[("gate", "up", "down").index(name)]
        return p.term(v, dv, ids) if p is not None else (0.0, 0.0)

    y, dy = ffn_bound(OF.bf16_to_f64(x_bf16), mats, lora, 2.0 ** -16 if len(x_bf16) <= 64 else HALF["bf16"])
    return final_bound(y, dy, base)


def mixed_ids(T, count, seed, run=1):
    """Adapters of T tokens in runs of up to `run`, none (-1) and ids outside the pool among them."""
    rng = np.random.default_rng([seed, T, count])
    ids = np.empty(0, np.int32)
    while len(ids) < T:
        a = rng.integers(-1, count + 1)
        a = {-1: int(rng.choice([-1, -2 ** 31])), count: int(rng.choice([count, 2 ** 31 - 1]))}.get(int(a), int(a))
        ids = np.concatenate([ids, np.full(rng.integers(1, run + 1), a, np.int32)])
    return ids[:T]
