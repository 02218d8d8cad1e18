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
