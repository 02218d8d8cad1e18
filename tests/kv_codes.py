"""Values and bounds that show whether attention took every step of a long request once."""
import numpy as np

from tests.resident_util import HALF, gamma

LONG = 20011


def positions_code(n, D, unit):
    """Values [n, D], 0 or 1: token t is 1 in the dimension of its unit of `unit` tokens, counted round."""
    v = np.zeros((n, D))
    v[np.arange(n), np.arange(n) // unit % D] = 1
    return v


def expected(v, scale=1.0):
    """The mean of the values and its bound.  All weights are 1 to their last bit, and sums of ones are exact in fp32 up to
    2^24 tokens, so there are the rounding of the quotient, of its product and of the scale (and 2^-126 a token), then
    bf16's."""
    n = len(v)
    assert n <= 1 << 24
    out = v.mean(0) * scale
    err = 4 * HALF["fp32"] * out + 2.0 ** -100
    return out, err + HALF["bf16"] * (out + err)


def lost(n, D, unit, step=32):
    """Steps whose absence, or presence twice, no output would show (none, for the sizes below)."""
    v = positions_code(n, D, unit)
    out, bound = expected(v)
    hidden = []
    for s in range(0, n, step):
        part = v[s:s + step]
        for sign, m in ((-1, n - len(part)), (1, n + len(part))):
            wrong = (v.sum(0) + sign * part.sum(0)) / m
            if (np.abs(wrong - out) <= bound).all():
                hidden.append((s, sign))
    return hidden


def long_row(q, k, v, scale, drop=None):
    """q [g, D], k, v [LONG, D] in fp64 -> out [g, D] and the bound of |kernel - out|, its bf16 rounding included; `drop`: a
    slice of tokens left out of out.

    As kv_util.attend_row, but with the roundings that the kernel's order of sums has.  626 steps of 32 tokens, two KV
    heads: 209 teams (256 for heads of 256), each of 6 steps (4) and up to 5 more where its cuts moved, over four waves (eight):
    at most 3 steps of a wave.  So a product passes 3 times 32 additions of either half of the weights and a rescale, 8
    of waves, two for each of the 8 parts of its run and two for each of at most 16 runs."""
    assert len(k) == LONG
    depth = 3 * (2 * 32 + 1) + 8 + 2 * 8 + 2 * 16
    keep = np.ones(LONG, bool)
    if drop is not None:
        keep[drop] = False
    s = scale * (q @ k.T)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    wk = w * keep
    total = wk.sum(1, keepdims=True)
    out = (wk @ v) / total
    u = HALF["fp32"]
    ds = abs(scale) * gamma(k.shape[1]) * (np.abs(q) @ np.abs(k).T) + 4 * u * (np.abs(s) + np.abs(s - m)) + 4 * u * np.abs(m)
    e = ds + 2.0 ** -21
    num = (w * (e + 2.0 ** -16 + gamma(depth))) @ np.abs(v) / total
    den = np.abs(out) * ((w * e).sum(1, keepdims=True) / total + gamma(depth))
    err = 1.05 * (num + den) + 2.0 ** -20 * np.abs(out)
    return out, err + HALF["bf16"] * (np.abs(out) + err) + 1e-37
