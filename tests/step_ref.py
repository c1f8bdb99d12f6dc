"""Plain references of a step's two ends, written from include/kvq.h: norm, rotation and transform of a row in
float64 with phases in Python integers, and a row of logits to probabilities token by token."""

from __future__ import annotations

import math

import numpy as np

MOST = 32767


# ---- rotary positions ---------------------------------------------------------------------------
def frequencies(rot, theta, kind="plain", factor=1.0, context=0.0, a=0.0, b=0.0):
    """Radians per token of every pair, and the factor of the rotated channels."""
    out = []
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        if kind == "linear":
            w = w / factor
        elif kind == "bands":
            turns = context * w / (2 * math.pi)          # in the original context
            if turns < a:
                w = w / factor
            elif turns <= b:
                s = (turns - a) / (b - a)
                w = (1 - s) * w / factor + s * w
        elif kind == "yarn":
            at = lambda t: rot * math.log(context / (t * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(math.floor(at(a)), 0), min(math.ceil(at(b)), rot - 1)
            ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = w / factor * ramp + w * (1 - ramp)
        out.append(w)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if kind == "yarn" and factor > 1 else 1.0)


def phases(freq, pos):
    """Angles in radians from the phases that the library keeps: freq, pos whole numbers."""
    f = [int(x) & (2**64 - 1) for x in freq]
    return np.array([[(int(p) * x % 2**64) / 2**64 * 2 * math.pi for x in f] for p in pos])


def placed(x, angle, interleaved, scale=1.0, w=None, eps=0.0):
    """Rows x [n, H, 128] float64 after norm and rotation by angle [n, rot / 2], and each channel's pair length."""
    y = np.array(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    m = np.abs(y)
    half = angle.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
    ya, yb = y[..., a], y[..., b]
    length = np.hypot(ya, yb) * scale
    out = y.copy()
    out[..., a], out[..., b] = ya * c - yb * s, yb * c + ya * s
    m[..., a] = m[..., b] = length
    return out, m


def hadamard():
    h = np.ones((1, 1))
    while len(h) < 128:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(128)


def transformed(y, m, mats, gqa):
    """(rows, bound): T y per head, and sum_j |T_ij| m_j; mats [Hkv, 128, 128]."""
    out, bound = np.empty_like(y), np.empty_like(y)
    for h in range(y.shape[1]):
        t = np.asarray(mats[h // gqa], np.float64)
        out[:, h], bound[:, h] = y[:, h] @ t.T, m[:, h] @ np.abs(t).T
    return out, bound


def near(got, want, bound):
    """got: bf16 values as float64.  Half a step of bf16 and the arithmetic's share."""
    return np.abs(got - want) <= 2.0**-8 * np.abs(want) * (1 + 2.0**-8) + 2.0**-17 * bound + 2.0**-133


# ---- logits ---------------------------------------------------------------------------------------
def values(logits, counts, above, rules, b, allowed):
    """One row's values before the softmax, float64, and the magnitudes that its roundings go by."""
    x = np.asarray(logits, np.float64).copy()
    size = np.where(np.isfinite(x), np.abs(x), 0.0)
    for t, v in rules.get("bias", {}).get(b, {}).items():
        x[t] += v
        if np.isfinite(v):
            size[t] += abs(v)
    c = np.zeros(len(x), np.int64) if counts is None else np.asarray(counts, np.int64) & 0xffff
    times, held = c & MOST, c != 0
    for t in above:
        times[t] += 1
        held[t] = True
    pick = lambda name, d: d if rules.get(name) is None else float(rules[name][b])  # noqa: E731
    r, f, a = pick("repetition", 1.0), pick("frequency", 0.0), pick("presence", 0.0)
    with np.errstate(invalid="ignore"):
        x = np.where(held, np.where(x > 0, x / r, x * r), x)
    size = np.where(held, size * max(r, 1 / r), size)
    x = x - f * times - a * (times > 0)
    size = size + abs(f) * times + abs(a) * (times > 0)
    if allowed is not None:
        x = np.where(allowed, x, -np.inf)
        size = np.where(allowed, size, 0.0)
    return x, size


def probabilities(x, size, heat):
    """(p, tolerance) of one row.

    Five roundings of 2^-24 lie between a logit and its value, each relative to at most the magnitudes in `size`; the
    difference to the maximum, the product with log2(e) / T and that factor add three more, relative to the
    difference; so the exponents are off by 8 * 2^-24 * 2 max(size) / T = 2^-20 max(size) / T at most, in the token and in
    the sum.  The exponential, the sums (a tree over slices, at most 2^6 additions in a row at these sizes) and the last product: 2^-17."""
    if heat == 0:
        p = np.zeros(len(x))
        p[int(np.argmax(x))] = 1.0
        return p, np.zeros(len(x))
    top = x.max()
    with np.errstate(over="ignore"):
        e = np.exp((x - top) / heat)
    p = e / e.sum()
    share = 2.0**-17 + 2 * 2.0**-20 * (size.max() + abs(top)) / heat
    return p, np.where(p > 0, p, 0.0) * min(share, 1e9) + 2.0**-120
