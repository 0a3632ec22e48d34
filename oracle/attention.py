"""64-bit references of moe_rope_append, moe_rope_frequencies and
moe_paged_attention, in numpy on the host, from their definitions in
include/moe.h.  Tests only."""

import math

import numpy as np

E4M3_MAX = 448.0
SCALE_FLOOR = 448.0 * 2.0 ** -126


def frequencies(R, theta, scaling="plain", factor=1.0, context=0, fast=32.0, slow=1.0):
    """(freq, rot_scale), pair by pair."""
    out = []
    for j in range(R // 2):
        f = theta ** (-2 * j / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "base":
            f = (theta * factor ** (R / (R - 2))) ** (-2 * j / R)
        elif scaling == "bands":
            def d(turns):
                return R * math.log(context / (2 * math.pi * turns)) / (2 * math.log(theta))
            lo, hi = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), R - 1)
            w = min(max((j - lo) / max(hi - lo, 0.001), 0), 1)
            f = f * (1 - w) + f / factor * w
        out.append(f)
    return np.array(out), 0.1 * math.log(factor) + 1 if scaling == "bands" else 1.0


def rotate(a, pos, freq, rot_scale, interleaved):
    """Rows a [n][D] of tokens at positions pos [n]; and what rounding errors
    scale with: the sum of both columns' magnitudes."""
    a = np.asarray(a, np.float64)
    out, mag = a.copy(), np.abs(a)
    half = len(freq)
    one = np.arange(half) * 2 if interleaved else np.arange(half)
    two = one + (1 if interleaved else half)
    angle = np.asarray(pos, np.float64)[:, None] * freq
    c, s = np.cos(angle) * rot_scale, np.sin(angle) * rot_scale
    out[:, one] = a[:, one] * c - a[:, two] * s
    out[:, two] = a[:, two] * c + a[:, one] * s
    mag[:, one] = mag[:, two] = (np.abs(a[:, one]) + np.abs(a[:, two])) * max(abs(rot_scale), 1)
    return out, mag


def head_norm(a, weight, eps):
    a = np.asarray(a, np.float64)
    if weight is None:
        return a
    return a / np.sqrt(np.mean(a * a, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def attend(q, k, v, pos, seen, scale, window=0):
    """One sequence: q [n][Hq][D] at positions pos [n], k and v [L][Hkv][D],
    seen [L]: positions that are there.  Returns out [n][Hq][D], and what its
    errors scale with: the weighted means of |v - out| and |v|, and per row
    the largest scale * sum |q k| [n][Hq][1]."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    at = np.arange(k.shape[0])
    out, spread, level, mag = (np.zeros((n, Hq, w)) for w in (D, D, D, 1))
    for i in range(n):
        keep = seen & (at <= pos[i])
        if window:
            keep &= at > pos[i] - window
        if not keep.any():
            continue
        for h in range(Hq):
            kk, vv = k[keep, h // G], v[keep, h // G]
            s = (kk @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv
            spread[i, h] = w @ np.abs(vv - out[i, h])
            level[i, h] = w @ np.abs(vv)
            mag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, spread, level, mag
