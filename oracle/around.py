"""64-bit references of the calls around the layer (moe_add_rmsnorm,
moe_scaled_linear, moe_sample), in numpy on the host, from their definitions
in include/moe.h.  Tests only."""

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
SCALE_FLOOR = 448.0 * 2.0 ** -126


def e4m3_values():
    """Value of each of the 256 e4m3 codes (sign, 4 exponent bits with bias
    7, 3 mantissa bits; 0x7F and 0xFF are NaN, there is no infinity)."""
    c = np.arange(256)
    sign = np.where(c & 128, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return sign * v


E4M3 = e4m3_values()


def rms_norm(v, weight, eps):
    """n [T][H] of rows v (the stored residual), in 64 bits."""
    v = np.asarray(v, np.float64)
    inv = 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    return v * inv * np.asarray(weight, np.float64)


def block_scales(n):
    """One scale per row and block of 128 columns, in 64 bits."""
    T, H = n.shape
    nb = -(-H // BLOCK)
    pad = np.zeros((T, nb * BLOCK))
    pad[:, :H] = np.abs(n)
    return np.maximum(pad.reshape(T, nb, BLOCK).max(axis=2), SCALE_FLOOR) / E4M3_MAX


def scaled_linear(x8, x_scale, w8, w_scale):
    """(out, abs): the product of the codes' values with their scales, and
    the same sum of absolute values (what rounding errors scale with)."""
    x = E4M3[x8] * np.repeat(x_scale.astype(np.float64), BLOCK, axis=1)[:, :x8.shape[1]]
    w = E4M3[w8] * np.repeat(np.repeat(w_scale.astype(np.float64), BLOCK, axis=0)[:w8.shape[0]],
                             BLOCK, axis=1)[:, :w8.shape[1]]
    return x @ w.T, np.abs(x) @ np.abs(w.T)


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, slack) of one row.  slack: the distance, as a
    share of the kept mass, from the draw and from the top-p cut to the
    nearest border where another token would be taken."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if not top > -np.inf:
        return -1, 0.0, 1.0
    order = np.argsort(-x, kind="stable")
    if not temperature > 0:
        return int(order[0]), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.exp(np.where(x == -np.inf, -np.inf, (x - top) / temperature)))
    w = np.where(x == -np.inf, 0.0, w)
    w = w[order]
    keep = (x[order] > -np.inf) & ~(w < min_p)
    keep[0] = True
    w = w[keep]
    order = order[keep]
    if top_k > 0:
        w, order = w[:top_k], order[:top_k]
    slack = 1.0
    u = 0.0 if not u > 0 else min(u, 1.0)
    if top_p < 1:
        cum = np.cumsum(w)
        n = int((cum < top_p * cum[-1]).sum()) + 1
        slack = min(slack, float(np.abs(cum - top_p * cum[-1]).min() / cum[-1]))
        w, order = w[:n], order[:n]
    cum = np.cumsum(w)
    at = min(int((cum <= u * cum[-1]).sum()), len(w) - 1)
    slack = min(slack, float(np.abs(cum[:-1] - u * cum[-1]).min() / cum[-1]) if len(w) > 1 else 1.0)
    return int(order[at]), float(w[at] / cum[-1]), slack
