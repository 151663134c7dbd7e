"""Plain 64-bit forms of the cached-attention path, for the tests only (numpy)."""
import numpy as np

from tests import mx_ref

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(bf16):
    return 2.0 ** -8 if bf16 else U


def group_weights(q4, scales, zeros, group):
    """(weights, magnitudes |s| (|nibble - 8| + |8 - z|)) of packed nibbles [N, K/2]."""
    n = np.stack((q4 & 15, q4 >> 4), -1).reshape(q4.shape[0], -1).astype(np.float64)
    s = np.repeat(scales.astype(np.float64), group, 1)
    z = np.full_like(s, 8.0) if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)
    return s * (n - z), np.abs(s) * (np.abs(n - 8) + np.abs(8 - z))


def norm_rope(x, weight, eps, pos, axes, theta, half):
    """(values, magnitude of the pair that each is made of)."""
    x = np.asarray(x, np.longdouble)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.longdouble(np.float32(eps)))
    if weight is not None:
        n = n * weight
    n = n.astype(np.float64)
    mag, turned = np.abs(n), sum(axes)
    if half:
        s = mag[..., :turned // 2] + mag[..., turned // 2:turned]
        mag[..., :turned] = np.concatenate((s, s), -1)
    else:
        mag[..., :turned] = np.repeat(mag[..., 0:turned:2] + mag[..., 1:turned:2], 2, -1)
    return mx_ref.rope(n, pos, axes, theta, half, False), mag


def cache_values(codes, scales):
    """fp64 values of a cache's codes [pages, heads, page, hd / 2]; scale bytes from 253 are NaN."""
    p, h, n, nb = scales.shape
    s = np.where(scales >= 253, 255, scales)
    v = mx_ref.decode(mx_ref.unpack(codes.reshape(-1, 16 * nb), "fp4"), s.reshape(-1, nb), "fp4")
    return v.reshape(p, h, n, 32 * nb)


def rows_of(values, table, b, length):
    """[heads, length, hd] of sequence b; a page that is not there reads as NaN."""
    pages, heads, page, hd = values.shape
    out = np.full((heads, length, hd), np.nan)
    for at in range(0, length, page):
        p, n = table[b, at // page], min(page, length - at)
        if 0 <= p < pages:
            out[:, at:at + n] = values[p, :, :n]
    return out


def attention(q, k, v, scale, causal, window, bf16):
    """One sequence: q [n, q_heads, hd], k and v [kv_heads, length, hd] ->
    (out, its tolerance before the output's rounding, lse, its tolerance).

    With u = 2^-24, a score's error is |scale| sum |q k| (hd + 8) u (the products
    are exact in more than 32 bits or rounded once, hd sums, the scale), the
    argument of its exponential gains 4 u (|s| + |m|) by the change to base 2 and
    the difference from the maximum, the exponential 4 u: p is off by its sum e,
    relatively; with bf16 queries by half a step of bf16 more where it meets v.
    Sums over n tokens are off by n u of the sum of magnitudes, in any order.
    Weights p below 2^-126, the smallest normal number, may be flushed to zero, and so
    may their products with |v| <= 1: each token is off by 2^-126 (|v| + 1) more,
    which is all there is of an element whose large weights all meet zeros."""
    n, heads, hd = q.shape
    length, share = k.shape[1], heads // k.shape[0]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    lse, ltol = np.full((n, heads), -np.inf), np.zeros((n, heads))
    j = np.arange(length)
    for i in range(n):
        at = length - n + i
        seen = np.ones(length, bool)
        if causal:
            seen = j <= at
            if window:
                seen &= j > at - window
        if not seen.any():
            continue
        for h in range(heads):
            kk, vv = k[h // share][seen], v[h // share][seen]
            s = scale * (kk @ q[i, h])
            if np.isnan(s).any() or np.isnan(q[i, h]).any():
                out[i, h], lse[i, h] = np.nan, np.nan
                continue
            m = s.max()
            p = np.exp(s - m)
            total = p.sum()
            out[i, h] = p @ vv / total
            lse[i, h] = m + np.log(total)
            e = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])) * (hd + 8) * U + 4 * U * (np.abs(s) + abs(m)) + 4 * U
            e = e.max() + (len(s) + 8) * U
            mag = np.abs(np.nan_to_num(vv))
            tol[i, h] = p @ mag / total * (2 * e + (2.0 ** -8 if bf16 else 0.0)) + 2.0 ** -126 * (mag + 1).sum(0)
            ltol[i, h] = e + 4 * U * (abs(m) + abs(lse[i, h]))
    return out, tol, lse, ltol
