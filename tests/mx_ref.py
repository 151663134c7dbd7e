"""Plain 64-bit forms of the microscaled path, for the tests only (numpy).

MX rows: blocks of 32, scale byte s = max(127 + floor(log2 max|x|) - e_max, 0),
elements by search for the nearest value of the type (ties to the even code)."""
import numpy as np

E_MAX = {"fp4": 2, "fp8": 8}
FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FP8 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9)
                                            for m in range(8) if (e, m) != (8, 7)]
GRID = {"fp4": np.array(FP4), "fp8": np.array(FP8)}


def nearest(a, fmt):
    """Code (without sign) of the nearest value to |a|, ties to even."""
    g = GRID[fmt]
    mid = (g[1:] + g[:-1]) / 2
    lo = np.searchsorted(mid, np.abs(a), side="left")
    hi = np.searchsorted(mid, np.abs(a), side="right")
    return np.where(lo % 2 == 0, lo, hi)


def scale_bytes(m, fmt):
    """Scale byte of blocks whose largest magnitude is m (finite)."""
    _, e = np.frexp(m)
    return np.where(m > 0, np.maximum(127 + e - 1 - E_MAX[fmt], 0), 0).astype(np.int64)


def quantize(x, fmt):
    """(element codes with sign [rows, d], scale bytes [rows, d/32]) of x."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    fin = np.isfinite(b).all(-1)
    m = np.where(fin, np.abs(np.where(np.isfinite(b), b, 0)).max(-1), 0)
    s = np.where(fin, scale_bytes(m, fmt), 255)
    v = np.where(fin[..., None], b, 0.0) / np.ldexp(1.0, np.where(fin, s, 127) - 127)[..., None]
    c = nearest(v, fmt) | (np.signbit(v).astype(np.int64) << (3 if fmt == "fp4" else 7))
    return np.where(fin[..., None], c, 0).reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def pack(codes, fmt):
    return codes if fmt == "fp8" else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed, fmt):
    if fmt == "fp8":
        return packed
    return np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1)


def decode(codes, scales, fmt):
    """fp64 values of element codes (unpacked) and scale bytes."""
    n = len(GRID[fmt])
    top = 7 if fmt == "fp4" else 127
    g = np.append(GRID[fmt], [np.nan] * (top + 1 - n))
    v = g[codes & top] * np.where(codes > top, -1.0, 1.0)
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(v.shape[0], -1, 32) * f[..., None]).reshape(v.shape)


def rope(x, pos, axes, theta, half, inverse):
    """fp64 rotary embedding of x [tokens, heads, head_dim]."""
    y = np.array(x, np.float64)
    x = y.copy()
    turned, j = sum(axes), 0
    for a, size in enumerate(axes):
        for i in range(size // 2):
            t = pos[:, a].astype(np.longdouble) * np.longdouble(theta) ** (-np.longdouble(2 * i) / size)
            t = -t if inverse else t
            c, s = (np.asarray(f(t), np.float64)[:, None] for f in (np.cos, np.sin))
            u, v = (j, j + turned // 2) if half else (2 * j, 2 * j + 1)
            y[..., u], y[..., v] = x[..., u] * c - x[..., v] * s, x[..., u] * s + x[..., v] * c
            j += 1
    return y
