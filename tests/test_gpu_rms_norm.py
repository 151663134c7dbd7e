"""Residual sum, RMS norm and modulation on the GPU against a plain 64-bit
form.

Tolerances, with u = 2^-24 (half an fp32 step).  h has one rounding of gate x
and one of the sum: dh = u (|g x| + |h|).  The mean of squares has at most
log2(16384) + 24 roundings on any path, the root and the products of y at most
10 more: a relative 40 u of y - shift, plus dh through the norm (twice: the
element's own and, at most as large, the row's), plus u |y| for the shift.
A stored bf16 value adds 2^-8 of itself, an fp32 one u.  Codes: the value they
stand for is nearest to some y within the tolerance above, under a scale of a
maximum within it."""
import numpy as np
import pytest

from tests import mx_ref as ref
from tests.gpu_util import bf16_to_np, host, say, to_device
import workloads as wl

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import torch
    import quantization_dit_linear_amd as q
    assert torch.cuda.is_available()
    q.lib()
    return q


def _round(x, bf16):
    x = np.asarray(x, np.float32)
    return wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(x)) if bf16 else x


def _dev(x, bf16):
    if x is None:
        return None
    return to_device(np.ascontiguousarray(wl.f32_to_bf16_bits(x) if bf16 else x))


def _np(t):
    import torch
    return bf16_to_np(t) if t.dtype == torch.bfloat16 else host(t).astype(np.float64)


def _inputs(rows, d, seed, bf16, pbf16, residual, weight, gate, mod, groups):
    r = np.random.default_rng([seed, 8])
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    c = {"x": _round(n(rows, d), bf16), "residual": None, "weight": None, "gate": None,
         "scale": None, "shift": None}
    if residual:
        v = n(rows, d) * np.exp(n(rows, 1))
        v[:, r.integers(0, d)] *= 40
        v[2::7] = 0
        c["x"][2::7] = 0
        c["residual"] = _round(v, bf16)
    if weight:
        c["weight"] = _round(1 + 0.1 * n(d), pbf16)
    m = _round(0.3 * n(groups, 6 * d), pbf16)
    if gate:
        c["gate"] = m[:, 2 * d:3 * d]
    if mod:
        c["scale"], c["shift"] = m[:, d:2 * d], m[:, :d]
    c["mod"] = m
    return c


def _want(c, per, eps):
    x = c["x"].astype(np.float64)
    row = np.arange(len(x)) // per
    gx = x * c["gate"].astype(np.float64)[row] if c["gate"] is not None else x
    h = gx + c["residual"] if c["residual"] is not None else gx
    dh = U * (np.abs(gx) + np.abs(h))
    k = np.ones_like(h)
    if c["weight"] is not None:
        k = k * c["weight"]
    if c["scale"] is not None:
        k = k * (1 + c["scale"].astype(np.float64)[row])
    inv = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    z = h * inv * k
    y = z + c["shift"].astype(np.float64)[row] if c["shift"] is not None else z
    dy = 2 * np.abs(k) * inv * dh.max(1, keepdims=True) + 40 * U * np.abs(z) + U * np.abs(y)
    return h, dh, y, dy


def _call(q, c, bf16, pbf16, per, eps, fmt=None, **kw):
    d = c["x"].shape[1]
    m = _dev(c["mod"], pbf16)
    part = lambda n, i: None if c[n] is None else m[:, i * d:(i + 1) * d]  # noqa: E731
    return q.add_rms_norm(_dev(c["x"], bf16), _dev(c["residual"], bf16),
                          weight=_dev(c["weight"], pbf16), gate=part("gate", 2),
                          scale=part("scale", 1), shift=part("shift", 0), rows_per_mod=per,
                          eps=eps, fmt=fmt, **kw)


def _check(q, rows, d, bf16, pbf16, fmt, groups=1, residual=True, weight=True, gate=False,
           mod=False, eps=1e-6):
    c = _inputs(rows, d, rows + d, bf16, pbf16, residual, weight, gate, mod, groups)
    per = -(-rows // groups)
    h, dh, y, dy = _want(c, per, eps)
    step = 2.0 ** -8 if bf16 else U
    got = _call(q, c, bf16, pbf16, per, eps, fmt)
    assert np.all(np.abs(_np(got[0]) - h) <= dh + step * (np.abs(h) + dh))
    if fmt is None:
        err, tol = np.abs(_np(got[1]) - y), dy + step * (np.abs(y) + dy) + 1e-45
        assert np.all(err <= tol), float(np.max(err / tol))
        return
    codes, s = ref.unpack(host(got[1]), fmt), host(got[2])
    yb, db = y.reshape(rows, -1, 32), dy.reshape(rows, -1, 32)
    big, slack = np.abs(yb).max(-1), db.max(-1)
    lo, hi = ref.scale_bytes(np.maximum(big - slack, 0), fmt), ref.scale_bytes(big + slack, fmt)
    assert np.all((lo <= s) & (s <= hi))
    unit = np.ldexp(1.0, s.astype(np.int64) - 127)[..., None]
    near = ref.GRID[fmt][ref.nearest(yb / unit, fmt)] * unit
    off = np.abs(ref.decode(codes, s, fmt).reshape(yb.shape) - yb)
    assert np.all(off <= np.abs(near - np.abs(yb)) + 2 * db)


SHAPES = [(1, 32), (1, 5120), (2, 64), (5, 96), (9, 2048), (33, 1568), (3, 2080), (4, 4096),
          (7, 5120), (2, 8224), (3, 16384), (700, 288)]


@pytest.mark.parametrize("fmt", [None, "fp8", "fp4"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_residual_and_weight(q, rows, d, bf16, fmt):
    say("rms norm", rows, d, bf16, fmt)
    _check(q, rows, d, bf16, bf16, fmt)


@pytest.mark.parametrize("fmt", [None, "fp8"])
@pytest.mark.parametrize("bf16,pbf16", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("rows,d,groups", [(1, 64, 1), (7, 160, 3), (10, 5120, 2), (65, 1024, 4),
                                           (3, 12288, 2), (2051, 512, 5)])
def test_gate_and_modulation(q, rows, d, groups, bf16, pbf16, fmt):
    """Slices of one [groups, 6 d] projection as they lie; the last group short."""
    say("rms norm mod", rows, d, groups, bf16, pbf16, fmt)
    _check(q, rows, d, bf16, pbf16, fmt, groups=groups, gate=True, mod=True)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,d,groups", [(1, 64, 1), (7, 160, 3), (10, 5120, 2), (3, 12288, 2), (515, 512, 5)])
def test_gate_and_modulation_into_four_bits(q, rows, d, groups, bf16):
    say("rms norm mod fp4", rows, d, groups, bf16)
    _check(q, rows, d, bf16, bf16, "fp4", groups=groups, gate=True, mod=True)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("gate,mod", [(False, False), (True, False), (False, True)])
def test_every_part_is_optional(q, residual, weight, gate, mod):
    say("rms norm parts", residual, weight, gate, mod)
    _check(q, 11, 352, True, True, None, groups=2, residual=residual, weight=weight, gate=gate,
           mod=mod)


@pytest.mark.parametrize("d", [96, 5120])
def test_single_parts_of_the_modulation(q, d):
    import torch
    x = torch.randn((5, d), device="cuda")
    p = torch.randn((5, d), device="cuda")
    _, plain = q.add_rms_norm(x)
    _, scaled = q.add_rms_norm(x, scale=p, rows_per_mod=1)
    _, shifted = q.add_rms_norm(x, shift=p, rows_per_mod=1)
    torch.testing.assert_close(scaled.double(), plain.double() * (1 + p.double()), rtol=4 * U, atol=0)
    torch.testing.assert_close(shifted.double(), plain.double() + p.double(), rtol=4 * U, atol=4e-7)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("d", [64, 5120, 16384])
def test_in_place_and_without_the_sum(q, d, bf16):
    import torch
    say("rms norm in place", d, bf16)
    t = torch.bfloat16 if bf16 else torch.float32
    x, r, w = (torch.randn(s, device="cuda").to(t) for s in ((37, d), (37, d), (d,)))
    h, y = q.add_rms_norm(x, r, weight=w)
    none, y2 = q.add_rms_norm(x, r, weight=w, sum_out=False)
    assert none is None
    torch.testing.assert_close(y2, y, rtol=0, atol=0)
    a, b = x.clone(), r.clone()
    h2, y3 = q.add_rms_norm(a, b, weight=w, sum_out=b, out=a)  # the stream's sum in the residual
    assert h2 is b and y3 is a
    torch.testing.assert_close(b, h, rtol=0, atol=0)
    torch.testing.assert_close(a, y, rtol=0, atol=0)
    a, b = x.clone(), r.clone()
    q.add_rms_norm(a, b, weight=w, sum_out=a, out=b)
    torch.testing.assert_close(a, h, rtol=0, atol=0)
    torch.testing.assert_close(b, y, rtol=0, atol=0)


@pytest.mark.parametrize("d", [128, 2048, 5120])
def test_zero_huge_and_non_finite_rows(q, d):
    """A zero row gives zeros, a row whose squares overflow fp32 its norm, and
    a row with a NaN or an infinity nothing to its neighbours."""
    import torch
    say("rms norm extremes", d)
    x = torch.randn((9, d), device="cuda")
    base = q.add_rms_norm(x)[1]
    y0 = x.clone()
    y0[1] = 0
    y0[3] *= 2.0 ** 90
    y0[5, 7] = float("nan")
    y0[7, d - 1] = float("inf")
    _, y = q.add_rms_norm(y0)
    assert bool((y[1] == 0).all())
    want = (y0[3].double() / y0[3].double().square().mean().sqrt())
    torch.testing.assert_close(y[3].double(), want, rtol=50 * U, atol=0)
    assert bool(y[5].isnan().all())
    assert bool(y[7, d - 1].isnan()) and bool((y[7, :d - 1] == 0).all())
    for k in (0, 2, 4, 6, 8):
        torch.testing.assert_close(y[k], base[k], rtol=0, atol=0)
    _, codes, scales = q.add_rms_norm(y0, fmt="fp8")
    assert bool((scales[5] == 255).all()) and bool((scales[7, -1] == 255).all())
    assert bool((scales[1] == 0).all()) and bool((codes[1] == 0).all())
    _, c2, s2 = q.add_rms_norm(x, fmt="fp8")
    for k in (0, 2, 4, 6, 8):
        assert torch.equal(codes[k], c2[k]) and torch.equal(scales[k], s2[k])


@pytest.mark.parametrize("eps", [1e30, 3e38])
@pytest.mark.parametrize("d", [128, 2048, 5120, 16384])
def test_the_largest_eps(q, d, eps):
    """Rows whose sum of squares, or whose mean with eps, passes fp32's range,
    beside ordinary ones: eps counts in each.  40 roundings as above."""
    say("rms norm eps", d, eps)
    r = np.random.default_rng([d, 12])
    x = (r.standard_normal((6, d)) * np.array([1.0, 1e15, 1e18, 4e18, 2e19, 1e25])[:, None]).astype(np.float32)
    x[4] = 1.8e19  # its sum of squares overflows, its mean is 3.2e38
    e = float(np.float32(eps))
    _, y = q.add_rms_norm(_dev(x, False), eps=eps)
    v = x.astype(np.float64)
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + e)
    assert np.all(np.abs(_np(y) - want) <= 40 * U * np.abs(want))


@pytest.mark.parametrize("mod", [False, True])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("d", [32, 128, 2048, 5120, 8192, 16384])
def test_rows_of_the_largest_values(q, d, bf16, mod):
    """Finite rows up to the type's largest value, whose norm passes 2^128,
    beside ordinary ones: the formula's values, also in codes.  The tolerance
    above, and where y is subnormal half of the type's smallest step (the
    normalised value's 2^-150 times at most 8 of weight and scale)."""
    say("rms norm largest", d, bf16, mod)
    top = 3.3895313892515355e38 if bf16 else 3.4028234663852886e38
    c = _inputs(9, d, d, bf16, bf16, mod, mod, mod, mod, 3)
    r = np.random.default_rng([d, 15])
    sign = r.choice([-1.0, 1.0], (9, d))
    x = c["x"].astype(np.float64)
    x[1] = sign[1] * top
    x[2] = sign[2] * r.uniform(3e36, 3e38, d)
    x[3, d // 2] = top
    x[4] = sign[4] * np.exp2(r.uniform(-100, 127, d))
    x[6] = sign[6] * 2.0 ** 116
    x[7] = sign[7] * 2.0 ** 121
    np.clip(c["mod"], -0.875, 0.875, out=c["mod"])  # gate x stays finite (gate, scale and shift are views)
    c["x"] = _round(x, bf16)
    assert np.isfinite(c["x"]).all()
    h, dh, y, dy = _want(c, 3, 1e-6)
    _, got = _call(q, c, bf16, bf16, 3, 1e-6)
    err = np.abs(_np(got) - y)
    tol = dy + (2.0 ** -8 if bf16 else U) * (np.abs(y) + dy) + 2.0 ** -147 + (2.0 ** -134 if bf16 else 0.0)
    assert np.all(err <= tol), (float(np.max(err / tol)), np.argwhere(err > tol)[:4])
    if not bf16:
        for fmt in ("fp8", "fp4"):
            _, codes, scales = _call(q, c, bf16, bf16, 3, 1e-6, fmt)
            want = q.mx_quantize(got, fmt)
            assert bool((codes == want[0]).all()) and bool((scales == want[1]).all())


def test_rows_do_not_depend_on_the_batch(q):
    """Row r alone gives the bits that it has in a batch."""
    import torch
    for d in (320, 5120):
        x, r = (torch.randn((1025, d), device="cuda").bfloat16() for _ in range(2))
        h, y = q.add_rms_norm(x, r)
        for k in (0, 1, 511, 1024):
            h1, y1 = q.add_rms_norm(x[k:k + 1], r[k:k + 1])
            assert torch.equal(h1[0], h[k]) and torch.equal(y1[0], y[k])


def test_offsets_beyond_32_bits(q):
    import torch
    rows, d = 262200, 16384
    say("rms norm far offsets", rows, d)
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    x[-5:].normal_()
    want = q.add_rms_norm(x[-5:].clone(), x[-5:].clone(), fmt="fp4")
    h, codes, scales = q.add_rms_norm(x, x, sum_out=x, fmt="fp4")
    assert h is x and torch.equal(h[-5:], want[0])
    assert torch.equal(codes[-5:], want[1]) and torch.equal(scales[-5:], want[2])
    assert bool((codes[:-5] == 0).all())


@pytest.mark.parametrize("d,per", [(32, 4), (2080, 2), (5152, 1)])
def test_more_rows_than_the_grid(q, d, per):
    """2^20 workgroups of one, two or four rows and more: some of them walk on
    to another row, also where a row's mean has overflowed."""
    import torch
    rows = per * 2 ** 20 + 1025
    say("rms norm walk", rows, d)
    x = torch.randn((rows, d), device="cuda", dtype=torch.bfloat16)
    for k in (1, per * 2 ** 20 - 2, per * 2 ** 20 + 2, rows - 2):
        x[k] *= 2.0 ** 120
    parts = [slice(0, 9), slice(per * 2 ** 20 - 7, per * 2 ** 20 + 9), slice(rows - 9, rows)]
    want = [q.add_rms_norm(x[s].clone(), sum_out=False)[1] for s in parts]
    q.add_rms_norm(x, sum_out=False, out=x)
    for s, w in zip(parts, want):
        assert torch.equal(x[s], w) and bool((w.double().square().mean(1) - 1).abs().max() < 0.02)


def test_empty(q):
    import torch
    h, y = q.add_rms_norm(torch.zeros((0, 64), device="cuda"))
    assert h.shape == y.shape == (0, 64)
