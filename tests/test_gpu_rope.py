"""Rotary embedding with several axes on the GPU against a plain form (angles
in extended precision).

Tolerance, u = 2^-24: the angle is exact to 2^-30 of a turn (its fixed-point
rate's rounding at a position of 2^31, and the fraction kept); as an fp32 angle
of at most half a turn and in sine and cosine it gains at most 2^-22; the
products and the sum three roundings.  All are of |u| + |v| at most: 2^-21
together, and the stored type's half step."""
import numpy as np
import pytest

from tests import mx_ref as ref
from tests.gpu_util import bf16_to_np, host, say, to_device
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    import quantization_dit_linear_amd as q
    assert torch.cuda.is_available()
    q.lib()
    return q


def _np(t):
    import torch
    return bf16_to_np(t) if t.dtype == torch.bfloat16 else host(t).astype(np.float64)


def _x(shape, seed, bf16):
    v = np.random.default_rng([seed, 4]).standard_normal(shape).astype(np.float32)
    return wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(v)) if bf16 else v


def _check(got, x, pos, axes, theta, half, inverse, bf16):
    want = ref.rope(x, pos, axes, theta, half, inverse)
    turned, mag = sum(axes), np.zeros(x.shape)
    a = np.abs(x.astype(np.float64))
    if half:
        s = a[..., :turned // 2] + a[..., turned // 2:turned]
        mag[..., :turned] = np.concatenate((s, s), -1)
    else:
        mag[..., :turned] = np.repeat(a[..., 0:turned:2] + a[..., 1:turned:2], 2, -1)
    tol = 2.0 ** -21 * mag + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(want) + 2.0 ** -21 * mag)
    err = np.abs(got - want)
    assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-30)))
    np.testing.assert_array_equal(got[..., turned:], x[..., turned:])


CASES = [(1, 1, 8, [8]), (1, 80, 128, [44, 42, 42]), (3, 5, 64, [20, 22, 22]),
         (257, 3, 72, [24, 24, 24]), (64, 24, 128, [16, 56, 56]), (1000, 2, 96, [96]),
         (33, 7, 256, [64, 64, 64, 64]), (5, 4, 512, [200, 156, 156]), (19, 6, 80, [10, 0, 22]),
         (2, 3, 64, [0, 0, 0]), (4097, 1, 16, [2, 4, 10])]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("tokens,heads,hd,axes", CASES)
def test_interleaved(q, tokens, heads, hd, axes, inverse, bf16):
    say("rope", tokens, heads, hd, axes, inverse, bf16)
    x = _x((tokens, heads, hd), tokens + hd, bf16)
    pos = np.random.default_rng(tokens).integers(-50, 4000, (tokens, len(axes))).astype(np.int32)
    import torch
    got = q.rope(to_device(wl.f32_to_bf16_bits(x) if bf16 else x), torch.from_numpy(pos).cuda(),
                 axes, inverse=inverse)
    _check(_np(got), x, pos, axes, 10000.0, False, inverse, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("tokens,heads,hd,axes",
                         [c for c in CASES if sum(c[3]) % 16 == 0 and c[2] > 8] + [(7, 3, 72, [32, 16, 16])])
def test_half_split(q, tokens, heads, hd, axes, inverse, bf16):
    say("rope half", tokens, heads, hd, axes, inverse, bf16)
    x = _x((tokens, heads, hd), tokens + hd, bf16)
    pos = np.random.default_rng(tokens).integers(-50, 4000, (tokens, len(axes))).astype(np.int32)
    import torch
    got = q.rope(to_device(wl.f32_to_bf16_bits(x) if bf16 else x), torch.from_numpy(pos).cuda(),
                 axes, half=True, inverse=inverse)
    _check(_np(got), x, pos, axes, 10000.0, True, inverse, bf16)


@pytest.mark.parametrize("theta", [1.0, 500.0, 10000.0, 1e6, 1e12])
def test_far_positions(q, theta):
    """Positions up to the ends of int32: the angle keeps its exactness."""
    import torch
    say("rope far", theta)
    pos = np.array([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], np.int32)
    pos = np.stack((pos, pos[::-1], np.roll(pos, 3)), 1)
    x = _x((8, 3, 96), 5, False)
    got = q.rope(to_device(x), torch.from_numpy(pos).cuda(), [32, 32, 32], theta=theta)
    _check(_np(got), x, pos, [32, 32, 32], theta, False, False, False)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_slices_of_a_fused_projection(q, half, bf16):
    """q|k read inside [tokens, 3 heads hd]; in place; values and padding
    rows behind the last token untouched; heads-first output."""
    import torch
    say("rope strided", half, bf16)
    T, H, D, axes = 45, 6, 64, [16, 24, 24]
    t = torch.bfloat16 if bf16 else torch.float32
    qkv = torch.randn((T + 3, 3 * H * D), device="cuda").to(t)
    pos = torch.randint(0, 100, (T, 3), device="cuda", dtype=torch.int32)
    qk = qkv[:T, :2 * H * D].unflatten(1, (2 * H, D))
    want = q.rope(qk.contiguous(), pos, axes, half=half)
    got = q.rope(qk, pos, axes, half=half)
    assert got.is_contiguous() and torch.equal(got, want)
    before = qkv.clone()
    res = q.rope(qk, pos, axes, half=half, out=qk)
    assert res is qk and torch.equal(qk, want)
    assert torch.equal(qkv[:T, 2 * H * D:], before[:T, 2 * H * D:]) and torch.equal(qkv[T:], before[T:])
    turned = torch.zeros((2 * H, T, D), device="cuda", dtype=t)
    q.rope(before[:T, :2 * H * D].unflatten(1, (2 * H, D)), pos, axes, half=half,
           out=turned.transpose(0, 1))
    assert torch.equal(turned.transpose(0, 1), want)
    one = before[:T, None, :D].expand(T, 3, D)  # one head read three times
    assert torch.equal(q.rope(one, pos, axes, half=half)[:, 2], want[:, 0])


def _tokens_a_workgroup(tokens, heads, hd, turned):
    """The launch's rule, to know that a case below runs what it is for."""
    half, per = turned // 2, hd // 8
    group = max(256 // half if half else 1, 1024 // (heads * per))
    group = min(group, 1024 // half if half else 64)
    return group if group >= 1 and tokens >= 1024 * group else 1


@pytest.mark.parametrize("half", [False, True], ids=["pairs", "halves"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("tokens,heads,hd,axes,group",
                         [(4099, 24, 128, [44, 42, 42], 4), (16387, 2, 128, [44, 42, 42], 16),
                          (32771, 3, 64, [20, 22, 22], 32), (131075, 1, 16, [2, 4, 10], 128),
                          (65543, 1, 80, [10, 0, 22], 64), (65539, 2, 64, [0, 0, 0], 64),
                          (4099, 2, 512, [200, 156, 156], 4)])
def test_several_tokens_a_workgroup(q, tokens, heads, hd, axes, group, bf16, half):
    """Enough tokens that a workgroup takes several, the last one fewer; the
    same inside a wider row, in place, with the elements around untouched."""
    import torch
    say("rope groups", tokens, heads, hd, axes, bf16, half)
    assert _tokens_a_workgroup(tokens, heads, hd, sum(axes)) == group and tokens % group
    x = _x((tokens, heads, hd), tokens + hd, bf16)
    pos = np.random.default_rng(tokens).integers(-50, 4000, (tokens, len(axes))).astype(np.int32)
    p, d = torch.from_numpy(pos).cuda(), to_device(wl.f32_to_bf16_bits(x) if bf16 else x)
    got = q.rope(d, p, axes, half=half)
    _check(_np(got), x, pos, axes, 10000.0, half, False, bf16)
    wide = torch.full((tokens, heads * hd + 16), 3.0, dtype=d.dtype, device="cuda")
    part = wide[:, 8:8 + heads * hd].unflatten(1, (heads, hd))
    part.copy_(d)
    q.rope(part, p, axes, half=half, out=part)
    assert torch.equal(part, got)
    assert bool((wide[:, :8] == 3).all()) and bool((wide[:, -8:] == 3).all())


@pytest.mark.parametrize("half", [False, True], ids=["pairs", "halves"])
def test_more_tokens_than_the_grid(q, half):
    """2^20 workgroups of four tokens and more: some of them walk on."""
    import torch
    tokens = 4 * 2 ** 20 + 4099
    say("rope walk", tokens, half)
    assert _tokens_a_workgroup(tokens, 1, 512, 512) == 4
    x = torch.randn((tokens, 1, 512), device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(-99, 9999, (tokens, 2), device="cuda", dtype=torch.int32)
    parts = [slice(0, 9), slice(4 * 2 ** 20 - 7, 4 * 2 ** 20 + 9), slice(tokens - 9, tokens)]
    want = [q.rope(x[s].clone(), pos[s].clone(), [256, 256], half=half) for s in parts]
    q.rope(x, pos, [256, 256], half=half, out=x)
    for s, w in zip(parts, want):
        assert torch.equal(x[s], w)


@pytest.mark.parametrize("half", [False, True])
def test_inverse_is_the_gradient(q, half):
    """<g, rope(x + e d) - rope(x - e d)> / 2e = <rope^-1(g), d>: the map is
    linear, so the difference is exact up to fp32 rounding of the sums; and
    the inverse undoes the embedding."""
    import torch
    say("rope gradient", half)
    g0 = torch.Generator(device="cuda").manual_seed(3)
    x, g, d = (torch.randn((31, 5, 96), device="cuda", generator=g0) for _ in range(3))
    pos = torch.randint(0, 1000, (31, 3), device="cuda", dtype=torch.int32, generator=g0)
    f = lambda v, **k: q.rope(v, pos, [32, 32, 32], half=half, **k).double()  # noqa: E731
    e = 0.5
    diff = ((f(x + e * d) - f(x - e * d)) / (2 * e) * g.double()).sum()
    grad = (f(g, inverse=True) * d.double()).sum()
    # every value differs by at most 2^-20 (|u| + |v|) on either side: about
    # 8 2^-20 a term at three sigma, summed over 14880 terms of random sign
    assert abs(float(diff - grad)) <= 8 * 2.0 ** -20 * 14880 ** 0.5 * 4
    back = f(f(x).float(), inverse=True)
    assert float((back - x.double()).abs().max()) <= 2 * 2.0 ** -21 * 2 * float(x.abs().max()) * 1.5


@pytest.mark.parametrize("half", [False, True])
def test_offsets_beyond_32_bits_and_unused_strides(q, half):
    """Three tokens 2^31 elements apart, and single tokens or heads whose
    strides are no multiple of 16 bytes."""
    import torch
    say("rope far offsets", half)
    x = torch.randn((3, 2, 64), device="cuda").bfloat16()
    pos = torch.tensor([[3], [70000], [-9]], dtype=torch.int32, device="cuda")
    want = q.rope(x, pos, [48], half=half)
    buf = torch.empty((2 * 2 ** 31 + 128,), dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((3, 2, 64), (2 ** 31, 64, 1))
    far.copy_(x)
    assert torch.equal(q.rope(far, pos, [48], half=half), want)
    q.rope(far, pos, [48], half=half, out=far)
    assert torch.equal(far, want)
    one = x[:1].as_strided((1, 2, 64), (7, 64, 1))
    assert torch.equal(q.rope(one, pos[:1], [48], half=half), want[:1])
    head = x[:, :1].as_strided((3, 1, 64), (128, 3, 1))
    assert torch.equal(q.rope(head, pos, [48], half=half), want[:, :1])


def test_empty(q):
    import torch
    x = torch.zeros((0, 4, 64), device="cuda")
    assert q.rope(x, torch.zeros((0, 1), dtype=torch.int32, device="cuda"), [64]).shape == (0, 4, 64)
    x = torch.zeros((4, 0, 64), device="cuda")
    assert q.rope(x, torch.zeros((4, 1), dtype=torch.int32, device="cuda"), [64]).shape == (4, 0, 64)
