"""The heads' RMS norm with the rotary embedding on the GPU against a plain form.

Tolerance, u = 2^-24: a head's sum of squares is off by at most head_dim u
(positive terms, any order), its root by half of that; mean, eps, root and the
products with the factor and the weight by 8 u: (head_dim / 2 + 8) u of the
normed element.  The turn adds 2^-21 of |u| + |v| as in the embedding alone
(angle, functions, products); then the type's half step."""
import numpy as np
import pytest

from tests import kv_ref as ref
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


def _dev(a, bf16):
    return to_device(wl.f32_to_bf16_bits(a) if bf16 else np.ascontiguousarray(a, np.float32))


def _check(got, x, w, eps, pos, axes, theta, half, bf16):
    want, mag = ref.norm_rope(x, w, eps, pos, axes, theta, half)
    e = mag * (2.0 ** -21 + (x.shape[-1] / 2 + 8) * ref.U)
    tol = e + ref.half_step(bf16) * (np.abs(want) + e)
    err = np.abs(got - want)
    assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-300)))


CASES = [(1, 1, 1, 8, [8]), (1, 40, 8, 128, [128]), (1, 1, 0, 128, [44, 42, 42]), (3, 5, 5, 64, [20, 22, 22]),
         (257, 3, 1, 72, [24, 24, 16]), (64, 24, 24, 128, [16, 56, 56]), (1000, 2, 2, 96, [96]),
         (33, 7, 1, 256, [64, 64, 64, 64]), (5, 4, 4, 512, [200, 152, 160]), (19, 6, 3, 80, [16, 0, 48]),
         (2, 3, 3, 64, [0, 0, 0]), (4097, 1, 1, 16, [16]), (3, 2, 1, 48, [32]), (2, 9, 2, 504, [0, 480]),
         (6, 1, 1, 320, [16, 16]), (1025, 130, 2, 64, [64]), (4, 3, 2, 512, [0]), (9, 0, 3, 128, [64])]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("tokens,qh,kh,hd,axes,half", [(*c, h) for c in CASES for h in (False, True)
                                                      if not h or sum(c[4]) % 16 == 0])
def test_heads(q, tokens, qh, kh, hd, axes, half, bf16):
    import torch
    say("qk norm rope", tokens, qh, kh, hd, axes, half, bf16)
    rng = np.random.default_rng([tokens, qh, hd])
    x = rng.standard_normal((tokens, qh + kh, hd)) * np.exp(rng.standard_normal((tokens, qh + kh, 1)))
    wq, wk = (1 + 0.2 * rng.standard_normal((2, hd))).astype(np.float32)
    pos = rng.integers(-50, 4000, (tokens, len(axes))).astype(np.int32)
    xd, wqd, wkd = _dev(x.astype(np.float32), bf16), _dev(wq, bf16), _dev(wk, bf16)
    qd, kd = xd[:, :qh], xd[:, qh:]
    qo, ko = q.qk_norm_rope(qd, kd if kh else None, torch.from_numpy(pos).cuda(), axes, q_weight=wqd,
                            k_weight=wkd if kh else None, half=half)
    if qh:
        _check(_np(qo), _np(qd), _np(wqd), 1e-6, pos, axes, 10000.0, half, bf16)
    if kh:
        _check(_np(ko), _np(kd), _np(wkd), 1e-6, pos, axes, 10000.0, half, bf16)
    else:
        assert ko is None


@pytest.mark.parametrize("weights", ["none", "q", "k"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_missing_and_other_typed_weights(q, weights, bf16):
    import torch
    say("qk norm rope weights", weights, bf16)
    rng = np.random.default_rng(5)
    x = rng.standard_normal((21, 5, 64)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal(64)).astype(np.float32)
    pos = rng.integers(0, 99, (21, 2)).astype(np.int32)
    xd, wd = _dev(x, bf16), _dev(w, not bf16)
    wq, wk = (wd if weights == n else None for n in "qk")
    qo, ko = q.qk_norm_rope(xd[:, :3], xd[:, 3:], torch.from_numpy(pos).cuda(), [32, 32], q_weight=wq,
                            k_weight=wk, eps=1e-5, theta=500.0)
    for got, at, w1 in ((qo, slice(0, 3), wq), (ko, slice(3, 5), wk)):
        _check(_np(got), _np(xd)[:, at], None if w1 is None else _np(w1), 1e-5, pos, [32, 32], 500.0, False, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("tokens", [1, 6, 1200])
def test_in_place_in_a_fused_projection(q, tokens, half, bf16):
    """The queries and keys of [q | k | v] and of heads by turns (q k v q k v),
    in place: the values, and everything else of the rows, stay."""
    import torch
    say("qk norm rope in place", tokens, half, bf16)
    rng, hd, pos = np.random.default_rng(tokens), 64, None
    pos = torch.from_numpy(rng.integers(0, 500, (tokens, 1)).astype(np.int32)).cuda()
    flat = _dev(rng.standard_normal((tokens, 7 * hd)).astype(np.float32), bf16)
    views = [lambda t: (t[:, :4 * hd].unflatten(1, (4, hd)), t[:, 4 * hd:6 * hd].unflatten(1, (2, hd)),
                        t[:, 6 * hd:])]
    turns = _dev(rng.standard_normal((tokens, 9 * hd)).astype(np.float32), bf16)
    views.append(lambda t: tuple(t.view(tokens, 3, 3, hd)[:, :, i] for i in range(3)))
    for t, view in zip((flat, turns), views):
        qs, ks, vs = view(t)
        want = q.qk_norm_rope(qs, ks, pos, [hd], half=half)
        kept = vs.clone()
        got = q.qk_norm_rope(qs, ks, pos, [hd], half=half, q_out=qs, k_out=ks)
        assert got[0] is qs and got[1] is ks
        assert torch.equal(qs, want[0]) and torch.equal(ks, want[1]) and torch.equal(vs, kept)


def test_a_head_does_not_depend_on_its_batch(q):
    import torch
    say("qk norm rope batch")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((3000, 6, 128), generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 9999, (3000, 3), generator=g, device="cuda", dtype=torch.int32)
    whole = q.qk_norm_rope(x[:, :4], x[:, 4:], pos, [44, 42, 42])
    one = q.qk_norm_rope(x[1234:1235, :4], x[1234:1235, 4:], pos[1234:1235], [44, 42, 42])
    for a, b in zip(whole, one):
        assert torch.equal(a[1234:1235], b)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    other = q.qk_norm_rope(heads_first[:, :4], heads_first[:, 4:], pos, [44, 42, 42])
    assert torch.equal(other[0], whole[0]) and torch.equal(other[1], whole[1])


@pytest.mark.parametrize("half", [False, True])
def test_extreme_heads(q, half):
    """Heads whose squares pass the fp32 range keep their norm, heads of tiny
    numbers and of zeros give tiny numbers and zeros, and one with a NaN or an
    infinity does not reach its neighbours."""
    import torch
    say("qk norm rope extremes", half)
    rng, hd = np.random.default_rng(2), 64
    x = rng.standard_normal((1, 9, hd)).astype(np.float32)
    for h, f in ((0, 1e30), (1, 3e37), (2, 1e-20), (3, 0.0), (4, 1e-38)):
        x[0, h] *= np.float32(f)
    x[0, 5, 9], x[0, 6, 63] = np.nan, np.inf
    pos = np.array([[77]], np.int32)
    y, _ = q.qk_norm_rope(_dev(x, False), None, torch.from_numpy(pos).cuda(), [hd], half=half)
    y = _np(y)
    ok = [0, 1, 2, 3, 4, 7, 8]
    _check(y[:, ok], x[:, ok].astype(np.float64), None, 1e-6, pos, [hd], 10000.0, half, False)
    assert np.isnan(y[0, 5]).all() and np.isnan(y[0, 6]).any()
    small = np.float32(np.finfo(np.float32).tiny)
    y, _ = q.qk_norm_rope(_dev(x[:, 1:2], True), None, torch.from_numpy(pos).cuda(), [hd], half=half, eps=small)
    _check(_np(y), _np(_dev(x[:, 1:2], True)), None, small, pos, [hd], 10000.0, half, True)


def test_graph(q):
    import torch
    say("qk norm rope graph")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((5, 12, 128), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((5, 1), dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    call = lambda **kw: q.qk_norm_rope(x[:, :8], x[:, 8:], pos, [128], half=True, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q_out=out[:, :8], k_out=out[:, 8:])
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        pos.fill_(1000 * i + 7)
        graph.replay()
        a, b = call()
        assert torch.equal(out[:, :8], a) and torch.equal(out[:, 8:], b)
