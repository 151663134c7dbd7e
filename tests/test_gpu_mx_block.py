"""The microscaled path as a block uses it: gated residual sum and norm into
codes, the fused projection on them, the rotary embedding on its queries and
keys where they lie -- against a 64-bit form of the whole, captured into graphs
that share buffers and are replayed, on a stream of its own, and beside the
library's other quantizer."""
import numpy as np
import pytest

from tests import mx_ref as ref
from tests.gpu_util import bf16_to_np, host, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    import quantization_dit_linear_amd as q
    assert torch.cuda.is_available()
    q.lib()
    return q


AXES, HEADS, HD = [24, 20, 20], 5, 64
D = HEADS * HD


def _state(tokens, seed, fmt_w):
    import torch
    import quantization_dit_linear_amd as q
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    s = {"x": n(tokens, D).bfloat16(), "res": (3 * n(tokens, D)).bfloat16(),
         "weight": (1 + 0.1 * n(D)).bfloat16(), "mod": (0.3 * n(2, 6 * D)).bfloat16(),
         "w": q.mx_quantize(0.05 * n(3 * D, D), fmt_w),
         "pos": torch.randint(0, 60, (tokens, 3), device="cuda", dtype=torch.int32, generator=g)}
    return s


def _block(q, s, fmt_a, fmt_w, stream=None):
    m, per = s["mod"], (len(s["x"]) + 1) // 2
    h, codes, scales = q.add_rms_norm(s["x"], s["res"], weight=s["weight"], gate=m[:, 2 * D:3 * D],
                                      scale=m[:, D:2 * D], shift=m[:, :D], rows_per_mod=per,
                                      fmt=fmt_a, stream=stream)
    qkv = q.mx_linear(codes, scales, fmt_a, *s["w"], fmt_w, stream=stream)
    qk = qkv[:, :2 * D].unflatten(1, (2 * HEADS, HD))
    q.rope(qk, s["pos"], AXES, out=qk, stream=stream)
    return h, codes, scales, qkv


@pytest.mark.parametrize("tokens", [1, 2, 77, 600])
@pytest.mark.parametrize("fmt_a,fmt_w", [("fp4", "fp4"), ("fp8", "fp4"), ("fp8", "fp8")])
def test_block_against_64_bits(q, tokens, fmt_a, fmt_w):
    """Each step against the 64-bit form of the step before it as the device
    holds it.  Linear: 2^-8 of the value and 2^-10 of each 64-step's largest
    product (see test_gpu_mx), then bf16 again after the turn: 2^-8."""
    say("mx block", tokens, fmt_a, fmt_w)
    s = _state(tokens, tokens, fmt_w)
    h, codes, scales, qkv = _block(q, s, fmt_a, fmt_w)
    m = bf16_to_np(s["mod"])
    row = np.arange(tokens) // ((tokens + 1) // 2)
    t = bf16_to_np(s["res"]) + bf16_to_np(s["x"]) * m[row, 2 * D:3 * D]
    assert np.all(np.abs(bf16_to_np(h) - t) <= 2.0 ** -8 * np.abs(t) + 1e-5)
    y = t / np.sqrt((t * t).mean(1, keepdims=True) + 1e-6) * bf16_to_np(s["weight"])
    y = y * (1 + m[row, D:2 * D]) + m[row, :D]
    a = ref.decode(ref.unpack(host(codes), fmt_a), host(scales), fmt_a)
    # the codes' own rounding: half a step at most of the block's largest
    # value (e2m1 above 6: a quarter; e4m3 above 448: an eighth)
    top = np.abs(y).reshape(tokens, -1, 32).max(-1).repeat(32, 1)
    assert np.all(np.abs(a - y) <= top * (0.25 if fmt_a == "fp4" else 0.125) * 1.001)
    w = ref.decode(ref.unpack(host(s["w"][0]), fmt_w), host(s["w"][1]), fmt_w)
    p = a @ w.T
    step = [np.abs(v).reshape(len(v), -1, 64).max(-1) for v in (a, w)]
    tol = 2.0 ** -8 * np.abs(p) + 2.0 ** -10 * (step[0] @ step[1].T)
    want = p.copy()
    qk = lambda v: v[:, :2 * D].reshape(tokens, 2 * HEADS, HD)  # noqa: E731
    want[:, :2 * D] = ref.rope(qk(p), host(s["pos"]), AXES, 10000.0, False, False).reshape(tokens, -1)
    pair = qk(tol).reshape(tokens, 2 * HEADS, -1, 2).sum(-1).repeat(2, -1)
    tol[:, :2 * D] = pair.reshape(tokens, -1) + 2.0 ** -7 * np.abs(want[:, :2 * D]) + 1e-6
    assert np.all(np.abs(bf16_to_np(qkv) - want) <= tol * 1.01)


def test_graphs_share_buffers_and_replay(q):
    """Two captured blocks of different sizes over one set of inputs each,
    replayed in turn with eager work between: every replay equals the eager
    result on the inputs of the moment."""
    import torch
    say("mx block graphs")
    states = [_state(t, 40 + t, "fp4") for t in (3, 300)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for s in states:
            _block(q, s, "fp8", "fp4")
    torch.cuda.synchronize()
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_block(q, s, "fp8", "fp4"))
        graphs.append(g)
    for turn in range(4):
        for s, g, o in zip(states, graphs, outs):
            s["x"].copy_(torch.randn_like(s["x"].float()).bfloat16())
            want = [t.clone() for t in _block(q, s, "fp8", "fp4")]
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(o, want):
                assert torch.equal(a, b), turn


def test_two_streams_at_once(q):
    import torch
    say("mx block two streams")
    states = [_state(t, 7 * t, "fp4") for t in (200, 513)]
    want = [[t.clone() for t in _block(q, s, "fp4", "fp4")] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [_block(q, s, "fp4", "fp4", stream=st) for s, st in zip(states, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_beside_the_rotating_quantizer(q):
    """The norm's bf16 rows feed rotate_quantize and the low-bit linear, and its
    sum the next block; results of those paths are what they are without it."""
    import torch
    say("mx block beside rotate_quantize")
    s = _state(50, 3, "fp4")
    h, y = q.add_rms_norm(s["x"], s["res"], weight=s["weight"])
    h2, y2 = q.add_rms_norm(y, h)
    codes, norms = q.rotate_quantize(y, 5, 4)
    again, norms2 = q.rotate_quantize(y.clone(), 5, 4)
    assert torch.equal(codes, again) and torch.equal(norms, norms2)
    t = h.double() + y.double()
    assert float((h2.double() - t).abs().max()) <= 2.0 ** -8 * float(t.abs().max())
