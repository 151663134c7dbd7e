"""The cached-attention path run together, as a block runs it for its new
tokens: projection by 4-bit group weights, norm and embedding of the heads in
place, keys and values into the cache, attention, projection back."""
import numpy as np
import pytest

from tests import kv_ref as ref
from tests import mx_ref
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    import quantization_dit_linear_amd as q
    assert torch.cuda.is_available()
    q.lib()
    return q


QH, KH, HD, D, PAGE, BATCH = 6, 2, 64, 384, 16, 3


def _step(q, s, n):
    """n new tokens of each sequence through the block; s["lengths"] counts them already."""
    qkv = q.rtn4_group_linear(s["x"], *s["w_in"])
    qs = qkv[:, :QH * HD].unflatten(1, (QH, HD))
    ks = qkv[:, QH * HD:(QH + KH) * HD].unflatten(1, (KH, HD))
    vs = qkv[:, (QH + KH) * HD:].unflatten(1, (KH, HD))
    q.qk_norm_rope(qs, ks, s["pos"], [HD], q_weight=s["qw"], k_weight=s["kw"], half=True, q_out=qs, k_out=ks)
    q.mx_kv_write(ks, vs, s["slots"], s["cache"])
    o = q.mx_kv_attention(qs, s["cache"], s["lengths"], table=s["table"], causal=True)
    return q.rtn4_group_linear(o.flatten(1), *s["w_out"]), qkv, o


def _state(q, n, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"x": rand(BATCH * n, D).bfloat16(), "qw": (1 + 0.1 * rand(HD)).bfloat16(), "kw": (1 + 0.1 * rand(HD)).bfloat16()}
    s["w_in"] = q.rtn4_group_prepare_weights((rand((QH + 2 * KH) * HD, D) / D ** 0.5).bfloat16(), 64, zeros=True)
    s["w_out"] = q.rtn4_group_prepare_weights((rand(D, QH * HD) / (QH * HD) ** 0.5).bfloat16(), 32)
    s["cache"] = q.mx_kv_cache(20, KH, PAGE, HD)
    s["table"] = torch.randperm(18, generator=g, device="cuda").int().view(BATCH, 6)
    s["lengths"] = torch.zeros(BATCH, dtype=torch.int32, device="cuda")
    s["pos"] = torch.zeros((BATCH * n, 1), dtype=torch.int32, device="cuda")
    s["slots"] = torch.zeros(BATCH * n, dtype=torch.int64, device="cuda")
    return s


def _advance(s, n):
    """The next n tokens of every sequence: positions, slots, lengths."""
    import torch
    p = s["lengths"][:, None].long() + torch.arange(n, device="cuda")
    s["pos"].copy_(p.reshape(-1, 1))
    s["slots"].copy_((s["table"].gather(1, p // PAGE).long() * PAGE + p % PAGE).flatten())
    s["lengths"].add_(n)


@pytest.mark.parametrize("n", [1, 5, 40])
def test_steps_follow_the_plain_form(q, n):
    """Every operator's outputs against the plain form of its own inputs, over
    steps that fill the cache: attention sees what all steps wrote."""
    import torch
    say("kv step", n)
    s, kept = _state(q, n, n), [[], []]
    for step in range(90 // n if n > 1 else 20):
        s["x"].copy_(torch.randn(s["x"].shape, device="cuda"))
        _advance(s, n)
        y, qkv, o = _step(q, s, n)
        x = qkv.double().cpu().numpy().reshape(BATCH, n, QH + 2 * KH, HD)
        kept[0].append(x[:, :, QH:QH + KH])
        kept[1].append(x[:, :, QH + KH:])
        got = o.double().cpu().numpy().reshape(BATCH, n, QH, HD)
        for b in range(BATCH):
            k, v = (np.concatenate([t[b] for t in kept[i]]) for i in range(2))
            k, v = (mx_ref.decode(*mx_ref.quantize(t.reshape(-1, HD), "fp4"), "fp4").reshape(t.shape).transpose(1, 0, 2)
                    for t in (k, v))
            want, tol, _, _ = ref.attention(x[b, :, :QH], k, v, np.float64(np.float32(HD ** -0.5)), True, 0, True)
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
            assert np.all(np.abs(got[b] - want) <= tol), (step, b)
        w, mag = ref.group_weights(host(s["w_out"][0]), host(s["w_out"][1].float()), None, 32)
        want, e = o.double().cpu().numpy().reshape(BATCH * n, -1), None
        e = (np.abs(want) @ mag.T) * (QH * HD + 8) * ref.U
        want = want @ w.T
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= e + 2.0 ** -8 * (np.abs(want) + e))


def test_a_captured_step(q):
    """One token a step in a graph: replays follow the positions, slots and
    lengths and give the eager steps' bits."""
    import torch
    say("kv step graph")
    a, b = _state(q, 1, 7), _state(q, 1, 7)
    y = _step(q, a, 1)[0]  # slot 0, length 0: warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = _step(q, a, 1)[0]
    for t in a["cache"]:
        t.zero_()
    for step in range(40):
        x = torch.randn(a["x"].shape, device="cuda")
        for s in (a, b):
            s["x"].copy_(x)
            _advance(s, 1)
        graph.replay()
        assert torch.equal(y, _step(q, b, 1)[0]), step
        assert all(torch.equal(t, u) for t, u in zip(a["cache"], b["cache"]))
