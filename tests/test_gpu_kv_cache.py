"""Keys and values into the 4-bit cache on the GPU, bit for bit against the plain
form (division by a power of two is exact: the codes are a function of the
input alone)."""
import numpy as np
import pytest

from tests import mx_ref
from tests.gpu_util import host, say, to_device
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    import quantization_dit_linear_amd as q
    assert torch.cuda.is_available()
    q.lib()
    return q


def _filled(q, pages, heads, page, hd, seed):
    """A cache of random bytes, and a copy of it on the host."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = q.mx_kv_cache(pages, heads, page, hd)
    for t in cache:
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return cache, [host(t).copy() for t in cache]


def _expected(before, x, slots, page):
    codes, scales = before
    tokens, heads, hd = x.shape
    c, s = mx_ref.quantize(x.reshape(-1, hd), "fp4")
    c = mx_ref.pack(c, "fp4").reshape(tokens, heads, -1)
    s = s.reshape(tokens, heads, -1)
    for t, slot in enumerate(slots):
        if 0 <= slot < codes.shape[0] * page:
            codes[slot // page, :, slot % page], scales[slot // page, :, slot % page] = c[t], s[t]
    return codes, scales


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("tokens,heads,hd,pages,page", [
    (1, 1, 32, 1, 1), (1, 8, 128, 3, 16), (5, 3, 96, 4, 7), (33, 2, 64, 2, 64), (100, 5, 160, 9, 16),
    (64, 40, 128, 64, 16), (1500, 2, 32, 11, 256), (17, 1, 256, 1, 100), (9, 13, 224, 30, 1), (2500, 1, 64, 50, 64)])
def test_write(q, tokens, heads, hd, pages, page, bf16):
    import torch
    say("kv write", tokens, heads, hd, pages, page, bf16)
    rng = np.random.default_rng([tokens, heads, hd])
    x = (rng.standard_normal((2, tokens, heads, hd)) * np.exp(2 * rng.standard_normal((2, tokens, heads, 1)))).astype(np.float32)
    x[:, 0, 0, :32] = 0
    x[0, -1, -1, -1], x[1, -1, 0, 3] = np.inf, np.nan
    if bf16:
        x = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(x))
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots = np.concatenate((slots, np.full(tokens - len(slots), -1))) if len(slots) < tokens else slots
    if tokens > 3:
        slots[rng.integers(0, tokens, 3)] = [-1, pages * page, -(2 ** 40)]
    cache, before = _filled(q, pages, heads, page, hd, 1)
    k, v = (to_device(wl.f32_to_bf16_bits(t) if bf16 else t) for t in x)
    q.mx_kv_write(k, v, torch.from_numpy(slots).cuda(), cache)
    for i in range(2):
        want = _expected(before[2 * i:2 * i + 2], x[i].astype(np.float64), slots, page)
        np.testing.assert_array_equal(host(cache[2 * i]), want[0])
        np.testing.assert_array_equal(host(cache[2 * i + 1]), want[1])


def test_strided_and_broadcast_inputs(q):
    """Slices of a fused projection's output, heads before tokens, and one token
    for every slot; the keys and the values with strides of their own."""
    import torch
    say("kv write strides")
    g = torch.Generator(device="cuda").manual_seed(4)
    heads, hd, page = 4, 96, 8
    qkv = torch.randn((10, 12 * hd), generator=g, device="cuda").bfloat16()
    k = qkv[:, 4 * hd:8 * hd].unflatten(1, (heads, hd))
    v = torch.randn((heads, 10, hd), generator=g, device="cuda").bfloat16().transpose(0, 1)
    one = k[:1].expand(10, heads, hd)
    slots = torch.randperm(24, generator=g, device="cuda")[:10]
    for a, b in ((k, v), (one, k)):
        got, want = q.mx_kv_cache(3, heads, page, hd), q.mx_kv_cache(3, heads, page, hd)
        q.mx_kv_write(a, b, slots, got)
        q.mx_kv_write(a.contiguous(), b.contiguous(), slots, want)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        values = q.mx_dequantize(got.v_codes.view(-1, hd // 2), got.v_scales.view(-1, hd // 32), "fp4")
        values = values.view(3, heads, page, hd).transpose(1, 2).flatten(0, 1)[slots]
        c, s = q.mx_quantize(b.contiguous().view(-1, hd), "fp4")
        assert torch.equal(values, q.mx_dequantize(c, s, "fp4").view(10, heads, hd))


def test_far_slots(q):
    """Rows behind 2^32 bytes of codes, and of scale bytes behind 2^31."""
    import torch
    say("kv write far")
    pages, heads, page, hd = 5, 8, 1 << 20, 256
    cache = q.mx_kv_cache(pages, heads, page, hd)
    assert cache.k_codes.numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = torch.randn((2, 3, heads, hd), generator=g, device="cuda").bfloat16()
    slots = torch.tensor([pages * page - 1, 0, 4 * page], device="cuda")
    q.mx_kv_write(k, v, slots, cache)
    for codes, scales, x in ((cache.k_codes, cache.k_scales, k), (cache.v_codes, cache.v_scales, v)):
        c, s = q.mx_quantize(x.reshape(-1, hd), "fp4")
        got = torch.stack([codes[p // page, :, p % page] for p in slots.tolist()])
        assert torch.equal(got.view(-1, hd // 2), c)
        got = torch.stack([scales[p // page, :, p % page] for p in slots.tolist()])
        assert torch.equal(got.view(-1, hd // 32), s)
        assert int((scales != 0).sum()) == s.numel()
    del cache
    torch.cuda.empty_cache()


def test_graph(q):
    import torch
    say("kv write graph")
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(4, device="cuda")
    cache, want = q.mx_kv_cache(4, 2, 4, 64), q.mx_kv_cache(4, 2, 4, 64)
    q.mx_kv_write(k, v, slots, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.mx_kv_write(k, v, slots, cache)
    for i in range(3):
        k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
        v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
        slots.copy_(torch.randperm(16, generator=g, device="cuda")[:4])
        graph.replay()
        q.mx_kv_write(k, v, slots, want)
        assert all(torch.equal(a, b) for a, b in zip(cache, want))
