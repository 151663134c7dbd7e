"""Attention over the 4-bit cache on the GPU against a plain 64-bit form; the
tolerances are derived in tests/kv_ref.py."""
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


def _queries(rng, shape, bf16, spread=1.0):
    v = (spread * rng.standard_normal(shape)).astype(np.float32)
    return to_device(wl.f32_to_bf16_bits(v) if bf16 else v)


def _cache(q, rng, pages, heads, page, hd):
    """Random codes; scales from 2^-5 to 2^1, so that values are of order one."""
    cache = []
    for _ in range(2):
        cache.append(rng.integers(0, 256, (pages, heads, page, hd // 2), dtype=np.uint8))
        cache.append(rng.integers(122, 128, (pages, heads, page, hd // 32)).astype(np.uint8))
    return cache, q.KVCache(*(to_device(t) for t in cache))


def _compare(q, qd, cache, dev, lengths, table, starts, causal, window, scale=None, **kw):
    """One call with its logarithms against the plain form, sequence by sequence; returns the outputs."""
    import torch
    hd, bf16 = qd.shape[-1], qd.dtype == torch.bfloat16
    out, lse = q.mx_kv_attention(
        qd, dev, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
        table=None if table is None else torch.from_numpy(table).cuda(),
        q_starts=None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda"),
        scale=scale, causal=causal, window=window, lse=True, **kw)
    k, v = ref.cache_values(*cache[:2]), ref.cache_values(*cache[2:])
    if table is None:
        table = np.arange(len(lengths))[:, None]
    if starts is None:
        starts = np.arange(len(lengths) + 1) * (qd.shape[0] // max(1, len(lengths)))
    x, got, glse = _np(qd), _np(out), host(lse).astype(np.float64)
    scale = np.float64(np.float32(hd ** -0.5 if scale is None else scale))
    cap = table.shape[1] * cache[0].shape[2]
    for b, n in enumerate(lengths):
        n = min(max(n, 0), cap)
        at = slice(starts[b], starts[b + 1])
        want, tol, wl_, ltol = ref.attention(x[at], ref.rows_of(k, table, b, n), ref.rows_of(v, table, b, n),
                                             scale, causal, window, bf16)
        nan = np.isnan(want)
        np.testing.assert_array_equal(np.isnan(got[at]), nan)
        err = np.abs(got[at] - want)[~nan]
        tol = (tol + ref.half_step(bf16) * (np.abs(want) + tol))[~nan]
        assert np.all(err <= tol), (b, float(np.max(err / np.maximum(tol, 1e-300))))
        none = np.isneginf(wl_)
        np.testing.assert_array_equal(np.isneginf(glse[at]), none)
        np.testing.assert_array_equal(np.isnan(glse[at]), np.isnan(wl_))
        ok = np.isfinite(wl_)
        assert np.all(np.abs(glse[at][ok] - wl_[ok]) <= ltol[ok]), b
        assert np.all(got[at][none] == 0)
    return out, lse


def _table(rng, lengths, page, pages, extra=0):
    """Pages in any order; numbers that are not pages where a sequence has no tokens."""
    width = max(1, max(-(-n // page) for n in lengths) + extra)
    table = np.full((len(lengths), width), -7, np.int32)
    order = rng.permutation(pages)
    at = 0
    for b, n in enumerate(lengths):
        used = -(-n // page)
        table[b, :used] = order[at:at + used]
        at += used
    return table


def _paged(q, seed, lengths, counts, qh, kh, hd, page, causal, window, bf16, spread=1.0, extra=0):
    rng = np.random.default_rng([seed, hd, page, qh])
    pages = sum(-(-n // page) for n in lengths) + 2
    cache, dev = _cache(q, rng, pages, kh, page, hd)
    table = _table(rng, lengths, page, pages, extra)
    uniform = len(set(counts)) == 1
    starts = None if uniform else [0, *np.cumsum(counts).tolist()]
    qd = _queries(rng, (sum(counts), qh, hd), bf16, spread)
    return _compare(q, qd, cache, dev, lengths, table, starts, causal, window)


HEADS = [(1, 1), (4, 4), (6, 2), (8, 1), (40, 8), (33, 1), (5, 5)]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("qh,kh", HEADS)
@pytest.mark.parametrize("hd", [32, 64, 96, 128, 160, 192, 224, 256])
def test_one_token_each(q, hd, qh, kh, bf16):
    say("kv attention one token", hd, qh, kh, bf16)
    lengths = [1, 63, 64, 65, 0, 200, 31, 129]
    _paged(q, 1, lengths, [1] * 8, qh, kh, hd, 16, True, 0, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 64, 100, 256])
def test_pages(q, page, bf16):
    say("kv attention pages", page, bf16)
    _paged(q, 2, [301, 5, 256, 99], [1] * 4, 8, 2, 64, page, True, 0, bf16, extra=2)
    _paged(q, 3, [301, 5, 256, 99], [33, 5, 64, 1], 4, 2, 64, page, True, 0, bf16)


MASKS = [(False, 0), (True, 0), (True, 1), (True, 37), (True, 64), (True, 1000)]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("hd,qh,kh", [(32, 2, 2), (64, 3, 1), (96, 4, 2), (128, 2, 1), (160, 1, 1), (192, 2, 2),
                                      (224, 1, 1), (256, 2, 1)])
def test_many_queries(q, hd, qh, kh, causal, window, bf16):
    """More queries than tokens (rows that see nothing), as many, fewer, none."""
    say("kv attention many", hd, qh, kh, causal, window, bf16)
    _paged(q, 4, [70, 130, 33, 0, 257, 90, 1], [100, 130, 1, 9, 65, 0, 3], qh, kh, hd, 16, causal, window, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("share", [1, 2, 3, 4, 5, 8, 16, 33])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 17])
def test_shared_heads_and_short_chunks(q, n, share, bf16):
    say("kv attention share", n, share, bf16)
    _paged(q, 5, [40, 300, 9], [n] * 3, 2 * share, 2, 64, 64, True, 0, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("length", [1000, 4097, 20000])
def test_long(q, length, bf16):
    """One token over a long cache, and a few queries at its end."""
    say("kv attention long", length, bf16)
    _paged(q, 6, [length], [1], 4, 1, 128, 64, True, 0, bf16)
    _paged(q, 7, [length, 777], [5, 2], 2, 1, 64, 256, True, 600, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_peaked_and_flat(q, bf16):
    """Scores from one token far ahead of the rest (weights that underflow) to all alike."""
    import torch
    for spread in (0.0, 0.01, 30.0):
        say("kv attention spread", spread, bf16)
        _paged(q, 8, [500, 64], [70, 64], 2, 1, 64, 16, True, 0, bf16, spread)
    rng = np.random.default_rng(9)
    cache, dev = _cache(q, rng, 2, 1, 64, 32)
    qd = _queries(rng, (2, 2, 32), bf16)
    for scale in (0.0, -0.3, 2.5):
        _compare(q, qd, cache, dev, [64, 50], None, None, False, 0, scale)
    assert torch.isfinite(qd.float()).all()


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 130])
def test_cache_without_a_table(q, n, bf16):
    """Sequence b is page b: one page a sequence, longer than its tokens."""
    say("kv attention no table", n, bf16)
    rng = np.random.default_rng([10, n])
    cache, dev = _cache(q, rng, 4, 2, 333, 96)
    qd = _queries(rng, (3 * n, 4, 96), bf16)
    _compare(q, qd, cache, dev, [333, 1, 170], None, None, False, 0)
    _compare(q, qd, cache, dev, [400, -5, 130], None, None, True, 0)  # taken as 333 and 0


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 64])
def test_pages_that_are_not_there(q, n, bf16):
    """Rows that see a token of such a page are NaN, the others are not; a page
    number behind the sequence's tokens does not matter."""
    say("kv attention missing pages", n, bf16)
    rng = np.random.default_rng([11, n])
    cache, dev = _cache(q, rng, 6, 1, 16, 64)
    table = np.array([[0, 1, 99, 3], [2, -1, 4, 5], [5, 4, 3, 2 ** 31 - 1], [1, 2, 0, -2 ** 31]], np.int32)
    qd = _queries(rng, (4 * n, 3, 64), bf16)
    out, _ = _compare(q, qd, cache, dev, [40, 64, 47, 48], table, None, True, 20)
    assert not np.isnan(_np(out)[2 * n:]).any()


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("hd", [64, 96, 128])
@pytest.mark.parametrize("n", [1, 6, 150])
def test_nan_blocks(q, n, hd, bf16):
    """Blocks that hold NaN (scale bytes 253 to 255) among the keys and the values:
    rows that see them are NaN (of the values only in the block's elements),
    rows that do not are as they would be without; so with what lies behind a
    sequence's end."""
    say("kv attention nan blocks", n, hd, bf16)
    rng = np.random.default_rng([12, n, hd])
    cache, _ = _cache(q, rng, 12, 2, 16, hd)
    for at, (page, head, row, block, s) in {1: (3, 0, 5, 0, 255), 3: (7, 1, 2, 1, 255)}.items():
        cache[at][page, head, row, block] = s
    cache[3][5, :, 9, 0], cache[3][2, 0, 0, 1], cache[1][11, 1, 15, 1] = 253, 254, 255
    cache[1][8, :, 4:], cache[3][8, :, 4:] = 255, 255  # behind the end of sequence 2
    dev = q.KVCache(*(to_device(t) for t in cache))
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7], [9, 10, 8, -1]], np.int32)
    for causal, window in ((True, 0), (True, 9), (False, 0)):
        qd = _queries(rng, (3 * n, 4, hd), bf16)
        _compare(q, qd, cache, dev, [64, 57, 36], table, None, causal, window)


@pytest.mark.parametrize("n", [1, 40])
def test_nan_queries(q, n):
    import torch
    say("kv attention nan queries", n)
    rng = np.random.default_rng([13, n])
    cache, dev = _cache(q, rng, 2, 1, 64, 64)
    for bf16 in (False, True):
        qd = _queries(rng, (2 * n, 2, 64), bf16)
        qd[0, 1, 3] = float("nan")
        qd[n, 0] = float("nan")
        out, lse = _compare(q, qd, cache, dev, [64, 64], None, None, False, 0)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[n, 0])
        assert torch.isfinite(out).sum() == out.numel() - 2 * 64


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_strides_and_rows_behind_the_last_sequence(q, bf16):
    """Queries as a slice of a fused projection, outputs heads first; tokens
    before the first and behind the last sequence keep what the outputs hold."""
    import torch
    say("kv attention strides", bf16)
    rng = np.random.default_rng(14)
    cache, dev = _cache(q, rng, 8, 2, 16, 64)
    table = np.arange(8, dtype=np.int32).reshape(2, 4)
    for n in (1, 50):
        rows = 2 * n + 9
        qkv = _queries(rng, (rows, 4 * 64 + 72), bf16)
        qd = qkv[:, 8:8 + 4 * 64].unflatten(1, (4, 64))
        starts = [3, 3 + n, 3 + 2 * n]
        out = torch.full((4, rows, 64), 7.0, dtype=qd.dtype, device="cuda").transpose(0, 1)
        lse = torch.full((rows, 4), 5.0, device="cuda")
        got = q.mx_kv_attention(qd, dev, torch.tensor([60, 33], dtype=torch.int32, device="cuda"),
                                table=torch.from_numpy(table).cuda(),
                                q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), causal=True,
                                out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        want, _ = _compare(q, qd[3:3 + 2 * n].contiguous(), cache, dev, [60, 33], table, None, True, 0)
        assert torch.equal(out[3:3 + 2 * n], want)
        for t, v in ((out, 7.0), (lse, 5.0)):
            assert (t[:3] == v).all() and (t[3 + 2 * n:] == v).all()


def test_starts_that_are_not_ascending(q):
    """Garbage in q_starts stays inside the arrays: what it names twice or out of
    range is unspecified, the call ends and rows that no sequence names stay."""
    import torch
    say("kv attention starts")
    rng = np.random.default_rng(15)
    _, dev = _cache(q, rng, 4, 1, 16, 32)
    qd = _queries(rng, (20, 1, 32), True)
    out = torch.full((20, 1, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    for starts in ([-9, 4, 2, 8, 8], [5, 5, 5, 5, 5], [2 ** 31 - 1, -2 ** 31, 0, 30, 8], [8, 6, 4, 2, 0]):
        q.mx_kv_attention(qd, dev, torch.full((4,), 16, dtype=torch.int32, device="cuda"),
                          q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), out=out)
        torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("tokens", [100, 2000])
def test_starts_that_name_tokens_many_times(q, tokens):
    """More tiles than the sizes allow: the call ends, touches nothing but its
    outputs and its workspace, and the next call is right."""
    import torch
    say("kv attention starts many times", tokens)
    rng = np.random.default_rng(16)
    cache, dev = _cache(q, rng, 8, 1, 16, 32)
    before = [c.clone() for c in dev]
    qd = _queries(rng, (tokens, 1, 32), True)
    around = torch.full((tokens + 64, 1, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    q.mx_kv_attention(qd, dev, torch.full((8,), 16, dtype=torch.int32, device="cuda"),
                      q_starts=torch.tensor([0, tokens] * 4 + [0], dtype=torch.int32, device="cuda"),
                      out=around[32:-32])
    torch.cuda.synchronize()
    assert (around[:32] == 3.0).all() and (around[-32:] == 3.0).all()
    assert all(torch.equal(a, b) for a, b in zip(before, dev))
    _compare(q, qd, cache, dev, [16] * 8, None, [0, 3, 3, 40, 41, 60, 61, tokens - 1, tokens], True, 0)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_same_bits_every_time_and_in_graphs(q, bf16):
    """Twice the same call, two captured graphs replayed by turns with eager work
    between them, and a call on another stream: the same bits; the graphs follow
    lengths that change."""
    import torch
    say("kv attention graphs", bf16)
    rng = np.random.default_rng(16)
    lengths = [3000, 17, 900]
    pages = sum(-(-n // 64) for n in lengths)
    _, dev = _cache(q, rng, pages, 2, 64, 128)
    table = torch.from_numpy(_table(rng, lengths, 64, pages)).cuda()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    inputs = [_queries(rng, (3 * m, 8, 128), bf16) for m in (1, 70)]
    outs = [torch.empty_like(x) for x in inputs]
    call = lambda i, **kw: q.mx_kv_attention(inputs[i], dev, n, table=table, causal=True, **kw)  # noqa: E731
    for i in range(2):
        assert torch.equal(call(i), call(i))
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, out=outs[i])
    for step in range(3):
        n.copy_(torch.tensor([3000 - 700 * step, 17 + step, 900 - 450 * step], dtype=torch.int32))
        inputs[0].mul_(1.25)
        for i in (step % 2, 1 - step % 2):
            graphs[i].replay()
        for i in range(2):
            assert torch.equal(outs[i], call(i)), (step, i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        want = call(i)
        got = call(i, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_two_streams_at_once(q):
    """Two calls in flight together have a workspace each."""
    import torch
    say("kv attention two streams")
    rng = np.random.default_rng(17)
    _, dev = _cache(q, rng, 64, 1, 256, 128)
    table = torch.randperm(64, device="cuda").int().view(1, 64)
    n = torch.tensor([64 * 256], dtype=torch.int32, device="cuda")
    xs = [_queries(rng, (1, 8, 128), True) for _ in range(2)]
    want = [q.mx_kv_attention(x, dev, n, table=table) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(q.mx_kv_attention(xs[i], dev, n, table=table))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_far_pages(q):
    """Pages behind 2^32 bytes of codes."""
    import torch
    say("kv attention far")
    pages, heads, page, hd = 5, 8, 1 << 20, 256
    cache = q.mx_kv_cache(pages, heads, page, hd)
    near = q.mx_kv_cache(1, heads, 64, hd)
    rng = np.random.default_rng(18)
    for far, small in zip(cache, near):
        v = torch.from_numpy(rng.integers(110, 126, small.shape).astype(np.uint8)).cuda()
        small.copy_(v)
        far[4, :, :64] = v[0]
    table = torch.tensor([[4]], dtype=torch.int32, device="cuda")
    for n in (1, 60):
        qd = _queries(rng, (n, 16, hd), True)
        length = torch.tensor([64], dtype=torch.int32, device="cuda")
        got = q.mx_kv_attention(qd, cache, length, table=table, causal=True)
        want, tol = q.mx_kv_attention(qd, near, length, causal=True), 2.0 ** -6
        assert torch.isfinite(got).all() and (got - want).abs().max() <= tol * want.abs().max()
    del cache, far
    torch.cuda.empty_cache()
