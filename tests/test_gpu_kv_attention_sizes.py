"""Attention over the 4-bit cache where the sizes choose other ways through the
kernels: more sequences than a wave has lanes, more tiles than are shared out
evenly, rows in more parts than a wave joins at once.  Against the plain 64-bit
form; tolerances as derived in tests/kv_ref.py."""
import numpy as np
import pytest

from tests import kv_ref as ref
from tests.gpu_util import host, say
from tests.test_gpu_kv_attention import _cache, _np, _queries, _table, q  # noqa: F401

pytestmark = pytest.mark.gpu


def _shared(q, qd, kh, batch, page, width):
    """Whether a call shares its steps out evenly: only then it needs a workspace."""
    tokens, qh, hd = qd.shape
    return q.lib().oq_mx_kv_attention_workspace(tokens, qh, kh, hd, batch, page, width) > 0


def _check(q, seed, lengths, counts, qh, kh, hd, page, causal, window, bf16, shared, starts=True, heads=None):
    """One call against the plain form, at the key heads `heads` (all of them by default).  Tokens
    that no sequence names keep what the outputs hold."""
    import torch
    rng = np.random.default_rng([seed, hd, page, qh])
    pages = sum(-(-n // page) for n in lengths) + 1
    cache, dev = _cache(q, rng, pages, kh, page, hd)
    table = _table(rng, lengths, page, pages)
    behind = 3 if starts else 0
    qd = _queries(rng, (sum(counts) + behind, qh, hd), bf16)
    assert _shared(q, qd, kh, len(lengths), page, table.shape[1]) == shared
    at = np.concatenate(([0], np.cumsum(counts)))
    out = torch.full(qd.shape, 7.0, dtype=qd.dtype, device="cuda")
    _, lse = q.mx_kv_attention(
        qd, dev, torch.tensor(lengths, dtype=torch.int32, device="cuda"), table=torch.from_numpy(table).cuda(),
        q_starts=torch.from_numpy(at.astype(np.int32)).cuda() if starts else None, causal=causal, window=window,
        out=out, lse=torch.full(qd.shape[:2], 5.0, device="cuda"))
    assert (out[at[-1]:] == 7.0).all() and (lse[at[-1]:] == 5.0).all()
    heads = list(range(kh)) if heads is None else heads
    share = qh // kh
    mine = [h * share + i for h in heads for i in range(share)]
    x, got, glse = _np(qd)[:, mine], _np(out)[:, mine], host(lse).astype(np.float64)[:, mine]
    k, v = (ref.cache_values(c[:, heads], s[:, heads]) for c, s in (cache[:2], cache[2:]))
    scale = np.float64(np.float32(hd ** -0.5))
    for b, n in enumerate(lengths):
        rows = slice(at[b], at[b + 1])
        want, tol, wl, ltol = ref.attention(x[rows], ref.rows_of(k, table, b, n), ref.rows_of(v, table, b, n),
                                            scale, causal, window, bf16)
        err, tol = np.abs(got[rows] - want), tol + ref.half_step(bf16) * (np.abs(want) + tol)
        assert np.all(err <= tol), (b, float(np.max(err / np.maximum(tol, 1e-300))))
        none = np.isneginf(wl)
        np.testing.assert_array_equal(np.isneginf(glse[rows]), none)
        assert np.all(np.abs(glse[rows][~none] - wl[~none]) <= ltol[~none]), b


def _lengths(n, top, empty):
    """n lengths spread over [0, top]; those of `empty` are 0."""
    v = [int(top * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    for i in empty:
        v[i] = 0
    return v


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("batch,top,shared", [(65, 300, True), (130, 200, True), (700, 90, True), (1100, 70, False)])
@pytest.mark.parametrize("starts", [False, True])
def test_many_sequences_of_one_token(q, starts, batch, top, shared, bf16):  # noqa: F811
    say("kv sizes one token", starts, batch, top, bf16)
    lengths = _lengths(batch, top, [0, 62, 63, 64, batch - 1])
    counts = [1] * batch
    if starts:
        for i in (5, 63, 64, batch - 2):  # sequences without queries around the 64th, and before the last
            counts[i] = 0
    _check(q, 1, lengths, counts, 4, 2, 64, 16, True, 0, bf16, shared, starts)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("batch,shared", [(70, True), (530, False)])
@pytest.mark.parametrize("window", [0, 9])
def test_many_sequences_of_few_rows(q, window, batch, shared, bf16):  # noqa: F811
    """Ragged chunks, none to three tiles of 16 rows each, the rows kernel."""
    say("kv sizes few rows", window, batch, bf16)
    counts = [(3 * i + i // 64) % 5 for i in range(batch)]
    _check(q, 2, _lengths(batch, 80, [64]), counts, 20, 2, 32, 24, True, window, bf16, shared)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 20)])
def test_many_sequences_of_many_rows(q, causal, window, bf16):  # noqa: F811
    """More than 64 sequences on the tiles kernel, some of them without queries."""
    say("kv sizes many rows", causal, window, bf16)
    counts = [0 if i in (0, 63, 64, 69) else 8 + i % 7 for i in range(70)]
    _check(q, 3, _lengths(70, 150, [3, 65]), counts, 8, 1, 64, 16, causal, window, bf16, True)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 50)])
@pytest.mark.parametrize("starts", [False, True])
def test_more_tiles_of_many_rows_than_are_shared(q, starts, causal, window, bf16):  # noqa: F811
    """A workgroup a tile and key head: sequences of one, two and no tiles."""
    say("kv sizes many groups", starts, causal, window, bf16)
    lengths, counts = ([200, 64, 30, 0, 333], [300, 70, 0, 9, 90]) if starts else ([280, 64, 301], [290] * 3)
    _check(q, 4, lengths, counts, 206, 206, 32, 16, causal, window, bf16, False, starts, [0, 1, 100, 204, 205])


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("hd,page", [(64, 64), (96, 16), (192, 64)])
@pytest.mark.parametrize("starts", [False, True])
def test_one_long_sequence_among_many_short_ones(q, starts, hd, page, bf16):  # noqa: F811
    """A row in more than 64 parts that a wave joins alone: shares are two steps at least, the long
    sequence has some 300 and the others' together no more."""
    say("kv sizes long among short", starts, hd, page, bf16)
    lengths = [5 + i for i in range(70)]
    lengths[40] = 20000 if hd < 192 else 10000
    counts = [1] * 70
    if starts:
        counts[39], counts[41] = 0, 2
    _check(q, 5, lengths, counts, 2, 1, hd, page, True, 0, bf16, True, starts)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 9, 130])
def test_large_values(q, n, bf16):  # noqa: F811
    """Values up to the stated range, 2^119 over the tokens that a row sees: here 64 of them,
    6 times 2^110 at most, all of one sign where the sums are largest.  And tiny ones, 2^-100."""
    import torch
    say("kv sizes large values", n, bf16)
    rng = np.random.default_rng([20, n])
    for codes, s in ((None, 127 + 110), (0x77, 127 + 110), (None, 127 - 100)):
        cache, _ = _cache(q, rng, 4, 2, 16, 64)
        cache[3][:] = s
        if codes is not None:
            cache[2][:] = codes  # 6 times the scale everywhere
        dev = q.KVCache(*(torch.from_numpy(t).cuda() for t in cache))
        table = np.array([[2, 0, 3, 1]], np.int32)
        qd = _queries(rng, (n, 4, 64), bf16)
        out = q.mx_kv_attention(qd, dev, torch.tensor([64], dtype=torch.int32, device="cuda"),
                                table=torch.from_numpy(table).cuda())
        k, v = ref.cache_values(*cache[:2]), ref.cache_values(*cache[2:])
        want, tol, _, _ = ref.attention(_np(qd), ref.rows_of(k, table, 0, 64), ref.rows_of(v, table, 0, 64),
                                        np.float64(np.float32(64 ** -0.5)), False, 0, bf16)
        err, tol = np.abs(_np(out) - want), tol + ref.half_step(bf16) * (np.abs(want) + tol)
        assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-300)))
