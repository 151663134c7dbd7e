"""INT4 weights with group scales on the GPU against plain forms.

The projection's tolerance, u = 2^-24: every order of summing K products is off
by at most K u of the sum of magnitudes S = sum |s| |x| (|nibble - 8| + |8 - z|)
(an implementation may take the zero point apart from the nibbles), the scale,
the zero point and a split of x by 8 u more; then half a step of bf16.  A
row's error over all outputs also has to be what that last rounding gives."""
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
    return to_device(wl.f32_to_bf16_bits(a) if bf16 else a.astype(np.float32))


def _weights(rng, N, K, group, zeros, scale_bf16):
    q4 = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = (0.01 * np.exp(rng.standard_normal((N, K // group)))).astype(np.float32)
    z = rng.uniform(0, 15, s.shape).astype(np.float32) if zeros else None
    s, z = (None if a is None else _dev(a, scale_bf16) for a in (s, z))
    return q4, s, z


def _check(y, x, q4, s, z, group):
    w, mag = ref.group_weights(q4, _np(s), None if z is None else _np(z), group)
    want, e = x @ w.T, (np.abs(x) @ mag.T) * (x.shape[1] + 8) * ref.U
    tol = e + 2.0 ** -8 * (np.abs(want) + e)
    assert np.all(np.abs(y - want) <= tol), float(np.max(np.abs(y - want) / np.maximum(tol, 1e-300)))
    assert np.linalg.norm(y - want) <= 2.0 ** -8 * np.linalg.norm(want) + np.linalg.norm(e)


SHAPES = [(1, 1, 32, 32), (1, 16, 64, 64), (1, 17, 96, 32), (2, 100, 1024, 128), (3, 5, 480, 96),
          (4, 257, 512, 512), (5, 33, 2048, 64), (8, 64, 256, 128), (9, 31, 160, 160), (16, 129, 1536, 64),
          (17, 48, 640, 128), (31, 130, 320, 32), (33, 15, 224, 224), (64, 66, 512, 64), (65, 16, 128, 32),
          (130, 40, 384, 128), (1, 515, 5120, 128), (2, 20, 16384, 16384), (7, 9, 16384, 64)]


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("scale_bf16", [False, True], ids=["s32", "s16"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_linear(q, M, N, K, group, bf16, scale_bf16, zeros):
    say("rtn4 group linear", M, N, K, group, bf16, scale_bf16, zeros)
    rng = np.random.default_rng([M, N, K, group])
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 100))] *= 100.0
    q4, s, z = _weights(rng, N, K, group, zeros, scale_bf16)
    xd = _dev(x, bf16)
    y = q.rtn4_group_linear(xd, to_device(q4), s, z)
    _check(_np(y), _np(xd), q4, s, z, group)


@pytest.mark.parametrize("zeros,scale_bf16", [(False, True), (True, False)], ids=["sym", "zeros"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(29, 8200, 320, 32), (33, 4161, 480, 96), (64, 4097, 256, 64),
                                         (17, 8191, 384, 128), (70, 2753, 1056, 352)])
def test_wide_tiles(q, M, N, K, group, bf16, scale_bf16, zeros):
    """Columns and rows enough for the tiles of 64 columns."""
    test_linear(q, M, N, K, group, bf16, scale_bf16, zeros)


@pytest.mark.parametrize("zeros,scale_bf16", [(False, False), (True, True)], ids=["sym", "zeros"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(1, 4130, 640, 128), (3, 4097, 320, 64), (4, 4111, 352, 32), (2, 4099, 672, 96),
                                         (5, 4105, 256, 128), (16, 4129, 448, 64), (12, 4098, 288, 32), (9, 4150, 320, 160),
                                         (17, 4100, 384, 128), (32, 5001, 704, 64), (20, 4321, 224, 32), (31, 8100, 480, 480)])
def test_pairs_of_tiles(q, M, N, K, group, bf16, scale_bf16, zeros):
    """Columns enough for two tiles a workgroup, too few for four."""
    test_linear(q, M, N, K, group, bf16, scale_bf16, zeros)


@pytest.mark.parametrize("zeros,scale_bf16", [(False, False), (True, True)], ids=["sym", "zeros"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(3, 40, 1088, 64), (12, 70, 1600, 64), (40, 70, 1344, 64), (40, 33, 1312, 32),
                                         (4, 5, 1952, 32), (2, 37, 3232, 3232), (20, 35, 2592, 288)])
def test_half_steps(q, M, N, K, group, bf16, scale_bf16, zeros):
    """K that ends within 128 coordinates, where some of the groups do."""
    test_linear(q, M, N, K, group, bf16, scale_bf16, zeros)


def test_many_rows(q):
    """More rows than one grid has tiles for."""
    import torch
    say("rtn4 group many rows")
    rng, M, N, K = np.random.default_rng(2), (1 << 20) + 37, 3, 32
    x = rng.standard_normal((M, K)).astype(np.float32)
    q4, s, _ = _weights(rng, N, K, 32, False, True)
    xd = _dev(x, True)
    y = q.rtn4_group_linear(xd, to_device(q4), s)
    rows = np.r_[0:70, (1 << 20) - 70:M]
    _check(_np(y[rows]), _np(xd[rows]), q4, s, None, 32)


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M", [1, 12, 40])
def test_wide_ranges(q, M, bf16):
    """Activations from 2^-60 to 2^60 side by side, groups of zeros, subnormals
    and the largest numbers: the sums keep what an fp32 sum keeps."""
    say("rtn4 group ranges", M, bf16)
    rng, N, K = np.random.default_rng(M), 48, 256
    x = (rng.standard_normal((M, K)) * 2.0 ** rng.integers(-60, 60, (M, K))).astype(np.float32)
    x[:, 32:64] = 0
    x[0, 64:96] = 2.0 ** -140
    x[-1, 96:128] = rng.standard_normal(32) * 2.0 ** 100
    q4, s, _ = _weights(rng, N, K, 32, False, False)
    xd = _dev(x, bf16)
    y = q.rtn4_group_linear(xd, to_device(q4), s)
    _check(_np(y), _np(xd), q4, s, None, 32)


@pytest.mark.parametrize("zeros,scale_bf16", [(False, False), (True, True)], ids=["sym", "zeros"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,N,group", [(1, 70, 64), (3, 4130, 64), (12, 70, 64), (12, 4130, 64), (40, 70, 64),
                                       (40, 2100, 64), (3, 70, 32), (12, 4130, 128), (40, 70, 96), (3, 4130, 96)])
def test_large_numbers_at_the_end(q, M, N, group, bf16, scale_bf16, zeros):
    """The last 16 bytes of a row up to the stated range (a group's |x| below 2^122),
    where K ends within a step of 128: what the step reads behind K counts nothing.
    Sums hold x (16 + nibble) and x (16 + z), as the header says, so each order of
    summing them is off by at most K u of |s| |x| (16 + nibble + 16 + z), where a
    column's weights at the end may all be 0; the rest as at the top."""
    say("rtn4 group large end", M, N, group, bf16, scale_bf16, zeros)
    for K in (group * 3, group * 17):
        rng = np.random.default_rng([M, K])
        x = rng.standard_normal((M, K)).astype(np.float32)
        last = 8 if bf16 else 4
        x[:, -last:] = 2.0 ** 121 / last
        q4, _, z = _weights(rng, N, K, group, zeros, scale_bf16)
        s = _dev(np.full((N, K // group), 2.0 ** -40, np.float32), scale_bf16)
        xd = _dev(x, bf16)
        y = q.rtn4_group_linear(xd, to_device(q4), s, z)
        x = _np(xd)
        w, _ = ref.group_weights(q4, _np(s), None if z is None else _np(z), group)
        n = np.stack((q4 & 15, q4 >> 4), -1).reshape(N, K)
        mag = 2.0 ** -40 * (32.0 + n + (8.0 if z is None else np.repeat(_np(z), group, 1)))
        want, e = x @ w.T, (np.abs(x) @ mag.T) * (K + 8) * ref.U
        err, tol = np.abs(_np(y) - want), e + 2.0 ** -8 * (np.abs(want) + e)
        assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("M", [1, 3, 20])
def test_not_finite(q, M):
    """A row with a NaN or an infinity does not reach the others."""
    import torch
    say("rtn4 group not finite", M)
    rng, N, K = np.random.default_rng(M), 33, 128
    x = rng.standard_normal((M + 2, K)).astype(np.float32)
    x[0, 5], x[M + 1, 77] = np.nan, np.inf
    q4, s, _ = _weights(rng, N, K, 64, False, True)
    xd = _dev(x, True)
    y = q.rtn4_group_linear(xd, to_device(q4), s)
    assert torch.isnan(y[0]).all() and not torch.isfinite(y[-1]).any()
    _check(_np(y)[1:-1], _np(xd)[1:-1], q4, s, None, 64)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale_bf16", [False, True], ids=["s32", "s16"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (7, 192, 96), (33, 512, 64), (5, 1024, 1024), (64, 256, 32)])
def test_prepare(q, N, K, group, bf16, scale_bf16, zeros):
    """Bit for bit the definition's fp32 operations (numpy's are IEEE's)."""
    import torch
    say("rtn4 group prepare", N, K, group, bf16, scale_bf16, zeros)
    rng = np.random.default_rng([N, K, group])
    W = rng.standard_normal((N, K)).astype(np.float32)
    W[0, :32] = 0
    W[-1] = np.abs(W[-1])
    if bf16:
        W = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(W))
    got = q.rtn4_group_prepare_weights(_dev(W, bf16), group, zeros=zeros,
                                       scale_dtype=torch.bfloat16 if scale_bf16 else torch.float32)
    g = W.reshape(N, -1, group)
    hi, lo = np.maximum(g.max(-1), 0), np.minimum(g.min(-1), 0)
    s = hi / np.float32(15) - lo / np.float32(15) if zeros else np.abs(g).max(-1) / np.float32(7)
    if scale_bf16:
        s = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(s))
    div = np.where(s > 0, s, np.float32(1))
    z = np.where(s > 0, np.clip(np.rint(-lo / div), 0, 15), 0) if zeros else np.full_like(s, 8)
    n = np.clip(np.where(s[..., None] > 0, np.rint(g / div[..., None]), 0) + z[..., None], 0, 15)
    n = n.astype(np.uint8).reshape(N, K)
    np.testing.assert_array_equal(host(got[0]), n[:, 0::2] | (n[:, 1::2] << 4))
    np.testing.assert_array_equal(_np(got[1]), s.astype(np.float64))
    if zeros:
        np.testing.assert_array_equal(_np(got[2]), z.astype(np.float64))
    x = rng.standard_normal((3, K)).astype(np.float32)
    y = q.rtn4_group_linear(_dev(x, False), *got)
    _check(_np(y), x.astype(np.float64), host(got[0]), got[1], got[2] if zeros else None, group)


def test_graph_and_stream(q):
    """Captured once and replayed over changing inputs, and on another stream."""
    import torch
    say("rtn4 group graph")
    rng, M, N, K = np.random.default_rng(0), 3, 200, 1024
    q4, s, z = _weights(rng, N, K, 128, True, True)
    q4d, x = to_device(q4), torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    q.rtn4_group_linear(x, q4d, s, z, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.rtn4_group_linear(x, q4d, s, z, out=out)
    for i in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)))
        g.replay()
        assert torch.equal(out, q.rtn4_group_linear(x, q4d, s, z))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = q.rtn4_group_linear(x, q4d, s, z, stream=side)
    side.synchronize()
    assert torch.equal(out, y)
