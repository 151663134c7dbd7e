"""Microscaled quantization, read-back and linear on the GPU against a plain
64-bit form (tests/mx_ref.py): codes, scale bytes and read-back values equal
bit for bit; linear outputs within one bf16 rounding plus the accumulation's
own error.

The linear's tolerance.  One bf16 rounding is 2^-8 |y|.  Products of 4-bit
elements are summed in fp32: at most K roundings of 2^-24 of sum |a w|.  Where
an operand is e4m3 the matrix instruction aligns the products of one step
(64 or 128 elements) to the largest of them and drops low bits: measured on
random codes at most 2^-11.3 of the step's largest product, so 2^-10 of it is
allowed, summed over 64-element steps with max|a| max|w| for the product."""
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


def _tokens(rows, d, seed, bf16):
    """Normal values with an outlier column, exact ties, zero blocks and rows,
    subnormals and blocks of widely different size."""
    r = np.random.default_rng([seed, 1])
    x = r.standard_normal((rows, d)).astype(np.float32)
    x[:, r.integers(0, d)] *= 60.0
    x *= np.exp2(r.integers(-20, 20, (rows, 1))).astype(np.float32)
    x[::5, :32] = r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.5, 0.0], 32)
    x[1::7, -32:] = 0.0
    x[2::11] = 0.0
    x[3::13, :32] = r.standard_normal(32) * np.float32(2.0 ** -130)
    x[4::13, -32:] = r.standard_normal(32) * np.float32(2.0 ** 120)
    return wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(x)) if bf16 else x


def _dev(x, bf16):
    return to_device(wl.f32_to_bf16_bits(x) if bf16 else x)


def _as_bf16(v):
    """fp64 values as the nearest bf16: the read-back's own rounding, which only
    e4m3 values below 2^-126 meet (their last bit lies below 2^-133)."""
    with np.errstate(over="ignore"):
        bits = wl.f32_to_bf16_bits(np.where(np.isnan(v), 0, v).astype(np.float32))
    return np.where(np.isnan(v), np.nan, wl.bf16_bits_to_f32(bits)).astype(np.float64)


SHAPES = [(1, 32), (1, 5120), (2, 64), (3, 96), (7, 160), (129, 1568), (5, 16384), (1000, 288)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_quantize_and_read_back(q, rows, d, bf16, fmt):
    import torch
    say("mx quantize", rows, d, bf16, fmt)
    x = _tokens(rows, d, rows + d, bf16)
    codes, scales = q.mx_quantize(_dev(x, bf16), fmt)
    rc, rs = ref.quantize(x, fmt)
    np.testing.assert_array_equal(host(scales), rs)
    np.testing.assert_array_equal(host(codes), ref.pack(rc, fmt))
    want = ref.decode(rc, rs, fmt)
    got = q.mx_dequantize(codes, scales, fmt, dtype=torch.float32)
    np.testing.assert_array_equal(host(got).astype(np.float64), want)
    np.testing.assert_array_equal(bf16_to_np(q.mx_dequantize(codes, scales, fmt)), _as_bf16(want))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_every_code_and_scale_reads_back(q, fmt):
    """All element codes under every scale byte, through both output types."""
    import torch
    say("mx every code", fmt)
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    c = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    packed = c if fmt == "fp8" else c[:, :128]
    packed = np.ascontiguousarray(packed)
    want = ref.decode(ref.unpack(packed, fmt), s, fmt)
    got = q.mx_dequantize(to_device(packed), to_device(s), fmt, dtype=torch.float32)
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(host(got), want.astype(np.float32))
    b = q.mx_dequantize(to_device(packed), to_device(s), fmt)
    np.testing.assert_array_equal(bf16_to_np(b), _as_bf16(want))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_bad_values_stay_in_their_block(q, fmt, bf16):
    say("mx non-finite", fmt, bf16)
    x = _tokens(6, 128, 9, bf16)
    clean = ref.quantize(x, fmt)
    x[0, 5] = np.nan
    x[2, 40], x[2, 41] = np.inf, 1.0
    x[5, 127] = -np.inf
    codes, scales = q.mx_quantize(_dev(x, bf16), fmt)
    rc, rs = ref.quantize(x, fmt)
    assert rs[0, 0] == rs[2, 1] == rs[5, 3] == 255
    np.testing.assert_array_equal(host(scales), rs)
    np.testing.assert_array_equal(host(codes), ref.pack(rc, fmt))
    same = rs != 255
    np.testing.assert_array_equal(rs[same], clean[1][same])
    v = bf16_to_np(q.mx_dequantize(codes, scales, fmt))
    assert np.isnan(v[0, :32]).all() and np.isfinite(v[0, 32:]).all()


def _codes(rows, K, fmt, seed):
    """Random finite codes and scales, some zero rows."""
    r = np.random.default_rng([seed, 3])
    x = r.standard_normal((rows, K)) * np.exp(r.standard_normal((rows, 1)))
    x[:, :: 37] *= 20.0
    x[3::9] = 0.0
    c, s = ref.quantize(x, fmt)
    return c, s


def _check_linear(q, M, N, K, fa, fw):
    ac, as_ = _codes(M, K, fa, M + K)
    wc, ws = _codes(N, K, fw, N + 3 * K)
    y = bf16_to_np(q.mx_linear(to_device(ref.pack(ac, fa)), to_device(as_), fa,
                               to_device(ref.pack(wc, fw)), to_device(ws), fw))
    a, w = ref.decode(ac, as_, fa), ref.decode(wc, ws, fw)
    want, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    tol = 2.0 ** -8 * np.abs(want) + K * 2.0 ** -24 * mag + 1e-37
    if "fp8" in (fa, fw):
        pad = -K % 64
        sa, sw = (np.abs(np.pad(v, ((0, 0), (0, pad)))).reshape(len(v), -1, 64).max(-1)
                  for v in (a, w))
        tol = tol + 2.0 ** -10 * (sa @ sw.T)
    assert np.all(np.abs(y - want) <= tol), float(np.max(np.abs(y - want) / tol))
    # the same through the norm of the difference: bf16 rounding is uniform,
    # so far below the worst case of every element at once
    assert np.linalg.norm(y - want) <= 2.0 ** -8 * np.linalg.norm(want) + 1e-37


# few rows; few tiles; resident 64, 128 and 256 tiles: each with whole and
# ragged edges, K below, at and above one load of scales
LINEAR = [(1, 1, 32), (1, 16, 64), (3, 5, 96), (16, 16, 128), (17, 33, 160), (31, 257, 256),
          (2, 640, 5120), (64, 64, 512), (128, 130, 544), (255, 257, 1024), (513, 300, 416),
          (300, 515, 2592), (1, 5120, 1024), (5, 128, 16384), (16, 1000, 3200), (33, 4096, 1280),
          (1000, 1000, 288), (1025, 2049, 480), (700, 900, 2592), (1500, 1600, 2080), (2900, 2950, 2592),
          (3000, 3100, 480), (2817, 3090, 32)]


@pytest.mark.parametrize("fa,fw", [("fp4", "fp4"), ("fp8", "fp4"), ("fp4", "fp8"), ("fp8", "fp8")])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(q, M, N, K, fa, fw):
    say("mx linear", M, N, K, fa, fw)
    _check_linear(q, M, N, K, fa, fw)


@pytest.mark.parametrize("fa", ["fp4", "fp8"])
@pytest.mark.parametrize("M,N,K", [(4, 48, 320), (40, 200, 320), (600, 520, 320), (1000, 900, 320), (1500, 1600, 320),
                                   (3000, 3100, 320)])
def test_linear_is_exact_on_small_integers(q, M, N, K, fa):
    """Elements in {-1, 0, 1} under scale 1: every sum is a whole number below
    256, which bf16 holds, so a misplaced element or scale shows at once."""
    say("mx linear exact", M, N, K, fa)
    r = np.random.default_rng(5)
    a, w = (r.choice([-1.0, 0.0, 1.0], p=[0.1, 0.8, 0.1], size=s) for s in ((M, K), (N, K)))
    one = lambda v, f: (ref.nearest(v, f) | (np.signbit(v) << (3 if f == "fp4" else 7))).astype(np.uint8)  # noqa: E731
    sa, sw = (np.full((n, K // 32), 127, np.uint8) for n in (M, N))
    y = bf16_to_np(q.mx_linear(to_device(ref.pack(one(a, fa), fa)), to_device(sa), fa,
                               to_device(ref.pack(one(w, "fp4"), "fp4")), to_device(sw), "fp4"))
    np.testing.assert_array_equal(y, a @ w.T)


@pytest.mark.parametrize("fa,fw", [("fp4", "fp4"), ("fp8", "fp4"), ("fp4", "fp8"), ("fp8", "fp8")])
@pytest.mark.parametrize("M,N", [(5, 70), (70, 90), (600, 520), (3000, 3100)])
def test_linear_over_the_range_of_the_scales(q, M, N, fa, fw):
    """Scale bytes from 0 to 254 against each other.  One element a block, one
    block a row holds a value, so an output is one product 2^(sa + sw - 254):
    exact where fp32 holds it as a normal number, infinite from 2^128 on, at
    most 2^-126 below the normal ones (the sum may flush them)."""
    say("mx linear scales", M, N, fa, fw)
    r = np.random.default_rng([M, 6])
    K, one = 96, {"fp4": 2, "fp8": 0x38}
    sa, sw = (r.choice([0, 1, 2, 60, 126, 127, 128, 190, 253, 254], (n, 3)).astype(np.uint8) for n in (M, N))
    ac, wc = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
    ac[:, 37], wc[:, 37] = one[fa], one[fw]
    y = bf16_to_np(q.mx_linear(to_device(ref.pack(ac, fa)), to_device(sa), fa,
                               to_device(ref.pack(wc, fw)), to_device(sw), fw))
    e = sa[:, 1].astype(int)[:, None] + sw[:, 1].astype(int)[None] - 254
    want = np.ldexp(1.0, e)
    normal = (e >= -126) & (e <= 127)
    np.testing.assert_array_equal(y[normal], want[normal])
    assert np.all(y[e >= 128] == np.inf)
    assert np.all(np.abs(y[e < -126]) <= 2.0 ** -126)


@pytest.mark.parametrize("fa,fw", [("fp4", "fp4"), ("fp8", "fp4"), ("fp8", "fp8")])
@pytest.mark.parametrize("M,N,K", [(5, 70, 160), (70, 90, 288), (520, 513, 160), (900, 800, 1184),
                                   (1500, 1600, 160), (2900, 3000, 544)])
def test_linear_nan_block_reaches_its_row_only(q, M, N, K, fa, fw):
    say("mx linear nan", M, N, K, fa, fw)
    ac, as_ = _codes(M, K, fa, 1)
    wc, ws = _codes(N, K, fw, 2)
    args = lambda: (to_device(ref.pack(ac, fa)), to_device(as_), fa, to_device(ref.pack(wc, fw)),  # noqa: E731
                    to_device(ws), fw)
    clean = bf16_to_np(q.mx_linear(*args()))
    as_[M - 1, K // 32 - 1] = 255
    ac[M - 1, -32:] = 0
    y = bf16_to_np(q.mx_linear(*args()))
    assert np.isnan(y[M - 1]).all()
    np.testing.assert_array_equal(y[:M - 1], clean[:M - 1])
    ws[0, 0] = 255
    wc[0, :32] = 0
    y = bf16_to_np(q.mx_linear(*args()))
    assert np.isnan(y[:, 0]).all()
    np.testing.assert_array_equal(y[:M - 1, 1:], clean[:M - 1, 1:])


def _whole_numbers(rows, K, fmt, seed):
    """Elements in {-1, 0, 1}, few of them not 0, under scales 1/2, 1 and 2:
    codes, scale bytes and the values on the device."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand((rows, K), device="cuda", generator=g)
    v = (u > 0.96).float() - (u < 0.04).float()
    e = torch.randint(-1, 2, (rows, K // 32), device="cuda", generator=g)
    one, sign = (2, 8) if fmt == "fp4" else (0x38, 0x80)
    c = (one * (v != 0) + sign * (v < 0)).to(torch.uint8)
    c = c[:, 0::2] | (c[:, 1::2] << 4) if fmt == "fp4" else c
    return c.contiguous(), (e + 127).to(torch.uint8), v * torch.exp2(e.float()).repeat_interleave(32, 1)


@pytest.mark.parametrize("fa,fw", [("fp4", "fp4"), ("fp8", "fp4"), ("fp4", "fp8"), ("fp8", "fp8")])
@pytest.mark.parametrize("M,N,K", [(5000, 5000, 544), (5000, 5003, 1056), (6000, 6000, 544), (5990, 6001, 2592),
                                   (8200, 8200, 288)])
def test_linear_over_many_tiles(q, M, N, K, fa, fw):
    """More tiles than the card holds at once (256 tiles at 5000 and 8200, 128
    tiles at 6000): workgroups walk to their next ones.  Sums of quarters below
    64 fit bf16, and every step's products differ by 2^4 at most, which no
    alignment drops, so every element is exact."""
    import torch
    say("mx linear many tiles", M, N, K, fa, fw)
    ac, as_, a = _whole_numbers(M, K, fa, M + K)
    wc, ws, w = _whole_numbers(N, K, fw, N + 3 * K)
    want = a @ w.t()
    assert torch.equal(want.bfloat16().float(), want)
    for _ in range(2):
        assert torch.equal(q.mx_linear(ac, as_, fa, wc, ws, fw).float(), want)


@pytest.mark.parametrize("fa,fw", [("fp8", "fp4"), ("fp4", "fp8"), ("fp8", "fp8")])
@pytest.mark.parametrize("M,N", [(20, 90), (600, 1000), (1500, 1600), (2900, 3000)])
def test_linear_after_a_call_full_of_nan(q, M, N, fa, fw):
    """K ends inside a stage: what lies behind it has to be zeros, not what the
    call before left on the chip (here NaN in every e4m3 element)."""
    import torch
    say("mx linear after nan", M, N, fa, fw)
    ac, as_, a = _whole_numbers(M, 160, fa, M)
    wc, ws, w = _whole_numbers(N, 160, fw, N)
    bad = lambda n, f: (torch.full((n, 1024 // (2 if f == "fp4" else 1)), 0x7f, device="cuda", dtype=torch.uint8),  # noqa: E731
                        torch.full((n, 32), 127, device="cuda", dtype=torch.uint8))
    ba, bw = bad(M, fa), bad(N, fw)
    for _ in range(2):
        assert bool(q.mx_linear(*ba, fa, *bw, fw).isnan().all())
        assert torch.equal(q.mx_linear(ac, as_, fa, wc, ws, fw).float(), a @ w.t())


def test_linear_writes_only_y(q):
    """Guard bytes around y stay as they were, at sizes that end inside a tile."""
    import torch
    for M, N, K in ((3, 19, 96), (65, 77, 128), (300, 270, 224), (900, 801, 96), (1500, 1607, 96),
                    (2900, 2951, 224)):
        say("mx linear guards", M, N, K)
        buf = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[2048:2048 + M * N].view(M, N)
        ac, as_ = _codes(M, K, "fp4", 1)
        wc, ws = _codes(N, K, "fp4", 2)
        a, w = ((to_device(ref.pack(c, "fp4")), to_device(s)) for c, s in ((ac, as_), (wc, ws)))
        y = q.mx_linear(*a, "fp4", *w, "fp4", out=out)
        assert y is out
        assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + M * N:] == 7).all())
        torch.testing.assert_close(out, q.mx_linear(*a, "fp4", *w, "fp4"), rtol=0, atol=0)


def test_linear_odd_output_address(q):
    """y at 2-byte alignment (one element into a buffer), whole and ragged N."""
    import torch
    for M, N, K in ((3, 64, 96), (300, 256, 128), (900, 800, 128), (1500, 1600, 128), (2900, 3000, 128)):
        say("mx linear odd y", M, N, K)
        ac, as_ = _codes(M, K, "fp8", 1)
        wc, ws = _codes(N, K, "fp4", 2)
        args = (to_device(ac), to_device(as_), "fp8", to_device(ref.pack(wc, "fp4")), to_device(ws),
                "fp4")
        buf = torch.zeros((M * N + 1,), dtype=torch.bfloat16, device="cuda")
        y = q.mx_linear(*args, out=buf[1:].view(M, N))
        torch.testing.assert_close(y, q.mx_linear(*args), rtol=0, atol=0)
        assert float(buf[0]) == 0.0


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_offsets_beyond_32_bits(q, fmt):
    """The last rows of arrays of more than 2^32 elements are the rows alone."""
    import torch
    rows, d = 262200, 16384
    say("mx far offsets", rows, d, fmt)
    x = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    x[:64].normal_()
    x[-64:].normal_()
    x[64:-64].zero_()
    codes, scales = q.mx_quantize(x, fmt)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        c, s = q.mx_quantize(x[part].contiguous(), fmt)
        assert torch.equal(codes[part], c) and torch.equal(scales[part], s)
    back = q.mx_dequantize(codes, scales, fmt, out=x)
    c, s = codes[-64:].contiguous(), scales[-64:].contiguous()
    assert torch.equal(back[-64:], q.mx_dequantize(c, s, fmt))
    w = q.mx_quantize(torch.randn((40, d), device="cuda"), "fp4")
    y = q.mx_linear(codes, scales, fmt, *w, "fp4")
    torch.testing.assert_close(y[-64:], q.mx_linear(c, s, fmt, *w, "fp4"), rtol=2.0 ** -7, atol=0.05)
    assert bool((y[64:-64] == 0).all())
    # y itself beyond 2^32 elements
    del x, back, codes, y
    a, b = (q.mx_quantize(torch.randn((n, 32), device="cuda"), fmt) for n in (140000, 32000))
    y = q.mx_linear(*a, fmt, *b, fmt)
    tail = tuple(t[-300:].contiguous() for t in a)
    torch.testing.assert_close(y[-300:], q.mx_linear(*tail, fmt, *b, fmt), rtol=2.0 ** -7, atol=1e-3)


def test_empty(q):
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    assert q.mx_linear(z(0, 64), z(0, 4), "fp4", z(8, 64), z(8, 4), "fp4").shape == (0, 8)
    assert q.mx_linear(z(8, 64), z(8, 4), "fp4", z(0, 64), z(0, 4), "fp4").shape == (8, 0)
    c, s = q.mx_quantize(torch.zeros((0, 64), device="cuda"), "fp8")
    assert c.shape == (0, 64) and s.shape == (0, 2)
    assert q.mx_dequantize(c, s, "fp8").shape == (0, 64)
