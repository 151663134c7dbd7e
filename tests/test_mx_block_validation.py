"""The microscaled path's refusals, without a GPU: the C entry points reject
bad arguments before any device work (the addresses below are never touched),
and the binding rejects mismatched buffers."""
import ctypes

import pytest
import torch

import quantization_dit_linear_amd as q

A, B, C, D, E = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000


def _caller(fn, ok):
    f = getattr(q.lib(), fn)

    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*dict(ok, **kw).values())
    return call


@pytest.mark.parametrize("fn", ["quantize", "dequantize"])
def test_quantize_and_read_back(fn):
    ok = (dict(x=A, dt=1, rows=8, d=64, fmt=4, codes=B, scales=C, stream=None) if fn == "quantize" else
          dict(codes=B, scales=C, fmt=4, rows=8, d=64, dt=1, x=A, stream=None))
    call = _caller("oq_mx_" + fn, ok)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(x=A + 8), dict(codes=B + 8),
               dict(dt=2), dict(dt=-1), dict(fmt=0), dict(fmt=5), dict(rows=-1), dict(d=0), dict(d=-32),
               dict(codes=A + 512), dict(x=B + 128), dict(scales=A + 1023), dict(x=C)):
        assert call(**kw) == q.OQ_EINVAL, kw
    for kw in (dict(d=48), dict(d=16), dict(d=16416), dict(rows=(1 << 30) + 1)):
        assert call(**kw) == q.OQ_EUNSUPPORTED, kw
    assert call(rows=0) == call(rows=0, x=None, codes=None, scales=None) == q.OQ_OK
    assert call(rows=0, d=48) == q.OQ_EUNSUPPORTED
    if fn == "quantize":
        assert call(scales=B + 255) == q.OQ_EINVAL


def test_linear():
    ok = dict(a=A, sa=B, fa=4, w=C, sw=D, fw=8, M=4, N=8, K=96, y=E, stream=None)
    call = _caller("oq_mx_linear", ok)
    for kw in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(a=A + 4),
               dict(w=C + 8), dict(y=E + 1), dict(fa=3), dict(fw=0), dict(M=-1), dict(N=-2), dict(K=0),
               dict(y=A), dict(y=B + 10), dict(y=C + 766), dict(y=D + 22), dict(y=A - 62)):
        assert call(**kw) == q.OQ_EINVAL, kw
    for kw in (dict(K=80), dict(K=16416), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1)):
        assert call(**kw) == q.OQ_EUNSUPPORTED, kw
    for kw in (dict(M=0), dict(N=0), dict(M=0, a=None, sa=None, y=None)):
        assert call(**kw) == q.OQ_OK


def test_norm():
    ok = dict(x=A, res=B, dt=1, rows=4, d=64, eps=1e-6, w=C, gate=D, scale=D + 128, shift=D + 256,
              pdt=1, per=2, stride=384, sum=E, fmt=0, y=E + 0x1000, ys=None, stream=None)
    call = _caller("oq_add_rms_norm", ok)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(x=None), dict(y=None), dict(dt=7), dict(pdt=7), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-40),
               dict(eps=nan), dict(eps=inf), dict(rows=-1), dict(d=0), dict(per=0), dict(stride=-8),
               dict(stride=32), dict(stride=388), dict(fmt=5), dict(fmt=8), dict(ys=E + 0x2000),
               dict(x=A + 8), dict(res=B + 2), dict(w=C + 4), dict(gate=D + 2), dict(sum=E + 8),
               dict(y=E + 0x1008), dict(sum=A + 128), dict(y=A + 128), dict(sum=C), dict(y=D),
               dict(y=E), dict(y=E + 256), dict(sum=D + 768), dict(fmt=8, ys=E + 0x1000),
               dict(fmt=4, y=A, ys=E + 0x2000), dict(fmt=8, ys=B + 511), dict(fmt=8, ys=E + 511)):
        assert call(**kw) == q.OQ_EINVAL, kw
    for kw in (dict(d=48), dict(d=16416), dict(rows=(1 << 30) + 1)):
        assert call(**kw) == q.OQ_EUNSUPPORTED, kw
    assert call(rows=0) == call(rows=0, x=None, y=None) == q.OQ_OK


def test_rope():
    dims = lambda *v: (ctypes.c_int * len(v))(*v)  # noqa: E731
    ok = dict(x=A, dt=1, tokens=4, heads=2, hd=64, xt=128, xh=64, pos=C, axes=3, dims=dims(24, 20, 20),
              theta=1e4, flags=0, y=B, yt=128, yh=64, stream=None)
    call = _caller("oq_rope", ok)
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(dims=None), dict(dt=3), dict(flags=4),
               dict(tokens=-1), dict(heads=-1), dict(hd=0), dict(axes=0), dict(theta=0.5),
               dict(theta=float("inf")), dict(theta=float("nan")), dict(dims=dims(24, 21, 20)),
               dict(dims=dims(24, -2, 20)), dict(dims=dims(24, 24, 24)), dict(x=A + 8), dict(y=B + 8),
               dict(pos=C + 2), dict(xt=132), dict(xh=60), dict(yt=129), dict(yh=-64), dict(xt=-128),
               dict(y=A + 128), dict(x=B + 512), dict(y=A, yh=128, yt=64), dict(yh=32), dict(yt=64),
               dict(yt=0), dict(pos=B + 64), dict(yt=1 << 60), dict(xt=1 << 60)):
        assert call(**kw) == q.OQ_EINVAL, kw
    for kw in (dict(hd=60), dict(hd=520), dict(axes=5, dims=dims(8, 8, 8, 8, 8)),
               dict(flags=q.OQ_ROPE_HALF, dims=dims(24, 20, 18)), dict(tokens=(1 << 30) + 1)):
        assert call(**kw) == q.OQ_EUNSUPPORTED, kw
    for kw in (dict(tokens=0), dict(heads=0), dict(tokens=0, x=None, y=None, pos=None)):
        assert call(**kw) == q.OQ_OK


def test_binding_rejects_mismatched_buffers():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cases = [
        (lambda: q.mx_quantize(bf(4, 64), "fp6"), "fmt"),
        (lambda: q.mx_quantize(bf(64), "fp4"), "rows"),
        (lambda: q.mx_quantize(bf(4, 64), "fp4", codes=u8(4, 64)), "codes"),
        (lambda: q.mx_quantize(bf(4, 64), "fp8", scales=u8(4, 1)), "scales"),
        (lambda: q.mx_quantize(bf(4, 64), "fp8"), "GPU"),
        (lambda: q.mx_dequantize(u8(4, 64), u8(4, 2), "fp4"), "codes"),
        (lambda: q.mx_dequantize(u8(4, 64), u8(4, 2), "fp8", out=bf(4, 32)), "out"),
        (lambda: q.mx_dequantize(u8(4, 64), u8(4, 2), "fp8", out=bf(4, 64), dtype=torch.float32), "out"),
        (lambda: q.mx_linear(u8(4, 64), u8(4, 2), "fp8", u8(3, 64), u8(3, 4), "fp4"), "columns"),
        (lambda: q.mx_linear(u8(4, 64), u8(4, 2), "fp4", u8(3, 64), u8(3, 2), "fp8"), "a_codes"),
        (lambda: q.mx_linear(u8(4, 64), u8(4, 2), "fp8", u8(3, 64), u8(2, 2), "fp8"), "w_codes"),
        (lambda: q.mx_linear(u8(4, 64), u8(4, 2), "fp8", u8(3, 64), u8(3, 2), "fp8", out=bf(3, 4)), "out"),
        (lambda: q.add_rms_norm(bf(4, 64), bf(4, 32)), "residual"),
        (lambda: q.add_rms_norm(bf(4, 64), weight=bf(32)), "weight"),
        (lambda: q.add_rms_norm(bf(4, 64), weight=bf(64), scale=torch.zeros(64)), "scale"),
        (lambda: q.add_rms_norm(bf(4, 64), weight=bf(1, 64)), "weight"),
        (lambda: q.add_rms_norm(bf(4, 64), gate=bf(2, 64), shift=bf(1, 64)), "groups"),
        (lambda: q.add_rms_norm(bf(4, 64), gate=bf(2, 64), rows_per_mod=1), "groups"),
        (lambda: q.add_rms_norm(bf(4, 64), out=bf(4, 32)), "out"),
        (lambda: q.add_rms_norm(bf(4, 64), sum_out=torch.zeros(4, 64)), "sum_out"),
        (lambda: q.add_rms_norm(bf(4, 64), scales_out=u8(4, 2)), "scales_out"),
        (lambda: q.add_rms_norm(bf(4, 64), fmt="fp4", out=u8(4, 64)), "codes"),
        (lambda: q.rope(bf(4, 64), torch.zeros((4, 1), dtype=torch.int32), [64]), "heads"),
        (lambda: q.rope(bf(4, 1, 64), torch.zeros((4, 2), dtype=torch.int32), [64]), "pos"),
        (lambda: q.rope(bf(4, 1, 64), torch.zeros((4, 1), dtype=torch.int64), [64]), "pos"),
        (lambda: q.rope(bf(4, 1, 64), torch.zeros((4, 1), dtype=torch.int32), [64], out=bf(4, 64, 1)), "out"),
        (lambda: q.rope(bf(4, 1, 64), torch.zeros((4, 1), dtype=torch.int32), [64], out=bf(4, 1, 64)), "GPU"),
    ]
    for call, what in cases:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError, match="codes"):
        q.mx_dequantize([1], u8(1, 1), "fp8")


def test_one_tensor_as_weight_and_modulation():
    """The same tensor as weight and as gate, scale or shift is both: its one
    group has to cover the rows like any other's."""
    w = torch.zeros(64, dtype=torch.bfloat16)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for name in ("gate", "scale", "shift"):
        with pytest.raises(ValueError, match="groups"):
            q.add_rms_norm(x, weight=w, rows_per_mod=1, **{name: w})


class _Recorder:
    """Stands for the library: keeps the arguments as the C side would see them."""

    def __init__(self, monkeypatch):
        self.args = []
        monkeypatch.setattr(q, "lib", lambda: self)
        monkeypatch.setattr(q, "_call_device", lambda *named: 0)
        monkeypatch.setattr(q, "_raw_stream", lambda stream, dev: None)

    def __getattr__(self, name):
        def call(*args):
            self.args = [t(a).value for t, a in zip(q._SIGS[name][1], args)]
            return q.OQ_OK
        return call


@pytest.mark.parametrize("per", [4, 5, 2 ** 31, 2 ** 63, 2 ** 64 + 1, 2 ** 65])
def test_rows_per_mod_of_any_size(monkeypatch, per):
    """One group covers every row, however large the number of rows it may
    have: the library has to see no more than one (2^64 + 1 would arrive as 1,
    and the rows behind the first would read past the group)."""
    seen = _Recorder(monkeypatch)
    p = torch.zeros((1, 64), dtype=torch.bfloat16)
    q._torch()
    q.add_rms_norm(torch.zeros((4, 64), dtype=torch.bfloat16), gate=p, rows_per_mod=per)
    rows, rows_per_mod = seen.args[3], seen.args[11]
    assert rows == 4 and rows_per_mod >= 4


def test_sizes_beyond_32_bits_are_refused(monkeypatch):
    """Sizes that the C calls take in 32 bits: a larger one is refused rather
    than cut (2^32 + 64 columns would be taken for 64)."""
    _Recorder(monkeypatch)
    far = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="meta")  # noqa: E731
    u8, d, pos = torch.uint8, 2 ** 32 + 64, torch.zeros((1, 1), dtype=torch.int32)
    q._torch()
    cases = [
        (lambda: q.mx_quantize(far(1, d), "fp4"), "x"),
        (lambda: q.mx_dequantize(far(1, d, t=u8), far(1, d // 32, t=u8), "fp8"), "codes"),
        (lambda: q.mx_linear(far(1, d, t=u8), far(1, d // 32, t=u8), "fp8", far(1, d, t=u8),
                             far(1, d // 32, t=u8), "fp8"), "codes"),
        (lambda: q.add_rms_norm(far(1, d)), "x"),
        (lambda: q.rope(far(1, d, 64), pos, [64]), "heads"),
        (lambda: q.rope(far(1, 1, d), pos, [64]), "head_dim"),
        (lambda: q.rope(far(1, 1, 64), pos, [d]), "axis_dims"),
        (lambda: q.rope(far(1, 1, 64), pos, [64 - 2 ** 32]), "axis_dims"),
    ]
    for call, what in cases:
        with pytest.raises(ValueError, match=what + ".*32 bits"):
            call()
