"""The cached-attention path's refusals, without a GPU: the C entry points reject
bad arguments before any device work (the addresses below are never touched),
and the binding rejects mismatched buffers."""
import ctypes

import pytest
import torch

import quantization_dit_linear_amd as q

A, B, C, D, E, F, G, H = (0x10000000 * i for i in range(1, 9))


def _caller(fn, ok):
    f = getattr(q.lib(), fn)

    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*dict(ok, **kw).values())
    return call


def _refused(call, invalid, unsupported):
    for kw in invalid:
        assert call(**kw) == q.OQ_EINVAL, kw
    for kw in unsupported:
        assert call(**kw) == q.OQ_EUNSUPPORTED, kw


def test_group_prepare():
    call = _caller("oq_rtn4_group_prepare_weights",
                   dict(w=A, dt=1, n=8, d=256, group=64, q4=B, s=C, z=D, sdt=1, stream=None))
    _refused(call, (dict(w=None), dict(q4=None), dict(s=None), dict(w=A + 2), dict(q4=B + 8), dict(s=C + 2),
                    dict(z=D + 2), dict(dt=2), dict(sdt=-1), dict(n=-1), dict(d=0), dict(group=0),
                    dict(group=-32), dict(group=96), dict(group=512), dict(q4=A), dict(s=A + 64), dict(s=B + 16),
                    dict(z=C), dict(z=C + 60), dict(z=A + 4092)),
             (dict(group=16), dict(d=16416, group=32), dict(n=(1 << 30) + 1)))
    for kw in (dict(n=0), dict(n=0, w=None, q4=None, s=None, z=None)):
        assert call(**kw) == q.OQ_OK


def test_group_linear():
    call = _caller("oq_rtn4_group_linear", dict(x=A, dt=1, m=4, q4=B, s=C, z=D, sdt=0, group=64, n=8, k=256,
                                                y=E, stream=None))
    _refused(call, (dict(x=None), dict(q4=None), dict(s=None), dict(y=None), dict(x=A + 8), dict(q4=B + 4),
                    dict(s=C + 2), dict(z=D + 2), dict(y=E + 1), dict(dt=5), dict(sdt=2), dict(m=-1), dict(n=-1),
                    dict(k=0), dict(group=0), dict(group=100), dict(group=3), dict(y=A), dict(y=A + 2046),
                    dict(y=B), dict(y=C + 126), dict(y=D - 62)),
             (dict(group=16), dict(k=16416, group=32), dict(m=(1 << 30) + 1), dict(n=(1 << 30) + 1),
              dict(n=(1 << 27) + 1)))
    for kw in (dict(m=0), dict(n=0), dict(m=0, x=None, y=None)):
        assert call(**kw) == q.OQ_OK


def _dims(*v):
    return (ctypes.c_int * len(v))(*v)


def test_qk_norm_rope():
    ok = dict(q=A, qh=2, qt=128, qs=64, k=B, kh=1, kt=64, ks=64, dt=1, tokens=4, hd=64, qw=C, kw=D, pdt=1,
              eps=1e-6, pos=E, axes=3, dims=_dims(24, 20, 20), theta=1e4, flags=0, qo=F, qot=128, qos=64, ko=G,
              kot=64, kos=64, stream=None)
    call = _caller("oq_qk_norm_rope", ok)
    _refused(call, (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(dims=None),
                    dict(dt=2), dict(pdt=2), dict(flags=q.OQ_ROPE_INVERSE), dict(flags=8), dict(eps=0.0),
                    dict(eps=1e-39), dict(eps=float("nan")), dict(eps=float("inf")), dict(tokens=-1), dict(qh=-1),
                    dict(kh=-1), dict(hd=0), dict(axes=0), dict(theta=0.5), dict(theta=float("nan")),
                    dict(dims=_dims(24, 21, 20)), dict(dims=_dims(24, -2, 20)), dict(dims=_dims(24, 24, 24)),
                    dict(q=A + 8), dict(k=B + 2), dict(qo=F + 8), dict(ko=G + 4), dict(qw=C + 8), dict(kw=D + 2),
                    dict(pos=E + 2), dict(qt=132), dict(qs=60), dict(kt=-64), dict(qot=64), dict(qos=32),
                    dict(kot=56), dict(kot=0), dict(qo=A + 128), dict(qo=A, qot=256), dict(qo=B), dict(ko=A),
                    dict(ko=F), dict(ko=F + 512), dict(qo=C), dict(ko=D - 128), dict(qo=E + 32), dict(qt=1 << 60),
                    dict(qot=1 << 60)),
             (dict(hd=60), dict(hd=520), dict(axes=5, dims=_dims(8, 8, 8, 8, 8)),
              dict(flags=q.OQ_ROPE_HALF, dims=_dims(24, 20, 18)), dict(tokens=(1 << 30) + 1),
              dict(qh=(1 << 24)), dict(kh=1 << 24)))
    for kw in (dict(tokens=0), dict(tokens=0, q=None, k=None, qo=None, ko=None, pos=None), dict(qh=0, kh=0)):
        assert call(**kw) == q.OQ_OK
    # keys inside the queries' heads of one projection, in place: a head of the one is the other's
    fused = dict(q=A, qo=A, qt=448, qot=448, k=A + 256, ko=A + 256, kt=448, kot=448)
    assert call(**dict(fused, k=A + 128, ko=A + 128)) == q.OQ_EINVAL
    assert call(**dict(fused, k=A + 840, ko=A + 840)) == q.OQ_EINVAL


def test_kv_write():
    ok = dict(k=A, v=B, dt=1, tokens=4, kt=128, ks=64, vt=128, vs=64, slots=C, kc=D, ksc=E, vc=F, vsc=G, pages=3,
              heads=2, page=16, hd=64, stream=None)
    call = _caller("oq_mx_kv_write", ok)
    _refused(call, (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(ksc=None), dict(vc=None),
                    dict(vsc=None), dict(k=A + 8), dict(v=B + 4), dict(slots=C + 4), dict(kc=D + 8),
                    dict(ksc=E + 8), dict(vsc=G + 1), dict(dt=3), dict(tokens=-1), dict(pages=-1), dict(heads=0),
                    dict(page=0), dict(hd=0), dict(kt=100), dict(vs=-64), dict(kc=A), dict(vc=B + 1008),
                    dict(ksc=C), dict(vc=D), dict(vsc=E + 176), dict(ksc=D + 3056), dict(kt=1 << 60)),
             (dict(hd=48), dict(hd=288), dict(heads=65536), dict(tokens=(1 << 30) + 1), dict(pages=1 << 45)))
    for kw in (dict(tokens=0), dict(pages=0), dict(tokens=0, k=None, v=None, slots=None)):
        assert call(**kw) == q.OQ_OK


def test_kv_attention():
    ok = dict(q=A, dt=1, tokens=4, qh=4, qt=256, qs=64, kc=B, ksc=B + 0x1000000, vc=C, vsc=C + 0x1000000, pages=8,
              kh=2, page=16, hd=64, batch=4, lengths=D, starts=D + 0x1000, table=E, width=2, scale=0.125, flags=1,
              window=0, out=F, ot=256, os=64, lse=G, ws=H, wsb=1 << 28, stream=None)
    call = _caller("oq_mx_kv_attention", ok)
    _refused(call, (dict(q=None), dict(out=None), dict(kc=None), dict(ksc=None), dict(vc=None), dict(vsc=None),
                    dict(lengths=None), dict(q=A + 8), dict(out=F + 8), dict(kc=B + 4), dict(vsc=C + 2),
                    dict(lengths=D + 2), dict(starts=D + 2), dict(table=E + 1), dict(lse=G + 2), dict(ws=H + 8),
                    dict(dt=2), dict(tokens=-1), dict(qh=0), dict(qh=3), dict(kh=0), dict(page=0), dict(hd=0),
                    dict(batch=-1), dict(pages=-1), dict(pages=0), dict(width=0), dict(flags=2), dict(window=-1),
                    dict(window=5, flags=0), dict(scale=float("nan")), dict(scale=float("inf")),
                    dict(starts=None, tokens=5), dict(table=None), dict(table=None, width=1, pages=3),
                    dict(qt=252), dict(os=32), dict(ot=0), dict(out=A), dict(out=A + 512), dict(out=B),
                    dict(out=C + 0x1000000), dict(lse=F), dict(lse=A + 16), dict(lse=D), dict(out=E + 16),
                    dict(qt=1 << 60)),
             (dict(hd=48), dict(hd=288), dict(kh=65536, qh=65536), dict(batch=(1 << 20) + 1), dict(width=1 << 27),
              dict(tokens=(1 << 27) + 1), dict(tokens=1 << 27)))
    for kw in (dict(tokens=0), dict(batch=0), dict(tokens=0, q=None, out=None, kc=None)):
        assert call(**kw) == q.OQ_OK


@pytest.mark.parametrize("scale", [2.0 ** 127 * 1.5, -3.4e38])
def test_kv_attention_scale(scale):
    """A scale that passes the fp32 range in base 2 (times log2 e) is refused: it would make a score of
    0 a NaN."""
    call = _caller("oq_mx_kv_attention", dict(
        q=A, dt=1, tokens=4, qh=4, qt=256, qs=64, kc=B, ksc=B + 0x1000000, vc=C, vsc=C + 0x1000000, pages=8, kh=2,
        page=16, hd=64, batch=4, lengths=D, starts=None, table=E, width=2, scale=0.125, flags=1, window=0, out=F,
        ot=256, os=64, lse=G, ws=H, wsb=1 << 28, stream=None))
    assert call(scale=scale) == q.OQ_EINVAL
    assert call(scale=scale, tokens=0) == q.OQ_EINVAL


def test_kv_attention_workspace():
    size = q.lib().oq_mx_kv_attention_workspace
    for args in ((1, 4, 3, 64, 1, 16, 1), (1, 4, 2, 48, 1, 16, 1), (-1, 4, 2, 64, 1, 16, 1), (1, 4, 2, 64, 1, 0, 1),
                 (1, 4, 2, 64, 1, 16, 0), (1, 4, 2, 64, 1, 16, 1 << 27), (1 << 27, 4, 2, 64, 1, 16, 1)):
        assert size(*args) == -1, args
    for args in ((0, 4, 2, 64, 1, 16, 1), (4, 4, 2, 64, 0, 16, 1)):
        assert size(*args) == 0, args
    for args in ((1, 1, 1, 32, 1, 1, 1), (1, 40, 8, 128, 1, 64, 512), (64, 32, 8, 128, 64, 64, 128),
                 (1560, 40, 40, 128, 1, 1560, 21), (1 << 25, 4, 1, 256, 1 << 20, 1 << 10, 1 << 20)):
        assert 0 <= size(*args) <= 1 << 31, args


def test_binding_rejects_mismatched_buffers():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64)  # noqa: E731
    cache = q.mx_kv_cache(4, 2, 16, 64, device="cpu")
    cases = [
        (lambda: q.rtn4_group_prepare_weights(bf(4, 64), 48), "group"),
        (lambda: q.rtn4_group_prepare_weights(bf(64), 32), "W"),
        (lambda: q.rtn4_group_prepare_weights(bf(4, 64), 32), "GPU"),
        (lambda: q.rtn4_group_linear(bf(64), u8(4, 32), bf(4, 2)), "x"),
        (lambda: q.rtn4_group_linear(bf(2, 64), u8(4, 64), bf(4, 2)), "q4"),
        (lambda: q.rtn4_group_linear(bf(2, 64), bf(4, 32), bf(4, 2)), "q4"),
        (lambda: q.rtn4_group_linear(bf(2, 64), u8(4, 32), bf(4, 3)), "groups"),
        (lambda: q.rtn4_group_linear(bf(2, 64), u8(4, 32), bf(4, 2), bf(4, 1)), "zeros"),
        (lambda: q.rtn4_group_linear(bf(2, 64), u8(4, 32), bf(4, 2), torch.zeros(4, 2)), "zeros"),
        (lambda: q.rtn4_group_linear(bf(2, 64), u8(4, 32), bf(4, 2), out=bf(4, 2)), "out"),
        (lambda: q.rtn4_group_linear(bf(2, 64), u8(4, 32), bf(4, 2)), "GPU"),
        (lambda: q.qk_norm_rope(bf(4, 64), None, i32(4, 1), [64]), "heads"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), bf(4, 1, 32), i32(4, 1), [64]), "k"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), bf(3, 1, 64), i32(4, 1), [64]), "k"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), torch.zeros(4, 1, 64), i32(4, 1), [64]), "k"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i32(4, 1), [64], k_weight=bf(64)), "k_weight"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i32(4, 1), [64], q_weight=bf(32)), "q_weight"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), bf(4, 1, 64), i32(4, 1), [64], q_weight=bf(64),
                                k_weight=torch.zeros(64)), "k_weight"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i32(4, 2), [64]), "pos"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i64(4, 1), [64]), "pos"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i32(4, 1), []), "axes"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i32(4, 1), [64], q_out=bf(4, 64, 2)), "q_out"),
        (lambda: q.qk_norm_rope(bf(4, 2, 64), None, i32(4, 1), [64]), "GPU"),
        (lambda: q.mx_kv_cache(4, 2, 16, 48, device="cpu"), "head_dim"),
        (lambda: q.mx_kv_write(bf(3, 64), bf(3, 2, 64), i64(3), cache), "k"),
        (lambda: q.mx_kv_write(bf(3, 1, 64), bf(3, 2, 64), i64(3), cache), "k"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), bf(3, 2, 32), i64(3), cache), "v"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), torch.zeros(3, 2, 64), i64(3), cache), "v"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), bf(3, 2, 64), i32(3), cache), "slots"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), bf(3, 2, 64), i64(4), cache), "slots"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), bf(3, 2, 64), i64(3), cache._replace(v_codes=u8(4, 2, 16, 31))),
         "v_codes"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), bf(3, 2, 64), i64(3), cache._replace(k_scales=u8(4, 2, 32))), "cache"),
        (lambda: q.mx_kv_write(bf(3, 2, 64), bf(3, 2, 64), i64(3), cache), "GPU"),
        (lambda: q.mx_kv_attention(bf(3, 2, 32), cache, i32(3)), "heads"),
        (lambda: q.mx_kv_attention(bf(3, 3, 64), cache, i32(3)), "heads"),
        (lambda: q.mx_kv_attention(bf(3, 64), cache, i32(3)), "q"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i64(3)), "lengths"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i32(3, 1)), "lengths"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i32(3), table=i32(2, 4)), "table"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i32(3), table=i64(3, 4)), "table"),
        (lambda: q.mx_kv_attention(bf(5, 2, 64), cache, i32(5)), "pages"),
        (lambda: q.mx_kv_attention(bf(4, 2, 64), cache, i32(3)), "evenly"),
        (lambda: q.mx_kv_attention(bf(4, 2, 64), cache, i32(3), q_starts=i32(3)), "q_starts"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i32(3), out=bf(3, 64, 2)), "out"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i32(3), lse=bf(3, 2)), "lse"),
        (lambda: q.mx_kv_attention(bf(3, 2, 64), cache, i32(3)), "GPU"),
    ]
    for call, what in cases:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError, match="lengths"):
        q.mx_kv_attention(bf(3, 2, 64), cache, [3])
    with pytest.raises(TypeError, match="q4"):
        q.rtn4_group_linear(bf(2, 64), [1], bf(4, 2))


def test_sizes_beyond_32_bits_are_refused(monkeypatch):
    """Sizes that the C calls take in 32 bits: a larger one is refused rather than cut."""
    monkeypatch.setattr(q, "_call_device", lambda *named: 0)
    far = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="meta")  # noqa: E731
    u8, d, pos = torch.uint8, 2 ** 32 + 64, torch.zeros((1, 1), dtype=torch.int32)
    cache = lambda h, p, hd: q.KVCache(*(far(1, h, p, hd // w, t=u8) for w in (2, 32, 2, 32)))  # noqa: E731
    n = torch.zeros(1, dtype=torch.int32)
    cases = [
        (lambda: q.rtn4_group_prepare_weights(far(1, d), 64), "W"),
        (lambda: q.rtn4_group_linear(far(1, d), far(1, d // 2, t=u8), far(1, d // 64)), "x"),
        (lambda: q.qk_norm_rope(far(1, d, 64), None, pos, [64]), "heads"),
        (lambda: q.qk_norm_rope(far(1, 1, 64), far(1, d, 64), pos, [64]), "heads"),
        (lambda: q.qk_norm_rope(far(1, 1, d), None, pos, [64]), "head_dim"),
        (lambda: q.qk_norm_rope(far(1, 1, 64), None, pos, [d]), "axis_dims"),
        (lambda: q.mx_kv_write(far(1, d, 64), far(1, d, 64), n.long(), cache(d, 16, 64)), "kv_heads"),
        (lambda: q.mx_kv_write(far(1, 1, 64), far(1, 1, 64), n.long(), cache(1, d, 64)), "page_size"),
        (lambda: q.mx_kv_attention(far(1, 1, d), cache(1, 1, d), n), "head_dim"),
        (lambda: q.mx_kv_attention(far(1, d, 64), cache(1, 16, 64), n), "heads"),
        (lambda: q.mx_kv_attention(far(1, 1, 64), cache(1, 16, 64), n, causal=True, window=d), "window"),
    ]
    for call, what in cases:
        with pytest.raises(ValueError, match=what + ".*32 bits"):
            call()
