"""OrbitQuant online quantized-linear path for MI355X (gfx950).

Thin Python binding over ``liborbitquant.so`` (C ABI in
``include/orbitquant.h``).  This module only marshals arguments: every step
of the path runs in the library's HIP kernels.  PyTorch supplies device
memory and the current stream, nothing else.  There is no CPU fallback: if
the library is missing or cannot run, the call raises.

Functions mirror the C entry points:

* :func:`codebook`        -> ``oq_codebook``
* :func:`rotate_quantize` -> ``oq_rotate_quantize``
* :func:`rotate`          -> ``oq_rotate_quantize`` with ``OQ_OUT_F32_ROTATED``
* :func:`fake_quantize`   -> ``oq_rotate_quantize`` with ``OQ_OUT_BF16_DEQUANT``
* :func:`prepare_weights` -> ``oq_prepare_weights``
* :func:`linear`          -> ``oq_linear``
* :func:`mx_quantize`, :func:`mx_dequantize` -> ``oq_mx_quantize``, ``oq_mx_dequantize``
* :func:`mx_linear`       -> ``oq_mx_linear``
* :func:`add_rms_norm`    -> ``oq_add_rms_norm``
* :func:`rope`            -> ``oq_rope``
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liborbitquant.so")

OQ_OK, OQ_EINVAL, OQ_EUNSUPPORTED, OQ_ENOMEM, OQ_EDEVICE = 0, -1, -2, -3, -4
OQ_F32, OQ_BF16 = 0, 1
OQ_ROT_NO_SIGNS, OQ_OUT_F32_ROTATED, OQ_OUT_BF16_DEQUANT, OQ_ROT_INPUT_PERMUTED = 1, 2, 4, 8
OQ_CODEBOOK_SPHERE = 16
OQ_MX_FP4, OQ_MX_FP8 = 4, 8
OQ_ROPE_HALF, OQ_ROPE_INVERSE = 1, 2

# every symbol the header declares, with (restype, argtypes)
_P = ctypes.c_void_p
_SIGS = {
    "oq_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "oq_version": (ctypes.c_int, []),
    "oq_codebook": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, _P, _P]),
    "oq_codes_bytes": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "oq_codebook_ex": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_uint32, _P, _P]),
    "oq_linear_ex": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, ctypes.c_int, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int, ctypes.c_uint32, _P, _P]),
    "oq_rotate_quantize": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                          ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int,
                                          _P, _P, _P]),
    "oq_prepare_weights": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                          ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int,
                                          _P, _P, _P]),
    "oq_linear": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, ctypes.c_int, ctypes.c_int64,
                                 ctypes.c_int64, ctypes.c_int, _P, _P]),
    "oq_release_plans": (ctypes.c_int, []),
    "oq_plan_create": (ctypes.c_int, [ctypes.c_int, ctypes.c_uint64, ctypes.c_uint32,
                                      ctypes.POINTER(ctypes.c_void_p)]),
    "oq_plan_destroy": (ctypes.c_int, [ctypes.c_void_p]),
    "oq_permute_rows": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_uint64,
                                       _P]),
    "oq_rtn4_prepare_weights": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                               _P, _P, _P]),
    "oq_rtn4_linear": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, _P, _P, ctypes.c_int64,
                                      ctypes.c_int, _P, _P]),
    "oq_mx_quantize": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                      _P, _P, _P]),
    "oq_mx_dequantize": (ctypes.c_int, [_P, _P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                        ctypes.c_int, _P, _P]),
    "oq_mx_linear": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, ctypes.c_int, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int, _P, _P]),
    "oq_add_rms_norm": (ctypes.c_int, [_P, _P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                       ctypes.c_float, _P, _P, _P, _P, ctypes.c_int,
                                       ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int, _P, _P,
                                       _P]),
    "oq_rope": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                               ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int, _P,
                               ctypes.c_double, ctypes.c_uint32, _P, ctypes.c_int64,
                               ctypes.c_int64, _P]),
    "oq_diag_mfma_f16": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, _P, _P]),
}

_lib = None


class OQError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


def lib():
    """The loaded ctypes library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first (python -m "
                "quantization_dit_linear_amd.build or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def strerror(status):
    return lib().oq_strerror(status).decode()


def _check(status, where):
    if status != OQ_OK:
        raise OQError(status, where)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on_device(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} lives on {t.device}, not on the current device "
                         f"cuda:{torch.cuda.current_device()}")


def _dev_ptr(t, name):
    _on_device(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _expect(t, shape, dtype, name):
    """The shape and dtype a buffer must have for the call (the library
    trusts its sizes): checked before anything touches the device."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


# ------------------------------------------------------------------- API --

def codebook(d, bits, *, sphere=False):
    """(levels float32[2^bits], thresholds float32[2^bits-1]) of C_{d,bits}
    (sphere: the exact-sphere-marginal family)."""
    L = 1 << bits
    lv = np.zeros(256, np.float32)
    th = np.zeros(256, np.float32)
    flags = OQ_CODEBOOK_SPHERE if sphere else 0
    _check(lib().oq_codebook_ex(d, bits, flags, lv.ctypes.data, th.ctypes.data), "oq_codebook_ex")
    return lv[:L].copy(), th[:L - 1].copy()


def codes_bytes(rows, d, bits):
    return lib().oq_codes_bytes(rows, d, bits)


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return OQ_BF16
    if t.dtype == torch.float32:
        return OQ_F32
    raise TypeError(f"unsupported input dtype {t.dtype} (bfloat16 or float32)")


def rotate_quantize(x, seed, bits, *, signs=True, permuted=False, sphere=False, out=None,
                    norms=None, stream=None):
    """Codes (uint8 [M, d*bits/8], storage order) and norms (float32 [M]).
    permuted=True: x's columns are already in rotation order (OQ_ROT_INPUT_PERMUTED);
    sphere=True: the exact-sphere-marginal codebook (OQ_CODEBOOK_SPHERE)."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [tokens, d]")
    M, d = x.shape
    if out is None:
        out = torch.empty((M, d * bits // 8), dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty((M,), dtype=torch.float32, device=x.device)
    _expect(out, (M, d * bits // 8), torch.uint8, "out")
    _expect(norms, (M,), torch.float32, "norms")
    flags = ((0 if signs else OQ_ROT_NO_SIGNS) | (OQ_ROT_INPUT_PERMUTED if permuted else 0)
             | (OQ_CODEBOOK_SPHERE if sphere else 0))
    rc = lib().oq_rotate_quantize(_dev_ptr(x, "x"), _dtype_code(x), M, d, seed, flags, bits,
                                  _dev_ptr(out, "out"), _dev_ptr(norms, "norms"),
                                  _stream(stream))
    _check(rc, "oq_rotate_quantize")
    return out, norms


def rotate(x, seed, *, signs=True, permuted=False, stream=None):
    """Rotated unit vectors z (float32 [M, d], coordinate order) and norms.
    bf16 tokens of the fast-path sizes run through the same kernel as the
    codes; permuted=True: x's columns are already in rotation order."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [tokens, d]")
    M, d = x.shape
    z = torch.empty((M, d), dtype=torch.float32, device=x.device)
    norms = torch.empty((M,), dtype=torch.float32, device=x.device)
    flags = (OQ_OUT_F32_ROTATED | (0 if signs else OQ_ROT_NO_SIGNS)
             | (OQ_ROT_INPUT_PERMUTED if permuted else 0))
    rc = lib().oq_rotate_quantize(_dev_ptr(x, "x"), _dtype_code(x), M, d, seed, flags, 4,
                                  _dev_ptr(z, "z"), _dev_ptr(norms, "norms"), _stream(stream))
    _check(rc, "oq_rotate_quantize")
    return z, norms


def fake_quantize(x, seed, bits, *, signs=True, sphere=False, out=None, norms=None,
                  stream=None):
    """Dequantized rotated rows (bfloat16 [M, d], coordinate order): row m,
    coordinate i holds s_m * C_{d,bits}[code_mi]; and the norms.  Works for
    activation tokens and weight rows alike (the same quantizer); a bf16 GEMM
    of two such matrices with the same seed is the fake-quantized product."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [rows, d]")
    M, d = x.shape
    if out is None:
        out = torch.empty((M, d), dtype=torch.bfloat16, device=x.device)
    if norms is None:
        norms = torch.empty((M,), dtype=torch.float32, device=x.device)
    _expect(out, (M, d), torch.bfloat16, "out")
    _expect(norms, (M,), torch.float32, "norms")
    flags = (OQ_OUT_BF16_DEQUANT | (0 if signs else OQ_ROT_NO_SIGNS)
             | (OQ_CODEBOOK_SPHERE if sphere else 0))
    rc = lib().oq_rotate_quantize(_dev_ptr(x, "x"), _dtype_code(x), M, d, seed, flags, bits,
                                  _dev_ptr(out, "out"), _dev_ptr(norms, "norms"),
                                  _stream(stream))
    _check(rc, "oq_rotate_quantize")
    return out, norms


def prepare_weights(W, seed, bits, *, signs=True, sphere=False, out=None, norms=None,
                    stream=None):
    """Weight codes (uint8 [N, K*bits/8]) and row norms (float32 [N])."""
    import torch
    if W.dim() != 2:
        raise ValueError("W must be [d_out, d_in]")
    N, K = W.shape
    if out is None:
        out = torch.empty((N, K * bits // 8), dtype=torch.uint8, device=W.device)
    if norms is None:
        norms = torch.empty((N,), dtype=torch.float32, device=W.device)
    _expect(out, (N, K * bits // 8), torch.uint8, "out")
    _expect(norms, (N,), torch.float32, "norms")
    flags = (0 if signs else OQ_ROT_NO_SIGNS) | (OQ_CODEBOOK_SPHERE if sphere else 0)
    rc = lib().oq_prepare_weights(_dev_ptr(W, "W"), _dtype_code(W), N, K, seed, flags, bits,
                                  _dev_ptr(out, "w_codes"), _dev_ptr(norms, "row_norms"),
                                  _stream(stream))
    _check(rc, "oq_prepare_weights")
    return out, norms


def linear(a_codes, a_norms, a_bits, w_codes, w_norms, w_bits, K, *, sphere=False, out=None,
           stream=None):
    """bf16 y [M, N] = s_m r_n sum_k C_w[p_nk] C_a[q_mk] (sphere: the
    exact-sphere-marginal codebooks, oq_linear_ex)."""
    import torch
    if a_codes.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("a_codes and w_codes must be [rows, K*bits/8]")
    M = a_codes.shape[0]
    N = w_codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_codes.device)
    _expect(a_codes, (M, K * a_bits // 8), torch.uint8, "a_codes")
    _expect(w_codes, (N, K * w_bits // 8), torch.uint8, "w_codes")
    _expect(a_norms, (M,), torch.float32, "a_norms")
    _expect(w_norms, (N,), torch.float32, "w_norms")
    _expect(out, (M, N), torch.bfloat16, "out")
    if sphere:
        rc = lib().oq_linear_ex(_dev_ptr(a_codes, "a_codes"), _dev_ptr(a_norms, "a_norms"),
                                a_bits, _dev_ptr(w_codes, "w_codes"), _dev_ptr(w_norms, "w_norms"),
                                w_bits, M, N, K, OQ_CODEBOOK_SPHERE, _dev_ptr(out, "y"),
                                _stream(stream))
    else:
        rc = lib().oq_linear(_dev_ptr(a_codes, "a_codes"), _dev_ptr(a_norms, "a_norms"), a_bits,
                             _dev_ptr(w_codes, "w_codes"), _dev_ptr(w_norms, "w_norms"), w_bits,
                             M, N, K, _dev_ptr(out, "y"), _stream(stream))
    _check(rc, "oq_linear")
    return out


def rtn4_prepare_weights(W, *, out=None, scales=None, stream=None):
    """INT4 weight-only RTN of the AdaLN projection weights W [N, K]:
    (uint8 [N, K/2] offset-binary nibbles, float32 scales [N])."""
    import torch
    N, K = W.shape
    if out is None:
        out = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N,), dtype=torch.float32, device=W.device)
    _expect(out, (N, K // 2), torch.uint8, "out")
    _expect(scales, (N,), torch.float32, "scales")
    rc = lib().oq_rtn4_prepare_weights(_dev_ptr(W, "W"), _dtype_code(W), N, K,
                                       _dev_ptr(out, "q4"), _dev_ptr(scales, "scales"),
                                       _stream(stream))
    _check(rc, "oq_rtn4_prepare_weights")
    return out, scales


def rtn4_linear(x, q4, scales, *, out=None, stream=None):
    """bf16 y [M, N] = scale_n sum_k x_mk q_nk (AdaLN projection)."""
    import torch
    M, K = x.shape
    N = q4.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _expect(q4, (N, K // 2), torch.uint8, "q4")
    _expect(scales, (N,), torch.float32, "scales")
    _expect(out, (M, N), torch.bfloat16, "out")
    rc = lib().oq_rtn4_linear(_dev_ptr(x, "x"), _dtype_code(x), M, _dev_ptr(q4, "q4"),
                              _dev_ptr(scales, "scales"), N, K, _dev_ptr(out, "y"),
                              _stream(stream))
    _check(rc, "oq_rtn4_linear")
    return out


# ------------------------------------------------- the microscaled path --
#
# Calls of a few microseconds: the checks below are the ones above, written for
# the case that passes (the slow forms name what is wrong).

_MX = {"fp4": OQ_MX_FP4, "fp8": OQ_MX_FP8}
_C_INTS = [ctypes.c_int * n for n in range(5)]
_T = None  # torch, from the first call on


def _torch():
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


def _mx(fmt, name="fmt"):
    try:
        return _MX[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be 'fp4' or 'fp8' (got {fmt!r})") from None


def _empty(shape, dtype, like, stream):
    """A fresh output beside `like`, owned by the stream that the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _torch().cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _shaped(t, shape, dtype, name):
    try:
        if t.shape == shape and t.dtype == dtype:
            return
    except AttributeError:
        pass
    _expect(t, shape, dtype, name)


def _call_device(*named):
    """The current device's index; every (tensor, name) must live there."""
    tensor, dev = _torch().Tensor, -1
    for t, name in named:
        if t is None:
            continue
        if not isinstance(t, tensor) or not t.is_cuda:
            _on_device(t, name)
        if dev < 0:
            dev = _T.cuda.current_device()
        if t.get_device() != dev:
            _on_device(t, name)
    return dev


def _fits(size, what):
    """Sizes that the C call takes as an int (ctypes would cut a larger one)."""
    if size > 2147483647:
        raise ValueError(f"{what} ({size}) must fit 32 bits")


def _ptr(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _strided_ptr(t, name):
    """Device pointer of a tensor whose last dimension is dense (the other
    strides are the call's arguments)."""
    if t.stride(-1) != 1 and t.numel():
        raise ValueError(f"{name} must be dense in its last dimension")
    return t.data_ptr()


def _raw_stream(stream, dev):
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream belongs to {stream.device}, not to the current device cuda:{dev}")
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _element(t):
    """OQ_F32 or OQ_BF16."""
    dtype = t.dtype
    return OQ_BF16 if dtype is _torch().bfloat16 else OQ_F32 if dtype is _T.float32 else _dtype_code(t)


def _check_mx_outputs(codes, scales, rows, d, bits):
    if codes is not None:
        _shaped(codes, (rows, d * bits // 8), _torch().uint8, "codes")
    if scales is not None:
        _shaped(scales, (rows, d // 32), _torch().uint8, "scales")


def _mx_outputs(codes, scales, rows, d, bits, like, stream):
    if codes is None:
        codes = _empty((rows, d * bits // 8), _T.uint8, like, stream)
    if scales is None:
        scales = _empty((rows, d // 32), _T.uint8, like, stream)
    return codes, scales


def _mx_pair(codes, scales, bits, codes_name, scales_name):
    """(rows, d) of a pair of MX arrays, whose shapes must agree."""
    torch = _torch()
    for t, n in ((codes, codes_name), (scales, scales_name)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if t.dim() != 2 or t.dtype is not torch.uint8:
            raise ValueError(f"{n} must be two-dimensional, of dtype torch.uint8")
    rows, d = scales.shape
    d *= 32
    _fits(d, codes_name + "'s row length")
    if codes.shape != (rows, d * bits // 8):
        _expect(codes, (rows, d * bits // 8), torch.uint8, codes_name)
    return rows, d


def mx_quantize(x, fmt, *, codes=None, scales=None, stream=None):
    """MX codes (uint8 [rows, d/2] for 'fp4', [rows, d] for 'fp8') and e8m0
    scale bytes (uint8 [rows, d/32]) of x [rows, d] (bfloat16 or float32):
    activations and weights alike."""
    bits = _mx(fmt)
    if x.dim() != 2:
        raise ValueError("x must be [rows, d]")
    rows, d = x.shape
    _fits(d, "x's row length")
    _check_mx_outputs(codes, scales, rows, d, bits)
    dev = _call_device((x, "x"), (codes, "codes"), (scales, "scales"))
    codes, scales = _mx_outputs(codes, scales, rows, d, bits, x, stream)
    rc = lib().oq_mx_quantize(_ptr(x, "x"), _element(x), rows, d, bits, _ptr(codes, "codes"),
                              _ptr(scales, "scales"), _raw_stream(stream, dev))
    _check(rc, "oq_mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, fmt, *, dtype=None, out=None, stream=None):
    """The values [rows, d] that MX codes stand for (bfloat16 unless dtype or
    out says float32)."""
    bits = _mx(fmt)
    rows, d = _mx_pair(codes, scales, bits, "codes", "scales")
    if out is not None:
        _shaped(out, (rows, d), dtype or out.dtype, "out")
    dev = _call_device((codes, "codes"), (scales, "scales"), (out, "out"))
    if out is None:
        out = _empty((rows, d), dtype or _T.bfloat16, codes, stream)
    rc = lib().oq_mx_dequantize(_ptr(codes, "codes"), _ptr(scales, "scales"), bits, rows, d,
                                _element(out), _ptr(out, "out"), _raw_stream(stream, dev))
    _check(rc, "oq_mx_dequantize")
    return out


def mx_linear(a_codes, a_scales, a_fmt, w_codes, w_scales, w_fmt, *, out=None, stream=None):
    """bf16 y [M, N] = A W^T of MX activations [M, K] and weights [N, K]."""
    a_bits, w_bits = _mx(a_fmt, "a_fmt"), _mx(w_fmt, "w_fmt")
    M, K = _mx_pair(a_codes, a_scales, a_bits, "a_codes", "a_scales")
    N, Kw = _mx_pair(w_codes, w_scales, w_bits, "w_codes", "w_scales")
    if K != Kw:
        raise ValueError(f"activations have {K} columns, weights {Kw}")
    if out is not None:
        _shaped(out, (M, N), _T.bfloat16, "out")
    dev = _call_device((a_codes, "a_codes"), (a_scales, "a_scales"), (w_codes, "w_codes"),
                       (w_scales, "w_scales"), (out, "out"))
    if out is None:
        out = _empty((M, N), _T.bfloat16, a_codes, stream)
    rc = lib().oq_mx_linear(_ptr(a_codes, "a_codes"), _ptr(a_scales, "a_scales"), a_bits,
                            _ptr(w_codes, "w_codes"), _ptr(w_scales, "w_scales"), w_bits, M, N, K,
                            _ptr(out, "out"), _raw_stream(stream, dev))
    _check(rc, "oq_mx_linear")
    return out


def add_rms_norm(x, residual=None, *, weight=None, gate=None, scale=None, shift=None,
                 rows_per_mod=None, eps=1e-6, fmt=None, sum_out=None, out=None, scales_out=None,
                 stream=None):
    """h = residual + gate * x and y = h / rms(h) * weight * (1 + scale) + shift.

    x, residual: [rows, d], bfloat16 or float32.  weight [d]; gate, scale and
    shift [groups, d] (or [d]) with one common row stride, row r taking group
    r // rows_per_mod (by default the rows split evenly); all parameters of one
    type, bfloat16 or float32.  Returns (h, y), or with fmt 'fp4' / 'fp8'
    (h, codes, scales): y in MX codes.  sum_out (for h) and out may be x or
    residual themselves; sum_out=False computes no h and returns None for it.
    """
    if x.dim() != 2:
        raise ValueError("x must be [rows, d]")
    rows, d = x.shape
    _fits(d, "x's row length")
    if residual is not None:
        _shaped(residual, (rows, d), x.dtype, "residual")
    first, groups, stride, mods = None, 1, d, False
    for p, n in ((weight, "weight"), (gate, "gate"), (scale, "scale"), (shift, "shift")):
        if p is None:
            continue
        first = p if first is None else first
        if p.shape[-1:] != (d,) or p.dtype != first.dtype:
            raise ValueError(f"{n} must have {d} columns and the other parameters' dtype")
        if n == "weight":  # by name: one tensor may be passed as several parameters
            if p.dim() != 1:
                raise ValueError("weight must be [d]")
            continue
        if p.dim() > 2:
            raise ValueError(f"{n} must be [groups, d] or [d]")
        g, st = (1, d) if p.dim() == 1 or p.shape[0] == 1 else (p.shape[0], p.stride(0))
        if mods and (g, st) != (groups, stride):
            raise ValueError("gate, scale and shift must have the same groups and row stride")
        groups, stride, mods = g, st, True
    if rows_per_mod is None:
        rows_per_mod = max(1, -(-rows // max(1, groups)))
    if mods and (rows_per_mod < 1 or -(-rows // rows_per_mod) > groups):
        raise ValueError(f"{rows} rows at {rows_per_mod} per group need more than {groups} groups")
    if rows_per_mod > rows:  # one group: as a number that the C call's 64 bits hold
        rows_per_mod = max(1, rows)
    if sum_out is not None and sum_out is not False:
        _shaped(sum_out, (rows, d), x.dtype, "sum_out")
    bits = 0
    if fmt is not None:
        bits = _mx(fmt)
        _check_mx_outputs(out, scales_out, rows, d, bits)
    elif scales_out is not None:
        raise ValueError("scales_out needs a fmt")
    elif out is not None:
        _shaped(out, (rows, d), x.dtype, "out")
    dev = _call_device((x, "x"), (residual, "residual"), (weight, "weight"), (gate, "gate"),
                       (scale, "scale"), (shift, "shift"), (None if sum_out is False else sum_out, "sum_out"),
                       (out, "out"), (scales_out, "scales_out"))
    if sum_out is None:
        sum_out = _empty((rows, d), x.dtype, x, stream)
    elif sum_out is False:
        sum_out = None
    scales = None
    if fmt is not None:
        out, scales = _mx_outputs(out, scales_out, rows, d, bits, x, stream)
    elif out is None:
        out = _empty((rows, d), x.dtype, x, stream)
    rc = lib().oq_add_rms_norm(
        _ptr(x, "x"), None if residual is None else _ptr(residual, "residual"), _element(x),
        rows, d, eps, None if weight is None else _ptr(weight, "weight"),
        None if gate is None else _strided_ptr(gate, "gate"),
        None if scale is None else _strided_ptr(scale, "scale"),
        None if shift is None else _strided_ptr(shift, "shift"),
        OQ_F32 if first is None else _element(first), rows_per_mod, stride,
        None if sum_out is None else _ptr(sum_out, "sum_out"), bits, _ptr(out, "out"),
        None if scales is None else _ptr(scales, "scales_out"), _raw_stream(stream, dev))
    _check(rc, "oq_add_rms_norm")
    return (sum_out, out) if fmt is None else (sum_out, out, scales)


def rope(x, pos, axis_dims, *, theta=10000.0, half=False, inverse=False, out=None, stream=None):
    """Rotary embedding of x [tokens, heads, head_dim] (bfloat16 or float32, any
    16-byte strides, dense heads: a slice of a fused projection's output is
    taken as it lies) at pos int32 [tokens, axes]; axis_dims: elements of a
    head that turn with each axis (one to four).  half: pairs (j, j + R/2)
    instead of (2j, 2j+1); inverse: the opposite turn, which is the gradient.
    out may be x."""
    if x.dim() != 3:
        raise ValueError("x must be [tokens, heads, head_dim]")
    tokens, heads, hd = x.shape
    axes = len(axis_dims)
    if not 1 <= axes <= 4:
        raise ValueError(f"axis_dims must name one to four axes (got {axes})")
    if max(heads, hd, *axis_dims) > 2147483647 or min(axis_dims) < -2147483647:
        for size, what in ((heads, "heads"), (hd, "head_dim"), *((abs(v), "axis_dims") for v in axis_dims)):
            _fits(size, what)
    _shaped(pos, (tokens, axes), _torch().int32, "pos")
    if out is not None:
        _shaped(out, (tokens, heads, hd), x.dtype, "out")
    dev = _call_device((x, "x"), (pos, "pos"), (out, "out"))
    if out is None:
        out = _empty((tokens, heads, hd), x.dtype, x, stream)
    flags = (OQ_ROPE_HALF if half else 0) | (OQ_ROPE_INVERSE if inverse else 0)
    rc = lib().oq_rope(_strided_ptr(x, "x"), _element(x), tokens, heads, hd, x.stride(0),
                       x.stride(1), _ptr(pos, "pos"), axes, _C_INTS[axes](*axis_dims), theta,
                       flags, _strided_ptr(out, "out"), out.stride(0), out.stride(1),
                       _raw_stream(stream, dev))
    _check(rc, "oq_rope")
    return out


def permute_rows(src, seed, *, out=None, stream=None):
    """dst row i = src row pi(i) for the rotation permutation of (d =
    src.shape[0], seed): folds pi into a producer's output rows (any dtype)."""
    import torch
    if out is None:
        out = torch.empty_like(src)
    _expect(out, tuple(src.shape), src.dtype, "out")
    rows = src.shape[0]
    row_bytes = src[0].numel() * src.element_size() if rows else 0
    rc = lib().oq_permute_rows(_dev_ptr(src, "src"), _dev_ptr(out, "dst"), rows, row_bytes,
                               seed, _stream(stream))
    _check(rc, "oq_permute_rows")
    return out


def release_plans():
    _check(lib().oq_release_plans(), "oq_release_plans")


class Plan:
    """Explicitly owned rotation plan of (current device, d, seed): built at
    construction, its device tables freed by close() (or on leaving a
    ``with`` block) once no other handle pins them."""

    def __init__(self, d, seed, *, signs=True):
        h = ctypes.c_void_p()
        flags = 0 if signs else OQ_ROT_NO_SIGNS
        _check(lib().oq_plan_create(d, seed, flags, ctypes.byref(h)), "oq_plan_create")
        self._h = h

    def close(self):
        if self._h is not None and self._h.value:
            h, self._h = self._h, None
            _check(lib().oq_plan_destroy(h), "oq_plan_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def diag_mfma_f16(blocks, iters, sink, stream=None):
    """Enqueue the matrix-core probe (orbitquant_diag.h); returns its flop
    count.  sink: float32 CUDA tensor of at least blocks * 512 elements."""
    if sink.numel() < blocks * 512:
        raise ValueError("sink too small")
    _check(lib().oq_diag_mfma_f16(blocks, iters, _dev_ptr(sink, "sink"), _stream(stream)),
           "oq_diag_mfma_f16")
    return blocks * 8 * iters * 32 * 16384
