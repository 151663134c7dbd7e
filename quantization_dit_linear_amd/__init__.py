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
* :func:`rtn4_group_prepare_weights`, :func:`rtn4_group_linear` -> ``oq_rtn4_group_*``
* :func:`qk_norm_rope`    -> ``oq_qk_norm_rope``
* :func:`mx_kv_write`, :func:`mx_kv_attention` -> ``oq_mx_kv_write``, ``oq_mx_kv_attention``
  (:func:`mx_kv_cache` allocates a cache for them)
"""
import collections
import ctypes
import math
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
OQ_ATTN_CAUSAL = 1

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
    "oq_rtn4_group_prepare_weights": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                                     ctypes.c_int, _P, _P, _P, ctypes.c_int, _P]),
    "oq_rtn4_group_linear": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, _P, _P, _P,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                            ctypes.c_int, _P, _P]),
    "oq_qk_norm_rope": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, _P,
                                       ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                       ctypes.c_int64, ctypes.c_int, _P, _P, ctypes.c_int,
                                       ctypes.c_float, _P, ctypes.c_int, _P, ctypes.c_double,
                                       ctypes.c_uint32, _P, ctypes.c_int64, ctypes.c_int64, _P,
                                       ctypes.c_int64, ctypes.c_int64, _P]),
    "oq_mx_kv_write": (ctypes.c_int, [_P, _P, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P, _P,
                                      _P, _P, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, _P]),
    "oq_mx_kv_attention_workspace": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                      ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                                      ctypes.c_int64]),
    "oq_mx_kv_attention": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                          ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P,
                                          ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int64, _P, _P, _P, ctypes.c_int64,
                                          ctypes.c_float, ctypes.c_uint32, ctypes.c_int, _P,
                                          ctypes.c_int64, ctypes.c_int64, _P, _P, ctypes.c_int64,
                                          _P]),
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


# ---------------------------------------------- the cached-attention path --

KVCache = collections.namedtuple("KVCache", "k_codes k_scales v_codes v_scales")


def _group_arrays(q4, scales, zeros, K):
    """(N, group) of 4-bit group weights, whose shapes must agree with K."""
    torch = _torch()
    for t, n in ((q4, "q4"), (scales, "scales")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if t.dim() != 2:
            raise ValueError(f"{n} must be two-dimensional")
    N, groups = scales.shape
    if q4.shape != (N, K // 2) or q4.dtype is not torch.uint8:
        _expect(q4, (N, K // 2), torch.uint8, "q4")
    if groups < 1 or K % groups:
        raise ValueError(f"scales has {groups} groups for {K} columns")
    if zeros is not None:
        _shaped(zeros, (N, groups), scales.dtype, "zeros")
    return N, K // groups


def rtn4_group_prepare_weights(W, group, *, zeros=False, scale_dtype=None, stream=None):
    """INT4 weights of W [N, K] (bfloat16 or float32) with a scale for every
    `group` columns: (uint8 [N, K/2], scales [N, K/group]), and with zeros=True
    zero points of the same shape as a third.  scale_dtype: bfloat16 (default)
    or float32."""
    torch = _torch()
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    _fits(K, "W's row length")
    if group < 1 or K % group:
        raise ValueError(f"group ({group}) must divide W's row length ({K})")
    dev = _call_device((W, "W"))
    scale_dtype = scale_dtype or torch.bfloat16
    q4 = _empty((N, K // 2), torch.uint8, W, stream)
    scales = _empty((N, K // group), scale_dtype, W, stream)
    zero = _empty((N, K // group), scale_dtype, W, stream) if zeros else None
    rc = lib().oq_rtn4_group_prepare_weights(_ptr(W, "W"), _element(W), N, K, group, q4.data_ptr(),
                                             scales.data_ptr(), zero.data_ptr() if zeros else None,
                                             _element(scales), _raw_stream(stream, dev))
    _check(rc, "oq_rtn4_group_prepare_weights")
    return (q4, scales, zero) if zeros else (q4, scales)


def rtn4_group_linear(x, q4, scales, zeros=None, *, out=None, stream=None):
    """bf16 y [M, N] = sum_g scales[n, g] sum_{k in g} x[m, k] (nibble[n, k] - zeros[n, g])
    for few rows x [M, K] (bfloat16 or float32); q4 uint8 [N, K/2], scales and
    zeros [N, K/group] of one type, bfloat16 or float32 (no zeros: 8)."""
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    _fits(K, "x's row length")
    N, group = _group_arrays(q4, scales, zeros, K)
    if out is not None:
        _shaped(out, (M, N), _T.bfloat16, "out")
    dev = _call_device((x, "x"), (q4, "q4"), (scales, "scales"), (zeros, "zeros"), (out, "out"))
    if out is None:
        out = _empty((M, N), _T.bfloat16, x, stream)
    rc = lib().oq_rtn4_group_linear(_ptr(x, "x"), _element(x), M, _ptr(q4, "q4"),
                                    _ptr(scales, "scales"),
                                    None if zeros is None else _ptr(zeros, "zeros"),
                                    _element(scales), group, N, K, _ptr(out, "out"),
                                    _raw_stream(stream, dev))
    _check(rc, "oq_rtn4_group_linear")
    return out


def qk_norm_rope(q, k, pos, axis_dims, *, q_weight=None, k_weight=None, eps=1e-6, theta=10000.0,
                 half=False, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [tokens, q_heads, head_dim] and k [tokens,
    k_heads, head_dim] (or None) with weights [head_dim] (or None), and the rotary
    embedding at pos int32 [tokens, axes] as :func:`rope` has it, in one pass:
    (q_out, k_out).  Strides as in rope: the slices of a fused projection's output
    are taken as they lie; q_out may be q and k_out k (in place)."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    tokens, q_heads, hd = q.shape
    axes = len(axis_dims)
    if not 1 <= axes <= 4:
        raise ValueError(f"axis_dims must name one to four axes (got {axes})")
    k_heads = 0
    if k is not None:
        k_heads = k.shape[1]
        _shaped(k, (tokens, k_heads, hd), q.dtype, "k")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need a k")
    if max(q_heads, k_heads, hd, *axis_dims) > 2147483647 or min(axis_dims) < -2147483647:
        for size, what in ((q_heads, "heads"), (k_heads, "heads"), (hd, "head_dim"),
                           *((abs(v), "axis_dims") for v in axis_dims)):
            _fits(size, what)
    _shaped(pos, (tokens, axes), _torch().int32, "pos")
    first = q_weight if q_weight is not None else k_weight
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _shaped(w, (hd,), first.dtype, n)
    for t, x, n in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if t is not None:
            _shaped(t, x.shape, x.dtype, n)
    dev = _call_device((q, "q"), (k, "k"), (pos, "pos"), (q_weight, "q_weight"),
                       (k_weight, "k_weight"), (q_out, "q_out"), (k_out, "k_out"))
    if q_out is None:
        q_out = _empty((tokens, q_heads, hd), q.dtype, q, stream)
    if k is not None and k_out is None:
        k_out = _empty((tokens, k_heads, hd), q.dtype, q, stream)
    ks = (None, 0, 0, 0) if k is None else (_strided_ptr(k, "k"), k_heads, k.stride(0), k.stride(1))
    ko = (None, 0, 0) if k is None else (_strided_ptr(k_out, "k_out"), k_out.stride(0), k_out.stride(1))
    rc = lib().oq_qk_norm_rope(
        _strided_ptr(q, "q"), q_heads, q.stride(0), q.stride(1), *ks, _element(q), tokens, hd,
        None if q_weight is None else _ptr(q_weight, "q_weight"),
        None if k_weight is None else _ptr(k_weight, "k_weight"),
        OQ_F32 if first is None else _element(first), eps, _ptr(pos, "pos"), axes,
        _C_INTS[axes](*axis_dims), theta, OQ_ROPE_HALF if half else 0, _strided_ptr(q_out, "q_out"),
        q_out.stride(0), q_out.stride(1), *ko, _raw_stream(stream, dev))
    _check(rc, "oq_qk_norm_rope")
    return q_out, k_out


def mx_kv_cache(pages, kv_heads, page_size, head_dim, *, device="cuda"):
    """An empty (zero) 4-bit key/value cache: k_codes, k_scales, v_codes, v_scales,
    uint8 [pages, kv_heads, page_size, head_dim / 2 and head_dim / 32]."""
    torch = _torch()
    if head_dim % 32:
        raise ValueError(f"head_dim ({head_dim}) must be a multiple of 32")
    shape = (pages, kv_heads, page_size)
    return KVCache(*(torch.zeros((*shape, head_dim // w), dtype=torch.uint8, device=device)
                     for w in (2, 32, 2, 32)))


def _cache_shape(cache):
    """(pages, kv_heads, page_size, head_dim) of a cache, whose arrays must agree."""
    torch = _torch()
    kc, ks, vc, vs = cache
    if not isinstance(ks, torch.Tensor):
        raise TypeError("cache must hold four torch.Tensors")
    if ks.dim() != 4:
        raise ValueError("the cache's arrays must be [pages, kv_heads, page_size, bytes]")
    shape, nb = ks.shape[:3], ks.shape[3]
    codes, scales = (*shape, 16 * nb), (*shape, nb)
    for t, want, n in ((kc, codes, "k_codes"), (ks, scales, "k_scales"), (vc, codes, "v_codes"),
                       (vs, scales, "v_scales")):
        _shaped(t, want, torch.uint8, n)
    if max(shape[1], shape[2], 32 * nb) > 2147483647:
        for size, what in ((shape[1], "kv_heads"), (shape[2], "page_size"), (32 * nb, "head_dim")):
            _fits(size, what)
    return (*shape, 32 * nb)


def mx_kv_write(k, v, slots, cache, *, stream=None):
    """Quantize k and v [tokens, kv_heads, head_dim] (bfloat16 or float32, strided
    as in rope) into the cache's slots int64 [tokens]: slot = page * page_size +
    offset; a token with a negative slot, or one past the cache, is not written."""
    pages, heads, page, hd = _cache_shape(cache)
    if k.dim() != 3:
        raise ValueError("k must be [tokens, kv_heads, head_dim]")
    tokens = k.shape[0]
    _shaped(k, (tokens, heads, hd), k.dtype, "k")
    _shaped(v, (tokens, heads, hd), k.dtype, "v")
    _shaped(slots, (tokens,), _T.int64, "slots")
    dev = _call_device((k, "k"), (v, "v"), (slots, "slots"), (cache[0], "k_codes"),
                       (cache[1], "k_scales"), (cache[2], "v_codes"), (cache[3], "v_scales"))
    rc = lib().oq_mx_kv_write(
        _strided_ptr(k, "k"), _strided_ptr(v, "v"), _element(k), tokens, k.stride(0), k.stride(1),
        v.stride(0), v.stride(1), _ptr(slots, "slots"), _ptr(cache[0], "k_codes"),
        _ptr(cache[1], "k_scales"), _ptr(cache[2], "v_codes"), _ptr(cache[3], "v_scales"), pages,
        heads, page, hd, _raw_stream(stream, dev))
    _check(rc, "oq_mx_kv_write")


def mx_kv_attention(q, cache, lengths, *, table=None, q_starts=None, scale=None, causal=False,
                    window=0, out=None, lse=False, stream=None):
    """Attention of q [tokens, q_heads, head_dim] (bfloat16 or float32, strided as
    in rope) over the cached keys and values of each query's sequence.

    lengths: int32 [batch], tokens that a sequence has in the cache (the new ones
    among them); table: int32 [batch, pages a sequence], or None where sequence b
    is page b; q_starts: int32 [batch + 1], sequence b's queries are
    q[q_starts[b]:q_starts[b + 1]], or None where every sequence has as many.
    Query i of n stands at position length - n + i; causal: it sees no later
    token, with window > 0 only the last `window`.  A query that sees none gets
    zeros.  scale: 1 / sqrt(head_dim) by default.  Returns out, or with lse=True
    (or an fp32 tensor [tokens, q_heads] for it) (out, lse): the logarithm of each
    row's sum of exponentials.  Rows behind the last sequence keep what out and
    lse hold."""
    pages, kv_heads, page, hd = _cache_shape(cache)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, head_dim]")
    tokens, q_heads, qd = q.shape
    if qd != hd or kv_heads < 1 or q_heads % kv_heads:
        raise ValueError(f"q has {q_heads} heads of {qd}, the cache {kv_heads} of {hd}")
    _fits(q_heads, "q's heads")
    _fits(abs(window), "window")
    if not isinstance(lengths, _T.Tensor):
        raise TypeError("lengths must be a torch.Tensor")
    batch = lengths.numel()
    _shaped(lengths, (batch,), _T.int32, "lengths")
    width = 1
    if table is not None:
        width = table.shape[-1]
        _shaped(table, (batch, width), _T.int32, "table")
    elif pages < batch:
        raise ValueError(f"{batch} sequences without a table need as many pages (got {pages})")
    if q_starts is not None:
        _shaped(q_starts, (batch + 1,), _T.int32, "q_starts")
    elif batch and tokens % batch:
        raise ValueError(f"{tokens} tokens do not split evenly over {batch} sequences: pass q_starts")
    if out is not None:
        _shaped(out, (tokens, q_heads, hd), q.dtype, "out")
    want_lse = lse is not None and lse is not False
    if want_lse and lse is not True:
        _shaped(lse, (tokens, q_heads), _T.float32, "lse")
    dev = _call_device((q, "q"), (cache[0], "k_codes"), (cache[1], "k_scales"),
                       (cache[2], "v_codes"), (cache[3], "v_scales"), (lengths, "lengths"),
                       (table, "table"), (q_starts, "q_starts"), (out, "out"),
                       (lse if want_lse and lse is not True else None, "lse"))
    if out is None:
        out = _empty((tokens, q_heads, hd), q.dtype, q, stream)
    if lse is True:
        lse = _empty((tokens, q_heads), _T.float32, q, stream)
    L = lib()
    need = L.oq_mx_kv_attention_workspace(tokens, q_heads, kv_heads, hd, batch, page, width)
    # of this call alone: the allocator hands it out again behind the call, in the stream's order
    space = _empty((need,), _T.uint8, q, stream) if need > 0 else None
    rc = L.oq_mx_kv_attention(
        _strided_ptr(q, "q"), _element(q), tokens, q_heads, q.stride(0), q.stride(1),
        _ptr(cache[0], "k_codes"), _ptr(cache[1], "k_scales"), _ptr(cache[2], "v_codes"),
        _ptr(cache[3], "v_scales"), pages, kv_heads, page, hd, batch, _ptr(lengths, "lengths"),
        None if q_starts is None else _ptr(q_starts, "q_starts"),
        None if table is None else _ptr(table, "table"), width,
        1.0 / math.sqrt(hd) if scale is None else scale, OQ_ATTN_CAUSAL if causal else 0, window,
        _strided_ptr(out, "out"), out.stride(0), out.stride(1),
        _ptr(lse, "lse") if want_lse else None, None if space is None else space.data_ptr(),
        max(need, 0), _raw_stream(stream, dev))
    _check(rc, "oq_mx_kv_attention")
    return (out, lse) if want_lse else out


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
