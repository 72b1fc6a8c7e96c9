"""Python binding of libzq (ctypes; argument marshalling only).

Every function mirrors one entry point of ``include/zq.h``: it checks the
tensors' device, dtype, shape and contiguity, passes their device pointers
and the current CUDA stream to the C ABI, and raises ``ZQError`` on a
non-zero status.  All arithmetic happens in the CUDA kernels; there is no
CPU or PyTorch fallback, and importing this module without a built
``libzq.so`` raises immediately.

``stream=`` runs a call on another stream than the current one.  Outputs that
are made by the call are then that stream's memory, as if they were made under
``torch.cuda.stream(stream)``.  What the caller passes in has to stay alive
until the stream is done with it (``Tensor.record_stream``), as for torch's own
calls.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzq.so")

ZQ_OK, ZQ_ERR_NULL, ZQ_ERR_SHAPE, ZQ_ERR_ALIGN, ZQ_ERR_UNSUPPORTED, ZQ_ERR_CUDA, ZQ_ERR_TIMEOUT = range(7)
OPT_GEMM_PATH, OPT_GEMM_BN, OPT_SPLIT_K, OPT_MAX_CTAS, OPT_CTA_PAIR = 1, 2, 3, 4, 5

EXPORTS = (
    "zq_status_str", "zq_abi_version", "zq_quantize_weights_groupwise", "zq_ln_quant",
    "zq_gemm_w8a8", "zq_gemm_w4a8", "zq_device_status", "zq_set_option", "zq_get_option",
    "zq_debug_wait_timeout", "zq_gemm_w8a8_noalloc", "zq_bias_act_quant", "zq_static_quant",
    "zq_gemm_w8a16", "zq_gemm_w4a16", "zq_launch_count", "zq_workspace_reserve",
    "zq_widen_int4_weights", "zq_quantize_weights_fp8", "zq_ln_quant_fp8", "zq_bias_act_quant_fp8",
    "zq_gemm_fp8", "zq_qk_norm_rope", "zq_rope_frequencies",
)


class ZQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} ({status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libzq.so is not built ({LIB_PATH}); run "
                          "`python -m int4_quantized_transformer_b200.build` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    sig = {
        "zq_status_str": ([I], ctypes.c_char_p),
        "zq_abi_version": ([], I),
        "zq_quantize_weights_groupwise": ([P, I, I, I, I, P, P, P], I),
        "zq_ln_quant": ([P, P, P, I, I, F, P, P, P, P], I),
        "zq_gemm_w8a8": ([P, P, P, P, I, P, I, I, I, P, P, P], I),
        "zq_gemm_w4a8": ([P, P, P, P, I, P, I, I, I, P, P, P], I),
        "zq_device_status": ([P, ctypes.POINTER(I)], I),
        "zq_set_option": ([I, I], I),
        "zq_get_option": ([I], I),
        "zq_debug_wait_timeout": ([P], I),
        "zq_gemm_w8a8_noalloc": ([P, P, P, P, I, P, I, I, I, P, P, P], I),
        "zq_bias_act_quant": ([P, P, I, I, I, P, P, P, P], I),
        "zq_static_quant": ([P, I, I, F, P, P, P], I),
        "zq_gemm_w8a16": ([P, P, P, I, P, I, I, I, P, P, P], I),
        "zq_gemm_w4a16": ([P, P, P, I, P, I, I, I, P, P, P], I),
        "zq_launch_count": ([], ctypes.c_ulonglong),
        "zq_workspace_reserve": ([ctypes.c_ulonglong], I),
        "zq_widen_int4_weights": ([P, I, I, P, P], I),
        "zq_quantize_weights_fp8": ([P, I, I, I, P, P, P], I),
        "zq_ln_quant_fp8": ([P, I, P, P, I, I, F, P, P, P, P], I),
        "zq_bias_act_quant_fp8": ([P, I, P, I, I, I, P, P, P, P], I),
        "zq_gemm_fp8": ([P, P, P, P, P, I, I, I, I, P, P], I),
        "zq_qk_norm_rope": ([P, P, I, I, I, I, F, P, P, I, I, F, P], I),
        "zq_rope_frequencies": ([I, ctypes.c_double, I, ctypes.c_double, ctypes.c_double,
                                 ctypes.c_double, I, ctypes.POINTER(F), ctypes.POINTER(F)], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def lib():
    return _lib


def status_str(s: int) -> str:
    return _lib.zq_status_str(int(s)).decode()


def abi_version() -> int:
    return _lib.zq_abi_version()


def _check(rc: int, what: str):
    if rc != ZQ_OK:
        raise ZQError(rc, what)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """A new tensor for the call's output, of the memory of the stream that
    writes it: the current stream's may still be in use by earlier work there,
    and would be given out again before `stream` has finished."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dev(t: torch.Tensor | None, dtype, shape, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def workspace_reserve(nbytes: int):
    """Grow the library workspace of the current device to nbytes now
    (zq_workspace_reserve)."""
    _check(_lib.zq_workspace_reserve(int(nbytes)), "zq_workspace_reserve")


def launch_count() -> int:
    """Kernel launches this library has issued in this process (zq_launch_count)."""
    return int(_lib.zq_launch_count())


def set_option(key: int, value: int):
    _check(_lib.zq_set_option(key, value), "zq_set_option")


def get_option(key: int) -> int:
    return _lib.zq_get_option(key)


class options:
    """Context manager that forces GEMM kernel variants (zq_set_option)."""

    def __init__(self, **kw):
        keys = {"path": OPT_GEMM_PATH, "bn": OPT_GEMM_BN, "split_k": OPT_SPLIT_K,
                "max_ctas": OPT_MAX_CTAS, "pair": OPT_CTA_PAIR}
        self.kw = {keys[k]: v for k, v in kw.items()}

    def __enter__(self):
        self.old = {k: get_option(k) for k in self.kw}
        for k, v in self.kw.items():
            set_option(k, v)
        return self

    def __exit__(self, *exc):
        for k, v in self.old.items():
            set_option(k, v)


def device_status(stream=None) -> tuple[int, int]:
    """Synchronize the stream; return (status, detail) of the device status word."""
    d = ctypes.c_int(0)
    rc = _lib.zq_device_status(_stream(stream), ctypes.byref(d))
    return rc, d.value


def quantize_weights_groupwise(W: torch.Tensor, g: int, bits: int, Wq=None, s_grp=None, stream=None):
    """Group-wise weight quantization (zq_quantize_weights_groupwise).
    Returns (Wq, s_grp): int8 [N,K] (bits 8) or uint8 [N,K/2] (bits 4), fp32 [g]."""
    N, K = W.shape
    if Wq is None:
        Wq = _empty((N, K) if bits == 8 else (N, K // 2), torch.int8 if bits == 8 else torch.uint8,
                    W.device, stream)
    if s_grp is None:
        s_grp = _empty(g, torch.float32, W.device, stream)
    wq_dtype = torch.int8 if bits == 8 else torch.uint8
    _check(_lib.zq_quantize_weights_groupwise(
        _dev(W, torch.float16, (N, K), "W"), N, K, g, bits,
        _dev(Wq, wq_dtype, (N, K) if bits == 8 else (N, K // 2), "Wq"),
        _dev(s_grp, torch.float32, (g,), "s_grp"), _stream(stream)), "zq_quantize_weights_groupwise")
    return Wq, s_grp


def ln_quant(X: torch.Tensor, gamma=None, beta=None, eps: float = 1e-5, Xq=None, s_tok=None,
             y_ln=None, stream=None):
    """Fused LayerNorm + token-wise INT8 quantization (zq_ln_quant); gamma=None
    is quant-only.  Returns (Xq int8 [T,K], s_tok fp32 [T])."""
    T, K = X.shape
    if Xq is None:
        Xq = _empty((T, K), torch.int8, X.device, stream)
    if s_tok is None:
        s_tok = _empty(T, torch.float32, X.device, stream)
    _check(_lib.zq_ln_quant(
        _dev(X, torch.float16, (T, K), "X"), _dev(gamma, torch.float16, (K,), "gamma"),
        _dev(beta, torch.float16, (K,), "beta"), T, K, float(eps),
        _dev(Xq, torch.int8, (T, K), "Xq"), _dev(s_tok, torch.float32, (T,), "s_tok"),
        _dev(y_ln, torch.float16, (T, K), "Y_ln"), _stream(stream)), "zq_ln_quant")
    return Xq, s_tok


ACT_NONE, ACT_GELU = 0, 1


def bias_act_quant(X: torch.Tensor, bias=None, act: int = ACT_NONE, Xq=None, s_tok=None, y=None,
                   stream=None):
    """Token-wise INT8 quantization fused into a bias-add (act=ACT_NONE) or a
    GeLU (act=ACT_GELU) (zq_bias_act_quant).  Returns (Xq int8 [T,K],
    s_tok fp32 [T]); y, if given, receives the fp16 activation."""
    T, K = X.shape
    if Xq is None:
        Xq = _empty((T, K), torch.int8, X.device, stream)
    if s_tok is None:
        s_tok = _empty(T, torch.float32, X.device, stream)
    _check(_lib.zq_bias_act_quant(
        _dev(X, torch.float16, (T, K), "X"), _dev(bias, torch.float16, (K,), "bias"), T, K,
        int(act), _dev(Xq, torch.int8, (T, K), "Xq"), _dev(s_tok, torch.float32, (T,), "s_tok"),
        _dev(y, torch.float16, (T, K), "Y_act"), _stream(stream)), "zq_bias_act_quant")
    return Xq, s_tok


def static_quant(X: torch.Tensor, amax: float, Xq=None, s_tok=None, stream=None):
    """Static (per-tensor) INT8 quantization with a calibrated range amax
    (zq_static_quant).  Returns (Xq int8 [T,K], s_tok fp32 [T] = amax/127)."""
    T, K = X.shape
    if Xq is None:
        Xq = _empty((T, K), torch.int8, X.device, stream)
    if s_tok is None:
        s_tok = _empty(T, torch.float32, X.device, stream)
    _check(_lib.zq_static_quant(
        _dev(X, torch.float16, (T, K), "X"), T, K, float(amax), _dev(Xq, torch.int8, (T, K), "Xq"),
        _dev(s_tok, torch.float32, (T,), "s_tok"), _stream(stream)), "zq_static_quant")
    return Xq, s_tok


def _gemm(fn, what, Xq, s_tok, Wq, s_grp, bias, N, Y, acc, stream, bits):
    T, K = Xq.shape
    g = s_grp.shape[0]
    if Y is None:
        Y = _empty((T, N), torch.float16, Xq.device, stream)
    wshape = (N, K) if bits == 8 else (N, K // 2)
    _check(fn(
        _dev(Xq, torch.int8, (T, K), "Xq"), _dev(s_tok, torch.float32, (T,), "s_tok"),
        _dev(Wq, torch.int8 if bits == 8 else torch.uint8, wshape, "Wq"),
        _dev(s_grp, torch.float32, (g,), "s_grp"), g, _dev(bias, torch.float16, (N,), "bias"),
        T, N, K, _dev(Y, torch.float16, (T, N), "Y"), _dev(acc, torch.int32, (T, N), "acc_dbg"),
        _stream(stream)), what)
    return Y


def gemm_w8a8(Xq, s_tok, Wq, s_grp, bias=None, Y=None, acc_dbg=None, stream=None):
    """Y = fp16(((acc * s_tok) * s_grp[group]) + bias), acc = Xq Wq^T in int32."""
    return _gemm(_lib.zq_gemm_w8a8, "zq_gemm_w8a8", Xq, s_tok, Wq, s_grp, bias, Wq.shape[0], Y,
                 acc_dbg, stream, 8)


def gemm_w4a8(Xq, s_tok, Wq4, s_grp, bias=None, Y=None, acc_dbg=None, stream=None):
    """As gemm_w8a8 with packed INT4 weights uint8 [N, K/2]."""
    return _gemm(_lib.zq_gemm_w4a8, "zq_gemm_w4a8", Xq, s_tok, Wq4, s_grp, bias, Wq4.shape[0], Y,
                 acc_dbg, stream, 4)


def widen_int4_weights(Wq4, K: int, Wq8=None, stream=None):
    """Packed INT4 codes uint8 [N, K/2] -> int8 codes [N, K] (zq_widen_int4_weights)."""
    N = Wq4.shape[0]
    if Wq8 is None:
        Wq8 = _empty((N, K), torch.int8, Wq4.device, stream)
    _check(_lib.zq_widen_int4_weights(
        _dev(Wq4, torch.uint8, (N, K // 2), "Wq4"), N, K, _dev(Wq8, torch.int8, (N, K), "Wq8"),
        _stream(stream)), "zq_widen_int4_weights")
    return Wq8


def gemm_w8a8_noalloc(Xq, s_tok, Wq, s_grp, bias=None, Y=None, acc_dbg=None, stream=None):
    """gemm_w8a8 without any device allocation by the library: the split-K
    scratch comes from a fixed array in device memory (zq_gemm_w8a8_noalloc)."""
    return _gemm(_lib.zq_gemm_w8a8_noalloc, "zq_gemm_w8a8_noalloc", Xq, s_tok, Wq, s_grp, bias,
                 Wq.shape[0], Y, acc_dbg, stream, 8)


def _gemm_a16(fn, what, X, Wq, s_grp, bias, N, Y, acc, stream, bits):
    T, K = X.shape
    g = s_grp.shape[0]
    if Y is None:
        Y = _empty((T, N), torch.float16, X.device, stream)
    wshape = (N, K) if bits == 8 else (N, K // 2)
    _check(fn(
        _dev(X, torch.float16, (T, K), "X"),
        _dev(Wq, torch.int8 if bits == 8 else torch.uint8, wshape, "Wq"),
        _dev(s_grp, torch.float32, (g,), "s_grp"), g, _dev(bias, torch.float16, (N,), "bias"),
        T, N, K, _dev(Y, torch.float16, (T, N), "Y"), _dev(acc, torch.float32, (T, N), "acc_dbg"),
        _stream(stream)), what)
    return Y


def gemm_w8a16(X, Wq, s_grp, bias=None, Y=None, acc_dbg=None, stream=None):
    """FP16 activations, INT8 weights: Y = fp16(acc * s_grp[group] + bias),
    acc = X Wq^T accumulated in fp32 on the tensor cores."""
    return _gemm_a16(_lib.zq_gemm_w8a16, "zq_gemm_w8a16", X, Wq, s_grp, bias, Wq.shape[0], Y,
                     acc_dbg, stream, 8)


def gemm_w4a16(X, Wq4, s_grp, bias=None, Y=None, acc_dbg=None, stream=None):
    """As gemm_w8a16 with packed INT4 weights uint8 [N, K/2]."""
    return _gemm_a16(_lib.zq_gemm_w4a16, "zq_gemm_w4a16", X, Wq4, s_grp, bias, Wq4.shape[0], Y,
                     acc_dbg, stream, 4)


# ------------------------------------------------- block-scaled FP8 (e4m3)
#
# The calls below serve single tokens too, where a kernel takes two or three
# microseconds: their checks take one fast path per tensor, and build the
# message of a refusal only when there is one.

FP8 = torch.float8_e4m3fn
FP8_BLOCK = 128
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}  # zq_dtype
_F32, _I32 = torch.float32, torch.int32
_MOST = 2**31 - 1  # the sizes are C ints
# the plain getters behind torch.cuda.current_device() and current_stream()
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)
# (shape, strides, dtype) -> a new tensor on the current device: torch's own
# short way there where it has one (0.8 us instead of 1.7)
_new = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None) \
    or (lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype, device="cuda"))


def _raw(stream, dev: int) -> int:
    """The handle of the stream to run on, which has to be one of the current
    device `dev`; None is that device's current stream."""
    if stream is None:
        return _current_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream must be on the current device cuda:{dev}, got {stream.device}")
    return stream.cuda_stream


def _out(shape, strides, dtype, dev, stream):
    """A new tensor on the current device `dev` for the call's output (_empty)."""
    if stream is None:
        return _new(shape, strides, dtype)
    _raw(stream, dev)
    with torch.cuda.stream(stream):
        return _new(shape, strides, dtype)


def _ptr(t, dtype, shape, name: str, dev: int):
    """The data pointer of a contiguous tensor of this dtype and shape on the
    current device `dev` (the kernels run there); None stays None."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.get_device() == dev):
        return t.data_ptr()
    _dev(t, dtype, shape, name)
    raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")


def _matrix(t, name: str):
    """(pointer, zq_dtype, rows, columns, device) of a 16-bit matrix."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(shape)}")
    if shape[0] > _MOST or shape[1] > _MOST:
        raise ValueError(f"{name} is too large: {tuple(shape)}")
    dev = _current_device()
    if not t.is_contiguous() or t.get_device() != dev:
        _ptr(t, t.dtype, shape, name, dev)
    return t.data_ptr(), d, shape[0], shape[1], dev


def _fp8_out(rows, cols, scale_rows, Xq, s_blk, dev, stream):
    """Codes and scales (made where not given) and their pointers."""
    kb = -(-cols // FP8_BLOCK)
    if Xq is None:
        Xq = _out((rows, cols), (cols, 1), FP8, dev, stream)
        q = Xq.data_ptr()
    else:
        q = _ptr(Xq, FP8, (rows, cols), "Xq" if rows == scale_rows else "Wq", dev)
    if s_blk is None:
        s_blk = _out((scale_rows, kb), (kb, 1), _F32, dev, stream)
        s = s_blk.data_ptr()
    else:
        s = _ptr(s_blk, _F32, (scale_rows, kb), "s_blk", dev)
    return Xq, s_blk, q, s


def quantize_weights_fp8(W: torch.Tensor, Wq=None, s_blk=None, stream=None):
    """Weights [N,K] (fp16 or bf16) to e4m3 with one scale for each 128 x 128
    block (zq_quantize_weights_fp8).  Returns (Wq float8_e4m3fn [N,K],
    s_blk fp32 [ceil(N/128), ceil(K/128)])."""
    w, dt, N, K, dev = _matrix(W, "W")
    Wq, s_blk, q, s = _fp8_out(N, K, -(-N // FP8_BLOCK), Wq, s_blk, dev, stream)
    rc = _lib.zq_quantize_weights_fp8(
        w, dt, N, K, q, s, _raw(stream, dev))
    if rc:
        _check(rc, "zq_quantize_weights_fp8")
    return Wq, s_blk


def ln_quant_fp8(X: torch.Tensor, gamma=None, beta=None, eps: float = 1e-5, Xq=None, s_blk=None,
                 y_ln=None, stream=None):
    """Fused LayerNorm + e4m3 quantization of token rows with one scale for
    each 128 values (zq_ln_quant_fp8); gamma=None is quant-only.  X, gamma,
    beta and y_ln share one dtype, fp16 or bf16.  Returns (Xq float8_e4m3fn
    [T,K], s_blk fp32 [T, ceil(K/128)])."""
    x, dt, T, K, dev = _matrix(X, "X")
    e = X.dtype
    g = None if gamma is None else _ptr(gamma, e, (K,), "gamma", dev)
    b = None if beta is None else _ptr(beta, e, (K,), "beta", dev)
    y = None if y_ln is None else _ptr(y_ln, e, (T, K), "Y_ln", dev)
    Xq, s_blk, q, s = _fp8_out(T, K, T, Xq, s_blk, dev, stream)
    rc = _lib.zq_ln_quant_fp8(x, dt, g, b, T, K, eps, q, s, y,
                              _raw(stream, dev))
    if rc:
        _check(rc, "zq_ln_quant_fp8")
    return Xq, s_blk


def bias_act_quant_fp8(X: torch.Tensor, bias=None, act: int = ACT_NONE, Xq=None, s_blk=None, y=None,
                       stream=None):
    """e4m3 quantization of token rows fused into a bias-add (act=ACT_NONE) or
    a bias-add and GeLU (act=ACT_GELU) (zq_bias_act_quant_fp8).  Returns as
    ln_quant_fp8; y, if given, receives the activation."""
    x, dt, T, K, dev = _matrix(X, "X")
    b = None if bias is None else _ptr(bias, X.dtype, (K,), "bias", dev)
    ya = None if y is None else _ptr(y, X.dtype, (T, K), "Y_act", dev)
    Xq, s_blk, q, s = _fp8_out(T, K, T, Xq, s_blk, dev, stream)
    rc = _lib.zq_bias_act_quant_fp8(x, dt, b, T, K, act, q, s, ya,
                                    _raw(stream, dev))
    if rc:
        _check(rc, "zq_bias_act_quant_fp8")
    return Xq, s_blk


def gemm_fp8(Xq, s_x, Wq, s_w, bias=None, Y=None, out_dtype=torch.float16, stream=None):
    """Y = (s_x Xq) (s_w Wq)^T + bias on block-scaled e4m3 codes
    (zq_gemm_fp8); Y and bias are of out_dtype, fp16 or bf16."""
    dt = _DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError(f"out_dtype must be torch.float16 or torch.bfloat16, got {out_dtype}")
    if not (isinstance(Xq, torch.Tensor) and isinstance(Wq, torch.Tensor) and Xq.is_cuda):
        raise TypeError("Xq and Wq must be CUDA tensors")
    xs, ws = Xq.shape, Wq.shape
    if len(xs) != 2 or len(ws) != 2:
        raise ValueError(f"Xq and Wq must have two dimensions, got {tuple(xs)} and {tuple(ws)}")
    T, K = xs
    N = ws[0]
    if T > _MOST or K > _MOST or N > _MOST:
        raise ValueError(f"Xq or Wq is too large: {tuple(xs)} and {tuple(ws)}")
    kb, dev = -(-K // FP8_BLOCK), _current_device()
    x, sx = _ptr(Xq, FP8, xs, "Xq", dev), _ptr(s_x, _F32, (T, kb), "s_x", dev)
    w, sw = _ptr(Wq, FP8, (N, K), "Wq", dev), _ptr(s_w, _F32, (-(-N // FP8_BLOCK), kb), "s_w", dev)
    b = None if bias is None else _ptr(bias, out_dtype, (N,), "bias", dev)
    if Y is None:
        Y = _out((T, N), (N, 1), out_dtype, dev, stream)
        y = Y.data_ptr()
    else:
        y = _ptr(Y, out_dtype, (T, N), "Y", dev)
    rc = _lib.zq_gemm_fp8(x, sx, w, sw, b, T, N, K, dt, y,
                          _raw(stream, dev))
    if rc:
        _check(rc, "zq_gemm_fp8")
    return Y


# ------------------------------------------- query/key norm and rotation

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_BANDS, ROPE_YARN = range(5)
_pack_heads = struct.Struct("@PPPPqqqqi4x").pack  # zq_heads


def rope_frequencies(R: int, base: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
                     low: float = 1.0, high: float = 32.0, trained_len: int = 0):
    """Frequencies of a rotation of R values and the factor on its cosine and
    sine (zq_rope_frequencies; host only).  Returns (inv_freq fp32 [R/2] on the
    CPU, scale): move inv_freq to the device once and keep it."""
    f = (ctypes.c_float * max(1, R // 2))()
    scale = ctypes.c_float(0.0)
    _check(_lib.zq_rope_frequencies(int(R), float(base), int(scaling), float(factor), float(low),
                                    float(high), int(trained_len), f, ctypes.byref(scale)),
           "zq_rope_frequencies")
    return torch.tensor(list(f), dtype=torch.float32), float(scale.value)


def _strided(v, shape, dtype, what, dev):
    """Token and head stride and pointer of a [T, heads, D] tensor with
    contiguous heads."""
    if not isinstance(v, torch.Tensor) or not v.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if v.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {v.dtype}")
    if v.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(v.shape)}")
    token, head, value = v.stride()
    if value != 1 and shape[2] > 1:
        raise ValueError(f"the values of a head of {what} must be contiguous")
    if v.get_device() != dev:
        raise ValueError(f"{what} must be on the current device cuda:{dev}, got {v.device}")
    # strides of dimensions of one element mean nothing and may be anything
    return token if shape[0] > 1 else 0, head if shape[1] > 1 else 0, v.data_ptr()


def _heads(t, out, weight, bias, T, D, dtype, name, dev, stream):
    """(zq_heads as bytes, out) of a strided [T, heads, D] tensor."""
    heads = 0
    if isinstance(t, torch.Tensor):
        if t.dim() != 3:
            raise ValueError(f"{name} must have shape ({T}, heads, {D}), got {tuple(t.shape)}")
        heads = t.shape[1]
    shape = (T, heads, D)
    it, ih, i = _strided(t, shape, dtype, name, dev)
    if out is None:
        ot, oh = heads * D, D
        out = _out(shape, (ot, oh, 1), dtype, dev, stream)
        o = out.data_ptr()
    else:
        ot, oh, o = _strided(out, shape, dtype, name + "_out", dev)
    w = 0 if weight is None else _ptr(weight, dtype, (D,), name + "_weight", dev)
    b = 0 if bias is None else _ptr(bias, dtype, (D,), name + "_bias", dev)
    return _pack_heads(i, o, w, b, it, ih, ot, oh, heads), out


def qk_norm_rope(q, k, positions, inv_freq, layout: int = ROPE_HALF, scale: float = 1.0,
                 norm: int = NORM_NONE, eps: float = 1e-6, q_weight=None, q_bias=None, k_weight=None,
                 k_bias=None, q_out=None, k_out=None, stream=None):
    """Norm of each query and key head and its rotation by position
    (zq_qk_norm_rope).  q [T, Hq, D] and k [T, Hk, D] (or None) are fp16 or
    bf16 with contiguous heads and any token and head strides that are
    multiples of 8, e.g. slices of a fused QKV output.  positions int32 [T] on
    the device (negative: the row is skipped), inv_freq fp32 [R/2] (R values of
    a head are rotated).  q_out=q works in place; without q_out a new tensor is
    made (its skipped rows are undefined).  Returns (q_out, k_out)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    e = q.dtype
    dt = _DTYPES.get(e)
    if dt is None:
        raise TypeError(f"q must be torch.float16 or torch.bfloat16, got {e}")
    if q.dim() != 3:
        raise ValueError(f"q must have shape (tokens, heads, head_dim), got {tuple(q.shape)}")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a tensor of one dimension")
    T, _, D = q.shape
    if T > _MOST or D > _MOST:
        raise ValueError(f"q is too large: {tuple(q.shape)}")
    half, dev = inv_freq.shape[0], _current_device()
    pos = _ptr(positions, _I32, (T,), "positions", dev)
    f = _ptr(inv_freq, _F32, (half,), "inv_freq", dev)
    if pos is None:
        raise TypeError("positions must be a CUDA tensor")
    hq, q_out = _heads(q, q_out, q_weight, q_bias, T, D, e, "q", dev, stream)
    hk = None
    if k is not None:
        hk, k_out = _heads(k, k_out, k_weight, k_bias, T, D, e, "k", dev, stream)
    rc = _lib.zq_qk_norm_rope(hq, hk, dt, T, D, norm, eps, pos, f, 2 * half, layout, scale,
                              _raw(stream, dev))
    if rc:
        _check(rc, "zq_qk_norm_rope")
    return q_out, k_out


def debug_wait_timeout(stream=None):
    _check(_lib.zq_debug_wait_timeout(_stream(stream)), "zq_debug_wait_timeout")
