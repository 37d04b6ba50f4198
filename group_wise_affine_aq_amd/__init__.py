"""group_wise_affine_aq_amd -- group-wise affine weight-only quantization for
AMD Instinct MI355X.

Python binding over the C ABI of ``libaq.so`` (``include/aq.h``).  The
functions here only marshal torch tensors (device memory, the current HIP
stream) into the C entry points of the same names; every step of the
computation runs in the library's HIP kernels.  There is no fallback: if the
library has not been built, or a call fails, an exception is raised.

Packed weights use the layout of the pages' container ("Tutorial 10:
Quantization", s.4): codes uint32 [N, K*bits/32] (stored in torch as int32),
scales and biases fp16 [N, K/group_size].  Consumers accept biases=None
(every bias +0).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

__all__ = [
    "AQError", "lib_path", "load_library", "aq_status_string", "aq_version", "aq_codes_words",
    "aq_qweight_bytes", "aq_quantize", "aq_quantize_mse", "aq_quantize_zp", "aq_dequantize",
    "aq_embedding", "aq_qmv", "aq_qmm",
    "aq_quantized_matmul", "aq_gather_qmv", "aq_gather_qmm", "aq_gather_quantized_matmul",
    "aq_quantize_fp", "aq_dequantize_fp", "aq_qmv_fp", "aq_matmul_fp", "aq_gather_matmul_fp", "aq_qmv_fp_describe",
    "FP_MODES", "aq_kv_append", "aq_kv_read", "aq_paged_attention", "aq_paged_attention_workspace",
]

AQ_OK = 0
AQ_F32, AQ_F16, AQ_BF16 = 0, 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    """The in-tree library, or the file AQ_LIB names (the sanitizer build)."""
    return os.environ.get("AQ_LIB") or os.path.join(_HERE, "libaq.so")


class AQError(RuntimeError):
    def __init__(self, status: int, fn: str):
        msg = _lib.aq_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


class _KVCache(ctypes.Structure):
    """aq_kv_cache of include/aq.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "k_biases",
                                                "v_codes", "v_scales", "v_biases")]
                + [("num_pages", ctypes.c_int64)]
                + [(n, ctypes.c_int32) for n in ("page_size", "kv_heads", "head_dim", "group_size",
                                                 "bits", "dtype")])


_pack_kv_cache = struct.Struct("@6Pq6i").pack  # (a third of the time that the structure takes)

_lib = None


def load_library():
    """Load libaq.so (built by ``python -m group_wise_affine_aq_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libaq.so not found at {path}; build it with "
                           "`python -m group_wise_affine_aq_amd.build`")
    lib = ctypes.CDLL(path)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    sigs = {
        "aq_status_string": ([i32], ctypes.c_char_p),
        "aq_version": ([], ctypes.c_char_p),
        "aq_codes_words": ([i64, i32], i64),
        "aq_qweight_bytes": ([i64, i64, i32, i32], i64),
        "aq_quantize": ([vp, i32, i64, i64, i32, i32, vp, vp, vp, vp], i32),
        "aq_quantize_mse": ([vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, vp], i32),
        "aq_quantize_zp": ([vp, i32, i64, i64, i32, i32, vp, vp, vp, vp, vp], i32),
        "aq_qmv_describe": ([i64, i64, i64, i32, i32, i32, ctypes.c_char_p, i32], i32),
        "aq_dequantize": ([vp, vp, vp, i64, i64, i32, i32, vp, i32, vp], i32),
        "aq_embedding": ([vp, vp, vp, i64, i64, i32, i32, vp, i64, vp, i32, vp], i32),
        "aq_qmv": ([vp, i32, i64, vp, vp, vp, i64, i64, i32, i32, vp, vp], i32),
        "aq_qmm": ([vp, i32, i64, vp, vp, vp, i64, i64, i32, i32, vp, vp], i32),
        "aq_quantized_matmul": ([vp, i32, i64, vp, vp, vp, i64, i64, i32, i32, vp, vp], i32),
        "aq_gather_qmv": ([vp, i32, i64, vp, vp, vp, i64, i64, i64, vp, i32, i32, i32, vp, vp],
                          i32),
        "aq_gather_qmm": ([vp, i32, i64, vp, vp, vp, i64, i64, i64, vp, i32, i32, i32, vp, vp],
                          i32),
        "aq_gather_quantized_matmul": (
            [vp, i32, i64, vp, vp, vp, i64, i64, i64, vp, i32, i32, i32, vp, vp], i32),
        "aq_quantize_fp": ([vp, i32, i64, i64, i32, i32, vp, vp, vp], i32),
        "aq_dequantize_fp": ([vp, vp, i64, i64, i32, i32, vp, i32, vp], i32),
        "aq_qmv_fp": ([vp, i32, vp, vp, i64, i64, i32, i32, vp, vp], i32),
        "aq_matmul_fp": ([vp, i32, i64, vp, vp, i64, i64, i32, i32, vp, vp], i32),
        "aq_gather_matmul_fp": ([vp, i32, i64, vp, vp, i64, i64, i64, vp, i32, i32, i32, vp, vp],
                                i32),
        "aq_qmv_fp_describe": ([i64, i64, i32, i32, ctypes.c_char_p, i32], i32),
        "aq_kv_append": ([vp, vp, i32, i64, i64, i64, vp, vp, vp], i32),
        "aq_kv_read": ([vp, i64, vp, vp, vp, i32, vp], i32),
        "aq_paged_attention": ([vp, i32, i64, i32, i32, i64, vp, vp, i64, vp, ctypes.c_float, vp,
                                vp, i64, vp], i32),
        "aq_paged_attention_workspace": ([i64, i32, i32, i32, i32], i64),
        "aq_bench_stream_read": ([vp, i64, i32, i32, vp, vp], i32),
        "aq_bench_read_oneshot": ([vp, i64, i32, i32, vp, vp], i32),
        "aq_bench_mfma_clock": ([i32, i32, vp, vp], i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ---- host helpers -------------------------------------------------------------------
def aq_status_string(status: int) -> str:
    return load_library().aq_status_string(status).decode()


def aq_version() -> str:
    return load_library().aq_version().decode()


def aq_codes_words(K: int, bits: int) -> int:
    return int(load_library().aq_codes_words(K, bits))


def aq_qweight_bytes(N: int, K: int, group_size: int, bits: int) -> int:
    return int(load_library().aq_qweight_bytes(N, K, group_size, bits))


# ---- marshalling -----------------------------------------------------------------------
_torch_module = None
_raw_stream = None  # the current stream's handle of a device, the short way if torch has it
_dtype_codes = {}


def _torch():
    global _torch_module, _raw_stream
    if _torch_module is None:
        import torch
        _dtype_codes.update({torch.float32: AQ_F32, torch.float16: AQ_F16, torch.bfloat16: AQ_BF16})
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    _torch()
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _torch_dtype(code: int):
    torch = _torch()
    return {AQ_F32: torch.float32, AQ_F16: torch.float16, AQ_BF16: torch.bfloat16}[code]


def _dev(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(st: int, fn: str):
    if st != AQ_OK:
        raise AQError(st, fn)


# ---- device operations -------------------------------------------------------------------
def aq_quantize(w, group_size: int, bits: int, codes=None, scales=None, biases=None, stream=None):
    """Quantize W [N, K] (fp32/fp16/bf16, device) -> (codes, scales, biases)."""
    torch = _torch()
    lib = load_library()
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K * bits // 32), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // group_size), dtype=torch.float16, device=w.device)
    if biases is None:
        biases = torch.empty((N, K // group_size), dtype=torch.float16, device=w.device)
    st = lib.aq_quantize(_dev(w, "w"), _dtype_code(w), N, K, group_size, bits,
                         _dev(codes, "codes"), _dev(scales, "scales"), _dev(biases, "biases"),
                         _stream(stream))
    _check(st, "aq_quantize")
    return codes, scales, biases


def aq_qmv_describe(M: int, N: int, K: int, group_size: int, bits: int, x_dtype="f16") -> str:
    """Name and compile-time shape of the kernel aq_qmv launches for this shape."""
    lib = load_library()
    code = {"f16": AQ_F16, "bf16": AQ_BF16}[x_dtype]
    buf = ctypes.create_string_buffer(160)
    n = lib.aq_qmv_describe(M, N, K, group_size, bits, code, buf, len(buf))
    if n < 0:
        raise AQError(-1, "aq_qmv_describe")
    return buf.value.decode()


def aq_quantize_mse(w, group_size: int, bits: int, steps: int, codes=None, scales=None,
                    biases=None, stream=None):
    """Range-search quantize W [N, K] over `steps` narrowed ranges -> (codes, scales, biases)."""
    torch = _torch()
    lib = load_library()
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K * bits // 32), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // group_size), dtype=torch.float16, device=w.device)
    if biases is None:
        biases = torch.empty((N, K // group_size), dtype=torch.float16, device=w.device)
    st = lib.aq_quantize_mse(_dev(w, "w"), _dtype_code(w), N, K, group_size, bits, steps,
                             _dev(codes, "codes"), _dev(scales, "scales"), _dev(biases, "biases"),
                             _stream(stream))
    _check(st, "aq_quantize_mse")
    return codes, scales, biases


def aq_quantize_zp(w, group_size: int, bits: int, codes=None, scales=None, biases=None,
                   zeros=None, stream=None):
    """Integer-zero-point quantize W [N, K] -> (codes, scales, biases, zeros),
    zeros uint8 [N, K/group_size] with bias = -zero * scale exactly."""
    torch = _torch()
    lib = load_library()
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K * bits // 32), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // group_size), dtype=torch.float16, device=w.device)
    if biases is None:
        biases = torch.empty((N, K // group_size), dtype=torch.float16, device=w.device)
    if zeros is None:
        zeros = torch.empty((N, K // group_size), dtype=torch.uint8, device=w.device)
    st = lib.aq_quantize_zp(_dev(w, "w"), _dtype_code(w), N, K, group_size, bits,
                            _dev(codes, "codes"), _dev(scales, "scales"), _dev(biases, "biases"),
                            _dev(zeros, "zeros"), _stream(stream))
    _check(st, "aq_quantize_zp")
    return codes, scales, biases, zeros


def aq_dequantize(codes, scales, biases, group_size: int, bits: int, out_dtype=None, out=None,
                  stream=None):
    """Dequantize packed weights -> [N, K] in out_dtype (default fp16)."""
    torch = _torch()
    lib = load_library()
    N = codes.shape[0]
    K = scales.shape[1] * group_size
    if out is None:
        out = torch.empty((N, K), dtype=out_dtype or torch.float16, device=codes.device)
    st = lib.aq_dequantize(_dev(codes, "codes"), _dev(scales, "scales"), _dev(biases, "biases"),
                           N, K, group_size, bits, _dev(out, "out"), _dtype_code(out),
                           _stream(stream))
    _check(st, "aq_dequantize")
    return out


def aq_embedding(ids, codes, scales, biases, group_size: int, bits: int, out_dtype=None,
                 out=None, stream=None):
    """Quantized embedding: out[t] = dequantize(table row ids[t]); ids int32 [T]."""
    torch = _torch()
    V = codes.shape[0]
    K = scales.shape[1] * group_size
    T = ids.numel()
    if out is None:
        out = torch.empty((T, K), dtype=out_dtype or torch.float16, device=codes.device)
    st = load_library().aq_embedding(_dev(codes, "codes"), _dev(scales, "scales"),
                                     _dev(biases, "biases"), V, K, group_size, bits,
                                     _dev(ids, "ids"), T, _dev(out, "out"), _dtype_code(out),
                                     _stream(stream))
    _check(st, "aq_embedding")
    return out


def _matmul(fname, x, codes, scales, biases, group_size, bits, y, stream):
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    st = getattr(lib, fname)(_dev(x, "x"), _dtype_code(x), M, _dev(codes, "codes"),
                             _dev(scales, "scales"), _dev(biases, "biases"), N, K, group_size,
                             bits, _dev(y, "y"), _stream(stream))
    _check(st, fname)
    return y


def aq_qmv(x, codes, scales, biases, group_size: int, bits: int, y=None, stream=None):
    """y = x @ W^T for x [M <= 8, K] (decode kernels)."""
    return _matmul("aq_qmv", x, codes, scales, biases, group_size, bits, y, stream)


def aq_qmm(x, codes, scales, biases, group_size: int, bits: int, y=None, stream=None):
    """y = x @ W^T for any M (matrix-core kernel)."""
    return _matmul("aq_qmm", x, codes, scales, biases, group_size, bits, y, stream)


def aq_quantized_matmul(x, codes, scales, biases, group_size: int, bits: int, y=None,
                        stream=None):
    """y = x @ W^T with the kernel chosen per shape."""
    return _matmul("aq_quantized_matmul", x, codes, scales, biases, group_size, bits, y, stream)


def aq_gather_qmv(x, codes, scales, biases, ids, group_size: int, bits: int, y=None,
                  stream=None):
    """MoE: y[t, j, :] = x[t] @ W_{ids[t, j]}^T; codes [E, N, K*bits/32]."""
    return _gather("aq_gather_qmv", x, codes, scales, biases, ids, group_size, bits, y, stream)


def aq_gather_qmm(x, codes, scales, biases, ids, group_size: int, bits: int, y=None,
                  stream=None):
    """MoE at prefill size (matrix cores): same operation as aq_gather_qmv."""
    return _gather("aq_gather_qmm", x, codes, scales, biases, ids, group_size, bits, y, stream)


def aq_gather_quantized_matmul(x, codes, scales, biases, ids, group_size: int, bits: int, y=None,
                               stream=None):
    """MoE with the kernel chosen by routed rows per expert."""
    return _gather("aq_gather_quantized_matmul", x, codes, scales, biases, ids, group_size, bits,
                   y, stream)


def _gather(name, x, codes, scales, biases, ids, group_size, bits, y, stream):
    torch = _torch()
    lib = load_library()
    T, K = x.shape
    E, N = codes.shape[0], codes.shape[1]
    topk = ids.shape[1]
    if y is None:
        y = torch.empty((T, topk, N), dtype=x.dtype, device=x.device)
    st = getattr(lib, name)(_dev(x, "x"), _dtype_code(x), T, _dev(codes, "codes"),
                            _dev(scales, "scales"), _dev(biases, "biases"), E, N, K,
                            _dev(ids, "ids"), topk, group_size, bits, _dev(y, "y"),
                            _stream(stream))
    _check(st, name)
    return y


# ---- measurement helpers (include/aq_bench.h) ----------------------------------------------
def aq_bench_stream_read(buf, blocks: int = 512, unroll: int = 4, sink=None, stream=None):
    """Read all of the device tensor `buf` once with a plain streaming kernel."""
    torch = _torch()
    if sink is None:
        sink = torch.zeros(4, dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    st = load_library().aq_bench_stream_read(_dev(buf, "buf"), nbytes, blocks, unroll,
                                             _dev(sink, "sink"), _stream(stream))
    _check(st, "aq_bench_stream_read")
    return sink


def aq_bench_read_oneshot(buf, threads: int = 256, unroll: int = 8, sink=None, stream=None):
    """Read all of the device tensor `buf` once, every thread's loads issued up
    front, one contiguous block per workgroup."""
    torch = _torch()
    if sink is None:
        sink = torch.zeros(4, dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    st = load_library().aq_bench_read_oneshot(_dev(buf, "buf"), nbytes, threads, unroll,
                                              _dev(sink, "sink"), _stream(stream))
    _check(st, "aq_bench_read_oneshot")
    return sink


def aq_bench_mfma_clock(blocks: int, iters: int, out=None, stream=None):
    """Per-wave (shader cycles, 100 MHz ticks) of an MFMA-only loop; int64 [4*blocks, 2]."""
    torch = _torch()
    if out is None:
        out = torch.zeros((4 * blocks, 2), dtype=torch.int64, device=torch.device("cuda"))
    st = load_library().aq_bench_mfma_clock(blocks, iters, _dev(out, "out"), _stream(stream))
    _check(st, "aq_bench_mfma_clock")
    return out


# ---- block-scaled float modes ---------------------------------------------------------
# mode -> (enum value, group size, code bits).  codes uint32 [N, K*bits/32]
# (int32 in torch); scales uint8 [N, K/group]: X + 127 for the mx modes, an
# E4M3 value for nvfp4 (with the tensor scale 2^tensor_exp).
FP_MODES = {"mxfp4": (0, 32, 4), "nvfp4": (1, 16, 4), "mxfp8": (2, 32, 8)}


def aq_quantize_fp(w, mode: str, tensor_exp: int = 0, codes=None, scales=None, stream=None):
    """Quantize W [N, K] (fp32/fp16/bf16, device) in a block-scaled float mode
    -> (codes, scales)."""
    torch = _torch()
    lib = load_library()
    m, g, bits = FP_MODES[mode]
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K * bits // 32), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // g), dtype=torch.uint8, device=w.device)
    st = lib.aq_quantize_fp(_dev(w, "w"), _dtype_code(w), N, K, m, tensor_exp,
                            _dev(codes, "codes"), _dev(scales, "scales"), _stream(stream))
    _check(st, "aq_quantize_fp")
    return codes, scales


def aq_dequantize_fp(codes, scales, K: int, mode: str, tensor_exp: int = 0, out_dtype=None,
                     out=None, stream=None):
    """Block-scaled codes/scales -> W^ [N, K] in out_dtype (default fp32)."""
    torch = _torch()
    lib = load_library()
    N = codes.shape[0]
    if out is None:
        out = torch.empty((N, K), dtype=out_dtype or torch.float32, device=codes.device)
    st = lib.aq_dequantize_fp(_dev(codes, "codes"), _dev(scales, "scales"), N, K,
                              FP_MODES[mode][0], tensor_exp, _dev(out, "out"), _dtype_code(out),
                              _stream(stream))
    _check(st, "aq_dequantize_fp")
    return out


def aq_qmv_fp(x, codes, scales, mode: str, tensor_exp: int = 0, y=None, stream=None):
    """y = x @ W^T for one row x [K] (or [1, K]) in fp16/bf16 and block-scaled W [N, K]."""
    torch = _torch()
    lib = load_library()
    K = x.shape[-1]
    if x.numel() != K:
        raise ValueError("aq_qmv_fp takes one row of x")
    N = codes.shape[0]
    if y is None:
        y = torch.empty(tuple(x.shape[:-1]) + (N,), dtype=x.dtype, device=x.device)
    st = lib.aq_qmv_fp(_dev(x, "x"), _dtype_code(x), _dev(codes, "codes"), _dev(scales, "scales"),
                       N, K, FP_MODES[mode][0], tensor_exp, _dev(y, "y"), _stream(stream))
    _check(st, "aq_qmv_fp")
    return y


def aq_matmul_fp(x, codes, scales, mode: str, tensor_exp: int = 0, y=None, stream=None):
    """y = x @ W^T for x [M, K] (fp16/bf16, device) and block-scaled W [N, K]."""
    torch = _torch()
    lib = load_library()
    M, K = (1, x.shape[-1]) if x.dim() == 1 else (x.shape[0], x.shape[1])
    if x.dim() > 2:
        raise ValueError("aq_matmul_fp takes x as [K] or [M, K]")
    N = codes.shape[0]
    if y is None:
        y = torch.empty(tuple(x.shape[:-1]) + (N,), dtype=x.dtype, device=x.device)
    st = lib.aq_matmul_fp(_dev(x, "x"), _dtype_code(x), M, _dev(codes, "codes"),
                          _dev(scales, "scales"), N, K, FP_MODES[mode][0], tensor_exp,
                          _dev(y, "y"), _stream(stream))
    _check(st, "aq_matmul_fp")
    return y


def aq_gather_matmul_fp(x, codes, scales, ids, mode: str, tensor_exp: int = 0, y=None,
                        stream=None):
    """y[t, j] = x[t] @ W_{ids[t, j]}^T: x [T, K] fp16/bf16, block-scaled experts
    codes [E, N, K*bits/32] (int32), scales [E, N, K/group] (uint8), ids [T, topk]
    (int32), all on the device; y [T, topk, N] in x's dtype."""
    torch = _torch()
    lib = load_library()
    T, K = x.shape
    E, N = codes.shape[0], codes.shape[1]
    topk = ids.shape[1]
    if y is None:
        y = torch.empty((T, topk, N), dtype=x.dtype, device=x.device)
    st = lib.aq_gather_matmul_fp(_dev(x, "x"), _dtype_code(x), T, _dev(codes, "codes"),
                                 _dev(scales, "scales"), E, N, K, _dev(ids, "ids"), topk,
                                 FP_MODES[mode][0], tensor_exp, _dev(y, "y"), _stream(stream))
    _check(st, "aq_gather_matmul_fp")
    return y


def aq_qmv_fp_describe(N: int, K: int, mode: str, x_dtype="f16") -> str:
    """Name and compile-time shape of the kernel aq_qmv_fp launches."""
    lib = load_library()
    code = {"f16": AQ_F16, "bf16": AQ_BF16}[x_dtype]
    buf = ctypes.create_string_buffer(160)
    n = lib.aq_qmv_fp_describe(N, K, FP_MODES[mode][0], code, buf, len(buf))
    if n < 0:
        raise AQError(-1, "aq_qmv_fp_describe")
    return buf.value.decode()


# ---- key-value cache and attention ------------------------------------------------------
# A cache is three arrays for K and three for V: codes int32 [pages, kv_heads, page_size,
# head_dim*bits/32], scales and biases fp16 [pages, kv_heads, page_size, head_dim/group_size];
# with bits = 16 the codes are the values, fp16 or bf16 [pages, kv_heads, page_size, head_dim],
# and scales and biases are None.  A decode step makes one such call per layer, so what runs
# before the launch is kept short.
def _queue(stream, t):
    """The stream's handle; without one, that of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream
    raw = _raw_stream
    return raw(t.get_device()) if raw else _torch().cuda.current_stream(t.device).cuda_stream


_same_stream = contextlib.nullcontext()


def _its(stream):
    """What a call makes for itself is made on the stream that it runs on: cleared there, and not
    another's again before it is done with it."""
    return _same_stream if stream is None else _torch_module.cuda.stream(stream)


def _rows(t, name):
    """Device address of [tokens, heads, head_dim] rows, heads and head_dim contiguous, and the
    tokens' distance in elements."""
    stride, inner, last = t.stride()
    n, h, d = t.shape
    if last != 1 or (h > 1 and inner != d) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor, heads and head_dim contiguous")
    return t.data_ptr(), (stride if n > 1 else h * d)


def _array(t, dtype, shape, name):
    """Device address of a contiguous array of that shape (None: any)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, {dtype} expected")
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous device tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, {tuple(shape)} expected")
    return t.data_ptr()


def _kv_cache(k_codes, k_scales, k_biases, v_codes, v_scales, v_biases, group_size, bits):
    """(the bytes of a _KVCache, kv_heads, head_dim)"""
    torch = _torch()
    codes = k_codes.shape
    pages, heads, page, words = codes
    if bits == 16:
        code = _dtype_code(k_codes)
        if code == AQ_F32:
            raise TypeError("a 16-bit cache holds float16 or bfloat16")
        kind = k_codes.dtype
        return _pack_kv_cache(_array(k_codes, kind, None, "k_codes"), 0, 0,
                              _array(v_codes, kind, codes, "v_codes"), 0, 0,
                              pages, page, heads, words, 0, 16, code), heads, words
    if bits != 4 and bits != 8:
        raise AQError(-2 if 2 <= bits <= 8 else -1, "aq_kv_cache")
    dim = words * 32 // bits
    if group_size < 1 or dim % group_size or k_scales is None or v_scales is None:
        raise AQError(-1, "aq_kv_cache")
    word, half, groups = torch.int32, torch.float16, (pages, heads, page, dim // group_size)
    return _pack_kv_cache(_array(k_codes, word, None, "k_codes"),
                          _array(k_scales, half, groups, "k_scales"),
                          0 if k_biases is None else _array(k_biases, half, groups, "k_biases"),
                          _array(v_codes, word, codes, "v_codes"),
                          _array(v_scales, half, groups, "v_scales"),
                          0 if v_biases is None else _array(v_biases, half, groups, "v_biases"),
                          pages, page, heads, dim, group_size, bits, 0), heads, dim


def aq_kv_append(k, v, slots, k_codes, k_scales, k_biases, v_codes, v_scales, v_biases,
                 group_size: int, bits: int, stream=None):
    """Quantize k, v [T, kv_heads, head_dim] (fp16/bf16; tokens may be strided) into the cache at
    slots int64 [T] = page * page_size + place (outside the cache: not written)."""
    lib = load_library()
    cache, heads, dim = _kv_cache(k_codes, k_scales, k_biases, v_codes, v_scales, v_biases,
                                  group_size, bits)
    T = slots.numel()
    shape = (T, heads, dim)
    if k.shape != shape or v.shape != shape or k.dtype is not v.dtype:
        raise ValueError(f"aq_kv_append: k and v must be {shape} of one dtype")
    kp, ks = _rows(k, "k")
    vp, vs = _rows(v, "v")
    st = lib.aq_kv_append(kp, vp, _dtype_code(k), T, ks, vs,
                          _array(slots, _torch_module.int64, None, "slots"), cache,
                          _queue(stream, slots))
    if st != AQ_OK:
        raise AQError(st, "aq_kv_append")


def aq_kv_read(slots, k_codes, k_scales, k_biases, v_codes, v_scales, v_biases, group_size: int,
               bits: int, out_dtype=None, k=None, v=None, stream=None):
    """Rows of the cache at slots int64 [T] -> (k, v) [T, kv_heads, head_dim] in out_dtype
    (default fp16); a slot outside the cache gives zeros."""
    lib = load_library()
    cache, H, D = _kv_cache(k_codes, k_scales, k_biases, v_codes, v_scales, v_biases, group_size,
                            bits)
    torch = _torch_module
    T = slots.numel()
    if k is None and v is None:
        with _its(stream):
            k = torch.empty((T, H, D), dtype=out_dtype or torch.float16, device=slots.device)
            v = torch.empty_like(k)
        kp, vp = k.data_ptr(), v.data_ptr()
    else:
        if k is None:
            with _its(stream):
                k = torch.empty((T, H, D), dtype=v.dtype, device=slots.device)
        elif v is None:
            with _its(stream):
                v = torch.empty((T, H, D), dtype=k.dtype, device=slots.device)
        if k.shape != (T, H, D) or v.shape != (T, H, D):
            raise ValueError(f"aq_kv_read: k and v must be {(T, H, D)}")
        kp, vp = _array(k, k.dtype, None, "k"), _array(v, k.dtype, None, "v")
    st = lib.aq_kv_read(_array(slots, torch.int64, None, "slots"), T, cache, kp, vp,
                        _dtype_code(k), _queue(stream, slots))
    if st != AQ_OK:
        raise AQError(st, "aq_kv_read")
    return k, v


def aq_paged_attention_workspace(B: int, L: int, q_heads: int, kv_heads: int,
                                 head_dim: int) -> int:
    """Bytes of workspace aq_paged_attention needs for this shape."""
    n = int(load_library().aq_paged_attention_workspace(B, L, q_heads, kv_heads, head_dim))
    if n < 0:
        raise AQError(-1, "aq_paged_attention_workspace")
    return n


def aq_paged_attention(q, k_codes, k_scales, k_biases, v_codes, v_scales, v_biases, page_table,
                       lengths, group_size: int, bits: int, scale: float | None = None, out=None,
                       workspace=None, stream=None):
    """Attention of the newest L tokens of every sequence over the paged cache: q [B, L, q_heads,
    head_dim] or [B, q_heads, head_dim] (L = 1; tokens may be strided), page_table int32 [B,
    max_pages], lengths int32 [B] (cached tokens, the L new ones included) -> out of q's shape.
    scale: default head_dim ** -0.5.  workspace: a device buffer of
    aq_paged_attention_workspace bytes, zeroed once before its first use; without one each call
    makes and clears its own."""
    lib = load_library()
    cache, heads, dim = _kv_cache(k_codes, k_scales, k_biases, v_codes, v_scales, v_biases,
                                  group_size, bits)
    torch = _torch_module
    shape, strides = q.shape, q.stride()
    if len(shape) == 3:
        B, Hq, D = shape
        L = 1
        step, inner, last = strides
    else:
        B, L, Hq, D = shape
        outer, step, inner, last = strides
        if L == 1:
            step = outer
        elif B > 1 and outer != L * step:
            raise ValueError("q: all tokens must lie at one distance")
    if D != dim:
        raise ValueError(f"q: head_dim {D}, the cache has {dim}")
    if last != 1 or (Hq > 1 and inner != D) or not q.is_cuda:
        raise ValueError("q: a device tensor, heads and head_dim contiguous")
    if B * L == 1:
        step = Hq * D
    rows, max_pages = page_table.shape
    if rows != B or lengths.numel() != B:
        raise ValueError(f"page_table must be [{B}, max_pages], lengths [{B}]")
    if out is None:
        with _its(stream):
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = out.data_ptr()
    else:
        if out.shape != shape:
            raise ValueError("out must have q's shape and dtype")
        op = _array(out, q.dtype, None, "out")
    if workspace is None:
        need = lib.aq_paged_attention_workspace(B, L, Hq, heads, D)
        with _its(stream):
            workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=q.device)
    int32 = torch.int32
    st = lib.aq_paged_attention(q.data_ptr(), _dtype_code(q), B, L, Hq, step, cache,
                                _array(page_table, int32, None, "page_table"), max_pages,
                                _array(lengths, int32, None, "lengths"),
                                D ** -0.5 if scale is None else scale, op,
                                _array(workspace, workspace.dtype, None, "workspace"),
                                workspace.nbytes, _queue(stream, q))
    if st != AQ_OK:
        raise AQError(st, "aq_paged_attention")
    return out
