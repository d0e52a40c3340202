"""Python binding of libaria_q.so: quantized linear layers for B200 (sm_100a).

Argument marshalling only. Every step of the path -- packing, activation
quantisation, the GEMMs and their epilogue -- runs in the library's CUDA
kernels; PyTorch provides device memory and streams. There is no CPU
fallback: if the library is missing or the tensors are not on a CUDA device,
the calls raise.

Method: "A Quantized Native Runtime for On-Device Semantic Audio Generation"
(aria project page): "What aria is" (weights packed from fp16 to 8 or 4
bits), "Results" (fp16, q8, W8A8 on integer tensor cores, q4), "Steering is
real" (a direction added at one block, bit-identical at alpha = 0), "Live
steering while streaming" (the strength lives inside the captured graph) and
"Run it" (the steer spec site:block:file:alpha:steps). Formats and argument
rules are documented in include/aria_q.h.

qgemm_act, qgemm_gated and gated_backward are the feed-forward operators on
the same formats: activation, steering and residual in the GEMM's epilogue, a
gated block's two projections in one kernel, and its gradients.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libaria_q.so")

ARIA_OK = 0
STATUS = {0: "ARIA_OK", 1: "ARIA_ERR_INVALID_ARG", 2: "ARIA_ERR_UNSUPPORTED",
          3: "ARIA_ERR_MISALIGNED", 4: "ARIA_ERR_CUDA", 5: "ARIA_ERR_TIMEOUT"}
FORMATS = {"q8": 1, "q4": 2, "w8a8": 3, "f16": 4}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
API = ("aria_status_string", "aria_last_error_message", "aria_qpack_size", "aria_qpack",
       "aria_act_quant", "aria_qgemm", "aria_qgemm_steer_dev", "aria_w8a8_workspace_size",
       "aria_qgemm_w8a8_fused", "aria_qgemm_w8a8_fused_noalloc", "aria_qgemm_s32",
       "aria_qgemm_act", "aria_qgemm_gated", "aria_gated_bwd_workspace_size", "aria_gated_bwd",
       "aria_selftest_bounded_wait", "aria_device_status")


class AriaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libaria_q.so (built by ``python -m int8_int4_b200.build``)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m int8_int4_b200.build`")
    lib = ctypes.CDLL(path)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "aria_status_string": ([I], ctypes.c_char_p),
        "aria_last_error_message": ([], ctypes.c_char_p),
        "aria_qpack_size": ([I, I, I64, I64, P, P], I),
        "aria_qpack": ([I, I, P, I64, I64, P, P, P], I),
        "aria_act_quant": ([P, I64, I64, P, P, P], I),
        "aria_qgemm": ([I, I, I64, I64, I64, P, P, P, P, P, P, ctypes.c_float, P, P], I),
        "aria_qgemm_steer_dev": ([I, I, I64, I64, I64, P, P, P, P, P, P, P, P, P], I),
        "aria_w8a8_workspace_size": ([I64, I64, P], I),
        "aria_qgemm_w8a8_fused": ([I64, I64, I64, P, P, P, P, P, ctypes.c_float, P, P, P,
                                   ctypes.c_size_t, P], I),
        "aria_qgemm_w8a8_fused_noalloc": ([I64, I64, I64, P, P, P, P, P, ctypes.c_float, P, P, P], I),
        "aria_qgemm_s32": ([I64, I64, I64, P, P, P, P], I),
        "aria_qgemm_act": ([I, I, I64, I64, I64, P, P, P, P, P, I, P, P, ctypes.c_float, P, P, P], I),
        "aria_qgemm_gated": ([I, I, I64, I64, I64, P, P, P, P, P, P, P, P, I, P, P, P, P], I),
        "aria_gated_bwd_workspace_size": ([I64, I64, I64, P], I),
        "aria_gated_bwd": ([I, I64, I64, I64, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P], I),
        "aria_selftest_bounded_wait": ([I64, I64, I64, P, P, P, P, P, ctypes.c_uint32, P], I),
        "aria_device_status": ([P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int):
    if status != ARIA_OK:
        msg = load_library().aria_last_error_message().decode()
        raise AriaError(status, msg)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor | None, name: str, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def same_device(**tensors):
    """Every given tensor (None skipped) on one device; returns it. The library
    launches on the current device and encodes tensor maps from raw pointers,
    so a tensor on another GPU would be read through the wrong device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other arguments on {dev}")
    return dev


@contextlib.contextmanager
def _on(dev):
    """Make `dev` the current CUDA device for the library call."""
    if dev is not None and dev.type == "cuda":
        with torch.cuda.device(dev):
            yield
    else:
        yield


def _group(fmt: str, group):
    return (32 if fmt == "q4" else 0) if group is None else int(group)


def _expect(t, name: str, shape, dtype):
    """Shape and dtype of an argument (checked before anything reaches the device:
    the C ABI takes raw pointers and cannot see a too-small buffer)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def check_gemm_args(fmt: str, X, Wq, scales, sx=None, bias=None, steer_vec=None, out=None,
                    alpha_dev=None):
    """The tensors of one GEMM call agree with each other and with the format
    (include/aria_q.h): X [M,K] (fp16; int8 for W8A8), Wq [N,K] int8 (q8, W8A8)
    or [N,K/2] uint8 (q4) or the fp16 weight [N,K] itself (f16), scales fp32
    [N] (q8, W8A8) or fp16 [N,K/32] (q4) or None (f16), sx fp32 [M] (W8A8
    only), bias fp16 [N], steer_vec fp32 [N], alpha_dev one fp32 element,
    out fp16 [M,N], all on one device. Returns (M, N, K)."""
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    if X.dim() != 2 or Wq.dim() != 2:
        raise ValueError("X and Wq must be 2-D")
    M, K = X.shape
    N = Wq.shape[0]
    _expect(X, "X", (M, K), torch.int8 if fmt == "w8a8" else torch.float16)
    if fmt == "q4":
        if K % 32:
            raise ValueError("q4 needs K % 32 == 0")
        _expect(Wq, "Wq", (N, K // 2), torch.uint8)
        _expect(scales, "scales", (N, K // 32), torch.float16)
    elif fmt == "f16":
        _expect(Wq, "W", (N, K), torch.float16)
        if scales is not None:
            raise ValueError("f16 weights take no scales")
    else:
        _expect(Wq, "Wq", (N, K), torch.int8)
        _expect(scales, "scales", (N,), torch.float32)
    if fmt == "w8a8":
        if sx is None:
            raise ValueError("w8a8 needs sx")
        _expect(sx, "sx", (M,), torch.float32)
    elif sx is not None:
        raise ValueError("sx is for w8a8 only")
    _expect(bias, "bias", (N,), torch.float16)
    _expect(steer_vec, "steer_vec", (N,), torch.float32)
    if alpha_dev is not None:
        if alpha_dev.numel() != 1 or alpha_dev.dtype != torch.float32:
            raise TypeError("alpha_dev must be one float32 element")
    _expect(out, "out", (M, N), torch.float16)
    same_device(X=X, Wq=Wq, scales=scales, sx=sx, bias=bias, steer_vec=steer_vec, out=out,
                alpha_dev=alpha_dev)
    return M, N, K


def qpack_size(fmt: str, N: int, K: int, group=None):
    wb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().aria_qpack_size(FORMATS[fmt], _group(fmt, group), N, K,
                                          ctypes.byref(wb), ctypes.byref(sb)))
    return wb.value, sb.value


def qpack(fmt: str, W: torch.Tensor, group=None, stream=None, out=None):
    """Pack fp16 W [N,K]: q8/w8a8 -> (int8 [N,K], fp32 [N]); q4 -> (uint8 [N,K/2], fp16 [N,K/32]).
    ``out`` = (Wq, scales) writes into existing tensors of those shapes."""
    N, K = W.shape
    g = _group(fmt, group)
    qpack_size(fmt, N, K, g)
    q4 = fmt == "q4"
    shapes = ((N, K // 2), (N, K // 32)) if q4 else ((N, K), (N,))
    dtypes = (torch.uint8, torch.float16) if q4 else (torch.int8, torch.float32)
    if out is None:
        Wq = torch.empty(*shapes[0], dtype=dtypes[0], device=W.device)
        S = torch.empty(*shapes[1], dtype=dtypes[1], device=W.device)
    else:
        Wq, S = out
        _expect(Wq, "Wq", shapes[0], dtypes[0])
        _expect(S, "scales", shapes[1], dtypes[1])
        same_device(W=W, Wq=Wq, scales=S)
    with _on(W.device):
        _check(load_library().aria_qpack(FORMATS[fmt], g, _dev(W, "W", torch.float16), N, K,
                                         Wq.data_ptr(), S.data_ptr(), _stream(stream)))
    return Wq, S


def act_quant(X: torch.Tensor, out=None, stream=None):
    """Per-token int8 quantisation of fp16 X [M,K] -> (Xq int8 [M,K], s_x fp32 [M])."""
    M, K = X.shape
    Xq, sx = out if out is not None else (
        torch.empty(M, K, dtype=torch.int8, device=X.device),
        torch.empty(M, dtype=torch.float32, device=X.device))
    _expect(Xq, "Xq", (M, K), torch.int8)
    _expect(sx, "sx", (M,), torch.float32)
    dev = same_device(X=X, Xq=Xq, sx=sx)
    with _on(dev):
        _check(load_library().aria_act_quant(_dev(X, "X", torch.float16), M, K,
                                             _dev(Xq, "Xq", torch.int8), _dev(sx, "sx", torch.float32),
                                             _stream(stream)))
    return Xq, sx


def qgemm(fmt: str, X: torch.Tensor, Wq: torch.Tensor, scales, sx=None,
          bias=None, steer_vec=None, alpha: float = 0.0, group=None, out=None, stream=None,
          alpha_dev=None):
    """Y [M,N] fp16 = X . dequant(W)^T + bias + alpha*v (see include/aria_q.h).

    fmt "f16" takes the fp16 weight [N,K] as Wq and scales=None. With
    ``alpha_dev`` (one fp32 element on the device, e.g. ``schedule[s:s+1]``)
    the strength is read from device memory when the kernel runs
    (aria_qgemm_steer_dev) and ``alpha`` is ignored.

    The weight and its scales may be read before the preceding kernel in the
    stream has ended (include/aria_q.h, stream order): qpack-then-qgemm is
    safe, but where another kernel has just written them (``copy_``, an
    optimiser's update of an fp16 weight), at least one kernel must lie
    between; qgemm_act reads fp16 weights in stream order."""
    if fmt != "f16" and scales is None:
        raise ValueError(f"{fmt} needs scales")
    M, N, K = check_gemm_args(fmt, X, Wq, scales, sx, bias, steer_vec, out, alpha_dev)
    Y = out if out is not None else torch.empty(M, N, dtype=torch.float16, device=X.device)
    xdt = torch.int8 if fmt == "w8a8" else torch.float16
    lib = load_library()
    args = (FORMATS[fmt], _group(fmt, group), M, N, K, _dev(X, "X", xdt),
            _dev(sx, "sx", torch.float32), _dev(Wq, "Wq"), _dev(scales, "scales"),
            _dev(bias, "bias", torch.float16), _dev(steer_vec, "steer_vec", torch.float32))
    with _on(X.device):
        if alpha_dev is not None:
            if not alpha_dev.is_cuda:
                raise ValueError("alpha_dev must be a CUDA tensor")
            _check(lib.aria_qgemm_steer_dev(*args, alpha_dev.data_ptr(), _dev(Y, "out"),
                                            _stream(stream)))
        else:
            _check(lib.aria_qgemm(*args, float(alpha), _dev(Y, "out"), _stream(stream)))
    return Y


def w8a8_workspace_size(M: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().aria_w8a8_workspace_size(M, K, ctypes.byref(n)))
    return n.value


def w8a8_workspace(M: int, K: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for qgemm_w8a8_fused (uint8, 256-byte aligned:
    the caching allocator's blocks are)."""
    ws = torch.zeros(w8a8_workspace_size(M, K), dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise RuntimeError("workspace is not 256-byte aligned")
    return ws


def workspace_codes(ws: torch.Tensor, M: int, K: int):
    """Views of the token scales fp32 [M] and codes int8 [M,K] that a fused
    call leaves in its workspace (the layout of include/aria_q.h)."""
    sx_bytes = (4 * M + 255) // 256 * 256
    sx = ws[256:256 + 4 * M].view(torch.float32)
    xq = ws[256 + sx_bytes:256 + sx_bytes + M * K].view(torch.int8).view(M, K)
    return xq, sx


def qgemm_w8a8_fused(X: torch.Tensor, Wq: torch.Tensor, sw: torch.Tensor, bias=None, steer_vec=None,
                     alpha: float = 0.0, alpha_dev=None, out=None, workspace=None, stream=None):
    """W8A8 from fp16 X [M,K] in one launch: per-token quantisation inside the
    GEMM kernel (include/aria_q.h, aria_qgemm_w8a8_fused). ``workspace``: a
    zero-filled uint8 tensor of w8a8_workspace_size(M, K) bytes (see
    w8a8_workspace); calls sharing one must not overlap on the GPU."""
    M, K = X.shape
    N = Wq.shape[0]
    _expect(X, "X", (M, K), torch.float16)
    _expect(Wq, "Wq", (N, K), torch.int8)
    _expect(sw, "scales", (N,), torch.float32)
    _expect(bias, "bias", (N,), torch.float16)
    _expect(steer_vec, "steer_vec", (N,), torch.float32)
    if alpha_dev is not None and (alpha_dev.numel() != 1 or alpha_dev.dtype != torch.float32):
        raise TypeError("alpha_dev must be one float32 element")
    Y = out if out is not None else torch.empty(M, N, dtype=torch.float16, device=X.device)
    _expect(Y, "out", (M, N), torch.float16)
    if workspace is None:
        raise ValueError("qgemm_w8a8_fused needs a workspace (w8a8_workspace(M, K, device))")
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    same_device(X=X, Wq=Wq, scales=sw, bias=bias, steer_vec=steer_vec, out=Y, workspace=workspace,
                alpha_dev=alpha_dev)
    with _on(X.device):
        _check(load_library().aria_qgemm_w8a8_fused(
            M, N, K, _dev(X, "X", torch.float16), _dev(Wq, "Wq", torch.int8), _dev(sw, "scales"),
            _dev(bias, "bias", torch.float16), _dev(steer_vec, "steer_vec", torch.float32),
            float(alpha), None if alpha_dev is None else _dev(alpha_dev, "alpha_dev"),
            _dev(Y, "out"), _dev(workspace, "workspace"), workspace.numel(), _stream(stream)))
    return Y


def qgemm_w8a8_fused_noalloc(X: torch.Tensor, Wq: torch.Tensor, sw: torch.Tensor, bias=None,
                             steer_vec=None, alpha: float = 0.0, alpha_dev=None, out=None, stream=None):
    """qgemm_w8a8_fused with the library's static scratch instead of a
    workspace, for callers that must not allocate device memory while they
    run (include/aria_q.h, aria_qgemm_w8a8_fused_noalloc). ``out`` must be
    given: this call allocates nothing, not even its output."""
    M, K = X.shape
    N = Wq.shape[0]
    if out is None:
        raise ValueError("qgemm_w8a8_fused_noalloc allocates nothing: pass out=")
    _expect(X, "X", (M, K), torch.float16)
    _expect(Wq, "Wq", (N, K), torch.int8)
    _expect(sw, "scales", (N,), torch.float32)
    _expect(bias, "bias", (N,), torch.float16)
    _expect(steer_vec, "steer_vec", (N,), torch.float32)
    _expect(out, "out", (M, N), torch.float16)
    if alpha_dev is not None and (alpha_dev.numel() != 1 or alpha_dev.dtype != torch.float32):
        raise TypeError("alpha_dev must be one float32 element")
    same_device(X=X, Wq=Wq, scales=sw, bias=bias, steer_vec=steer_vec, out=out, alpha_dev=alpha_dev)
    with _on(X.device):
        _check(load_library().aria_qgemm_w8a8_fused_noalloc(
            M, N, K, _dev(X, "X", torch.float16), _dev(Wq, "Wq", torch.int8), _dev(sw, "scales"),
            _dev(bias, "bias", torch.float16), _dev(steer_vec, "steer_vec", torch.float32),
            float(alpha), None if alpha_dev is None else _dev(alpha_dev, "alpha_dev"),
            _dev(out, "out"), _stream(stream)))
    return out


def qgemm_s32(Xq: torch.Tensor, Wq: torch.Tensor, out=None, stream=None):
    """Raw int32 accumulators C [M,N] = Xq . Wq^T on the integer tensor cores."""
    M, K = Xq.shape
    N = Wq.shape[0]
    _expect(Wq, "Wq", (N, K), torch.int8)
    C = out if out is not None else torch.empty(M, N, dtype=torch.int32, device=Xq.device)
    _expect(C, "out", (M, N), torch.int32)
    dev = same_device(Xq=Xq, Wq=Wq, out=C)
    with _on(dev):
        _check(load_library().aria_qgemm_s32(M, N, K, _dev(Xq, "Xq", torch.int8),
                                             _dev(Wq, "Wq", torch.int8), _dev(C, "out", torch.int32),
                                             _stream(stream)))
    return C


# --------------------------------------------------- feed-forward operators --

_F16, _F32, _I8, _U8 = torch.float16, torch.float32, torch.int8, torch.uint8


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    return ACTS[act]


def _arg(t, name: str, shape: tuple, dtype, di: int):
    """Check one argument (None passes as NULL) and return its device pointer;
    `di` is the index of the call's CUDA device. A call checks up to ten: the
    common outcome is one expression."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.get_device() == di and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != di:
        raise ValueError(f"{name} is on {t.device}, the other arguments on cuda:{di}")
    raise ValueError(f"{name} must be contiguous")


def _weight_args(fmt: str, W, scales, sfx: str, N: int, K: int, di: int):
    """Pointers of one packed weight [N,K] of the given format and its scales."""
    if fmt == "f16":
        if scales is not None:
            raise ValueError("f16 weights take no scales")
        return _arg(W, "W" + sfx, (N, K), _F16, di), None
    if scales is None:
        raise ValueError(f"{fmt} needs scales")
    if fmt == "q4":
        if K % 32:
            raise ValueError("q4 needs K % 32 == 0")
        return (_arg(W, "W" + sfx, (N, K // 2), _U8, di),
                _arg(scales, "scales" + sfx, (N, K // 32), _F16, di))
    return (_arg(W, "W" + sfx, (N, K), _I8, di),
            _arg(scales, "scales" + sfx, (N,), _F32, di))


def _x_args(fmt: str, X, W, sx):
    """Sizes, device index and pointers of the activations: (M, N, K, di, X, sx)."""
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and the weights must be 2-D")
    di = X.get_device()
    if di < 0:
        raise ValueError("X must be a CUDA tensor (no CPU path exists)")
    shape = X.shape
    M, K = shape
    if fmt == "w8a8":
        if sx is None:
            raise ValueError("w8a8 needs sx")
        px = _arg(X, "X", shape, _I8, di)
        sx = _arg(sx, "sx", (M,), _F32, di)
    else:
        if sx is not None:
            raise ValueError("sx is for w8a8 only")
        px = _arg(X, "X", shape, _F16, di)
    return M, W.shape[0], K, di, px, sx


def _here(di: int, stream):
    """The current stream's handle where the call runs on it and on the current
    device, as almost every call does; None where _running_on is needed. (The
    handle without a Stream object: 0.1 instead of 3 us of a call's 9.)"""
    if stream is None and di == torch.cuda.current_device():
        return torch._C._cuda_getCurrentRawStream(di)
    return None


@contextlib.contextmanager
def _running_on(di: int, stream):
    """Device and stream of one call: yields the stream's handle. With a stream
    of the caller's, tensors that the call allocates come from that stream's
    pool, so the memory is not still in use by work on another one."""
    dev = getattr(stream, "device", None)
    if dev is not None and dev.index != di:
        raise ValueError(f"the stream belongs to {dev}, the arguments to cuda:{di}")
    with torch.cuda.device(di):
        if stream is None:
            yield torch._C._cuda_getCurrentRawStream(di)
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(
                _stream(stream), device=di)
            with torch.cuda.stream(s):
                yield s.cuda_stream


def qgemm_act(fmt: str, X: torch.Tensor, Wq: torch.Tensor, scales, sx=None, bias=None, act: str = "none",
              residual=None, steer_vec=None, alpha: float = 0.0, group=None, out=None, stream=None,
              alpha_dev=None):
    """Y [M,N] fp16 = act(X . dequant(W)^T + bias) + alpha*v + residual, in one
    kernel (include/aria_q.h, aria_qgemm_act).

    Formats and arguments as for qgemm; ``act`` is one of ACTS; ``residual``
    fp16 [M,N] may be ``out`` itself. With ``alpha_dev`` the strength is read
    from device memory and ``alpha`` is ignored. "f16" weights are read in
    stream order, so they may be written right before the call; packed weights
    follow qgemm's rule."""
    M, N, K, di, px, psx = _x_args(fmt, X, Wq, sx)
    pw, ps = _weight_args(fmt, Wq, scales, "", N, K, di)
    mn, n = (M, N), (N,)
    pb = _arg(bias, "bias", n, _F16, di)
    pr = _arg(residual, "residual", mn, _F16, di)
    pv = _arg(steer_vec, "steer_vec", n, _F32, di)
    if alpha_dev is None:
        pa = None
    elif alpha_dev.numel() != 1:
        raise ValueError("alpha_dev must be one element")
    else:
        pa = _arg(alpha_dev, "alpha_dev", alpha_dev.shape, _F32, di)
    a, g, f = _act(act), _group(fmt, group), FORMATS[fmt]
    po = _arg(out, "out", mn, _F16, di)
    fn = load_library().aria_qgemm_act
    raw = _here(di, stream)
    if raw is not None:
        if out is None:
            out = torch.empty(mn, dtype=_F16, device=X.device)
            po = out.data_ptr()
        st = fn(f, g, M, N, K, px, psx, pw, ps, pb, a, pr, pv, alpha, pa, po, raw)
    else:
        with _running_on(di, stream) as raw:
            if out is None:
                out = torch.empty(mn, dtype=_F16, device=X.device)
                po = out.data_ptr()
            st = fn(f, g, M, N, K, px, psx, pw, ps, pb, a, pr, pv, alpha, pa, po, raw)
    if st:
        _check(st)
    return out


def qgemm_gated(fmt: str, X: torch.Tensor, Wg: torch.Tensor, scales_g, Wu: torch.Tensor, scales_u, sx=None,
                bias_g=None, bias_u=None, act: str = "silu", group=None, out=None, save=None, stream=None):
    """H [M,N] fp16 = act(g) * u with g = X . dequant(Wg)^T + bias_g and
    u = X . dequant(Wu)^T + bias_u, in one kernel (include/aria_q.h,
    aria_qgemm_gated).

    Both weights have one format and shape (as Wq and scales of qgemm; "f16"
    takes the fp16 weights and None for the scales). ``save`` = (G, U): fp16
    [M,N] tensors that receive g and u, for gated_backward. The weights are
    read in stream order for "f16" and wherever ``save`` is given; packed
    weights otherwise follow qgemm's rule."""
    M, N, K, di, px, psx = _x_args(fmt, X, Wg, sx)
    pg, psg = _weight_args(fmt, Wg, scales_g, "g", N, K, di)
    pu, psu = _weight_args(fmt, Wu, scales_u, "u", N, K, di)
    mn, n = (M, N), (N,)
    pbg = _arg(bias_g, "bias_g", n, _F16, di)
    pbu = _arg(bias_u, "bias_u", n, _F16, di)
    if save is None:
        pG = pU = None
    elif len(save) != 2 or save[0] is None or save[1] is None:
        raise ValueError("save is (G, U)")
    else:
        pG = _arg(save[0], "save[0]", mn, _F16, di)
        pU = _arg(save[1], "save[1]", mn, _F16, di)
    a, gr, f = _act(act), _group(fmt, group), FORMATS[fmt]
    po = _arg(out, "out", mn, _F16, di)
    fn = load_library().aria_qgemm_gated
    raw = _here(di, stream)
    if raw is not None:
        if out is None:
            out = torch.empty(mn, dtype=_F16, device=X.device)
            po = out.data_ptr()
        st = fn(f, gr, M, N, K, px, psx, pg, psg, pu, psu, pbg, pbu, a, po, pG, pU, raw)
    else:
        with _running_on(di, stream) as raw:
            if out is None:
                out = torch.empty(mn, dtype=_F16, device=X.device)
                po = out.data_ptr()
            st = fn(f, gr, M, N, K, px, psx, pg, psg, pu, psu, pbg, pbu, a, po, pG, pU, raw)
    if st:
        _check(st)
    return out


def gated_backward_workspace_size(M: int, N: int, K: int, device=None) -> int:
    """Bytes that gated_backward needs on `device` (the current one if None):
    the number of its SMs decides how dX's sum is divided."""
    n = ctypes.c_size_t()
    with contextlib.nullcontext() if device is None else torch.cuda.device(torch.device(device)):
        _check(load_library().aria_gated_bwd_workspace_size(M, N, K, ctypes.byref(n)))
    return n.value


def gated_backward(dH: torch.Tensor, X, Wg, Wu, G: torch.Tensor, U: torch.Tensor, act: str = "silu",
                   input_grad: bool = True, weight_grad: bool = True, bias_grad: bool = True, out=None,
                   workspace=None, stream=None):
    """Gradients of qgemm_gated("f16", ...) from the pre-activations it kept
    (include/aria_q.h, aria_gated_bwd): (dX [M,K], dWg [N,K], dWu [N,K],
    dbg [N], dbu [N]), fp16, None for those not asked for.

    ``out``: a tuple of five tensors to write (None where nothing is asked
    for). ``workspace``: a uint8 tensor of gated_backward_workspace_size(M, N, K,
    dH.device) bytes; calls sharing one must not overlap on the GPU. X is needed for the
    weight gradients only and the weights for dX only; K comes from any of them."""
    if dH.dim() != 2:
        raise ValueError("dH must be 2-D")
    di = dH.get_device()
    if di < 0:
        raise ValueError("dH must be a CUDA tensor (no CPU path exists)")
    if not (input_grad or weight_grad or bias_grad):
        raise ValueError("no gradient is asked for")
    M, N = dH.shape
    src = X if X is not None else Wg if Wg is not None else Wu
    if src is None:
        if input_grad or weight_grad:
            raise ValueError("dX needs Wg and Wu, dWg and dWu need X")
        K = 16  # the bias gradients alone do not depend on it
    elif src.dim() != 2:
        raise ValueError("X and the weights must be 2-D")
    else:
        K = src.shape[1]
    if input_grad and (Wg is None or Wu is None):
        raise ValueError("dX needs Wg and Wu")
    if weight_grad and X is None:
        raise ValueError("dWg and dWu need X")
    mn, mk, nk = (M, N), (M, K), (N, K)
    pin = (_arg(dH, "dH", mn, _F16, di), _arg(G, "G", mn, _F16, di), _arg(U, "U", mn, _F16, di),
           _arg(X, "X", mk, _F16, di), _arg(Wg, "Wg", nk, _F16, di), _arg(Wu, "Wu", nk, _F16, di))
    if pin[1] is None or pin[2] is None:
        raise ValueError("G and U are needed (qgemm_gated's save=)")
    a = _act(act)
    shapes = (mk, nk, nk, (N,), (N,))
    asked = (input_grad, weight_grad, weight_grad, bias_grad, bias_grad)
    names = ("dX", "dWg", "dWu", "dbg", "dbu")
    if out is not None:
        if len(out) != 5:
            raise ValueError("out is (dX, dWg, dWu, dbg, dbu)")
        for t, on, n, sh in zip(out, asked, names, shapes):
            if (t is not None) != on:
                raise ValueError(f"out: {n} is {'needed' if on else 'not asked for'}")
            _arg(t, n, sh, _F16, di)
    if workspace is not None:
        _arg(workspace, "workspace", workspace.shape, _U8, di)
        if workspace.numel() < 4 * M * N:
            raise ValueError(f"workspace of {workspace.numel()} bytes, more than {4 * M * N} needed")
    raw = _here(di, stream)
    if raw is not None:
        return _gated_backward_on(raw, a, M, N, K, pin, dH, X, Wg, Wu, input_grad, weight_grad, bias_grad, out,
                                  workspace)
    with _running_on(di, stream) as raw:
        return _gated_backward_on(raw, a, M, N, K, pin, dH, X, Wg, Wu, input_grad, weight_grad, bias_grad, out,
                                  workspace)


def _gated_backward_on(raw, act, M, N, K, pin, dH, X, Wg, Wu, input_grad, weight_grad, bias_grad, out, ws):
    """The checked call on stream `raw`, with what is not given allocated (the
    inputs are contiguous, so the tensors like them are). The device of the
    tensors is current: the workspace is planned for it."""
    need = gated_backward_workspace_size(M, N, K)
    if ws is not None and ws.numel() < need:
        raise ValueError(f"workspace of {ws.numel()} bytes, {need} needed")
    if out is None:
        dX = dWg = dWu = dbg = dbu = None
        if input_grad:
            dX = dH.new_empty((M, K)) if X is None else torch.empty_like(X)
        if weight_grad:
            dWg = dH.new_empty((N, K)) if Wg is None else torch.empty_like(Wg)
            dWu = torch.empty_like(dWg)
        if bias_grad:
            dbg = dH.new_empty(N)
            dbu = torch.empty_like(dbg)
        out = (dX, dWg, dWu, dbg, dbu)
    if ws is None:
        ws = dH.new_empty(need, dtype=_U8)
    st = load_library().aria_gated_bwd(act, M, N, K, *pin, *[None if t is None else t.data_ptr() for t in out],
                                       ws.data_ptr(), ws.numel(), raw)
    if st:
        _check(st)
    return tuple(out)


def selftest_bounded_wait(Xq, sx, Wq, sw, out=None, wait_limit_us: int = 50000, stream=None):
    """Failure-detection self-test (include/aria_q.h): a W8A8 launch whose
    first pipeline stage never fills, with every bounded wait limited to
    wait_limit_us. Returns the output tensor (contents unspecified); the
    following device_status() raises AriaError with ARIA_ERR_TIMEOUT."""
    M, K = Xq.shape
    N = Wq.shape[0]
    _expect(sx, "sx", (M,), torch.float32)
    _expect(Wq, "Wq", (N, K), torch.int8)
    _expect(sw, "scales", (N,), torch.float32)
    Y = out if out is not None else torch.empty(M, N, dtype=torch.float16, device=Xq.device)
    _expect(Y, "out", (M, N), torch.float16)
    same_device(Xq=Xq, sx=sx, Wq=Wq, sw=sw, out=Y)
    with _on(Xq.device):
        _check(load_library().aria_selftest_bounded_wait(
            M, N, K, _dev(Xq, "Xq", torch.int8), _dev(sx, "sx", torch.float32), _dev(Wq, "Wq", torch.int8),
            _dev(sw, "scales", torch.float32), _dev(Y, "out"), int(wait_limit_us), _stream(stream)))
    return Y


def device_status(stream=None):
    """Synchronise the stream and raise if a kernel's bounded wait ran out."""
    _check(load_library().aria_device_status(_stream(stream)))


# ------------------------------------------------------- steering schedule --

def parse_steer_spec(spec: str) -> dict:
    """Parse a steer spec ``site:block:file:alpha:steps`` ("Run it", e.g.
    ``residual:19:directions/small/sour.atns:0.1:0-7``) into its fields.
    ``steps`` is an inclusive range ``a-b`` or a single step ``a``. The file
    is only named here: the direction itself is passed to the GEMM as a
    device vector. Raises ValueError on a malformed spec."""
    parts = spec.split(":")
    if len(parts) != 5:
        raise ValueError(f"steer spec needs 5 fields site:block:file:alpha:steps, got {spec!r}")
    site, block, path, alpha, steps = parts
    if not site:
        raise ValueError("empty steering site")
    try:
        block_i = int(block)
        alpha_f = float(alpha)
    except ValueError as e:
        raise ValueError(f"bad block or alpha in {spec!r}") from e
    if block_i < 0:
        raise ValueError("block must be >= 0")
    a, sep, b = steps.partition("-")
    try:
        s0 = int(a)
        s1 = int(b) if sep else s0
    except ValueError as e:
        raise ValueError(f"bad step range {steps!r}") from e
    if s0 < 0 or s1 < s0:
        raise ValueError(f"bad step range {steps!r}")
    return {"site": site, "block": block_i, "file": path, "alpha": alpha_f, "steps": (s0, s1)}


def steer_schedule(spec, n_steps: int) -> list:
    """Per-step strengths of a steer spec (a string or parse_steer_spec's
    dict): alpha inside the inclusive step window, 0.0 outside it (a zero
    strength skips the add, so those steps are bit-identical to unsteered
    ones). Feed it to a device tensor read through ``alpha_dev``."""
    d = parse_steer_spec(spec) if isinstance(spec, str) else spec
    s0, s1 = d["steps"]
    return [d["alpha"] if s0 <= s < s1 + 1 else 0.0 for s in range(n_steps)]
