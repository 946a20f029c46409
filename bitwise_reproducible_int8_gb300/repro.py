"""Thin Python binding of librepro.so (include/repro.h): argument marshalling
only.  Every step of the path runs in the library's CUDA kernels; torch is used
for device memory and streams.  There is no fallback: if the library is not
built, or a call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librepro.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "repro.h")

REPRO_OK = 0
STATUS_NAMES = {
    0: "REPRO_OK", -1: "REPRO_ERR_ARG", -2: "REPRO_ERR_SHAPE", -3: "REPRO_ERR_ALIGN",
    -4: "REPRO_ERR_ARCH", -5: "REPRO_ERR_LAUNCH", -6: "REPRO_ERR_TIMEOUT",
    -7: "REPRO_ERR_WORKSPACE", -8: "REPRO_ERR_ALIAS", -9: "REPRO_ERR_SELFTEST",
    -10: "REPRO_ERR_NONFINITE", -11: "REPRO_ERR_INDEX",
}
REPRO_ERR_TIMEOUT = -6
REPRO_ERR_NONFINITE = -10
REPRO_ERR_INDEX = -11
REPRO_DEBUG_CHECK_FINITE = 1
REPRO_SCALE_WEIGHT_MEANABS = 0
REPRO_SCALE_ACT_AMAX = 1
REPRO_BWD_DW_ACCUMULATE = 1
REPRO_QMAX = 127
REPRO_MAX_REPLICAS = 64
REPRO_F32, REPRO_BF16, REPRO_I8 = 0, 1, 2
REPRO_EMBED_MAX_V = 16777215
REPRO_EMBED_MAX_N = 1 << 30
REPRO_QK_INTERLEAVED = 2
REPRO_QK_MAX_D = 512
REPRO_DISTILL_BLOCK = 1024
REPRO_DISTILL_STATS = 8
REPRO_DISTILL_STAT_LSE = 2
REPRO_DISTILL_LOGPROBS = 1


class ReproError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)} "
                         f"({lib().repro_status_str(status).decode()})")


class AdamWHparams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_float) for k in
                ("lr", "beta1", "beta2", "eps", "weight_decay", "max_norm")]


class DistillHparams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_float) for k in ("tau", "w_kd", "w_ce", "w_z")]


class LaunchCfg(ctypes.Structure):
    _fields_ = [("bwd_segment_log2", ctypes.c_int), ("reduce_block_log2", ctypes.c_int),
                ("fwd_path", ctypes.c_int), ("elementwise_blocks", ctypes.c_int),
                ("bwd_kernel", ctypes.c_int), ("fwd_selftest", ctypes.c_int)]


_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_sz = ctypes.c_size_t

_SIGNATURES = {
    "repro_wscale": (_int, [_vp, _i64, _int, _int, _vp, _vp, _sz, _vp]),
    "repro_wscale_ws_bytes": (_sz, [_i64]),
    "repro_wscale_noalloc": (_int, [_vp, _i64, _int, _int, _vp, _vp]),
    "repro_quant_i8": (_int, [_vp, _i64, _vp, _int, _vp, _vp]),
    "repro_wscale_multi": (_int, [ctypes.POINTER(_vp), ctypes.POINTER(_i64), _int, _int, _int,
                                  _vp, _vp, _sz, _vp]),
    "repro_wscale_multi_ws_bytes": (_sz, [ctypes.POINTER(_i64), _int]),
    "repro_quant_i8_multi": (_int, [ctypes.POINTER(_vp), ctypes.POINTER(_i64), _int, _vp, _int,
                                    ctypes.POINTER(_vp), _vp]),
    "repro_linear_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "repro_linear_fwd_ws_bytes": (_sz, [_i64, _i64, _i64]),
    "repro_linear_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int,
                                _vp, _sz, _vp]),
    "repro_linear_bwd_ws_bytes": (_sz, [_i64, _i64, _i64]),
    "repro_grad_accum": (_int, [_vp, _vp, _i64, _vp]),
    "repro_treefold": (_int, [ctypes.POINTER(_vp), _int, _i64, _vp, _vp]),
    "repro_running_sum": (_int, [ctypes.POINTER(_vp), _int, _i64, _vp, _vp]),
    "repro_sumsq": (_int, [_vp, _i64, _vp, _vp, _sz, _vp]),
    "repro_sumsq_ws_bytes": (_sz, [_i64]),
    "repro_adamw_step": (_int, [_vp, _vp, _vp, _vp, _i64, _vp, ctypes.POINTER(AdamWHparams),
                                _i64, _vp]),
    "repro_state_hash": (_int, [ctypes.POINTER(_vp), ctypes.POINTER(_i64), _int, _vp, _vp, _sz,
                                _vp]),
    "repro_state_hash_ws_bytes": (_sz, [ctypes.POINTER(_i64), _int]),
    "repro_attn_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                              _i64, _vp, _sz, _vp]),
    "repro_attn_fwd_ws_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "repro_attn_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                              _i64, _i64, _i64, _i64, _vp, _sz, _vp, _sz, _vp]),
    "repro_attn_bwd_ws_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "repro_embed_fwd": (_int, [_vp, _int, _i64, _vp, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _i64,
                               _vp, _int, _i64, _vp]),
    "repro_embed_bwd": (_int, [_vp, _int, _i64, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _i64, _vp,
                               _i64, _int, _vp, _sz, _vp]),
    "repro_embed_bwd_ws_bytes": (_sz, [_i64, _i64, _i64]),
    "repro_qk_norm_rope_fwd": (_int, [_vp, _i64, _i64, _vp, _i64, _i64, _int, _vp, _vp, _vp, _i64, _vp, _i64,
                                      ctypes.c_float, _i64, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp]),
    "repro_qk_norm_rope_bwd": (_int, [_vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _int, _vp, _vp, _vp, _i64,
                                      _vp, _i64, ctypes.c_float, _i64, _i64, _i64, _i64, _i64, _int, _vp, _i64,
                                      _i64, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "repro_qk_norm_rope_bwd_ws_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "repro_distill_fwd": (_int, [_vp, _int, _i64, _vp, _vp, _int, _vp, _int, _i64, _i64, _i64,
                                 ctypes.POINTER(DistillHparams), _int, _vp, _vp, _vp, _sz, _vp]),
    "repro_distill_ws_bytes": (_sz, [_i64, _i64]),
    "repro_distill_bwd": (_int, [_vp, _int, _i64, _vp, _vp, _int, _i64, _i64, _i64,
                                 ctypes.POINTER(DistillHparams), _vp, _vp, _i64, _vp, _i64, _vp]),
    "repro_selftest": (_int, [_vp, _sz, _vp]),
    "repro_selftest_ws_bytes": (_sz, []),
    "repro_status_str": (ctypes.c_char_p, [_int]),
    "repro_version": (_int, []),
    "repro_device_check": (_int, [_vp]),
    "repro_wait_probe": (_int, [_int, _vp]),
    "repro_launch_count": (ctypes.c_uint64, []),
    "repro_set_launch_cfg": (_int, [ctypes.POINTER(LaunchCfg)]),
    "repro_set_debug": (_int, [_int]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "bitwise_reproducible_int8_gb300.build_lib.build() (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def declared_functions() -> list:
    """Names of the functions declared in include/repro.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+char\s*\*|int|size_t|uint64_t)\s+(repro_\w+)\s*\(",
                                 text, flags=re.M)))


# ------------------------------------------------------------------ marshalling

def _stream(stream) -> int:
    if stream is None:
        # the current stream's handle, without the Stream object around it: a call's
        # host time is a few microseconds and building that object was most of it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check(fn: str, status: int) -> None:
    if status != REPRO_OK:
        raise ReproError(fn, status)


def _workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """A workspace for one call on `stream`: memory of that stream, whichever is current,
    so that its owners before and after this call are in the stream's order."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) \
            else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ the calls

def repro_wscale_ws_bytes(n: int) -> int:
    return int(lib().repro_wscale_ws_bytes(int(n)))


def repro_wscale(x: torch.Tensor, mode: int, scale_out: torch.Tensor, ws=None,
                 qmax: int = REPRO_QMAX, stream=None) -> None:
    """scale_out[0] <- weight (mode 0) or activation (mode 1) scale of x."""
    n = x.numel()
    if ws is None:
        ws = _workspace(repro_wscale_ws_bytes(n), x.device, stream)
    _check("repro_wscale", lib().repro_wscale(
        _ptr(x, torch.float32, "x"), n, int(mode), int(qmax),
        _ptr(scale_out, torch.float32, "scale_out"), _ptr(ws, None, "ws"),
        ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 1 << 62,
        _stream(stream)))


def repro_wscale_noalloc(x: torch.Tensor, mode: int, scale_out: torch.Tensor,
                         qmax: int = REPRO_QMAX, stream=None) -> None:
    """repro_wscale without a workspace, for callers that cannot allocate
    device memory; scratch comes from a fixed array inside the library."""
    _check("repro_wscale_noalloc", lib().repro_wscale_noalloc(
        _ptr(x, torch.float32, "x"), x.numel(), int(mode), int(qmax),
        _ptr(scale_out, torch.float32, "scale_out"), _stream(stream)))


def repro_quant_i8(x: torch.Tensor, scale: torch.Tensor, q_out: torch.Tensor,
                   qmax: int = REPRO_QMAX, stream=None) -> None:
    if q_out.numel() != x.numel():
        raise ValueError("q_out must have as many elements as x")
    _check("repro_quant_i8", lib().repro_quant_i8(
        _ptr(x, torch.float32, "x"), x.numel(), _ptr(scale, torch.float32, "scale"), int(qmax),
        _ptr(q_out, torch.int8, "q_out"), _stream(stream)))


def _tables(tensors, dtype, name):
    n = len(tensors)
    ptrs = (_vp * max(n, 1))(*[_ptr(t, dtype, name) for t in tensors])
    sizes = (_i64 * max(n, 1))(*[int(t.numel()) for t in tensors])
    return ptrs, sizes


def repro_wscale_multi_ws_bytes(sizes) -> int:
    arr = (_i64 * max(len(sizes), 1))(*[int(v) for v in sizes])
    return int(lib().repro_wscale_multi_ws_bytes(arr, len(sizes)))


def repro_wscale_multi(xs, mode: int, scales_out: torch.Tensor, ws=None,
                       qmax: int = REPRO_QMAX, stream=None) -> None:
    """scales_out[t] <- the scale of xs[t] (mode 0 weight, 1 activation) for
    every t, in one pass; the bits of repro_wscale on each tensor."""
    ptrs, sizes = _tables(xs, torch.float32, "x")
    if scales_out.numel() < len(xs):
        raise ValueError("scales_out needs one float per tensor")
    if ws is None:
        ws = _workspace(repro_wscale_multi_ws_bytes([x.numel() for x in xs]), xs[0].device, stream)
    _check("repro_wscale_multi", lib().repro_wscale_multi(
        ptrs, sizes, len(xs), int(mode), int(qmax), _ptr(scales_out, torch.float32, "scales_out"),
        _ptr(ws, None, "ws"), ws.numel() * ws.element_size(), _stream(stream)))


def repro_quant_i8_multi(xs, scales: torch.Tensor, q_outs, qmax: int = REPRO_QMAX,
                         stream=None) -> None:
    """q_outs[t] <- int8 codes of xs[t] with scales[t], every t in one launch."""
    if len(q_outs) != len(xs) or any(q.numel() != x.numel() for q, x in zip(q_outs, xs)):
        raise ValueError("one q_out of x's size per tensor")
    ptrs, sizes = _tables(xs, torch.float32, "x")
    qptrs, _ = _tables(q_outs, torch.int8, "q_out")
    _check("repro_quant_i8_multi", lib().repro_quant_i8_multi(
        ptrs, sizes, len(xs), _ptr(scales, torch.float32, "scales"), int(qmax), qptrs,
        _stream(stream)))


def repro_linear_fwd_ws_bytes(M: int, N: int, K: int) -> int:
    return int(lib().repro_linear_fwd_ws_bytes(int(M), int(N), int(K)))


def repro_linear_fwd(xq: torch.Tensor, wq: torch.Tensor, s_x: torch.Tensor, s_w: torch.Tensor,
                     y: torch.Tensor, ws=None, stream=None) -> None:
    M, K = xq.shape
    N, K2 = wq.shape
    if K != K2 or tuple(y.shape) != (M, N):
        raise ValueError("shape mismatch: xq [M,K], wq [N,K], y [M,N]")
    if ws is None:
        need = repro_linear_fwd_ws_bytes(M, N, K)
        ws = _workspace(need, y.device, stream) if need > 0 else None
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("repro_linear_fwd", lib().repro_linear_fwd(
        _ptr(xq, torch.int8, "xq"), _ptr(wq, torch.int8, "wq"), _ptr(s_x, torch.float32, "s_x"),
        _ptr(s_w, torch.float32, "s_w"), _ptr(y, torch.float32, "y"), M, N, K,
        _ptr(ws, None, "ws"), ws_bytes, _stream(stream)))


def repro_linear_bwd_ws_bytes(M: int, N: int, K: int) -> int:
    return int(lib().repro_linear_bwd_ws_bytes(int(M), int(N), int(K)))


def repro_linear_bwd(dy: torch.Tensor, xq, wq, s_x, s_w, dx=None, dw=None,
                     accumulate: bool = False, ws=None, stream=None) -> None:
    M, N = dy.shape
    K = (xq if xq is not None else wq).shape[1]
    if dx is not None and tuple(dx.shape) != (M, K):
        raise ValueError("dx must be [M,K]")
    if dw is not None and tuple(dw.shape) != (N, K):
        raise ValueError("dw must be [N,K]")
    if ws is None:
        need = repro_linear_bwd_ws_bytes(M, N, K)
        ws = _workspace(need, dy.device, stream) if need > 0 else None
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("repro_linear_bwd", lib().repro_linear_bwd(
        _ptr(dy, torch.float32, "dy"), _ptr(xq, torch.int8, "xq"), _ptr(wq, torch.int8, "wq"),
        _ptr(s_x, torch.float32, "s_x"), _ptr(s_w, torch.float32, "s_w"),
        _ptr(dx, torch.float32, "dx"), _ptr(dw, torch.float32, "dw"), M, N, K,
        REPRO_BWD_DW_ACCUMULATE if accumulate else 0, _ptr(ws, None, "ws"), ws_bytes,
        _stream(stream)))


def repro_grad_accum(acc: torch.Tensor, g: torch.Tensor, stream=None) -> None:
    if acc.numel() != g.numel():
        raise ValueError("acc and g must have the same number of elements")
    _check("repro_grad_accum", lib().repro_grad_accum(
        _ptr(acc, torch.float32, "acc"), _ptr(g, torch.float32, "g"), acc.numel(),
        _stream(stream)))


def repro_running_sum(parts, out: torch.Tensor, stream=None) -> None:
    """out <- left fold of the partials in the given (mesh) order."""
    S = len(parts)
    n = out.numel()
    if any(p.numel() != n for p in parts):
        raise ValueError("every partial must have out.numel() elements")
    arr = (_vp * max(S, 1))(*[_ptr(p, torch.float32, "part") for p in parts])
    _check("repro_running_sum", lib().repro_running_sum(arr, S, n, _ptr(out, torch.float32, "out"),
                                                        _stream(stream)))


def repro_treefold(parts, out: torch.Tensor, stream=None) -> None:
    R = len(parts)
    n = out.numel()
    if any(p.numel() != n for p in parts):
        raise ValueError("every partial must have out.numel() elements")
    arr = (_vp * max(R, 1))(*[_ptr(p, torch.float32, "part") for p in parts])
    _check("repro_treefold", lib().repro_treefold(arr, R, n, _ptr(out, torch.float32, "out"),
                                                  _stream(stream)))


def repro_attn_fwd_ws_bytes(B: int, T: int, Hq: int, W: int = 0) -> int:
    return int(lib().repro_attn_fwd_ws_bytes(int(B), int(T), int(Hq), int(W)))


def repro_attn_fwd(q: torch.Tensor, k: torch.Tensor, vq: torch.Tensor, s_v: torch.Tensor,
                   o: torch.Tensor, m: torch.Tensor, l: torch.Tensor, W: int = 0, ws=None,
                   stream=None) -> None:
    """q, o [B,T,Hq,128] fp32; k [B,T,Hkv,128] fp32; vq [B,T,Hkv,128] int8;
    s_v [1]; m, l [B,T,Hq] outputs.  W: sliding window (0: full causal).
    ws: optional logit cache of repro_attn_fwd_ws_bytes bytes (None: the
    second pass recomputes the logits; same bits)."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check("repro_attn_fwd", lib().repro_attn_fwd(
        _ptr(q, torch.float32, "q"), _ptr(k, torch.float32, "k"), _ptr(vq, torch.int8, "vq"),
        _ptr(s_v, torch.float32, "s_v"), _ptr(o, torch.float32, "o"),
        _ptr(m, torch.float32, "m"), _ptr(l, torch.float32, "l"), B, T, Hq, Hkv, D, int(W),
        _ptr(ws, None, "ws"), ws_bytes, _stream(stream)))


def repro_attn_bwd_ws_bytes(B: int, T: int, Hq: int, W: int = 0) -> int:
    """Workspace of repro_attn_bwd for window W; W = -1: a call without the
    forward's cache."""
    return int(lib().repro_attn_bwd_ws_bytes(int(B), int(T), int(Hq), int(W)))


def repro_attn_bwd(q, k, vq, s_v, o, dout, m, l, dq, dk, dv, W: int = 0, ws=None,
                   fwd_ws=None, stream=None) -> None:
    """dq [B,T,Hq,128], dk and dv [B,T,Hkv,128] from the forward's inputs,
    output o, row statistics m, l and the upstream gradient dout.  fwd_ws:
    optionally the logit cache repro_attn_fwd filled for these inputs."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    if ws is None:
        ws = _workspace(repro_attn_bwd_ws_bytes(B, T, Hq, int(W) if fwd_ws is not None else -1),
                        q.device, stream)
    f32 = torch.float32
    _check("repro_attn_bwd", lib().repro_attn_bwd(
        _ptr(q, f32, "q"), _ptr(k, f32, "k"), _ptr(vq, torch.int8, "vq"), _ptr(s_v, f32, "s_v"),
        _ptr(o, f32, "o"), _ptr(dout, f32, "dout"), _ptr(m, f32, "m"), _ptr(l, f32, "l"),
        _ptr(dq, f32, "dq"), _ptr(dk, f32, "dk"), _ptr(dv, f32, "dv"), B, T, Hq, Hkv, D, int(W),
        _ptr(ws, None, "ws"), ws.numel() * ws.element_size(), _ptr(fwd_ws, None, "fwd_ws"),
        fwd_ws.numel() * fwd_ws.element_size() if fwd_ws is not None else 0, _stream(stream)))


_FLOAT_TYPES = {torch.float32: REPRO_F32, torch.bfloat16: REPRO_BF16}


def _dev_ptr(t, name, contiguous=True):
    """Data pointer of a CUDA tensor (None: NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _float_type(t, name) -> int:
    if t.dtype not in _FLOAT_TYPES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return _FLOAT_TYPES[t.dtype]


def _index_bytes(name, *ts) -> int:
    kinds = {t.dtype for t in ts if t is not None}
    if len(kinds) > 1 or not kinds <= {torch.int32, torch.int64}:
        raise ValueError(f"{name} must be int32 or int64 (all of one type)")
    return 4 if kinds == {torch.int32} else 8


def _rows2d(t, name):
    """(rows, width, row stride) of a matrix, or of an array whose leading
    dimensions collapse into one; elements of a row adjacent."""
    shape = t.shape
    if len(shape) < 2:
        raise ValueError(f"{name} must have at least two dimensions")
    D = shape[-1]
    if t.is_contiguous():
        return (t.numel() // D if D else 0), D, D
    strides = t.stride()
    if D > 1 and strides[-1] != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    n, ld = 1, None
    for size, stride in zip(shape[-2::-1], strides[-2::-1]):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif t.numel() > 0 and stride != ld * n:
            raise ValueError(f"{name}: the rows must lie at one stride")
        n *= size
    return n, D, D if ld is None else int(ld)


def repro_embed_fwd(table: torch.Tensor, tokens: torch.Tensor, out: torch.Tensor, scale: float = 1.0,
                    s_w=None, pad: int = -1, stream=None) -> None:
    """out[..., D] <- table[tokens] (x) scale; +0 rows where a token equals pad.
    table [V, D] float32, bfloat16, or int8 codes with their scale s_w [1]; rows
    of table and out at any stride; tokens int32 or int64."""
    V, D, table_ld = _rows2d(table, "table")
    n, D2, out_ld = _rows2d(out, "out")
    if D2 != D or n != tokens.numel():
        raise ValueError("shape mismatch: table [V, D], out [..., D] with a row per token")
    if table.dtype == torch.int8:
        if s_w is None:
            raise ValueError("an int8 table needs its scale s_w")
        kind = REPRO_I8
    else:
        kind = _float_type(table, "table")
    _check("repro_embed_fwd", lib().repro_embed_fwd(
        _dev_ptr(table, "table", False), kind, table_ld, _ptr(s_w, torch.float32, "s_w"),
        _dev_ptr(tokens, "tokens"), _index_bytes("tokens", tokens), n, V, D, float(scale), int(pad),
        _dev_ptr(out, "out", False), _float_type(out, "out"), out_ld, _stream(stream)))


def repro_embed_bwd_ws_bytes(n: int, V: int, D: int) -> int:
    return int(lib().repro_embed_bwd_ws_bytes(int(n), int(V), int(D)))


def repro_embed_bwd(dout: torch.Tensor, tokens: torch.Tensor, dtable: torch.Tensor, scale: float = 1.0,
                    pad: int = -1, accumulate: bool = False, ws=None, stream=None) -> None:
    """dtable [V, D] <- (or (+)=) the sum of dout's rows by token, in canonical
    order over ascending positions, (x) scale."""
    n, D, dout_ld = _rows2d(dout, "dout")
    V, D2, dtable_ld = _rows2d(dtable, "dtable")
    if D2 != D or n != tokens.numel():
        raise ValueError("shape mismatch: dout [..., D] with a row per token, dtable [V, D]")
    if dtable.dtype != torch.float32:
        raise ValueError(f"dtable must be {torch.float32}, got {dtable.dtype}")
    if ws is None:
        ws = _workspace(repro_embed_bwd_ws_bytes(n, V, D), dtable.device, stream)
    _check("repro_embed_bwd", lib().repro_embed_bwd(
        _dev_ptr(dout, "dout", False), _float_type(dout, "dout"), dout_ld, _dev_ptr(tokens, "tokens"),
        _index_bytes("tokens", tokens), n, V, D, float(scale), int(pad), _dev_ptr(dtable, "dtable", False),
        dtable_ld, REPRO_BWD_DW_ACCUMULATE if accumulate else 0, _dev_ptr(ws, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def _heads(t, name):
    """(tokens, heads, width, token stride, head stride) of [n, H, D] or [B, T, H, D]."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 3:
        n, ld = shape[0], strides[0]
    elif len(shape) == 4:
        B, T = shape[:2]
        n = B * T
        ld = strides[0] if T == 1 else strides[1]
        if B > 1 and T > 1 and strides[0] != T * ld:
            raise ValueError(f"{name}: the tokens must lie at one stride")
    else:
        raise ValueError(f"{name} must be [n, H, D] or [B, T, H, D]")
    H, D = shape[-2:]
    if D > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the elements of a head must be adjacent")
    return n, H, D, (ld if n > 1 else max(ld, 1)), (strides[-2] if H > 1 else D)


def _qk_common(q, k, rope, g_q, g_k, positions):
    n, Hq, D, q_ld, q_hs = _heads(q, "q")
    kind = _float_type(q, "q")
    Hkv, k_ld, k_hs = 0, D, D
    if k is not None:
        nk, Hkv, Dk, k_ld, k_hs = _heads(k, "k")
        if nk != n or Dk != D or k.dtype != q.dtype:
            raise ValueError("k must have q's tokens, width and type")
    P, R = (rope.shape if rope is not None else (0, 0))
    for g, name in ((g_q, "g_q"), (g_k, "g_k")):
        if g is not None and g.numel() != D:
            raise ValueError(f"{name} must have D elements")
    if positions is not None and positions.numel() != n:
        raise ValueError("positions must have an entry per token")
    T = q.shape[1] if q.dim() == 4 else n
    return n, Hq, D, q_ld, q_hs, Hkv, k_ld, k_hs, kind, P, R, max(int(T), 1)


def repro_qk_norm_rope_fwd(q: torch.Tensor, k, rope, q_out: torch.Tensor, k_out, g_q=None, g_k=None,
                           positions=None, eps: float = 1e-6, interleaved: bool = False,
                           stream=None) -> None:
    """q_out, k_out <- the RMS-normalised heads of q, k (gains g_q, g_k [D] if
    given), turned by the positions' angles.  q [B, T, Hq, D] or [n, Hq, D], k the
    same with its own heads (or None), float32 or bfloat16, at any token and head
    strides; rope [P, R] float32, cosines then sines (None: no rotation);
    positions int32 per token (None: 0 .. T - 1 in every sequence); outputs dense
    float32."""
    f32 = torch.float32
    n, Hq, D, q_ld, q_hs, Hkv, k_ld, k_hs, kind, P, R, T = _qk_common(q, k, rope, g_q, g_k, positions)
    if q_out.numel() != n * Hq * D or (k is not None and k_out.numel() != n * Hkv * D):
        raise ValueError("outputs must have the inputs' sizes")
    _check("repro_qk_norm_rope_fwd", lib().repro_qk_norm_rope_fwd(
        _dev_ptr(q, "q", False), q_ld, q_hs, _dev_ptr(k, "k", False), k_ld, k_hs, kind,
        _ptr(g_q, f32, "g_q"), _ptr(g_k, f32, "g_k"), _ptr(rope, f32, "rope"), P,
        _ptr(positions, torch.int32, "positions"), T, float(eps), n, Hq, Hkv, D, R,
        REPRO_QK_INTERLEAVED if interleaved else 0, _ptr(q_out, f32, "q_out"),
        _ptr(k_out if k is not None else None, f32, "k_out"), _stream(stream)))


def repro_qk_norm_rope_bwd_ws_bytes(n: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().repro_qk_norm_rope_bwd_ws_bytes(int(n), int(Hq), int(Hkv), int(D)))


def repro_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out, q: torch.Tensor, k, rope, dq: torch.Tensor, dk,
                           g_q=None, g_k=None, dg_q=None, dg_k=None, positions=None, eps: float = 1e-6,
                           interleaved: bool = False, accumulate: bool = False, ws=None,
                           stream=None) -> None:
    """dq, dk (q's type, any token and head strides that keep their heads apart;
    both may lie in one buffer) and the gains' gradients
    dg_q, dg_k [D] (added to with accumulate) from the gradients dq_out, dk_out
    of the forward's outputs (dense float32) and the forward's inputs."""
    f32 = torch.float32
    n, Hq, D, q_ld, q_hs, Hkv, k_ld, k_hs, kind, P, R, T = _qk_common(q, k, rope, g_q, g_k, positions)
    strides = []
    for t, g, x, H, name in ((dq, dq_out, q, Hq, "q"), (dk, dk_out, k, Hkv, "k")):
        if x is None:
            strides.append((D, D))
            continue
        nd, Hd, Dd, ld, hs = _heads(t, "d" + name)
        if (nd, Hd, Dd) != (n, H, D) or t.dtype != q.dtype or g.numel() != n * H * D:
            raise ValueError(f"d{name} must have {name}'s shape and type, d{name}_out its size")
        strides.append((ld, hs))
    for g, name in ((dg_q, "dg_q"), (dg_k, "dg_k")):
        if g is not None and g.numel() != D:
            raise ValueError(f"{name} must have D elements")
    if ws is None and (g_q is not None or g_k is not None):
        ws = _workspace(repro_qk_norm_rope_bwd_ws_bytes(n, Hq, Hkv, D), q.device, stream)
    flags = (REPRO_QK_INTERLEAVED if interleaved else 0) | (REPRO_BWD_DW_ACCUMULATE if accumulate else 0)
    has_k = k is not None
    _check("repro_qk_norm_rope_bwd", lib().repro_qk_norm_rope_bwd(
        _ptr(dq_out, f32, "dq_out"), _ptr(dk_out if has_k else None, f32, "dk_out"),
        _dev_ptr(q, "q", False), q_ld, q_hs, _dev_ptr(k, "k", False), k_ld, k_hs, kind,
        _ptr(g_q, f32, "g_q"), _ptr(g_k, f32, "g_k"), _ptr(rope, f32, "rope"), P,
        _ptr(positions, torch.int32, "positions"), T, float(eps), n, Hq, Hkv, D, R, flags,
        _dev_ptr(dq, "dq", False), *strides[0], _dev_ptr(dk if has_k else None, "dk", False), *strides[1],
        _ptr(dg_q, f32, "dg_q"), _ptr(dg_k, f32, "dg_k"), _dev_ptr(ws, "ws"),
        ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def repro_distill_ws_bytes(n: int, V: int) -> int:
    return int(lib().repro_distill_ws_bytes(int(n), int(V)))


def _distill_common(logits, t_idx, labels, tau, w_kd, w_ce, w_z):
    n, V, ld = _rows2d(logits, "logits")
    if t_idx.dim() < 2 or t_idx.numel() != n * t_idx.shape[-1]:
        raise ValueError("t_idx must be [..., K] with a row per row of logits")
    if labels is not None and labels.numel() != n:
        raise ValueError("labels must have an entry per row of logits")
    hp = DistillHparams(tau, w_kd, w_ce, w_z)
    return n, V, ld, int(t_idx.shape[-1]), _index_bytes("t_idx and labels", t_idx, labels), hp


def repro_distill_fwd(logits: torch.Tensor, t_idx: torch.Tensor, t_logits: torch.Tensor, loss: torch.Tensor,
                      stats: torch.Tensor, labels=None, tau: float = 1.0, w_kd: float = 1.0,
                      w_ce: float = 0.0, w_z: float = 0.0, logprobs: bool = False, ws=None,
                      stream=None) -> None:
    """loss [n] <- w_kd tau^2 KL(teacher, student) over the teacher's K entries a
    row (t_idx [n, K], negative: empty; t_logits [n, K], or its log-probabilities
    with logprobs) + w_ce cross entropy of labels (negative: none) + w_z lse^2.
    Without a teacher (w_kd 0) t_idx and t_logits may have K = 0 columns.
    logits [n, V] float32 or bfloat16, rows at any stride; tau from 1e-4 to 1e4; stats
    [n, REPRO_DISTILL_STATS + K] float32 is the backward's input."""
    n, V, ld, K, ib, hp = _distill_common(logits, t_idx, labels, tau, w_kd, w_ce, w_z)
    if t_logits.shape != t_idx.shape:
        raise ValueError("t_logits must have t_idx's shape")
    if loss.numel() != n or stats.numel() != n * (REPRO_DISTILL_STATS + K):
        raise ValueError("loss must be [n], stats [n, REPRO_DISTILL_STATS + K]")
    if ws is None:
        ws = _workspace(repro_distill_ws_bytes(n, V), logits.device, stream)
    _check("repro_distill_fwd", lib().repro_distill_fwd(
        _dev_ptr(logits, "logits", False), _float_type(logits, "logits"), ld, _dev_ptr(t_idx, "t_idx"),
        _dev_ptr(t_logits, "t_logits"), _float_type(t_logits, "t_logits"), _dev_ptr(labels, "labels"), ib,
        n, V, K, ctypes.byref(hp), REPRO_DISTILL_LOGPROBS if logprobs else 0,
        _ptr(loss, torch.float32, "loss"), _ptr(stats, torch.float32, "stats"), _dev_ptr(ws, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def repro_distill_bwd(logits: torch.Tensor, t_idx: torch.Tensor, stats: torch.Tensor, g: torch.Tensor,
                      dlogits: torch.Tensor, labels=None, tau: float = 1.0, w_kd: float = 1.0,
                      w_ce: float = 0.0, w_z: float = 0.0, logprobs: bool = False, stream=None) -> None:
    """dlogits [n, V] (logits' type; may be logits itself) <- the gradient of the
    rows' losses for upstream gradients g ([n], or [1] for every row), from the
    forward's arguments and stats (logprobs is accepted so that one set of
    keywords serves both calls; stats holds its effect)."""
    n, V, ld, K, ib, hp = _distill_common(logits, t_idx, labels, tau, w_kd, w_ce, w_z)
    nd, Vd, dld = _rows2d(dlogits, "dlogits")
    if (nd, Vd) != (n, V) or dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must have the shape and type of logits")
    if stats.numel() != n * (REPRO_DISTILL_STATS + K):
        raise ValueError("stats must be [n, REPRO_DISTILL_STATS + K]")
    _check("repro_distill_bwd", lib().repro_distill_bwd(
        _dev_ptr(logits, "logits", False), _float_type(logits, "logits"), ld, _dev_ptr(t_idx, "t_idx"),
        _dev_ptr(labels, "labels"), ib, n, V, K, ctypes.byref(hp), _ptr(stats, torch.float32, "stats"),
        _ptr(g, torch.float32, "g"), g.numel(), _dev_ptr(dlogits, "dlogits", False), dld, _stream(stream)))


def repro_selftest(device=None, stream=None) -> int:
    """Runs the tensor-core forward's exactness self-test; returns the status
    (REPRO_OK when every output matches the exact CUDA-core path)."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    ws = _workspace(int(lib().repro_selftest_ws_bytes()), dev, stream)
    return int(lib().repro_selftest(_ptr(ws, None, "ws"), ws.numel(), _stream(stream)))


REPRO_HASH_LEAF_BYTES = 4096


def _hash_tables(buffers):
    nb = len(buffers)
    ptrs = (_vp * max(nb, 1))(*[_ptr(b, None, "buffer") if b.numel() else None for b in buffers])
    sizes = (_i64 * max(nb, 1))(*[b.numel() * b.element_size() for b in buffers])
    return ptrs, sizes, nb


def repro_state_hash_ws_bytes(buffers) -> int:
    """Workspace for hashing these tensors (their bytes, in order)."""
    _, sizes, nb = _hash_tables(buffers)
    return int(lib().repro_state_hash_ws_bytes(sizes, nb))


def repro_state_hash(buffers, digest: torch.Tensor, ws=None, stream=None) -> None:
    """digest (32 uint8, device) <- Merkle Tree Hash of the tensors' bytes."""
    for b in buffers:
        if not b.is_contiguous():
            raise ValueError("state buffers must be contiguous")
    ptrs, sizes, nb = _hash_tables(buffers)
    if digest.numel() != 32 or digest.dtype != torch.uint8:
        raise ValueError("digest must be 32 uint8")
    if ws is None:
        ws = _workspace(int(lib().repro_state_hash_ws_bytes(sizes, nb)), digest.device, stream)
    _check("repro_state_hash", lib().repro_state_hash(
        ptrs, sizes, nb, _ptr(digest, torch.uint8, "digest"), _ptr(ws, None, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def repro_sumsq_ws_bytes(n: int) -> int:
    return int(lib().repro_sumsq_ws_bytes(int(n)))


def repro_sumsq(g: torch.Tensor, out: torch.Tensor, ws=None, stream=None) -> None:
    """out[0] <- canonical sum of g_i (x) g_i."""
    n = g.numel()
    if ws is None:
        ws = _workspace(repro_sumsq_ws_bytes(n), g.device, stream)
    _check("repro_sumsq", lib().repro_sumsq(
        _ptr(g, torch.float32, "g"), n, _ptr(out, torch.float32, "out"), _ptr(ws, None, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def repro_adamw_step(p: torch.Tensor, m: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     sumsq: torch.Tensor, t: int, lr: float = 4.5e-4, beta1: float = 0.9,
                     beta2: float = 0.95, eps: float = 1e-8, weight_decay: float = 0.1,
                     max_norm: float = 1.0, stream=None) -> None:
    """Clip to the global norm sqrt(sumsq) and apply AdamW step t in place."""
    n = p.numel()
    if not (m.numel() == v.numel() == g.numel() == n):
        raise ValueError("p, m, v and g must have the same number of elements")
    hp = AdamWHparams(lr, beta1, beta2, eps, weight_decay, max_norm)
    _check("repro_adamw_step", lib().repro_adamw_step(
        _ptr(p, torch.float32, "p"), _ptr(m, torch.float32, "m"), _ptr(v, torch.float32, "v"),
        _ptr(g, torch.float32, "g"), n, _ptr(sumsq, torch.float32, "sumsq"), ctypes.byref(hp),
        int(t), _stream(stream)))


def repro_status_str(status: int) -> str:
    return lib().repro_status_str(int(status)).decode()


def repro_version() -> int:
    return int(lib().repro_version())


def repro_launch_count() -> int:
    return int(lib().repro_launch_count())


def repro_device_check(stream=None) -> int:
    return int(lib().repro_device_check(_stream(stream)))


def repro_wait_probe(arrive: int, stream=None) -> int:
    """Enqueue the bounded-wait probe; arrive=0 makes the wait run out."""
    return int(lib().repro_wait_probe(int(arrive), _stream(stream)))


def repro_set_debug(flags: int) -> None:
    """Debug checks (REPRO_DEBUG_CHECK_FINITE: scan every float input; a NaN or
    an infinity makes the next repro_device_check return REPRO_ERR_NONFINITE)."""
    _check("repro_set_debug", lib().repro_set_debug(int(flags)))


def repro_set_launch_cfg(bwd_segment_log2: int = -1, reduce_block_log2: int = -1,
                         fwd_path: int = -1, elementwise_blocks: int = -1, bwd_kernel: int = -1,
                         fwd_selftest: int = -1, reset: bool = False):
    if reset:
        _check("repro_set_launch_cfg", lib().repro_set_launch_cfg(None))
        return
    cfg = LaunchCfg(bwd_segment_log2, reduce_block_log2, fwd_path, elementwise_blocks, bwd_kernel,
                    fwd_selftest)
    _check("repro_set_launch_cfg", lib().repro_set_launch_cfg(ctypes.byref(cfg)))
