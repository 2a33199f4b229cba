"""Python binding of libmoe.so, the MI355X MoE FFN layer library.

Argument marshalling only: every function below packs its arguments and calls
the C entry point of the same name (declared in include/moe.h); all of the
layer's work runs in the library's HIP kernels.  PyTorch supplies device
memory and the stream.  Tensors are passed by ``data_ptr()``; bf16 tensors may
be torch.bfloat16 or raw uint16/int16 bit patterns, MXFP4 tensors uint8.

If the library is not built the import still succeeds, but every call raises
``MoeLibraryMissing`` (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(6)
MOE_WFMT_BF16, MOE_WFMT_MXFP4, MOE_WFMT_MXFP4_PACKED = 0, 1, 2
MOE_PACK_GATE_UP, MOE_PACK_DOWN = 0, 1
MOE_DT_BF16, MOE_DT_F16, MOE_DT_F32 = 0, 1, 2
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1
MOE_NORM_NONE, MOE_NORM_RMS, MOE_NORM_LAYER = 0, 1, 2
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
MOE_PATH_AUTO, MOE_PATH_SKINNY, MOE_PATH_TILED, MOE_PATH_TILED_DEQUANT, MOE_PATH_TILED_MX = 0, 1, 2, 3, 4

EXPORTED = ("moe_workspace_size", "moe_route", "moe_permute", "moe_gate_up", "moe_down", "moe_grouped_ffn",
            "moe_combine", "moe_forward", "moe_forward_noalloc", "moe_backward_workspace_size", "moe_backward",
            "moe_mxfp4_quantize", "moe_mxfp4_fakequant", "moe_mxfp4_pack", "moe_mx_split", "moe_strerror",
            "moe_last_error", "moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_workspace_size",
            "moe_grouped_mm_wgrad", "moe_w4_matvec", "moe_norm_in", "moe_norm_out", "moe_norm_workspace_size",
            "moe_norm_in_backward", "moe_norm_out_backward")


class MoeLibraryMissing(RuntimeError):
    pass


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn} failed: {text} (code {code})")
        self.code = code


class moe_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("wfmt", ctypes.c_int32), ("path", ctypes.c_int32)]


class moe_expert_weights(ctypes.Structure):
    _fields_ = [("gate_up", ctypes.c_void_p), ("gate_up_scale", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("down_scale", ctypes.c_void_p)]


class moe_gmm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "E", "T", "k", "dtype", "out_dtype", "accumulate",
                                              "reserved")] + [("lda", ctypes.c_int64), ("ldc", ctypes.c_int64)]


class moe_w4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "E", "T", "k", "group", "dtype", "out_dtype", "act")]


class moe_norm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "dtype", "wdtype", "kind", "gate")] + \
               [(n, ctypes.c_float) for n in ("eps", "res_scale", "dropout_p")]


_lib = None


def library(path: str | None = None):
    """Load libmoe.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    # torch ships its own libamdhip64 (same soname): load it first so the
    # process holds a single HIP runtime and torch's streams are valid here.
    import torch  # noqa: F401
    if not os.path.exists(p):
        raise MoeLibraryMissing(f"{p} is not built; run `python -m mixture_experts_ffn_05_amd.build`")
    lib = ctypes.CDLL(p)
    V, I32, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    D, W = ctypes.POINTER(moe_dims), ctypes.POINTER(moe_expert_weights)
    G, N = ctypes.POINTER(moe_gmm), ctypes.POINTER(moe_norm)
    sig = {
        "moe_workspace_size": [D, ctypes.POINTER(SZ)],
        "moe_route": [D, V, V, V, V, V, SZ, V],
        "moe_permute": [D, V, V, V, V, V, SZ, V],
        "moe_gate_up": [D, V, V, V, W, V, V, SZ, V],
        "moe_down": [D, V, V, W, V, V, SZ, V],
        "moe_grouped_ffn": [D, V, V, V, W, V, V, SZ, V],
        "moe_combine": [D, V, V, V, V, V],
        "moe_forward": [D, V, V, W, V, V, V, V, SZ, V],
        "moe_forward_noalloc": [D, V, V, W, V, V, V, V],
        "moe_backward_workspace_size": [D, ctypes.POINTER(SZ)],
        "moe_backward": [D, V, V, W, V, V, V, V, V, V, SZ, V],
        "moe_mxfp4_quantize": [ctypes.c_int64, ctypes.c_int32, V, V, V, V],
        "moe_mxfp4_fakequant": [ctypes.c_int64, ctypes.c_int32, V, V, V],
        "moe_mxfp4_pack": [D, ctypes.c_int32, V, V, V, V, V],
        "moe_mx_split": [ctypes.c_int64, ctypes.c_int32, V, V, V, V],
        "moe_grouped_mm": [G, V, V, V, V, V, V, V],
        "moe_grouped_mm_dgrad": [G, V, V, V, V, V],
        "moe_grouped_mm_workspace_size": [G, ctypes.POINTER(SZ)],
        "moe_grouped_mm_wgrad": [G, V, V, V, V, V, V, V, SZ, V],
        "moe_w4_matvec": [ctypes.POINTER(moe_w4), V, V, V, V, V, V, V, V, V],
        "moe_norm_in": [N, V, V, V, V, V],
        "moe_norm_out": [N, V, V, V, V, V, V, V, V],
        "moe_norm_workspace_size": [N, ctypes.POINTER(SZ)],
        "moe_norm_in_backward": [N, V, V, V, V, V, V, V, V, SZ, V],
        "moe_norm_out_backward": [N, V, V, V, V, V, V, V, V, V, V, V, SZ, V],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = I32
    lib.moe_strerror.argtypes = [I32]
    lib.moe_strerror.restype = ctypes.c_char_p
    lib.moe_last_error.argtypes = []
    lib.moe_last_error.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        lib = library()
        text = lib.moe_strerror(rc).decode()
        if rc == MOE_ERR_HIP:
            text += ": " + lib.moe_last_error().decode()
        raise MoeError(fn, rc, text)


def dims(T: int, H: int, E: int, k: int, I: int, wfmt: int = MOE_WFMT_BF16, path: int = MOE_PATH_AUTO) -> moe_dims:
    return moe_dims(T, H, E, k, I, wfmt, path)


def expert_weights(gate_up, down, gate_up_scale=None, down_scale=None) -> moe_expert_weights:
    return moe_expert_weights(_ptr(gate_up), _ptr(gate_up_scale), _ptr(down), _ptr(down_scale))


def strerror(code: int) -> str:
    return library().moe_strerror(code).decode()


def moe_workspace_size(d: moe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_workspace_size", library().moe_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def moe_route(d, x, w_router, topk_idx, topk_w, ws, ws_bytes, stream=None):
    _check("moe_route", library().moe_route(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(topk_idx), _ptr(topk_w),
                                           _ptr(ws), ws_bytes, _stream(stream)))


def moe_permute(d, topk_idx, expert_offsets, sorted_pairs, pair_rank, ws, ws_bytes, stream=None):
    _check("moe_permute", library().moe_permute(ctypes.byref(d), _ptr(topk_idx), _ptr(expert_offsets),
                                               _ptr(sorted_pairs), _ptr(pair_rank), _ptr(ws), ws_bytes,
                                               _stream(stream)))


def moe_gate_up(d, x, expert_offsets, sorted_pairs, weights: moe_expert_weights, h, ws, ws_bytes, stream=None):
    _check("moe_gate_up", library().moe_gate_up(ctypes.byref(d), _ptr(x), _ptr(expert_offsets), _ptr(sorted_pairs),
                                               ctypes.byref(weights), _ptr(h), _ptr(ws), ws_bytes, _stream(stream)))


def moe_down(d, h, expert_offsets, weights: moe_expert_weights, y_sorted, ws, ws_bytes, stream=None):
    _check("moe_down", library().moe_down(ctypes.byref(d), _ptr(h), _ptr(expert_offsets), ctypes.byref(weights),
                                         _ptr(y_sorted), _ptr(ws), ws_bytes, _stream(stream)))


def moe_grouped_ffn(d, x, expert_offsets, sorted_pairs, weights: moe_expert_weights, y_sorted, ws, ws_bytes,
                    stream=None):
    _check("moe_grouped_ffn", library().moe_grouped_ffn(ctypes.byref(d), _ptr(x), _ptr(expert_offsets),
                                                       _ptr(sorted_pairs), ctypes.byref(weights), _ptr(y_sorted),
                                                       _ptr(ws), ws_bytes, _stream(stream)))


def moe_combine(d, y_sorted, pair_rank, topk_w, y, stream=None):
    _check("moe_combine", library().moe_combine(ctypes.byref(d), _ptr(y_sorted), _ptr(pair_rank), _ptr(topk_w),
                                               _ptr(y), _stream(stream)))


def moe_forward(d, x, w_router, weights: moe_expert_weights, y, topk_idx_out, topk_w_out, ws, ws_bytes, stream=None):
    _check("moe_forward", library().moe_forward(ctypes.byref(d), _ptr(x), _ptr(w_router), ctypes.byref(weights),
                                               _ptr(y), _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(ws), ws_bytes,
                                               _stream(stream)))


def moe_forward_noalloc(d, x, w_router, weights: moe_expert_weights, y, topk_idx_out, topk_w_out, stream=None):
    _check("moe_forward_noalloc", library().moe_forward_noalloc(ctypes.byref(d), _ptr(x), _ptr(w_router),
                                                               ctypes.byref(weights), _ptr(y), _ptr(topk_idx_out),
                                                               _ptr(topk_w_out), _stream(stream)))


MOE_NOALLOC_SCRATCH_BYTES = 32 << 20


def moe_backward_workspace_size(d: moe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_backward_workspace_size", library().moe_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def moe_backward(d, x, w_router, weights: moe_expert_weights, dy, dx, dw_router, dgate_up, ddown, ws, ws_bytes,
                 stream=None):
    _check("moe_backward", library().moe_backward(ctypes.byref(d), _ptr(x), _ptr(w_router), ctypes.byref(weights),
                                                 _ptr(dy), _ptr(dx), _ptr(dw_router), _ptr(dgate_up), _ptr(ddown),
                                                 _ptr(ws), ws_bytes, _stream(stream)))


def moe_mxfp4_quantize(rows: int, cols: int, w, packed, scales, stream=None):
    _check("moe_mxfp4_quantize", library().moe_mxfp4_quantize(rows, cols, _ptr(w), _ptr(packed), _ptr(scales),
                                                             _stream(stream)))


def moe_mxfp4_fakequant(rows: int, cols: int, w, out, stream=None):
    _check("moe_mxfp4_fakequant", library().moe_mxfp4_fakequant(rows, cols, _ptr(w), _ptr(out), _stream(stream)))


def moe_mxfp4_pack(d: moe_dims, which: int, w, scales, w_packed, scales_packed, stream=None):
    _check("moe_mxfp4_pack", library().moe_mxfp4_pack(ctypes.byref(d), which, _ptr(w), _ptr(scales), _ptr(w_packed),
                                                     _ptr(scales_packed), _stream(stream)))


def moe_mx_split(rows: int, cols: int, x, codes, scales, stream=None):
    _check("moe_mx_split", library().moe_mx_split(rows, cols, _ptr(x), _ptr(codes), _ptr(scales), _stream(stream)))


# --------------------------------------------------------------------- stand-alone operators


class _DTypes:
    """torch dtype -> MOE_DT_*."""

    def __getitem__(self, dtype):
        import torch
        return {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16, torch.float32: MOE_DT_F32}[dtype]


DTYPE = _DTypes()


def _stream_for(stream, *tensors):
    """The stream of a call on these tensors: the given one, or the current one
    of the current device.  Tensors on another device are refused: they would be
    reached over a link, if at all, and without ordering."""
    import torch
    dev = None
    for t in tensors:
        if t is None or type(t) is int:
            continue
        at = t.get_device()  # -1: host memory
        if dev is None and at >= 0:
            dev = torch.cuda.current_device()
        if at < 0 or at != dev:
            raise ValueError(f"tensor on {t.device}, not on the current device" + ("" if dev is None else f" (cuda:{dev})"))
    if stream is None:
        # the raw handle: torch.cuda.current_stream() builds an object around it,
        # which costs more than the call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    return _stream(stream)


def gmm(M: int, N: int, K: int, E: int, T: int = 0, k: int = 1, dtype: int = MOE_DT_BF16, out_dtype: int | None = None,
        accumulate: bool = False, lda: int = 0, ldc: int = 0) -> moe_gmm:
    return moe_gmm(M, N, K, E, T, k, dtype, dtype if out_dtype is None else out_dtype, int(accumulate), 0, lda, ldc)


def w4(M: int, N: int, K: int, E: int, T: int = 0, k: int = 1, group: int = 128, dtype: int = MOE_DT_BF16,
       out_dtype: int | None = None, act: int = MOE_ACT_NONE) -> moe_w4:
    return moe_w4(M, N, K, E, T, k, group, dtype, dtype if out_dtype is None else out_dtype, act)


def norm(T: int, H: int, dtype: int = MOE_DT_BF16, wdtype: int | None = None, kind: int = MOE_NORM_RMS,
         eps: float = 1e-5, gate: int = MOE_GATE_NONE, res_scale: float = 1.0, dropout_p: float = 0.0) -> moe_norm:
    return moe_norm(T, H, dtype, dtype if wdtype is None else wdtype, kind, gate, eps, res_scale, dropout_p)


def moe_grouped_mm(g, a, expert_offsets, sorted_pairs, b, bias, c, stream=None):
    st = _stream_for(stream, a, expert_offsets, sorted_pairs, b, bias, c)
    _check("moe_grouped_mm", library().moe_grouped_mm(ctypes.byref(g), _ptr(a), _ptr(expert_offsets),
                                                     _ptr(sorted_pairs), _ptr(b), _ptr(bias), _ptr(c),
                                                     st))


def moe_grouped_mm_dgrad(g, dc, expert_offsets, b, da, stream=None):
    st = _stream_for(stream, dc, expert_offsets, b, da)
    _check("moe_grouped_mm_dgrad", library().moe_grouped_mm_dgrad(ctypes.byref(g), _ptr(dc), _ptr(expert_offsets),
                                                                 _ptr(b), _ptr(da), st))


def moe_grouped_mm_workspace_size(g) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_grouped_mm_workspace_size", library().moe_grouped_mm_workspace_size(ctypes.byref(g), ctypes.byref(n)))
    return n.value


def moe_grouped_mm_wgrad(g, a, expert_offsets, sorted_pairs, dc, db, dbias, ws, ws_bytes, stream=None):
    st = _stream_for(stream, a, expert_offsets, sorted_pairs, dc, db, dbias, ws)
    _check("moe_grouped_mm_wgrad", library().moe_grouped_mm_wgrad(ctypes.byref(g), _ptr(a), _ptr(expert_offsets),
                                                                 _ptr(sorted_pairs), _ptr(dc), _ptr(db), _ptr(dbias),
                                                                 _ptr(ws), ws_bytes, st))


def moe_w4_matvec(d, x, expert_offsets, sorted_pairs, codes, scales, zeros, bias, y, stream=None):
    st = _stream_for(stream, x, expert_offsets, sorted_pairs, codes, scales, zeros, bias, y)
    _check("moe_w4_matvec", library().moe_w4_matvec(ctypes.byref(d), _ptr(x), _ptr(expert_offsets), _ptr(sorted_pairs),
                                                   _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(bias), _ptr(y),
                                                   st))


def moe_norm_in(d, x, weight, bias, y, stream=None):
    st = _stream_for(stream, x, weight, bias, y)
    _check("moe_norm_in", library().moe_norm_in(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y),
                                               st))


def moe_norm_out(d, f, residual, weight, bias, gate, rng, out, stream=None):
    st = _stream_for(stream, f, residual, weight, bias, gate, rng, out)
    _check("moe_norm_out", library().moe_norm_out(ctypes.byref(d), _ptr(f), _ptr(residual), _ptr(weight), _ptr(bias),
                                                 _ptr(gate), _ptr(rng), _ptr(out), st))


def moe_norm_workspace_size(d) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_norm_workspace_size", library().moe_norm_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def moe_norm_in_backward(d, x, weight, dy, dres, dx, dweight, dbias, ws, ws_bytes, stream=None):
    st = _stream_for(stream, x, weight, dy, dres, dx, dweight, dbias, ws)
    _check("moe_norm_in_backward", library().moe_norm_in_backward(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(dy),
                                                                 _ptr(dres), _ptr(dx), _ptr(dweight), _ptr(dbias),
                                                                 _ptr(ws), ws_bytes, st))


def moe_norm_out_backward(d, f, weight, bias, gate, rng, dout, df, dweight, dbias, dgate, ws, ws_bytes, stream=None):
    st = _stream_for(stream, f, weight, bias, gate, rng, dout, df, dweight, dbias, dgate, ws)
    _check("moe_norm_out_backward", library().moe_norm_out_backward(ctypes.byref(d), _ptr(f), _ptr(weight), _ptr(bias),
                                                                   _ptr(gate), _ptr(rng), _ptr(dout), _ptr(df),
                                                                   _ptr(dweight), _ptr(dbias), _ptr(dgate), _ptr(ws),
                                                                   ws_bytes, st))


__all__ = ["library", "dims", "expert_weights", "strerror", "moe_workspace_size", "moe_route", "moe_permute",
           "moe_gate_up", "moe_down", "moe_grouped_ffn", "moe_combine", "moe_forward", "moe_forward_noalloc",
           "MOE_NOALLOC_SCRATCH_BYTES", "moe_backward_workspace_size",
           "moe_backward", "moe_mxfp4_quantize",
           "moe_mxfp4_fakequant", "moe_mxfp4_pack", "moe_mx_split", "moe_dims",
           "moe_expert_weights", "moe_gmm", "moe_w4", "moe_norm", "gmm", "w4", "norm", "DTYPE", "moe_grouped_mm",
           "moe_grouped_mm_dgrad", "moe_grouped_mm_workspace_size", "moe_grouped_mm_wgrad", "moe_w4_matvec",
           "moe_norm_in", "moe_norm_out", "moe_norm_workspace_size", "moe_norm_in_backward", "moe_norm_out_backward",
           "MoeError", "MoeLibraryMissing", "EXPORTED", "LIB_PATH"]
